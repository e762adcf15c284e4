"""The rotation's frequencies against 60 digits: the header that the library is
built from, compiled for the host."""
from __future__ import annotations

import subprocess
from fractions import Fraction

import pytest

from tests import ropeexact as X
from w8a8_int8_gemm_amd import build as wb

MAIN = """
#include <cstdio>
#include <cstdlib>
#include "rope.h"
int main(int n, char **v) {
  w8a8_rope_t r{};
  r.axes = 1;
  r.scaling = atoi(v[2]);
  r.theta = atof(v[3]);
  r.factor = atof(v[4]);
  r.original = atof(v[5]);
  r.beta_fast = atof(v[6]);
  r.beta_slow = atof(v[7]);
  const int p = r.pairs[0] = atoi(v[1]);
  double q[W8A8_ROPE_MAX_PAIRS];
  w8a8::rope_quarters(r, p, q);
  for (int i = 0; i < p; ++i) printf("%a\\n", q[i]);
}
"""

KINDS = ["none", "linear", "ntk", "yarn"]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("rope")
    src = at / "rope.cpp"
    src.write_text(MAIN)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off",
                    f"-I{wb.ROOT / 'include'}", f"-I{wb.CSRC}", str(src), "-o",
                    str(at / "rope")], check=True)
    return at / "rope"


CASES = [(p, dict(theta=theta)) for p in (1, 3, 40, 64, 256)
         for theta in (1.0001, 256.0, 10000.0, 1e6, 1e300)] + [
    (p, dict(scaling="linear", factor=factor)) for p in (7, 64)
    for factor in (1.0, 3.7, 64.0)] + [
    (p, dict(scaling="ntk", theta=theta, factor=factor)) for p in (1, 2, 64, 127)
    for theta, factor in ((1e4, 8.0), (5e5, 1000.0), (1e10, 1e120))] + [
    (p, dict(scaling="yarn", theta=theta, factor=factor, original=original))
    for p in (16, 64, 256)
    for theta, factor, original in ((1e4, 4.0, 4096.0), (1e6, 40.0, 32768.0),
                                    (150.0, 1e6, 100.0))]


@pytest.mark.parametrize("p,kw", CASES)
def test_frequencies(program, p, kw):
    full = dict(scaling="none", theta=1e4, factor=1.0, original=0.0,
                beta_fast=32.0, beta_slow=1.0)
    full.update(kw)
    args = [p, KINDS.index(full["scaling"])] + [repr(full[n]) for n in (
        "theta", "factor", "original", "beta_fast", "beta_slow")]
    got = subprocess.run([str(program), *map(str, args)], check=True,
                         capture_output=True, text=True).stdout.split()
    want = X.frequencies(p, **kw)
    assert len(got) == p
    # The header's bounds: 1.25 * 2^-52, and 1.75 * 2^-53 for small theta, factor.
    small = full["theta"] < 2**20 and full["factor"] < 2**20
    most = Fraction(7 if small else 10, 2**55)
    for g, w in zip(got, want):
        with X.localcontext(X.DIGITS):
            exact = Fraction(w * 2 / X.PI)
        assert abs(Fraction(float.fromhex(g)) - exact) <= most * exact

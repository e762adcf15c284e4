"""NaN, Inf and rows beyond binary32's squares in the block norms: they reach
every output of their row, the codes' scale among them, and no other row."""
from __future__ import annotations

import pytest

from tests.test_gpu_norm import call, inputs, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

NAN = float("nan")

# one wave a row, several waves, two rows a work group with an odd last one
SHAPES = [(9, 64), (21, 1000), (11, 5376), (1201, 5376)]


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def check_rows(before, after, bad, quantize, residual):
    """Rows `bad` have a NaN in each output (codes: the scale); the others are
    what they were."""
    assert bad.any() and not bad.all()
    names = (["r"] if residual else []) + (["q", "s"] if quantize else ["y"])
    for name, a, b in zip(names, before, after):
        assert same_bits(a[~bad].contiguous(), b[~bad].contiguous()), name
        if name == "s":
            assert b[bad].isnan().all(), name
            assert a.isfinite().all()
        elif name != "q":
            assert b[bad].isnan().any(1).all(), name


def listed(t):
    return [c.clone() for c in (t if isinstance(t, (tuple, list)) else [t])]


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_nan_in_a_row(M, H, norm):
    """A NaN of x or of the branch, at the ends and inside."""
    for quantize in (False, True):
        for where in ("x", "branch"):
            for post in (("none", "rms") if where == "branch" else ("rms",)):
                say(f"nan row {M}x{H} {norm} q={quantize} {where} {post}")
                residual = where == "branch"
                x, kw = inputs(M, H, 3, post=post, norm=norm, mods="index",
                               branch=residual)
                before = listed(call(x, kw, quantize))
                t = kw["branch"] if residual else x
                rows = [0, M // 2, M - 1]
                for i, m in enumerate(rows):
                    t[m, (0, H // 2 + 1, H - 1)[i]] = NAN
                bad = torch.zeros(M, dtype=torch.bool, device="cuda")
                bad[rows] = True
                check_rows(before, listed(call(x, kw, quantize)), bad,
                           quantize, residual)


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_nan_in_a_modulation_row(M, H, norm):
    """A NaN of one row of scale, shift or gate reaches the tokens of that row;
    padding tokens and those of other rows keep their values."""
    for quantize in (False, True):
        for name in ("scale", "shift", "gate"):
            say(f"nan modulation {M}x{H} {norm} q={quantize} {name}")
            x, kw = inputs(M, H, 4, post="none", norm=norm, mods="index")
            row = (torch.arange(M, device="cuda") % 5).to(torch.int32)
            row[1] = -1
            kw["mod_row"] = row
            before = listed(call(x, kw, quantize))
            kw[name][2, H - 3] = NAN
            after = listed(call(x, kw, quantize))
            if name == "gate":
                check_rows(before, after, row == 2, quantize, True)
            else:
                assert same_bits(before[0], after[0])
                check_rows(before[1:], after[1:], row == 2, quantize, False)


@pytest.mark.parametrize("name,norm", [
    ("weight", "rms"), ("weight", "layer"), ("bias", "layer"),
    ("post_weight", "rms"), ("post_bias", "layer")])
@pytest.mark.parametrize("M,H", SHAPES)
def test_nan_in_a_vector(M, H, name, norm):
    """A NaN of a norm's weight or bias reaches every token but padding."""
    for quantize in (False, True):
        say(f"nan vector {M}x{H} {name} {norm} q={quantize}")
        how = dict(post=norm) if name.startswith("post") else dict(norm=norm)
        x, kw = inputs(M, H, 6, mods="index", **how)
        kw["mod_row"][M // 2] = -1
        before = listed(call(x, kw, quantize))
        kw[name][H // 3] = NAN
        after = listed(call(x, kw, quantize))
        if not name.startswith("post"):
            assert same_bits(before.pop(0), after.pop(0))
        check_rows(before, after, kw["mod_row"] >= 0, quantize,
                   name.startswith("post"))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_squares_beyond_the_range(M, H, kind):
    """Finite values whose squares overflow binary32, behind a norm of the
    branch and of the row itself: the row is NaN, not quietly without them."""
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[0, M - 2]] = True
    for quantize in (False, True):
        say(f"overflow {M}x{H} {kind} q={quantize}")
        x, kw = inputs(M, H, 7, post=kind, norm="none", mods="vector")
        before = listed(call(x, kw, quantize))
        kw["branch"][bad] = kw["branch"][bad] * 2.0 ** 100
        check_rows(before, listed(call(x, kw, quantize)), bad, quantize, True)
        x, kw = inputs(M, H, 8, norm=kind, branch=False, mods="vector")
        before = listed(call(x, kw, quantize))
        x[bad] = x[bad] * 2.0 ** 100
        assert x.isfinite().all()
        check_rows(before, listed(call(x, kw, quantize)), bad, quantize, False)
    # the residual alone
    x, kw = inputs(M, H, 9, post=kind, norm=None, mods="vector")
    before = listed(call(x, kw))
    kw["branch"][bad] = kw["branch"][bad] * 2.0 ** 100
    after = listed(call(x, kw))
    assert same_bits(before[0][~bad], after[0][~bad])
    assert after[0][bad].isnan().all()


@pytest.mark.parametrize("M,H", SHAPES)
def test_bf16_row_with_nan_or_inf(M, H):
    """To BF16: a row with a NaN is NaN behind either norm; one with an Inf has
    no finite value behind them."""
    for kind in ("rms", "layer"):
        x, kw = inputs(M, H, 10, norm=kind, branch=False, mods="none")
        want = call(x, kw)
        x[2, H // 2] = NAN
        x[5, 1] = float("inf")
        got = call(x, kw)
        assert got[2].isnan().all()
        assert not got[5].isfinite().any()
        fine = [m for m in range(M) if m not in (2, 5)]
        assert same_bits(want[fine], got[fine])
        s = call(x, kw, True)[1]
        assert s[[2, 5]].isnan().all() and s[fine].isfinite().all()


@pytest.mark.parametrize("M,H", SHAPES)
def test_inf_to_codes_without_a_norm(M, H):
    """The scale of a row with an Inf is not finite, and spoils no other row."""
    x, kw = inputs(M, H, 11, norm="none", branch=False, mods="none")
    want = listed(call(x, kw, True))
    x[1, H - 1] = -float("inf")
    got = listed(call(x, kw, True))
    fine = [m for m in range(M) if m != 1]
    assert not got[1][1].isfinite()
    for a, b in zip(want, got):
        assert same_bits(a[fine], b[fine])

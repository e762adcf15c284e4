"""No wave signals a barrier with LDS operations of its own under way: behind the
barrier other waves overwrite what it reads, and read what it writes."""
from __future__ import annotations

import subprocess
from pathlib import Path

import pytest

from tests import lds_waits
from w8a8_int8_gemm_amd import build as wb


# Not the GEMM: its ring of four stages frees the stage before the one that the
# reads under way are of.
@pytest.mark.parametrize("src", ["attention.hip", "norm.hip", "w4.hip",
                                 "rowwise.hip"])
def test_lds_is_waited_for_before_every_barrier(src, tmp_path):
    out = tmp_path / (Path(src).stem + ".s")
    cmd = [wb.HIPCC, *[f for f in wb.FLAGS if f not in ("-shared", "-fPIC")],
           "--cuda-device-only", "-S", "-o", str(out), str(wb.CSRC / src)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    at = lds_waits.barriers(out.read_text())
    assert sum(map(len, at.values())) > 0
    assert {k: v for k, v in at.items() if any(v)} == {}


KERNEL = """
k:
\tds_read_b128 v[0:3], v4
{before}
.LBB0_1:
{inside}
\ts_barrier
\ts_cbranch_scc1 .LBB0_1
\ts_endpgm
.Lfunc_end0:
\t.amdhsa_kernel k
"""


@pytest.mark.parametrize("before,inside,want", [
    ("", "", 1),
    ("\ts_waitcnt lgkmcnt(0)", "", 0),
    ("\ts_waitcnt vmcnt(0)", "", 1),
    ("\ts_waitcnt vmcnt(0) lgkmcnt(0)", "", 0),
    # one of two is still under way; an exchange does not begin a wait
    ("\tds_read_b32 v5, v6\n\ts_waitcnt lgkmcnt(1)", "", 1),
    ("\ts_waitcnt lgkmcnt(0)", "\tds_bpermute_b32 v5, v6, v7", 0),
    # the loop goes round without a wait: as many as are counted
    ("\ts_waitcnt lgkmcnt(0)", "\tds_write_b32 v5, v6", 16),
    ("", "\tds_read_b64_tr_b16 v[6:7], v8", 16),
    # waited for on one of two paths
    ("\ts_cbranch_vccz .LBB0_1\n\ts_waitcnt lgkmcnt(0)", "", 1),
])
def test_what_counts_as_waited_for(before, inside, want):
    got = lds_waits.barriers(KERNEL.format(before=before, inside=inside))
    assert got == {"k": [want]}

"""The residual alone at every number of chunks and rows that a work group
takes, and rows whose squares are next to nothing beside the least eps."""
from __future__ import annotations

import pytest

from tests.test_gpu_norm import (WIDTHS, call, inputs, rand, gen, run_case, say,
                                 verify)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("H", WIDTHS)
def test_residual_alone_widths(H):
    say(f"residual alone H={H}")
    run_case(7, H, H, False, post="layer", norm=None, mods="token")
    run_case(7, H, H + 1, False, post="rms", norm=None, mods="index")
    run_case(7, H, H + 2, False, post="none", norm=None, mods="none")


@pytest.mark.parametrize("H,M", [
    (5376, 600), (7168, 500), (12296, 401), (16384, 301), (8, 750001),
    (512, 12001), (1000, 6001), (1536, 4001), (1544, 4001), (3064, 2001),
    (5376, 1201), (12288, 601), (24576, 301), (24584, 301), (32768, 201)])
def test_residual_alone_many_values(H, M):
    """From two chunks a thread on, and past the size where work groups take
    two rows; odd row counts, runs of equal modulation rows, padding."""
    say(f"residual alone many H={H} M={M}")
    for post in ("rms", "layer", "none"):
        for mods in ("index", "token", "broadcast"):
            x, kw = inputs(M, H, H + M, post=post, norm=None, mods=mods)
            if mods == "index":
                row = (torch.arange(M, device="cuda") // 7 % 5).to(torch.int32)
                row[M // 2::5] = -1
                kw["mod_row"] = row
            verify(x, kw, False, call(x, kw))


def test_residual_alone_in_place():
    for M, H in ((33, 1000), (1201, 5376)):
        x, kw = inputs(M, H, 3, post="rms", norm=None, mods="index",
                       padded=True)
        want = call(x, kw).clone()
        got = call(x, kw, out=x)
        assert got.data_ptr() == x.data_ptr()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [8, 520, 5376])
def test_rows_as_small_as_the_least_eps(H, kind):
    """Mean squares from 2^-130 to 2^-120 beside an eps of 2^-126."""
    x = (rand(gen(1), 23, H).float()
         * 2.0 ** (-65 + 0.25 * torch.arange(23, device="cuda"))[:, None]
         ).to(torch.bfloat16)
    for branch in (False, True):
        kw = {"norm_kind": kind, "eps": 2.0 ** -126}
        if branch:
            kw = {"branch": x, "post_norm": kind, "post_eps": 2.0 ** -126}
        say(f"least eps H={H} {kind} branch={branch}")
        verify(torch.zeros_like(x) if branch else x, kw, False,
               call(torch.zeros_like(x) if branch else x, kw))

"""Attention whose scores are as large as binary32 holds: one key, or several of
the same score, take all of a row's weight."""
from __future__ import annotations

import pytest

from tests import headref as R
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16

# (queries, keys, heads, width): tiles of 32, 64, 128 (few and many), 256 rows,
# whole and in parts.
SHAPES = [(1, 700, 2, 64), (1, 9000, 2, 64), (40, 700, 2, 128),
          (300, 700, 2, 64), (300, 3000, 3, 32), (300, 700, 64, 32),
          (300, 500, 260, 16), (300, 2500, 64, 40), (600, 2500, 80, 16)]


def scores(Lq, Lk, H, D, power, seed):
    """q, k whose scores are whole numbers below 2^8 times 2^power, exactly, of
    either sign and many of them equal, and v; the whole numbers [Lk, H]."""
    g = torch.Generator("cuda").manual_seed(seed)
    j = torch.randint(-120, 121, (Lk, H), generator=g, device="cuda")
    q = torch.zeros(Lq, H, D, device="cuda")
    k = torch.zeros(Lk, H, D, device="cuda")
    up = power // 2
    q[..., 0] = 2.0 ** up
    q[1::2, :, 0] *= -1  # every other row: the smallest number wins
    k[..., 0] = j * 2.0 ** (power - up)
    v = torch.randn(Lk, H, D, generator=g, device="cuda")
    return q.to(BF), k.to(BF), v.to(BF), j


@pytest.mark.parametrize("power", [9, 17, 24, 27, 30, 31, 40, 64, 100, 118])
@pytest.mark.parametrize("Lq,Lk,H,D", SHAPES)
def test_all_weight_on_the_largest(Lq, Lk, H, D, power):
    q, k, v, j = scores(Lq, Lk, H, D, power, power)
    got = B.attention(q, k, v, scale=1.0)
    # Scores differ by 2^9 or not at all, so other weights are below 2^-700.
    for rows, best in ((slice(0, None, 2), j.amax(0)),
                       (slice(1, None, 2), j.amin(0))):
        mine = got[rows]
        if not mine.shape[0]:
            continue
        on = (j == best).double()  # [Lk, H]
        n = on.sum(0)
        x = v.double()
        want = (on[..., None] * x).sum(0) / n[:, None]
        # n equal weights: as many roundings of the sums, a few of joins and
        # the division
        bound = (n[:, None] + 16) * R.U * (
            (on[..., None] * x.abs()).sum(0) / n[:, None])
        R.check_bf16(mine, want.expand(mine.shape), bound.expand(mine.shape))


@pytest.mark.parametrize("power", [20, 31, 60, 100])
@pytest.mark.parametrize("Lq,Lk,H,D", [s for s in SHAPES if s[0] > 1])
def test_rows_of_ordinary_scores_beside_them(Lq, Lk, H, D, power):
    """Rows share their keys and their wave with rows of large scores: what the
    others do costs them no more than their own roundings."""
    q, k, v, j = scores(Lq, Lk, H, D, power, power)
    g = torch.Generator("cuda").manual_seed(1)
    near = torch.zeros(Lq, dtype=torch.bool, device="cuda")
    near[::3] = True
    k[..., 1:] = torch.randn(Lk, H, D - 1, generator=g, device="cuda").to(BF)
    q[near] = torch.randn(int(near.sum()), H, D, generator=g,
                          device="cuda").to(BF)
    q[near, :, 0] = 0
    got = B.attention(q, k, v, scale=1.0)
    assert got.isfinite().all()
    heads = [0, H // 2, H - 1]
    one = [t[:, heads] for t in (q[near], k, v)]
    one[1] = one[1].clone()
    one[1][..., 0] = 0  # these rows' scores do not see it
    want, bound, _ = R.attention(*one, R.sequences(one[0].shape[0], Lk, 1), 1.0)
    R.check_bf16(got[near][:, heads], want, bound)


@pytest.mark.parametrize("Lq,Lk,H,D", SHAPES)
def test_maximum_that_rises_through_all_sizes(Lq, Lk, H, D):
    """Scores from -2^100 up to 2^100 in the order of the keys: the last takes
    everything, and in the other order the first."""
    q = torch.zeros(Lq, H, D, device="cuda")
    q[..., 0] = 2.0 ** 50
    step = torch.linspace(-100, 100, Lk, device="cuda").round()
    k = torch.zeros(Lk, H, D, device="cuda")
    k[..., 0] = (step.sign() * 2.0 ** (step.abs() - 50))[:, None]
    k[-1, :, 0] = 2.0 ** 51  # alone at the top
    g = torch.Generator("cuda").manual_seed(2)
    v = torch.randn(Lk, H, D, generator=g, device="cuda").to(BF)
    q, k = q.to(BF), k.to(BF)
    got = B.attention(q, k, v, scale=1.0)
    assert torch.equal(got, v[-1].expand(got.shape))
    k, v = k.flip(0).contiguous(), v.flip(0).contiguous()
    got = B.attention(q, k, v, scale=1.0)
    assert torch.equal(got, v[0].expand(got.shape))

"""The rotary table and the head norms with rotation on the GPU against the same
formulas in 64 bits."""
from __future__ import annotations

import pytest

from tests import headref as R
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rand(g, *shape, std=1.0, mean=0.0):
    return (mean + std * torch.randn(*shape, generator=g, device="cuda")).to(BF)


def angles(g, rows, P):
    a = 6.3 * torch.rand(rows, P, generator=g, device="cuda")
    return torch.stack([a.cos(), a.sin()], 1)


# ---------------------------------------------------------------------------
# table
# ---------------------------------------------------------------------------

def check_table(got, want, bound):
    off = (got.double().cpu() - want).abs()
    assert got.shape == want.shape and (off <= bound).all(), (
        (off / bound).max().item())


@pytest.mark.parametrize("T,pairs,reach,kw", [
    (1, (1,), 5, {}), (1, (64,), 2**20, {}), (7, (3,), 100, {}),
    (1000, (22, 21, 21), 64, {}), (33, (1, 2, 3, 5), 1000, {}),
    (5, (256,), 2**31 - 1, {}), (257, (32,), 131072, dict(theta=5e5)),
    (129, (64,), 32768, dict(scaling="linear", factor=4.0)),
    (129, (64,), 32768, dict(scaling="ntk", factor=8.0)),
    (129, (1, 16), 32768, dict(scaling="ntk", factor=8.0)),
    (129, (64,), 131072, dict(scaling="yarn", factor=32.0, original=4096.0)),
    (40, (20, 7), 131072, dict(scaling="yarn", factor=1.0, original=300.0,
                               beta_fast=8.0, beta_slow=2.0)),
    (40, (4,), 1000, dict(scaling="yarn", factor=2.0, original=3.0)),
    (40, (16,), 1000, dict(amplitude=-0.75)),
    (65537, (3,), 1 << 24, {}),
])
@pytest.mark.parametrize("dtype", [torch.int32, torch.float32])
def test_table(T, pairs, reach, kw, dtype):
    pos = torch.randint(-(reach // 3), reach, (T, len(pairs)),
                        generator=gen(T), device="cuda", dtype=torch.int32)
    if dtype == torch.float32:
        pos = pos.float() + 0.25
    got = B.rope_table(pos, pairs, **kw)
    kw = dict(kw)
    if kw.get("scaling") == "yarn" and kw["factor"] > 1:
        import math
        kw["amplitude"] = 0.1 * math.log(kw["factor"]) + 1
    check_table(got, *R.table(pos, pairs, **kw))


def test_table_one_axis_forms_and_nonfinite_positions():
    pos = torch.tensor([0.0, INF, NAN, -INF, 2.5, 3e38], device="cuda")
    got = B.rope_table(pos, 6)
    again = B.rope_table(pos[:, None].contiguous(), (6,),
                         out=torch.empty_like(got))
    assert torch.equal(got.nan_to_num(9.0), again.nan_to_num(9.0))
    assert got[1:4].isnan().all() and not got[[0, 4]].isnan().any()
    assert (got[0, 0] == 1).all() and (got[0, 1] == 0).all()
    # any angle has a cosine and a sine
    assert ((got[5].double() ** 2).sum(0) - 1).abs().max() < 1e-5


# ---------------------------------------------------------------------------
# head norms with rotation
# ---------------------------------------------------------------------------

def case(M, Hq, Hk, D, norm, P, seed, affine="shared", fused=True, rows=None,
         pad=False):
    g = gen(seed)
    qkv = rand(g, M, (Hq + 2 * Hk) * D + (0 if fused else 8), std=1.5, mean=0.3)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    kw = dict(norm=norm)
    for n, H in (("q", Hq), ("k", Hk)):
        shape = (H, D) if affine == "head" else (D,)
        if affine and norm != "none":
            kw[n + "_weight"] = rand(g, *shape, std=0.2, mean=1.0)
        if affine and norm == "layer":
            kw[n + "_bias"] = rand(g, *shape, std=0.2)
    if P:
        rows = M if rows is None else rows
        kw["table"] = angles(g, rows, P)
        if rows not in (1, M) or pad:
            row = torch.randint(0, rows, (M,), generator=g, device="cuda",
                                dtype=torch.int32)
            if pad:
                row[M // 2:] = torch.tensor(
                    [-1, rows, -2**31, 2**31 - 1], device="cuda",
                    dtype=torch.int32).repeat(M)[:M - M // 2]
            kw["row"] = row
    return q, k, kw


def expected(x, n, kw):
    return R.heads(x, kw["norm"], kw.get(n + "_weight"), kw.get(n + "_bias"),
                   table=kw.get("table"), row=kw.get("row"),
                   interleaved=kw.get("interleaved", False))


def check(q, k, kw, out=None):
    got = B.head_norm_rope(q, k, out=out, **kw)
    R.check_bf16(got[0], *expected(q, "q", kw))
    R.check_bf16(got[1], *expected(k, "k", kw))
    return got


@pytest.mark.parametrize("M,Hq,Hk,D,P", [
    (1, 1, 1, 8, 4), (1, 56, 56, 128, 64), (3, 5, 1, 16, 4), (7, 3, 3, 24, 12),
    (2, 6, 2, 40, 12), (64, 8, 2, 64, 32), (33, 20, 4, 80, 20), (5, 2, 2, 96, 48),
    (9, 4, 4, 104, 20), (300, 42, 42, 128, 32), (3, 2, 1, 136, 68),
    (5, 3, 1, 256, 128), (2, 2, 2, 256, 4), (2, 4096, 1, 8, 4),
    (1200, 56, 56, 128, 64), (4000, 9, 7, 32, 16),
])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_against_64_bits(M, Hq, Hk, D, P, norm, interleaved):
    q, k, kw = case(M, Hq, Hk, D, norm, P, M + D)
    kw["interleaved"] = interleaved
    check(q, k, kw)


@pytest.mark.parametrize("norm,affine", [("rms", "head"), ("layer", "head"),
                                         ("rms", None), ("layer", None)])
@pytest.mark.parametrize("rows,pad", [(1, False), (11, False), (11, True),
                                      (37, True)])
def test_weights_and_rows(norm, affine, rows, pad):
    q, k, kw = case(37, 10, 6, 72, norm, 36, 3, affine, rows=rows, pad=pad,
                    fused=False)
    got = check(q, k, kw)
    if pad:
        assert (got[0][37 // 2:] == 0).all() and (got[1][37 // 2:] == 0).all()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_without_a_table_and_without_k(norm):
    q, k, kw = case(21, 7, 7, 128, norm, 0, 4)
    check(q, k, kw)
    only = {n: kw[n] for n in kw if not n.startswith("k_")}
    R.check_bf16(B.head_norm_rope(q, **only), *expected(q, "q", kw))


def test_rotation_alone_is_the_rotation_without_a_norm():
    q, k, kw = case(50, 6, 6, 64, "none", 16, 5)
    got = B.head_norm_rope(q, k, **kw)
    assert torch.equal(B.rope(q, kw["table"]), got[0])
    # values past the rotated part are copied bit for bit
    assert torch.equal(got[1][..., 32:], k[..., 32:])


def test_in_place_within_the_fused_output():
    q, k, kw = case(45, 12, 4, 128, "rms", 64, 6)
    want = B.head_norm_rope(q, k, **kw)
    base = q._base.clone()
    v = base[:, 16 * 128:].clone()
    q2 = base[:, :12 * 128].unflatten(1, (12, 128))
    k2 = base[:, 12 * 128:16 * 128].unflatten(1, (4, 128))
    got = B.head_norm_rope(q2, k2, out=(q2, k2), **kw)
    assert got[0] is q2 and torch.equal(q2, want[0]) and \
        torch.equal(k2, want[1])
    assert torch.equal(base[:, 16 * 128:], v)


@pytest.mark.parametrize("D,P", [(8, 4), (80, 20), (128, 64)])
def test_nothing_is_written_past_the_outputs(D, P):
    q, k, kw = case(13, 3, 2, D, "rms", P, 7)
    bufs = [torch.full((15, H + 2, D), 7.0, dtype=BF, device="cuda")
            for H in (3, 2)]
    outs = tuple(b[1:14, 1:-1] for b in bufs)
    check(q, k, kw, out=outs)
    for b in bufs:
        b[1:14, 1:-1] = 7.0
        assert (b == 7.0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_nonfinite_values_stay_where_they_are(interleaved):
    q, k, kw = case(9, 4, 4, 128, "none", 20, 8)
    kw["interleaved"] = interleaved
    clean = B.head_norm_rope(q, k, **kw)
    q, k = q.clone(), k.clone()
    q[2, 1, 3], q[4, 0, 100], k[5, 2, 39] = INF, NAN, -INF
    got = B.head_norm_rope(q, k, **kw)
    partner = {3: (2 if interleaved else 23), 100: None,
               39: (38 if interleaved else 19)}
    for a, c, (m, h, d) in ((got[0], clean[0], (2, 1, 3)),
                            (got[0], clean[0], (4, 0, 100)),
                            (got[1], clean[1], (5, 2, 39))):
        assert not a[m, h, d].isfinite()
        a[m, h, d] = c[m, h, d]
        if partner[d] is not None:
            assert not a[m, h, partner[d]].isfinite()
            a[m, h, partner[d]] = c[m, h, partner[d]]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_nonfinite_heads_behind_a_norm(norm):
    q, k, kw = case(9, 4, 4, 128, norm, 64, 9)
    clean = B.head_norm_rope(q, k, **kw)
    q = q.clone()
    q[2, 1, 3], q[4, 0, 100] = INF, NAN
    q[6, 2] = torch.finfo(BF).max  # squares beyond the range
    got = B.head_norm_rope(q, k, **kw)
    for m, h in ((2, 1), (4, 0), (6, 2)):
        assert got[0][m, h].isnan().all()
        got[0][m, h] = clean[0][m, h]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # padding is zero whatever it and the vectors hold
    kw["row"] = torch.full((9,), -1, dtype=torch.int32, device="cuda")
    kw["q_weight"] = torch.full_like(kw["q_weight"], NAN)
    assert (B.head_norm_rope(q, k, **kw)[0] == 0).all()


def test_zero_and_constant_heads():
    x = torch.zeros(2, 3, 64, dtype=BF, device="cuda")
    assert (B.head_norm_rope(x) == 0).all()
    x[:] = 3.0
    assert (B.head_norm_rope(x, norm="layer") == 0).all()


def test_far_rows_of_a_long_stride():
    """Token offsets past 2^32 bytes."""
    M, stride = 70000, 1 << 15
    big = torch.empty(M * stride, dtype=BF, device="cuda")
    x = big.as_strided((M, 1, 64), (stride, 64, 1))
    x.copy_(rand(gen(10), M, 1, 64))
    t = angles(gen(11), M, 32)
    got = B.head_norm_rope(x, table=t, out=x)
    assert got.data_ptr() == big.data_ptr()
    dense = rand(gen(10), M, 1, 64)
    assert torch.equal(got, B.head_norm_rope(dense, table=t))
    R.check_bf16(got[-9:], *R.heads(dense[-9:], "rms", table=t[-9:]))


def test_other_stream_and_graph():
    q, k, kw = case(40, 8, 8, 128, "rms", 64, 12)
    want = B.head_norm_rope(q, k, **kw)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    t = B.rope_table(pos, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = B.head_norm_rope(q, k, stream=s, **kw)
    t2 = B.rope_table(pos, 64, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(t, t2)
    outs = tuple(torch.empty_like(w) for w in want)
    x = q._base
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.rope_table(pos, 64, out=t)
        B.head_norm_rope(q, k, norm="rms", table=t, out=outs)
    for i in range(3):
        x.copy_(rand(gen(20 + i), *x.shape))
        pos.add_(100 * i)
        g.replay()
        torch.cuda.synchronize()
        eager = B.head_norm_rope(q, k, norm="rms", table=B.rope_table(pos, 64))
        assert torch.equal(outs[0], eager[0])
        assert torch.equal(outs[1], eager[1])


def test_binding_refuses():
    q, k, kw = case(6, 4, 2, 64, "rms", 32, 13)
    t = kw["table"]
    bad = [
        dict(norm="l2"), dict(table=t[:3]), dict(table=t[:, :1]),
        dict(table=t.double()), dict(row=torch.zeros(6, device="cuda")),
        dict(q_weight=kw["q_weight"][:32]),
        dict(q_weight=kw["q_weight"].expand(3, 64)),
        dict(q_bias=kw["q_weight"].expand(4, 64).contiguous(), norm="layer"),
        dict(out=(torch.empty_like(q),)), dict(out=(q.clone(), q.clone())),
        dict(table=t.cpu()),
    ]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            B.head_norm_rope(q, k, **{**kw, **b})
    for x in (q.float(), q[:, :, ::2], q[:, ::2], q.transpose(0, 1), q[0], None):
        with pytest.raises((ValueError, TypeError)):
            B.head_norm_rope(x, **dict(norm="rms"))
    with pytest.raises(ValueError):
        B.head_norm_rope(q, k[:5])
    with pytest.raises(ValueError):
        B.head_norm_rope(q, k_weight=kw["k_weight"])
    with pytest.raises(ValueError):
        B.head_norm_rope(q, row=torch.zeros(6, dtype=torch.int32,
                                            device="cuda"))
    with pytest.raises(ValueError):
        B.rope(q, None)
    # refused by the library
    for call in (lambda: B.head_norm_rope(q, k, out=(q, q[:, :2])),
                 lambda: B.head_norm_rope(q[:, :, :12].contiguous()),
                 lambda: B.rope(q, angles(gen(1), 6, 36)),
                 lambda: B.rope(q, angles(gen(1), 6, 6)),
                 lambda: B.head_norm_rope(q, eps=0.0)):
        with pytest.raises(B.W8A8Error):
            call()
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for args in ((pos, 8), (pos, (8, 8, 8)), (pos, (8, 0)), (pos, (200, 100)),
                 (pos.long(), (8, 8)), (pos[:, :1], (8,)), (pos.cpu(), (8, 8))):
        with pytest.raises(ValueError):
            B.rope_table(*args)
    with pytest.raises(ValueError):
        B.rope_table(pos, (8, 8), scaling="log")
    for more in (dict(theta=1.0), dict(scaling="linear", factor=0.5),
                 dict(scaling="yarn", factor=2.0)):
        with pytest.raises(B.W8A8Error):
            B.rope_table(pos, (8, 8), **more)

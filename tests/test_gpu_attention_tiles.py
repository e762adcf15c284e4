"""Every tile of the attention against 64 bits, whole and with its keys in parts:
each width's padding, shared heads, ragged and empty sequences, padding that holds
anything.

`plan` states the library's rule, so that each case says which tile it means; that
a case is split shows in the workspace."""
from __future__ import annotations

import pytest

from tests import headref as R
from tests.test_gpu_attention import check, gen, ints, rand, starts
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")
WIDTHS = [24, 32, 56, 64, 88, 96, 120, 128]
ROWS = dict(few=32, some=64, mid=128, short=128, many=256)


def plan(Tq, Tk, n, packed, Hq, Hk):
    """(tile, parts)"""
    G = Hq // Hk
    tiles = lambda rows: (Tq * G // rows + n if packed else
                          n * -(-(Tq // n * G) // rows)) * Hk
    rows, keys = -(-Tq // n) * G, Tk // n
    large = tiles(256)
    tile = ("few" if rows <= 32 else "some" if rows <= 64 or large < 64 else
            "many" if keys > 2048 else
            "mid" if keys > 1024 or large <= 512 else "short")
    groups, stages = tiles(ROWS[tile]), -(-keys // 128)
    parts = min(1 if groups >= 256 else 256 // groups, stages, 64)
    return tile, parts if stages - -(-stages // max(parts, 1)) >= 4 else 1


# tile, parts, sequences, queries and keys of each, query and key heads
CASES = [("mid", 1, 4, 300, 700, 16, 16), ("mid", 1, 4, 100, 700, 48, 16),
         ("mid", 2, 4, 200, 1200, 16, 16), ("mid", 2, 4, 67, 1200, 48, 16),
         ("many", 1, 4, 600, 2100, 12, 12), ("many", 1, 4, 200, 2100, 36, 12),
         ("many", 3, 4, 600, 2100, 6, 6), ("many", 3, 4, 120, 2100, 30, 6),
         ("short", 1, 4, 300, 150, 130, 65),
         ("some", 1, 4, 60, 300, 3, 3), ("some", 6, 3, 200, 1300, 4, 2),
         ("few", 1, 5, 3, 400, 9, 3), ("few", 8, 4, 1, 1100, 32, 8)]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("tile,parts,n,Lq,Lk,Hq,Hk", CASES)
def test_padded_batch(tile, parts, n, Lq, Lk, Hq, Hk, D):
    assert plan(n * Lq, n * Lk, n, False, Hq, Hk) == (tile, parts)
    need = B.attention_workspace_bytes(n * Lq, n * Lk, Hq, Hk, D, B=n)
    assert need == (parts > 1) * parts * n * Lq * Hq * (4 * D + 8)
    g = gen(Lq + D)
    q = rand(g, n, Lq, Hq, D, std=1.5)
    k, v = rand(g, n, Lk, Hk, D, std=1.5), rand(g, n, Lk, Hk, D)
    lens = [Lk - 1, 0, Lk // 2 + 1, 1, Lk][:n]
    junk = [NAN, INF, -INF, torch.finfo(BF).min]
    for b, m in enumerate(lens):
        k[b, m:], v[b, m:] = junk[b % 4], junk[(b + 1) % 4]
    wide = torch.full((n * Lq + 2, Hq, D), 5.0, dtype=BF, device="cuda")
    out = wide[1:-1].unflatten(0, (n, Lq))
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    assert B.attention(q, k, v, k_lens=ints(lens), out=out, workspace=ws) is out
    assert (wide[0] == 5).all() and (wide[-1] == 5).all()
    flat = [t.flatten(0, 1) for t in (q, k, v)]
    want, bound, _ = R.attention(*flat, R.sequences(n * Lq, n * Lk, n,
                                                    k_lens=ints(lens)))
    R.check_bf16(out.flatten(0, 1), want, bound)
    assert (out[1] == 0).all()
    assert torch.equal(B.attention(q, k, v, k_lens=ints(lens)), out)


@pytest.mark.parametrize("D", [32, 56, 96, 128])
@pytest.mark.parametrize("tile,parts,q_len,k_len,Hq,Hk", [
    ("mid", 1, [500, 0, 129, 256], [700, 50, 0, 1300], 16, 16),
    ("mid", 2, [170, 0, 133], [2000, 100, 1500], 33, 11),
    ("many", 1, [1100, 1, 0, 257], [5000, 0, 3000, 700], 16, 16),
    ("many", 2, [300, 1, 0, 257], [5000, 0, 3000, 700], 32, 8),
    ("short", 1, [700, 3, 0, 130, 300], [64, 0, 40, 333, 1], 130, 65),
    ("some", 9, [100, 0, 90, 1], [4000, 10, 1, 1000], 4, 4),
    ("few", 8, [1, 0, 3, 1], [4000, 10, 0, 1300], 24, 8)])
def test_packed(tile, parts, q_len, k_len, Hq, Hk, D):
    n, Tq, Tk = len(q_len), sum(q_len) + 3, sum(k_len) + 2
    assert plan(Tq, Tk, n, True, Hq, Hk) == (tile, parts)
    need = B.attention_workspace_bytes(Tq, Tk, Hq, Hk, D, B=n, packed=True)
    assert (need > 0) == (parts > 1)
    g = gen(Tq + D)
    q = rand(g, Tq, Hq, D, std=1.5)
    k, v = rand(g, Tk, Hk, D, std=1.5), rand(g, Tk, Hk, D)
    k[sum(k_len):], v[sum(k_len):] = NAN, INF
    kw = dict(q_offsets=ints([x + 2 for x in starts(q_len)]),
              k_offsets=ints(starts(k_len)))
    check(q, k, v, n, **kw)
    kw["k_lens"] = ints([x // 2 for x in k_len])
    check(q, k, v, n, **kw)


@pytest.mark.parametrize("Lq,Lk,Hq,Hk", [(1, 5000, 8, 2), (600, 2100, 24, 24),
                                         (300, 700, 64, 64)])
def test_two_calls_at_once(Lq, Lk, Hq, Hk):
    """On two streams, each with a workspace of its own or the binding's."""
    sets = [(rand(gen(i), Lq, Hq, 64, std=1.5), rand(gen(9 + i), Lk, Hk, 64),
             rand(gen(99 + i), Lk, Hk, 64)) for i in range(2)]
    want = [B.attention(*s) for s in sets]
    need = max(B.attention_workspace_bytes(Lq, Lk, Hq, Hk, 64), 16)
    streams = [torch.cuda.Stream() for _ in sets]
    for own in (False, True):
        kw = [dict(workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
              if own else {} for _ in sets]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [[], []]
        for _ in range(5):
            for i, s in enumerate(streams):
                got[i].append(B.attention(*sets[i], stream=s, **kw[i]))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for w, outs in zip(want, got):
            assert all(torch.equal(o, w) for o in outs)

"""The block norms on the GPU against the same formulas in 64 bits."""
from __future__ import annotations

import pytest

from tests import normref as R
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rand(g, *shape, std=1.0, mean=0.0):
    return (mean + std * torch.randn(*shape, generator=g, device="cuda")).to(BF)


def guarded(shape, dtype):
    """A tensor with 4 KiB of canary on both sides, and its check."""
    n = torch.empty(0, dtype=dtype).element_size()
    for s in shape:
        n *= s
    raw = torch.full((8192 + n,), 0xA5, dtype=torch.uint8, device="cuda")
    t = raw[4096:4096 + n].view(dtype).view(*shape)

    def check():
        assert (raw[:4096] == 0xA5).all() and (raw[4096 + n:] == 0xA5).all()
    return t, check


def inputs(M, H, seed, post="rms", norm="rms", mods="broadcast", branch=True,
           affine=True, padded=False, outliers=True):
    """Arguments of a call, as the reference and the binding take them."""
    g = gen(seed)
    x = rand(g, M, H)
    if outliers:
        x = torch.where(torch.rand(M, H, generator=g, device="cuda") < 0.001,
                        20 * x, x)
    kw = {}
    if branch:
        kw["branch"] = rand(g, M, H, std=2.0, mean=0.5)
        kw["post_norm"] = post
        kw["residual_scale"] = 0.7
        if affine and post != "none":
            kw["post_weight"] = rand(g, H, mean=1.0, std=0.2)
        if affine and post == "layer":
            kw["post_bias"] = rand(g, H, std=0.2)
    if norm is not None:
        kw["norm_kind"] = norm
        if affine and norm != "none":
            kw["weight"] = rand(g, H, mean=1.0, std=0.2)
        if affine and norm == "layer":
            kw["bias"] = rand(g, H, std=0.2)
    rows = {"none": 0, "vector": 1, "broadcast": 1, "token": M,
            "index": min(M, 5)}[mods]
    if rows:
        table = rand(g, rows, 6 * H, std=0.3)
        part = lambda i: (table[0, i * H:(i + 1) * H] if mods == "vector" else
                          table[:, i * H:(i + 1) * H])
        if branch:
            kw["gate"] = part(2)
        if norm is not None:
            kw["shift"], kw["scale"] = part(0), part(1)
    if mods == "index" or padded:
        row = torch.randint(0, max(rows, 1), (M,), generator=g, device="cuda",
                            dtype=torch.int32)
        if padded:
            row[M // 2:] = torch.tensor([-1, max(rows, 1), -2**31, 2**31 - 1],
                                        device="cuda", dtype=torch.int32)[
                torch.arange(M - M // 2, device="cuda") % 4]
        kw["mod_row"] = row
    return x, kw


def call(x, kw, quantize=False, out=None, stream=None):
    """The binding's outputs for reference arguments."""
    kw = dict(kw)
    branch, norm = kw.pop("branch", None), kw.pop("norm_kind", None)
    if norm is not None:
        kw["norm"] = norm
    kw.update(out=out, stream=stream)
    if branch is None:
        f = B.norm_modulate_quantize if quantize else B.norm_modulate
        return f(x, **kw)
    if norm is None:
        return B.gated_residual(x, branch, **kw)
    f = B.gated_residual_norm_quantize if quantize else B.gated_residual_norm
    return f(x, branch, **kw)


def verify(x, kw, quantize, got):
    r, y = R.block(x, **kw)
    got = list(got) if isinstance(got, (tuple, list)) else [got]
    if r is not None:
        R.check_bf16(got.pop(0), *r)
    if y is not None:
        if quantize:
            R.check_codes(got[0], got[1], *y)
        else:
            R.check_bf16(got[0], *y)


def run_case(M, H, seed, quantize, **how):
    x, kw = inputs(M, H, seed, **how)
    shapes = []
    if how.get("branch", True):
        shapes.append(((M, H), BF))
    if how.get("norm", "rms") is not None:
        shapes += ([((M, H), torch.int8), ((M,), torch.float32)] if quantize
                   else [((M, H), BF)])
    outs, checks = zip(*[guarded(*s) for s in shapes])
    got = call(x, kw, quantize, out=outs[0] if len(outs) == 1 else outs)
    torch.cuda.synchronize()
    for c in checks:
        c()
    verify(x, kw, quantize, got)


# one lane's chunk, a partial wave, one wave, several rows a group, ragged
# chunks at every number of chunks a thread holds, the widest row
WIDTHS = [8, 16, 504, 512, 520, 1000, 1024, 2048, 2056, 4096, 4104, 5376,
          7168, 8192, 8200, 14336, 16384, 16392, 32768]


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, quantize):
    M = 7
    say(f"norm widths H={H} quantize={quantize}")
    run_case(M, H, H, quantize, post="layer", norm="layer", mods="token")
    run_case(M, H, H + 1, quantize, branch=False, norm="rms", mods="index")


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("norm", [None, "none", "rms", "layer"])
@pytest.mark.parametrize("mods", ["none", "vector", "broadcast", "token",
                                  "index"])
def test_kinds(post, norm, mods):
    say(f"norm kinds post={post} norm={norm} mods={mods}")
    for quantize in ([False] if norm is None else [False, True]):
        for affine in (False, True):
            run_case(33, 1000, 5, quantize, post=post, norm=norm, mods=mods,
                     affine=affine)
            if norm is not None:
                run_case(33, 1000, 6, quantize, norm=norm, mods=mods,
                         branch=False, affine=affine)


@pytest.mark.parametrize("M", [1, 2, 3, 5, 64, 255, 1025, 4097, 9001])
def test_tokens(M):
    say(f"norm tokens M={M}")
    for quantize in (False, True):
        run_case(M, 5376, M, quantize, post="rms", norm="layer", mods="index")
        run_case(M, 136, M, quantize, branch=False, norm="rms", mods="token")


@pytest.mark.parametrize("H,M", [
    (8, 250001), (512, 12001), (520, 12001), (1000, 6001), (1536, 4001),
    (1544, 4001), (3064, 2001), (5376, 1201), (8192, 801), (12288, 601),
    (16384, 401), (24576, 301), (24584, 301), (32768, 201)])
def test_many_values(H, M):
    """Past the size where work groups take two rows: odd row counts, runs of
    equal modulation rows, changes inside a pair, padding, one row each."""
    say(f"norm many H={H} M={M}")
    for quantize in (False, True):
        for mods in ("index", "token", "broadcast"):
            x, kw = inputs(M, H, H + M, post="rms", norm="layer", mods=mods,
                           padded=mods == "index")
            if mods == "index":
                row = (torch.arange(M, device="cuda") // 7 % 5).to(torch.int32)
                row[M // 2::5] = -1
                kw["mod_row"] = row
            verify(x, kw, quantize, call(x, kw, quantize))
            if mods != "token":
                x, kw = inputs(M, H, H, branch=False, norm="rms", mods=mods)
                verify(x, kw, quantize, call(x, kw, quantize))


@pytest.mark.parametrize("H", [136, 5376])
@pytest.mark.parametrize("quantize", [False, True])
def test_padding_rows(H, quantize):
    """Indices outside the table: r keeps x bit for bit, the rest is zero, and
    what the branch and x hold there (NaN, Inf) reaches nothing else."""
    M = 41
    say(f"norm padding H={H} quantize={quantize}")
    x, kw = inputs(M, H, 9, mods="index", padded=True)
    dead = M // 2
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0],
                       device="cuda", dtype=BF)
    x[dead:] = bad[torch.arange(H, device="cuda") % 4]
    kw["branch"][dead:] = float("nan")
    got = call(x, kw, quantize)
    live = {k: v[:dead] if k in ("branch", "mod_row") else v
            for k, v in kw.items()}
    verify(x[:dead], live, quantize, [t[:dead] for t in got])
    assert torch.equal(got[0][dead:].view(torch.int16),
                       x[dead:].view(torch.int16))
    assert all((t[dead:] == 0).all() for t in got[1:])
    # without vectors the index says only what is padding
    plain = {"mod_row": kw["mod_row"].clamp_max(2**31 - 2), "branch":
             kw["branch"], "norm_kind": "rms"}
    plain["mod_row"] = torch.where(torch.arange(M, device="cuda") < dead,
                                   plain["mod_row"].abs(), -1).to(torch.int32)
    got = call(x, plain, quantize)
    verify(x[:dead], {"branch": kw["branch"][:dead], "norm_kind": "rms"},
           quantize, [t[:dead] for t in got])
    assert torch.equal(got[0][dead:].view(torch.int16),
                       x[dead:].view(torch.int16))
    # every token padding, the norm alone
    none = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    got = call(x, {"norm_kind": "layer", "mod_row": none}, quantize)
    assert all((t == 0).all() for t in (got if quantize else [got]))


def test_special_rows():
    """Rows of zeros, of one value, with a mean far above their spread, near
    the ends of the range; a row with NaN or Inf spoils only itself."""
    H = 1000
    g = gen(3)
    x = rand(g, 10, H)
    x[0] = 0
    x[1] = 3.5
    x[2] = 256 + rand(g, H)
    x[3] = x[3] * 2.0**40
    x[4] = x[4] * 2.0**-60
    x[5] = torch.where(torch.arange(H, device="cuda") == 999, 5.0, 0.0)
    x[7, 17] = float("nan")
    x[8, 3] = float("inf")
    fine = [0, 1, 2, 3, 4, 5, 6, 9]
    for kind in ("rms", "layer", "none"):
        for quantize in (False, True):
            say(f"norm special kind={kind} quantize={quantize}")
            kw = {"norm_kind": kind}
            got = call(x, kw, quantize)
            got = got if quantize else [got]
            verify(x[fine], kw, quantize, [t[fine] for t in got])
        if not quantize and kind != "none":
            assert got[0][7].isnan().all()
    y = call(x, {"norm_kind": "rms"})
    assert y[7].isnan().all() and y[8].isnan().any()
    one = torch.full((3, 5376), 0.7, dtype=BF, device="cuda")
    assert (call(one, {"norm_kind": "layer"}) == 0).all()  # exactly
    for kind in ("rms", "layer"):
        s = call(x, {"norm_kind": kind}, True)[1]
        assert s[[7, 8]].isnan().all() and s[fine].isfinite().all()


def test_scales_down_to_subnormal():
    """Rows whose code scale is tiny, subnormal, or rounds to zero, through
    the map of one value to codes (no norm)."""
    H = 256
    base = rand(gen(2), 40, H).float()
    base[:, 0] = 4.0
    x = (base * 2.0 ** -torch.arange(90, 130, device="cuda").float()[:, None]
         ).to(BF)
    x[39, :] = 0
    x[39, :3] = 2.0 ** -133
    q, s = B.norm_modulate_quantize(x, norm="none")
    amax = x.double().abs().amax(1)
    assert ((s.double() - amax / 127).abs() <=
            amax / 127 * 2.0 ** -23 + 2.0 ** -150).all()
    v = x.double() / torch.where(s == 0, 1.0, s)[:, None].double()
    off = (q.double() - v.clamp(-127, 127)).abs()
    assert (off <= torch.where(s == 0, 1.0, 0.5 + 2.0 ** -14)[:, None]).all()
    assert (q[s == 0] == 0).all() and (q >= -127).all()


@pytest.mark.parametrize("eps", [2.0**-126, 1e-12, 1e-5, 10.0])
def test_eps(eps):
    x, kw = inputs(9, 520, 1, mods="vector")
    x[0] = 0
    kw.update(eps=eps, post_eps=2 * eps)
    verify(x, kw, False, call(x, kw))


def test_in_place_and_repeatable():
    x, kw = inputs(301, 5376, 12, mods="index", padded=True)
    want = [t.clone() for t in call(x, kw)]
    again = call(x, kw)
    for a, b in zip(want, again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    y = torch.empty_like(x)
    got = call(x, kw, out=(x, y))
    assert got[0].data_ptr() == x.data_ptr()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_fused_agrees_with_parts():
    """One pass against gated_residual, then norm_modulate of its BF16 sum:
    the sum is the same bit for bit, the norm within the sum's rounding."""
    x, kw = inputs(65, 5376, 4, mods="index")
    r, y = call(x, kw)
    res = {k: v for k, v in kw.items() if k not in
           ("norm_kind", "weight", "bias", "scale", "shift")}
    alone = call(x, res)
    assert torch.equal(alone.view(torch.int16), r.view(torch.int16))
    # a row of y by itself: the norm of one token equals that of the batch
    m = 17
    one = {k: v[m:m + 1] if k in ("branch", "mod_row") else v
           for k, v in kw.items()}
    r1, y1 = call(x[m:m + 1], one)
    assert torch.equal(r1.view(torch.int16), r[m:m + 1].view(torch.int16))
    assert torch.equal(y1.view(torch.int16), y[m:m + 1].view(torch.int16))


def test_index_of_every_order():
    """Neighbouring tokens with equal, alternating and random rows give what
    the same tokens give one by one."""
    M, H = 130, 5376
    x, kw = inputs(M, H, 8, mods="index")
    t = torch.arange(M, device="cuda", dtype=torch.int32)
    for row in (t * 0, t % 2, (t // 7) % 5, (t * 3 + 1) % 5, 4 - t % 5,
                torch.where(t % 3 == 0, -1, t % 5)):
        kw["mod_row"] = row.to(torch.int32)
        verify(x, kw, False, call(x, kw))
        verify(x, kw, True, call(x, kw, True))


def test_table_row_stride_zero_and_wide():
    M, H = 20, 256
    x, kw = inputs(M, H, 2, mods="none")
    g = gen(7)
    row = torch.arange(M, device="cuda", dtype=torch.int32) % 3
    one = rand(g, 1, H, std=0.3)
    kw.update(scale=one.expand(3, H), shift=rand(g, 3, 4 * H, std=0.3)[:, H:2 * H],
              gate=rand(g, 6, H)[::2], mod_row=row)
    assert kw["scale"].stride(0) == 0
    verify(x, kw, False, call(x, kw))


def test_other_stream():
    x, kw = inputs(513, 5376, 21, mods="index")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(x, kw, True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    verify(x, kw, True, got)


def test_graph_replay():
    """Captured once, replayed with new inputs and eager calls in between."""
    x, kw = inputs(129, 5376, 31, mods="index", padded=True)
    outs = (torch.empty_like(x), torch.empty(x.shape, dtype=torch.int8,
                                             device="cuda"),
            torch.empty(x.shape[0], device="cuda"))
    call(x, kw, True, out=outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, kw, True, out=outs)
    for i in range(3):
        x2, kw2 = inputs(129, 5376, 40 + i, mods="index", padded=True)
        x.copy_(x2)
        kw["branch"].copy_(kw2["branch"])
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        eager = call(x, kw, True)
        for a, b in zip(got, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        verify(x, kw, True, got)


def test_offsets_past_32_bits():
    """More than 2^31 values and 2^32 bytes a tensor: the last rows."""
    M, H = 70001, 32768
    say("norm 70001 x 32768")
    x = torch.zeros(M, H, dtype=BF, device="cuda")
    b = torch.zeros(M, H, dtype=BF, device="cuda")
    at = [0, 1, 65535, 65536, M - 2, M - 1]
    g = gen(1)
    x[at] = rand(g, len(at), H)
    b[at] = rand(g, len(at), H)
    kw = {"norm_kind": "rms", "post_norm": "layer"}
    got = call(x, {"branch": b, **kw})
    verify(x[at], {"branch": b[at], **kw}, False, [t[at] for t in got])
    del got
    got = call(x, {"branch": b, **kw}, True)
    verify(x[at], {"branch": b[at], **kw}, True, [t[at] for t in got])


def test_empty_is_refused():
    with pytest.raises(B.W8A8Error):
        B.norm_modulate(torch.empty(0, 64, dtype=BF, device="cuda"))

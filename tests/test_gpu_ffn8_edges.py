"""Edges of what surrounds the W8A8 products: scales of a few subnormal units, rows of
2^20 values and more, zeros' signs, GELU's tail, launches whose last tokens go apart, 9 to
16 tokens of few channels, tokens quantized by every workgroup, outputs on inputs.

Tolerances as in test_gpu_ffn8.py (u = 2^-24), whose references are used here."""
import math

import numpy as np
import pytest

from test_gpu_ffn8 import U, act_case, assert_within, gen, half_of, norm_ref, ops

from w4a4_quantized_gemm_quantize_amd import _lib

pytestmark = pytest.mark.gpu


# ------------------------------------------------- scales of a few subnormal units

@pytest.mark.parametrize("K", [64, 4096, 33024])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_codes_of_subnormal_scales(K, residual):
    """a / 127 rounds to so few units of 2^-149 that t / fl32(a / 127) passes 127: the codes stop there."""
    import torch
    tops = [1, 63, 64, 100, 127, 128, 190, 191, 254, 318, 320, 500, 2000, 20000]
    x = torch.randint(-64, 65, (len(tops), K), generator=gen(K), device="cuda").half()
    for i, a in enumerate(tops):
        x[i] = (x[i] * (a / 64)).round().clamp(-a, a)
        x[i, K // 3], x[i, K // 2] = a, -a
    w = torch.full((K,), 2.0 ** -149, device="cuda")
    r = torch.zeros_like(x) if residual else None
    q, s = ops().w8a8_rmsnorm_quantize(x, w, residual=r)[:2]
    t = (x.float() * w).cpu().numpy()
    a = np.abs(t).max(axis=1, keepdims=True)
    st = a / np.float32(127)
    with np.errstate(all="ignore"):
        ref = np.where(st > 0, np.clip(np.rint(t / st), -127, 127), 0)
    assert np.array_equal(a[:, 0] / np.float32(2.0 ** -149), tops) and float(np.abs(t / np.maximum(st, 1e-45)).max()) > 127.5
    assert np.array_equal(q.cpu().numpy(), ref)
    y = norm_ref(x, w, 1e-6)[3]
    assert_within(s, y.abs().amax(dim=1) / 127, 2.0 ** -149, "scale")


def test_moe_codes_of_subnormal_scales():
    """h of a few units of 2^-149: the codes of its row stop at 127, of either sign."""
    import torch
    H = I = 64
    unit, big = 2.0 ** -149, 2.0 ** 120
    for act in (None, "relu"):
        xq = torch.zeros((3, H), dtype=torch.int8, device="cuda")
        xq[:, 0] = torch.tensor([2, 3, 4], device="cuda")
        xs = torch.ones(3, device="cuda")
        c = torch.randint(-46, 47, (I,), generator=gen(1), device="cuda")
        c[5], c[9] = 47, -47                                      # largest h: 188, 423 and 752 units
        w13 = torch.zeros((1, 2 * I, H), dtype=torch.int8, device="cuda")
        w13[0, 0::2, 0] = c.to(torch.int8)                        # gate: c units times the token's code
        w13[0, 1::2, 0] = 1                                       # up: that code
        s13 = torch.ones((1, 2 * I), device="cuda")
        s13[0, 0::2] = unit
        w2 = torch.eye(H, dtype=torch.int8, device="cuda")[None].contiguous()
        s2 = torch.full((1, H), big, device="cuda")
        ids, f = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.full((3, 1), 2.0 ** 29, device="cuda")
        y = ops().w8a8_moe(xq, xs, ids, f, w13, s13, w2, s2, activation=act)
        n = xq[:, :1].double()
        h = c.double() * n * n                                    # in units
        if act == "relu":
            h = h.clamp_min(0)
        s = (h.abs().amax(dim=1, keepdim=True) / 127).round()     # fl32(a / 127): whole units
        assert bool((h.abs() / s).amax() > 127.5)
        assert torch.equal(y.double(), (h / s).round().clamp(-127, 127) * s), act


# ------------------------------------------------------------------- long rows

@pytest.mark.parametrize("K", [65552, 1 << 17, (1 << 20) + 16, 1 << 24])
def test_norm_of_long_rows(K):
    """The sum of squares of long rows keeps its bound: rows of one value, and others."""
    import torch
    for dtype in (torch.float16, torch.bfloat16):
        x = torch.full((2, K), 1.7, device="cuda").to(dtype)
        x[1] = torch.randn(K, generator=gen(K), device="cuda").to(dtype)
        w = torch.ones(K, dtype=dtype, device="cuda")
        w[K // 2:] = 0.75
        for r in (None, torch.ones_like(x)):
            got = ops().w8a8_rmsnorm_quantize(x, w, residual=r)
            h, q, s, _ = norm_ref(x, w, 1e-6, r)
            assert np.array_equal(got[0].cpu().numpy(), q)
            assert_within(got[1], s, 76 * U * s, f"scale {dtype}")
    big = torch.full((1, K), 3e25, dtype=torch.bfloat16, device="cuda")       # squares past fp32's range
    s = norm_ref(big, w, 1e-6)[2]
    assert_within(ops().w8a8_rmsnorm_quantize(big, w)[1], s, 76 * U * s, "scale, rescaled")


@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_more_than_2_22_rows(residual):
    """Rows past a launch's 2^22, in every input and output."""
    import torch
    M, K = (1 << 22) + 37, 16
    x = torch.randn(M, K, generator=gen(1), device="cuda").half()
    r = torch.randn(M, K, generator=gen(2), device="cuda").half() if residual else None
    w = torch.rand(K, generator=gen(3), device="cuda") + 0.5
    got = ops().w8a8_rmsnorm_quantize(x, w, residual=r, return_normed=True)
    m = (1 << 22) - 40
    part = ops().w8a8_rmsnorm_quantize(x[m:].clone(), w, residual=r[m:].clone() if residual else None, return_normed=True)
    for a, b in zip(got, part):
        assert torch.equal(a[m:], b)
    h, q, s, y = norm_ref(x[:64], w, 1e-6, r[:64] if residual else None)
    assert np.array_equal(got[0][:64].cpu().numpy(), q)
    assert_within(got[1][:64], s, 76 * U * s, "scale")


# ---------------------------------------------------------------- zeros' signs

@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("residual", [False, True])
def test_act_bits_of_zeros(act, gated, residual):
    """Closed gates and saturated activations: the sign bit of a zero is the same from the
    streaming kernel, the tiles, and the sums with their join."""
    import torch
    o, g = ops(), gen(7)
    M, N, K = 300, 272, 64
    C = 2 * N if gated else N
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (C, K), generator=g, device="cuda", dtype=torch.int8)
    wq[::5] = 0
    ws = 0.02 * torch.rand(C, generator=g, device="cuda")           # |v| up to some thousands: sigmoids of 0 and 1
    s = torch.randn(M, generator=g, device="cuda")
    s[::7] = 0
    r = torch.zeros((M, N), dtype=torch.float16, device="cuda") if residual else None
    if residual:
        r[::2] = -0.0
    call = lambda m, out: o.w8a8_gemm_act(q[:m], s[:m], wq, ws, activation=act, gated=gated,
                                          residual=None if r is None else r[:m], out_dtype=torch.float16, out=out)
    bits = lambda t: t.contiguous().view(torch.int16)
    tiles = call(M, None)
    narrow = torch.empty((M, N + 1), dtype=torch.float16, device="cuda")[:, :N]       # no 16-byte stores: the join
    assert _lib.workspace_bytes("w8a8_gemm_act_workspace", M, N, K, int(gated), 1) == 0
    assert _lib.workspace_bytes("w8a8_gemm_act_workspace", M, N, K, int(gated), 0) > 0
    assert bool((tiles == 0).any())
    assert torch.equal(bits(call(M, narrow)), bits(tiles))
    for m in (3, 16):
        assert torch.equal(bits(call(m, None)), bits(tiles[:m]))


# ------------------------------------------------------------------ GELU's tail

@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gelu_tail(dtype):
    """v Phi(v) from -13 up, without a residual and with one that takes its leading bits away."""
    import torch
    o, N, K = ops(), 4096, 16
    dtype = getattr(torch, dtype)
    v = torch.linspace(-13, 6, N, device="cuda")
    wq = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    wq[:, 0] = torch.where(v < 0, -1, 1).to(torch.int8)
    ws = v.abs()
    v = v.double()
    r = v.abs() * torch.special.erfc(v.abs() / math.sqrt(2)) / 2      # |v| Phi(-|v|)
    y = v.clamp_min(0) - r
    z = v.abs().clamp_max(16)
    bound = r * (z * z + 32) * 2 * U + U * y.abs()                    # v itself is exact
    rel, tiny = half_of(dtype)
    back = -y.to(dtype)                                               # with it: act(v) - rounded act(v)
    for M in (1, 16, 40):
        q = torch.zeros((M, K), dtype=torch.int8, device="cuda")
        q[:, 0] = 1
        s = torch.ones(M, device="cuda")
        got = o.w8a8_gemm_act(q, s, wq, ws, activation="gelu", out_dtype=dtype)
        assert_within(got, y.expand(M, N), bound * (1 + rel) + rel * y.abs() + tiny, "Y")
        got = o.w8a8_gemm_act(q, s, wq, ws, activation="gelu", residual=back.expand(M, N).contiguous(), out_dtype=dtype)
        left = y + back.double()
        assert_within(got, left.expand(M, N), (bound + U * left.abs()) * (1 + rel) + rel * left.abs() + tiny, "Y - round(Y)")
        odd = torch.empty((M, N + 1), dtype=dtype, device="cuda")[:, :N]
        assert torch.equal(o.w8a8_gemm_act(q, s, wq, ws, activation="gelu", out=odd),
                           o.w8a8_gemm_act(q, s, wq, ws, activation="gelu", out_dtype=dtype))


# ------------------------------------- the last tokens in a launch of their own

# (tokens, outputs, K, gated, bytes of int32 sums): the tail in 8 K ranges behind whole tiles; in whole tiles itself; both
# launches in K ranges, 2 of them for the first one's 512 tokens, in one workspace
TAILS = [(2070, 4096, 4096, False, 8 * 22 * 4096 * 4), (1185, 16192, 1760, True, 0),
         (530, 3840, 23888, False, 2 * 512 * 3840 * 4)]


@pytest.mark.parametrize("M,N,K,gated,sums", TAILS)
def test_act_last_tokens_in_tiles_of_their_own(M, N, K, gated, sums):
    import torch
    o = ops()
    dtype = torch.bfloat16
    need = _lib.workspace_bytes("w8a8_gemm_act_workspace", M, N, K, int(gated), 1)
    assert need == sums                                              # the launch that is meant
    x, q, s, wq, ws, b, r, y = act_case(M, N, K, "silu", gated, True, True, dtype, seed=3)
    guard = 1 << 16
    space = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    out = r.clone()
    o.w8a8_gemm_act(q, s, wq, ws, bias=b, activation="silu", gated=gated, residual=out, out=out, workspace=space[:need])
    assert torch.equal(out, y) and bool((space[need:] == 0x5A).all())
    m = M // 256 * 256
    for rows in (slice(0, m), slice(m, M)):                          # each part as a call of its own
        assert torch.equal(o.w8a8_gemm_act(q[rows].contiguous(), s[rows].contiguous(), wq, ws, bias=b, activation="silu",
                                           gated=gated, residual=r[rows], out_dtype=dtype), y[rows])
    total = _lib.workspace_bytes("w8a8_linear_act_workspace", M, N, K, int(gated), 1)
    space = torch.full((total + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    out.copy_(r)
    o.w8a8_linear_act(x, wq, ws, bias=b, activation="silu", gated=gated, residual=out, out=out, workspace=space[:total])
    assert torch.equal(out, y) and bool((space[total:] == 0x5A).all())
    wide = torch.full((M + 2, N + 24), 7.0, dtype=dtype, device="cuda")
    view = wide[1:M + 1, 8:8 + N]
    view.copy_(r)
    o.w8a8_gemm_act(q, s, wq, ws, bias=b, activation="silu", gated=gated, residual=view, out=view)
    assert torch.equal(view, y)
    view.fill_(7)
    assert bool((wide == 7).all())


# ------------------------------------------------ 9 to 16 tokens of few channels

@pytest.mark.parametrize("M,N,K", [(9, 200, 33040), (16, 2048, 32784), (13, 17, 65536), (16, 640, 131056)])
def test_few_channels_of_long_k(M, N, K):
    """In tiles of K ranges, as 8 of the tokens from the streaming kernel."""
    import torch
    o = ops()
    x, q, s, wq, ws, b, r, y = act_case(M, N, K, "silu", False, True, True, torch.float16, seed=K)
    assert torch.equal(y[:8], o.w8a8_gemm_act(q[:8], s[:8], wq, ws, bias=b, activation="silu", residual=r[:8]))
    for dtype in (torch.float32, torch.bfloat16):
        full = o.w8a8_gemm(q, s, wq, ws, bias=b, out_dtype=dtype)
        assert torch.equal(full[-8:], o.w8a8_gemm(q[-8:], s[-8:], wq, ws, bias=b, out_dtype=dtype))
        assert torch.equal(full, o.w8a8_linear(x, wq, ws, bias=b, out_dtype=dtype))
    if N % 2 == 0:
        act_case(M, N // 2, K, "gelu", True, False, True, torch.bfloat16, seed=N)


# ------------------------------------------- few tokens quantized by every workgroup

@pytest.mark.parametrize("M,N,K", [(4, 24600, 2064), (1, 30005, 4176), (8, 8200, 4096), (16, 9000, 512), (8, 8190, 4112)])
def test_few_tokens_of_many_channels(M, N, K):
    """One launch, W turned by LDS or not, or two: as the product on the tokens' codes."""
    import torch
    o = ops()
    for i, xdtype in enumerate((torch.float16, torch.bfloat16)):
        act_case(M, N, K, (None, "relu")[i], False, True, i == 0, (torch.bfloat16, torch.float16)[i], seed=N, xdtype=xdtype)
        x, q, s, wq, ws, b, _, _ = act_case(M, N // 2, K, "silu", True, False, True, torch.float16, seed=K, xdtype=xdtype)
        for bias in (None, torch.arange(len(ws), device="cuda").float()):
            y = o.w8a8_linear(x, wq, ws, bias=bias)
            assert torch.equal(y, o.w8a8_gemm(q, s, wq, ws, bias=bias))
            assert torch.equal(y[:1], o.w8a8_linear(x[:1], wq, ws, bias=bias))


# ------------------------------------------------------------------- refusals

def test_outputs_on_other_rows_tokens_are_refused():
    """Codes and scales over tokens that other workgroups still read, and outputs on one another."""
    import torch
    o = ops()
    raw = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    x = raw[:1024].view(torch.float16).view(8, 64)
    x.fill_(1)
    keep = raw.clone()
    r, w = torch.ones_like(x), torch.ones(64, device="cuda")
    codes = lambda at: raw[at:at + 512].view(torch.int8).view(8, 64)
    floats = lambda at: raw[at:at + 32].view(torch.float32)
    halfs = lambda at: raw[at:at + 1024].view(torch.float16).view(8, 64)
    fine = (codes(2048), floats(4096), halfs(8192), halfs(16384))
    for i, bad in [(0, codes(0)), (0, codes(1008)), (1, floats(512)), (1, floats(2048)), (2, halfs(2048)), (2, halfs(4000)),
                   (3, halfs(2048)), (3, halfs(8192)), (3, halfs(0)), (0, codes(8192)), (1, floats(16384)), (1, w[:8])]:
        with pytest.raises((ValueError, _lib.W4A4Error)):
            o.w8a8_rmsnorm_quantize(x, w, residual=r, return_normed=True, out=(*fine[:i], bad, *fine[i + 1:]))
    for bad in (halfs(0), halfs(512)):
        with pytest.raises((ValueError, _lib.W4A4Error)):                              # no residual: normed over x
            o.w8a8_rmsnorm_quantize(x, w, return_normed=True, out=(*fine[:2], bad))
    q, s = codes(2048), floats(4096)
    wq, ws = torch.ones((64, 64), dtype=torch.int8, device="cuda"), raw[32768:33024].view(torch.float32)
    bias = raw[33024:33280].view(torch.float32)
    for at in (1536, 2048, 2304, 3584, 32256, 33024):
        with pytest.raises((ValueError, _lib.W4A4Error)):
            o.w8a8_gemm_act(q, s, wq, ws, bias=bias, out=halfs(at))
    for at in (0, 512, 32256, 33024):
        with pytest.raises((ValueError, _lib.W4A4Error)):
            o.w8a8_linear_act(x, wq, ws, bias=bias, out=halfs(at))
    logits = raw[:2048].view(torch.float32).view(8, 64)
    ids = lambda at: raw[at:at + 128].view(torch.int32).view(8, 4)
    for a, b in [(256, 4096), (4096, 2016), (4096, 4096), (4096, 4160)]:
        with pytest.raises((ValueError, _lib.W4A4Error)):
            o.moe_route(logits, 4, out=(ids(a), ids(b).view(torch.float32)))
    e = [torch.ones(s, dtype=d, device="cuda") for s, d in [((8, 64), torch.int8), ((8,), torch.float32)]]
    w13, s13 = torch.ones((2, 64, 64), dtype=torch.int8, device="cuda"), torch.ones((2, 64), device="cuda")
    w2, s2 = raw[40960:45056].view(torch.int8).view(2, 64, 32), raw[45056:45568].view(torch.float32).view(2, 64)
    some, f = ids(4096), ids(4224).view(torch.float32)
    for at in (3584, 4096, 4224, 40960, 44544, 45056):
        with pytest.raises((ValueError, _lib.W4A4Error)):
            o.w8a8_moe(*e, some, f, w13, s13, w2, s2, out=halfs(at))
    assert torch.equal(raw, keep)                                    # nothing was launched
    o.w8a8_rmsnorm_quantize(x, w, residual=r, return_normed=True, out=fine)
    for a, b in zip(fine, o.w8a8_rmsnorm_quantize(x, w, residual=r, return_normed=True)):
        assert torch.equal(a, b)
    # a run in the gap between two rows, and columns of one buffer, are apart
    wide = torch.full((8, 160), 1.0, dtype=torch.float16, device="cuda")
    gap = wide.view(torch.float32)[3, 64:72]
    o.w8a8_rmsnorm_quantize(wide[:, :64], w, residual=r, return_normed=True, out=(q, gap, wide[:, 64:128], halfs(16384)))
    assert torch.equal(wide[:, 64:128], wide[:, :64] + r) and torch.equal(gap, fine[1])


def test_norm_of_a_residual_that_is_x():
    """Inputs may be the same tensor, whichever outputs are given."""
    import torch
    o = ops()
    x = torch.randn(5, 96, generator=gen(4), device="cuda").half()
    w = torch.rand(96, generator=gen(5), device="cuda").half()
    for normed in (False, True):
        want = o.w8a8_rmsnorm_quantize(x, w, residual=x, return_normed=normed)
        out = tuple(torch.empty_like(t) for t in want)
        for a, b in zip(o.w8a8_rmsnorm_quantize(x, w, residual=x, return_normed=normed, out=out), want):
            assert torch.equal(a, b)
        keep = x.clone()
        for a, b in zip(o.w8a8_rmsnorm_quantize(x, w, residual=x, return_normed=normed, out=(*out[:2], x, *out[3:])), want):
            assert torch.equal(a, b)
        x.copy_(keep)

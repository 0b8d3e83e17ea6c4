"""What surrounds the W8A8 products against its definitions in 64 bits: the RMS norm
that emits INT8 codes, products with an epilogue, the router, the experts' layer.

Tolerances, with u = 2^-24 (half a step of fp32) and `half` that of the output's type
(2^-11 fp16, 2^-8 bf16, relative; 2^-25 absolute below fp16's normal range):

* norm: the codes are exact (they depend on no sum). A lane sums at most 128 squares
  in a row and a tree of 12 steps joins them, so a sum of squares is off by 140 u and its
  root by 70 u; mean, eps, root, reciprocal and the two products of the scale round
  6 times more: 76 u.
* epilogues: v = P sx sw + b is off by dv = 3 u |P sx sw| + u |v|. The activations have
  slopes up to 1.13. v sigmoid(z): the argument of the exponential is off by 4 u |z|
  (its polynomial and the factor log2 e), which is the exponential's relative error, and
  exponential, sum, reciprocal and product add at most 2^-21 (one step of 2^-23 each for
  exponential and reciprocal, half a one for the others): (4 |z| u + 2^-21) |act|, and 2^-120 where
  the exponential overflows. GELU = max(v, 0) - r, r = z Phi(-z) within (z^2 + 32) 2 u,
  whose polynomial is within 1.3e-7 = 2.2 u and takes 14 roundings. Then the
  gate's product, the residual's sum and the output's rounding.
* experts: h carries the epilogue's error; where it moves a quotient h / s across
  the middle of two codes, the code may be one off, which moves the output by a step
  of h times that weight. Sums of k terms round k times.
"""
import math

import numpy as np
import pytest

from w4a4_quantized_gemm_quantize_amd import _lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}


def ops():
    from w4a4_quantized_gemm_quantize_amd import ops as o
    return o


def dt(name):
    import torch
    return getattr(torch, name)


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def half_of(dtype):
    return HALF[str(dtype).split(".")[1]]


def assert_within(got, ref, bound, what):
    import torch
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first "
                                 f"{torch.nonzero(bad)[:4].tolist()}, worst ratio "
                                 f"{float(((got.double() - ref).abs() / bound).nan_to_num(nan=math.inf).max()):.3g}")


# ------------------------------------------------------------------- norm

def norm_ref(x, w, eps, r=None):
    """(h, codes, scale, normed rows): codes in binary32 as they are defined, the rest in 64 bits."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    t = (h.float() * w.float()).cpu().numpy()
    a = np.abs(t).max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        st = a / np.float32(127)
        q = np.where(st > 0, np.rint(t / st), 0)
    h64 = h.double()
    rstd = 1 / ((h64 ** 2).mean(dim=1, keepdim=True) + eps).sqrt()
    y = h64 * w.double() * rstd
    return h, q, y.abs().amax(dim=1) / 127, y


def check_norm(x, w, eps=1e-6, residual=None, normed=False, out=None, keep=None):
    """keep: copies of x and residual from before, where `out` overwrites one of them."""
    x0, r0 = keep or (x, residual)
    got = ops().w8a8_rmsnorm_quantize(x, w, eps=eps, residual=residual, return_normed=normed, out=out)
    h, q, s, y = norm_ref(x0, w, eps, r0)
    assert np.array_equal(got[0].cpu().numpy(), q)
    assert_within(got[1], s, 76 * U * s + 2.0 ** -149, "scale")
    if r0 is not None:
        assert bool((got[2] == h).all())
    if normed:
        rel, tiny = half_of(x.dtype)
        assert_within(got[-1], y, (rel * (1 + 2.0 ** -18) + 76 * U) * y.abs() + tiny, "normed")
    return got


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (5, 1024), (4, 1040), (2, 4096), (7, 4112), (3, 8192), (2, 8208),
                                 (3, 11008), (2, 16400), (2, 28672), (2, 33024), (301, 256)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(M, K, dtype, residual):
    import torch
    g = gen(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(dt(dtype))
    x[:, K // 3] *= 50
    r = (3 * torch.randn(M, K, generator=g, device="cuda")).to(dt(dtype)) if residual else None
    for wdt in (dt(dtype), torch.float32):
        w = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(wdt)
        check_norm(x, w, residual=r, normed=wdt is torch.float32)


@pytest.mark.parametrize("K", [64, 4096, 33024])
def test_norm_strided_and_in_place(K):
    import torch
    g = gen(K)
    M = 6
    wide = torch.randn(M, K + 24, generator=g, device="cuda").half()
    wide_r = torch.randn(M, K + 8, generator=g, device="cuda").half()
    w = torch.rand(K, generator=g, device="cuda")
    x, r = wide[:, :K], wide_r[:, 8:]
    x0, r0, tail = x.clone(), r.clone(), wide[:, K:].clone()
    check_norm(x, w, residual=r, normed=True)
    new = lambda: (torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"))
    got = check_norm(x, w, residual=r, out=(*new(), r), keep=(x0, r0))
    assert got[2].data_ptr() == r.data_ptr() and torch.equal(x, x0)
    r.copy_(r0)
    check_norm(x, w, residual=r, out=(*new(), x), keep=(x0, r0))
    assert torch.equal(r, r0) and torch.equal(wide[:, K:], tail)


@pytest.mark.parametrize("K", [512, 4096, 16384])
def test_norm_rows_that_are_special(K):
    """Zero rows, rows of one value, rows that are not finite (scale NaN), beside ordinary ones."""
    import torch
    for dtype in (torch.float16, torch.bfloat16):
        x = torch.randn(7, K, generator=gen(1), device="cuda").to(dtype)
        x[1] = 0
        x[2] = 0
        x[2, K - 1] = 3
        x[3, 5] = float("nan")
        x[4, K // 2] = float("inf")
        x[5] = -1
        w = torch.ones(K, device="cuda")
        q, s, y = ops().w8a8_rmsnorm_quantize(x, w, return_normed=True)
        fine = [0, 1, 2, 5, 6]
        _, rq, rs, ry = norm_ref(x[fine], w, 1e-6)
        assert np.array_equal(q[fine].cpu().numpy(), rq)
        assert_within(s[fine], rs, 76 * U * rs, "scale")
        assert bool(s[[3, 4]].isnan().all()) and float(s[1]) == 0 and not bool(q[1].any()) and not bool(y[1].any())
        # a value that is not finite meets a weight of zero
        w[5] = 0
        w[K // 2] = 0
        assert bool(ops().w8a8_rmsnorm_quantize(x, w)[1][[3, 4]].isnan().all())


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e15, 1e19, 1e30, 1e37])
@pytest.mark.parametrize("K", [256, 8192, 33024])
def test_norm_bf16_range(scale, K):
    """Squares that pass fp32's range at both ends."""
    import torch
    x = (scale * torch.randn(3, K, generator=gen(2), device="cuda").clamp(-3, 3)).bfloat16()
    check_norm(x, (1 + 0.2 * torch.rand(K, generator=gen(3), device="cuda")), normed=True)
    check_norm(x, torch.full((K,), 1e-4, device="cuda"), residual=x.flip(0))


def test_norm_residual_that_overflows():
    import torch
    x = torch.full((2, 64), 60000.0, dtype=torch.float16, device="cuda")
    x[1] = 1
    got = ops().w8a8_rmsnorm_quantize(x, torch.ones(64, device="cuda"), residual=x)
    assert bool(got[1][0].isnan()) and bool(got[2][0].isinf().all()) and abs(float(got[1][1]) - 1 / 127) < 1e-6


# -------------------------------------------------------- products with an epilogue

def act_ref(v, name, dv):
    """(activation in 64 bits, bound of its error for an argument off by dv)."""
    import torch
    a = v.abs()
    if name is None:
        return v, dv
    if name == "relu":
        return v.clamp_min(0), dv
    if name == "gelu":
        y = v * torch.special.ndtr(v)
        z = a.clamp_max(16)
        r = z * torch.special.ndtr(-z)
        return y, 1.13 * dv + r * (z * z + 32) * 2 * U + U * y.abs()
    z = v if name == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    y = v * torch.sigmoid(z)
    # where |z| is large and positive its error multiplies exp(-z); where negative, the value is tiny
    return y, 1.13 * dv + y.abs() * (4 * z.abs().clamp_max(128) * U + 2.0 ** -21) + 2.0 ** -120


def epilogue_ref(p, q, s, wq, ws, bias, act, gated, residual):
    """(Y in 64 bits, bound before the output's rounding) from codes."""
    t = (q.double() @ wq.double().t()) * s.double()[:, None] * ws.double()
    v = t if bias is None else t + bias.double()
    dv = 3 * U * t.abs() + U * v.abs()
    if gated:
        a, da = act_ref(v[:, 0::2], act, dv[:, 0::2])
        u, du = v[:, 1::2], dv[:, 1::2]
        y, dy = a * u, u.abs() * da + a.abs() * du + da * du + U * (a * u).abs()
    else:
        y, dy = act_ref(v, act, dv)
    if residual is not None:
        y = y + residual.double()
        dy = dy + U * y.abs()
    return y, dy


def check_epilogue(y, q, s, wq, ws, bias, act, gated, residual):
    ref, bound = epilogue_ref(None, q, s, wq, ws, bias, act, gated, residual)
    rel, tiny = half_of(y.dtype)
    assert_within(y, ref, bound * (1 + rel) + rel * ref.abs() + tiny, "Y")


def act_case(M, N, K, act, gated, bias, residual, dtype, seed=0, xdtype=None):
    import torch
    o, g = ops(), gen(seed)
    C = 2 * N if gated else N
    x = (torch.randn(M, K, generator=g, device="cuda") * 2).to(xdtype or dtype)
    wq = torch.randint(-127, 128, (C, K), generator=g, device="cuda", dtype=torch.int8)
    ws = (0.02 + 0.01 * torch.rand(C, generator=g, device="cuda")) / (73 * math.sqrt(K) * 0.02)
    b = torch.randn(C, generator=g, device="cuda") if bias else None
    r = (2 * torch.randn(M, N, generator=g, device="cuda")).to(dtype) if residual else None
    q, s = o.w8a8_quantize_act(x)
    y = o.w8a8_gemm_act(q, s, wq, ws, bias=b, activation=act, gated=gated, residual=r, out_dtype=dtype)
    assert y.shape == (M, N) and y.dtype == dtype
    check_epilogue(y, q, s, wq, ws, b, act, gated, r)
    assert torch.equal(y, o.w8a8_linear_act(x, wq, ws, bias=b, activation=act, gated=gated, residual=r, out_dtype=dtype))
    return x, q, s, wq, ws, b, r, y


ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
# streaming kernel, 128 x 128 tiles whole and in K ranges, 256 x 128, 256 x 256, several tiles a workgroup; odd widths
SHAPES = [(1, 1, 16), (1, 200, 80), (5, 33, 144), (16, 256, 256), (3, 4096, 4096), (17, 100, 1040), (33, 304, 512),
          (64, 17, 2064), (130, 512, 4096), (300, 1000, 336), (515, 260, 128), (2048, 4096, 256), (4000, 4088, 256),
          (4200, 8200, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_act(M, N, K, gated):
    import torch
    acts = ACTS if M * N < 1 << 21 else [ACTS[(M + N) % 2], "silu", "gelu"]
    for i, act in enumerate(acts):
        act_case(M, N, K, act, gated, bias=(i + M) % 2 == 0, residual=i % 2 == 0 or act == "gelu",
                 dtype=(torch.float16, torch.bfloat16)[(i + N) % 2], seed=M + N + K + i,
                 xdtype=(torch.bfloat16, torch.float16)[i % 2])


@pytest.mark.parametrize("M,N,K,gated", [(1, 11008, 4096, True), (16, 4096, 11008, False), (8, 3584, 18944, False),
                                         (48, 3584, 18944, False), (128, 4096, 4096, True), (777, 18944, 3584, False),
                                         (2048, 11008, 4096, True)])
def test_act_model_shapes(M, N, K, gated):
    import torch
    act_case(M, N, K, "silu" if gated else None, gated, False, not gated, torch.bfloat16, seed=1)


@pytest.mark.parametrize("M,N,K,gated", [(1030, 8192, 512, True), (4100, 8192, 512, False), (2052, 8192, 1024, False)])
def test_act_tokens_past_a_multiple_of_256(M, N, K, gated):
    """The last tokens take a launch of their own."""
    import torch
    x, q, s, wq, ws, b, r, y = act_case(M, N, K, "gelu", gated, True, True, torch.bfloat16, seed=2)
    m = M - 20
    assert torch.equal(y[m:], ops().w8a8_gemm_act(q[m:].contiguous(), s[m:].contiguous(), wq, ws, bias=b, activation="gelu",
                                                  gated=gated, residual=r[m:], out_dtype=torch.bfloat16))


def test_act_without_an_epilogue_is_the_gemm():
    import torch
    for M, N, K in [(3, 96, 256), (70, 512, 1024), (300, 72, 336), (300, 71, 336)]:
        _, q, s, wq, ws, b, _, y = act_case(M, N, K, None, False, True, False, torch.float16, seed=9)
        assert torch.equal(y, ops().w8a8_gemm(q, s, wq, ws, bias=b, out_dtype=torch.float16))


@pytest.mark.parametrize("M,N,K", [(4, 64, 256), (130, 512, 4096), (300, 272, 256), (2048, 4096, 256)])
@pytest.mark.parametrize("gated", [False, True])
def test_act_strided_in_place_and_around(M, N, K, gated):
    import torch
    for pad, lead in ((16, 8), (9, 1)):                       # rows of 16-byte stores, and others
        x, q, s, wq, ws, b, r, y = act_case(M, N, K, "silu", gated, True, True, torch.float16, seed=5)
        big = torch.full((M + 2, N + pad), 7.0, dtype=torch.float16, device="cuda")
        view = big[1:M + 1, lead:lead + N]
        ops().w8a8_gemm_act(q, s, wq, ws, bias=b, activation="silu", gated=gated, residual=r, out=view)
        assert torch.equal(view, y)
        view.copy_(r)                                         # the residual stream, updated in place
        ops().w8a8_linear_act(x, wq, ws, bias=b, activation="silu", gated=gated, residual=view, out=view)
        assert torch.equal(view, y)
        assert bool((big[0] == 7).all()) and bool((big[M + 1] == 7).all())
        assert bool((big[:, :lead] == 7).all()) and bool((big[:, lead + N:] == 7).all())


def test_act_extremes():
    """Saturated activations, zero and NaN scales, the largest sums."""
    import torch
    o = ops()
    K = 64
    q = torch.full((20, K), 127, dtype=torch.int8, device="cuda")
    q[10:] = -127
    w = torch.full((32, K), 127, dtype=torch.int8, device="cuda")
    s = torch.ones(20, device="cuda")
    s[3] = 0
    s[5] = float("nan")
    for rows in (20, 7):                                     # tiles and the streaming kernel
        for top in (1e-9, 1e-6, 4e-5, 1e-3, 1.0):            # |v| up to 1e6: exp overflows
            ws = torch.full((32,), top, device="cuda")
            for act in ACTS:
                for gated in (False, True):
                    y = o.w8a8_gemm_act(q[:rows], s[:rows], w, ws, activation=act, gated=gated, out_dtype=torch.bfloat16)
                    keep = [i for i in range(rows) if i != 5]
                    assert bool(y[5].isnan().all()) and not bool(y[keep].isnan().any()) and not bool(y[3].any())
                    check_epilogue(y[keep], q[keep], s[keep], w, ws, None, act, gated, None)


def test_act_captured_and_on_another_stream():
    import torch
    o = ops()
    for M, N, K, gated in [(4, 512, 2048, True), (130, 512, 4096, False)]:
        x, q, s, wq, ws, b, r, y = act_case(M, N, K, "gelu_tanh", gated, True, True, torch.bfloat16, seed=3)
        call = lambda: o.w8a8_linear_act(x, wq, ws, bias=b, activation="gelu_tanh", gated=gated, residual=r,
                                         out_dtype=torch.bfloat16)
        replayed(call, y, lambda i: x.copy_(torch.randn(M, K, generator=gen(i), device="cuda")))


def replayed(call, y0, change):
    """The call on another stream, and captured: every replay as the eager call on the same inputs."""
    import torch
    same = lambda a, b: all(torch.equal(i, j) for i, j in zip(a, b)) if isinstance(a, tuple) else torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = call()
    torch.cuda.current_stream().wait_stream(side)
    assert same(y0, y1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = call()
    for i in range(3):
        change(i)
        graph.replay()
        torch.cuda.synchronize()
        assert same(y2, call()), f"replay {i}"


def test_pack_gated():
    import torch
    g = gen(4)
    for shape in ((6, 32), (3, 6, 32)):
        a, b = (torch.randn(*shape, generator=g, device="cuda").half() for _ in range(2))
        wq, ws = ops().w8a8_pack_gated(a, b)
        for half, w in ((0, a), (1, b)):
            q, s = ops().w8a8_pack_weight(w.reshape(-1, 32))
            assert torch.equal(wq[..., half::2, :].reshape(-1, 32), q) and torch.equal(ws[..., half::2].reshape(-1), s)


# ------------------------------------------------------------------- router

def check_route(logits, k, renorm):
    import torch
    ids, w = ops().moe_route(logits, k, renormalize=renorm)
    x = logits.double()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x).clamp_max(torch.finfo(torch.float32).max)
    order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    v = torch.gather(x, 1, order)
    none = v == -math.inf
    e = torch.where(none, torch.zeros_like(v), torch.exp(v - v[:, :1]))
    total = e.sum(1, keepdim=True) if renorm else torch.exp(x - v[:, :1]).nan_to_num(nan=0.0).sum(1, keepdim=True)
    ref = torch.where(none, torch.zeros_like(v), e / total)
    got_k = order.shape[1]
    assert torch.equal(ids[:, :got_k].long(), torch.where(none, torch.full_like(order, -1), order))
    assert bool((ids[:, got_k:] == -1).all()) and not bool(w[:, got_k:].any())
    # the difference rounds once (up to |l| u absolute, the exponential's relative error), the exponential by 2 u more, sums of up to
    # 512 terms in a lane's 8 and a tree, a division
    spread = (v[:, :1] - v).nan_to_num(posinf=0.0).abs()
    assert_within(w[:, :got_k], ref, ref * (2 * spread + 40) * U + 2.0 ** -126, "weights")


@pytest.mark.parametrize("T,E", [(1, 1), (1, 64), (5, 8), (3, 63), (7, 65), (130, 128), (4, 129), (6, 256), (9, 511),
                                 (1030, 512)])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_route(T, E, dtype):
    import torch
    x = (3 * torch.randn(T, E, generator=gen(T + E), device="cuda")).to(dt(dtype))
    for k in sorted({1, min(8, E), min(64, E), min(E + 3, 64)}):
        for renorm in (False, True):
            check_route(x, k, renorm)


def test_route_ties_masks_and_infinities():
    import torch
    for E in (8, 100, 256, 300):
        x = torch.randint(-2, 3, (40, E), generator=gen(E), device="cuda").float()
        x[x == 0] *= -1                                       # -0 and +0 are equal
        x[3] = -math.inf
        x[4, 2:] = -math.inf
        x[5, ::2] = math.nan
        x[6, 7] = math.inf
        x[7] = math.inf
        x[8, 1:4] = torch.finfo(torch.float32).min
        x[9] = torch.finfo(torch.float32).max
        x[10] = 0.0
        x[10, ::3] = -0.0
        x[11, 3:] = math.nan
        for k in (1, 6, 8):
            for renorm in (False, True):
                check_route(x, k, renorm)
        wide = torch.full((40, E + 5), 99.0, device="cuda")
        wide[:, :E] = x
        a, b = ops().moe_route(wide[:, :E], 4), ops().moe_route(x, 4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_route_empty_and_captured():
    import torch
    ids, w = ops().moe_route(torch.zeros((0, 16), device="cuda"), 4)
    assert ids.shape == w.shape == (0, 4)
    x = torch.randn(9, 60, generator=gen(1), device="cuda")
    call = lambda: ops().moe_route(x, 6)
    replayed(call, call(), lambda i: x.copy_(torch.randn(9, 60, generator=gen(i), device="cuda")))


# ------------------------------------------------------------------ experts

def moe_inputs(T, H, I, E, k, seed=0, ids=None):
    import torch
    g = gen(seed)
    o = ops()
    xq, xs = o.w8a8_quantize_act(torch.randn(T, H, generator=g, device="cuda").half())
    if ids is None:
        ids, weights = o.moe_route(torch.randn(T, E, generator=g, device="cuda") +
                                   torch.randn(E, generator=g, device="cuda"), k)
    else:
        weights = torch.rand(T, k, generator=g, device="cuda")
    code = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)
    scale = lambda n, *s: (1 + 0.3 * torch.rand(*s, generator=g, device="cuda")) / (73 * math.sqrt(n))
    return (xq, xs, ids, weights, code(E, 2 * I, H), 2 * scale(H, E, 2 * I), code(E, H, I), scale(I, E, H))


def moe_ref(args, act):
    """(Y in 64 bits, bound before the output's rounding)."""
    import torch
    xq, xs, ids, weights, w13, s13, w2, s2 = args
    (T, H), E = xq.shape, w13.shape[0]
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    dy, size = torch.zeros_like(y), torch.zeros_like(y)
    host = ids.cpu()
    for e in sorted({int(i) for i in host.flatten() if 0 <= i < E}):
        t, j = torch.nonzero(host == e, as_tuple=True)
        t, j = t.cuda(), j.cuda()
        h, dh = epilogue_ref(None, xq[t], xs[t], w13[e], s13[e], None, act, True, None)
        top = h.abs().amax(dim=1, keepdim=True)
        s = top / 127
        ds = torch.where(s > 0, dh.amax(dim=1, keepdim=True) / top.clamp_min(1e-300), torch.zeros_like(s)) + 3 * U
        x = torch.where(s > 0, h / s, torch.zeros_like(h))
        # a code that may be one off: its quotient is that near to the middle of two
        off = torch.where(s > 0, dh / s + x.abs() * ds, torch.zeros_like(x)) + U * x.abs()
        near = ((x - torch.floor(x)) - 0.5).abs() <= off
        part = (x.round() @ w2[e].double().t()) * s * s2[e].double()
        flips = (near.double() @ w2[e].double().abs().t()) * s * s2[e].double()
        f = weights[t, j].double()[:, None]
        y.index_add_(0, t, f * part)
        size.index_add_(0, t, (f * part).abs())
        dy.index_add_(0, t, f.abs() * (flips * 1.01 + part.abs() * (ds + 4 * U)))
    return y, dy + (ids.shape[1] + 1) * U * size


def check_moe(args, act="silu", dtype="float16", out=None):
    import torch
    y = ops().w8a8_moe(*args, activation=act, out_dtype=dt(dtype), out=out)
    ref, bound = moe_ref(args, act)
    rel, tiny = half_of(y.dtype)
    assert_within(y, ref, bound * (1 + rel) + rel * ref.abs() + tiny, "Y")
    assert torch.equal(y, ops().w8a8_moe(*args, activation=act, out_dtype=dt(dtype)))       # no order changes it
    return y


# one token; odd widths; the fused quantizer and the separate one; many rows an expert; every pair of 512
MOE = [(1, 64, 32, 4, 2), (1, 16, 16, 1, 1), (3, 80, 48, 5, 3), (1, 2048, 1024, 16, 8), (2, 512, 4112, 8, 4),
       (16, 512, 2368, 8, 4), (16, 272, 144, 60, 6), (13, 3584, 592, 32, 4), (17, 256, 1376, 8, 2), (32, 256, 80, 3, 2),
       (40, 256, 128, 4, 4), (64, 512, 256, 64, 8), (64, 4096, 96, 16, 8), (512, 64, 64, 7, 1), (8, 1024, 64, 512, 64)]


@pytest.mark.parametrize("T,H,I,E,k", MOE)
def test_moe(T, H, I, E, k):
    for i, act in enumerate(ACTS if T * I < 1 << 14 else ["silu", "gelu_tanh"]):
        check_moe(moe_inputs(T, H, I, E, k, seed=T + H + i), act, ("float16", "bfloat16")[(i + T) % 2])


@pytest.mark.parametrize("T,H,I,E,k", [(12, 400, 1040, 24, 4), (20, 1040, 704, 60, 8), (33, 272, 3232, 10, 3),
                                       (9, 2560, 1056, 16, 6), (170, 512, 592, 130, 3)])
def test_moe_few_channels(T, H, I, E, k):
    # the second stage in shares of the experts, against tokens on their own
    import torch
    args = moe_inputs(T, H, I, E, k, seed=H)
    ids = args[2]
    ids[1::3, 0] = -1
    ids[2::4, k - 1] = ids[2::4, 1]
    ids[T // 2] = E
    buf = torch.full((T + 1, H + 5), 3.0, dtype=torch.float16, device="cuda")
    out = buf[:T, 3:3 + H]
    ops().w8a8_moe(*args, out=out)
    for t in range(T):
        one = [a[t:t + 1].contiguous() if i < 4 else a for i, a in enumerate(args)]
        assert torch.equal(ops().w8a8_moe(*one)[0], out[t])
    assert bool((out[T // 2] == 0).all())
    assert bool((buf[T] == 3).all()) and bool((buf[:, :3] == 3).all()) and bool((buf[:, 3 + H:] == 3).all())
    check_moe(moe_inputs(T, H, I, E, k, seed=T), "gelu", "bfloat16")
    # two captured calls with their own workspaces, replayed in turn with eager ones
    calls = [moe_inputs(T, H, I, E, k, seed=s) for s in (1, 2)]
    want = [ops().w8a8_moe(*a) for a in calls]
    graph, got = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for a in calls:
            got.append(ops().w8a8_moe(*a))
    for _ in range(3):
        for y in got:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ops().w8a8_moe(*calls[0]), want[0])
        assert all(torch.equal(y, w) for y, w in zip(got, want))


def test_moe_ids_that_repeat_or_are_no_expert():
    import torch
    for T, k, E in [(1, 4, 8), (5, 4, 3), (20, 6, 4), (64, 8, 16)]:
        ids = torch.randint(-2, E + 2, (T, k), generator=gen(T), device="cuda", dtype=torch.int32)
        ids[0] = -1                                           # a token without any
        if T > 1:
            ids[1] = 2                                        # the same expert every time
            ids[2, 0], ids[2, 1] = 2 ** 31 - 1, -2 ** 31
        args = moe_inputs(T, 128, 96, E, k, ids=ids)
        y = check_moe(args)
        assert not bool(y[0].any())
    none = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    assert not bool(check_moe(moe_inputs(3, 64, 32, 4, 4, ids=none)).any())
    one = torch.full((64, 8), 3, dtype=torch.int32, device="cuda")                # 512 rows of one expert
    check_moe(moe_inputs(64, 128, 64, 5, 8, ids=one))


def test_moe_zero_and_nan_rows():
    import torch
    args = list(moe_inputs(6, 128, 64, 4, 2))
    args[1] = args[1].clone()
    args[1][2] = 0
    y = check_moe(args)
    assert not bool(y[2].any())
    args[1][4] = float("nan")
    y = ops().w8a8_moe(*args)
    assert bool(y[4].isnan().all()) and not bool(y[[0, 1, 2, 3, 5]].isnan().any())


def test_moe_strided_output_leaves_the_rest():
    import torch
    args = moe_inputs(5, 64, 32, 4, 2)
    for pad in (8, 3):
        big = torch.full((7, 64 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        check_moe(args, dtype="bfloat16", out=big[1:6, :64])
        assert bool((big[0] == 7).all()) and bool((big[6] == 7).all()) and bool((big[:, 64:] == 7).all())


def test_moe_experts_past_2_31_bytes():
    """The last expert's weights lie beyond 32-bit offsets."""
    import torch
    T, H, I, E = 2, 4096, 8192, 36                            # w13: 2.25 GiB
    ids = torch.tensor([[E - 1, 0], [E - 2, E - 1]], dtype=torch.int32, device="cuda")
    check_moe(moe_inputs(T, H, I, E, 2, ids=ids))


def test_moe_workspace_given_and_captured():
    import torch
    o = ops()
    for T, I in ((2, 96), (20, 2368)):
        args = moe_inputs(T, 256, I, 8, 2)
        need = _lib.workspace_bytes("w8a8_moe_workspace", T, 2, 8, 256, I)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")            # h is NaN where nothing writes it
        y = o.w8a8_moe(*args, workspace=ws)
        assert torch.equal(y, o.w8a8_moe(*args))
        with pytest.raises(ValueError):
            o.w8a8_moe(*args, workspace=ws[:-16])
        call = lambda: o.w8a8_moe(*args)

        def change(i):
            args[2].copy_(torch.randint(-1, 8, (T, 2), generator=gen(i), device="cuda", dtype=torch.int32))
        replayed(call, y, change)


def test_moe_of_no_token():
    import torch
    args = moe_inputs(1, 64, 32, 4, 2)
    y = ops().w8a8_moe(args[0][:0], args[1][:0], args[2][:0], args[3][:0], *args[4:])
    assert y.shape == (0, 64)


# ---------------------------------------------------------------- together

def test_a_block_of_all_of_them():
    """Norm, router, experts and a dense gated layer on one residual stream, each step
    against its definition on the step's own inputs; then the whole, captured."""
    import torch
    o, g = ops(), gen(11)
    T, H, I, E, k = 6, 512, 192, 8, 2
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, stream = rand(T, H).bfloat16(), rand(T, H).bfloat16()
    w = (1 + 0.1 * rand(H)).bfloat16()
    router = (rand(E, H) / math.sqrt(H)).bfloat16()
    w13, s13 = o.w8a8_pack_gated((0.05 * rand(E, I, H)).half(), (0.05 * rand(E, I, H)).half())
    w2, s2 = (t.view(E, H, -1) for t in o.w8a8_pack_weight((0.05 * rand(E * H, I)).half()))
    s2 = s2.view(E, H)
    up, up_s = o.w8a8_pack_gated((0.05 * rand(I, H)).half(), (0.05 * rand(I, H)).half())
    down, down_s = o.w8a8_pack_weight((0.05 * rand(H, I)).half())

    def block():
        q, s, h, n = o.w8a8_rmsnorm_quantize(x, w, residual=stream, return_normed=True)
        ids, f = o.moe_route(n @ router.t(), k)
        m = o.w8a8_moe(q, s, ids, f, w13, s13, w2, s2, out_dtype=torch.bfloat16)
        d = o.w8a8_gemm_act(q, s, up, up_s, activation="silu", gated=True, out_dtype=torch.bfloat16)
        y = o.w8a8_linear_act(d, down, down_s, residual=m, out_dtype=torch.bfloat16)
        return q, s, h, n, ids, f, m, d, y

    q, s, h, n, ids, f, m, d, y = block()
    check_norm(x, w, residual=stream, normed=True)
    check_route(n @ router.t(), k, True)
    args = (q, s, ids, f, w13, s13, w2, s2)
    check_moe(args, dtype="bfloat16")
    check_epilogue(d, q, s, up, up_s, None, "silu", True, None)
    dq, ds = o.w8a8_quantize_act(d)
    check_epilogue(y, dq, ds, down, down_s, None, None, False, m)
    out = lambda: block()[-1]
    replayed(out, y, lambda i: stream.copy_(rand(T, H)))


# ---------------------------------------------------------------- refusals

def test_outputs_that_meet_inputs_are_refused():
    import torch
    o = ops()
    buf = torch.ones((6, 192), dtype=torch.float16, device="cuda")
    x, r, h, y = buf[:4, :64], buf[:4, 64:128], buf[:4, 128:], torch.ones((4, 64), dtype=torch.float16, device="cuda")
    w = torch.ones(64, device="cuda")
    q, s = o.w8a8_quantize_act(x)
    norm = lambda h, y: o.w8a8_rmsnorm_quantize(x, w, residual=r, return_normed=True, out=(q, s, h, y))
    for bad in ((buf[1:5, :64], y), (buf[:4, 8:72], y), (buf[2:, 64:128], y), (h, x), (h, r), (h, h), (h, buf[:4, 96:160])):
        with pytest.raises(ValueError):
            norm(*bad)
    wq, ws = torch.ones((64, 64), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    for call, a in ((o.w8a8_gemm_act, (q, s)), (o.w8a8_linear_act, (x,))):
        for bad in (buf[1:5, 64:128], buf[:4, 72:136]):
            with pytest.raises(ValueError):
                call(*a, wq, ws, residual=r, out=bad)
    assert bool((buf == 1).all()) and bool((y == 1).all())
    apart = o.w8a8_linear_act(x, wq, ws, residual=r, out=h)      # three columns of one buffer
    assert torch.equal(apart, o.w8a8_linear_act(x.clone(), wq, ws, residual=r.clone()))
    norm(h, y)
    assert torch.equal(h, x + r)


def test_refusals_launch_nothing():
    import torch
    o = ops()
    x = torch.ones((4, 64), dtype=torch.float16, device="cuda")
    w = torch.ones(64, device="cuda")
    q, s = o.w8a8_quantize_act(x)
    for bad, exc in [(dict(weight=w[:32]), ValueError), (dict(weight=w.double()), TypeError), (dict(eps=0.0), ValueError),
                     (dict(eps=float("nan")), ValueError), (dict(residual=x[:2]), ValueError),
                     (dict(residual=x.bfloat16()), TypeError), (dict(out=(q, s, x)), ValueError),
                     (dict(out=(q, s[:2])), ValueError), (dict(weight=w.bfloat16()), TypeError)]:
        with pytest.raises(exc):
            o.w8a8_rmsnorm_quantize(**dict(dict(x=x, weight=w), **bad))
    with pytest.raises(_lib.W4A4Error):
        o.w8a8_rmsnorm_quantize(x[:, :40].contiguous(), w[:40].clone())
    with pytest.raises(TypeError):
        o.w8a8_rmsnorm_quantize(x.float(), w)
    y = torch.empty((4, 4), dtype=torch.float16, device="cuda")
    for bad, exc in [(dict(out_dtype=torch.float32), TypeError), (dict(activation="swish"), ValueError),
                     (dict(out=y[:, :3]), ValueError), (dict(residual=y.bfloat16()), TypeError),
                     (dict(residual=y[:2]), ValueError), (dict(gated=True, out=y), ValueError),
                     (dict(bias=torch.zeros(3, device="cuda")), ValueError)]:
        with pytest.raises(exc):
            o.w8a8_gemm_act(q, s, q, s, **bad)
        with pytest.raises(exc):
            o.w8a8_linear_act(x, q, s, **bad)
    with pytest.raises(ValueError):
        o.w8a8_gemm_act(q, s, q[:3], s[:3], gated=True)
    square, ones = torch.zeros((64, 64), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        o.w8a8_linear_act(x, square, ones, residual=x, out=x)
    wide = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        o.w8a8_linear_act(wide[:, :64], square, ones, out=wide[:, 32:96])
    with pytest.raises(ValueError):
        o.w8a8_gemm_act(q, s, torch.zeros((4, 80), dtype=torch.int8, device="cuda"), s)
    for k in (0, 65, -1, 2.0, True):
        with pytest.raises((ValueError, _lib.W4A4Error)):
            o.moe_route(w[None], k)
    with pytest.raises(_lib.W4A4Error):
        o.moe_route(torch.zeros((2, 513), device="cuda"), 2)
    args = moe_inputs(4, 64, 32, 4, 2)
    for i, t in enumerate(args):
        with pytest.raises((TypeError, ValueError)):
            o.w8a8_moe(*args[:i], t.double(), *args[i + 1:])
        with pytest.raises(ValueError):
            o.w8a8_moe(*args[:i], t[:3] if i < 4 else t[:, :16], *args[i + 1:])
    with pytest.raises(TypeError):
        o.w8a8_moe(*args, out_dtype=torch.float32)
    with pytest.raises(_lib.W4A4Error):
        o.w8a8_moe(*(t.repeat(65, *[1] * (t.dim() - 1)) if i < 4 else t for i, t in enumerate(args)))

"""W8A8 linear layers against their definition: codes and scales bit-exact
(symmetric INT8, one scale per row), the product against exact integer sums.

Tolerance of Y: the int32 sum is exact, its conversion, the product of the
scales, their product and the bias addition round once each to fp32 (2^-24
relative), the output rounds once to its type (2^-11 fp16, 2^-8 bf16, half a
smallest subnormal absolute)."""
import numpy as np
import pytest

from w4a4_quantized_gemm_quantize_amd import _lib, synth

pytestmark = pytest.mark.gpu

HALF_STEP = {"float32": (0.0, 0.0), "float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 0.0)}


def ops():
    from w4a4_quantized_gemm_quantize_amd import ops as o
    return o


def quant_ref(x32):
    """Codes and scales of a float32 matrix, in IEEE binary32 divisions."""
    a = np.abs(x32).max(axis=1).astype(np.float32)
    s = (a / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x32 / s[:, None])
    return np.where(s[:, None] > 0, q, 0).astype(np.int8), s


def check_quant(x, **kw):
    q, s = ops().w8a8_quantize_act(x, **kw)
    rq, rs = quant_ref(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    return q, s


def check_y(y, q, s, wq, ws, bias=None):
    import torch
    rel, tiny = HALF_STEP[str(y.dtype).split(".")[1]]
    y = y.double()
    t = (q.double() @ wq.double().t()) * s.double()[:, None] * ws.double()[None, :]
    ref = t if bias is None else t + bias.double()
    bound = 3 * 2.0 ** -24 * t.abs() + 2.0 ** -24 * ref.abs() + rel * (1 + 2.0 ** -20) * ref.abs() + tiny
    bad = (y - ref).abs() > bound
    assert not bool(bad.any()), f"{int(bad.sum())} outputs out of tolerance, first {torch.nonzero(bad)[:4].tolist()}"


def gemm_case(M, N, K, dtype, seed=0, bias=False, xdtype=None):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(M, K, generator=g, device="cuda") * 3).to(xdtype or torch.float16)
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).half()
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    o = ops()
    q, s = o.w8a8_quantize_act(x)
    wq, ws = o.w8a8_pack_weight(w)
    y = o.w8a8_gemm(q, s, wq, ws, bias=b, out_dtype=dtype)
    assert y.dtype == dtype and y.shape == (M, N)
    check_y(y, q, s, wq, ws, b)
    assert torch.equal(y, o.w8a8_linear(x, wq, ws, bias=b, out_dtype=dtype))
    return y


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (5, 1024), (4, 1040), (2, 4096), (7, 4112), (3, 11008), (2, 28672),
                                 (2, 33024), (300, 256)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantize_matches_definition(M, K, dtype):
    import torch
    x = torch.from_numpy(synth.activations(M, K, dist="t3", seed=M + K)).cuda().to(getattr(torch, dtype))
    x[M // 2] = 0                                       # a row of zeros: scale 0, codes 0
    check_quant(x)
    wide = torch.zeros((M, K + 24), dtype=x.dtype, device="cuda")
    wide[:, :K] = x
    check_quant(wide[:, :K])


def test_quantize_every_fp16_pair():
    """Every (maximum, value) pair of mantissas, value below the maximum by 0 to
    8 binary places: rne(fl32(x / s)) with IEEE divisions."""
    import torch
    man = torch.arange(1024, 2048, dtype=torch.float32)
    for shift in range(9):
        x = (man / 1024 * 2.0 ** -shift)[None, :].expand(1024, 1024).clone()
        top = man / 1024
        x = torch.minimum(x, top[:, None])              # a value above the maximum is not a pair
        x[:, 0] = top
        check_quant(torch.cat([x, -x], dim=1).half().cuda())


@pytest.mark.parametrize("scale", [2.0 ** -133, 2.0 ** -126, 2.0 ** -66, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 120])
def test_quantize_bf16_range(scale):
    """Rows whose scale is subnormal in fp32, at the border of the rescaling, and large."""
    import torch
    man = torch.arange(128, 256, dtype=torch.float64) / 128
    x = torch.stack([torch.minimum(man * 2.0 ** (-i % 8), man[i]) for i in range(128)])
    x[:, 0] = man
    x[:, 1::2] *= -1
    check_quant((x * scale).to(torch.bfloat16).cuda())


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 200, 80), (2, 33, 144), (16, 256, 256), (17, 100, 1040),
                                   (33, 300, 512), (64, 17, 2064), (65, 640, 1024), (130, 257, 400),
                                   (256, 512, 896), (300, 1000, 336), (515, 260, 128), (1, 4096, 4096)])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gemm(M, N, K, dtype):
    import torch
    gemm_case(M, N, K, getattr(torch, dtype), seed=M + N + K, bias=(M + N) % 2 == 1,
              xdtype=torch.bfloat16 if K % 32 else torch.float16)


@pytest.mark.parametrize("M,N,K", [(1, 11008, 4096), (16, 8192, 28672), (8, 1024, 8192), (48, 3584, 18944),
                                   (777, 3584, 18944), (128, 8192, 4096), (2048, 4096, 11008)])
def test_gemm_model_shapes(M, N, K):
    import torch
    gemm_case(M, N, K, torch.float16, seed=1)


def test_gemm_extreme_codes_and_longest_k():
    """-128 against -128 over the longest K: the largest sum that int32 holds."""
    import torch
    o = ops()
    K = 131056
    for M, N in [(1, 16), (20, 33), (129, 130)]:
        q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        w[0] = 127
        s, t = torch.ones(M, device="cuda"), torch.full((N,), 2.0 ** -20, device="cuda")
        check_y(o.w8a8_gemm(q, s, w, t), q, s, w, t)


def test_gemm_is_exact_where_fp32_is():
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    for M, N, K in [(3, 70, 1024), (200, 300, 1024)]:
        q = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        y = ops().w8a8_gemm(q, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"))
        assert torch.equal(y.double(), q.double() @ w.double().t())


def test_gemm_strided_output_leaves_the_rest():
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    for M, N, K in [(5, 40, 256), (300, 270, 256)]:
        x = torch.randn(M, K, generator=g, device="cuda").half()
        wq, ws = ops().w8a8_pack_weight(torch.randn(N, K, generator=g, device="cuda").half())
        for dt in (torch.float32, torch.bfloat16):
            big = torch.full((M + 2, N + 9), 7.0, dtype=dt, device="cuda")
            ops().w8a8_linear(x, wq, ws, out=big[1:M + 1, :N])
            assert torch.equal(big[1:M + 1, :N], ops().w8a8_linear(x, wq, ws, out_dtype=dt))
            assert bool((big[0] == 7).all()) and bool((big[M + 1] == 7).all()) and bool((big[:, N:] == 7).all())


def test_empty_and_one_row():
    import torch
    o = ops()
    wq, ws = o.w8a8_pack_weight(torch.ones((8, 64), dtype=torch.float16, device="cuda"))
    assert o.w8a8_linear(torch.zeros((0, 64), dtype=torch.float16, device="cuda"), wq, ws).shape == (0, 8)
    row = torch.ones((4, 64), dtype=torch.float16, device="cuda")[::4]      # one row of any stride
    assert o.w8a8_linear(row, wq, ws).shape == (1, 8)
    assert o.w8a8_gemm(*o.w8a8_quantize_act(row), wq[:0], ws[:0]).shape == (1, 0)


def test_captured_and_on_another_stream():
    import torch
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(7)
    for M, N, K in [(4, 512, 2048), (200, 300, 4096)]:
        x = torch.randn(M, K, generator=g, device="cuda").half()
        wq, ws = o.w8a8_pack_weight(torch.randn(N, K, generator=g, device="cuda").half())
        y0 = o.w8a8_linear(x, wq, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y1 = o.w8a8_linear(x, wq, ws)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y0, y1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y2 = o.w8a8_linear(x, wq, ws)
        for i in range(3):
            x.copy_(torch.randn(M, K, generator=g, device="cuda").half())
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y2, o.w8a8_linear(x, wq, ws)), f"replay {i}"


def test_refusals_launch_nothing():
    import torch
    o = ops()
    q = torch.zeros((4, 64), dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    for bad, exc in [(dict(out=torch.empty((4, 3), device="cuda")), ValueError),
                     (dict(out=torch.empty((4, 4), device="cuda", dtype=torch.float64)), TypeError),
                     (dict(bias=torch.zeros(3, device="cuda")), ValueError),
                     (dict(bias=torch.zeros(4, device="cuda", dtype=torch.float16)), TypeError),
                     (dict(out_dtype=torch.int32), TypeError)]:
        with pytest.raises(exc):
            o.w8a8_gemm(q, s, q, s, **bad)
    with pytest.raises(ValueError):
        o.w8a8_gemm(q, s[:3], q, s)
    with pytest.raises(ValueError):
        o.w8a8_gemm(q, s, torch.zeros((4, 80), dtype=torch.int8, device="cuda"), s)
    with pytest.raises(_lib.W4A4Error):
        o.w8a8_quantize_act(torch.zeros((4, 40), dtype=torch.float16, device="cuda"))
    with pytest.raises(_lib.W4A4Error):
        o.w8a8_quantize_act(torch.zeros((4, 68), dtype=torch.float16, device="cuda")[:, 1:65])
    with pytest.raises(TypeError):
        o.w8a8_quantize_act(torch.zeros((4, 64), device="cuda"))

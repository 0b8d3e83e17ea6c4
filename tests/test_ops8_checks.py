"""Argument validation of the 8-bit calls (CPU only): statuses of the C ABI,
which returns before any HIP call, and the tensor wrappers' refusals."""
import pytest
import torch

from w4a4_quantized_gemm_quantize_amd import _lib, ops

OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE = 0, 1, 2, 4, 5
F32, F16, BF16 = 0, 1, 2
P = 0x10000          # a fake, aligned "device pointer"


def test_quantize_validation():
    q = lambda *a: _lib.status_of("w8a8_quantize_act", *a)
    assert q(P, F32, 4, 64, 64, P, P, None) == E_DTYPE
    assert q(P, F16, -1, 64, 64, P, P, None) == E_SHAPE
    assert q(P, F16, 4, 0, 64, P, P, None) == E_SHAPE
    assert q(P, F16, 4, 72, 72, P, P, None) == E_SHAPE          # K % 16
    assert q(P, F16, 4, 64, 56, P, P, None) == E_SHAPE          # ldx < K
    assert q(P, BF16, 4, 64, 68, P, P, None) == E_ALIGN         # ldx % 8
    assert q(None, F16, 0, 64, 64, None, None, None) == OK
    assert q(None, F16, 4, 64, 64, P, P, None) == E_NULL
    assert q(P, F16, 4, 64, 64, P, None, None) == E_NULL
    assert q(P + 2, F16, 4, 64, 64, P, P, None) == E_ALIGN
    assert q(P, F16, 4, 64, 64, P + 8, P, None) == E_ALIGN
    assert _lib.status_of("w8a8_pack_weight", P, 7, 4, 64, P, P, None) == E_DTYPE


def test_gemm_validation():
    g = lambda *a: _lib.status_of("w8a8_gemm", *a)
    assert g(P, P, P, P, None, 4, 4, 72, None, 0, P, F32, 4, None) == E_SHAPE
    assert g(P, P, P, P, None, 4, 4, 131072, None, 0, P, F32, 4, None) == E_SHAPE    # 128^2 K = 2^31
    assert g(P, P, P, P, None, 4, -4, 64, None, 0, P, F32, 4, None) == E_SHAPE
    assert g(P, P, P, P, None, 1 << 31, 4, 64, None, 0, P, F32, 4, None) == E_SHAPE
    assert g(P, P, P, P, None, 4, 4, 64, None, 0, P, 3, 4, None) == E_DTYPE
    assert g(P, P, P, P, None, 4, 4, 64, None, 0, P, F32, 3, None) == E_SHAPE        # ldy < N
    assert g(P, P, None, P, None, 4, 4, 64, None, 0, P, F32, 4, None) == E_NULL
    assert g(P, P, P, P, P + 2, 4, 4, 64, None, 0, P, F32, 4, None) == E_ALIGN
    assert g(P, P, P + 8, P, None, 4, 4, 64, None, 0, P, F32, 4, None) == E_ALIGN
    assert g(P, P, P, P, None, 4, 4, 64, None, 0, P + 1, BF16, 4, None) == E_ALIGN
    assert g(None, None, None, None, None, 0, 4, 64, None, 0, None, F32, 4, None) == OK
    ws = _lib.load_library().w8a8_gemm_workspace
    assert ws(4, 4, 72) == -1 and ws(-1, 4, 64) == -1 and ws(0, 4, 64) == 0


def test_linear_validation():
    f = lambda x=P, xdt=F16, M=32, K=64, ldx=64, wq=P, ws=P, bias=None, N=4, wsp=P, wb=1 << 30, y=P, ydt=F16, ldy=4: \
        _lib.status_of("w8a8_linear", x, xdt, M, K, ldx, wq, ws, bias, N, wsp, wb, y, ydt, ldy, None)
    assert f(K=72) == E_SHAPE and f(M=-1) == E_SHAPE and f(ldx=56) == E_SHAPE and f(ldy=3) == E_SHAPE
    assert f(xdt=F32) == E_DTYPE and f(ydt=9) == E_DTYPE
    assert f(ldx=68) == E_ALIGN and f(x=P + 8) == E_ALIGN and f(wsp=P + 8) == E_ALIGN and f(bias=P + 2) == E_ALIGN
    assert f(x=None) == E_NULL and f(wq=None) == E_NULL and f(wsp=None) == E_NULL and f(y=None) == E_NULL
    assert f(x=None, wsp=None, wb=0, M=0) == OK and f(N=0) == OK
    need = _lib.load_library().w8a8_linear_workspace(32, 4, 64)
    assert need >= 32 * 64 + 4 * 32 and f(wb=need - 1) == E_SHAPE
    assert _lib.load_library().w8a8_linear_workspace(1, 4, 64) == 0      # one launch, which keeps nothing
    assert _lib.load_library().w8a8_linear_workspace(4, 4, 72) == -1


KV = dict(num_pages=8, heads=2, page=16, dim=64, table=P, ld=4, cu=P, lens=P, B=3, T=5, max_new=2, max_len=64)


def kv(**kw):
    d = dict(KV, **kw)
    return [d[k] for k in ("num_pages", "heads", "page", "dim", "table", "ld", "cu", "lens", "B", "T", "max_new",
                           "max_len")]


BAD_EXTENTS = [dict(num_pages=-1), dict(heads=0), dict(page=8), dict(page=48), dict(page=512), dict(dim=32),
               dict(dim=96), dict(dim=320), dict(B=-1), dict(B=65536), dict(T=-1), dict(max_new=-1),
               dict(max_len=-1), dict(max_len=65)]


def test_append_and_gather_validation():
    a = lambda x=F16, st=(128, 64, 128, 64), k=P, kc=P, **kw: _lib.status_of(
        "kv8_append", k, P, x, *st, kc, P, P, P, *kv(**kw), None)
    g = lambda y=F16, k=P, kc=P, **kw: _lib.status_of("kv8_gather", kc, P, P, P, *kv(**kw), k, P, y, None)
    for bad in BAD_EXTENTS:
        assert a(**bad) == E_SHAPE and g(**bad) == E_SHAPE, bad
    assert a(x=F32) == E_DTYPE and g(y=3) == E_DTYPE
    assert a(st=(128, 64, 128, 60)) == E_ALIGN and a(st=(-8, 64, 128, 64)) == E_SHAPE
    for empty in (dict(B=0), dict(T=0), dict(max_new=0)):
        assert a(k=None, kc=None, **empty) == OK and g(k=None, kc=None, **empty) == OK
    assert a(max_len=0) == OK                            # nothing can be stored
    for f in (a, g):
        assert f(k=None) == E_NULL and f(kc=None) == E_NULL and f(cu=None) == E_NULL and f(table=None) == E_NULL
        assert f(k=P + 8) == E_ALIGN and f(kc=P + 4) == E_ALIGN and f(lens=P + 2) == E_ALIGN


def test_attention_validation():
    def f(x=F16, qt=256, qh=64, hq=4, q=P, kc=P, scale=0.125, causal=1, window=0, ws=P, wbytes=1 << 40, y=P, ydt=F16,
          lse=None, **kw):
        return _lib.status_of("kv8_attention", q, x, qt, qh, hq, kc, P, P, P, *kv(**kw), scale, causal, window, ws,
                              wbytes, y, ydt, lse, None)
    for bad in BAD_EXTENTS:
        assert f(**bad) == E_SHAPE, bad
    assert f(x=F32) == E_DTYPE and f(ydt=5) == E_DTYPE
    assert f(hq=3) == E_SHAPE and f(hq=0) == E_SHAPE and f(window=-1) == E_SHAPE
    assert f(hq=2048, T=1 << 20) == E_SHAPE              # T q_heads = 2^31
    assert f(qt=252) == E_ALIGN and f(qt=-8) == E_SHAPE
    assert f(q=None) == E_NULL and f(kc=None) == E_NULL and f(y=None) == E_NULL
    assert f(q=P + 2) == E_ALIGN and f(lse=P + 2) == E_ALIGN and f(y=P + 8) == E_ALIGN
    assert f(q=None, T=0) == OK
    big = dict(max_len=1 << 20, ld=1 << 16, B=1, T=1, max_new=1)
    need = _lib.load_library().kv8_attention_workspace(4, 2, 16, 64, 1, 1, 1, 1 << 20, 1, 0)
    assert need > 0                                       # a long context is split
    assert f(wbytes=need - 1, **big) == E_SHAPE
    assert f(ws=None, wbytes=need, **big) == E_NULL
    assert f(ws=P + 4, wbytes=need, **big) == E_ALIGN
    w = _lib.load_library().kv8_attention_workspace
    assert w(3, 2, 16, 64, 1, 1, 1, 64, 1, 0) == -1 and w(4, 2, 0, 64, 1, 1, 1, 64, 1, 0) == -1
    assert w(4, 2, 16, 64, 0, 1, 1, 64, 1, 0) == 0


def test_wrappers_refuse_host_tensors_and_bad_numbers():
    x = torch.zeros((4, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        ops.w8a8_quantize_act(x)
    with pytest.raises(TypeError):
        ops.w8a8_gemm(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))
    with pytest.raises(ValueError):
        ops.kv8_new_cache(4, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError):
        ops.kv8_new_cache(4, 2, 16, 80, device="cpu")
    cache = ops.kv8_new_cache(4, 2, 16, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        ops.kv8_append(x, x, *cache, i[None], i, i[:1], 1)
    for bad in (-1, 1.0, True, None):
        with pytest.raises(ValueError):
            ops._need_max(bad, "max_new")
    with pytest.raises(ValueError):
        ops._heads_strides(torch.zeros(3, 2, 60), "k", 2, 64)
    with pytest.raises(ValueError):
        ops._heads_strides(torch.zeros(3, 64, 2).transpose(1, 2), "k", 2, 64)
    assert ops._heads_strides(torch.zeros(3, 6, 64)[:, 2:4], "k", 2, 64) == (384, 64)


def test_public_names():
    import w4a4_quantized_gemm_quantize_amd as pkg
    for name in ("w8a8_linear", "w8a8_gemm", "kv8_new_cache", "kv8_append", "kv8_gather", "kv8_attention"):
        assert getattr(pkg, name) is getattr(ops, name)


def test_nine_to_sixteen_tokens_of_few_channels_and_long_k_split_k():
    """Tiles in K ranges, which need a workspace, where 16 channels a workgroup would leave CUs idle."""
    w = _lib.load_library().w8a8_gemm_workspace
    for M in (9, 16):
        for N, K in [(16, 131056), (640, 40960), (1024, 98304), (2048, 53248), (2048, 32784)]:
            assert w(M, N, K) >= 2 * M * N * 4, (M, N, K)
        for N, K in [(2048, 28672), (1024, 16384), (2064, 53248), (8192, 28672)]:
            assert w(M, N, K) == 0, (M, N, K)
    assert w(8, 1024, 98304) == 0

"""Calls of the 8-bit operators at the edges of what their documentation allows:
bounds that are wrong on purpose (too small: nothing may leave the tensors),
empty pools and tables, negative and zero softmax scales, calls side by side on
two streams, two captured graphs, shapes whose K is split without wide stores."""
import math

import pytest

from w4a4_quantized_gemm_quantize_amd import _lib

from test_gpu_kv8 import Batch, attention_ref, check
from test_gpu_w8a8 import check_quant, check_y, gemm_case

pytestmark = pytest.mark.gpu


def ops():
    from w4a4_quantized_gemm_quantize_amd import ops as o
    return o


# ------------------------------------------------------------------- linears

@pytest.mark.parametrize("M,N,K", [
    (9, 20001, 4096), (16, 20001, 4096), (12, 8192, 8208),     # few tokens on tiles; N odd: element stores
    (9, 4097, 4112), (8, 20001, 4096), (16, 520, 16384),       # the streaming kernel, both workgroup sizes
    (64, 1001, 8192), (40, 130, 30000),                        # K split, odd rows of partial sums
])
@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_few_tokens_and_splits(M, N, K, dtype):
    import torch
    gemm_case(M, N, K, getattr(torch, dtype), seed=M + N, bias=True)


def test_linear_reads_strided_rows_and_broadcast_ones():
    import torch
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(40, 5 * 256, generator=g, device="cuda").half()
    wq, ws = o.w8a8_pack_weight(torch.randn(96, 256, generator=g, device="cuda").half())
    for M in (1, 5, 40):
        x = wide[:M, 512:768]
        assert torch.equal(o.w8a8_linear(x, wq, ws), o.w8a8_linear(x.contiguous(), wq, ws))
        same = wide[:1, 512:768].expand(M, 256)                # row stride 0
        if M > 1:
            with pytest.raises(_lib.W4A4Error):
                o.w8a8_linear(same, wq, ws)
        else:
            assert torch.equal(o.w8a8_linear(same, wq, ws), o.w8a8_linear(x, wq, ws))


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 16, 1024), (1, 17, 1040), (3, 100, 2064), (2, 8193, 4112),
                                   (4, 9000, 4096), (16, 40, 2000), (7, 300, 4096), (1, 500, 32768), (16, 8200, 1008)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_few_tokens_quantized_where_they_are_used(M, N, K, dtype):
    """The linear layer of few tokens (one launch) against its two steps, rows of
    zeros, of wide range and strided ones included."""
    import torch
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    wide = torch.randn(M, K + 8, generator=g, device="cuda") * 2.0 ** (torch.arange(M, device="cuda") - M // 2)[:, None]
    x = wide.to(getattr(torch, dtype))[:, :K]
    x[M // 2] = 0
    x[0, K - 1] = 30.0
    wq, ws = o.w8a8_pack_weight(torch.randn(N, K, generator=g, device="cuda").half())
    b = torch.randn(N, generator=g, device="cuda")
    y = o.w8a8_linear(x, wq, ws, bias=b, out_dtype=torch.float32)
    q, s = o.w8a8_quantize_act(x)
    assert torch.equal(y, o.w8a8_gemm(q, s, wq, ws, bias=b))
    check_y(y, q, s, wq, ws, b)


def test_linear_rows_of_zeros_give_the_bias():
    import torch
    o = ops()
    for M in (3, 100):
        x = torch.zeros((M, 128), dtype=torch.bfloat16, device="cuda")
        wq, ws = o.w8a8_pack_weight(torch.ones((48, 128), dtype=torch.bfloat16, device="cuda"))
        b = torch.arange(48, dtype=torch.float32, device="cuda")
        assert torch.equal(o.w8a8_linear(x, wq, ws, bias=b), b.expand(M, 48))
        zq, zs = o.w8a8_pack_weight(torch.zeros((48, 128), dtype=torch.bfloat16, device="cuda"))
        assert bool((o.w8a8_linear(x + 1, zq, zs) == 0).all()) and bool((zs == 0).all())


def test_linears_on_two_streams_and_in_two_graphs():
    """A K-split and a tiled product side by side, then captured into two graphs
    that are replayed in turn."""
    import torch
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(2)
    cases = []
    for M, N, K in [(48, 640, 8192), (300, 256, 1024), (2, 640, 2048)]:
        x = torch.randn(M, K, generator=g, device="cuda").half()
        wq, ws = o.w8a8_pack_weight(torch.randn(N, K, generator=g, device="cuda").half())
        cases.append((x, wq, ws))
    want = [o.w8a8_linear(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(8):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(o.w8a8_linear(*c))
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)
    graphs, outs = [], []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(o.w8a8_linear(*c))
    for _ in range(3):
        for x, _, _ in cases:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, o.w8a8_linear(*c)) for y, c in zip(outs, cases))


def test_quantize_one_long_row_and_the_largest_values():
    import torch
    x = torch.zeros((2, 40000), dtype=torch.float16, device="cuda")
    x[0, 39999], x[1, 0] = -65504.0, 2.0 ** -24
    check_quant(x)
    big = torch.finfo(torch.bfloat16).max
    check_quant(torch.tensor([[big, -big] + [1e38] * 14], device="cuda").bfloat16())


# --------------------------------------------------------------------- cache

@pytest.mark.parametrize("scale", [-0.11, 0.0, -30.0])
@pytest.mark.parametrize("new,lens", [([1, 2], [700, 40]), ([1], [5000]), ([9, 5], [300, 77]), ([120, 3], [300, 77])])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_softmax_scales_of_any_sign(scale, new, lens, dtype):
    B = Batch(new, lens, 2, 128, 64, dtype, seed=31)
    check(B, 6, scale=scale, window=0 if lens[0] % 2 == 0 else 50)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50), (False, 40), (True, 700)])
@pytest.mark.parametrize("new,lens,heads,kv", [([9, 3], [600, 3], 6, 2), ([5, 0, 4], [70, 33, 9], 28, 4), ([17], [17], 1, 1),
                                               ([8, 6], [5000, 260], 8, 1), ([32, 10], [1500, 900], 8, 2),
                                               ([100, 128], [2000, 600], 3, 3)])
@pytest.mark.parametrize("dim,page,dtype", [(64, 16, "float16"), (128, 32, "bfloat16"), (128, 256, "float16")])
def test_17_to_128_rows_per_kv_head(new, lens, heads, kv, causal, window, dim, page, dtype):
    B = Batch(new, lens, kv, dim, page, dtype, seed=39 + len(lens))
    check(B, heads, causal=causal, window=window, scale=-0.1 if window == 50 else None)


def test_bad_pages_and_nan_rows_of_drafts():
    import torch
    B = Batch([9, 6], [300, 130], 2, 128, 32, seed=40)
    B.table_host[0, 2], B.table_host[0, 9], B.table_host[1, 0] = 1 << 29, -1, B.kc.shape[0]
    B.table = B.table_host.cuda()
    ref = Batch([9, 6], [300, 130], 2, 128, 32, seed=40)
    q = B.rand(8)
    y = ops().kv8_attention(q, *B.pool, B.max_new, B.max_len)
    o, _, bound = attention_ref(ref, q, True, 0, 128 ** -0.5, {0: [(64, 96), (288, 300)], 1: [(0, 32)]})
    t = B.cu_host[-1]
    assert bool(((y.double() - o).abs()[:t] <= (bound + 2.0 ** -10 * o.abs() + 2.0 ** -24)[:t]).all())
    q[3, 5] = float("nan")
    z = ops().kv8_attention(q, *B.pool, B.max_new, B.max_len)
    keep = torch.ones(B.total, 8, dtype=torch.bool)
    keep[3, 5] = False
    keep[t:] = False
    assert bool(torch.isnan(z[3, 5]).all()) and torch.equal(z[keep.cuda()], y[keep.cuda()])


@pytest.mark.parametrize("new", [1, 5, 20, 90])
def test_pool_without_pages_and_sequences_without_positions(new):
    """No page in the pool, or no column in the table: every query sees nothing,
    tokens read back as zeros, nothing is stored."""
    import torch
    o = ops()
    B = Batch([new, 0, new], [new + 3, 0, new], 2, 64, 16, seed=32)
    q, k = B.rand(4), B.rand(2)
    t = B.cu_host[-1]
    none = o.kv8_new_cache(0, 2, 16, 64)
    no_column = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    for pool, table, max_len in ((none, B.table, B.max_len), (B.pool[:4], no_column, 0), (B.pool[:4], B.table, 0)):
        batch = (table, B.cu, B.sl)
        y, lse = o.kv8_attention(q, *pool, *batch, B.max_new, max_len, return_lse=True)
        assert bool((y[:t] == 0).all()) and bool((lse[:t] == -math.inf).all())
        if max_len == 0 and table is B.table:
            continue
        o.kv8_append(k, k, *pool, *batch, B.max_new)
        a, b = o.kv8_gather(*pool, *batch, B.total, B.max_new)
        assert bool((a[:t] == 0).all()) and bool((b[:t] == 0).all())


@pytest.mark.parametrize("new,lens,max_new,max_len", [([7, 2], [300, 900], 2, 912), ([90, 200], [400, 200], 64, 400),
                                                      ([3, 1], [700, 90], 3, 256), ([130], [2000], 20, 1024)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 40), (True, 33)])
def test_bounds_that_are_too_small_cut_the_batch(new, lens, max_new, max_len, causal, window):
    """Results are those of the cut batch: at most max_new new tokens, at most
    max_len positions. Everything else is left as it was."""
    import torch
    o = ops()
    B = Batch(new, lens, 2, 64, 16, seed=33)
    q, t = B.rand(4), B.cu_host[-1]
    out = torch.full_like(q, 7.0)
    need = o._workspace_size("kv8_attention_workspace", 4, 2, 16, 64, len(new), B.total, max_new, max_len, int(causal), window)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    o.kv8_attention(q, *B.pool, max_new, max_len, causal=causal, window=window, out=out, workspace=ws)
    assert bool((ws[need:] == 255).all())
    seen = torch.zeros(B.total, dtype=torch.bool, device="cuda")
    for b, (n, length) in enumerate(zip(new, lens)):
        n1, l1, t0 = min(n, max_new), min(length, max_len), B.cu_host[b]
        cu = torch.tensor([0, n1], dtype=torch.int32, device="cuda")
        sl = torch.tensor([l1], dtype=torch.int32, device="cuda")
        C = Batch([n1], [l1], 2, 64, 16, seed=33, tail=0)
        C.kc, C.vc, C.ks, C.vs, C.table, C.cu, C.sl = *B.pool[:4], B.table[b:b + 1], cu, sl
        qq = q[t0:t0 + n1].contiguous()
        o1, _, bound = attention_ref(C, qq, causal, window, 64 ** -0.5)
        y = out[t0:t0 + n1].double()
        assert bool(((y - o1).abs() <= bound + 2.0 ** -11 * (o1.abs() + bound) + 2.0 ** -25).all())
        seen[t0:t0 + n1] = True
    assert bool((out[~seen] == 7).all())
    # storing and reading back: the same tokens
    k, v = B.rand(2), B.rand(2)
    o.kv8_append(k, v, *B.pool, max_new)
    a = torch.full((B.total, 2, 64), 9.0, dtype=torch.float16, device="cuda")
    c = a.clone()
    o.kv8_gather(*B.pool, B.total, max_new, out=(a, c))
    seen[:] = False
    for b, n in enumerate(new):
        seen[B.cu_host[b]:B.cu_host[b] + min(n, max_new)] = True
    assert bool((a[~seen] == 9).all()) and bool((c[~seen] == 9).all())
    # half a step of the largest stored scale, and fp16's own half step
    for x, got, s in ((k, a, B.ks), (v, c, B.vs)):
        step = torch.nan_to_num(s).max()
        assert bool(((x - got)[seen].float().abs() <= 0.51 * step + 2.0 ** -10 * x[seen].abs().float()).all())
    del t


def test_cu_seqlens_out_of_range_stay_inside():
    """Starts and ends past the packed tokens, running backwards, negative: read as
    cut to them, without an access outside."""
    import torch
    o = ops()
    B = Batch([4, 4], [40, 40], 2, 64, 16, seed=34, tail=0)
    q = B.rand(4)
    for cu, live in (([-5, 4, 1000], [(0, 4), (4, 8)]), ([6, 2, 2], []), ([0, 0, 8], [(0, 0), (0, 8)])):
        B.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 7.0)
        o.kv8_attention(q, *B.pool, 8, B.max_len, out=out)
        touched = torch.zeros(8, dtype=torch.bool, device="cuda")
        for lo, hi in live:
            touched[lo:hi] = True
        assert bool((out[~touched] == 7).all()) and not bool((out[touched] == 7).all(dim=2).any())
    for lens in ([-3, 1 << 30], [0, 40]):
        B.cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
        B.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        y = o.kv8_attention(q, *B.pool, 4, B.max_len)
        assert bool((y[:4] == 0).all()) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("new,lens", [([1, 1], [9000, 700]), ([100, 20], [400, 20])])
def test_attention_on_two_streams_and_in_two_graphs(new, lens):
    import torch
    o = ops()
    Bs = [Batch(new, lens, 2, 128, 64, seed=35 + i) for i in range(2)]
    qs = [B.rand(8) for B in Bs]
    t = Bs[0].cu_host[-1]

    def run(i):
        return o.kv8_attention(qs[i], *Bs[i].pool, Bs[i].max_new, Bs[i].max_len)
    want = [run(i)[:t] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(i))
    torch.cuda.synchronize()
    assert all(torch.equal(y[:t], want[i]) for i in range(2) for y in got[i])
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(i))
    for _ in range(3):
        for q, B in zip(qs, Bs):
            q.copy_(B.rand(8))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i][:t], run(i)[:t]) for i in range(2))


def test_keys_and_values_shared_between_heads_by_a_view():
    """Head stride 0: every kv head stores the same rows."""
    import torch
    B = Batch([5, 40], [21, 40], 3, 64, 16, seed=37)
    one = B.rand(1)
    k = one.expand(-1, 3, -1)
    ops().kv8_append(k, k, *B.pool, B.max_new)
    a, c = ops().kv8_gather(*B.pool, B.total, B.max_new, out_dtype=torch.float32)
    whole = slice(B.cu_host[1], B.cu_host[2])                 # its pages hold new tokens only
    assert torch.equal(a[whole, 0], a[whole, 2]) and torch.equal(a[whole], c[whole])


def test_a_sequence_twice_reads_the_same_pages():
    """Two rows of the table name the same pages (a shared prefix): reading is fine."""
    import torch
    B = Batch([1, 1], [300, 300], 2, 64, 16, seed=38)
    B.table = B.table[:1].expand(2, -1).contiguous()
    q = B.rand(4)
    q[1] = q[0]
    y = ops().kv8_attention(q, *B.pool, B.max_new, B.max_len)
    assert torch.equal(y[0], y[1])


def test_gemm_checks_its_split_workspace():
    import torch
    o = ops()
    q = torch.randint(-127, 128, (48, 8192), device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (640, 8192), device="cuda", dtype=torch.int8)
    s, t = torch.rand(48, device="cuda"), torch.rand(640, device="cuda")
    need = o._workspace_size("w8a8_gemm_workspace", 48, 640, 8192)
    assert need > 0
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    check_y(o.w8a8_gemm(q, s, w, t, workspace=ws), q, s, w, t)
    assert bool((ws[need:] == 255).all())
    with pytest.raises(ValueError):
        o.w8a8_gemm(q, s, w, t, workspace=ws[:need - 1])

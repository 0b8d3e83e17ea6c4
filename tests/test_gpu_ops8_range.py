"""The 8-bit operators at the ends of the range of their inputs."""
import copy
import math

import numpy as np
import pytest

from test_gpu_kv8 import Batch, attention_ref, check_append

pytestmark = pytest.mark.gpu

# new tokens, positions, query heads over 2 kv heads of 128 dimensions: a call of
# at most 16, at most 128 and more query rows per kv head
KERNELS = {"decode": ([1, 2], [300, 517], 8), "draft": ([9, 5], [300, 517], 8), "prefill": ([70, 40], [300, 517], 8)}


def ops():
    from w4a4_quantized_gemm_quantize_amd import ops as o
    return o


def attend(B, q, scale=None, **kw):
    return ops().kv8_attention(q, *B.pool, B.max_new, B.max_len, scale=scale, return_lse=True, **kw)


# ------------------------------------------------------- value scales of zero

@pytest.mark.parametrize("kernel", KERNELS)
def test_values_of_scale_zero_give_zeros(kernel):
    """Softmax weights sum to one whatever the values are: zeros give zeros, with
    the log-sum-exp of the scores."""
    import torch
    new, lens, heads = KERNELS[kernel]
    B = Batch(new, lens, 2, 128, 64, seed=51)
    B.vs[:] = 0.0
    q = B.rand(heads)
    y, lse = attend(B, q)
    t = B.cu_host[-1]
    _, want, _ = attention_ref(B, q, True, 0, 128 ** -0.5)
    assert bool((y[:t] == 0).all())
    assert bool(((lse[:t].double() - want[:t]).abs() <= 2.0 ** -10).all())
    # a pool as kv8_new_cache returns it: every key and value is zero
    fresh = ops().kv8_new_cache(B.kc.shape[0], 2, 64, 128)
    y, lse = ops().kv8_attention(q, *fresh, *B.pool[4:], B.max_new, B.max_len, causal=False, return_lse=True)
    assert bool((y[:t] == 0).all())
    for b, length in enumerate(lens):
        rows = lse[B.cu_host[b]:B.cu_host[b + 1]]
        # exp2 and log2 of one ulp each, the conversion to natural logarithms
        assert bool(((rows - math.log(length)).abs() <= 2.0 ** -20 * math.log(length)).all())


@pytest.mark.parametrize("page", [64, 256])
@pytest.mark.parametrize("kernel", KERNELS)
def test_whole_pages_that_are_none_of_the_pool(kernel, page):
    """64 and more consecutive positions without a page are masked."""
    new, lens, heads = KERNELS[kernel]
    B = Batch(new, lens, 2, 128, page, seed=52)
    B.table_host[0, 0], B.table_host[1, 1] = -1, 1 << 29
    B.table = B.table_host.cuda()
    ref = Batch(new, lens, 2, 128, page, seed=52)
    q = B.rand(heads)
    y, _ = attend(B, q)
    o, _, bound = attention_ref(ref, q, True, 0, 128 ** -0.5, {0: [(0, page)], 1: [(page, 2 * page)]})
    t = B.cu_host[-1]
    assert bool(((y.double() - o).abs()[:t] <= (bound + 2.0 ** -11 * (o.abs() + bound) + 2.0 ** -25)[:t]).all())


# ------------------------------------------------------- negative positions

def seen_ref(B, q, causal, window, max_len=None):
    """As attention_ref, for sequences with more new tokens than positions (their
    first tokens see nothing), lengths cut to max_len."""
    import torch
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    bound, lse = torch.zeros_like(o), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(zip(B.new, B.lens)):
        length = length if max_len is None else min(length, max_len)
        C = copy.copy(B)
        C.new, C.lens, C.cu_host, C.table = [min(n, length)], [length], [0, min(n, length)], B.table[b:b + 1]
        rows = slice(B.cu_host[b + 1] - C.new[0], B.cu_host[b + 1])
        o[rows], lse[rows], bound[rows] = attention_ref(C, q[rows].contiguous(), causal, window, B.dim ** -0.5)
    return o, lse, bound


@pytest.mark.parametrize("causal,window", [(False, 0), (False, 3), (False, 100), (True, 0), (True, 100)])
@pytest.mark.parametrize("new,lens,max_len", [([5, 2], [3, 1], None), ([4, 4], [130, 3], 3), ([20, 25], [7, 90], None),
                                              ([30, 6], [200, 100], 17), ([90, 150], [70, 200], None),
                                              ([150, 100], [300, 300], 100), ([6, 200], [0, 1], None)])
@pytest.mark.parametrize("dim", [128, 192])
def test_tokens_at_negative_positions_see_nothing(new, lens, max_len, causal, window, dim):
    import torch
    B = Batch(new, lens, 2, dim, 16, seed=53)
    q = B.rand(6)
    y, lse = ops().kv8_attention(q, *B.pool, B.max_new, B.max_len if max_len is None else max_len, causal=causal,
                                 window=window, return_lse=True)
    o, want, bound = seen_ref(B, q, causal, window, max_len)
    t = B.cu_host[-1]
    assert torch.equal(torch.isinf(lse[:t]), torch.isinf(want[:t])), "which rows see something"
    assert bool((y[:t][torch.isinf(want[:t])] == 0).all())
    assert bool(((y.double() - o).abs()[:t] <= (bound + 2.0 ** -11 * (o.abs() + bound) + 2.0 ** -25)[:t]).all())


# ------------------------------------------------- results half way between two

@pytest.mark.parametrize("top", [2.0, 6.0, 10.0, 12.0, 14.0, 96.0])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_rescaled_codes_round_their_product_first(top, dtype):
    """Every code of a page with maximum 1 when the maximum becomes `top`: rne(fl32(q
    fl32(s_old / s))), whose product lies within a rounding of a half for many."""
    import torch
    B = Batch([1, 3], [33, 18], 2, 64, 64, dtype, seed=54)
    B.kc[:] = ((torch.arange(B.kc.numel(), device="cuda") % 255) - 127).to(torch.int8).view(B.kc.shape)
    B.vc[:] = ((torch.arange(B.vc.numel(), device="cuda") % 255) - 127).to(torch.int8).view(B.vc.shape)
    one = torch.tensor(np.float32(1) / np.float32(127), device="cuda")
    B.ks[:], B.vs[:] = one, one
    k, v = B.rand(2, 0.01), B.rand(2, 0.01)
    k[0, :, 5], k[1, :, 9] = top, -top
    v[0, :, 63], v[1, :, 0] = -top, top
    check_append(B, k, v)


def test_a_page_filled_token_by_token_stays_within_its_bound():
    """A value stored and then rescaled g times is off by at most half a step of the
    scale at each of the g + 1 roundings (steps never shrink): (g + 1) / 2 steps
    of the last one. The quotients and products round to fp32 before: up to 127
    units times 2 roundings of 2^-24 each."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(55)
    page, dim = 32, 64
    pool = ops().kv8_new_cache(1, 1, page, dim)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x = torch.randn(2, page, 1, dim, generator=g, device="cuda").clamp(-3, 3)
    x[:, :, 0, 7] = 3.0 + 0.02 * torch.arange(page, device="cuda")     # the maximum rises with every token
    x = x.half()
    for i in range(page):
        sl = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        ops().kv8_append(x[0, i:i + 1], x[1, i:i + 1], *pool, table, cu, sl, 1)
    every = torch.tensor([0, page], dtype=torch.int32, device="cuda")
    got = ops().kv8_gather(*pool, table, every, sl, page, page, out_dtype=torch.float32)
    roundings = page - torch.arange(page, device="cuda").double()
    for side, back, scale in zip(x, got, pool[2:]):
        off = (side.double() - back.double()).abs().amax(dim=(1, 2)) / scale[0, 0].double()
        assert bool((off <= roundings * (0.5 + 127 * 2 * 2.0 ** -24)).all())


@pytest.mark.parametrize("M,N,K", [(1, 130, 256), (7, 8200, 1024), (12, 300, 4112), (33, 100, 4096), (64, 130, 8192),
                                   (130, 256, 512), (300, 520, 1024), (2048, 512, 256)])
def test_bias_is_added_to_the_rounded_product(M, N, K):
    """fl32(fl32(fl32(P) fl32(xs ws)) + bias), bit for bit: the streaming kernel, the
    tiles with element and with wide stores, the join of K ranges."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(56)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    s, t = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    b = torch.randn(N, generator=g, device="cuda") * 100
    p = (q.double() @ w.double().t()).cpu().numpy()                   # exact: below 2^53
    sc = s.cpu().numpy()[:, None] * t.cpu().numpy()[None, :]
    want = p.astype(np.float32) * sc + b.cpu().numpy()[None, :]
    assert want.dtype == np.float32
    y = ops().w8a8_gemm(q, s, w, t, bias=b)
    assert np.array_equal(y.cpu().numpy(), want)
    zero = torch.zeros_like(b)
    assert np.array_equal(ops().w8a8_gemm(q, s, w, t, bias=zero).cpu().numpy(), p.astype(np.float32) * sc)


# ------------------------------------------------------------- large scores

@pytest.mark.parametrize("dtype,ks,exp", [("float16", 1817 / 127, 0), ("float16", 40.0, 0), ("float16", 1e4, 0),
                                          ("bfloat16", 40.0, 0), ("bfloat16", 300.0, 40)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_one_key_far_above_the_others(kernel, dtype, ks, exp):
    """Scores of 3e7 and more, where a rounding of one moves its weight by whole
    powers of two: one key of a head is above the others by half its score and
    takes all the weight. The output is that key's values: its weight is rounded to
    11 bits, and a page's scale may pass through its log2 (below 16, so steps of
    2^-20: three of them, and the sums)."""
    import torch
    new, lens, heads = KERNELS[kernel]
    for page in (64, 16):
        B = Batch(new, lens, 2, 128, page, dtype, seed=57)
        B.kc[:] = torch.randint(-40, 41, B.kc.shape, generator=B.g, device="cuda", dtype=torch.int8)
        B.ks[:] = ks
        best = [[70, 141], [3, 400]]
        t = B.cu_host[-1]
        q = (torch.rand(B.total, heads, 128, generator=B.g, device="cuda") * 800 + 1000).to(B.dtype) * 2.0 ** exp
        want = torch.zeros((t, heads, 128), dtype=torch.float64, device="cuda")
        top = torch.zeros((t, heads), dtype=torch.float64, device="cuda")
        for b in range(2):
            rows = slice(B.cu_host[b], B.cu_host[b + 1])
            for h in range(2):
                at = best[b][h]
                B.kc[int(B.table_host[b, at // page]), h, at % page] = 127
                v = B.values(b, torch.float64)[1][h, at]
                want[rows, 4 * h:4 * h + 4] = v
                top[rows, 4 * h:4 * h + 4] = 127 * float(B.ks[0, 0]) * 128 ** -0.5 * q[rows, 4 * h:4 * h + 4].double().sum(-1)
        y, lse = attend(B, q, out_dtype=torch.float32)
        y, lse = y[:t].double(), lse[:t].double()
        assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(lse).all())
        assert bool(((y - want).abs() <= (2.0 ** -11 + 2.0 ** -18) * want.abs()).all())
        # 128 products of one sign summed in fp32, the factors' roundings
        assert bool(((lse - top).abs() <= (128 + 16) * 2.0 ** -24 * top).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_large_scores_that_rise_by_little(kernel):
    """Scores of 6e7 (in units of ln 2) that rise by 2 of their roundings from one
    chunk of positions to the next: whatever the weights are, they are weights:
    outputs lie between the values."""
    import torch
    new, lens, heads = KERNELS[kernel]
    for q0 in (1024.0, 1023.0, 1020.0, 1001.0):
        B = Batch(new, lens, 2, 128, 64, seed=58)
        B.kc[:] = 0
        B.ks[:] = 1.0
        for b, length in enumerate(lens):
            for j in range(-(-length // 64)):
                page = int(B.table_host[b, j])
                B.kc[page, :, :, 0] = 127
                B.kc[page, :, :, 1] = j
        q = torch.zeros(B.total, heads, 128, dtype=torch.float16, device="cuda")
        q[..., 0], q[..., 1] = q0, 2.0 ** -6
        t = B.cu_host[-1]
        for scale in (512 * math.log(2), -512 * math.log(2)):
            y, lse = attend(B, q if scale > 0 else -q, scale=scale, out_dtype=torch.float32)
            assert bool(torch.isfinite(y[:t]).all()) and bool(torch.isfinite(lse[:t]).all())
            for b in range(len(lens)):
                rows = slice(B.cu_host[b], B.cu_host[b + 1])
                big = B.values(b, torch.float64)[1].abs().amax(dim=1).repeat_interleave(heads // 2, 0)
                # weights rounded to 11 bits, their sum to fp32
                assert bool((y[rows].double().abs() <= big[None] * (1 + 2.0 ** -10)).all())


# ------------------------------------------------------- small value scales

@pytest.mark.parametrize("exp", [-100, -112, -118, -121, -126, -130])
@pytest.mark.parametrize("kernel", KERNELS)
def test_values_down_to_subnormal_scales(kernel, exp):
    """Every value scale in [2^exp, 2^(exp + 1)): the outputs keep their relative
    precision (the bound of attention_ref, whose absolute term is a share of the
    largest page scale, 2^-120 at least), the log-sum-exp does not depend on them."""
    import torch
    new, lens, heads = KERNELS[kernel]
    for page in (64, 16):
        B = Batch(new, lens, 2, 128, page, seed=59)
        B.vs = torch.ldexp(1 + torch.rand(B.vs.shape, generator=B.g, device="cuda"), torch.tensor(exp, device="cuda"))
        q = B.rand(heads)
        t = B.cu_host[-1]
        o, want, bound = attention_ref(B, q, True, 0, 128 ** -0.5)
        y, lse = attend(B, q, out_dtype=torch.float32)
        assert bool(((lse[:t].double() - want[:t]).abs() <= 2.0 ** -10).all())
        # the output's step, 2^-24 or half a subnormal one, and that of a subnormal factor of the largest scale
        tiny = max(lens) * 127 * 2.0 ** -34 * 2.0 ** -120 + 2.0 ** -150
        err = (y.double() - o).abs()[:t]
        assert bool((err <= (bound + (2.0 ** -24 + 2.0 ** -14) * o.abs())[:t] + tiny).all()), float((err / o.abs()[:t]).max())


# -------------------------------------------------- inputs that are not finite

BAD = [float("nan"), -float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("M,N,K", [(3, 40, 512), (5, 40, 4096), (9, 8200, 1024), (4, 40, 40000), (40, 40, 8192), (2, 20, 20000)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_a_token_that_is_not_finite_gives_nan(M, N, K, dtype):
    """A NaN or an infinity in a token, beside its largest finite values: the token's
    outputs are NaN, the other tokens' are as without it."""
    import torch
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(60)
    x = torch.randn(M, K, generator=g, device="cuda").to(getattr(torch, dtype))
    wq, ws = o.w8a8_pack_weight(torch.randn(N, K, generator=g, device="cuda").half())
    clean, s0 = o.w8a8_linear(x, wq, ws), o.w8a8_quantize_act(x)[1]
    for i, bad in enumerate(BAD):
        for at in (0, 5, K // 2 + 3, K - 1):
            z = x.clone()
            row = (at + i) % M
            z[row, at // 16 * 16:at // 16 * 16 + 16] = 1000.0
            z[row, at] = bad
            keep = torch.arange(M, device="cuda") != row
            q, s = o.w8a8_quantize_act(z)
            assert bool(torch.isnan(s[row])) and torch.equal(s[keep], s0[keep])
            for y in (o.w8a8_linear(z, wq, ws), o.w8a8_gemm(q, s, wq, ws)):
                assert bool(torch.isnan(y[row]).all()) and torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_a_page_that_is_not_finite_says_so(bad, dtype):
    """The scale of the page and head that a NaN or an infinity is stored in becomes
    NaN, and stays so while the page is filled; the others are as without it; the
    page starts afresh when it is used again. Queries that see it get NaN."""
    import torch
    o = ops()
    B = Batch([20, 3], [37, 40], 2, 64, 16, dtype, seed=61)
    k, v = B.rand(2), B.rand(2)
    kc, vc, ks, vs = (x.clone() for x in B.pool[:4])
    o.kv8_append(k, v, kc, vc, ks, vs, *B.pool[4:], B.max_new)
    bk, bv = k.clone(), v.clone()
    bk[4, 1, 7], bv[15, 0, 60] = bad, bad                # positions 21 and 32 of sequence 0: pages 1 and 2
    pk, pv = int(B.table_host[0, 1]), int(B.table_host[0, 2])
    o.kv8_append(bk, bv, *B.pool, B.max_new)
    assert bool(torch.isnan(B.ks[pk, 1])) and bool(torch.isnan(B.vs[pv, 0]))
    for a, b, at in ((B.ks, ks, (pk, 1)), (B.vs, vs, (pv, 0)), (B.kc, kc, (pk, 1)), (B.vc, vc, (pv, 0))):
        a, b = a.clone(), b.clone()
        a[at], b[at] = 0, 0
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    last = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for heads, cu, n in ((4, B.cu, 20), (16, B.cu, 20), (4, last, 1)):    # 40, 160 and 2 query rows per kv head
        q, g = B.rand(heads), heads // 2
        y, lse = o.kv8_attention(q, *B.pool[:5], cu, B.sl, n, B.max_len, causal=False, return_lse=True)
        clean, clean_lse = o.kv8_attention(q, kc, vc, ks, vs, B.table, cu, B.sl, n, B.max_len, causal=False, return_lse=True)
        assert bool(torch.isnan(y[:n]).all()), "values of its first kv head, keys of its second"
        assert torch.equal(lse[:n, :g], clean_lse[:n, :g]) and bool(torch.isnan(lse[:n, g:]).all())
        rest = slice(n, int(cu[2]))
        assert torch.equal(y[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    # 3 more tokens on the page: its scale still says so
    B.sl = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 3], dtype=torch.int32, device="cuda")
    o.kv8_append(k, v, *B.pool[:5], cu, B.sl, 3)
    assert bool(torch.isnan(B.vs[pv, 0]))
    # used again from its first position
    sl = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    table = B.table.clone()
    table[0, 0] = pv
    o.kv8_append(k, v, *B.pool[:4], table, torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda"), sl, 2)
    assert bool(torch.isfinite(B.vs[pv]).all()) and bool(torch.isfinite(B.ks[pv]).all())


# --------------------------------------------------------- small weights

@pytest.mark.parametrize("new,lens,heads", [([1, 3], [300, 900], 8), ([9, 5], [300, 517], 8), ([30, 8], [400, 100], 8),
                                            ([1], [5000], 16), ([7, 2], [900, 90], 4)])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_small_weights_of_few_rows(new, lens, heads, dim, page):
    """Up to 128 rows per kv head a weight in fp16's subnormal range is off by half
    its step, 2^-25, relative to 2^15 for the largest page scale: 2^-40 of it
    (many rows: 2^-34)."""
    import torch
    B = Batch(new, lens, 2, dim, page, seed=62)
    B.vs[::2] *= 2.0 ** -16                               # pages whose values are small beside the largest
    q = B.rand(heads, 6.0)
    o, _, bound = attention_ref(B, q, True, 0, dim ** -0.5)
    t = B.cu_host[-1]
    for b in range(len(lens)):
        pages = B.table[b, :-(-lens[b] // page)].long()
        top = max(float(torch.nan_to_num(B.vs[pages]).max()), 0.0)
        bound[B.cu_host[b]:B.cu_host[b + 1]] -= lens[b] * 127 * (2.0 ** -34 - 2.0 ** -40) * top
    y, _ = attend(B, q, out_dtype=torch.float32)
    assert bool(((y.double() - o).abs()[:t] <= (bound + 2.0 ** -24 * o.abs())[:t]).all())


@pytest.mark.parametrize("single", [5, 1])
def test_single_tokens_and_chunks_in_two_calls(single):
    """A mixed batch in one call, and its single tokens and chunks each in a call of
    their own that fills its rows of one output."""
    import torch
    B = Batch([1] * single + [90, 40], [300 + 7 * i for i in range(single)] + [200, 40], 2, 128, 64, seed=63)
    q = B.rand(8)
    o, _, bound = attention_ref(B, q, True, 0, 128 ** -0.5)
    t = B.cu_host[-1]
    out = torch.full_like(q, 7.0)
    for part, new in ((slice(0, single), 1), (slice(single, None), 90)):
        cu = B.cu[:single + 1] if new == 1 else B.cu[single:]
        ops().kv8_attention(q, *B.pool[:4], B.table[part], cu, B.sl[part], new, B.max_len, out=out)
    for y in (out, ops().kv8_attention(q, *B.pool, B.max_new, B.max_len)):
        assert bool(((y.double() - o).abs()[:t] <= (bound + 2.0 ** -11 * (o.abs() + bound) + 2.0 ** -25)[:t]).all())
    assert bool((out[t:] == 7).all())

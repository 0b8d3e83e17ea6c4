"""The 8-bit operators at the ends of the range of their inputs."""
import math

import pytest

from test_gpu_kv8 import Batch, attention_ref

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

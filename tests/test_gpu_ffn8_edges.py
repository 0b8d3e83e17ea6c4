"""Edges of what surrounds the W8A8 products: scales of a few subnormal units, rows of
2^20 values and more, zeros' signs, GELU's tail, launches whose last tokens go apart.

Tolerances as in test_gpu_ffn8.py (u = 2^-24), whose references are used here."""
import math

import numpy as np
import pytest

from test_gpu_ffn8 import U, act_case, assert_within, check_epilogue, gen, half_of, norm_ref, ops

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

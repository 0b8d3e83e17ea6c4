"""Argument validation of what surrounds the W8A8 products (CPU only): statuses of the
C ABI, which returns before any HIP call, and the tensor wrappers' refusals."""
import pytest
import torch

from w4a4_quantized_gemm_quantize_amd import _lib, ops

OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE = 0, 1, 2, 4, 5
F32, F16, BF16 = 0, 1, 2
P = 0x10000          # a fake, aligned "device pointer"


def test_rmsnorm_validation():
    def f(x=P, dt=F16, ldx=64, r=None, ldr=0, w=P, wdt=F32, eps=1e-6, M=4, K=64, q=P, s=P, h=None, ldh=0, y=None, ldy=0):
        return _lib.status_of("w8a8_rmsnorm_quantize", x, dt, ldx, r, ldr, w, wdt, eps, M, K, q, s, h, ldh, y, ldy, None)
    assert f(dt=F32) == E_DTYPE and f(wdt=BF16) == E_DTYPE and f(dt=BF16, wdt=F16) == E_DTYPE
    assert f(M=-1) == E_SHAPE and f(M=1 << 24) == E_SHAPE and f(K=0) == E_SHAPE and f(K=72, ldx=72) == E_SHAPE
    assert f(ldx=56) == E_SHAPE and f(ldx=68) == E_ALIGN
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == E_SHAPE
    res = dict(r=P, ldr=64, h=P, ldh=64)
    assert f(**dict(res, ldr=56)) == E_SHAPE and f(**dict(res, ldh=56)) == E_SHAPE
    assert f(**dict(res, ldr=68)) == E_ALIGN and f(**dict(res, ldh=68)) == E_ALIGN
    assert f(**dict(res, h=None)) == E_NULL and f(**dict(res, h=P + 8)) == E_ALIGN and f(**dict(res, r=P + 2)) == E_ALIGN
    assert f(y=P, ldy=56) == E_SHAPE and f(y=P, ldy=68) == E_ALIGN and f(y=P + 2, ldy=64) == E_ALIGN
    assert f(x=None) == E_NULL and f(w=None) == E_NULL and f(q=None) == E_NULL and f(s=None) == E_NULL
    assert f(x=P + 8) == E_ALIGN and f(w=P + 4) == E_ALIGN and f(q=P + 8) == E_ALIGN and f(s=P + 2) == E_ALIGN
    assert f(x=None, w=None, q=None, s=None, M=0) == OK


def gemm_act(xq=P, xs=P, wq=P, ws=P, bias=None, act=0, gated=0, res=None, ldr=0, M=32, N=8, K=64, wsp=P, wb=1 << 30, y=P,
             dt=F16, ldy=8):
    return _lib.status_of("w8a8_gemm_act", xq, xs, wq, ws, bias, act, gated, res, ldr, M, N, K, wsp, wb, y, dt, ldy, None)


def linear_act(x=P, xdt=F16, M=32, K=64, ldx=64, wq=P, ws=P, bias=None, act=0, gated=0, res=None, ldr=0, N=8, wsp=P,
               wb=1 << 30, y=P, dt=F16, ldy=8):
    return _lib.status_of("w8a8_linear_act", x, xdt, M, K, ldx, wq, ws, bias, act, gated, res, ldr, N, wsp, wb, y, dt, ldy,
                          None)


def test_act_validation():
    for f in (gemm_act, linear_act):
        assert f(K=72) == E_SHAPE and f(K=131072) == E_SHAPE and f(M=-1) == E_SHAPE and f(N=-1) == E_SHAPE
        assert f(M=1 << 24) == E_SHAPE and f(N=1 << 24, ldy=1 << 24) == E_SHAPE
        assert f(N=1 << 22, ldy=1 << 22) == E_SHAPE and f(N=1 << 21, ldy=1 << 21, gated=1) == E_SHAPE    # 2^22 channels
        assert f(act=5) == E_SHAPE and f(act=-1) == E_SHAPE
        assert f(dt=F32) == E_DTYPE and f(dt=9) == E_DTYPE
        assert f(ldy=7) == E_SHAPE and f(res=P, ldr=7) == E_SHAPE
        assert f(wq=None) == E_NULL and f(ws=None) == E_NULL and f(y=None) == E_NULL
        assert f(wq=P + 8) == E_ALIGN and f(bias=P + 2) == E_ALIGN and f(y=P + 1) == E_ALIGN
        assert f(res=P + 1, ldr=8) == E_ALIGN and f(wsp=P + 8) == E_ALIGN
        assert f(M=0) == OK and f(N=0) == OK
    assert gemm_act(xq=None) == E_NULL and gemm_act(xs=None) == E_NULL and gemm_act(xq=P + 8) == E_ALIGN
    assert linear_act(x=None) == E_NULL and linear_act(xdt=F32) == E_DTYPE and linear_act(ldx=68) == E_ALIGN
    assert linear_act(ldx=56) == E_SHAPE and linear_act(x=P + 8) == E_ALIGN


def test_act_workspace():
    gemm, lin = _lib.load_library().w8a8_gemm_act_workspace, _lib.load_library().w8a8_linear_act_workspace
    assert gemm(4, 8, 72, 0, 1) == -1 and lin(4, 8, 72, 0, 1) == -1 and gemm(0, 8, 64, 0, 1) == 0
    assert gemm(300, 1000, 336, 0, 1) == 0                               # tiles write the outputs
    assert gemm(300, 1000, 336, 0, 0) == 300 * 1000 * 4                  # other rows: int32 sums first
    assert gemm(300, 1001, 336, 0, 1) == 300 * 1004 * 4                  # in rows of whole 16-byte stores
    assert gemm(300, 1001, 336, 1, 1) == 300 * 2004 * 4
    for M, N, K in [(64, 8192, 8192), (4096, 4096, 4096), (17, 100, 1040), (512, 4096, 11008)]:
        for gated in (0, 1):
            assert gemm(M, N, K, gated, 0) >= gemm(M, N, K, gated, 1)
            assert lin(M, N, K, gated, 1) >= M * K + 4 * M + gemm(M, N, K, gated, 1)
    assert lin(1, 4096, 4096, 1, 1) == 0                                 # one launch
    need = gemm(64, 8192, 8192, 0, 1)
    assert need > 0
    big = dict(M=64, N=8192, K=8192, ldy=8192)
    assert gemm_act(**big, wb=need - 1) == E_SHAPE and gemm_act(**big, wsp=None, wb=need) == E_NULL
    assert linear_act(**big, ldx=8192, wb=need) == E_SHAPE


def test_route_validation():
    def f(x=P, dt=F32, T=4, E=64, ld=64, k=8, ids=P, w=P):
        return _lib.status_of("moe_route", x, dt, T, E, ld, k, 1, ids, w, None)
    assert f(dt=3) == E_DTYPE and f(T=-1) == E_SHAPE and f(T=1 << 24) == E_SHAPE
    assert f(E=0) == E_SHAPE and f(E=513, ld=513) == E_SHAPE and f(ld=63) == E_SHAPE
    assert f(k=0) == E_SHAPE and f(k=65) == E_SHAPE
    assert f(x=None) == E_NULL and f(ids=None) == E_NULL and f(w=None) == E_NULL
    assert f(x=P + 2) == E_ALIGN and f(x=P + 1, dt=F16) == E_ALIGN and f(ids=P + 2) == E_ALIGN and f(w=P + 1) == E_ALIGN
    assert f(x=None, ids=None, w=None, T=0) == OK


def test_moe_validation():
    def f(xq=P, xs=P, ids=P, w=P, T=4, k=2, w13=P, s13=P, w2=P, s2=P, E=8, H=64, I=32, act=2, wsp=P, wb=1 << 30, y=P,
          dt=F16, ldy=64):
        return _lib.status_of("w8a8_moe", xq, xs, ids, w, T, k, w13, s13, w2, s2, E, H, I, act, wsp, wb, y, dt, ldy, None)
    assert f(T=-1) == E_SHAPE and f(T=257) == E_SHAPE and f(k=0) == E_SHAPE and f(T=1, k=513) == E_SHAPE
    assert f(T=1 << 62, k=8) == E_SHAPE                                  # no overflow on the way
    assert f(E=0) == E_SHAPE and f(E=513) == E_SHAPE
    assert f(H=72, ldy=72) == E_SHAPE and f(I=24) == E_SHAPE and f(H=131072, ldy=131072) == E_SHAPE and f(I=0) == E_SHAPE
    assert f(act=7) == E_SHAPE and f(dt=F32) == E_DTYPE and f(ldy=63) == E_SHAPE
    need = _lib.load_library().w8a8_moe_workspace(4, 2, 8, 64, 32)
    assert need >= 8 * 32 * 5 and f(wb=need - 1) == E_SHAPE
    assert _lib.load_library().w8a8_moe_workspace(4, 2, 8, 64, 24) == -1
    assert _lib.load_library().w8a8_moe_workspace(0, 2, 8, 64, 32) == 0
    for name in ("xq", "xs", "ids", "w", "w13", "s13", "w2", "s2", "y", "wsp"):
        assert f(**{name: None}) == E_NULL, name
    for name in ("xq", "w13", "w2", "wsp"):
        assert f(**{name: P + 8}) == E_ALIGN, name
    for name in ("xs", "ids", "w", "s13", "s2"):
        assert f(**{name: P + 2}) == E_ALIGN, name
    assert f(y=P + 1) == E_ALIGN
    assert f(xq=None, T=0) == OK


def test_wrappers_refuse_host_tensors_and_bad_names():
    x = torch.zeros((4, 64), dtype=torch.float16)
    q, s = x.to(torch.int8), torch.ones(4)
    with pytest.raises(TypeError):
        ops.w8a8_rmsnorm_quantize(x, torch.ones(64))
    with pytest.raises(TypeError):
        ops.w8a8_gemm_act(q, s, q, s)
    with pytest.raises(TypeError):
        ops.w8a8_linear_act(x, q, s)
    with pytest.raises(TypeError):
        ops.moe_route(x, 2)
    with pytest.raises(TypeError):
        ops.w8a8_moe(q, s, q.int(), x.float(), q[None], s[None], q[None], s[None])
    for bad in ("swish", 1, True, ""):
        with pytest.raises(ValueError):
            ops._activation(bad)
    with pytest.raises(ValueError):
        ops.w8a8_pack_gated(x, x[:2])


def test_overlap():
    t = torch.zeros((8, 64), dtype=torch.float16)
    assert ops._overlap(t, t) and ops._overlap(t[:4], t[3:])
    assert not ops._overlap(t[:4], t[4:]) and not ops._overlap(t[:0], t) and not ops._overlap(t[0:1, :32], t[0:1, 32:])


def test_overlap_of_columns_and_in_place():
    t = torch.zeros((8, 64), dtype=torch.float16)
    assert not ops._overlap(t[:, :32], t[:, 32:]) and not ops._overlap(t[:, 32:], t[:, :32])
    assert not ops._overlap(t[:6, 48:], t[2:, :48]) and not ops._overlap(t[1:7, :8], t[:, 56:])
    assert ops._overlap(t[:, :33], t[:, 32:]) and ops._overlap(t[:, 16:48], t[2:, :17])
    assert ops._overlap(t[1:, 60:], t[:7].view(-1)[56:].as_strided((7, 16), (64, 1)))      # round the row's end
    assert ops._overlap(t[:, :8], t.view(16, 32)[:, 16:])                                  # other strides: as ranges
    ops._in_place_or_apart(t, t, "a and b")
    ops._in_place_or_apart(t[:, :8], t[:, 8:16], "a and b")
    ops._in_place_or_apart(t[:1], t.view(16, 32)[:1], "a and b")
    for a, b in ((t[1:], t[:7]), (t[:, 1:9], t[:, :8]), (t[:4], t.view(16, 32)[:4])):
        with pytest.raises(ValueError):
            ops._in_place_or_apart(a, b, "a and b")


def test_public_names():
    import w4a4_quantized_gemm_quantize_amd as pkg
    for name in ("w8a8_rmsnorm_quantize", "w8a8_gemm_act", "w8a8_linear_act", "w8a8_pack_gated", "moe_route", "w8a8_moe"):
        assert getattr(pkg, name) is getattr(ops, name)


def test_rmsnorm_eps_is_a_normal_number():
    """Squares below fp32's normal range lose bits that only a larger eps hides."""
    f = lambda eps: _lib.status_of("w8a8_rmsnorm_quantize", P, F16, 64, None, 0, P, F32, eps, 0, 64, P, P, None, 0, None, 0,
                                   None)
    assert f(2.0 ** -126) == OK and f(1e-6) == OK
    for eps in (2.0 ** -127, 2.0 ** -149, 1e-40):
        assert f(eps) == E_SHAPE


def test_act_channels_whose_padded_sums_reach_2_31_bytes():
    """128 rows of 2^22 int32 sums are 2^31 bytes, more than a buffer resource spans: 2^22 - 3 channels pad to that."""
    gemm, lin = _lib.load_library().w8a8_gemm_act_workspace, _lib.load_library().w8a8_linear_act_workspace
    top = (1 << 22) - 4
    for N, gated in [(top + 1, 0), (top + 3, 0), ((top + 2) // 2, 1)]:
        assert gemm(32, N, 64, gated, 0) == -1 and lin(32, N, 64, gated, 0) == -1
        for f in (gemm_act, linear_act):
            assert f(N=N, ldy=N, gated=gated, wb=1 << 62) == E_SHAPE and f(M=0, N=N, ldy=N, gated=gated) == E_SHAPE
    for N, gated in [(top, 0), (top // 2, 1)]:
        assert gemm(32, N, 64, gated, 0) == 32 * top * 4
        for f in (gemm_act, linear_act):
            assert f(M=0, N=N, ldy=N, gated=gated) == OK


E_OVERLAP = 8
FAR = 1 << 20        # between the fake buffers below


def test_norm_outputs_that_meet_buffers():
    """Codes, scales, sums and normed rows apart from one another and from the inputs, whatever is absent."""
    M, K = 8, 64
    base = dict(x=P, ldx=64, r=P + FAR, ldr=64, w=P + 2 * FAR, q=P + 3 * FAR, s=P + 4 * FAR, h=P + 5 * FAR, ldh=64,
                y=P + 6 * FAR, ldy=64)

    def f(**k):
        a = dict(base, **k)
        return _lib.status_of("w8a8_rmsnorm_quantize", a["x"], F16, a["ldx"], a["r"], a["ldr"], a["w"], F32, 1e-6, M, K,
                              a["q"], a["s"], a["h"], a["ldh"], a["y"], a["ldy"], None)
    inputs = [base[n] for n in ("x", "r", "w")]
    for name in ("q", "s", "y"):
        for at in inputs + [base[n] for n in ("q", "s", "h", "y") if n != name]:
            assert f(**{name: at}) == E_OVERLAP, (name, at)
    assert f(q=P + 1008) == E_OVERLAP and f(q=P - 496) == E_OVERLAP and f(s=P + 1020) == E_OVERLAP     # by their ends
    assert f(h=P + 16) == E_OVERLAP and f(h=P + 2 * FAR) == E_OVERLAP and f(h=P + FAR + 128) == E_OVERLAP
    assert f(h=P, ldh=72) == E_OVERLAP                                          # x itself, at another stride
    assert f(r=None, h=None, q=P) == E_OVERLAP and f(r=None, h=None, y=None, s=P) == E_OVERLAP
    # columns of one buffer that touch by one
    assert f(ldx=200, r=P + 126, ldr=200, h=P + 240, ldh=200) == E_ALIGN and f(ldx=200, h=P + 112, ldh=200) == E_OVERLAP
    assert f(ldx=200, h=P + 384, ldh=200) == E_OVERLAP                          # round the row's end


def test_act_outputs_that_meet_buffers():
    for gated in (0, 1):
        C = 8 << gated
        for f, tokens in ((gemm_act, "xq"), (linear_act, "x")):
            base = {tokens: P, "wq": P + FAR, "ws": P + 2 * FAR, "bias": P + 3 * FAR, "res": P + 4 * FAR, "ldr": 8,
                    "wsp": P + 5 * FAR, "y": P + 6 * FAR, "gated": gated}
            if tokens == "xq":
                base["xs"] = P + 7 * FAR
            call = lambda **k: f(**dict(base, **k))
            for name in (tokens, "wq", "ws", "bias", *(["xs"] if tokens == "xq" else [])):
                assert call(y=base[name]) == E_OVERLAP, name
            assert call(y=P + FAR + C * 64 - 2) == E_OVERLAP and call(y=P + FAR - 2) == E_OVERLAP
            assert call(y=P + 4 * FAR + 16) == E_OVERLAP and call(y=P + 4 * FAR, ldy=16) == E_OVERLAP
            # the workspace, where there is one
            big = dict(M=64, N=8192 >> gated, K=8192, ldy=8192 >> gated, ldr=8192 >> gated)
            big = {n: big[n] for n in big} | ({"ldx": 8192} if tokens == "x" else {})
            far = {n: P + i * (1 << 34) for i, n in enumerate(n for n in base if n not in ("ldr", "gated"))}
            for name in far:
                if name != "wsp":
                    assert f(**dict(far, gated=gated, wsp=far[name], **big)) == E_OVERLAP, name


def test_route_and_moe_outputs_that_meet_buffers():
    def route(x=P, ids=P + FAR, w=P + 2 * FAR, ld=64):
        return _lib.status_of("moe_route", x, F32, 4, 64, ld, 8, 1, ids, w, None)
    assert route(ids=P) == E_OVERLAP and route(w=P + 1020) == E_OVERLAP and route(w=P + FAR + 124) == E_OVERLAP
    assert route(ids=P + 3 * 400 + 252, ld=100) == E_OVERLAP and route(ids=P - 4, ld=100) == E_OVERLAP
    T, k, E, H, I = 4, 2, 8, 64, 32
    names = ("xq", "xs", "ids", "w", "w13", "s13", "w2", "s2", "wsp", "y")
    base = {n: P + i * FAR for i, n in enumerate(names)}

    def moe(**a):
        a = dict(base, **a)
        return _lib.status_of("w8a8_moe", a["xq"], a["xs"], a["ids"], a["w"], T, k, a["w13"], a["s13"], a["w2"], a["s2"], E,
                              H, I, 2, a["wsp"], 1 << 30, a["y"], F16, 64, None)
    for name in ("ids", "w", "w2", "s2", "wsp"):
        assert moe(y=base[name]) == E_OVERLAP, name
    for name in names:
        if name != "wsp":
            assert moe(wsp=base[name]) == E_OVERLAP, name
    assert moe(y=base["w2"] + E * H * I - 2) == E_OVERLAP and moe(y=base["ids"] - 2) == E_OVERLAP
    assert _lib.load_library().w4a4_status_str(E_OVERLAP) != b"unknown status"

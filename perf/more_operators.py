"""The operators of an 8-bit feed-forward block as they are measured: the norm that
emits INT8 codes, products with an epilogue, the router, and the experts' layer.

``run`` computes a case with elementary torch operations in 32 bits
(``own`` false) or with this package's operators (``own`` true); ``exact`` gives
the same outputs from the definitions in 64 bits.

Four kinds of case:

* ``norm``: add the residual, RMS norm, INT8 codes with one scale per token.
* ``linear``: INT8 product of tokens quantized on the way, with bias, activation,
  gate and residual in its epilogue.
* ``route``: the k largest router logits of every token and their weights.
* ``moe``: a mixture-of-experts layer of few tokens on INT8 experts.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode token in front of the projections of the 7B-sized model: latency
        dict(name="norm 1x4096", kind="norm", M=1, K=4096, dtype="bf16", weight="bf16", residual=True, normed=False),
        # a ragged prompt in front of a router, which reads the normed tokens too
        dict(name="norm 777x3584, normed", kind="norm", M=777, K=3584, dtype="fp16", weight="fp32", residual=False,
             normed=True),
        # a full prefill chunk of the 70B-sized model, the residual stream updated on the way
        dict(name="norm 4096x8192", kind="norm", M=4096, K=8192, dtype="bf16", weight="bf16", residual=True,
             normed=False),
        # one decode token through gate and up projections of the 7B-sized model
        dict(name="linear 1x4096, gated 11008", kind="linear", M=1, K=4096, N=11008, dtype="fp16", act="silu",
             gated=True, bias=False, residual=False),
        # a small decode batch through its down projection, onto the residual stream
        dict(name="linear 16x11008x4096, residual", kind="linear", M=16, K=11008, N=4096, dtype="bf16", act="none",
             gated=False, bias=False, residual=True),
        # a ragged prompt through an up projection with bias and GELU
        dict(name="linear 777x3584x18944, gelu", kind="linear", M=777, K=3584, N=18944, dtype="bf16", act="gelu",
             gated=False, bias=True, residual=False),
        # a full prefill chunk through gate and up projections of the 70B-sized model: matrix bound
        dict(name="linear 4096x8192, gated 28672", kind="linear", M=4096, K=8192, N=28672, dtype="fp16", act="silu",
             gated=True, bias=False, residual=False),
        # the router of one decode token: latency
        dict(name="route 1x64, 8", kind="route", T=1, E=64, k=8, dtype="fp32", renorm=True),
        # the router of a prefill chunk over many experts
        dict(name="route 4096x256, 8", kind="route", T=4096, E=256, k=8, dtype="bf16", renorm=False),
        # one decode token through 8 of 64 small experts: latency, then the weights' stream
        dict(name="moe 1, 8 of 64", kind="moe", T=1, H=2048, I=1024, E=64, k=8, dtype="bf16", act="silu"),
        # a small decode batch over fewer, larger experts: most of them are read
        dict(name="moe 13, 4 of 32", kind="moe", T=13, H=3584, I=2368, E=32, k=4, dtype="fp16", act="gelu_tanh"),
        # a full decode batch: every expert is read, 8 tokens each
        dict(name="moe 64, 8 of 64", kind="moe", T=64, H=4096, I=1376, E=64, k=8, dtype="bf16", act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# no drawn case costs more than the largest listed ones
MAX_LINEAR = 2 * 4096 * 8192 * 2 * 28672
MAX_EXPERTS = 64 * 3 * 1376 * 4096


def draw(rng):
    kind = rng.choice(["norm", "linear", "linear", "route", "moe", "moe"])
    dtype = rng.choice(["fp16", "bf16"])
    if kind == "norm":
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 4096), K=16 * _log(rng, 4, 1792), dtype=dtype,
                     weight=rng.choice(["fp32", dtype]), residual=rng.random() < 0.6, normed=rng.random() < 0.3)
            if c["M"] * c["K"] <= 4096 * 8192:
                return c
    if kind == "linear":
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 4096), K=16 * _log(rng, 16, 1792), N=_log(rng, 64, 28672), dtype=dtype,
                     act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), gated=rng.random() < 0.4,
                     bias=rng.random() < 0.4, residual=rng.random() < 0.4)
            if rng.random() < 0.7:
                c["N"] = max(64, c["N"] // 64 * 64)    # widths of layers; the others are odd
            if work(c)["flops"] <= MAX_LINEAR:
                return c
    if kind == "route":
        E = _log(rng, 4, 512)
        return dict(kind=kind, T=_log(rng, 1, 4096), E=E, k=min(E, rng.choice([1, 2, 4, 6, 8, 10])),
                    dtype=rng.choice(["fp32", "fp16", "bf16"]), renorm=rng.random() < 0.5)
    while True:
        E = rng.choice([8, 16, 32, 60, 64, 128])
        c = dict(kind=kind, T=_log(rng, 1, 64), H=16 * _log(rng, 16, 448), I=16 * _log(rng, 8, 224), E=E,
                 k=min(E, rng.choice([1, 2, 4, 6, 8])), dtype=dtype, act=rng.choice(["silu", "gelu", "gelu_tanh"]))
        if 3 * E * c["H"] * c["I"] <= MAX_EXPERTS:
            return c


def work(case):
    kind = case["kind"]
    if kind == "norm":
        n = case["M"] * case["K"]
        per = 2 + 1 + (4 if case["residual"] else 0) + (2 if case["normed"] else 0)
        return {"bytes": per * n + 4 * case["M"] + DTYPES[case["weight"]].itemsize * case["K"], "flops": 8 * n}
    if kind == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        rows = 2 * N if case["gated"] else N
        return {"bytes": 2 * M * K + rows * K + 4 * rows + (4 * rows if case["bias"] else 0) +
                (4 if case["residual"] else 2) * M * N, "flops": 2 * M * rows * K}
    T, E, k = case["T"], case["E"], case["k"]
    if kind == "route":
        return {"bytes": DTYPES[case["dtype"]].itemsize * T * E + 8 * T * k, "flops": 4 * T * E}
    H, I = case["H"], case["I"]
    used = E * (1 - (1 - k / E) ** T)                  # experts that at least one token chose
    return {"bytes": used * (3 * H * I + 4 * (2 * I + H)) + T * H + 4 * T + 8 * T * k + 2 * T * H,
            "flops": 6 * T * k * H * I}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, M, K):
    """Heavy-tailed activations with 1 % outlier channels, as in front of a linear layer."""
    x = 0.5 * _randn(g, M, K)
    x /= torch.sqrt((_randn(g, M, K) ** 2 + _randn(g, M, K) ** 2 + _randn(g, M, K) ** 2) / 3).clamp_min(1e-3)
    x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 30
    return x.clamp(-60000, 60000)


def _codes(g, *shape):
    """Weight codes of normal values whose largest is near 127."""
    return (36.0 * _randn(g, *shape)).round_().clamp_(-127, 127).to(torch.int8)


def _quantize_rows(x):
    """Symmetric INT8 codes and one scale per row of a float32 tensor."""
    s = x.abs().amax(dim=-1, keepdim=True) / 127
    q = torch.where(s > 0, torch.round(x / s), torch.zeros_like(s))
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    dt = DTYPES[case["dtype"]]
    if kind == "norm":
        M, K = case["M"], case["K"]
        x = _activations(g, M, K)
        weight = (1.0 + 0.3 * _randn(g, K)).to(DTYPES[case["weight"]])
        residual = (3.0 * _randn(g, M, K)).to(dt) if case["residual"] else None
        return dict(case=case, x=x.to(dt), weight=weight, residual=residual)
    if kind == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        rows = 2 * N if case["gated"] else N
        # scales of weights near 0.02 whose codes are spread as above; gated: rows 2n gate, 2n + 1 up
        return dict(case=case, x=_activations(g, M, K).to(dt), wq=_codes(g, rows, K),
                    ws=0.02 / 36 * torch.exp(0.1 * _randn(g, rows)),
                    bias=0.5 * _randn(g, rows) if case["bias"] else None,
                    residual=(3.0 * _randn(g, M, N)).to(dt) if case["residual"] else None)
    T, E, k = case["T"], case["E"], case["k"]
    # some experts are liked more than others
    logits = _randn(g, T, E) + 0.5 * _randn(g, E)
    if kind == "route":
        return dict(case=case, logits=logits.to(dt))
    H, I = case["H"], case["I"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    xq, xs = _quantize_rows(_activations(g, T, H))
    return dict(case=case, xq=xq.to(torch.int8), xs=xs[:, 0].contiguous(), ids=ids[:, :k].int().contiguous(),
                weights=torch.softmax(top[:, :k], dim=1).contiguous(),
                w13=_codes(g, E, 2 * I, H), s13=0.02 / 36 * torch.exp(0.1 * _randn(g, E, 2 * I)),
                w2=_codes(g, E, H, I), s2=0.02 / 36 * torch.exp(0.1 * _randn(g, E, H)))


# ----------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(state["case"], state)
    return {"norm": _norm, "linear": _linear, "route": _route, "moe": _moe}[kind](state["case"], state)


def _run_own(case, state):
    from w4a4_quantized_gemm_quantize_amd import ops
    kind = case["kind"]
    act = case.get("act")
    act = None if act == "none" else act
    if kind == "norm":
        got = ops.w8a8_rmsnorm_quantize(state["x"], state["weight"], eps=1e-6, residual=state["residual"],
                                        return_normed=case["normed"])
        return _norm_outputs(case, state, *got)
    if kind == "linear":
        return ops.w8a8_linear_act(state["x"], state["wq"], state["ws"], bias=state["bias"], activation=act,
                                   gated=case["gated"], residual=state["residual"], out_dtype=DTYPES[case["dtype"]])
    if kind == "route":
        ids, weights = ops.moe_route(state["logits"], case["k"], renormalize=case["renorm"])
        return {"ids": ids, "weights": weights}
    return ops.w8a8_moe(state["xq"], state["xs"], state["ids"], state["weights"], state["w13"], state["s13"],
                        state["w2"], state["s2"], activation=act, out_dtype=DTYPES[case["dtype"]])


def _norm_outputs(case, state, q, s, *more):
    """The codes as the values they stand for, in one operation; then the scales, the
    residual stream and the normed tokens, where the case has them."""
    out = {"x": torch.mul(q, s[:, None], out=torch.empty_like(state["x"])), "scale": s}
    out.update(zip([n for n in ("residual", "normed") if (case[n] if n == "normed" else state[n] is not None)], more))
    return out


def _norm(case, state):
    x, r = state["x"], state["residual"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    t = h.float() * state["weight"].float()
    rstd = torch.rsqrt(h.float().square().mean(dim=1, keepdim=True) + 1e-6)
    q, _ = _quantize_rows(t)
    s = t.abs().amax(dim=1) * rstd[:, 0] / 127
    more = ([] if r is None else [h]) + ([(t * rstd).to(x.dtype)] if case["normed"] else [])
    return _norm_outputs(case, state, q, s, *more)


def _act(v, name):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def _gated(v, name):
    """act(gate) * up of interleaved channels."""
    return _act(v[..., 0::2], name) * v[..., 1::2]


def _linear(case, state):
    q, s = _quantize_rows(state["x"].float())
    v = (q @ state["wq"].float().t()) * (s * state["ws"])
    if state["bias"] is not None:
        v = v + state["bias"]
    y = _gated(v, case["act"]) if case["gated"] else _act(v, case["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(DTYPES[case["dtype"]])


def _route(case, state):
    x = state["logits"].float()
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)
    v, ids = v[:, :case["k"]], ids[:, :case["k"]]
    e = torch.exp(v - v[:, :1])
    total = e.sum(dim=1, keepdim=True) if case["renorm"] else torch.exp(x - v[:, :1]).sum(dim=1, keepdim=True)
    return {"ids": ids.int(), "weights": e / total}


def _moe(case, state):
    # every expert that some token chose, on every token; then each token's share of it
    used = torch.unique(state["ids"])
    U, T, I = used.numel(), case["T"], case["I"]
    share = torch.where(state["ids"][:, :, None] == used, state["weights"][:, :, None], 0.0).sum(dim=1)     # [T, U]
    v = torch.matmul(state["xq"].float(), state["w13"][used].float().transpose(1, 2))                       # [U, T, 2 I]
    v = v * state["xs"][None, :, None] * state["s13"][used][:, None, :]
    hq, hs = _quantize_rows(_gated(v, case["act"]))
    y = torch.matmul(hq, state["w2"][used].float().transpose(1, 2)) * hs * state["s2"][used][:, None, :]    # [U, T, H]
    return (y * share.t()[:, :, None]).sum(dim=0).to(DTYPES[case["dtype"]])


# -------------------------------------------------- the definitions in 64 bits

def _activation64(v, name):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
    return v


def _codes64(x):
    """INT8 codes of rows, and the row's scale."""
    s = x.abs().max(dim=-1, keepdim=True).values / 127
    return torch.where(s > 0, x / s, torch.zeros_like(x)).round(), s


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        h, r = state["x"], state["residual"]
        out = {}
        if r is not None:
            h = (h.double() + r.double()).float().to(h.dtype)       # the stored stream is rounded by definition
            out["residual"] = h.double()
        y = h.double() * state["weight"].double()
        y /= torch.sqrt((h.double() ** 2).sum(dim=1, keepdim=True) / case["K"] + 1e-6)
        q, s = _codes64(y)
        out["x"], out["scale"] = q * s, s[:, 0]
        if case["normed"]:
            out["normed"] = y
        return out
    if kind == "linear":
        q, s = _codes64(state["x"].double())
        N = state["wq"].shape[0]
        y = torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
        for n in range(0, N, 8192):                                 # channels by the block: float64 weights
            v = (q @ state["wq"][n:n + 8192].double().t()) * s * state["ws"][n:n + 8192].double()
            if state["bias"] is not None:
                v += state["bias"][n:n + 8192].double()
            if case["gated"]:
                y[:, n // 2:n // 2 + 4096] = _activation64(v[:, 0::2], case["act"]) * v[:, 1::2]
            else:
                y[:, n:n + 8192] = _activation64(v, case["act"])
        return y if state["residual"] is None else y + state["residual"].double()
    if kind == "route":
        x = state["logits"].double()
        # position of an expert in its token's order: those above it, and equal ones before it
        at = torch.arange(case["E"], device="cuda")
        p = torch.softmax(x, dim=1)
        ids = torch.empty((case["T"], case["k"]), dtype=torch.int32, device="cuda")
        for t in range(0, case["T"], 256):
            a = x[t:t + 256]
            ahead = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) & (at[None, :] < at[:, None]))
            rank = ahead.sum(dim=2)
            ids[t:t + 256] = torch.argsort(rank, dim=1)[:, :case["k"]].int()
        w = torch.gather(p, 1, ids.long())
        return {"ids": ids, "weights": w / w.sum(dim=1, keepdim=True) if case["renorm"] else w}
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    x = state["xq"].double() * state["xs"].double()[:, None]
    ids = state["ids"].cpu()
    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            t, j = t.cuda(), j.cuda()
            w13 = state["w13"][e].double() * state["s13"][e].double()[:, None]
            gate, up = x[t] @ w13[0::2].t(), x[t] @ w13[1::2].t()
            q, s = _codes64(_activation64(gate, case["act"]) * up)
            part = (q @ state["w2"][e].double().t()) * s * state["s2"][e].double()
            y.index_add_(0, t, part * state["weights"][t, j].double()[:, None])
    return y

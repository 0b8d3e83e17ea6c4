"""The 8-bit operators as they are measured: W8A8 linear layers, and attention
over an INT8 key/value cache with one scale per page of tokens and kv head.

``run`` computes a case with elementary torch operations in 32 bits
(``own`` false) or with this package's operators (``own`` true); ``exact`` gives
the same outputs from the definitions in 64 bits.

Three kinds of case:

* ``linear``: quantize X[M, K] per token, multiply with INT8 weights that carry
  one scale per output channel, scale, add a bias if there is one.
* ``append``: quantize new keys and values into the pages of a cache, then read
  the touched pages back as values.
* ``attention``: queries of ragged sequences against their cached pages.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode token through the up projection of the 7B-sized model: latency
        dict(name="linear 1x4096x11008", kind="linear", M=1, K=4096, N=11008, dtype="fp16", out="fp16", bias=False),
        # a small decode batch through the down projection of the 70B-sized model: one read of the weights
        dict(name="linear 16x28672x8192", kind="linear", M=16, K=28672, N=8192, dtype="bf16", out="bf16", bias=False),
        # a short ragged prompt through a down projection with a bias: few tiles, long reduction
        dict(name="linear 777x18944x3584", kind="linear", M=777, K=18944, N=3584, dtype="bf16", out="bf16", bias=True),
        # a full prefill chunk through the up projection of the 70B-sized model: matrix bound
        dict(name="linear 4096x8192x28672", kind="linear", M=4096, K=8192, N=28672, dtype="fp16", out="fp16",
             bias=False),
        # one decode step of 64 sequences: one new token each, in pages that may have to be rescaled
        dict(name="append 64 sequences, 1 token", kind="append", batch=64, new=1, even=True, ctx=2048, heads_kv=8,
             dim=128, page=64, dtype="fp16"),
        # four draft tokens for each of 33 sequences, small pages and heads
        dict(name="append 33 sequences, 4 tokens", kind="append", batch=33, new=4, even=True, ctx=700, heads_kv=5,
             dim=64, page=16, dtype="bf16"),
        # ragged prompts being stored after the prefill
        dict(name="append 24 prompts up to 1500", kind="append", batch=24, new=1500, even=False, ctx=0, heads_kv=8,
             dim=128, page=64, dtype="bf16"),
        # the first tokens of one chat, every head with its own keys: latency
        dict(name="decode 1 of 257", kind="attention", batch=1, new=1, even=True, ctx=256, even_ctx=True, heads=32,
             heads_kv=32, dim=128, page=64, dtype="fp16", causal=True, window=0),
        # a serving batch: 64 ragged sequences, 8 query heads to a kv head
        dict(name="decode 64 up to 4096", kind="attention", batch=64, new=1, even=True, ctx=4095, even_ctx=False,
             heads=64, heads_kv=8, dim=128, page=64, dtype="fp16", causal=True, window=0),
        # one very long context
        dict(name="decode 1 of 131072", kind="attention", batch=1, new=1, even=True, ctx=131071, even_ctx=True,
             heads=64, heads_kv=8, dim=128, page=128, dtype="bf16", causal=True, window=0),
        # speculative decoding with a sliding window: 5 tokens a sequence, 7 query heads to a kv head
        dict(name="verify 24 x 5 of 6000, window 1024", kind="attention", batch=24, new=5, even=True, ctx=6000,
             even_ctx=False, heads=28, heads_kv=4, dim=128, page=32, dtype="bf16", causal=True, window=1024),
        # chunked prefill: ragged chunks of four prompts on top of what is cached already
        dict(name="prefill 4 chunks up to 4096", kind="attention", batch=4, new=4096, even=False, ctx=4096,
             even_ctx=False, heads=64, heads_kv=8, dim=128, page=64, dtype="fp16", causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# no drawn case costs more than the largest listed ones
MAX_LINEAR = 2 * 4096 * 8192 * 28672
MAX_ATTENTION = 4 * 128 * 64 * 4 * 4096 * 4096 // 2


def draw(rng):
    kind = rng.choice(["linear", "append", "attention", "attention"])
    if kind == "linear":
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 4096), K=16 * _log(rng, 16, 1792), N=_log(rng, 64, 28672),
                     dtype=rng.choice(["fp16", "bf16"]), out=rng.choice(["fp16", "bf16", "fp32"]),
                     bias=rng.random() < 0.5)
            if work(c)["flops"] <= MAX_LINEAR:
                return c
    heads_kv = rng.choice([1, 2, 4, 5, 8])
    c = dict(kind=kind, batch=_log(rng, 1, 64), dim=rng.choice([64, 128, 128, 192, 256]),
             page=rng.choice([16, 32, 64, 128]), heads_kv=heads_kv, dtype=rng.choice(["fp16", "bf16"]))
    if kind == "append":
        c.update(new=_log(rng, 1, 1024), even=rng.random() < 0.5, ctx=_log(rng, 1, 2048) - 1)
        return c
    c.update(heads=heads_kv * rng.choice([1, 3, 4, 7, 8, 16]), even=rng.random() < 0.5, even_ctx=rng.random() < 0.3,
             causal=rng.random() < 0.85, window=0)
    # decode steps, drafts and prompts in equal parts
    c["new"] = rng.choice([1, rng.randint(2, 8), _log(rng, 16, 2048)])
    c["ctx"] = _log(rng, 1, 65536 if c["new"] <= 8 else 8192) - 1
    if c["causal"] and rng.random() < 0.3:
        c["window"] = _log(rng, 16, 4096)
    while work(c)["flops"] > MAX_ATTENTION or _cache_bytes(c) > 1 << 30:
        c["batch"] = (c["batch"] + 1) // 2
        c["ctx"] //= 2
        c["new"] = (c["new"] + 1) // 2
    return c


def _lens(case):
    """(new tokens, cached length after them) of every sequence: from the case
    alone. Ragged batches hold a sequence of the largest size, and where there
    are several, one with nothing new."""
    rng = random.Random(case["batch"] * 1000003 + case["new"] * 1009 + case["ctx"])
    out = []
    for b in range(case["batch"]):
        n = case["new"]
        if not case["even"] and b:
            n = rng.randint(0, case["new"]) if b > 1 else 0
        c = case["ctx"]
        if not case.get("even_ctx", False) and b:
            c = rng.randint(0, case["ctx"])
        out.append((n, n + c))
    return out


def _span(case, n, length):
    """(keys a sequence's queries touch, visible (query, key) pairs)."""
    if n == 0 or length == 0:
        return 0, 0
    if not case["causal"]:
        return length, n * length
    w, p0 = case["window"], length - n
    if w == 0:
        return length, n * p0 + n * (n + 1) // 2
    pairs = sum(min(p + 1, w) for p in range(p0, length))
    return length - max(0, p0 + 1 - w), pairs


def _cache_bytes(case):
    return sum(2 * length * case["heads_kv"] * case["dim"] for _, length in _lens(case))


def work(case):
    if case["kind"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        size = DTYPES[case["out"]].itemsize
        return {"bytes": 2 * M * K + N * K + 4 * N + size * M * N + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    h, d, p = case["heads_kv"], case["dim"], case["page"]
    if case["kind"] == "append":
        new = back = pages = 0
        for n, length in _lens(case):
            if n:
                first = (length - n) // p
                new += n
                back += length - first * p
                pages += -(-length // p) - first
        # new keys and values read, codes and scales written, touched pages written back as 16-bit values
        return {"bytes": 2 * h * (2 * d * new + d * new + 4 * pages + 2 * d * back), "flops": 4 * h * d * (new + back)}
    hq = case["heads"]
    keys = pairs = new = 0
    for n, length in _lens(case):
        k, q = _span(case, n, length)
        keys, pairs, new = keys + k, pairs + q, new + n
    return {"bytes": 2 * h * d * keys + 8 * h * (keys // p) + 4 * hq * d * new, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _quantize_rows(x):
    """Symmetric INT8 codes and one scale per row."""
    a = x.abs().amax(dim=-1, keepdim=True).float()
    s = a / 127
    q = torch.where(s > 0, torch.round(x.float() / s), torch.zeros_like(s)).clamp(-127, 127)
    return q.to(torch.int8), s[..., 0]


def prepare(case, seed):
    g = _gen(seed)
    if case["kind"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        # heavy-tailed activations with 1 % outlier channels, as in front of a linear layer
        x = 0.5 * _randn(g, M, K)
        x /= torch.sqrt(sum(_randn(g, M, K) ** 2 for _ in range(3)) / 3).clamp_min(1e-3)
        hot = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]
        x[:, hot] *= 30
        w = 0.02 * _randn(g, N, K)
        wq, ws = _quantize_rows(w.half())
        bias = 0.5 * _randn(g, N) if case["bias"] else None
        return dict(case=case, x=x.clamp(-60000, 60000).to(DTYPES[case["dtype"]]), wq=wq, ws=ws, bias=bias)

    lens = _lens(case)
    h, d, p = case["heads_kv"], case["dim"], case["page"]
    dt = DTYPES[case["dtype"]]
    need = [-(-length // p) for _, length in lens]
    width, total = max(max(need), 1), sum(need)
    pages = total + 3                                  # a pool with pages to spare
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    state = dict(case=case, lens=lens, table=table, total=cu[-1], max_new=max(n for n, _ in lens),
                 max_len=max(length for _, length in lens),
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 lens_dev=torch.tensor([length for _, length in lens], dtype=torch.int32, device="cuda"))

    def cache(*shape):
        # codes of normal values whose page maximum is near 127, scales that differ by page and head
        codes = (36.0 * _randn(g, *shape)).round_().clamp_(-127, 127).to(torch.int8)
        scale = 0.03 * torch.exp(0.5 * _randn(g, pages, h))
        scale[perm[total:].long()] = float("nan")      # pages that belong to no one
        return codes, scale
    state["kc"], state["ks"] = cache(pages, h, p, d)
    state["vc"], state["vs"] = cache(pages, h, d, p)
    if case["kind"] == "append":
        state["k"] = (2.0 * _randn(g, cu[-1], h, d)).to(dt)
        state["v"] = _randn(g, cu[-1], h, d).to(dt)
        # the tokens of the touched pages, as the last tokens of each sequence
        back = [length - (length - n) // p * p if n else 0 for n, length in lens]
        cb = [0]
        for n in back:
            cb.append(cb[-1] + n)
        state.update(back=back, back_total=cb[-1], back_max=max(back),
                     back_cu=torch.tensor(cb, dtype=torch.int32, device="cuda"))
        # for the plain form: touched pages, the new token in each slot (or none), slots with an older token
        ids, slot, older = [], [], []
        for b, (n, length) in enumerate(lens):
            for j in range((length - n) // p, -(-length // p) if n else 0):
                pos = range(j * p, (j + 1) * p)
                ids.append((b, j))
                slot.append([cu[b] + t - (length - n) if length - n <= t < length else cu[-1] for t in pos])
                older.append([t < length - n for t in pos])
        ij = torch.tensor(ids, device="cuda").view(-1, 2)
        state["touched"] = table[ij[:, 0], ij[:, 1]].long()
        state["slot"] = torch.tensor(slot, device="cuda").view(-1, p)
        state["older"] = torch.tensor(older, device="cuda").view(-1, p)
        state["read"] = _positions(state, back, p)
    else:
        # queries sharp enough that the softmax picks some keys out
        state["q"] = (2.0 * _randn(g, cu[-1], case["heads"], d)).to(dt)
    return state


def _positions(state, back, p):
    """(page, slot) of the last back[b] tokens of each sequence."""
    pg, sl = [], []
    for b, (n, (_, length)) in enumerate(zip(back, state["lens"])):
        t = torch.arange(length - n, length, device="cuda")
        pg.append(state["table"][b, t // p].long())
        sl.append(t % p)
    return torch.cat(pg), torch.cat(sl)


# ----------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["kind"] == "linear":
        return _linear(case, state)
    if case["kind"] == "append":
        return _append(case, state)
    return _attention(case, state)


def _run_own(case, state):
    from w4a4_quantized_gemm_quantize_amd import ops
    if case["kind"] == "linear":
        return ops.w8a8_linear(state["x"], state["wq"], state["ws"], bias=state["bias"],
                               out_dtype=DTYPES[case["out"]])
    pool = (state["kc"], state["vc"], state["ks"], state["vs"], state["table"])
    if case["kind"] == "append":
        ops.kv8_append(state["k"], state["v"], *pool, state["cu"], state["lens_dev"], state["max_new"])
        k, v = ops.kv8_gather(*pool, state["back_cu"], state["lens_dev"], state["back_total"], state["back_max"],
                              out_dtype=DTYPES[case["dtype"]])
        return {"k": k, "v": v, "k_scale": state["ks"][state["touched"]], "v_scale": state["vs"][state["touched"]]}
    return ops.kv8_attention(state["q"], *pool, state["cu"], state["lens_dev"], state["max_new"], state["max_len"],
                             causal=case["causal"], window=case["window"])


def _linear(case, state):
    x, wq = state["x"], state["wq"]
    q, s = _quantize_rows(x)
    M, K, N = case["M"], case["K"], case["N"]
    acc = torch.empty((M, N), device="cuda", dtype=torch.float64)
    # sums of products up to 127^2 K pass 2^24: blocks of K whose sums fp32 holds exactly
    acc.zero_()
    step = 1024
    for k in range(0, K, step):
        acc += q[:, k:k + step].float() @ wq[:, k:k + step].float().t()
    y = acc.float() * (s[:, None] * state["ws"][None, :])
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(DTYPES[case["out"]])


def _store(x, codes, scale, state):
    """New rows into the touched pages; codes [pages, H, P, D]."""
    pg, slot, older = state["touched"], state["slot"], state["older"]
    new = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[slot].float().permute(0, 2, 1, 3)   # [n, H, P, D]
    s_new = new.abs().amax(dim=(2, 3)) / 127
    has_old = older.any(dim=1)[:, None]
    s_old = torch.where(has_old, scale[pg], torch.zeros_like(s_new))
    s = torch.maximum(s_old, s_new)
    grown = has_old & (s > s_old)
    ratio = torch.where(grown, s_old / s, torch.ones_like(s))
    old = codes[pg].float()
    old = torch.round(old * ratio[:, :, None, None])
    q = torch.where(s[:, :, None, None] > 0, torch.round(new / s[:, :, None, None]), torch.zeros_like(new))
    fresh = (slot < x.shape[0])[:, None, :, None]
    keep = older[:, None, :, None]
    codes[pg] = torch.where(fresh, q.clamp(-127, 127), torch.where(keep, old, codes[pg].float())).to(torch.int8)
    scale[pg] = s


def _append(case, state):
    _store(state["k"], state["kc"], state["ks"], state)
    _store(state["v"], state["vc"].transpose(2, 3), state["vs"], state)
    pg, sl = state["read"]
    dt = DTYPES[case["dtype"]]
    k = state["kc"][pg, :, sl].float() * state["ks"][pg][:, :, None]
    v = state["vc"][pg, :, :, sl].float() * state["vs"][pg][:, :, None]
    return {"k": k.to(dt), "v": v.to(dt), "k_scale": state["ks"][state["touched"]],
            "v_scale": state["vs"][state["touched"]]}


def _values(state, b, length, real, p):
    """K [H, L, D] and V [H, L, D] of a sequence as real numbers."""
    pg = state["table"][b, :-(-length // p)].long()
    k = state["kc"][pg].to(real) * state["ks"][pg].to(real)[:, :, None, None]
    v = state["vc"][pg].to(real) * state["vs"][pg].to(real)[:, :, None, None]
    k = k.permute(1, 0, 2, 3).reshape(k.shape[1], -1, k.shape[3])[:, :length]
    v = v.permute(1, 0, 3, 2).reshape(v.shape[1], -1, v.shape[2])[:, :length]
    return k, v


def _attention(case, state):
    q, p, d = state["q"], case["page"], case["dim"]
    hk, grp = case["heads_kv"], case["heads"] // case["heads_kv"]
    out = torch.zeros_like(q)
    at = 0
    for b, (n, length) in enumerate(state["lens"]):
        if n and length:
            k, v = _values(state, b, length, torch.float32, p)
            kt = k.transpose(1, 2)
            rows = max(1, min(n, (1 << 28) // (hk * grp * length)))     # scores within 1 GiB
            for i in range(0, n, rows):
                m = min(rows, n - i)
                qq = q[at + i:at + i + m].float().view(m, hk, grp, d).permute(1, 2, 0, 3).reshape(hk, grp * m, d)
                s = (qq @ kt).view(hk, grp, m, length) * (1.0 / math.sqrt(d))
                if case["causal"]:
                    pos = torch.arange(length - n + i, length - n + i + m, device="cuda")[:, None]
                    key = torch.arange(length, device="cuda")[None, :]
                    hide = key > pos
                    if case["window"]:
                        hide = hide | (key <= pos - case["window"])
                    s.masked_fill_(hide, float("-inf"))
                s = torch.exp(s - s.amax(dim=-1, keepdim=True))
                o = s.view(hk, grp * m, length) @ v
                o = o.view(hk, grp, m, d) / s.sum(dim=-1, keepdim=True)
                out[at + i:at + i + m] = o.permute(2, 0, 1, 3).reshape(m, hk * grp, d).to(out.dtype)
        at += n
    return out


# -------------------------------------------------- the definitions in 64 bits

def _codes64(x, s):
    """rne(fl32(x / s)): the quotient is rounded to 32 bits by definition."""
    return torch.where(s > 0, (x / s).float().double().round(), torch.zeros_like(x)).clamp(-127, 127)


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "linear":
        x = state["x"].double()
        s = (x.abs().max(dim=1, keepdim=True).values / 127).float().double()
        y = _codes64(x, s) @ state["wq"].double().t()
        y *= s
        y *= state["ws"].double()
        return y if state["bias"] is None else y + state["bias"].double()
    p = case["page"]
    if case["kind"] == "append":
        outs = {"k": [], "v": [], "k_scale": [], "v_scale": []}
        at = 0
        for b, (n, length) in enumerate(state["lens"]):
            for j in range((length - n) // p, -(-length // p) if n else 0):
                page, p0 = int(state["table"][b, j]), length - n
                lo, hi = max(j * p, p0), min(length, (j + 1) * p)
                held = max(0, min(p0 - j * p, p))               # tokens of the page that were there before
                for name, x, codes, scale in (("k", state["k"], state["kc"][page], state["ks"]),
                                              ("v", state["v"], state["vc"][page].transpose(1, 2), state["vs"])):
                    rows = x[at + lo - p0:at + hi - p0].double().transpose(0, 1)     # [H, new, D]
                    s = (rows.abs().flatten(1).max(dim=1).values / 127).float().double()
                    old = codes[:, :held].double()
                    if held:
                        before = scale[page].double()
                        after = torch.maximum(before, s)
                        ratio = (before / after).float().double()
                        old = torch.where((after > before)[:, None, None],
                                          (old * ratio[:, None, None]).float().double().round(), old)
                        s = after
                    s3 = s[:, None, None]
                    outs[name].append((torch.cat([old, _codes64(rows, s3)], dim=1) * s3).transpose(0, 1))
                    outs[name + "_scale"].append(s[None])
            at += n
        return {key: torch.cat(v) for key, v in outs.items()}
    grp = case["heads"] // case["heads_kv"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(state["lens"]):
        if n and length:
            k, v = _values(state, b, length, torch.float64, p)
            key = torch.arange(length, device="cuda")
            for h in range(case["heads"]):
                for i in range(0, n, 4096):
                    m = min(4096, n - i)
                    s = state["q"][at + i:at + i + m, h].double() @ k[h // grp].t() / math.sqrt(case["dim"])
                    if case["causal"]:
                        ahead = key[None, :] - (length - n + i + torch.arange(m, device="cuda"))[:, None]
                        s[(ahead > 0) | (ahead <= -(case["window"] or length))] = -math.inf
                    out[at + i:at + i + m, h] = torch.softmax(s, dim=1) @ v[h // grp]
        at += n
    return out

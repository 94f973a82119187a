"""Cases and plain forms of the 8-bit prefix operators.

A prefix enters the action expert through three operators that belong together:

  linear      y = (rows of x, each in 8 bits) times (weight rows in 8 bits):
              one scale per token and one per output channel, optionally with
              the RMSNorm that prefix production puts before its projection;
  cache       K/V rows quantised into a slot cache as they are written (one
              scale per token and KV head), and read back;
  attention   queries over such a cache: single tokens, the denoise loop's
              chunk of action tokens with its own fresh keys, causal prompts.

Plain forms are elementary torch operations in 32 bits (64 where a value sits
next to a rounding border); `exact` is the definition in 64 bits.  Shapes are
the pi0.5 expert's (width 1024, 8 query heads on 1 KV head of 256, MLP 4096,
prefixes of 512 to 1024 tokens with 968 = 3 x 256 + 200 the usual one, chunks
of 50, batches of 1 to 32, prefix width 2048) and generic ones around them.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ES = {"bf16": 2, "fp32": 4}
TINY = 2.0 ** -120  # rows whose scale is smaller are stored as zeros
EPS = 1e-6


# ---------------------------------------------------------------------- cases
def listed():
    lin = dict(op="linear", dtype="bf16", rms=False)
    att = dict(op="attention", heads=8, kv_heads=1, dim=256, causal=False, fresh=0)
    return [
        # the expert's q/k/v rows for one token: the smallest call, latency alone
        dict(lin, name="linear one token", tokens=1, k=1024, n=2560),
        # gate and up of one 50-token chunk: weight streaming
        dict(lin, name="linear chunk", tokens=50, k=1024, n=8192),
        # key and value rows of one observation, as prefix production computes them
        dict(lin, name="linear prefix", tokens=968, k=2048, n=512, rms=True),
        # the down projection at batch 32, 32-bit activations in and out
        dict(lin, name="linear batch fp32", tokens=1600, k=4096, n=1024, dtype="fp32"),
        # a prefix model's wide projection over eight observations, ragged
        dict(lin, name="linear wide", tokens=7743, k=2048, n=16384),
        # one new token for each of 32 sequences
        dict(op="cache", name="cache one token each", seqs=32, lo=1, hi=1, start=968, kv_heads=1, dim=256, dtype="bf16"),
        # 16 ragged prefixes of one observation each, several KV heads, 32-bit rows
        dict(op="cache", name="cache ragged prefixes", seqs=16, lo=512, hi=1024, start=0, kv_heads=4, dim=128, dtype="fp32"),
        # one query token over one prefix: the smallest call
        dict(att, name="attention one token", seqs=1, queries=1, lo=968, hi=968),
        # single tokens of 48 sequences over caches from one position to long ones
        dict(att, name="attention tokens", seqs=48, queries=1, lo=1, hi=8192),
        # the denoise loop at batch 1: 50 action tokens over [prefix | 50 fresh keys]
        dict(att, name="attention chunk", seqs=1, queries=50, lo=968, hi=968, fresh=50),
        # the same at batch 32
        dict(att, name="attention chunk batch", seqs=32, queries=50, lo=968, hi=968, fresh=50),
        # the 200 text tokens of eight prompts behind their 768 image tokens
        dict(att, name="attention causal prompt", seqs=8, queries=200, lo=968, hi=968, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "cache", "attention", "attention", "attention"])
    if op == "linear":
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 7743), k=16 * _log(rng, 8, 256), n=_log(rng, 40, 16384),
                     dtype=rng.choice(["bf16", "bf16", "fp32"]), rms=rng.random() < 0.4)
            if c["tokens"] * c["n"] <= 40_000_000:
                return c
    dim = rng.choice([64, 128, 256, 256])
    kv_heads = rng.choice([1, 1, 2, 4])
    if op == "cache":
        while True:
            hi = _log(rng, 1, 4096)
            c = dict(op=op, seqs=_log(rng, 1, 48), lo=rng.randint(0, hi), hi=hi, start=rng.choice([0, 0, _log(rng, 1, 2000)]),
                     kv_heads=kv_heads, dim=dim, dtype=rng.choice(["bf16", "bf16", "fp32"]))
            if c["seqs"] * hi * kv_heads * dim <= 8_000_000 and c["seqs"] * hi >= 1:
                return c
    while True:
        form = rng.choice(["token", "token", "chunk", "prompt"])
        hi = _log(rng, 1, 8192)
        c = dict(op=op, seqs=_log(rng, 1, 48), queries=1, lo=rng.randint(0, hi), hi=hi, heads=kv_heads * rng.choice([1, 2, 4, 8]),
                 kv_heads=kv_heads, dim=dim, causal=False, fresh=0)
        if form == "chunk":
            c["queries"] = _log(rng, 2, 200)
            c["fresh"] = rng.choice([0, c["queries"], c["queries"]])
        elif form == "prompt":
            c["queries"] = _log(rng, 2, 400)
            c["causal"] = True
        keys = c["seqs"] * (hi + c["fresh"])
        if keys * kv_heads * dim <= 48 * 8192 * 256 and keys * c["queries"] * c["heads"] * dim <= 32 * 1018 * 50 * 8 * 256:
            return c


def _lens(c):
    """Lengths of the sequences: spread over [lo, hi], the same for every seed."""
    n, lo, hi = c["seqs"], c["lo"], c["hi"]
    if n == 1:
        return [hi]
    return [lo + ((hi - lo) * ((i * 7919 + 3) % n)) // (n - 1) for i in range(n)]


# --------------------------------------------------------------------- inputs
def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _quantize(x):
    """Rows (last dimension) -> (codes as float32, scale float32): scale =
    max|x| / 127 rounded to 32 bits, codes = round(x / scale), ties to even.
    The quotient is taken in 64 bits: codes next to a half stay the definition's."""
    amax = x.float().abs().amax(-1)
    s = (amax.double() / 127.0).float()
    s = torch.where(s < TINY, torch.zeros_like(s), s)
    d = torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1)
    q = torch.round(x.double() / d).float()
    q = torch.where(s.unsqueeze(-1) > 0, q, torch.zeros_like(q))
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    st = {"case": case}
    if case["op"] == "linear":
        T, K, N, dt = case["tokens"], case["k"], case["n"], DT[case["dtype"]]
        # hidden states: unit rows of different size, a few channels that stand out
        gain = 1.0 + 7.0 * (torch.rand(K, generator=g, device="cuda") < 0.01).float()
        size = torch.exp(0.5 * _normal(g, (T, 1)))
        st["x"] = (_normal(g, (T, K)) * gain * size).to(dt)
        # weights are quantised once, when a program loads them
        w, st["w_scale"] = _quantize(0.02 * _normal(g, (N, K)))
        st["w"] = w.to(torch.int8)
        return st
    lens = _lens(case)
    B, Hk, d = case["seqs"], case["kv_heads"], case["dim"]
    if case["op"] == "cache":
        T, dt = sum(lens), DT[case["dtype"]]
        st["total"] = T
        st["k"], st["v"] = _normal(g, (T, Hk, d), dt), _normal(g, (T, Hk, d), dt)
        st["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
        st["start"] = torch.full((B,), case["start"], dtype=torch.int32, device="cuda")
        cap = case["start"] + max(lens)
        if own:
            import flow_matching_action_pi0_b200 as fm
            st["cache"] = fm.KvCacheInt8(B, Hk, cap, d)
        else:
            st["row_slot"] = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).cuda()
            st["row_pos"] = torch.cat([torch.arange(n) + case["start"] for n in lens]).cuda()
            st["codes"] = torch.zeros(2, B, Hk, cap, d, dtype=torch.int8, device="cuda")
            st["scales"] = torch.zeros(2, B, Hk, cap, dtype=torch.float32, device="cuda")
        return st
    cap = max(max(lens), 1)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["q"] = _normal(g, (B, case["queries"], case["heads"], d), torch.bfloat16)
    codes, scales = [], []
    for _ in range(2):
        q = torch.empty(B, Hk, cap, d, dtype=torch.int8, device="cuda")
        s = torch.empty(B, Hk, cap, dtype=torch.float32, device="cuda")
        for b in range(B):
            qb, s[b] = _quantize(_normal(g, (Hk, cap, d), torch.bfloat16))
            q[b] = qb.to(torch.int8)
        codes.append(q)
        scales.append(s)
    if case["fresh"]:
        st["k_new"] = _normal(g, (B, case["fresh"], Hk, d), torch.bfloat16)
        st["v_new"] = _normal(g, (B, case["fresh"], Hk, d), torch.bfloat16)
    if own:
        import flow_matching_action_pi0_b200 as fm
        cache = fm.KvCacheInt8(B, Hk, cap, d)
        for dst, src in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), codes + scales):
            dst.copy_(src)
        st["cache"] = cache
        st["plan"] = cache.plan(B, case["queries"], case["heads"], fresh=case["fresh"])
    else:
        st["codes"], st["scales"] = codes, scales
    return st


# ---------------------------------------------------------------- plain forms
def _plain_linear(st):
    c, x = st["case"], st["x"]
    q, s = _quantize(x)
    if c["rms"]:
        xf = x.float()
        s = s * torch.rsqrt((xf * xf).mean(-1) + EPS)
    y = (q @ st["w"].float().t()) * s.unsqueeze(-1) * st["w_scale"]
    return y.to(x.dtype)


def _plain_cache(st):
    slot, pos = st["row_slot"], st["row_pos"]
    out = []
    for i, x in enumerate((st["k"], st["v"])):
        q, s = _quantize(x)
        st["codes"][i][slot, :, pos] = q.to(torch.int8)
        st["scales"][i][slot, :, pos] = s
        out.append((st["codes"][i][slot, :, pos].float() * st["scales"][i][slot, :, pos].unsqueeze(-1)).to(x.dtype))
    return tuple(out)


def _attend(st, real):
    """o = softmax(q k / sqrt(d)) v over the visible keys, in `real` arithmetic."""
    c = st["case"]
    B, Hq, Hk, d, nq = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["queries"]
    G = Hq // Hk
    k, v = [q.to(real) * s.to(real).unsqueeze(-1) for q, s in zip(st["codes"], st["scales"])]  # [B, Hk, cap, d]
    cap, dev = k.shape[2], k.device
    at, last = torch.arange(cap, device=dev), st["lens"].long()
    if c["causal"]:  # query i stands at position len - queries + i
        limit = last.view(B, 1) - nq + 1 + torch.arange(nq, device=dev).view(1, nq)
    else:
        limit = last.view(B, 1).expand(B, nq)
    seen = at.view(1, 1, cap) < limit.unsqueeze(-1)  # [B, nq, cap]
    if c["fresh"]:
        k = torch.cat([k, st["k_new"].to(real).transpose(1, 2)], 2)
        v = torch.cat([v, st["v_new"].to(real).transpose(1, 2)], 2)
        seen = torch.cat([seen, torch.ones(B, nq, c["fresh"], dtype=torch.bool, device=dev)], 2)
    q = st["q"].to(real).view(B, nq, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * nq, d)
    s = (q @ k.transpose(2, 3)).view(B, Hk, G, nq, -1) / math.sqrt(d)
    s = s.masked_fill(~seen.view(B, 1, 1, nq, -1), float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, G * nq, -1) @ v).view(B, Hk, G, nq, d)
    o = torch.where(z > 0, o / torch.where(z > 0, z, torch.ones_like(z)), torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(B, nq, Hq, d)


def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "linear":
            return _plain_linear(state)
        if c["op"] == "cache":
            return _plain_cache(state)
        return _attend(state, torch.float32).to(torch.bfloat16)
    import flow_matching_action_pi0_b200 as fm
    if c["op"] == "linear":
        x = state["x"]
        q, s = fm.quantize_rows(x, rms_eps=EPS if c["rms"] else None)
        return fm.linear_i8(q, s, state["w"], state["w_scale"], out_dtype=x.dtype)
    if c["op"] == "cache":
        state["cache"].write(state["k"], state["v"], state["cu"], state["start"])
        return state["cache"].read(state["cu"], state["start"], state["total"], dtype=state["k"].dtype)
    return state["cache"].attend(state["q"], state["lens"], causal=c["causal"], k_new=state.get("k_new"),
                                 v_new=state.get("v_new"), plan=state["plan"])


# ------------------------------------------------------------------ the exact
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "attention":
        # one sequence and KV head at a time, keys gathered rather than masked
        B, nq, Hq, d = st["q"].shape
        Hk, G = case["kv_heads"], case["heads"] // case["kv_heads"]
        out = torch.zeros(B, nq, Hq, d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case)):
            for h in range(Hk):
                kk, vv = [q[b, h, :n].double() * s[b, h, :n].double()[:, None] for q, s in zip(st["codes"], st["scales"])]
                if case["fresh"]:
                    kk, vv = torch.cat([kk, st["k_new"][b, :, h].double()]), torch.cat([vv, st["v_new"][b, :, h].double()])
                if kk.shape[0] == 0:
                    continue
                for g in range(h * G, h * G + G):
                    t = st["q"][b, :, g].double() @ kk.T * d ** -0.5
                    if case["causal"]:
                        i, j = torch.meshgrid(torch.arange(nq, device="cuda"), torch.arange(n, device="cuda"), indexing="ij")
                        t[j - i > n - nq] = -math.inf
                    some = ~torch.isinf(t).all(1)
                    out[b, some, g] = torch.softmax(t[some], 1) @ vv
        return out
    one = np.float64(127.0)

    def codes_of(x):
        """(codes, scale) in float64 from the definition: the scale is a 32-bit number by definition."""
        a = x.double()
        s = (a.abs().max(-1, keepdim=True).values / one).float().double()
        s[s < TINY] = 0.0
        return torch.where(s > 0, torch.round(a / torch.where(s > 0, s, 1.0)), 0.0), s

    if case["op"] == "cache":
        return tuple((lambda qs: qs[0] * qs[1])(codes_of(x)) for x in (st["k"], st["v"]))
    q, s = codes_of(st["x"])
    if case["rms"]:
        s = s / torch.sqrt((st["x"].double() ** 2).mean(-1, keepdim=True) + EPS)
    return torch.einsum("tk,nk->tn", q, st["w"].double()) * s * st["w_scale"].double()[None, :]


# ----------------------------------------------------------------------- work
def work(case):
    if case["op"] == "linear":
        T, K, N, es = case["tokens"], case["k"], case["n"], ES[case["dtype"]]
        return {"bytes": T * K * es + N * K + 4 * N + T * N * es, "flops": 2 * T * K * N}
    lens = _lens(case)
    Hk, d = case["kv_heads"], case["dim"]
    if case["op"] == "cache":
        rows = 2 * sum(lens) * Hk
        # rows in, codes and scales written and read again, rows out
        return {"bytes": rows * (2 * d * ES[case["dtype"]] + 2 * (d + 4)), "flops": 4 * rows * d}
    nq, Hq, fresh = case["queries"], case["heads"], case["fresh"]
    pairs = 0  # visible (query, key) pairs
    for n in lens:
        pairs += sum(max(0, n - nq + 1 + i) for i in range(nq)) if case["causal"] else nq * (n + fresh)
    return {"bytes": 2 * sum(lens) * Hk * (d + 4) + 4 * case["seqs"] * fresh * Hk * d + 4 * case["seqs"] * nq * Hq * d,
            "flops": 4 * pairs * Hq * d}

"""The cases on which the library's layer-step and sampling operators are measured.

Three operators of a decoder's serving step, each as a plain computation in elementary torch
operations and as the call a user makes of the library:

* ``rope``: the position rotation of a step's queries and keys, with the keys and values appended
  to the paged cache on the way (``pa_rope_store_kv``); positions with one axis, or with three
  (time, height, width) of which each frequency takes one.
* ``chunk``: attention of a chunk of new tokens of each sequence over its paged cache, causal,
  with or without a sliding window (``pa_chunk_attn``).
* ``sample``: one token per row from its logits with temperature, top-k, top-p and min-p and a
  given random number (``pa_sample``).

A case is a dict of plain values. Lengths are drawn from the case's own ``lens`` number, so that
its work is a function of the case alone; values and block placements come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of a handful of sequences: launch latency is all of it
        _rope("rope_decode_tiny", T=4, Hq=4, Hkv=2, D=64, bs=16, dtype="f16"),
        # a decode step of a full batch, q, k and v as slices of one projection's output; the last
        # tokens are the padding of a captured batch size
        _rope("rope_decode_batch", T=256, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", fused=True, pad=5),
        # the tokens of 64 packed prompts
        _rope("rope_prefill", T=33673, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", fused=True),
        # a prompt of text and images with (time, height, width) positions in three sections
        _rope("rope_axes_prefill", T=9001, Hq=14, Hkv=2, D=64, bs=16, dtype="f16", axes=3, fused=True),
        # single decode tokens after such prompts, the axes in turn over the frequencies
        _rope("rope_axes_decode", T=32, Hq=16, Hkv=8, D=128, bs=16, dtype="bf16", axes=3, turns=True),
        # one short draft to verify: latency
        _chunk("chunk_draft_tiny", S=4, q_lo=1, q_hi=5, ctx_lo=5, ctx_hi=255, Hq=4, Hkv=2, D=64, bs=16, dtype="f16", lens=1),
        # few sequences with long caches and drafts of a few tokens: the cache has to be split
        _chunk("chunk_draft_long", S=3, q_lo=3, q_hi=8, ctx_lo=9000, ctx_hi=16384, Hq=14, Hkv=2, D=64, bs=16, dtype="f16", lens=2),
        # drafts of up to 5 tokens for a full batch: the cache's bytes are all of it
        _chunk("chunk_draft_batch", S=256, q_lo=1, q_hi=5, ctx_lo=100, ctx_hi=4096, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", lens=3, pad=7),
        # pieces of long prompts, each with what is cached of its prompt: matrix work
        _chunk("chunk_prefill_long", S=2, q_lo=1900, q_hi=2048, ctx_lo=12000, ctx_hi=16384, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", lens=4),
        # a layer with a sliding window, chunks of ragged prompts
        _chunk("chunk_window", S=12, q_lo=20, q_hi=700, ctx_lo=2000, ctx_hi=6000, Hq=32, Hkv=8, D=128, bs=16, dtype="bf16", lens=5, window=1024),
        # one request's next token
        dict(name="sample_one", op="sample", B=1, V=151936, dtype="bf16", mix="nucleus"),
        # a full batch of requests with settings of their own
        dict(name="sample_batch", op="sample", B=256, V=151936, dtype="f32", mix="all"),
    ]


def _rope(name, T, Hq, Hkv, D, bs, dtype, rot=0, axes=1, turns=False, pairs=False, fused=False, pad=0):
    return dict(name=name, op="rope", T=T, Hq=Hq, Hkv=Hkv, D=D, bs=bs, dtype=dtype, rot=rot or D, axes=axes,
                turns=turns, pairs=pairs, fused=fused, pad=pad)


def _chunk(name, S, q_lo, q_hi, ctx_lo, ctx_hi, Hq, Hkv, D, bs, dtype, lens, window=0, pad=0):
    return dict(name=name, op="chunk", S=S, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, Hq=Hq, Hkv=Hkv,
                D=D, bs=bs, dtype=dtype, lens=lens, window=window, pad=pad)


HEADS = [(4, 2), (14, 2), (16, 8), (32, 4), (6, 6), (20, 5), (16, 2), (9, 3), (5, 1)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "sample"])
    if op == "rope":
        Hq, Hkv = rng.choice(HEADS)
        D = rng.choice([64, 80, 128, 128, 256])
        T = _log(rng, 1, min(33000, 33673 * 32 * 128 // ((Hq + 2 * Hkv) * D)))
        rot = D if rng.random() < 0.7 else rng.choice([16, 32, 48, 64])
        axes = rng.choice([1, 1, 3])
        c = _rope("", T, Hq, Hkv, D, rng.choice([1, 16, 16, 48, 256]), rng.choice(["f16", "bf16"]), rot=rot, axes=axes,
                  turns=rng.random() < 0.5, pairs=rng.random() < 0.3, fused=rng.random() < 0.6,
                  pad=min(T - 1, rng.choice([0, 0, 3, 17])))
    elif op == "chunk":
        Hq, Hkv = rng.choice(HEADS)
        D = rng.choice([64, 128])
        q_hi = _log(rng, 1, 2000)
        ctx_hi = max(q_hi, _log(rng, 64, 16000))
        # the scores of the plain form in 32 bits, and the cache's rows, within the listed ones
        most = min(2 * 16 * 2048 * 16384 // (Hq * q_hi * ctx_hi), 256 * 8 * 128 * 2000 // (Hkv * D * ctx_hi))
        S = _log(rng, 1, max(1, min(300, most)))
        c = _chunk("", S, rng.randint(0, q_hi), q_hi, rng.randint(1, ctx_hi), ctx_hi, Hq, Hkv, D,
                   rng.choice([16, 16, 64, 256, 24, 4]), rng.choice(["f16", "bf16"]), rng.randint(0, 9999),
                   window=0 if rng.random() < 0.6 else _log(rng, 1, 5000), pad=rng.choice([0, 0, 5]))
    else:
        V = rng.choice([32000, 50257, 128256, 151936, 262144, _log(rng, 200, 200000)])
        B = _log(rng, 1, max(1, min(300, 256 * 151936 // V)))
        c = dict(op="sample", B=B, V=V, dtype=rng.choice(["f32", "bf16", "f16"]),
                 mix=rng.choice(["all", "nucleus", "top_k", "plain", "greedy"]))
    c.pop("name", None)
    return c


def _lengths(c):
    """(new tokens, context length with them) of each sequence of a chunk case."""
    r = random.Random(c["lens"] * 7919 + c["S"])
    q = [r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["S"])]
    return q, [max(n, r.randint(c["ctx_lo"], c["ctx_hi"])) for n in q]


def work(case):
    c = case
    if c["op"] == "rope":
        T, e = c["T"] - c["pad"], 2
        rows = T if c["axes"] == 1 else min(T, 100)  # of the table: the patches of an image share theirs
        return {"bytes": T * c["D"] * e * (2 * c["Hq"] + 4 * c["Hkv"]) + T * (4 + 4 * c["axes"]) + rows * c["rot"] * 4,
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "chunk":
        q, ctx = _lengths(c)
        W = c["window"]
        seen = read = 0
        for n, k in zip(q, ctx):
            if n:
                p0 = k - n
                seen += sum(min(p + 1, W) for p in range(p0, k)) if W else n * p0 + n * (n + 1) // 2
                read += k - max(0, p0 - W + 1) if W else k
        return {"bytes": 2 * 2 * read * c["Hkv"] * c["D"] + 2 * 2 * sum(q) * c["Hq"] * c["D"] + 4 * sum(-(-k // c["bs"]) for k in ctx),
                "flops": 4 * c["D"] * c["Hq"] * seen}
    return {"bytes": c["B"] * (c["V"] * SIZE[c["dtype"]] + 24), "flops": 4 * c["B"] * c["V"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pair_axis(c):
    """Which axis each rotated pair takes its position from: sections in the ratio 1 : 1.5 : 1.5
    one after the other, or in turns over the first frequencies and time for the rest."""
    n = c["rot"] // 2
    if c["axes"] == 1:
        return [0] * n
    h = 3 * n // 8
    if c["turns"]:
        return [i % 3 if i < 3 * h and i % 3 else 0 for i in range(n)]
    return [0] * (n - 2 * h) + [1] * h + [2] * h


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "rope":
        return _prepare_rope(c, g)
    if c["op"] == "chunk":
        return _prepare_chunk(c, g, seed)
    return _prepare_sample(c, g)


def _prepare_rope(c, g):
    T, Hq, Hkv, D, dt = c["T"], c["Hq"], c["Hkv"], c["D"], DT[c["dtype"]]
    if c["fused"]:
        qkv = _normal(g, T, Hq + 2 * Hkv, D, dtype=dt)
        c["q"], c["k"], c["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        c["q"], c["k"], c["v"] = (_normal(g, T, h, D, dtype=dt) for h in (Hq, Hkv, Hkv))
    nb = -(-T // c["bs"]) + max(1, T // (4 * c["bs"]))
    c["k_cache"], c["v_cache"] = (_normal(g, nb, c["bs"], Hkv, D, dtype=dt) for _ in range(2))
    blocks = torch.randperm(nb, generator=g, device="cuda")[: -(-T // c["bs"])]
    t = torch.arange(T, device="cuda")
    slots = blocks[t // c["bs"]] * c["bs"] + t % c["bs"]
    if c["pad"]:
        slots[T - c["pad"]:] = -1
    c["slots"] = slots.to(torch.int32)
    # the table of a model that takes 32768 positions: cosines, then sines, of each position's
    # angles, computed in 64 bits and rounded once
    n = c["rot"] // 2
    inv = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    a = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * inv
    c["table"] = torch.cat([a.cos(), a.sin()], 1).float()
    if c["axes"] == 1:
        start = int(torch.randint(0, 28000, (1,), generator=g, device="cuda"))
        c["positions"] = ((start + t) % 32768).to(torch.int32)
    else:  # images of 36 x 28 patches: time stands still over an image
        start = int(torch.randint(0, 20000, (1,), generator=g, device="cuda"))
        c["positions"] = torch.stack([start + t // 1008 * 36, start + t // 28 % 36, start + t % 28]).to(torch.int32)
    c["pair_axis"] = bytes(_pair_axis(c))
    c["axis_of"] = torch.tensor(_pair_axis(c), device="cuda")
    c["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    return c


def _prepare_chunk(c, g, seed):
    S, Hq, Hkv, D, bs, dt = c["S"], c["Hq"], c["Hkv"], c["D"], c["bs"], DT[c["dtype"]]
    q, ctx = _lengths(c)
    used = [-(-k // bs) for k in ctx]
    nb = sum(used) + max(1, sum(used) // 4)
    c["k_cache"], c["v_cache"] = (_normal(g, nb, bs, Hkv, D, dtype=dt) for _ in range(2))
    perm = np.random.default_rng(seed).permutation(nb).astype(np.int32)
    bt = np.full((S, max(used)), -1, np.int32)
    at = 0
    for s, n in enumerate(used):
        bt[s, :n] = perm[at:at + n]
        if c["window"]:  # what lies before the first token's window has been given back
            bt[s, : max(0, ctx[s] - q[s] - c["window"] + 1) // bs] = -1
        at += n
    c["block_tables"] = torch.from_numpy(bt).cuda()
    c["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, device="cuda")
    c["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    c["max_q"], c["max_ctx"] = max(q), max(ctx)
    Tq = sum(q) + c["pad"]
    c["q"] = _normal(g, Tq, Hq, D, dtype=dt)
    c["out"] = torch.zeros(Tq, Hq, D, dtype=dt, device="cuda")
    c["scale"] = D ** -0.5
    if own:
        import paged_kv_cache_83_gb300 as pa
        n = pa.pa_chunk_attn_workspace_size(S, Hq, Hkv, D)
        c["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return c


def _prepare_sample(c, g):
    B, V = c["B"], c["V"]
    # a bulk of unlikely tokens and a few dozen likely ones, as a language model gives them
    x = torch.randn(B, V, generator=g, device="cuda") * 2.0
    n = min(V, 40)
    at = torch.randint(0, V, (B, n), generator=g, device="cuda")
    x.scatter_add_(1, at, 10.0 * torch.rand(B, n, generator=g, device="cuda"))
    c["logits"] = x.to(DT[c["dtype"]])
    r = torch.arange(B, device="cuda")
    temperature = 0.5 + torch.rand(B, generator=g, device="cuda")
    top_k = torch.randint(1, 101, (B,), generator=g, device="cuda")
    top_p = 0.7 + 0.29 * torch.rand(B, generator=g, device="cuda")
    min_p = 0.01 + 0.09 * torch.rand(B, generator=g, device="cuda")
    mix = c["mix"]
    kind = r % 6 if mix == "all" else torch.full_like(r, {"greedy": 0, "top_k": 1, "nucleus": 2, "plain": 3}[mix])
    # 0 greedy, 1 top-k, 2 top-p, 3 temperature alone, 4 top-k and top-p, 5 min-p
    c["temperature"] = torch.where(kind == 0, 0.0, temperature).float()
    c["top_k"] = torch.where((kind == 1) | (kind == 4), top_k, 0).to(torch.int32)
    c["top_p"] = torch.where((kind == 2) | (kind == 4), top_p, 1.0).float()
    c["min_p"] = torch.where(kind == 5, min_p, 0.0).float()
    c["u"] = torch.rand(B, generator=g, device="cuda")
    c["tokens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return c


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_rope(s):
    T, D, R, dt = s["T"], s["D"], s["rot"], DT[s["dtype"]]
    n = R // 2
    pos = s["positions"].reshape(s["axes"], T)[s["axis_of"]].t().long()  # [T, n]: each pair's position
    i = torch.arange(n, device="cuda")
    cos, sin = s["table"][pos, i][:, None], s["table"][pos, n + i][:, None]

    def rotate(x):
        x = x.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["pairs"] else (x[..., :n], x[..., n:R])
        y0, y1 = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y0, y1], -1).flatten(-2) if s["pairs"] else torch.cat([y0, y1], -1)
        return torch.cat([y, x[..., R:]], -1).to(dt)

    keep = s["slots"] >= 0
    s["q_out"].copy_(torch.where(keep[:, None, None], rotate(s["q"]), s["q_out"]))
    kept = s["slots"][: T - s["pad"]].long()  # the padding comes last
    s["k_cache"].view(-1, s["Hkv"], D)[kept] = rotate(s["k"])[: T - s["pad"]]
    s["v_cache"].view(-1, s["Hkv"], D)[kept] = s["v"][: T - s["pad"]]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_rope(s):
    import paged_kv_cache_83_gb300 as pa
    pa.pa_rope_store_kv(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                        s["table"], pair_axis=s["pair_axis"] if s["axes"] > 1 else None, interleaved=s["pairs"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_chunk(s):
    S, Hq, Hkv, D, bs, W = s["S"], s["Hq"], s["Hkv"], s["D"], s["bs"], s["window"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    if s["max_q"] == 0:
        return s["out"]
    n = cu[1:] - cu[:-1]
    r = torch.arange(s["max_q"], device="cuda")
    j = torch.arange(s["max_ctx"], device="cuda")
    valid = r < n[:, None]
    rows = torch.where(valid, cu[:-1, None] + r, 0)
    slot = (s["block_tables"].long()[:, j // bs] * bs + j % bs).clamp(min=0)
    k = s["k_cache"].view(-1, Hkv, D)[slot].float().permute(0, 2, 3, 1)             # [S, Hkv, D, K]
    v = s["v_cache"].view(-1, Hkv, D)[slot].float().permute(0, 2, 1, 3)             # [S, Hkv, K, D]
    q = s["q"][rows].float().view(S, -1, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)  # [S, Hkv, G, Q, D]
    x = torch.matmul(q.reshape(S, Hkv, -1, D) * s["scale"], k).view(S, Hkv, Hq // Hkv, -1, s["max_ctx"])
    p = (ctx - n)[:, None] + r
    seen = (j <= p[..., None]) & valid[..., None]
    if W:
        seen &= j > p[..., None] - W
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    o = torch.matmul(x.view(S, Hkv, -1, s["max_ctx"]), v).view(S, Hkv, Hq // Hkv, -1, D) / x.sum(-1, keepdim=True)
    s["out"][rows[valid]] = o.permute(0, 3, 1, 2, 4).reshape(S, -1, Hq, D)[valid].to(DT[s["dtype"]])
    return s["out"]


def _own_chunk(s):
    import paged_kv_cache_83_gb300 as pa
    pa.pa_chunk_attn(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["cu"], s["ctx"], s["max_q"],
                     s["scale"], window=s["window"], workspace=s["workspace"])
    return s["out"]


def _plain_sample(s):
    V = s["V"]
    x, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    T = s["temperature"].double()[:, None]
    rank = torch.arange(V, device="cuda")
    # 64 bits: the sums are long and a token is decided at a border of them
    w = torch.where(T > 0, torch.exp((x.double() - x[:, :1].double()) / torch.where(T > 0, T, 1.0)), (rank == 0).double())
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    w = w * (rank < k)
    before = w.cumsum(1) - w
    p = s["top_p"].double()[:, None]
    w = w * ((p >= 1) | (before < p * w.sum(1, keepdim=True)) | (rank == 0)) * (w >= s["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, w)
    upto = w.cumsum(1)
    s["tokens"].copy_((upto <= s["u"].double()[:, None] * upto[:, -1:]).sum(1))
    return s["tokens"]


def _own_sample(s):
    import paged_kv_cache_83_gb300 as pa
    pa.pa_sample(s["tokens"], s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                 min_p=s["min_p"])
    return s["tokens"]


_plain = {"rope": _plain_rope, "chunk": _plain_chunk, "sample": _plain_sample}
_own = {"rope": _own_rope, "chunk": _own_chunk, "sample": _own_sample}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "chunk": _exact_chunk, "sample": _exact_sample}[s["op"]](s)


def _exact_rope(s):
    """y = x e^(i angle) on the pairs as complex numbers, from the table's cosines and sines."""
    T, n, D = s["T"], s["rot"] // 2, s["D"]
    axis = s["axis_of"]
    pos = s["positions"].view(s["axes"], T)
    tab = s["table"].double()
    turn = torch.complex(tab[:, :n], tab[:, n:])
    z = torch.stack([turn[pos[int(axis[i])].long(), i] for i in range(n)], 1)[:, None]  # [T, 1, n]

    def rotate(x):
        y = x.double().clone()
        even, odd = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if s["pairs"] else (slice(0, n), slice(n, 2 * n))
        t = torch.complex(y[..., even], y[..., odd]) * z
        y[..., even], y[..., odd] = t.real, t.imag
        return y

    kept = s["slots"] >= 0
    q = s["q_out"].double().clone()
    q[kept] = rotate(s["q"])[kept]
    at = s["slots"][kept].long()
    k, v = s["k_cache"].double().clone(), s["v_cache"].double().clone()
    k.view(-1, s["Hkv"], D)[at] = rotate(s["k"])[kept]
    v.view(-1, s["Hkv"], D)[at] = s["v"].double()[kept]
    return {"q": q, "k_cache": k, "v_cache": v}


def _exact_chunk(s):
    """Sequence by sequence and kv head by kv head, 64-bit softmax attention over the visible keys."""
    out = s["out"].double().clone()
    cu, ctx, bt = s["cu"].tolist(), s["ctx"].tolist(), s["block_tables"].cpu().numpy()
    G, bs = s["Hq"] // s["Hkv"], s["bs"]
    for i in range(s["S"]):
        a, b, n = cu[i], cu[i + 1], ctx[i]
        if a == b:
            continue
        p0 = n - (b - a)
        first = max(0, p0 - s["window"] + 1) if s["window"] else 0
        j = np.arange(first, n)
        at = torch.from_numpy(bt[i][j // bs].astype(np.int64) * bs + j % bs).cuda()
        pos, key = torch.arange(p0, n, device="cuda")[:, None], torch.arange(first, n, device="cuda")[None]
        hidden = key > pos
        if s["window"]:
            hidden |= pos - key >= s["window"]
        for h in range(s["Hq"]):
            k = s["k_cache"].view(-1, s["Hkv"], s["D"])[at, h // G].double()
            v = s["v_cache"].view(-1, s["Hkv"], s["D"])[at, h // G].double()
            x = (s["q"][a:b, h].double() @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
            out[a:b, h] = torch.softmax(x, 1) @ v
    return out


def _exact_sample(s):
    """Row by row in numpy: the kept set by rank, then the token where the sum in the order of the
    vocabulary first exceeds u times the whole."""
    x = s["logits"].double().cpu().numpy()
    T, K, P, M, U = (s[k].double().cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u"))
    got = np.zeros(s["B"], np.int64)
    for i in range(s["B"]):
        if not T[i] > 0:
            got[i] = int(np.argmax(x[i]))
            continue
        w = np.exp((x[i] - x[i].max()) / T[i])
        kept = np.ones(s["V"], bool)
        if K[i] > 0 or P[i] < 1:
            order = np.argsort(-x[i], kind="stable")
            if K[i] > 0:
                order = order[: int(K[i])]
            if P[i] < 1:
                c = np.cumsum(w[order])
                order = order[: max(1, int(np.sum(np.concatenate([[0.0], c[:-1]]) < P[i] * c[-1])))]
            kept[:] = False
            kept[order] = True
        kept &= w >= M[i]
        c = np.cumsum(np.where(kept, w, 0.0))
        got[i] = int(np.searchsorted(c, U[i] * c[-1], side="right"))
    return torch.from_numpy(got.astype(np.int32))

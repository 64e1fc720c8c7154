"""The cases on which the operators of a step over an 8-bit cache with verified drafts are measured.

Three operators, each as a plain computation in elementary torch operations and as the call a user
makes of the library:

* ``store``: norms of a step's queries and keys for each head, the position rotation, and the append of
  keys and values to the paged cache, in the storage type or in 8 bits (e4m3) with a scale for each
  row of a slot and kv head (``pa_norm_rope_store_kv``).
* ``attn``: causal attention of one or more new tokens of each sequence over such an 8-bit cache, with or
  without a sliding window (``pa_chunk_attn_q8``).
* ``verify``: drafted tokens against the target's probabilities, from given random numbers
  (``pa_verify``).

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
E4M3 = torch.float8_e4m3fn
LEAST_SCALE = 2.0 ** -90


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of a handful of sequences, cache in the storage type: launch latency is all of it
        _store("store_decode_tiny", T=4, Hq=4, Hkv=2, D=64, bs=16, dtype="f16", q8=False),
        # a decode step of a full batch into the 8-bit cache, q, k and v as slices of one projection's
        # output; the last tokens are the padding of a captured batch size
        _store("store_decode_batch", T=256, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", fused=True, pad=5),
        # the tokens of 64 packed prompts into the 8-bit cache
        _store("store_prefill", T=33673, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", fused=True),
        # a prompt of text and images with (time, height, width) positions, cache in the storage type
        _store("store_axes_prefill", T=9001, Hq=14, Hkv=2, D=64, bs=16, dtype="f16", axes=3, q8=False, fused=True),
        # the next tokens of a few short sequences: latency
        _attn("attn_decode_tiny", S=4, q_lo=1, q_hi=1, ctx_lo=5, ctx_hi=255, Hq=4, Hkv=2, D=64, bs=16, dtype="f16", lens=1),
        # the next tokens of a full batch: the cache's bytes are all of it
        _attn("attn_decode_batch", S=256, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=4096, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", lens=2, pad=3),
        # few sequences with long caches and drafts of a few tokens: the cache has to be split
        _attn("attn_draft_long", S=3, q_lo=3, q_hi=8, ctx_lo=9000, ctx_hi=16384, Hq=14, Hkv=2, D=64, bs=16, dtype="f16", lens=3),
        # pieces of long prompts, each with what is cached of its prompt: matrix work
        _attn("attn_prefill_long", S=2, q_lo=1900, q_hi=2048, ctx_lo=12000, ctx_hi=16384, Hq=16, Hkv=8, D=128, bs=256, dtype="bf16", lens=4),
        # a layer with a sliding window, chunks of ragged prompts
        _attn("attn_window", S=12, q_lo=20, q_hi=700, ctx_lo=2000, ctx_hi=6000, Hq=32, Hkv=8, D=128, bs=16, dtype="bf16", lens=5, window=1024),
        # one request's draft of four tokens, from a drafter without probabilities (its tokens are certain)
        dict(name="verify_one", op="verify", S=1, n_lo=4, n_hi=4, V=151936, dtype="bf16", drafter="certain", lens=1),
        # the drafts of a full batch, each with its drafter's probabilities
        dict(name="verify_batch", op="verify", S=256, n_lo=0, n_hi=4, V=151936, dtype="f32", drafter="probs", lens=2),
    ]


def _store(name, T, Hq, Hkv, D, bs, dtype, q8=True, norm=True, rot=-1, axes=1, turns=False, pairs=False, fused=False, pad=0):
    return dict(name=name, op="store", T=T, Hq=Hq, Hkv=Hkv, D=D, bs=bs, dtype=dtype, q8=q8, norm=norm,
                rot=D if rot < 0 else rot, axes=axes, turns=turns, pairs=pairs, fused=fused, pad=pad)


def _attn(name, S, q_lo, q_hi, ctx_lo, ctx_hi, Hq, Hkv, D, bs, dtype, lens, window=0, pad=0):
    return dict(name=name, op="attn", S=S, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, Hq=Hq, Hkv=Hkv,
                D=D, bs=bs, dtype=dtype, lens=lens, window=window, pad=pad)


HEADS = [(4, 2), (14, 2), (16, 8), (32, 4), (6, 6), (20, 5), (16, 2), (9, 3), (5, 1)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "verify"])
    if op == "store":
        Hq, Hkv = rng.choice(HEADS)
        D = rng.choice([64, 80, 128, 128, 256])
        T = _log(rng, 1, min(33000, 33673 * 32 * 128 // ((Hq + 2 * Hkv) * D)))
        rot = D if rng.random() < 0.7 else rng.choice([0, 16, 32, 48, 64])
        c = _store("", T, Hq, Hkv, D, rng.choice([1, 16, 16, 48, 256]), rng.choice(["f16", "bf16"]), q8=rng.random() < 0.6,
                   norm=rng.random() < 0.8, rot=rot, axes=rng.choice([1, 1, 3]) if rot else 1, turns=rng.random() < 0.5,
                   pairs=rng.random() < 0.3, fused=rng.random() < 0.6, pad=min(T - 1, rng.choice([0, 0, 3, 17])))
    elif op == "attn":
        Hq, Hkv = rng.choice(HEADS)
        D = rng.choice([64, 128])
        q_hi = 1 if rng.random() < 0.3 else _log(rng, 1, 2000)
        ctx_hi = max(q_hi, _log(rng, 64, 16000))
        # the scores of the plain form in 32 bits, and the cache's rows, within the listed ones
        most = min(2 * 16 * 2048 * 16384 // (Hq * q_hi * ctx_hi), 256 * 8 * 128 * 2000 // (Hkv * D * ctx_hi))
        S = _log(rng, 1, max(1, min(300, most)))
        c = _attn("", S, rng.randint(min(q_hi, 1 - (S > 1)), q_hi), q_hi, rng.randint(1, ctx_hi), ctx_hi, Hq, Hkv, D,
                  rng.choice([16, 16, 64, 256, 24, 4]), rng.choice(["f16", "bf16"]), rng.randint(0, 9999),
                  window=0 if rng.random() < 0.6 else _log(rng, 1, 5000), pad=rng.choice([0, 0, 5]))
    else:
        V = rng.choice([32000, 50257, 128256, 151936, 262144, _log(rng, 200, 200000)])
        n_hi = rng.randint(0, 8)
        S = _log(rng, 1, max(1, min(300, 256 * 3 * 151936 // (V * (n_hi + 1)))))
        c = dict(op="verify", S=S, n_lo=rng.randint(0, n_hi), n_hi=n_hi, V=V, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                 drafter=rng.choice(["probs", "probs", "certain"]), lens=rng.randint(0, 9999))
    c.pop("name", None)
    return c


def _lengths(c):
    """(new tokens, context length with them) of each sequence of an attention case."""
    r = random.Random(c["lens"] * 7919 + c["S"])
    q = [r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["S"])]
    return q, [max(n, r.randint(c["ctx_lo"], c["ctx_hi"])) for n in q]


def _drafts(c):
    """(drafted tokens, how many of them are accepted) of each sequence of a verification case."""
    r = random.Random(c["lens"] * 7919 + c["S"])
    n = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["S"])]
    return n, [r.randint(0, k) for k in n]


def work(case):
    c = case
    if c["op"] == "store":
        T, e, D = c["T"] - c["pad"], 2, c["D"]
        rows = T if c["axes"] == 1 else min(T, 100)  # of the table: the patches of an image share theirs
        cache = 2 * c["Hkv"] * (D + 4 if c["q8"] else D * e)
        return {"bytes": T * (D * e * (2 * c["Hq"] + 2 * c["Hkv"]) + cache + 4 + 4 * c["axes"]) + rows * c["rot"] * 4,
                "flops": T * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + (4 * D if c["norm"] else 0))}
    if c["op"] == "attn":
        q, ctx = _lengths(c)
        W = c["window"]
        seen = read = 0
        for n, k in zip(q, ctx):
            if n:
                p0 = k - n
                seen += sum(min(p + 1, W) for p in range(p0, k)) if W else n * p0 + n * (n + 1) // 2
                read += k - max(0, p0 - W + 1) if W else k
        return {"bytes": 2 * read * c["Hkv"] * (c["D"] + 4) + 2 * 2 * sum(q) * c["Hq"] * c["D"] + 4 * sum(-(-k // c["bs"]) for k in ctx),
                "flops": 4 * c["D"] * c["Hq"] * seen}
    n, kept = _drafts(c)
    rejected = sum(k < m for m, k in zip(n, kept)) if c["drafter"] == "probs" else 0
    return {"bytes": (c["S"] + rejected) * c["V"] * SIZE[c["dtype"]] + 24 * (sum(n) + c["S"]), "flops": 4 * c["S"] * c["V"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _quantise(x):
    """e4m3 values and the scale of each row (the last dimension) of fp32 numbers."""
    scale = (x.abs().amax(-1) / 448.0).clamp(min=LEAST_SCALE)
    return (x / scale[..., None]).to(E4M3), scale


def _q8_pool(g, nb, bs, Hkv, D):
    """A pool of e4m3 rows and its scales [nb, Hkv, bs]; rows of different sizes, as norm weights make them."""
    x = torch.randn(nb, bs, Hkv, D, generator=g, device="cuda")
    x *= 0.5 + torch.rand(nb, bs, Hkv, 1, generator=g, device="cuda")
    x, scale = _quantise(x)
    return x, scale.transpose(1, 2).contiguous()


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
    if c["op"] == "store":
        return _prepare_store(c, g)
    if c["op"] == "attn":
        return _prepare_attn(c, g, seed)
    return _prepare_verify(c, g)


def _prepare_store(c, g):
    T, Hq, Hkv, D, dt = c["T"], c["Hq"], c["Hkv"], c["D"], DT[c["dtype"]]
    if c["fused"]:
        qkv = _normal(g, T, Hq + 2 * Hkv, D, dtype=dt)
        c["q"], c["k"], c["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        c["q"], c["k"], c["v"] = (_normal(g, T, h, D, dtype=dt) for h in (Hq, Hkv, Hkv))
    c["q_weight"], c["k_weight"] = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2))
    c["eps"] = 1e-6
    nb = -(-T // c["bs"]) + max(1, T // (4 * c["bs"]))
    if c["q8"]:
        (c["k_cache"], c["k_scale"]), (c["v_cache"], c["v_scale"]) = (_q8_pool(g, nb, c["bs"], Hkv, D) for _ in range(2))
    else:
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
    inv = 1e6 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / max(n, 1))
    a = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * inv
    c["table"] = torch.cat([a.cos(), a.sin()], 1).float()
    if c["axes"] == 1:
        start = int(torch.randint(0, 28000, (1,), generator=g, device="cuda"))
        c["positions"] = ((start + t) % 32768).to(torch.int32)
    else:  # images of 36 x 28 patches: time stands still over an image
        start = int(torch.randint(0, 20000, (1,), generator=g, device="cuda"))
        c["positions"] = torch.stack([start + t // 1008 * 36, start + t // 28 % 36, start + t % 28]).to(torch.int32)
    c["pair_axis"] = bytes(_pair_axis(c))
    c["axis_of"] = torch.tensor(_pair_axis(c), device="cuda", dtype=torch.int64)
    c["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    return c


def _prepare_attn(c, g, seed):
    S, Hq, Hkv, D, bs, dt = c["S"], c["Hq"], c["Hkv"], c["D"], c["bs"], DT[c["dtype"]]
    q, ctx = _lengths(c)
    used = [-(-k // bs) for k in ctx]
    nb = sum(used) + max(1, sum(used) // 4)
    (c["k_cache"], c["k_scale"]), (c["v_cache"], c["v_scale"]) = (_q8_pool(g, nb, bs, Hkv, D) for _ in range(2))
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
        n = pa.pa_chunk_attn_q8_workspace_size(S, Hq, Hkv, D)
        c["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return c


def _prepare_verify(c, g):
    S, V, dt = c["S"], c["V"], DT[c["dtype"]]
    n, kept = _drafts(c)
    cu = np.concatenate([[0], np.cumsum(np.array(n) + 1)])
    R = int(cu[-1])
    c["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    c["max_rows"] = max(n) + 1
    # a bulk of unlikely tokens and a few dozen likely ones, as a language model gives them; the
    # drafter's distribution lies near the target's
    x = torch.randn(R, V, generator=g, device="cuda") * 2.0
    m = min(V, 40)
    at = torch.randint(0, V, (R, m), generator=g, device="cuda")
    x.scatter_add_(1, at, 10.0 * torch.rand(R, m, generator=g, device="cuda"))
    p = torch.softmax(x, 1).to(dt)
    q = torch.softmax(x + torch.randn(R, V, generator=g, device="cuda"), 1).to(dt)
    del x
    certain = c["drafter"] == "certain"
    # the draft that a row verifies: a likely one, or where the row is to reject it, one that the drafter overrates
    row = torch.arange(R, device="cuda")
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(n, device="cuda") + 1)
    place = row - c["cu"].long()[seq]
    takes = place < torch.tensor(kept, device="cuda")[seq]
    r = 0.05 + 0.95 * torch.rand(R, V, generator=g, device="cuda")
    likely = (p.float() * r if certain else q.float() * r).argmax(1)
    overrated = likely if certain else ((q.float() - p.float()) * r).argmax(1)
    del r
    draft = torch.where(takes, likely, overrated)
    px = p[row, draft].double()
    ratio = (px / (1.0 if certain else q[row, draft].double())).clamp(max=1.0)
    u = torch.rand(R, generator=g, device="cuda").double()
    u = torch.where(takes, ratio * u * 0.999, ratio + (1 - ratio) * (0.001 + 0.998 * u))
    last = place == torch.tensor(n, device="cuda")[seq]
    c["u"] = torch.where(last, torch.rand(R, generator=g, device="cuda").double(), u).float()
    # the chunk's tokens: the last one of the text, then the drafts (row r verifies token r + 1)
    tokens = torch.randint(0, V, (R,), generator=g, device="cuda")
    tokens[1:] = torch.where(last[:-1], tokens[1:], draft[:-1])
    c["tokens"] = tokens.to(torch.int32)
    c["probs"], c["draft_probs"] = p, None if certain else q
    c["next_tokens"] = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    c["accepted"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    return c


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _stored(s):
    r = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {**r, "k_scale": s["k_scale"], "v_scale": s["v_scale"]} if s["q8"] else r


def _plain_store(s):
    T, D, R, Hkv, bs, dt = s["T"], s["D"], s["rot"], s["Hkv"], s["bs"], DT[s["dtype"]]
    n = R // 2
    pos = s["positions"].reshape(s["axes"], T)[s["axis_of"]].t().long()  # [T, n]: each pair's position
    i = torch.arange(n, device="cuda")
    cos, sin = s["table"][pos, i][:, None], s["table"][pos, n + i][:, None]

    def turned(x, weight):
        x = x.float()
        if s["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["pairs"] else (x[..., :n], x[..., n:R])
        y0, y1 = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y0, y1], -1).flatten(-2) if s["pairs"] else torch.cat([y0, y1], -1)
        return torch.cat([y, x[..., R:]], -1)

    keep = s["slots"] >= 0
    s["q_out"].copy_(torch.where(keep[:, None, None], turned(s["q"], s["q_weight"]).to(dt), s["q_out"]))
    count = T - s["pad"]  # the padding comes last
    slot = s["slots"][:count].long()
    for name, x in (("k", turned(s["k"], s["k_weight"])[:count]), ("v", s["v"][:count].float())):
        if s["q8"]:
            x, scale = _quantise(x)
            s[name + "_scale"][slot // bs, :, slot % bs] = scale
            s[name + "_cache"].view(torch.uint8).view(-1, Hkv, D)[slot] = x.view(torch.uint8)
        else:
            s[name + "_cache"].view(-1, Hkv, D)[slot] = x.to(dt)
    return _stored(s)


def _own_store(s):
    import paged_kv_cache_83_gb300 as pa
    pa.pa_norm_rope_store_kv(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"],
                             q_weight=s["q_weight"] if s["norm"] else None, k_weight=s["k_weight"] if s["norm"] else None,
                             eps=s["eps"], positions=s["positions"] if s["rot"] else None,
                             cos_sin=s["table"] if s["rot"] else None, pair_axis=s["pair_axis"] if s["axes"] > 1 else None,
                             interleaved=s["pairs"], k_scale=s["k_scale"] if s["q8"] else None,
                             v_scale=s["v_scale"] if s["q8"] else None)
    return _stored(s)


def _plain_attn(s):
    S, Hq, Hkv, D, bs, W = s["S"], s["Hq"], s["Hkv"], s["D"], s["bs"], s["window"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    if s["max_q"] == 0:
        return s["out"]
    n = cu[1:] - cu[:-1]
    r = torch.arange(s["max_q"], device="cuda")
    j = torch.arange(s["max_ctx"], device="cuda")
    valid = r < n[:, None]
    rows = torch.where(valid, cu[:-1, None] + r, 0)
    block = s["block_tables"].long()[:, j // bs].clamp(min=0)  # [S, K]
    slot = block * bs + j % bs

    def rows_of(name):
        x = s[name + "_cache"].view(torch.uint8).view(-1, Hkv, D)[slot].view(E4M3).float()
        return x * s[name + "_scale"][block, :, j % bs][..., None]

    k = rows_of("k").permute(0, 2, 3, 1)                                            # [S, Hkv, D, K]
    v = rows_of("v").permute(0, 2, 1, 3)                                            # [S, Hkv, K, D]
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


def _own_attn(s):
    import paged_kv_cache_83_gb300 as pa
    pa.pa_chunk_attn_q8(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_tables"], s["cu"],
                        s["ctx"], s["max_q"], s["scale"], window=s["window"], workspace=s["workspace"])
    return s["out"]


def _plain_verify(s):
    S, V = s["S"], s["V"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1] - 1
    r = torch.arange(s["max_rows"], device="cuda")
    row = (cu[:-1, None] + r).clamp(max=s["tokens"].numel() - 1)
    x = s["tokens"].long()[(row + 1).clamp(max=s["tokens"].numel() - 1)]
    # 64 bits: the products of the test and the sums of the weights are exact there
    px = s["probs"][row, x].double()
    qx = s["draft_probs"][row, x].double() if s["draft_probs"] is not None else torch.ones_like(px)
    takes = (s["u"].double()[row] * qx < px) & (r < n[:, None])
    a = takes.long().cumprod(1).sum(1)
    at = cu[:-1] + a
    p = s["probs"][at].float()
    if s["draft_probs"] is not None:
        d = p - s["draft_probs"][at].float()
    else:
        d = p.scatter(1, s["tokens"].long()[(at + 1).clamp(max=s["tokens"].numel() - 1)][:, None], 0.0)
    d = torch.where((a < n)[:, None], d, p).clamp(0.0, 1.0)
    w = (d.double() * 2.0 ** 44).round().long()
    bare = w.sum(1, keepdim=True) == 0  # nothing is left where the drafter is nowhere below the target
    w = torch.where(bare, (p.clamp(0.0, 1.0).double() * 2.0 ** 44).round().long(), w)
    upto = w.cumsum(1)
    # the first token whose running sum exceeds u times the whole; u in steps of 2^-31
    u = (s["u"].double()[cu[1:] - 1] * 2.0 ** 31).floor().long()[:, None]
    whole = upto[:, -1:]
    border = (whole >> 31) * u + ((whole & (2 ** 31 - 1)) * u >> 31)
    token = (upto <= border).sum(1)
    chunk = torch.where(r < a[:, None], x, torch.where(r == a[:, None], token[:, None], -1))
    mine = r <= n[:, None]
    s["next_tokens"][row[mine]] = chunk[mine].to(torch.int32)
    s["accepted"].copy_(a)
    return {"tokens": s["next_tokens"], "accepted": s["accepted"]}


def _own_verify(s):
    import paged_kv_cache_83_gb300 as pa
    pa.pa_verify(s["next_tokens"], s["accepted"], s["tokens"], s["probs"], s["cu"], s["u"], draft_probs=s["draft_probs"])
    return {"tokens": s["next_tokens"], "accepted": s["accepted"]}


_plain = {"store": _plain_store, "attn": _plain_attn, "verify": _plain_verify}
_own = {"store": _own_store, "attn": _own_attn, "verify": _own_verify}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "attn": _exact_attn, "verify": _exact_verify}[s["op"]](s)


def _exact_store(s):
    """Norms as a division by the root mean square, y = x e^(i angle) on the pairs as complex numbers, 8-bit
    values as the nearest of the finite e4m3 numbers."""
    T, n, Hkv, bs = s["T"], s["rot"] // 2, s["Hkv"], s["bs"]
    axis = s["axis_of"]
    pos = s["positions"].view(s["axes"], T)
    tab = s["table"].double()
    turn = torch.complex(tab[:, :n], tab[:, n:])
    z = torch.stack([turn[pos[int(axis[i])].long(), i] for i in range(n)], 1)[:, None] if n else None

    def turned(x, weight):
        y = x.double().clone()
        if s["norm"]:
            y = weight.double() * (y / (y.square().sum(-1, keepdim=True) / s["D"] + s["eps"]).sqrt())
        if n:
            even, odd = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if s["pairs"] else (slice(0, n), slice(n, 2 * n))
            t = torch.complex(y[..., even], y[..., odd]) * z
            y[..., even], y[..., odd] = t.real, t.imag
        return y

    kept = s["slots"] >= 0
    at = s["slots"][kept].long()
    got = {"q": s["q_out"].double().clone()}
    got["q"][kept] = turned(s["q"], s["q_weight"])[kept]
    for name, x in (("k", turned(s["k"], s["k_weight"])[kept]), ("v", s["v"].double()[kept])):
        pool = s[name + "_cache"].float().double()
        if s["q8"]:
            scale = torch.maximum(x.abs().max(-1).values / 448, torch.tensor(LEAST_SCALE, device="cuda", dtype=torch.float64))
            x = x / scale[..., None]
            # spacing 2^(e - 3) from 2^e on, 2^-9 below 2^-6
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
            scales = s[name + "_scale"].double().clone()
            scales[at // bs, :, at % bs] = scale
            got[name + "_scale"] = scales
        pool.view(-1, Hkv, s["D"])[at] = x
        got[name + "_cache"] = pool
    return got


def _exact_attn(s):
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
        block, off = (torch.from_numpy(t.astype(np.int64)).cuda() for t in (bt[i][j // bs], j % bs))
        pos, key = torch.arange(p0, n, device="cuda")[:, None], torch.arange(first, n, device="cuda")[None]
        hidden = key > pos
        if s["window"]:
            hidden |= pos - key >= s["window"]
        k8, v8 = (s[x].view(torch.uint8)[block, off].view(E4M3).float().double() for x in ("k_cache", "v_cache"))
        for g in range(s["Hkv"]):
            k = k8[:, g] * s["k_scale"][block, g, off].double()[:, None]
            v = v8[:, g] * s["v_scale"][block, g, off].double()[:, None]
            for h in range(g * G, g * G + G):
                x = (s["q"][a:b, h].double() @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
                out[a:b, h] = torch.softmax(x, 1) @ v
    return out


def _exact_verify(s):
    """Sequence by sequence in whole numbers."""
    cu, tokens, u = s["cu"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
    next_tokens, accepted = s["next_tokens"].tolist(), []
    for i in range(s["S"]):
        row, last = cu[i], cu[i + 1] - 1
        while row < last:
            x = tokens[row + 1]
            p = float(s["probs"][row, x])
            q = 1.0 if s["draft_probs"] is None else float(s["draft_probs"][row, x])
            if not u[row] * q < p:
                break
            next_tokens[row] = x
            row += 1
        p = s["probs"][row].float().cpu().numpy()
        d = p.copy()
        if row < last:
            if s["draft_probs"] is None:
                d[tokens[row + 1]] = 0
            else:
                d -= s["draft_probs"][row].float().cpu().numpy()
        w = np.rint(np.clip(d, 0, 1).astype(np.float64) * 2.0 ** 44).astype(np.int64)
        if not w.any():
            w = np.rint(np.clip(p, 0, 1).astype(np.float64) * 2.0 ** 44).astype(np.int64)
        upto = np.cumsum(w)
        border = int(upto[-1]) * int(u[last] * 2.0 ** 31) >> 31
        next_tokens[row] = int(np.searchsorted(upto, border, side="right"))
        next_tokens[row + 1:last + 1] = [-1] * (last - row)
        accepted.append(row - cu[i])
    return {"tokens": torch.tensor(next_tokens, dtype=torch.int32), "accepted": torch.tensor(accepted, dtype=torch.int32)}

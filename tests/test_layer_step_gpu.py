"""The operators together, as an engine runs them: blocks from the block manager, prompts in chunks and
drafts of several tokens beside single decode tokens, each step rotation + append, attention over the cache,
logits and a sampled token. Attention is checked against 64-bit attention over the whole history, the
cache against the other entry points, tokens against the definition on the step's own logits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa
from tests.test_rope_store_gpu import table
from tests.test_sample_gpu import choose

pytestmark = pytest.mark.gpu

V = 500


class Model:
    """One attention layer over random embeddings: q, k, v of a token depend on its id alone."""

    def __init__(self, Hq, Hkv, D, dt, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.dt = Hq, Hkv, D, dt
        self.qkv = torch.randn(V, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
        self.head = (torch.randn(Hq * D, V, generator=g, device="cuda") * 0.1).to(dt)
        self.cos_sin = table(4096, D)

    def rotated(self, x, pos):
        n = self.D // 2
        c, s = self.cos_sin[pos, :n].double()[:, None], self.cos_sin[pos, n:].double()[:, None]
        a, b = x[..., :n].double(), x[..., n:].double()
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def attention(self, ids, first):
        """64-bit rows of tokens first .. of a whole sequence of ids, keys rounded as the cache holds them."""
        ids = torch.tensor(ids, device="cuda")
        pos = torch.arange(len(ids), device="cuda")
        x = self.qkv[ids]
        G = self.Hq // self.Hkv
        q = self.rotated(x[:, :self.Hq], pos).to(self.dt).double()[first:]
        k = self.rotated(x[:, self.Hq:self.Hq + self.Hkv], pos).to(self.dt).double().repeat_interleave(G, 1)
        v = x[:, self.Hq + self.Hkv:].double().repeat_interleave(G, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) * self.D ** -0.5
        s = s.masked_fill(pos > pos[first:, None], -torch.inf)
        return torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v)


@pytest.mark.parametrize("Hq,Hkv,D,bs,dt", [(16, 8, 128, 256, torch.bfloat16), (14, 2, 64, 16, torch.float16),
                                            (4, 4, 64, 4, torch.float16)])
def test_prompts_in_chunks_then_drafts_then_single_tokens(Hq, Hkv, D, bs, dt):
    m = Model(Hq, Hkv, D, dt)
    r = np.random.default_rng(D + bs)
    nb = 4000 // bs + 8
    bm = pa.BlockManager(nb, bs)
    kc, vc = (torch.full((nb, bs, Hkv, D), float("nan"), device="cuda", dtype=dt) for _ in range(2))
    seqs = {s: [int(t) for t in r.integers(0, V, n)] for s, n in ((0, 700), (1, 33), (2, 261))}
    done = {}
    for s, ids in seqs.items():
        done[s] = 0
        bm.allocate(s, ids)
    ws = torch.empty(pa.pa_chunk_attn_workspace_size(4, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # With u = eps / 2 and values under 5: P's rounding moves a row by at most 5 u, the output's by 5 u. The
    # kernel rotates in fp32, the reference in 64 bits, so that a q or k element may round to its other
    # neighbour (2 u of itself): one score in some thousand by up to 2 u 4 4 / sqrt(D), which moves an
    # output by under 5 u. The fp32 sums add under u.
    tol = 20 * torch.finfo(dt).eps / 2
    for step in range(8):
        # how many tokens each sequence feeds: pieces of its prompt, then 1 to 5 at the end (drafts)
        feed = {s: min(len(ids) - done[s], (300, 150, 64)[s] if step < 4 else 5) for s, ids in seqs.items()}
        tables = [bm.block_table(s) for s in seqs]
        bt = np.full((4, max(map(len, tables))), -1, np.int32)
        tok, pos, slots, cu = [], [], [], [0]
        for i, (s, ids) in enumerate(seqs.items()):
            bt[i, :len(tables[i])] = tables[i]
            for p in range(done[s], done[s] + feed[s]):
                tok.append(ids[p])
                pos.append(p)
                slots.append(tables[i][p // bs] * bs + p % bs)
            cu.append(cu[-1] + feed[s])
        cu.append(cu[-1])  # a padded batch: a sequence without tokens, and padding tokens behind
        n, pad = len(tok), 3
        ctx = [done[s] + feed[s] for s in seqs] + [0]
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        x = m.qkv[torch.tensor(tok + [0] * pad, device="cuda")]
        q = torch.full((n + pad, Hq, D), 9.0, device="cuda", dtype=dt)
        out = torch.full_like(q, 9.0)
        pa.pa_rope_store_kv(q, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, i32(slots + [-1] * pad),
                            i32(pos + [0] * pad), m.cos_sin, err=err)
        pa.pa_chunk_attn(out, q, kc, vc, i32(bt), i32(cu), i32(ctx), max(1, *feed.values()), D ** -0.5, workspace=ws,
                         err=err)
        rows = [cu[i + 1] - 1 for i, s in enumerate(seqs) if feed[s]]
        logits = out[rows].view(len(rows), -1).float() @ m.head.float()
        u = torch.tensor(r.uniform(0, 1, len(rows)), dtype=torch.float32, device="cuda")
        T = i32([0] * len(rows)).float() + 0.7
        tokens = i32([-1] * len(rows))
        pa.pa_sample(tokens, logits, u, temperature=T, top_k=i32([40] * len(rows)), top_p=T + 0.2, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert (out[n:] == 9).all() and (q[n:] == 9).all()
        want = [choose(logits[b].double().cpu().numpy(), T=np.float32(0.7), k=40, p=float((T + 0.2)[0]), u=float(u[b]))
                for b in range(len(rows))]
        assert tokens.tolist() == want
        b = 0
        for i, (s, ids) in enumerate(seqs.items()):
            if not feed[s]:
                continue
            ref = m.attention(ids[:done[s] + feed[s]], done[s])
            assert float((out[cu[i]:cu[i + 1]].double() - ref).abs().max()) <= tol, (step, s)
            done[s] += feed[s]
            if done[s] == len(ids):  # the token, and from step 4 on a draft of more behind it
                for t in [int(tokens[b])] + [int(t) for t in r.integers(0, V, (0 if step < 4 else 4))]:
                    bm.append(s, t)
                    ids.append(t)
            b += 1
    # the last state through the other entry points: one prefill of a whole sequence over the pool
    s = 0
    ids = seqs[s][:done[s]]
    x = m.qkv[torch.tensor(ids, device="cuda")]
    q = m.rotated(x[:, :Hq], torch.arange(len(ids), device="cuda")).to(dt).contiguous()
    out = torch.empty_like(q)
    cu = torch.tensor([0, len(ids)], dtype=torch.int32, device="cuda")
    bt = torch.tensor([bm.block_table(s)], dtype=torch.int32, device="cuda")
    pa.pa_prefill_varlen(out, q, None, None, kc, vc, cu, cu, len(ids), len(ids), bt, Hkv=Hkv, scale=D ** -0.5)
    torch.cuda.synchronize()
    assert float((out.double() - m.attention(ids, 0)).abs().max()) <= tol


class Overlap:
    """A rotation of several waves and the attention that reads its queries and pool rows, with nothing between
    the two calls: the attention's kernels may start while the rotation's last blocks run."""

    def __init__(self, form, D, bs, dt, seed):
        # query rows a kv head: whole chunks (128-row tiles), or up to 16, 32 and 64
        Hq, Hkv, q, S = {"wide": (16, 8, 700, 16), "rows16": (16, 8, 8, 1400), "rows32": (8, 2, 8, 1400),
                         "rows64": (8, 1, 8, 1400)}[form]
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        ctx = q + r.integers(0, 60, S)
        used = -(-ctx // bs)
        nb = int(used.sum()) + 2
        ids = r.permutation(nb)
        bt = np.zeros((S, used.max()), np.int64)
        slots, pos, at = [], [], 0
        for s in range(S):
            bt[s, :used[s]] = ids[at:at + used[s]]
            at += used[s]
            p = np.arange(ctx[s] - q, ctx[s])
            slots.append(bt[s, p // bs] * bs + p % bs)
            pos.append(p)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        self.slots, self.pos, self.bt, self.ctx = i32(np.concatenate(slots)), i32(np.concatenate(pos)), i32(bt), i32(ctx)
        self.cu = i32(np.arange(S + 1) * q)
        n, self.most, self.scale = S * q, q, D ** -0.5
        x = torch.randn(n, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
        self.qkv = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        self.base = [torch.randn(nb, bs, Hkv, D, generator=g, device="cuda").to(dt) for _ in range(2)]
        for pool in self.base:
            pool.view(-1, Hkv, D)[self.slots.long()] = float("nan")
        self.pools = [torch.empty_like(p) for p in self.base]
        self.q = torch.empty(n, Hq, D, dtype=dt, device="cuda")
        self.out = torch.empty_like(self.q)
        self.table = table(1024, D)
        self.ws = torch.empty(pa.pa_chunk_attn_workspace_size(S, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def poison(self):
        for pool, base in zip(self.pools, self.base):
            pool.copy_(base)
        self.q.fill_(float("nan"))
        self.out.fill_(float("nan"))
        torch.cuda.synchronize()

    def rotate(self):
        pa.pa_rope_store_kv(self.q, *self.qkv, *self.pools, self.slots, self.pos, self.table, err=self.err)

    def attend(self):
        pa.pa_chunk_attn(self.out, self.q, *self.pools, self.bt, self.cu, self.ctx, self.most, self.scale, workspace=self.ws,
                         err=self.err)

    def result(self):
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        return self.out.clone()


@pytest.mark.parametrize("bs", [16, 4])
@pytest.mark.parametrize("D,dt", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("form", ["wide", "rows16", "rows32", "rows64"])
def test_attention_directly_behind_its_rotation(form, D, dt, bs):
    o = Overlap(form, D, bs, dt, D + bs)
    o.poison()
    o.rotate()
    torch.cuda.synchronize()
    o.attend()
    want = o.result()
    assert torch.isfinite(want).all()
    for _ in range(15):
        o.poison()
        o.rotate()
        o.attend()
        assert torch.equal(o.result(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o.rotate()
        o.attend()
    for _ in range(15):
        o.poison()
        g.replay()
        assert torch.equal(o.result(), want)


@pytest.mark.parametrize("Hq,Hkv,D,dt,B,most", [(16, 8, 128, torch.bfloat16, 5000, 250), (14, 2, 64, torch.float16, 5000, 250),
                                                (16, 8, 128, torch.bfloat16, 700, 2000), (14, 2, 64, torch.float16, 900, 2000)])
def test_decode_directly_behind_its_rotation(Hq, Hkv, D, dt, B, most):
    """Single tokens: pa_decode's kernels (short tables and long ones) start beside the rotation too."""
    bs = 16
    g = torch.Generator(device="cuda").manual_seed(B)
    r = np.random.default_rng(B)
    ctx = r.integers(1, most, B)
    used = -(-ctx // bs)
    nb = int(used.sum())
    ids, at = r.permutation(nb), 0
    bt = np.zeros((B, -(-most // bs)), np.int64)
    for b in range(B):
        bt[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = i32(bt[np.arange(B), (ctx - 1) // bs] * bs + (ctx - 1) % bs)
    btd, cl, pos, cos_sin = i32(bt), i32(ctx), i32(ctx - 1), table(most, D)
    x = torch.randn(B, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
    base = [torch.randn(nb, bs, Hkv, D, generator=g, device="cuda").to(dt) for _ in range(2)]
    for pool in base:
        pool.view(-1, Hkv, D)[slots.long()] = float("nan")
    pools = [torch.empty_like(p) for p in base]
    q = torch.empty(B, Hq, D, dtype=dt, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(max(16, pa.pa_decode_workspace_size(B, Hq, Hkv, D, bt.shape[1], bs)), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(apart):
        for pool, b in zip(pools, base):
            pool.copy_(b)
        q.fill_(float("nan")), out.fill_(float("nan"))
        torch.cuda.synchronize()
        pa.pa_rope_store_kv(q, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *pools, slots, pos, cos_sin, err=err)
        if apart:
            torch.cuda.synchronize()
        pa.pa_decode(out, q, *pools, btd, cl, D ** -0.5, workspace=ws, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return out.clone()

    want = step(True)
    assert torch.isfinite(want).all()
    for _ in range(10):
        got = step(False)
        assert torch.isfinite(got).all()
        # the split form hands its last units out as CTAs come free, so that sums may be joined in another order
        assert float((got.double() - want.double()).abs().max()) <= (4e-3 if dt == torch.float16 else 2e-2)


def test_layers_in_a_row():
    """Layer by layer into the same buffers, nothing between the calls: a layer's rotation must not overtake the
    attention that still reads them."""
    layers = [Overlap(form, 128, 16, torch.bfloat16, 40 + i) for i, form in enumerate(["wide", "rows16", "wide", "rows16"])]
    for a, b in zip(layers, layers[2:]):  # the same shapes: one q, one set of pools' room, one workspace
        b.q, b.ws = a.q, a.ws
    want = []
    for o in layers:
        o.poison()
        o.rotate()
        torch.cuda.synchronize()
        o.attend()
        want.append(o.result())
    for _ in range(10):
        for o in layers:
            o.poison()
        for o in layers:
            o.rotate()
            o.attend()
        for o, w in zip(layers, want):
            assert torch.equal(o.result(), w)


def test_lengths_and_tables_from_a_kernel_that_lets_its_dependents_start():
    """The rotation lets what follows start early. Here its output, bit for bit its input (cosines 1, sines 0), is the
    attention's lengths and page table, written by its last blocks; what lies there before is valid and empty."""
    T, S, Hq, Hkv, D, bs = 60000, 20, 4, 2, 64, 16
    r = np.random.default_rng(5)
    for q in (3, 200):
        ctx = q + r.integers(0, 512 - 200, S)
        bt = r.permutation(S * 32).reshape(S, 32)
        words = torch.zeros(T, 32, dtype=torch.int32)
        words[T - S:] = torch.from_numpy(bt)
        words[T - S - 1, :S] = torch.from_numpy(ctx)
        words[T - S - 2, :S + 1] = torch.arange(S + 1) * q
        words = words.cuda()
        moved = torch.zeros_like(words)
        src, dst = (w.view(torch.float16).view(T, 1, D) for w in (words, moved))
        kc, vc = (torch.randn(S * 32, bs, Hkv, D, device="cuda").half() for _ in range(2))
        k, sink = torch.zeros(T, 1, D, device="cuda").half(), torch.zeros(T // 16, 16, 1, D, device="cuda").half()
        spare = torch.zeros_like(sink)
        slots, first = torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
        turn = torch.cat([torch.ones(1, 8), torch.zeros(1, 8)], 1).cuda()
        x = torch.randn(S * q, Hq, D, device="cuda").half()
        out = torch.zeros_like(x)
        ws = torch.empty(pa.pa_chunk_attn_workspace_size(S, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")

        def attend(w):
            pa.pa_chunk_attn(out, x, kc, vc, w[T - S:], w[T - S - 2, :S + 1], w[T - S - 1, :S], q, D ** -0.5, workspace=ws, err=err)

        attend(words)
        torch.cuda.synchronize()
        want = out.clone()
        assert int(err.item()) == 0 and (want != 0).any(-1).all()
        for _ in range(20):
            moved.zero_()
            out.zero_()
            torch.cuda.synchronize()
            pa.pa_rope_store_kv(dst, src, k, k, sink, spare, slots, first, turn, err=err)
            attend(moved)
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            assert torch.equal(moved, words)
            assert torch.equal(out, want)


def test_attention_between_other_kernels_that_use_tensor_memory():
    """Matrix products, prefill and chunk attention behind one another, on one stream and on two, and captured."""
    layers = [Overlap(form, D, 16, torch.bfloat16, 60 + i) for i, (form, D) in
              enumerate([("wide", 128), ("rows16", 64), ("wide", 64), ("rows64", 128)])]
    want = []
    for o in layers:
        o.poison()
        o.rotate()
        o.attend()
        want.append(o.result())
    a = torch.randn(2048, 2048, device="cuda").bfloat16()
    c = torch.empty_like(a)
    torch.matmul(a, a, out=c)
    cwant = c.clone()
    cu = torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
    x = torch.randn(3000, 16 + 2 * 8, 128, device="cuda").bfloat16()
    q, k, v = (t.contiguous() for t in (x[:, :16], x[:, 16:24], x[:, 24:]))
    p = torch.empty_like(q)

    def prefill():
        pa.pa_prefill_varlen(p, q, k, v, None, None, cu, cu, 3000, 3000, None, Hkv=8, scale=128 ** -0.5)

    prefill()
    torch.cuda.synchronize()
    pwant = p.clone()

    def step(beside=None):
        for o in layers:
            o.rotate()
            torch.matmul(a, a, out=c)
            o.attend()
            if beside is None:
                torch.matmul(a, a, out=c)
                prefill()
            else:
                with torch.cuda.stream(beside):
                    prefill()

    def same():
        torch.cuda.synchronize()
        for o, w in zip(layers, want):
            assert torch.equal(o.result(), w)
        assert torch.equal(c, cwant) and torch.equal(p, pwant)

    side = torch.cuda.Stream()
    for beside in (None, side):
        for _ in range(10):
            for o in layers:
                o.poison()
            c.zero_(), p.zero_()
            torch.cuda.synchronize()
            step(beside)
            same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(10):
        for o in layers:
            o.poison()
        g.replay()
        same()

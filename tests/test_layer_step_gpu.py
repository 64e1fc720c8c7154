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

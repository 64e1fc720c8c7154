"""The operators of an 8-bit cache together, as an engine runs them: steps of norms + rotation + append, attention over the cache,
probabilities and verification of drafts, each directly behind the one whose output it reads, over prompts in chunks, drafts and
single tokens. The cache is checked against the definition, attention against 64 bits over the values that the cache stands for,
tokens against the definition on the step's own probabilities."""
import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa
from tests.test_norm_rope_store_gpu import near8, normed, turned
from tests.test_rope_store_gpu import table
from tests.test_verify_gpu import choose

pytestmark = pytest.mark.gpu

V = 300
E4M3 = torch.float8_e4m3fn


class Engine:
    """One attention layer over random embeddings, with sequences in a paged 8-bit cache; what has not been written is NaN."""

    def __init__(self, Hq, Hkv, D, bs, dt, lens, room, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.bs, self.dt = Hq, Hkv, D, bs, dt
        self.qkv = torch.randn(V, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dt)
        self.qw, self.kw = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2))
        self.head = torch.randn(Hq * D, V, generator=g, device="cuda").to(dt)
        self.tab = table(4096, D)
        S, maxb = len(lens), -(-room // bs)
        nb = S * maxb + 2
        self.kc, self.vc = (torch.full((nb, bs, Hkv, D), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
        self.ks, self.vs = (torch.full((nb, Hkv, bs), float("nan"), device="cuda") for _ in range(2))
        self.bt = torch.from_numpy(np.random.default_rng(seed).permutation(nb)[:S * maxb].reshape(S, maxb).astype(np.int32)).cuda()
        self.done = [0] * S                     # tokens whose keys are in the cache
        self.ids = [list(map(int, np.random.default_rng(seed + s).integers(0, V, n))) for s, n in enumerate(lens)]
        self.ws = torch.empty(pa.pa_chunk_attn_q8_workspace_size(S, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, chunks, pad=0):
        """Runs the chunk of tokens of each sequence behind what is cached; the output rows."""
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        n = [len(c) for c in chunks]
        bt = self.bt.tolist()
        pos = [self.done[s] + i for s, k in enumerate(n) for i in range(k)] + [0] * pad
        slots = [bt[s][p // self.bs] * self.bs + p % self.bs for s, k in enumerate(n) for p in range(self.done[s], self.done[s] + k)]
        self.tokens = i32([t for c in chunks for t in c] + [0] * pad)
        self.slots, self.pos = i32(slots + [-1] * pad), i32(pos)
        self.cu, self.ctx, self.max_q = i32(np.concatenate([[0], np.cumsum(n)])), i32([d + k for d, k in zip(self.done, n)]), max(n)
        self.x = self.qkv[self.tokens.long()]
        self.q, self.out = (torch.zeros(len(pos), self.Hq, self.D, dtype=self.dt, device="cuda") for _ in range(2))
        self.launch()
        return n

    def launch(self):
        Hq, Hkv = self.Hq, self.Hkv
        pa.pa_norm_rope_store_kv(self.q, self.x[:, :Hq], self.x[:, Hq:Hq + Hkv], self.x[:, Hq + Hkv:], self.kc, self.vc, self.slots,
                                 self.qw, self.kw, 1e-6, self.pos, self.tab, k_scale=self.ks, v_scale=self.vs, err=self.err)
        pa.pa_chunk_attn_q8(self.out, self.q, self.kc, self.vc, self.ks, self.vs, self.bt, self.cu, self.ctx, self.max_q,
                            self.D ** -0.5, workspace=self.ws, err=self.err)

    def cached(self, pool, scale, s, n):
        p = torch.arange(n, device="cuda")
        block = self.bt[s].long()[p // self.bs]
        rows = pool.view(torch.uint8)[block, p % self.bs].view(E4M3)
        return rows, scale[block, :, p % self.bs]

    def check(self, n, full):
        """The step's outputs, and with `full` the whole cache of every sequence."""
        torch.cuda.synchronize()
        assert int(self.err) == 0
        G = self.Hq // self.Hkv
        cu = self.cu.tolist()
        for s, k in enumerate(n):
            upto = self.done[s] + k
            (kr, ksc), (vr, vsc) = self.cached(self.kc, self.ks, s, upto), self.cached(self.vc, self.vs, s, upto)
            if full:
                x = self.qkv[torch.tensor(self.ids[s][:upto], device="cuda")]
                p = torch.arange(upto, device="cuda", dtype=torch.int32)[None]
                want = turned(normed(x[:, self.Hq:self.Hq + self.Hkv], self.kw, 1e-6), p, self.tab, [0] * (self.D // 2), False)
                near8(kr, ksc, want)
                near8(vr, vsc, x[:, self.Hq + self.Hkv:].double())
            if not k:
                continue
            kk, vv = ((r.float().double() * sc.double()[..., None]).repeat_interleave(G, 1) for r, sc in ((kr, ksc), (vr, vsc)))
            q = self.q[cu[s]:cu[s] + k].double()
            j = torch.arange(upto, device="cuda")
            sc = torch.einsum("qhd,khd->hqk", q, kk) * self.D ** -0.5
            w = torch.softmax(sc.masked_fill(j > torch.arange(self.done[s], upto, device="cuda")[:, None], -torch.inf), -1)
            want = torch.einsum("hqk,khd->qhd", w, vv)
            got = self.out[cu[s]:cu[s] + k].double()
            assert not got.isnan().any()
            # (as in the operator's own test)
            assert float((got - want).norm()) <= 2.0 ** -8 * float(want.norm())

    def probs(self):
        return torch.softmax((self.out.view(len(self.out), -1).float() @ self.head.float()) * 0.05, 1)


@pytest.mark.parametrize("Hq,Hkv,D,bs,dt", [(16, 8, 128, 256, torch.bfloat16), (14, 2, 64, 16, torch.float16), (4, 4, 64, 4, torch.bfloat16),
                                            (8, 1, 128, 16, torch.float16)])
def test_prompts_in_chunks_then_verified_drafts(Hq, Hkv, D, bs, dt):
    lens = [700, 33, 261, 1]
    e = Engine(Hq, Hkv, D, bs, dt, lens, 900, seed=D + bs)
    r = np.random.default_rng(bs)
    # the prompts but for their last token, in chunks of 300
    while any(d < n - 1 for d, n in zip(e.done, lens)):
        n = e.step([e.ids[s][d:min(d + 300, lens[s] - 1)] for s, d in enumerate(e.done)], pad=2)
        e.check(n, full=False)
        e.done = [d + k for d, k in zip(e.done, n)]
    accepted = 0
    for turn in range(6):
        drafts = [[int(t) for t in r.integers(0, V, r.integers(0, 5))] for _ in lens]
        if turn == 4:
            drafts = [[] for _ in lens]  # single tokens
        e.step([[e.ids[s][-1]] + drafts[s] for s in range(len(lens))])
        p = e.probs()
        q = torch.full_like(p, 1.0 / V)
        u = torch.rand(len(p), generator=torch.Generator().manual_seed(turn)).cuda()
        u[1::3] *= 0.05  # that some drafts stand
        nxt, acc = torch.full_like(e.tokens, -7), torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        pa.pa_verify(nxt, acc, e.tokens, p, e.cu, u, draft_probs=q, err=e.err)
        n = [len(d) + 1 for d in drafts]
        for s in range(len(lens)):
            e.ids[s] += drafts[s]
        e.check(n, full=True)
        cu, got, count = e.cu.tolist(), nxt.tolist(), acc.tolist()
        pn, qn, un = p.cpu().numpy(), q.cpu().numpy(), u.cpu().numpy()
        for s in range(len(lens)):
            a, b = cu[s], cu[s + 1]
            k, row = choose(pn[a:b], qn[a:b], e.tokens.tolist()[a:b], un[a:b], V)
            assert (count[s], got[a:b]) == (k, row)
            # what was refused is overwritten in the next step
            e.ids[s] = e.ids[s][:len(e.ids[s]) - len(drafts[s])] + row[:k + 1]
            e.done[s] += k + 1
            accepted += k
    assert accepted > 0


def test_a_captured_step_replayed_with_other_inputs():
    lens = [300, 40, 120]
    a, b = (Engine(16, 8, 128, 64, torch.bfloat16, lens, 400, seed=5) for _ in range(2))
    for e in (a, b):
        e.done = [0, 0, 0]
        n = e.step([i[:-1] for i in e.ids])
        e.done = [k for k in n]
    u = torch.rand(9, generator=torch.Generator().manual_seed(1)).cuda() * 0.3
    first = [[i[-1], 5, 6] for i in a.ids]
    a.step(first)  # (the buffers that the graph will use)
    nxt, acc = torch.full_like(a.tokens, -7), torch.zeros(3, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.launch()
        p = a.probs()
        pa.pa_verify(nxt, acc, a.tokens, p, a.cu, u, err=a.err)
    for turn, more in enumerate((first, [[7, 8, 9], [1, 2, 3], [250, 251, 252]])):
        b.step(more)
        for name in ("tokens", "slots", "pos", "cu", "ctx", "x"):
            getattr(a, name).copy_(getattr(b, name))
        graph.replay()
        nb, ab = torch.full_like(b.tokens, -7), torch.zeros(3, dtype=torch.int32, device="cuda")
        pa.pa_verify(nb, ab, b.tokens, b.probs(), b.cu, u, err=b.err)
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and torch.equal(nxt, nb) and torch.equal(acc, ab)
        assert torch.equal(a.kc.view(torch.uint8), b.kc.view(torch.uint8)) and int(a.err) == int(b.err) == 0
        b.done = [d + 3 for d in b.done]

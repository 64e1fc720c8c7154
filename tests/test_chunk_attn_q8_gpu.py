"""pa_chunk_attn_q8 on the GPU against softmax attention in 64 bits over the values that the cache stands for.

Bounds, with u = finfo.eps / 2 of the output's type and A = sum_j softmax_j |v_j| of an element:
* a weight is held in two e4m3 numbers of four bits each: off by 2^-8 of itself, or by 2^-16 where the largest weight under the
  first keys' reference is 2^4: the reference lies at most 8 + 4 above 2^-20 of a later largest, so that
  this is 2^-20 of the largest weight * scale per key;
* a query's element is exact above 2^-14 of its row's largest, below that off by 2^-24 (bf16) of it: D 2^-24 max|q| max|k| scale,
  natural units, beside the fp32 sums of D products in D / 32 instructions per piece, each off by 2^-22 of sum |q k| scale, 16
  in all; a score that is off by e_s moves the output by 2 e_s A;
* the fp32 sums over n keys, the exponentials and logarithms by (n / 16 + 16) 2^-22 A;
* the output is rounded once, u |out|."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
NAN = float("nan")


class Case:
    """Sequences of (new tokens, context length); the pool's unused slots, their scales and every table entry that
    is not to be read are filled with what would be seen: NaN and -1 (or an index far outside)."""

    def __init__(self, lens, Hq, Hkv, D, bs, dt, window=0, pad=0, seed=0, lead=0, max_q=None, width=None, sizes=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        self.lens, self.D, self.Hq, self.Hkv, self.bs, self.window, self.dt = lens, D, Hq, Hkv, bs, window, DT[dt]
        S = len(lens)
        used = [-(-n // bs) for _, n in lens]
        nb = sum(used) + 3
        self.kc, self.vc = (torch.full((nb, bs, Hkv, D), 0x7f, device="cuda", dtype=torch.uint8) for _ in range(2))
        self.ks, self.vs = (torch.full((nb, Hkv, bs), NAN, device="cuda") for _ in range(2))
        ids = r.permutation(nb)
        bt = np.full((S, width or max(used + [1])), -1, np.int64)
        bt[:, 1::2] = 1 << 30
        at = 0
        for s, (q, n) in enumerate(lens):
            first = max(0, n - q - window + 1) if window else 0
            mine = ids[at:at + used[s]]
            at += used[s]
            for b in range(first // bs, used[s]):
                bt[s, b] = mine[b]
            j = torch.arange(first, n, device="cuda")
            block = torch.from_numpy(mine).cuda()[j // bs]
            for pool, scale in ((self.kc, self.ks), (self.vc, self.vs)):
                x = torch.randn(n - first, Hkv, D, generator=g, device="cuda")
                x *= torch.exp2(sizes * torch.randn(n - first, Hkv, 1, generator=g, device="cuda") - 1)
                sc = (x.abs().amax(-1) / 448).clamp(min=2.0 ** -90)
                pool[block, j % bs] = (x / sc[..., None]).to(E4M3).view(torch.uint8)
                scale[block, :, j % bs] = sc
        self.kc, self.vc = self.kc.view(E4M3), self.vc.view(E4M3)
        self.bt = torch.from_numpy(bt.astype(np.int32)).cuda()
        self.cu = torch.tensor(lead + np.concatenate([[0], np.cumsum([q for q, _ in lens])]), dtype=torch.int32, device="cuda")
        self.ctx = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda")
        self.Tq = lead + sum(q for q, _ in lens) + pad
        self.max_q = max([q for q, _ in lens]) if max_q is None else max_q
        self.q = torch.randn(self.Tq, Hq, D, generator=g, device="cuda").to(self.dt)
        self.out = torch.full((self.Tq, Hq, D), 7.0, device="cuda", dtype=self.dt)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5
        n = pa.pa_chunk_attn_q8_workspace_size(S, Hq, Hkv, D)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere

    def run(self, **kw):
        pa.pa_chunk_attn_q8(self.out, self.q, self.kc, self.vc, self.ks, self.vs, self.bt, self.cu, self.ctx, self.max_q, self.scale,
                            window=self.window, workspace=self.ws, err=self.err, **kw)

    def rows(self, pool, scale, s, j):
        block = self.bt[s].long()[j // self.bs]
        x = pool.view(torch.uint8)[block, j % self.bs].view(E4M3).float().double()
        return (x * scale[block, :, j % self.bs].double()[..., None]).repeat_interleave(self.Hq // self.Hkv, 1)

    def reference(self, s):
        """(output in 64 bits, bound) of sequence s: [q, Hq, D]."""
        q, n = self.lens[s]
        first = max(0, n - q - self.window + 1) if self.window else 0
        a = int(self.cu[s])
        j = torch.arange(first, n, device="cuda")
        k, v = self.rows(self.kc, self.ks, s, j), self.rows(self.vc, self.vs, s, j)
        x = self.q[a:a + q].double()
        pos = torch.arange(n - q, n, device="cuda")[:, None]
        hidden = (j > pos) | ((pos - j >= self.window) if self.window else False)
        sc = torch.einsum("qhd,khd->hqk", x, k) * self.scale
        w = torch.softmax(sc.masked_fill(hidden, -torch.inf), -1)
        size = (torch.einsum("qhd,khd->hqk", x.abs(), k.abs()) * self.scale).masked_fill(hidden, 0).amax(-1)
        lost = x.abs().amax(-1).t() * k.abs().amax(-1).amax(0)[:, None] * self.D * 2.0 ** -24 * self.scale  # [Hq, q]
        out, A = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
        u = torch.finfo(self.dt).eps / 2
        e_s = (16 * 2.0 ** -22 * size + lost).t()[..., None]
        bound = A * (2.0 ** -8 + 2 * e_s + (n / 16 + 16) * 2.0 ** -22)
        # weights below 2^-20 of the largest (weight * scale of its value): each is off by that, times an e4m3 number of at most 448
        vscale = (v.abs().amax(-1) / 448).t()  # [Hq, k]
        bound = bound + ((w * vscale[:, None]).amax(-1) * 448 * (n - first) * 2.0 ** -20).t()[..., None] * (v.abs() > 0).any(0)[None]
        return out, bound + u * (out.abs() + bound) + torch.finfo(self.dt).smallest_normal * u

    def check(self, zero=(), run=True):
        if run:
            self.run()
        torch.cuda.synchronize()
        lo, hi = int(self.cu[0]), int(self.cu[-1])
        assert (self.out[:lo] == 7).all() and (self.out[hi:] == 7).all()  # outside every sequence
        for s, (q, _) in enumerate(self.lens):
            got = self.out[int(self.cu[s]):int(self.cu[s]) + q].double()
            if s in zero:
                assert (got == 0).all(), s
            elif q:
                ref, bound = self.reference(s)
                bad = (got - ref).abs() - bound
                assert not torch.isnan(got).any(), s
                assert (bad <= 0).all(), (s, float(bad.max()), float((got - ref).abs().max()))
                # and as a whole: a rounding of two pieces is off by 2^-8 / sqrt(3) of a weight at most in the mean
                # square, the output's by u / sqrt(3); weights and roundings are independent
                off, norm = float((got - ref).norm()), float(ref.norm())
                assert off <= 2.0 ** -8 * norm, (s, off / norm)
        return self


@pytest.mark.parametrize("lens,Hq,Hkv,D,bs,dt,kw", [
    ([(1, 1)], 1, 1, 64, 16, "f16", {}),
    ([(1, 1)], 1, 1, 128, 16, "bf16", {}),
    ([(1, 1), (1, 17), (3, 100), (5, 255)], 4, 2, 64, 16, "f16", {}),
    ([(4, 4), (0, 50), (7, 130), (1, 128), (2, 129)], 16, 8, 128, 256, "bf16", dict(pad=5)),
    ([(3, 9000)], 14, 2, 64, 16, "f16", {}),                  # one long cache over all SMs
    ([(8, 5003), (1, 16000), (2, 700)], 16, 8, 128, 256, "bf16", {}),
    ([(128, 128), (129, 129), (127, 400), (257, 1025), (64, 64)], 8, 4, 128, 16, "bf16", {}),
    ([(300, 2000), (1, 3000), (1, 40), (77, 77)], 14, 2, 64, 16, "f16", dict(pad=3, lead=2)),
    ([(50, 333)], 3, 1, 128, 8, "bf16", {}),
    ([(41, 333), (90, 100)], 5, 1, 64, 24, "bf16", {}),       # boxes of 8 rows
    ([(33, 600), (18, 18), (19, 300)], 14, 2, 128, 64, "f16", {}),
    ([(1, 500), (2, 60), (9, 301)], 8, 1, 128, 4, "bf16", {}),  # rows gathered one by one
    ([(70, 500), (1, 60)], 4, 4, 64, 1, "f16", {}),
    ([(6, 700), (3, 95)], 6, 6, 64, 20, "bf16", {}),
    ([(1, 4096)] * 3 + [(1, 5)] * 40, 32, 4, 128, 128, "f16", {}),
])
def test_against_64_bits(lens, Hq, Hkv, D, bs, dt, kw):
    assert int(Case(lens, Hq, Hkv, D, bs, dt, **kw).check().err) == 0


@pytest.mark.parametrize("D,bs,dt", [(64, 16, "f16"), (128, 64, "bf16"), (128, 4, "f16")])
@pytest.mark.parametrize("window", [1, 7, 128, 129, 1000])
def test_window(window, D, bs, dt):
    Case([(1, 900), (4, 1000), (200, 700), (1, 3), (90, 90)], 8, 4, D, bs, dt, window=window).check()
    Case([(1, 900), (2, 1000), (2, 130), (1, 1)], 8, 4, D, bs, dt, window=window, seed=1).check()


@pytest.mark.parametrize("Hq,Hkv,q", [(1, 1, 1), (2, 1, 8), (3, 1, 5), (3, 1, 6), (7, 1, 4), (7, 1, 5), (8, 1, 2), (8, 1, 3), (8, 1, 8), (8, 1, 9), (5, 1, 13)])
@pytest.mark.parametrize("D,dt", [(64, "bf16"), (128, "f16")])
def test_rows(Hq, Hkv, q, D, dt):
    Case([(q, q), (q, 127 + q), (max(q - 1, 0), 400), (q, 1500)], Hq, Hkv, D, 16, dt).check()


@pytest.mark.parametrize("q", [1, 5, 40])
def test_growing_scores_move_the_reference(q):
    c = Case([(q, 3000), (q, 500)], 8, 4, 128, 64, "bf16")
    for s, (_, n) in enumerate(c.lens):
        j = torch.arange(n, device="cuda")
        block = c.bt[s].long()[j // c.bs]
        c.ks[block, :, j % c.bs] *= (1 + j[:, None] / 40.0)
    c.check()


def test_scales_of_every_size():
    # values that differ by 2^20 from key to key, keys by 2^6
    Case([(1, 700), (3, 2000)], 4, 2, 64, 16, "bf16", sizes=4.0).check()
    c = Case([(2, 300)], 4, 2, 128, 16, "bf16")
    c.vs *= 2.0 ** 40
    c.check()
    c.vs *= 2.0 ** -120
    c.check()


def test_rows_of_zeros():
    # a row of zeros has the least scale, 2^-90, and takes its weight all the same
    c = Case([(1, 300), (2, 40)], 4, 2, 128, 16, "bf16")
    c.vc.view(torch.uint8)[int(c.bt[0, 0])] = 0
    c.vs[int(c.bt[0, 0])] = 2.0 ** -90
    c.kc.view(torch.uint8)[int(c.bt[0, 1])] = 0
    c.ks[int(c.bt[0, 1])] = 2.0 ** -90
    c.check()
    c.vc.view(torch.uint8)[:] = 0
    c.vs[:] = 2.0 ** -90
    c.run()
    assert (c.out == 0).all()


@pytest.mark.parametrize("q,Hq,Hkv", [(1, 4, 2), (3, 14, 2), (40, 8, 4)])
def test_a_query_that_is_not_finite_stays_alone(q, Hq, Hkv):
    for bad in (NAN, float("inf")):
        c = Case([(q, 400), (q, 90)], Hq, Hkv, 64, 16, "bf16")
        c.run()
        torch.cuda.synchronize()
        ref = c.out.clone()
        c.q[0, 1, 3] = bad
        c.run()
        torch.cuda.synchronize()
        assert c.out[0, 1].isnan().all()
        ref[0, 1] = c.out[0, 1]
        assert torch.equal(ref.view(torch.int16), c.out.view(torch.int16))


def test_queries_of_every_size():
    c = Case([(4, 400), (1, 3)], 4, 2, 128, 16, "bf16")
    c.q[0] = 0
    c.q[1] *= 2.0 ** -60
    c.q[2] *= 30
    c.q[3, 0, :64] *= 2.0 ** -12
    c.check()


def test_a_row_that_held_a_nan_is_seen_and_others_are_not():
    c = Case([(1, 300), (1, 200)], 4, 2, 128, 16, "bf16")
    c.vs[int(c.bt[0, 3]), 1, 2] = float("inf")
    c.run()
    torch.cuda.synchronize()
    assert c.out[0, 2:].isnan().all() and c.out[0, :2].isfinite().all() and c.out[1].isfinite().all()
    c.vs[int(c.bt[0, 3]), 1, 2] = 1.0
    c.ks[int(c.bt[0, 3]), 0, 2] = NAN
    c.run()
    torch.cuda.synchronize()
    assert c.out[0, :2].isnan().all() and c.out[0, 2:].isfinite().all() and c.out[1].isfinite().all()


def test_lengths_outside_the_contract():
    c = Case([(2, 50), (3, 40), (1, 30), (2, 60)], 4, 2, 64, 16, "f16")
    c.ctx[0], c.ctx[2] = 1, 1 << 20
    c.check(zero=(0, 2))
    assert int(c.err) == pa.PA_DEVERR_LENGTH


@pytest.mark.parametrize("bs,q", [(16, 1), (16, 100), (4, 2)])
def test_bad_table_entries(bs, q):
    c = Case([(q, 300), (q, 200)], 4, 2, 128, bs, "bf16")
    c.bt[1, 2] = -1
    c.check(zero=(1,)) if q < 32 else c.run()
    torch.cuda.synchronize()
    assert int(c.err) & pa.PA_DEVERR_TABLE
    if q >= 32:
        assert (c.out[q:] == 0).all()


def test_nothing_to_do():
    c = Case([(0, 30), (0, 5)], 4, 2, 64, 16, "f16", max_q=4, pad=3)
    c.run()
    torch.cuda.synchronize()
    assert (c.out == 7).all() and int(c.err) == 0


def test_many_sequences():
    r = np.random.default_rng(0)
    lens = [(int(a), int(a + b)) for a, b in zip(r.integers(0, 4, 700), r.integers(0, 300, 700))]
    Case(lens, 4, 2, 64, 16, "bf16").check()


@pytest.mark.parametrize("Hq,Hkv,q", [(8, 1, 1), (7, 1, 1), (14, 2, 1), (3, 1, 2), (4, 1, 2), (2, 1, 4), (6, 6, 8), (5, 5, 7)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 256), (128, 8)])
def test_up_to_eight_rows(Hq, Hkv, q, D, bs):
    c = Case([(q, 2000), (max(q - 1, 1), 129), (q, q), (q, 700)], Hq, Hkv, D, bs, "bf16", window=0 if D == 64 else 300)
    c.check()
    for s, (_, n) in enumerate(c.lens):  # scores that grow along the keys: references move
        j = torch.arange(max(0, n - q - 299) if c.window else 0, n, device="cuda")
        c.ks[c.bt[s].long()[j // bs], :, j % bs] *= (1 + j[:, None] / 40.0)
    c.check()


@pytest.mark.parametrize("Hq,Hkv,window", [(320, 320, 0), (96, 48, 0), (33, 11, 50)])
def test_many_heads(Hq, Hkv, window):
    # more heads than CTAs, and shares that begin and end inside of a head's sequences; some sequences without work
    c = Case([(1, 300), (0, 40), (2, 129), (3, 60), (1, 5)], Hq, Hkv, 64, 16, "bf16", window=window, max_q=2)
    c.check(zero=(3,))  # longer than max_seqlen_q
    assert int(c.err) == pa.PA_DEVERR_LENGTH


def test_repeated_calls_are_equal_and_out_may_be_q():
    c = Case([(2, 4000), (1, 100), (70, 900)], 16, 8, 128, 64, "bf16", seed=3)
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone()
    for _ in range(3):
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    q = c.q.clone()
    pa.pa_chunk_attn_q8(q, q, c.kc, c.vc, c.ks, c.vs, c.bt, c.cu, c.ctx, c.max_q, c.scale, workspace=c.ws)
    assert torch.equal(first, q)


def test_captured_with_other_lengths_at_replay():
    c = Case([(3, 900), (1, 2000), (2, 300)], 16, 8, 128, 64, "bf16")
    c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.lens = [(1, 700), (3, 1999), (2, 2)]
    c.cu.copy_(torch.tensor([0, 1, 4, 6], dtype=torch.int32))
    c.ctx.copy_(torch.tensor([n for _, n in c.lens], dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    c.check(run=False)


def test_two_streams_with_workspaces_of_their_own():
    a, b = Case([(2, 4000)] * 4, 16, 8, 128, 64, "bf16", seed=1), Case([(1, 7000), (60, 600)], 14, 2, 64, 16, "f16", seed=2)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(stream=sa)
        b.run(stream=sb)
    torch.cuda.synchronize()
    a.check(run=False)
    b.check(run=False)


def test_calls_in_a_row_share_a_workspace():
    cases = [Case([(1, 3000), (1, 9)], 16, 8, 128, 64, "bf16"), Case([(100, 500)], 16, 8, 128, 16, "bf16"),
             Case([(3, 800)], 16, 8, 128, 4, "bf16"), Case([(7, 5000)], 16, 8, 128, 256, "bf16"), Case([(16, 600)], 16, 8, 128, 64, "f16")]
    ws = torch.full((max(c.ws.numel() for c in cases),), 255, dtype=torch.uint8, device="cuda")
    for c in cases:
        c.ws = ws
    for _ in range(3):
        for c in cases:
            c.run()
    torch.cuda.synchronize()
    for c in cases:
        c.check(run=False)


def test_the_first_call_of_a_thread():
    c = Case([(1, 300)], 4, 2, 64, 16, "f16")
    torch.cuda.synchronize()
    with ThreadPoolExecutor(1) as ex:
        ex.submit(c.run).result()
    c.check(run=False)


def test_a_cache_of_more_than_four_gigabytes():
    bs, Hkv, D, nb = 256, 8, 128, 17000  # 4.46 GB a pool
    kc, vc = (torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(nb, Hkv, bs, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(0)
    blocks = [nb - 1, 0, nb - 2, 16390]
    for b in blocks:
        for pool, scale in ((kc, ks), (vc, vs)):
            pool[b] = torch.randn(bs, Hkv, D, generator=g, device="cuda").to(E4M3).view(torch.uint8)
            scale[b] = torch.rand(Hkv, bs, generator=g, device="cuda")
    c = Case([(2, 1000)], 16, 8, D, bs, "bf16")
    c.kc, c.vc, c.ks, c.vs = kc.view(E4M3), vc.view(E4M3), ks, vs
    c.bt = torch.tensor([blocks], dtype=torch.int32, device="cuda")
    c.check()


def test_against_the_16_bit_cache():
    # the same numbers in a bf16 cache (e4m3 times a power of two is exact there)
    c = Case([(1, 2000), (4, 300), (60, 500)], 16, 8, 128, 64, "bf16")
    c.ks = torch.where(c.ks.isnan(), c.ks, torch.full_like(c.ks, 2.0 ** -8))
    c.vs = torch.where(c.vs.isnan(), c.vs, torch.full_like(c.vs, 2.0 ** -7))
    c.check()
    kc, vc = (x.float() * s.transpose(1, 2)[..., None] for x, s in ((c.kc, c.ks), (c.vc, c.vs)))
    other = torch.empty_like(c.out)
    ws = torch.empty(pa.pa_chunk_attn_workspace_size(3, 16, 8, 128), dtype=torch.uint8, device="cuda")
    pa.pa_chunk_attn(other, c.q, kc.to(c.dt), vc.to(c.dt), c.bt, c.cu, c.ctx, c.max_q, c.scale, workspace=ws)
    # each is within 2^-8 of the norm
    assert float((other.double() - c.out.double()).norm()) <= 2.0 ** -7 * float(c.out.double().norm())


# chunks of more than 64 query rows a kv head: items of two row tiles of 128, loaders that widen the cache's rows


@pytest.mark.parametrize("D,bs,dt", [(64, 16, "bf16"), (128, 4, "bf16"), (128, 256, "f16")])
def test_wide_many_short_sequences(D, bs, dt):
    # segments of one key tile, some without rows in the second row tile, and sequences without new tokens between them
    r = np.random.default_rng(1)
    lens = [(int(a), int(a + b)) for a, b in zip(r.integers(0, 70, 400), r.integers(0, 60, 400))]
    assert int(Case(lens, 4, 2, D, bs, dt, max_q=70, pad=1, lead=1).check().err) == 0


@pytest.mark.parametrize("Hq,Hkv,q", [(1, 1, 65), (1, 1, 127), (1, 1, 128), (1, 1, 129), (1, 1, 255), (1, 1, 256), (1, 1, 257), (3, 1, 43),
                                      (3, 1, 85), (5, 1, 26), (6, 1, 22), (7, 1, 18), (7, 1, 19), (7, 1, 37), (8, 1, 16), (8, 1, 33)])
@pytest.mark.parametrize("D,dt", [(64, "f16"), (128, "bf16")])
def test_wide_rows(Hq, Hkv, q, D, dt):
    Case([(q, q), (1, 1), (q - 1, 127 + q), (q, 1500)], Hq, Hkv, D, 16, dt).check()


@pytest.mark.parametrize("D,dt", [(64, "bf16"), (128, "bf16"), (128, "f16")])
def test_wide_scales_of_every_size(D, dt):
    Case([(100, 700), (40, 2000)], 4, 2, D, 16, dt, sizes=4.0).check()
    c = Case([(100, 300)], 4, 2, D, 16, dt)
    if dt == "bf16":  # (fp16 outputs hold no such numbers)
        c.vs *= 2.0 ** 40
        c.check()
        c.vs *= 2.0 ** -40
    # rows of zeros have the least scale and take their weight
    c.vc.view(torch.uint8)[int(c.bt[0, 0])] = 0
    c.vs[int(c.bt[0, 0])] = 2.0 ** -90
    c.check()


def test_wide_captured_with_other_lengths_at_replay():
    c = Case([(80, 900), (1, 2000), (70, 300)], 4, 2, 128, 64, "bf16")
    c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.lens = [(1, 700), (70, 1999), (80, 280)]
    c.cu.copy_(torch.tensor([0, 1, 71, 151], dtype=torch.int32))
    c.ctx.copy_(torch.tensor([n for _, n in c.lens], dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    c.check(run=False)


@pytest.mark.parametrize("D,dt", [(64, "f16"), (128, "bf16")])
def test_wide_lengths_outside_the_contract(D, dt):
    c = Case([(200, 500), (100, 400), (90, 300), (130, 600)], 4, 2, D, 16, dt)
    c.ctx[0], c.ctx[2] = 199, 1 << 20
    c.check(zero=(0, 2))
    assert int(c.err) == pa.PA_DEVERR_LENGTH

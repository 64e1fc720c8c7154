"""pa_chunk_attn on the GPU against softmax attention in 64 bits.

Bounds, with u = finfo.eps / 2 of the storage type and A = sum_j softmax_j |v_j| of an element: P is
rounded to the storage type (u A; below 2^-14, fp16's rounding is 2^-25 of the row's largest weight
a key); a score is off by at most e_s, from its fp32 sum of D products (each of the D / 16 matrix
instructions and the sums inside them off by at most 2^-22 of sum |q k| scale, 16 in all), which moves weights by e_s
and so the output by 2 e_s A; the fp32 sums over n keys, the base-2 exponential and the sum of
weights by (n / 16 + 16) 2^-22 A; the output is rounded once, u |out|.
"""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    """Sequences of (new tokens, context length); the pool's unused slots and every table entry that
    is not to be read are filled with what would be seen: NaN and -1 (or an index far outside)."""

    def __init__(self, lens, Hq, Hkv, D, bs, dt, window=0, pad=0, seed=0, lead=0, max_q=None, width=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        self.lens, self.D, self.Hq, self.Hkv, self.bs, self.window, self.dt = lens, D, Hq, Hkv, bs, window, DT[dt]
        S = len(lens)
        used = [-(-n // bs) for _, n in lens]
        nb = sum(used) + 3
        shape = (nb, bs, Hkv, D)
        self.kc = torch.full(shape, float("nan"), device="cuda", dtype=self.dt)
        self.vc = torch.full(shape, float("nan"), device="cuda", dtype=self.dt)
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
            slot = torch.from_numpy(mine).cuda()[j // bs] * bs + j % bs
            for pool in (self.kc, self.vc):
                pool.view(-1, Hkv, D)[slot] = torch.randn(n - first, Hkv, D, generator=g, device="cuda").to(self.dt)
        self.bt = torch.from_numpy(bt.astype(np.int32)).cuda()
        self.cu = torch.tensor(lead + np.concatenate([[0], np.cumsum([q for q, _ in lens])]), dtype=torch.int32,
                               device="cuda")
        self.ctx = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda")
        self.Tq = lead + sum(q for q, _ in lens) + pad
        self.max_q = max([q for q, _ in lens]) if max_q is None else max_q
        self.q = torch.randn(self.Tq, Hq, D, generator=g, device="cuda").to(self.dt)
        self.out = torch.full((self.Tq, Hq, D), 7.0, device="cuda", dtype=self.dt)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5
        n = pa.pa_chunk_attn_workspace_size(S, Hq, Hkv, D)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere

    def run(self, **kw):
        pa.pa_chunk_attn(self.out, self.q, self.kc, self.vc, self.bt, self.cu, self.ctx, self.max_q, self.scale,
                         window=self.window, workspace=self.ws, err=self.err, **kw)

    def reference(self, s):
        """(output in 64 bits, bound) of sequence s: [q, Hq, D]."""
        q, n = self.lens[s]
        first = max(0, n - q - self.window + 1) if self.window else 0
        a = int(self.cu[s])
        j = torch.arange(first, n, device="cuda")
        slot = self.bt[s].long()[j // self.bs] * self.bs + j % self.bs
        G = self.Hq // self.Hkv
        k = self.kc.view(-1, self.Hkv, self.D)[slot].double().repeat_interleave(G, 1)
        v = self.vc.view(-1, self.Hkv, self.D)[slot].double().repeat_interleave(G, 1)
        x = self.q[a:a + q].double()
        pos = torch.arange(n - q, n, device="cuda")[:, None]
        hidden = (j > pos) | ((pos - j >= self.window) if self.window else False)
        sc = torch.einsum("qhd,khd->hqk", x, k) * self.scale
        w = torch.softmax(sc.masked_fill(hidden, -torch.inf), -1)
        size = (torch.einsum("qhd,khd->hqk", x.abs(), k.abs()) * self.scale).masked_fill(hidden, 0).amax(-1)
        out, A = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
        u = torch.finfo(self.dt).eps / 2
        e_s = (16 * 2.0 ** -22 * size).t()[..., None]
        rel = u + 2 * e_s + (n / 16 + 16) * 2.0 ** -22
        bound = A * rel
        if self.dt == torch.float16:
            bound = bound + n * 2.0 ** -25 * v.abs().amax(0)
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


@pytest.mark.parametrize("lens,Hq,Hkv,D,bs,dt,kw", [
    ([(1, 1)], 1, 1, 64, 16, "f16", {}),
    ([(1, 1), (1, 17), (3, 100), (5, 255)], 4, 2, 64, 16, "f16", {}),
    ([(4, 4), (0, 50), (7, 130), (1, 128), (2, 129)], 16, 8, 128, 256, "bf16", dict(pad=5)),
    ([(3, 9000)], 14, 2, 64, 16, "f16", {}),                  # one long cache over all SMs
    ([(8, 5003), (1, 16000), (2, 700)], 16, 8, 128, 256, "bf16", {}),
    ([(128, 128), (129, 129), (127, 400), (257, 1025), (64, 64)], 8, 4, 128, 16, "bf16", {}),
    ([(300, 2000), (1, 3000), (1, 40), (77, 77)], 14, 2, 64, 16, "f16", dict(pad=3, lead=2)),
    ([(50, 333)], 3, 1, 128, 8, "bf16", {}),                  # 42 tokens a row tile
    ([(41, 333), (90, 100)], 5, 1, 64, 24, "bf16", {}),       # boxes of 8 rows
    ([(33, 600), (18, 18), (19, 300)], 14, 2, 128, 64, "f16", {}),
    ([(40, 700)], 12, 2, 64, 32, "bf16", {}),
    ([(140, 300), (256, 256)], 2, 2, 128, 128, "f16", {}),    # no grouping
    ([(17, 900), (100, 130)], 16, 2, 64, 16, "bf16", {}),
    ([(9, 300), (130, 411), (1, 5)], 4, 2, 64, 1, "f16", {}), # rows gathered one by one
    ([(9, 300), (1, 1), (200, 700)], 6, 2, 128, 12, "bf16", {}),
    ([(70, 77)], 8, 1, 128, 5, "f16", {}),
])
def test_against_64_bits(lens, Hq, Hkv, D, bs, dt, kw):
    c = Case(lens, Hq, Hkv, D, bs, dt, seed=len(lens) + bs, **kw)
    c.check()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("window", [1, 2, 127, 128, 129, 1000, 100000])
@pytest.mark.parametrize("Hq,Hkv,D,bs,dt", [(8, 2, 128, 16, "bf16"), (7, 1, 64, 64, "f16"), (4, 2, 64, 3, "bf16")])
def test_window(window, Hq, Hkv, D, bs, dt):
    """Blocks that lie before the window are not in the table and their slots hold NaN."""
    c = Case([(1, 1), (5, 4000), (200, 1500), (64, 64), (1, 129), (130, 130)], Hq, Hkv, D, bs, dt, window=window, seed=window)
    c.check()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("window", [0, 1, 130, 1000])
@pytest.mark.parametrize("D,bs,dt", [(64, 16, "f16"), (128, 256, "bf16"), (128, 24, "f16"), (64, 3, "bf16"), (128, 2, "bf16")])
@pytest.mark.parametrize("Hq,Hkv,q", [(2, 2, 16), (8, 8, 17), (14, 2, 9), (8, 2, 4), (8, 1, 8), (3, 1, 1), (5, 1, 12)])
def test_few_rows(Hq, Hkv, q, D, bs, dt, window):
    """Chunks of up to 16, 32 and 64 query rows a kv head (and the least that are more), single key
    tiles, odd and even numbers of them, whole and shared ones."""
    c = Case([(q, 4000), (1, 1), (min(q, 3), 128), (q, 129), (0, 7), (q, 256), (1, 257), (q, 700), (max(1, q - 1), 384)],
             Hq, Hkv, D, bs, dt, window=window, seed=q + bs, pad=2)
    c.check()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,q", [(2, 2, 5), (14, 2, 4), (8, 1, 8)])
def test_few_rows_growing_scores(Hq, Hkv, q):
    """Keys that grow along the sequence, so that every tile moves the running maximum, and a column
    of equal scores; large scores in both directions."""
    for f in (lambda j: 0.02 * j, lambda j: 40 - 0.02 * j, lambda j: 0 * j):
        c = Case([(q, 2000), (q, 300)], Hq, Hkv, 128, 16, "bf16", seed=3)
        for s, (_, n) in enumerate(c.lens):
            j = torch.arange(n, device="cuda")
            slot = c.bt[s].long()[j // 16] * 16 + j % 16
            c.kc.view(-1, Hkv, 128)[slot] = f(j.float())[:, None, None].expand(n, Hkv, 128).bfloat16()
        c.q[:, 0].fill_(1.0)
        c.q[:, -1].fill_(-1.0)
        c.check()


@pytest.mark.parametrize("q,Hq,Hkv,D", [(4, 4, 2, 64), (9, 14, 2, 128), (200, 8, 2, 128)])
def test_a_query_that_is_not_finite_stays_alone(q, Hq, Hkv, D):
    """NaN and infinities in one query row: every other row keeps its result."""
    c = Case([(q, 1500), (2, 300)], Hq, Hkv, D, 16, "bf16", seed=7)
    c.run()
    torch.cuda.synchronize()
    want = c.out.clone()
    for value in (float("nan"), float("inf"), float("-inf")):
        keep = c.q[1, 1].clone()
        c.q[1, 1, 3:9] = value
        c.out.fill_(7)
        c.run()
        torch.cuda.synchronize()
        c.q[1, 1] = keep
        same = torch.ones(c.Tq, Hq, dtype=torch.bool, device="cuda")
        same[1, 1] = False
        assert torch.equal(c.out[same], want[same])
        assert not torch.isfinite(c.out[1, 1]).any()


def test_keys_that_some_rows_do_not_see_may_be_nan():
    """A key that is NaN reaches the rows that see it and no other (its value is finite)."""
    for q, Hq, Hkv in ((4, 4, 2), (100, 8, 2)):
        c = Case([(q, 700)], Hq, Hkv, 64, 16, "f16")
        c.run()
        torch.cuda.synchronize()
        want = c.out.clone()
        slot = int(c.bt[0, 699 // 16]) * 16 + 699 % 16
        c.kc.view(-1, Hkv, 64)[slot] = float("nan")
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out[: q - 1], want[: q - 1])
        assert torch.isnan(c.out[q - 1]).all()


def test_a_cache_of_more_than_four_gigabytes():
    """Slots whose byte offsets pass 2^32, by boxes and gathered row by row."""
    for bs, q in ((16, 3), (16, 100), (4, 3)):
        c = Case([(q, 1000)], 16, 8, 128, bs, "bf16")
        nb = (5 << 30) // (bs * 8 * 128 * 2)
        kc, vc = (torch.zeros(nb, bs, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        n = c.kc.shape[0]
        kc[-n:], vc[-n:] = c.kc, c.vc
        c.kc, c.vc = kc, vc
        c.bt = torch.where((c.bt >= 0) & (c.bt < n), c.bt + nb - n, c.bt)
        c.check()
        assert int(c.err.item()) == 0


def test_the_largest_group_and_lengths_that_fill_the_table():
    c = Case([(8, 4096), (1, 4096), (8, 8)], 8, 1, 128, 256, "f16")
    c.check()
    c = Case([(64, 4096), (128, 4096), (65, 128)], 2, 2, 64, 256, "bf16")
    c.check()


def test_many_sequences():
    """More sequences than a CTA has threads, single tokens and drafts, empty ones among them."""
    r = np.random.default_rng(5)
    lens = [(int(q), int(max(q, n))) for q, n in zip(r.integers(0, 6, 1000), r.integers(1, 300, 1000))]
    c = Case(lens, 4, 2, 64, 16, "bf16", pad=9)
    c.check()
    assert int(c.err.item()) == 0


def test_single_tokens_equal_decode():
    c = Case([(1, n) for n in (1, 16, 17, 300, 2000, 4096)], 16, 8, 128, 16, "f16")
    c.check()
    out = torch.empty_like(c.out)
    n = pa.pa_decode_workspace_size(6, 16, 8, 128, c.bt.shape[1], 16)
    pa.pa_decode(out, c.q, c.kc, c.vc, c.bt, c.ctx, c.scale, workspace=torch.empty(max(16, n), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert float((out.double() - c.out.double()).abs().max()) <= 2e-3


def test_lengths_outside_the_contract():
    c = Case([(3, 50), (5, 60), (4, 70), (2, 80), (40, 90)], 8, 2, 64, 16, "f16", max_q=39)
    c.ctx[1] = 4                       # fewer keys than new tokens
    c.ctx[3] = c.bt.shape[1] * 16 + 1  # more than the table covers
    c.check(zero=(1, 3, 4))            # and one longer than max_seqlen_q
    assert int(c.err.item()) == pa.PA_DEVERR_LENGTH


def test_rows_outside_q():
    """cu_seqlens_q that runs backwards, or past total_q: flagged, nothing outside q and out is touched."""
    c = Case([(3, 50), (5, 60), (4, 70)], 8, 2, 64, 16, "f16")
    good = c.cu.clone()
    for cu, rows in (([0, 3, 8, 20], 12), ([0, 3, 2, 2], None), ([-1, 3, 8, 12], None)):
        c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        c.err.zero_()
        c.run()
        torch.cuda.synchronize()
        assert int(c.err.item()) == pa.PA_DEVERR_LENGTH
        if rows:
            assert (c.out[8:] == 0).all()
    c.cu = good
    c.err.zero_()
    c.check()


@pytest.mark.parametrize("bs,q", [(16, 3), (16, 200), (1, 3), (1, 200)])
def test_bad_table_entries(bs, q):
    """The rows of an item that needs the block are zero, whichever CTA meets it; other sequences
    are not touched by it."""
    c = Case([(2, 300), (q, 4000), (5, 600)], 8, 2, 64, bs, "f16")
    c.bt[1, 1000 // bs] = c.kc.shape[0]
    c.check(zero=(1,))
    assert int(c.err.item()) == pa.PA_DEVERR_TABLE


def test_nothing_to_do():
    c = Case([(0, 5), (0, 0)], 8, 2, 64, 16, "f16", pad=4, max_q=3)
    c.ctx[1] = -5  # not looked at
    c.check()
    assert int(c.err.item()) == 0 and (c.out == 7).all()


def test_scores_of_every_size():
    """Large scores (a running maximum that jumps by thousands), and a zero scale, which is refused."""
    c = Case([(60, 2000), (3, 900)], 8, 2, 64, 16, "bf16")
    c.q.mul_(30)
    c.check()
    c.scale = 0.0
    with pytest.raises(pa.PagedAttnError) as e:
        c.run()
    assert e.value.status == 2


def test_repeated_calls_are_equal():
    c = Case([(8, 5003), (300, 1600), (2, 700)], 16, 8, 128, 256, "bf16")
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(7)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)


def test_captured_with_other_lengths_at_replay():
    """The shares follow the device's lengths: a captured call replays with others (in place)."""
    c = Case([(4, 2000), (4, 300), (4, 77)], 8, 2, 128, 16, "bf16", width=200)
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.lens = [(2, 100), (0, 5), (3, 77)]
    c.ctx.copy_(torch.tensor([100, 5, 77], dtype=torch.int32))
    c.cu.copy_(torch.tensor([0, 2, 2, 5], dtype=torch.int32))
    c.out.fill_(7)
    torch.cuda.synchronize()
    g.replay()
    c.check(run=False)


def test_two_streams_with_workspaces_of_their_own():
    a = Case([(8, 6000), (100, 900)], 16, 8, 128, 16, "bf16", seed=1)
    b = Case([(5, 7000), (333, 1900)], 14, 2, 64, 16, "f16", seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    a.check(run=False)
    b.check(run=False)


def mixed_cases():
    """Calls of every kind: few and many rows, pages that tile a box and pages that do not, windows, long caches."""
    r = np.random.default_rng(11)
    cases = []
    for i in range(24):
        Hkv, G = int(r.choice([1, 2, 8])), int(r.integers(1, 9))
        most = int(r.choice([1, 4, 8, 30, 100, 400]))
        new = [int(n) for n in r.integers(1, most + 1, r.choice([1, 3, 10]))]
        lens = [(n, max(n, int(r.integers(1, 4000)))) for n in new]
        cases.append(Case(lens, G * Hkv, Hkv, int(r.choice([64, 128])), int(r.choice([4, 16, 64, 256])),
                          str(r.choice(["f16", "bf16"])), window=int(r.choice([0, 0, 200])), seed=i))
    return cases


def test_calls_in_a_row_share_a_workspace():
    # on one stream, with nothing between: the set-up of a call overlaps the end of the one before it
    cases = mixed_cases()
    ws = max((c.ws for c in cases), key=lambda t: t.numel())
    for c in cases:
        c.ws = ws
        c.check()
        c.want = c.out.clone()
    r = np.random.default_rng(12)
    for _ in range(20):
        for c in cases:
            c.out.fill_(7)
        for i in r.permutation(len(cases)):
            cases[i].run()
        torch.cuda.synchronize()
        for c in cases:
            assert torch.equal(c.out, c.want)
            assert int(c.err.item()) == 0


def test_an_input_written_by_the_work_before():
    # the queries, the lengths and the page table come from kernels queued directly before the call
    c = Case([(4, 900), (1, 77), (7, 3000)], 16, 8, 128, 16, "bf16", seed=3)
    c.check()
    want, q, ctx, bt = c.out.clone(), c.q.clone(), c.ctx.clone(), c.bt.clone()
    for _ in range(20):
        c.q.zero_(), c.ctx.zero_(), c.bt.fill_(0), c.out.fill_(7)
        torch.cuda.synchronize()
        c.bt.copy_(bt), c.ctx.copy_(ctx), c.q.copy_(q)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)


def test_calls_from_threads():
    cases = mixed_cases()[:8]
    for c in cases:
        c.check()
        c.want = c.out.clone()
        c.out.fill_(7)
    torch.cuda.synchronize()

    def work(c):
        stream = torch.cuda.Stream()
        for _ in range(20):
            c.run(stream=stream.cuda_stream)
        stream.synchronize()

    with ThreadPoolExecutor(len(cases)) as ex:
        list(ex.map(work, cases))
    for c in cases:
        assert torch.equal(c.out, c.want)
        assert int(c.err.item()) == 0


def test_the_first_call_of_a_thread():
    # nothing has bound a context to the thread before
    c = Case([(4, 900), (300, 1200)], 16, 8, 128, 16, "bf16", seed=4)
    stream = torch.cuda.current_stream().cuda_stream
    with ThreadPoolExecutor(1) as ex:
        ex.submit(c.run, stream=stream).result()
    c.check(run=False)


@pytest.mark.parametrize("lens,Hq,Hkv,D,bs", [
    ([(8, 5003), (300, 1600), (2, 700)], 16, 8, 128, 256), ([(300, 2000), (1, 3000), (77, 77)], 14, 2, 64, 16),
    ([(2000, 2000), (600, 9000)], 8, 1, 128, 16), ([(4, 2000), (1, 300), (3, 77)], 8, 2, 128, 16),
    ([(9, 4000), (1, 1), (5, 128)], 14, 2, 64, 16), ([(8, 4000), (7, 129)], 8, 2, 64, 4)])
def test_out_is_q(lens, Hq, Hkv, D, bs):
    """In place: whole items and joined ones, neighbours' rows in the same load of queries."""
    c = Case(lens, Hq, Hkv, D, bs, "bf16", seed=17)
    c.check()
    q, c.out = c.q.clone(), c.q
    want = None
    for _ in range(10):
        c.q.copy_(q)
        c.run()
        torch.cuda.synchronize()
        want = c.out.clone() if want is None else want
        assert torch.equal(c.out, want)
    c.q = q
    c.check(run=False)

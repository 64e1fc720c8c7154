"""Verification of drafts against the definition in whole numbers, token for token."""
import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

NAN = float("nan")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def units(x):
    x = np.where(np.isnan(x), np.float32(0), x)
    return np.rint(np.clip(x, 0, 1).astype(np.float64) * 2.0 ** 44).astype(np.int64)


def choose(p, q, tokens, u, V):
    """(accepted, next tokens) of one sequence; p, q fp32 arrays of rows (q None: certain drafts)."""
    n = len(tokens) - 1
    k, ended = 0, False
    while k < n:
        x = tokens[k + 1]
        if not 0 <= x < V:
            ended = True
            break
        if not float(u[k]) * (1.0 if q is None else float(q[k, x])) < float(p[k, x]):
            break
        k += 1
    r = p[k].copy()
    if k < n and not ended:
        if q is None:
            r[tokens[k + 1]] = 0
        else:
            with np.errstate(invalid="ignore"):
                r = r - q[k]
    w = units(r)
    if not w.any():
        w = units(p[k])
    if not w.any():
        t = -1
    else:
        last = float(u[n])
        last = 0.0 if not last > 0 else min(last, 1 - 2.0 ** -31)
        upto = np.cumsum(w)
        border = int(upto[-1]) * int(last * 2.0 ** 31) >> 31
        t = int(np.searchsorted(upto, border, side="right"))
    return k, list(tokens[1:k + 1]) + [t] + [-1] * (n - k)


class Drafts:
    def __init__(self, lens, V, dtype, certain=False, seed=0, ahead=0, behind=0, spread=2.0, stride=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.V, self.S = V, len(lens)
        R = ahead + sum(lens) + behind
        self.cu = torch.tensor(np.concatenate([[ahead], ahead + np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        x = spread * torch.randn(R, V, generator=g, device="cuda")
        room = torch.zeros(R, stride or V, dtype=DTYPES[dtype], device="cuda")
        self.p = room[:, :V]
        self.p.copy_(torch.softmax(x, 1))
        self.q = None if certain else torch.softmax(x + torch.randn(R, V, generator=g, device="cuda"), 1).to(DTYPES[dtype])
        # likely drafts, so that some stand
        likely = (self.p if certain else self.q).float()
        self.tokens = torch.multinomial(likely / likely.sum(1, keepdim=True), 1, generator=g)[:, 0].roll(1).to(torch.int32)
        self.u = torch.rand(R, generator=g, device="cuda")
        if certain:
            self.u *= 0.3
        self.next = torch.full((R,), -7, dtype=torch.int32, device="cuda")
        self.accepted = torch.full((self.S,), -7, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        pa.pa_verify(self.next, self.accepted, self.tokens, self.p, self.cu, self.u, draft_probs=self.q, err=self.err, stream=stream)

    def wanted(self):
        cu, tokens, u = self.cu.tolist(), self.tokens.tolist(), self.u.cpu().numpy()
        p, q = self.p.float().cpu().numpy(), None if self.q is None else self.q.float().cpu().numpy()
        nxt, acc = [-7] * len(tokens), []
        for a, b in zip(cu, cu[1:]):
            if a == b:
                acc.append(0)
                continue
            k, row = choose(p[a:b], None if q is None else q[a:b], tokens[a:b], u[a:b], self.V)
            acc.append(k)
            nxt[a:b] = row
        return acc, nxt

    def check(self, err=0):
        self.run()
        acc, nxt = self.wanted()
        assert self.accepted.tolist() == acc
        assert self.next.tolist() == nxt
        assert int(self.err) == err
        return acc


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4096, 4097, 8191, 32000, 50257, 151936, 262144])
def test_against_the_definition(V, dtype, certain):
    Drafts([1, 4, 0, 2, 9, 5], V, dtype, certain, seed=V).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_sequences(dtype):
    acc = Drafts(list(np.random.default_rng(1).integers(0, 7, 300)), 1500, dtype, seed=3, ahead=3, behind=6).check()
    assert min(acc) == 0 and max(acc) > 2


def test_more_drafts_than_a_warp():
    d = Drafts([80, 33, 34, 1, 65], 40, "f32", spread=0.1)
    assert max(d.check()) < 32
    d.u[:] *= 0.001  # nearly every draft stands
    acc = d.check()
    assert max(acc) > 64 and acc[1:3] == [32, 33]


@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_rows_off_the_16_byte_grid(off):
    for dtype in DTYPES:
        d = Drafts([3, 4, 5, 2], 5000, dtype, seed=off, stride=5000 + off)  # p and q rows lie differently
        d.check()
        room = torch.zeros(d.p.numel() + off, dtype=d.p.dtype, device="cuda")
        room[off:] = d.p.reshape(-1)
        d.p = room[off:].view(d.p.shape)
        d.check()


def test_a_draft_outside_the_vocabulary_ends_the_drafts():
    for bad in (-1, 1000, 2 ** 31 - 1, -2 ** 31):
        d = Drafts([6, 6, 6], 1000, "f32", seed=5)
        d.u[:] = 1e-6
        d.tokens[3] = bad
        d.tokens[7] = bad
        assert d.check()[:2] == [2, 0]
        # the token comes from the target's own row, drafter or not
        e = Drafts([3], 1000, "f32", seed=5)
        e.p, e.q, e.u, e.tokens, e.cu = d.p[:3], d.q[:3], torch.cat([d.u[:2], d.u[5:6]]), d.tokens[:3], torch.tensor([0, 3], dtype=torch.int32, device="cuda")
        e.check()
        assert e.next[2] == d.next[2]


def test_where_the_drafter_is_nowhere_below_the_target_its_row_is_taken():
    d = Drafts([2, 2, 2], 777, "f32", seed=6)
    d.q = d.p.clone()
    d.u[0::2] = 1.0           # refused all the same
    assert d.check() == [0, 0, 0]
    d = Drafts([2], 3, "f32", certain=True)
    d.p[0] = torch.tensor([0.0, 1.0, 0.0], device="cuda")
    d.tokens[1] = 1
    d.u[0] = 1.0
    assert d.check() == [0] and d.next[0] == 1


def test_rows_without_weight():
    d = Drafts([3, 1, 2], 5000, "f32", seed=7)
    d.p[3] = 0
    d.p[4] = NAN
    d.check(err=pa.PA_DEVERR_ROW)
    assert d.next[3] == -1 and d.next[4] == -1


def test_odd_numbers():
    # NaN, infinities, numbers below 0 and above 1, weights below 2^-45; random numbers out of range
    d = Drafts([2, 2, 2, 2, 2, 2, 1, 1, 1, 1], 600, "f32", seed=8)
    d.u[1::2] = 0.5
    d.p[0, 5] = NAN
    d.p[2, 7] = float("inf")
    d.p[4, 3], d.q[4, 4] = -1.0, NAN
    d.q[6] = 0
    d.p[8] = 1e-14
    d.p[8, 599] = 2e-14
    d.q[8] = 0
    d.u[8] = NAN
    d.u[12:16] = torch.tensor([0.0, 1.0, NAN, -3.0], device="cuda")
    d.u[10], d.u[11] = 2.0, 7.0
    d.check(err=pa.PA_DEVERR_ROW)  # 2e-14 * 2^44 = 0.35: row 8 has no weight
    assert d.next[8] == -1
    d.err.zero_()
    d.p[8, 599] = 4e-14  # 0.70: one unit
    d.check()
    assert d.next[8] == 599
    d.u[12:16] = torch.tensor([1 - 2.0 ** -24, 2.0 ** -149, 2.0 ** -31, float("inf")], device="cuda")
    d.check()


@pytest.mark.parametrize("V", [700, 151936])
def test_every_token_of_a_flat_row_can_be_drawn(V):
    # a uniform number in the middle of a token's share draws that token, at the borders of slices as elsewhere
    S = 600
    d = Drafts([1] * S, V, "f32", certain=True, spread=0.0)
    want = torch.linspace(0, V - 1, S, device="cuda").round()
    d.u[:] = ((want.double() + 0.5) / V).float()
    d.check()
    if V == 700:
        assert torch.equal(d.next.double(), want.double())


def test_the_share_of_accepted_drafts_and_of_tokens_is_that_of_the_distributions():
    # 60,000 sequences of one draft from q: the tokens that come out have the target's distribution, whatever q is.
    # Five standard deviations of a share of 60,000 are 5 * sqrt(0.25 / 60000) = 0.0102 at most.
    S, g = 60000, torch.Generator(device="cuda").manual_seed(1)
    p, q = torch.tensor([0.5, 0.2, 0.2, 0.1], device="cuda"), torch.tensor([0.1, 0.2, 0.3, 0.4], device="cuda")
    cu = torch.arange(0, 2 * S + 1, 2, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(2 * S, dtype=torch.int32, device="cuda")
    tokens[1::2] = torch.multinomial(q, S, replacement=True, generator=g).to(torch.int32)
    nxt, acc = torch.empty_like(tokens), torch.empty(S, dtype=torch.int32, device="cuda")
    u = torch.rand(2 * S, generator=g, device="cuda")
    pa.pa_verify(nxt, acc, tokens, p.expand(2 * S, 4).contiguous(), cu, u, draft_probs=q.expand(2 * S, 4).contiguous())
    share = torch.bincount(nxt[0::2].long(), minlength=4).double() / S
    assert float((share - p.double()).abs().max()) <= 0.0102
    assert abs(float(acc.double().mean()) - float(torch.minimum(p, q).sum())) <= 0.0102


def test_bad_spans():
    d = Drafts([3, 4, 2], 100, "f32")
    good = d.cu.clone()
    for at, value in ((1, 10), (1, -1), (3, 10)):
        d.cu = good.clone()
        d.cu[at] = value
        d.next.fill_(-7)
        d.err.zero_()
        d.run()
        cu = d.cu.tolist()
        bad = [not 0 <= a <= b <= 9 for a, b in zip(cu, cu[1:])]
        assert any(bad) and int(d.err) == pa.PA_DEVERR_LENGTH
        for s in range(3):
            if bad[s]:
                assert int(d.accepted[s]) == 0


def test_another_stream_a_captured_step_and_the_same_again():
    a, b, c = (Drafts([5] * 40, 30000, "bf16", seed=2) for _ in range(3))
    a.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.run(stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seed in (3, 4):
        other = Drafts([5] * 40, 30000, "bf16", seed=seed)
        for name in ("p", "q", "u", "tokens"):
            getattr(c, name).copy_(getattr(other, name))
        graph.replay()
        other.run()
        torch.cuda.synchronize()
        assert torch.equal(c.next, other.next) and torch.equal(c.accepted, other.accepted)
    assert torch.equal(a.next, b.next) and torch.equal(a.accepted, b.accepted)


def test_empty():
    d = Drafts([2], 10, "f32")
    pa.pa_verify(d.next[:0], d.accepted[:0], d.tokens[:0], d.p[:0], d.cu[:1], d.u[:0])
    d.cu[:] = 0
    pa.pa_verify(d.next[:0], d.accepted, d.tokens[:0], d.p[:0], d.cu, d.u[:0])
    assert d.accepted.tolist() == [0]

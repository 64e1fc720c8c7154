"""pa_sample on the GPU against the definition in 64 bits, token for token.

Why equality: with N kept tokens a wrong token needs u within about sqrt(N) 2^-31 of a border of the
running sum (the weights' errors are below 2^-31 of themselves and independent), which has
probability below N^1.5 2^-31 / N = sqrt(N) 2^-31 a row, 2^-22 at the largest vocabulary here; a top-p border moves
the choice with less. At borders that are hit on purpose (equal weights) both sides are exact.
"""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def choose(x, T=1.0, k=0, p=1.0, m=0.0, u=0.0):
    """The definition, one row in float64."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    top = x.max()
    if top == -np.inf:
        return -1
    if not T > 0:
        return int(np.argmax(x))
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / np.float64(T)))
    order = np.argsort(-x, kind="stable")
    if 0 < k < len(x):
        order = order[:k]
    if p < 1:
        c = np.cumsum(w[order])
        before = np.concatenate([[0.0], c[:-1]])
        n = int(np.sum(before < max(p, 0.0) * c[-1]))
        order = order[: max(n, 1)]
    kept = np.zeros(len(x))
    kept[order] = w[order]
    if m > 0:
        kept[w < min(m, 1.0)] = 0
    c = np.cumsum(kept)
    u = 0.0 if not u > 0 else u
    if u >= 1:
        return int(np.flatnonzero(kept)[-1])
    return int(np.searchsorted(c, u * c[-1], side="right"))


def model_logits(B, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 2 * torch.randn(B, V, generator=g, device="cuda")
    n = min(V, 30)
    x.scatter_add_(1, torch.randint(0, V, (B, n), generator=g, device="cuda"), 9 * torch.rand(B, n, generator=g, device="cuda"))
    return x


def run(x, err=None, **kw):
    B = x.shape[0]
    tokens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    args = {}
    for name, v in kw.items():
        dt = torch.int32 if name == "top_k" else torch.float32
        args[name] = torch.tensor(np.broadcast_to(np.asarray(v), (B,)).copy(), dtype=dt, device="cuda")
    pa.pa_sample(tokens, x, err=err, **args)
    torch.cuda.synchronize()
    return tokens.cpu().numpy()


def check(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.0):
    """Whole rows against the definition; the settings as the float32 the call takes."""
    B = x.shape[0]
    f = [np.broadcast_to(np.asarray(v, dtype=np.float32), (B,)) for v in (temperature, top_p, min_p, u)]
    k = np.broadcast_to(np.asarray(top_k), (B,))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(x, err=err, temperature=f[0], top_k=k, top_p=f[1], min_p=f[2], u=f[3])
    xs = x.double().cpu().numpy()
    want = np.array([choose(xs[b], f[0][b], int(k[b]), float(f[1][b]), float(f[2][b]), float(f[3][b])) for b in range(B)])
    assert np.array_equal(got, want), np.flatnonzero(got != want)
    assert int(err.item()) == (pa.PA_DEVERR_ROW if (want < 0).any() else 0)
    return got


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 512, 4096, 4097, 8191, 16385, 50257, 151936, 262144])
def test_settings_of_every_kind(V, dt):
    B = 24
    r = np.random.default_rng(V)
    x = model_logits(B, V, V).to(DT[dt])
    b = np.arange(B)
    check(x, temperature=np.where(b % 8 == 0, 0.0, r.uniform(0.3, 2.0, B)),
          top_k=np.where(np.isin(b % 8, (1, 4, 6)), r.integers(1, 200, B), 0),
          top_p=np.where(np.isin(b % 8, (2, 4, 7)), r.uniform(0.05, 0.999, B), 1.0),
          min_p=np.where(np.isin(b % 8, (5, 6, 7)), r.uniform(0.001, 0.3, B), 0.0), u=r.uniform(0, 1, B))


def test_defaults():
    x = model_logits(5, 1000, 1)
    assert np.array_equal(run(x), run(x, u=0.0))          # no settings at all: temperature 1, u 0
    got = run(x, temperature=0.0)
    assert np.array_equal(got, x.argmax(1).cpu().numpy())


@pytest.mark.parametrize("dt,V,stride,offset", [("f32", 1003, 1009, 1), ("f16", 1003, 1003, 3), ("bf16", 5001, 5007, 7),
                                                ("bf16", 9, 11, 5), ("f32", 40001, 40003, 3)])
def test_rows_off_the_grid(dt, V, stride, offset):
    """Rows that start anywhere, with neighbours that would win if they were read."""
    B = 9
    flat = torch.full((offset + B * stride + 64,), 1000.0, device="cuda").to(DT[dt])
    x = flat[offset:offset + B * stride].view(B, stride)[:, :V]
    x.copy_(model_logits(B, V, 3).to(DT[dt]))
    r = np.random.default_rng(1)
    check(x, temperature=np.where(np.arange(B) % 3 == 0, 0.0, 1.0), top_p=0.95, u=r.uniform(0, 1, B))


def test_equals():
    """Equal logits: the lowest indexes stay, borders are met exactly."""
    V = 3000
    x = torch.zeros(8, V, device="cuda")
    u = np.array([0, 0.25, 0.5, 0.999, 1 - 2.0 ** -24, 1 / 3, 0.75, 0.125])
    check(x, u=u)
    check(x, top_k=8, u=u)
    check(x, top_p=0.5, u=u)
    check(x, top_k=100, top_p=0.25, u=u)
    check(x, top_p=1e-9, u=u)
    check(x, min_p=1.0, u=u)
    check(x, temperature=0.0)
    y = torch.zeros(8, V, device="cuda")
    y[:, 1::2] = -0.0                                    # equal to 0
    check(y, top_k=5, u=u)
    z = torch.randint(-2, 3, (8, V), device="cuda").float()
    for k in (1, 2, 500, 700, 2999, 3000, 4000):
        check(z, top_k=k, u=u)
    for p in (0.1, 0.6, 0.9, 0.999999):
        check(z, top_p=p, u=u)
        check(z, top_p=p, top_k=900, u=u)


def test_masked_and_odd_logits():
    V = 5000
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    x = model_logits(12, V, 9)
    x[0, :] = -inf                                       # nothing left: -1
    x[1, :] = nan
    x[2, 100:] = -inf
    x[3, :] = low                                        # the lowest value is a value
    x[4, :-7] = low
    x[5, 17] = nan
    x[6, 4000] = inf                                     # all of the weight
    x[7, [5, 17, 900, 901, 4999]] = inf
    x[8, :] = -inf
    x[8, 4321] = -3e38
    x[9, ::2] = -inf
    x[10, :] = low
    x[10, 77] = torch.finfo(torch.float32).max
    x[11, 1:] = nan
    r = np.random.default_rng(2)
    u = r.uniform(0, 1, 12)
    check(x, u=u)
    check(x, temperature=0.0)
    check(x, top_k=3, u=u)
    check(x, top_p=0.9, u=u)
    check(x, top_k=200, top_p=0.5, min_p=0.01, u=u)


@pytest.mark.parametrize("T", [1e-38, 1e-6, 0.01, 100.0, 1e30, float("inf"), -1.0, float("nan"), 1e-45])
def test_temperatures(T):
    x = model_logits(6, 2000, 4)
    check(x, temperature=T, u=np.linspace(0.01, 0.99, 6))
    check(x, temperature=T, top_p=0.7, u=np.linspace(0.01, 0.99, 6))


def test_settings_at_their_ends():
    x = model_logits(6, 2000, 5)
    u = np.linspace(0, 1 - 2.0 ** -24, 6)
    nan = float("nan")
    for kw in (dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=2.0), dict(top_p=nan), dict(min_p=1.0), dict(min_p=7.0), dict(min_p=nan),
               dict(min_p=-1.0), dict(top_k=-3), dict(top_k=1), dict(top_k=1999), dict(top_k=2000), dict(top_k=2 ** 31 - 1)):
        check(x, u=u, **kw)
    assert np.array_equal(check(x, u=1.0), check(x, u=5.0))  # the last token with weight
    assert np.array_equal(check(x, u=nan), check(x, u=-2.0))


def test_a_long_flat_tail():
    """Kept sets of tens of thousands of tokens."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 0.05 * torch.randn(16, 100000, generator=g, device="cuda")
    u = np.random.default_rng(3).uniform(0, 1, 16)
    check(x, u=u)
    check(x, top_p=0.9, u=u)
    check(x, top_k=70001, u=u)
    check(x, top_k=70001, top_p=0.5, min_p=0.9, u=u)


def test_many_rows():
    x = model_logits(700, 3001, 8).bfloat16()
    r = np.random.default_rng(8)
    check(x, temperature=r.uniform(0.2, 2, 700), top_k=r.integers(0, 60, 700), top_p=r.uniform(0.5, 1.1, 700),
          min_p=r.uniform(0, 0.1, 700), u=r.uniform(0, 1, 700))


def test_every_token_has_its_share():
    """A sweep of u over one row chooses each kept token as often as its weight says."""
    x = torch.tensor([[0.0, 3.0, 1.0, 2.0, 2.0, -1.0, 2.5]], device="cuda").expand(4096, 7).contiguous()
    got = run(x, temperature=1.0, top_k=4, u=(np.arange(4096) + 0.5) / 4096)
    w = np.exp(np.array([0, 3, 0, 2, 0, 0, 2.5]))
    w[[0, 2, 4, 5]] = 0
    w[4] = np.exp(2.0)                                   # four stay: 3, 2.5, and both 2s
    share = np.bincount(got, minlength=7) / 4096
    assert np.abs(share - w / w.sum()).max() <= 1 / 4096


def test_captured_and_on_another_stream():
    x = model_logits(33, 40000, 6).half()
    B = 33
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    u = torch.rand(B, device="cuda")
    p = torch.full((B,), 0.9, device="cuda")
    pa.pa_sample(tokens, x, u, top_p=p)
    torch.cuda.synchronize()
    want = tokens.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_sample(tokens, x, u, top_p=p)
    tokens.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, want)
    side = torch.cuda.Stream()
    tokens.zero_()
    torch.cuda.synchronize()
    pa.pa_sample(tokens, x, u, top_p=p, stream=side)
    side.synchronize()
    assert torch.equal(tokens, want)


def test_the_first_call_of_a_thread():
    x = model_logits(33, 40000, 6).half()
    tokens, u = torch.zeros(33, dtype=torch.int32, device="cuda"), torch.rand(33, device="cuda")
    pa.pa_sample(tokens, x, u)
    torch.cuda.synchronize()
    want = tokens.clone()
    tokens.zero_()
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    with ThreadPoolExecutor(1) as ex:
        ex.submit(pa.pa_sample, tokens, x, u, stream=stream).result()
    torch.cuda.synchronize()
    assert torch.equal(tokens, want)


def test_empty_batch():
    pa.pa_sample(torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, 10, device="cuda"))


def test_subnormal_logits():
    """Logits below the smallest normal number, of either sign and among zeros, are ordered like any others: at
    temperature 1 all weights are equal (to 2^-126), so that top-k's and top-p's choice is that order alone."""
    r = np.random.default_rng(21)
    small = r.integers(-3000, 3001, (8, 700))
    for x in (torch.tensor([[-1.0, 1e-39, 2e-39, 0.0, -0.0]] * 8),
              torch.from_numpy(small * 2.0 ** -149).float(),
              torch.from_numpy(np.clip(small, -120, 120) * 2.0 ** -133).bfloat16(),
              torch.from_numpy(np.clip(small, -900, 900) * 2.0 ** -24).half()):
        u = r.uniform(0, 1, 8)
        x = x.cuda()
        check(x, temperature=0.0)
        for k in (1, 2, 40, 650):
            check(x, top_k=k, u=u)
        check(x, top_p=0.3, u=u)
        check(x, top_k=500, top_p=0.5, u=u)


@pytest.mark.parametrize("T", [2.0 ** -149, 7 * 2.0 ** -149, 1e-40, 2.0 ** -126, 1e-30, 2.0 ** -63, (1 - 2.0 ** -24) * 2.0 ** -62, 2.0 ** -62,
                               2.0 ** -60])
def test_cold_temperatures(T):
    """Logits a few temperatures apart, and equal ones, at temperatures whose inverse fp32 does not hold."""
    r = np.random.default_rng(22)
    step = r.integers(-40, 1, (12, 300)).astype(np.float64)
    u = np.linspace(0.02, 0.98, 12)
    for x in (step * T, (step + 17) * T, np.where(step < -2, -np.inf, step * T), np.where(step == -1, 1.0, step * T),
              np.where(step < -3, -1e30, 0.75), np.where(step < -3, 1e-6, 2e-6)):
        x = torch.from_numpy(x).float().cuda()
        check(x, temperature=T, u=u)
        check(x, temperature=T, top_k=5, u=u)
        check(x, temperature=T, top_p=0.6, u=u)
        check(x, temperature=T, top_k=90, top_p=0.9, min_p=0.04, u=u)


def test_hot_temperatures():
    x = torch.from_numpy(np.random.default_rng(23).normal(0, 2.0 ** 100, (12, 300))).float().cuda()
    u = np.linspace(0.02, 0.98, 12)
    for kw in ({}, dict(top_k=7), dict(top_p=0.4), dict(min_p=0.2)):
        check(x, temperature=2.0 ** 100, u=u, **kw)


def kinds(B, r):
    """Settings of B rows: greedy, top-k of few and of many, top-p, min-p and their combinations, plain."""
    i = np.arange(B) % 8
    return dict(temperature=np.where(i == 0, 0.0, r.uniform(0.3, 2.0, B)),
                top_k=np.where(np.isin(i, (1, 4)), r.integers(1, 200, B), np.where(i == 6, r.integers(300, 20000, B), 0)),
                top_p=np.where(np.isin(i, (2, 4, 7)), r.uniform(0.05, 0.999, B), 1.0),
                min_p=np.where(np.isin(i, (5, 6, 7)), r.uniform(0.001, 0.3, B), 0.0), u=r.uniform(0, 1, B))


def check_in_parts(x, n, **kw):
    """check(), n rows a call: few long rows take wider clusters than many do."""
    for b in range(0, x.shape[0], n):
        check(x[b:b + n], **{k: np.broadcast_to(np.asarray(v), x.shape[:1])[b:b + n] for k, v in kw.items()})


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [32768, 32769, 50257, 151936, 262144])
@pytest.mark.parametrize("n", [1, 4, 5])
def test_few_long_rows(n, V, dt):
    r = np.random.default_rng(V + n)
    check_in_parts(model_logits(8, V, V + 1).to(DT[dt]), n, **kinds(8, r))


@pytest.mark.parametrize("dt,V,stride,offset", [("f32", 40001, 40003, 3), ("f16", 50257, 50261, 5), ("bf16", 151935, 151943, 1)])
def test_few_long_rows_off_the_grid(dt, V, stride, offset):
    flat = torch.full((offset + 8 * stride + 64,), 1000.0, device="cuda").to(DT[dt])
    x = flat[offset:offset + 8 * stride].view(8, stride)[:, :V]
    x.copy_(model_logits(8, V, 13).to(DT[dt]))
    for n in (1, 3):
        check_in_parts(x, n, **kinds(8, np.random.default_rng(n)))


@pytest.mark.parametrize("n", [1, 2])
def test_few_long_rows_of_equals(n):
    """Borders among equal logits that lie in every CTA of the cluster."""
    V = 100003
    u = np.array([0, 0.25, 0.999, 1 / 3])
    x = torch.zeros(4, V, device="cuda")
    z = torch.randint(-2, 3, (4, V), device="cuda").float()
    for y in (x, z):
        check_in_parts(y, n, u=u)
        check_in_parts(y, n, temperature=0.0)
        for k in (1, 2, 255, 700, 30000, V - 1, V, V + 1):
            check_in_parts(y, n, top_k=k, u=u)
        for p in (1e-9, 0.25, 0.6, 0.999999):
            check_in_parts(y, n, top_p=p, u=u)
            check_in_parts(y, n, top_p=p, top_k=9000, u=u)
        check_in_parts(y, n, min_p=1.0, u=u)


@pytest.mark.parametrize("n", [1, 4])
def test_few_long_flat_tails(n):
    g = torch.Generator(device="cuda").manual_seed(31)
    x = 0.05 * torch.randn(4, 200000, generator=g, device="cuda")
    u = np.random.default_rng(31).uniform(0, 1, 4)
    check_in_parts(x, n, u=u)
    check_in_parts(x, n, top_p=0.9, u=u)
    check_in_parts(x, n, top_k=70001, top_p=0.5, min_p=0.9, u=u)


def test_few_long_rows_with_nothing_left():
    inf, nan = float("inf"), float("nan")
    x = model_logits(6, 90000, 14)
    x[0, :] = -inf
    x[1, :] = nan
    x[2, 1:] = nan
    x[3, [5, 40000, 89999]] = inf
    x[4, :-1] = -inf
    for kw in ({}, dict(temperature=0.0), dict(top_k=3), dict(top_p=0.9), dict(top_k=200, top_p=0.5, min_p=0.01)):
        check_in_parts(x, 1, u=0.6, **kw)
        check_in_parts(x, 3, u=0.6, **kw)

"""Norms + rotation + append against the definition in 64 bits, for pools of the storage type and of 8 bits.

Tolerances: q and 16-bit pools are rounded once, half a step (eps / 2 of the value), after fp32 arithmetic whose error
is at most 2^-17 of the row's largest magnitude (a sum of D <= 512 squares, a root, three products and a
difference, each within 2^-24 of what it works on). An 8-bit value is half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6) from
the row divided by its scale; the scale is within 2^-17 of its own."""
import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa
from tests.test_rope_store_gpu import table

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
NAN = float("nan")
FP32 = 2.0 ** -17


def normed(x, w, eps):
    x = x.double()
    if w is None:
        return x
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def turned(y, pos, tab, axis, pairs):
    """pos [axes, T], tab [max_pos, rot], axis: of each pair."""
    if tab is None:
        return y
    n = tab.shape[1] // 2
    at = pos.long().clamp(0, tab.shape[0] - 1)[torch.tensor(axis, device=y.device)].t()  # [T, n]; refused ones are not compared
    i = torch.arange(n, device=y.device)
    c, s = tab.double()[at, i][:, None], tab.double()[at, n + i][:, None]
    even, odd = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairs else (slice(0, n), slice(n, 2 * n))
    z = y.clone()
    z[..., even] = y[..., even] * c - y[..., odd] * s
    z[..., odd] = y[..., odd] * c + y[..., even] * s
    return z


class Step:
    def __init__(self, T, Hq, Hkv, D, bs, dt, q8, rot=None, axes=1, pairs=False, weights=(True, True), fused=True, pad=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.Hq, self.Hkv, self.D, self.bs, self.dt, self.q8 = T, Hq, Hkv, D, bs, dt, q8
        self.pairs, self.eps = pairs, 1e-6
        rot = D // 16 * 16 if rot is None else rot
        rot = min(rot, 256)
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda") * (0.1 + 3 * torch.rand(T, 1, 1, generator=g, device="cuda"))
        qkv = qkv.to(dt)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.qw, self.kw = ((torch.randn(D, generator=g, device="cuda") + 1).to(dt) if on else None for on in weights)
        self.nb = -(-T // bs) + 2
        slots = torch.randperm(self.nb * bs, generator=g, device="cuda")[:T].to(torch.int32)
        if pad:
            slots[T - pad:] = -1
        self.slots = slots
        shape = (self.nb, bs, Hkv, D)
        if q8:
            self.kc, self.vc = (torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8).view(E4M3) for _ in range(2))
            self.ks, self.vs = (torch.rand(self.nb, Hkv, bs, generator=g, device="cuda") for _ in range(2))
        else:
            self.kc, self.vc = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
            self.ks = self.vs = None
        self.tab = table(500, rot) if rot else None
        self.pos = torch.randint(0, 500, (axes, T), generator=g, device="cuda", dtype=torch.int32)
        self.axis = [i % axes for i in range(rot // 2)]
        self.q_out = torch.full((T, Hq, D), NAN, device="cuda", dtype=dt)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        pa.pa_norm_rope_store_kv(self.q_out, self.q, self.k, self.v, self.kc, self.vc, self.slots, self.qw, self.kw, self.eps,
                                 self.pos if self.tab is not None else None, self.tab,
                                 bytes(self.axis) if len(self.pos) > 1 else None, self.pairs, self.ks, self.vs, err=self.err,
                                 stream=stream)

    def check(self, kept=None):
        """Runs the call and compares everything that it may write, and that nothing else is written."""
        q, k, v = (x.clone() for x in (self.q, self.k, self.v))
        before = [None if x is None else x.clone() for x in (self.q_out, self.kc, self.vc, self.ks, self.vs)]
        self.run()
        torch.cuda.synchronize()
        kept = self.slots >= 0 if kept is None else kept
        wq = turned(normed(q, self.qw, self.eps), self.pos, self.tab, self.axis, self.pairs)
        wk = turned(normed(k, self.kw, self.eps), self.pos, self.tab, self.axis, self.pairs)
        near(self.q_out[kept], wq[kept], self.dt)
        assert torch.equal(self.q_out[~kept].view(torch.int16), before[0][~kept].view(torch.int16))
        at = self.slots[kept].long()
        rest = torch.ones(self.nb * self.bs, dtype=torch.bool, device="cuda")
        rest[at] = False
        for got, was, scale, was_scale, want in ((self.kc, before[1], self.ks, before[3], wk), (self.vc, before[2], self.vs, before[4], v.double())):
            got, was = (x.view(torch.uint8).view(self.nb * self.bs, self.Hkv, -1) for x in (got, was))
            assert torch.equal(got[rest], was[rest])
            rows = got[at].view(E4M3 if self.q8 else self.dt)
            if not self.q8:
                near(rows, want[kept], self.dt)
                continue
            scale, was_scale = (x.transpose(1, 2).reshape(-1, self.Hkv) for x in (scale, was_scale))
            assert torch.equal(scale[rest], was_scale[rest])
            near8(rows, scale[at], want[kept])
        return self


def near(got, want, dt):
    half, least = torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    slack = FP32 * want.abs().amax(-1, keepdim=True)
    far = (got.double() - want).abs() - (half * want.abs() + (1 + half) * slack + least)
    assert got.numel() == 0 or float(far.max()) <= 0, float(far.max())


def near8(rows, scale, want):
    ideal = (want.abs().amax(-1) / 448).clamp(min=2.0 ** -90)
    assert bool(((scale.double() - ideal).abs() <= FP32 * ideal).all())
    x = want / scale.double()[..., None]
    far = (rows.float().double() - x).abs() - (2.0 ** -4 * x.abs() + 2.0 ** -10 + 2 * FP32 * 448)
    assert rows.numel() == 0 or float(far.max()) <= 0, float(far.max())


HEADS = [(4, 2, 64), (16, 8, 128), (14, 2, 64), (5, 1, 80), (3, 3, 256), (2, 1, 512), (2, 2, 8), (4, 1, 24), (1, 1, 16), (6, 2, 192)]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_against_the_definition(Hq, Hkv, D, dt, q8):
    rot = 0 if D < 16 else None
    assert int(Step(37, Hq, Hkv, D, 16, dt, q8, rot, pad=3).check().err) == 0


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T,bs", [(1, 1), (2, 256), (1301, 48), (9001, 16)])
def test_lengths(T, bs, q8):
    Step(T, 16, 8, 128, bs, torch.bfloat16, q8, fused=T % 2 == 1).check()
    Step(T, 5, 1, 80, bs, torch.float16, q8, pairs=True, pad=min(T - 1, 5)).check()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rot,axes,pairs,weights", [(0, 1, False, (True, True)), (32, 1, False, (True, False)), (128, 3, False, (False, True)),
                                                    (48, 4, True, (True, True)), (16, 2, True, (False, False)), (0, 1, False, (False, False))])
def test_forms(rot, axes, pairs, weights, q8):
    for T in (9, 2500):
        Step(T, 6, 3, 128, 16, torch.bfloat16, q8, rot, axes, pairs, weights).check()


def test_without_norms_the_rows_are_those_of_the_rotation_alone():
    a = Step(200, 8, 4, 128, 16, torch.bfloat16, False, weights=(False, False))
    q, kc, vc = torch.empty_like(a.q_out), a.kc.clone(), a.vc.clone()
    pa.pa_rope_store_kv(q, a.q, a.k, a.v, kc, vc, a.slots, a.pos[0].contiguous(), a.tab)
    a.run()
    assert torch.equal(q, a.q_out) and torch.equal(kc, a.kc) and torch.equal(vc, a.vc)


@pytest.mark.parametrize("q8", [False, True])
def test_in_place(q8):
    a, b = (Step(300, 16, 8, 128, 16, torch.bfloat16, q8, seed=4) for _ in range(2))
    a.run()
    b.q_out = b.q
    b.run()
    assert torch.equal(a.q_out, b.q) and torch.equal(a.kc.view(torch.uint8), b.kc.view(torch.uint8))
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


@pytest.mark.parametrize("q8", [False, True])
def test_bad_slots_and_positions_are_skipped(q8):
    a = Step(50, 4, 2, 64, 16, torch.float16, q8)
    a.slots[7] = a.nb * a.bs
    a.pos[0, 20] = 500
    a.pos[0, 21] = -1
    kept = torch.ones(50, dtype=torch.bool, device="cuda")
    kept[[7, 20, 21]] = False
    a.check(kept)
    assert int(a.err) == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_POSITION


def test_rows_of_zeros_tiny_rows_and_rows_with_nan_or_infinity():
    a = Step(6, 2, 1, 64, 16, torch.bfloat16, True, rot=0, weights=(True, False))
    for x in (a.k, a.v):
        x[0] = 0
        x[1] = 0
        x[1, 0, 5] = 2.0 ** -120   # its scale is the least one: it reads back as 0
        x[2, 0, 3] = NAN
        x[3, 0, 9] = float("inf")
        x[4, 0, 9] = 3e38
    a.run()
    torch.cuda.synchronize()
    at = a.slots.long()
    for c, s in ((a.kc, a.ks), (a.vc, a.vs)):
        rows = c.view(torch.uint8).view(-1, 64)[at].view(E4M3).float()
        scale = s.transpose(1, 2).reshape(-1)[at]
        back = rows * scale[:, None]
        assert bool((scale[:2] == 2.0 ** -90).all()) and bool((back[:2] == 0).all())
        assert bool(back[2:4].isnan().all())
        assert bool(back[4:].isfinite().all())
    # the neighbours are none the worse
    near8(a.kc.view(torch.uint8).view(-1, 1, 64)[at[4:]].view(E4M3), a.ks.transpose(1, 2).reshape(-1, 1)[at[4:]], a.k[4:].double())


def test_the_largest_magnitude_is_held_exactly_and_ties_go_to_even():
    a = Step(1, 1, 1, 16, 1, torch.float16, True, rot=0, weights=(False, False))
    # scale 1: 17 and 19 lie half-way between e4m3 numbers (16, 18, 20), 2^-10 between 0 and 2^-9
    row = torch.tensor([448, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -17, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9], device="cuda")
    a.k[0, 0] = row.to(torch.float16)
    a.run()
    got = a.kc.view(-1, 16)[int(a.slots[0])].float().tolist()
    assert got == [448, 16, 20, 0, 2 * 2.0 ** -9, -16, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9]
    assert float(a.ks.view(-1)[int(a.slots[0])]) == 1.0


def test_another_stream_and_a_captured_step():
    a, b, c = (Step(64, 16, 8, 128, 256, torch.bfloat16, True, seed=9) for _ in range(3))
    a.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.run(stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x in (b, c):
        assert torch.equal(a.q_out, x.q_out) and torch.equal(a.ks, x.ks) and torch.equal(a.vs, x.vs)
        assert torch.equal(a.kc.view(torch.uint8), x.kc.view(torch.uint8)) and torch.equal(a.vc.view(torch.uint8), x.vc.view(torch.uint8))


def test_no_tokens():
    a = Step(1, 4, 2, 64, 16, torch.float16, True)
    pa.pa_norm_rope_store_kv(a.q_out[:0], a.q[:0], a.k[:0], a.v[:0], a.kc, a.vc, a.slots[:0], k_scale=a.ks, v_scale=a.vs)

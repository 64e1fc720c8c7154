"""pa_rope_store_kv on the GPU against the rotation in 64 bits.

Bounds: a rotated element is x0 c - x1 s (or x1 c + x0 s) in fp32, then one rounding to the storage
type. The two products and their sum are each off by at most 2^-24 of their size, together under
2^-22 (|x0 c| + |x1 s|); the rounding is off by half a step, finfo.eps / 2 of the value (half the
smallest subnormal below the normal range). Values, unrotated elements and everything that is not
written are compared bit for bit.
"""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def table(max_pos, rot, base=10000.0):
    n = rot // 2
    a = np.arange(max_pos)[:, None] * base ** (-np.arange(n) / n)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, bs, dt, axes=1, pairs=False, fused=False, pad=0, max_pos=5000, seed=0,
                 pair_axis=None):
        g = torch.Generator(device="cuda").manual_seed(seed + T)
        self.rot, self.pairs, self.axes, self.D, self.Hkv = rot, pairs, axes, D, Hkv

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda").to(DT[dt])

        if fused:
            x = normal(T, Hq + 2 * Hkv, D)
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
        nb = -(-T // bs) + 3
        self.kc, self.vc = normal(nb, bs, Hkv, D), normal(nb, bs, Hkv, D)
        slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T]
        if pad:
            slots[torch.randperm(T, generator=g, device="cuda")[:pad]] = -1
        self.slots = slots.to(torch.int32)
        self.table = table(max_pos, rot)
        pos = torch.randint(0, max_pos, (axes, T), generator=g, device="cuda").to(torch.int32)
        pos[0, 0], pos[-1, -1] = max_pos - 1, 0
        self.pos = pos[0].contiguous() if axes == 1 else pos
        self.pair_axis = pair_axis
        if axes > 1 and pair_axis is None:
            self.pair_axis = bytes(np.random.default_rng(seed).integers(0, axes, rot // 2).astype(np.uint8))
        self.q_out = normal(T, Hq, D)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rotated(self, x):
        """(the rotation in 64 bits, its bound) of [T, H, D]."""
        n = self.rot // 2
        x = x.double().cpu().numpy()
        pos = self.pos.cpu().numpy().reshape(self.axes, -1)
        tab = self.table.cpu().numpy().astype(np.float64)
        pos = np.clip(pos, 0, len(tab) - 1)  # of tokens that are skipped
        ax = np.frombuffer(self.pair_axis, np.uint8) if self.pair_axis else np.zeros(n, int)
        y, mag = x.copy(), np.zeros_like(x)
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if self.pairs else (i, n + i)
            c, s = tab[pos[ax[i]], i][:, None], tab[pos[ax[i]], n + i][:, None]
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
            mag[..., a] = abs(x[..., a] * c) + abs(x[..., b] * s)
            mag[..., b] = abs(x[..., b] * c) + abs(x[..., a] * s)
        f = torch.finfo(self.kc.dtype)
        wide = 2.0 ** -22 * mag
        return y, wide + f.eps / 2 * (abs(y) + wide) + np.where(mag > 0, f.smallest_normal * f.eps / 2, 0.0)

    def run(self, q_out=None):
        pa.pa_rope_store_kv(self.q_out if q_out is None else q_out, self.q, self.k, self.v, self.kc, self.vc, self.slots,
                            self.pos, self.table, pair_axis=self.pair_axis, interleaved=self.pairs, err=self.err)

    def check(self, q_out=None, keep=None):
        """One call against the reference; `keep`: the tokens that are to be written."""
        q0, kc0, vc0 = self.q_out.clone(), self.kc.clone(), self.vc.clone()
        (qr, qb), (kr, kb) = self.rotated(self.q), self.rotated(self.k)
        v0 = self.v.clone()
        self.run(q_out)
        torch.cuda.synchronize()
        out = self.q_out if q_out is None else q_out
        slots = self.slots.cpu().numpy()
        keep = slots >= 0 if keep is None else keep
        d = abs(out.double().cpu().numpy() - qr)
        assert (d[keep] <= qb[keep]).all(), float((d - qb)[keep].max())
        if q_out is None:
            assert torch.equal(out[torch.from_numpy(~keep)], q0[torch.from_numpy(~keep)])
        at = slots[keep]
        got = self.kc.view(-1, self.Hkv, self.D)[torch.from_numpy(at).long()].double().cpu().numpy()
        assert (abs(got - kr[keep]) <= kb[keep]).all()
        kc0.view(-1, self.Hkv, self.D)[torch.from_numpy(at).long().cuda()] = \
            self.kc.view(-1, self.Hkv, self.D)[torch.from_numpy(at).long().cuda()]
        assert torch.equal(self.kc, kc0)  # every other slot as it was
        vc0.view(-1, self.Hkv, self.D)[torch.from_numpy(at).long().cuda()] = v0[torch.from_numpy(keep).cuda()]
        assert torch.equal(self.vc, vc0)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,bs,dt,kw", [
    (1, 1, 1, 16, 16, 1, "f16", {}),
    (4, 4, 2, 64, 64, 16, "f16", {}),
    (37, 14, 2, 64, 64, 16, "bf16", dict(pad=9)),
    (130, 16, 8, 128, 128, 256, "bf16", dict(fused=True, pad=3)),
    (5, 3, 1, 24, 16, 3, "f16", dict(pairs=True)),          # one chunk behind the rotated part
    (33, 5, 5, 40, 32, 16, "bf16", {}),
    (19, 7, 1, 128, 48, 5, "f16", dict(fused=True)),        # rotated in part, five units to pass on
    (64, 16, 8, 128, 128, 16, "f16", dict(pairs=True, fused=True)),
    (3, 2, 2, 512, 256, 8, "bf16", {}),
    (2000, 16, 8, 128, 128, 256, "bf16", dict(pad=17)),     # several rows a thread
    (9001, 5, 1, 80, 80, 16, "f16", dict(fused=True)),
    (9003, 16, 8, 128, 128, 256, "bf16", dict(fused=True, pad=5)),  # more than stays in L2
    (8300, 16, 8, 128, 64, 16, "f16", dict(pairs=True)),
    (900, 32, 8, 64, 32, 16, "bf16", dict(pairs=True)),
    (77, 16, 8, 128, 128, 16, "bf16", dict(axes=3, pair_axis=pa.rope_pair_axis([16, 24, 24]))),
    (77, 16, 8, 128, 128, 16, "bf16", dict(axes=3, pair_axis=pa.rope_pair_axis([24, 20, 20], interleaved=True))),
    (50, 14, 2, 64, 64, 16, "f16", dict(axes=4)),           # any axis on any pair
    (3000, 14, 2, 64, 48, 16, "f16", dict(axes=2, pairs=True, fused=True, pad=100)),
])
def test_rotation_and_append(T, Hq, Hkv, D, rot, bs, dt, kw):
    c = Case(T, Hq, Hkv, D, rot, bs, dt, **kw)
    c.check()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fused", [False, True])
def test_in_place_on_q(fused):
    c = Case(211, 14, 2, 64, 64, 16, "bf16", fused=fused, pad=11)
    k0, v0, skipped = c.k.clone(), c.v.clone(), (c.slots < 0).cpu().numpy()
    q0 = c.q.clone()
    c.check(q_out=c.q)
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)
    assert torch.equal(c.q[torch.from_numpy(skipped)], q0[torch.from_numpy(skipped)])


def test_no_rotation_equals_the_plain_store():
    """At position 0 of a table whose angles are all zero the call stores what pa_store_kv stores."""
    c = Case(300, 16, 8, 128, 128, 16, "f16", pad=20)
    c.pos.zero_()
    kc, vc = c.kc.clone(), c.vc.clone()
    pa.pa_store_kv(c.k, c.v, kc, vc, c.slots)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.kc, kc) and torch.equal(c.vc, vc)
    keep = c.slots >= 0
    assert torch.equal(c.q_out[keep], c.q[keep])


@pytest.mark.parametrize("T", [6, 2500])
def test_bad_slots_and_positions_are_flagged_and_skipped(T):
    c = Case(T, 16, 8, 128, 128, 16, "bf16", axes=3)
    n = c.kc.shape[0] * 16
    c.slots[1] = n                      # behind the pool
    c.pos[2, 3] = 5000                  # behind the table
    c.pos[0, 4] = -1
    keep = np.ones(T, bool)
    keep[[1, 3, 4]] = False
    c.check(keep=keep)
    assert int(c.err.item()) == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_POSITION


def test_padding_tokens_hold_anything():
    """Rows, positions and table entries of a padding token are not read: NaN there, and a position
    outside the table, change nothing and raise no error bit."""
    c = Case(40, 4, 2, 64, 64, 16, "f16", pad=13)
    for t in torch.nonzero(c.slots < 0)[:, 0].tolist():
        c.q[t], c.k[t], c.v[t] = float("nan"), float("nan"), float("nan")
        c.pos[t] = -7
    c.check()
    assert int(c.err.item()) == 0


def test_empty_step():
    c = Case(8, 4, 2, 64, 64, 16, "f16")
    kc = c.kc.clone()
    pa.pa_rope_store_kv(c.q_out[:0], c.q[:0], c.k[:0], c.v[:0], c.kc, c.vc, c.slots[:0], c.pos[:0], c.table)
    torch.cuda.synchronize()
    assert torch.equal(c.kc, kc)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,kw", [
    (9001, 14, 2, 64, 64, dict(fused=True, axes=3, pad=7)),  # three rows a thread, none left over
    (4999, 3, 1, 128, 64, dict(pairs=True, pad=3)),          # five rows by threes
    (3500, 5, 1, 128, 128, {}),                              # seven rows by fours
    (2500, 16, 8, 128, 96, dict(axes=2)),                    # four, none left over
    (700, 64, 1, 256, 256, {}),                              # 66: three
    (160000, 1, 1, 16, 16, dict(pairs=True)),            # three rows: one thread a token
])
def test_many_tokens(T, Hq, Hkv, D, rot, kw):
    c = Case(T, Hq, Hkv, D, rot, 16, "bf16", **kw)
    c.check()
    assert int(c.err.item()) == 0


def test_captured_and_on_another_stream():
    c = Case(57, 16, 8, 128, 128, 16, "bf16", fused=True)
    c.check()
    want_q, want_k = c.q_out.clone(), c.kc.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.run()
    c.q_out.zero_()
    c.kc.view(-1, 8, 128)[c.slots.long()] = 0
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, want_q) and torch.equal(c.kc, want_k)
    c.q_out.zero_()
    torch.cuda.synchronize()
    pa.pa_rope_store_kv(c.q_out, c.q, c.k, c.v, c.kc, c.vc, c.slots, c.pos, c.table, stream=side)
    side.synchronize()
    assert torch.equal(c.q_out, want_q)


def test_the_first_call_of_a_thread():
    c = Case(57, 16, 8, 128, 128, 16, "bf16", fused=True)
    c.check()
    want = c.q_out.clone()
    c.q_out.zero_()
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    with ThreadPoolExecutor(1) as ex:
        ex.submit(pa.pa_rope_store_kv, c.q_out, c.q, c.k, c.v, c.kc, c.vc, c.slots, c.pos, c.table, stream=stream).result()
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, want)


def test_slots_behind_two_gigabytes():
    """Byte offsets into a pool past 2^32."""
    nb, Hkv, D = 2_200_000, 8, 128
    kc = torch.zeros(nb, 1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(3, Hkv, D, generator=g, device="cuda").bfloat16()
    slots = torch.tensor([nb - 1, 5, 1_100_000], dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty_like(k)
    pa.pa_rope_store_kv(out, k, k, k, kc, vc, slots, pos, table(4, 128))
    torch.cuda.synchronize()
    assert torch.equal(kc[slots.long(), 0], k) and torch.equal(vc[slots.long(), 0], k) and torch.equal(out, k)
    assert int(kc.ne(0).any(3).any(2).sum()) == 3

"""Rows that held an infinity or a NaN in the 8-bit cache: what sees them is NaN throughout, whichever kernel the number of query
rows chooses, and the other kv heads and sequences are what they would be without."""
import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")
HEADS = (4, 2)


class Cached:
    """Two sequences of n keys, written by pa_norm_rope_store_kv; the last q tokens of each are the chunk."""

    def __init__(self, q, D, dtype, bs=16, n=300):
        g = torch.Generator(device="cuda").manual_seed(q + D)
        Hq, Hkv = HEADS
        i32 = dict(dtype=torch.int32, device="cuda")
        self.q, self.n, self.bs, self.D = q, n, bs, D
        nb = -(-n // bs)
        self.k, self.v = (torch.randn(2 * n, Hkv, D, generator=g, device="cuda").to(dtype) for _ in range(2))
        self.kc, self.vc = (torch.zeros(2 * nb, bs, Hkv, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
        self.ks, self.vs = (torch.zeros(2 * nb, Hkv, bs, device="cuda") for _ in range(2))
        t = torch.arange(n, **i32)
        self.slots = torch.cat([t, t + nb * bs])
        self.bt = torch.arange(2 * nb, **i32).view(2, nb)
        self.cu, self.ctx = torch.tensor([0, q, 2 * q], **i32), torch.tensor([n, n], **i32)
        self.x = torch.randn(2 * q, Hq, D, generator=g, device="cuda").to(dtype)
        self.ws = torch.empty(pa.pa_chunk_attn_q8_workspace_size(2, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def append(self):
        any_q = torch.zeros(2 * self.n, HEADS[0], self.D, dtype=self.k.dtype, device="cuda")
        pa.pa_norm_rope_store_kv(torch.empty_like(any_q), any_q, self.k, self.v, self.kc, self.vc, self.slots, k_scale=self.ks, v_scale=self.vs)

    def attend(self):
        out = torch.zeros_like(self.x)
        pa.pa_chunk_attn_q8(out, self.x, self.kc, self.vc, self.ks, self.vs, self.bt, self.cu, self.ctx, self.q, self.D ** -0.5,
                            workspace=self.ws)
        torch.cuda.synchronize()
        return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,bs", [(1, 16), (8, 16), (12, 64), (30, 16), (100, 16), (100, 64), (100, 4), (2, 4)])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_rows_that_held_one(q, bs, D, dtype, bad):
    c = Cached(q, D, dtype, bs)
    c.append()
    clean = c.attend()
    assert clean.isfinite().all()
    for name in ("k", "v"):
        x = getattr(c, name)
        was = x[150, 1, 7].clone()
        x[150, 1, 7] = bad  # key 150 of the first sequence, kv head 1: queries of both signs see it
        c.append()
        out = c.attend()
        assert out[:q, 2:].isnan().all(), (name, int(out[:q, 2:].isfinite().sum()))
        assert torch.equal(out[q:], clean[q:])
        assert torch.equal(out[:q, :2], clean[:q, :2])
        x[150, 1, 7] = was


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q,bs", [(1, 16), (8, 16), (30, 16), (100, 16), (2, 4)])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_a_scale_alone(q, bs, dtype, which):
    # the row itself is ordinary: scores of both signs, zeros among the values
    c = Cached(q, 128, dtype, bs)
    c.append()
    clean = c.attend()
    block, at = 150 // bs, 150 % bs
    c.vc.view(torch.uint8)[block, at, 1, ::2] = 0
    for bad in (INF, NAN):
        getattr(c, which)[block, 1, at] = bad
        out = c.attend()
        assert out[:q, 2:].isnan().all()
        assert torch.equal(out[q:], clean[q:]) and torch.equal(out[:q, :2], clean[:q, :2])

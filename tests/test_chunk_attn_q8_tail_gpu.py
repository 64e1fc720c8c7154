"""pa_chunk_attn_q8 where one key outweighs a long tail of others: a first key (an attention sink) with 2^13 to 2^21 times the
weight of each of 20,000 keys behind it. Each of those counts for little, all of them together do not, and in half of the
elements the sink's value is zero, so that the tail is all there is.

As many pairs of sequence and kv head as there are CTAs: a CTA then walks the whole of a sequence's keys, with one
reference for the weights, as it does in any batch of long sequences. All sequences read the same blocks.

Bounds, with u = finfo.eps / 2 of the output's type: a weight is within r of itself (bf16: 2^-8, fp16: 2^-11) or within f of the
largest one (bf16: 2^-30, the pieces end at 2^-19 where the reference leaves the largest at 2^11; fp16: 2^-24, 2^-20 where
it is at 2^4); the score of the sink, some 15, is a sum of one product of two numbers that the pieces hold exactly, off by 2^-22 of itself with
the factors of its scale, which moves a weight by 2 * 15 * 2^-22; sums of n keys and the exponentials by (n / 16 + 16) 2^-22;
the output is rounded once."""
import math

import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,q", [(16, 8, 128, 64, 1), (16, 8, 128, 64, 5), (16, 8, 128, 256, 15), (16, 8, 128, 64, 31),
                                           (8, 8, 64, 16, 2), (32, 8, 64, 16, 4), (16, 8, 128, 4, 1), (16, 8, 128, 64, 70)])
def test_the_tail_behind_a_sink_keeps_its_weight(Hq, Hkv, D, bs, q, dt):
    n, dtype = 20480, DT[dt]
    g = torch.Generator(device="cuda").manual_seed(0)
    S = torch.cuda.get_device_properties(0).multi_processor_count // Hkv
    scale = D ** -0.5
    kc = torch.zeros(n, Hkv, D, dtype=torch.uint8, device="cuda")
    ks = torch.full((n, Hkv), 2.0 ** -90, device="cuda")
    kc[0, :, 0] = 0x7e                                              # 448
    ks[0] = 13 * math.log(2.0) / (scale * 448)
    v8 = (448 * (0.5 + 0.5 * torch.rand(n, Hkv, D, generator=g, device="cuda"))).to(E4M3)
    v8.view(torch.uint8)[0, :, :D // 2] = 0
    vs = torch.full((n, Hkv), 2.0 ** -9, device="cuda")

    def pools(x, s):
        return x.view(n // bs, bs, Hkv, D).view(E4M3), s.view(n // bs, bs, Hkv).transpose(1, 2).contiguous()

    (kp, ksp), (vp, vsp) = pools(kc, ks), pools(v8, vs)
    x = torch.rand(S * q, Hq, D, generator=g, device="cuda") - 0.5
    x[..., 0] = 1 + 0.6 * torch.rand(S * q, Hq, generator=g, device="cuda")
    x = x.to(dtype)
    out = torch.zeros_like(x)
    i32 = dict(dtype=torch.int32, device="cuda")
    bt = torch.arange(n // bs, **i32).repeat(S, 1)
    cu, ctx, err = torch.arange(S + 1, **i32) * q, torch.full((S,), n, **i32), torch.zeros(1, **i32)
    ws = torch.empty(pa.pa_chunk_attn_q8_workspace_size(S, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    pa.pa_chunk_attn_q8(out, x, kp, vp, ksp, vsp, bt, cu, ctx, q, scale, workspace=ws, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0

    G = Hq // Hkv
    v = v8.double() * vs.double()[..., None]
    seen = torch.arange(n - q, n, device="cuda")                    # the tail's keys that a token sees: 1 .. seen
    tail = (v.cumsum(0)[seen] - v[0]).repeat_interleave(G, 1)       # [q, Hq, D]
    heavy = torch.exp(scale * x[..., 0].double() * 448 * ks[0].double().repeat_interleave(G)).view(S, q, Hq, 1)
    first = v[0].repeat_interleave(G, 0)
    want = (heavy * first + tail) / (heavy + seen.view(q, 1, 1))
    got = out.double().view(S, q, Hq, D)
    u = torch.finfo(dtype).eps / 2
    r, f = (2.0 ** -8, 2.0 ** -30) if dt == "bf16" else (2.0 ** -11, 2.0 ** -24)
    bound = want * (r + 30 * 2.0 ** -22 + (n / 16 + 16) * 2.0 ** -22) + n * f * heavy / (heavy + seen.view(q, 1, 1))
    bound = bound + u * (want + bound)
    far = (got - want).abs() - bound
    assert float(far.max()) <= 0, (float(far.max()), float(((got - want).abs() / want).max()))

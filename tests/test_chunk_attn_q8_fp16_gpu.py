"""pa_chunk_attn_q8 in fp16, to fp16's precision, against softmax attention in 64 bits over the values that the cache stands for.

Bounds, with u = 2^-11 and A = sum_j softmax_j |v_j| of an element:
* a weight is within 2^-11 of itself, and up to 64 query rows a kv head within 2^-24 of the largest weight times scale under the first keys'
  reference, beyond that within 2^-25 of the largest: where references lie up to 8 above, 2^-17 per key of that largest is the
  most that a later, larger one leaves; the cases here have none so far above the first keys' (sizes differ by 2^3): 2^-20;
* a query's element is off by at most 2^-27 of its row's largest (three e4m3 pieces, the last in steps of 2^-19 where the largest is from 2^7 on;
  exact beyond 64 rows): D 2^-27 max|q| max|k| scale; the fp32 sums of D products as in the test of both types, 16 * 2^-22 of sum |q k|
  scale; a score that is off by e moves the output by 2 e A;
* fp32 sums over n keys, exponentials and logarithms by (n / 16 + 16) 2^-22 A; the output is rounded once, u |out|.
As a whole: two independent roundings of at most 2^-11, each 2^-11 / sqrt(3) in the mean square, are sqrt(2 / 3) 2^-11 together:
2^-11 of the norm leaves a fifth for the rest."""
import pytest
import torch

from tests.test_chunk_attn_q8_gpu import Case

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def check(c):
    c.run()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for s, (q, n) in enumerate(c.lens):
        if not q:
            continue
        first = max(0, n - q - c.window + 1) if c.window else 0
        a = int(c.cu[s])
        j = torch.arange(first, n, device="cuda")
        k, v = c.rows(c.kc, c.ks, s, j), c.rows(c.vc, c.vs, s, j)
        x = c.q[a:a + q].double()
        pos = torch.arange(n - q, n, device="cuda")[:, None]
        hidden = (j > pos) | ((pos - j >= c.window) if c.window else False)
        w = torch.softmax((torch.einsum("qhd,khd->hqk", x, k) * c.scale).masked_fill(hidden, -torch.inf), -1)
        size = (torch.einsum("qhd,khd->hqk", x.abs(), k.abs()) * c.scale).masked_fill(hidden, 0).amax(-1)
        lost = x.abs().amax(-1).t() * k.abs().amax(-1).amax(0)[:, None] * c.D * 2.0 ** -27 * c.scale
        out, A = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
        e = (16 * 2.0 ** -22 * size + lost).t()[..., None]
        vscale = (v.abs().amax(-1) / 448).t()
        bound = A * (U + 2 * e + (n / 16 + 16) * 2.0 ** -22)
        bound = bound + ((w * vscale[:, None]).amax(-1) * 448 * (n - first) * 2.0 ** -20).t()[..., None]
        bound = bound + U * (out.abs() + bound) + 2.0 ** -25
        got = c.out[a:a + q].double()
        far = (got - out).abs() - bound
        assert float(far.max()) <= 0, (s, float(far.max()))
        off, norm = float((got - out).norm()), float(out.norm())
        assert off <= U * norm, (s, off / norm)


@pytest.mark.parametrize("lens,Hq,Hkv,D,bs,window", [
    ([(1, 1), (1, 17), (1, 255)], 4, 2, 64, 16, 0),
    ([(1, 700), (1, 4000), (1, 129)], 16, 8, 128, 256, 0),   # sixteen columns
    ([(12, 700), (3, 300)], 4, 2, 128, 64, 0),               # thirty-two
    ([(9, 5000), (8, 640)], 14, 2, 64, 16, 0),               # both streams' columns
    ([(30, 900), (2, 80)], 8, 4, 128, 16, 200),
    ([(2, 700), (1, 90)], 8, 4, 128, 4, 0),                  # rows gathered one by one
    ([(150, 900), (40, 300)], 4, 2, 64, 16, 0),              # items of two row tiles
    ([(100, 1500), (65, 400)], 8, 4, 128, 64, 0),
    ([(200, 1500), (65, 65)], 14, 2, 128, 16, 300),
    ([(90, 500)], 4, 2, 128, 4, 0),
])
def test_to_the_precision_of_fp16(lens, Hq, Hkv, D, bs, window):
    check(Case(lens, Hq, Hkv, D, bs, "f16", window=window))

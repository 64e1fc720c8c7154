"""What the pieces that stand for queries and softmax weights beside an 8-bit cache hold: the bounds that include/pa.h states for
pa_chunk_attn_q8 up to 64 query rows a kv head, by the arithmetic of csrc/chunk_attn_q8.cu, step for step, on the CPU.

The pieces are cut from fp16 numbers, whose least step is 2^-24: that rounding adds 2^-25 to the absolute bounds."""
import pytest
import torch


def e4m3(x):
    return x.to(torch.float8_e4m3fn).float()


def numbers(bits, low, high):
    """Every number of so many bits of mantissa from 2^low up to 2^high, both signs."""
    m = torch.arange(1 << (bits - 1), 1 << bits).double() / (1 << (bits - 1))
    x = (m[None] * 2.0 ** torch.arange(low, high).double()[:, None]).flatten()
    return torch.cat([x, -x])


def test_the_conversions_round_to_nearest_even():
    assert e4m3(torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]


@pytest.mark.parametrize("pieces,bits,bound", [(2, 8, 2.0 ** -22), (3, 11, 2.0 ** -27)])
@pytest.mark.parametrize("most", [128.0, 255.0])
def test_query_elements(pieces, bits, bound, most):
    # beside a largest magnitude that has been brought to [128, 256)
    x = numbers(bits, -30, 8)
    x = x[x.abs() <= most]
    v, got = x.half(), torch.zeros_like(x)
    for i in range(pieces):
        a = e4m3(v.float())
        got += a.double() / 32.0 ** i
        v = (v.float() * 32 - a * 32).half()  # exact
    off = (got - x).abs()
    assert float(off.max()) <= bound * most + 2.0 ** -25
    assert float(off[x.abs() >= most * 2.0 ** -14].max()) == 0
    assert float(off.max()) > bound * most / 4  # (and no better than that)


def weights(high):
    g = torch.Generator().manual_seed(0)
    x = torch.rand(2_000_000, generator=g, dtype=torch.float64) * (high + 45) - 45
    return torch.exp2(torch.cat([x, torch.arange(-45, high + 1).double()])).float()


def test_weights_beside_fp16():
    w = weights(8)
    v, got = w.half(), torch.zeros(len(w), dtype=torch.float64)
    for i in range(3):
        a = e4m3(v.float())
        got += a.double() / 32.0 ** i
        v = (v.float() * 32 - a * 32).half()
    off = (got - w.double()).abs()
    # the largest seen with the first keys lies at 2^4
    assert bool((off <= w.double() * 2.0 ** -11 + 16 * 2.0 ** -24 + 2.0 ** -25).all())


def test_weights_beside_bf16():
    w = weights(15)
    h = w.half()

    def upper(v, nearest):  # the upper byte of each half: e5m2
        i = v.view(torch.int16).to(torch.int32) & 0xffff
        i = (i + (0x80 if nearest else 0)) & 0xff00
        return torch.where(i >= 0x8000, i - 0x10000, i).to(torch.int16).view(torch.float16)

    w0 = upper(h, True)
    r = ((h.float() - w0.float()) * 8).half()
    assert torch.equal(r.float(), (h.float() - w0.float()) * 8)  # exact
    w1 = upper(r, True)
    r2 = (r.float() - w1.float()).half()
    assert torch.equal(r2.float(), r.float() - w1.float())
    w2 = upper(r2, False)
    for piece in (w0, w1, w2):
        assert torch.equal(piece.float().to(torch.float8_e5m2).float(), piece.float())
    got = w0.double() + (w1.double() + w2.double()) / 8
    off = (got - w.double()).abs()
    # the largest seen with the first keys lies at 2^11
    assert bool((off <= torch.maximum(w.double() * 2.0 ** -8, torch.tensor(2.0 ** 11 * 2.0 ** -30 + 2.0 ** -25))).all())

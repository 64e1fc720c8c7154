"""Verification where the numbers are extreme: subnormal ones in the tests, rows of many large ones. Token for token against the
definition in whole numbers."""
import pytest
import torch

from tests.test_verify_gpu import DTYPES, Drafts

pytestmark = pytest.mark.gpu

# the least subnormal of each type, and its largest
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
MOST = {"f32": 2.0 ** -126 - 2.0 ** -149, "bf16": 2.0 ** -126 - 2.0 ** -133, "f16": 2.0 ** -14 - 2.0 ** -24}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("certain", [False, True])
def test_subnormal_numbers_in_a_test_are_what_they_are(dtype, certain):
    lo, hi = LEAST[dtype], MOST[dtype]
    # (p, q, u) of a draft; a certain draft has q = 1
    cases = [(lo, 1.0, 0.0), (hi, 1.0, 0.0), (0.0, 1.0, 0.0), (lo, lo, 0.5), (lo, lo, 1.0), (hi, lo, 1.0), (lo, hi, 0.0), (lo, hi, 1.0), (hi, hi, 1 - 2.0 ** -10),
             (lo, 0.0, 0.5), (0.5, lo, 2.0 ** -149), (lo, 1.0, 2.0 ** -149), (hi, 1.0, 2.0 ** -149), (0.0, lo, 2.0 ** -149), (hi, 0.5, 2.0 ** -130),
             (lo, 0.5, 2.0 ** -126)]
    d = Drafts([2] * len(cases), 100, dtype, certain)
    stands = []
    for s, (p, q, u) in enumerate(cases):
        d.tokens[2 * s + 1] = 40 + s
        d.p[2 * s, 40 + s] = p
        if certain:
            q = 1.0
        else:
            d.q[2 * s, 40 + s] = q
        d.u[2 * s] = u
        assert float(d.p[2 * s, 40 + s]) == p and (certain or float(d.q[2 * s, 40 + s]) == q) and float(d.u[2 * s]) == u
        stands.append(int(u * q < p))  # exact in 64 bits
    assert d.check() == stands and 0 < sum(stands) < len(stands)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [1, 400])
@pytest.mark.parametrize("V", [9000, 262144])
def test_rows_of_ones(V, S, dtype):
    # each number counts as 1 (larger ones do too): their sum is far from 1, and the token that of the definition. With 400 sequences a
    # sequence has one CTA, and a lane up to 704 of these numbers.
    d = Drafts([1] * S, V, dtype, certain=True)
    d.p[:] = 1
    d.p[:, V // 3:V // 2] = 2
    d.u[:] = torch.linspace(0, 1 - 2.0 ** -24, S, device="cuda") if S > 1 else 0.7
    d.check()

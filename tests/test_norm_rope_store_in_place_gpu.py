"""In place, with the rows of a token dealt out to several warps (up to 16 tokens an SM) and with a warp a token: what one warp
stores is not what another still has to read."""
import pytest
import torch

from tests.test_norm_rope_store_gpu import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [1, 3, 1000, 2432, 2433])
@pytest.mark.parametrize("Hq,Hkv,D,pairs", [(16, 8, 128, False), (14, 2, 64, False), (5, 1, 80, True), (32, 4, 128, True)])
def test_in_place_is_as_out_of_place(Hq, Hkv, D, pairs, T, q8):
    for dt in (torch.bfloat16, torch.float16):
        a, b = (Step(T, Hq, Hkv, D, 16, dt, q8, pairs=pairs, seed=T) for _ in range(2))
        a.check()
        b.q_out = b.q
        b.run()
        assert torch.equal(a.q_out, b.q) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
        for x, y in ((a.kc, b.kc), (a.vc, b.vc)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        if q8:
            assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)

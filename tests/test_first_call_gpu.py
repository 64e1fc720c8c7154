"""The first call of a thread: nothing has bound a context to it before. (Rotation, chunk attention and sampling have
theirs in their own files.)"""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import paged_kv_cache_83_gb300 as pa

pytestmark = pytest.mark.gpu


def on_a_new_thread(f):
    with ThreadPoolExecutor(1) as ex:
        ex.submit(f).result()
    torch.cuda.synchronize()


@pytest.mark.parametrize("Hq,Hkv,D,n", [(4, 2, 64, 200), (4, 2, 64, 1000), (16, 8, 128, 1000), (8, 1, 128, 1000), (14, 2, 64, 1000)])
def test_decode_and_prefill(Hq, Hkv, D, n):
    bs, B = 16, 3
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    w = -(-n // bs)
    base = [torch.randn(B * w, bs, Hkv, D, device="cuda").half() for _ in range(2)]
    kc, vc = (t.clone() for t in base)
    q, new = torch.randn(B, Hq, D, device="cuda").half(), torch.randn(2, B, Hkv, D, device="cuda").half()
    bt, cl = i32([[b * w + i for i in range(w)] for b in range(B)]), i32([n, n - 1, n // 2])
    ws = torch.empty(max(16, pa.pa_decode_workspace_size(B, Hq, Hkv, D, w, bs)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    cu, cuk = i32([0, 1, 2, 3]), i32([0, n, 2 * n - 1, 2 * n - 1 + n // 2])
    stream = torch.cuda.current_stream().cuda_stream
    calls = [lambda: pa.pa_decode(out, q, kc, vc, bt, cl, D ** -0.5, workspace=ws, stream=stream),
             lambda: pa.pa_store_decode(out, q, new[0], new[1], kc, vc, bt, cl, D ** -0.5, workspace=ws, stream=stream),
             lambda: pa.pa_prefill_varlen(out, q, None, None, kc, vc, cu, cuk, 1, n, bt, Hkv=Hkv, scale=D ** -0.5, stream=stream)]
    if ws.numel() <= pa.PA_DECODE_NOALLOC_SCRATCH_BYTES:
        calls.append(lambda: pa.pa_decode_noalloc(out, q, kc, vc, bt, cl, D ** -0.5, stream=stream))
    for call in calls:
        results = []
        for run in (lambda f: f(), on_a_new_thread):
            for pool, b in zip((kc, vc), base):
                pool.copy_(b)
            out.zero_()
            torch.cuda.synchronize()
            run(call)
            torch.cuda.synchronize()
            results.append(out.clone())
        # a context's pieces may be joined in another order: two results within the contract of one
        assert float((results[0].double() - results[1].double()).abs().max()) <= 4e-3
        assert (results[1] != 0).any(-1).all()

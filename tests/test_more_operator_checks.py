"""What norms + rotation + append, attention over the 8-bit cache and verification refuse, without a GPU: the status codes of the C entry points and the
exceptions of the binding. Every call here fails a host-side check or is an empty no-op."""
import pytest
import torch

import paged_kv_cache_83_gb300 as pa
from paged_kv_cache_83_gb300 import binding

NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
FAKE = 1 << 20  # a non-null, 16-byte aligned address that no launch ever sees
FAR = 1 << 30   # another, clear of FAKE's spans


@pytest.fixture(scope="module")
def lib():
    if not binding.LIB_PATH.exists():
        from paged_kv_cache_83_gb300 import build
        build.build()
    return pa.load()


def _norm(lib, **kw):
    a = dict(qo=FAR, qos=256, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, sm=FAKE,
             qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, axes=1, pair=None, table=FAKE, max_pos=100, rot=64, inter=0, T=4, nb=8, bs=16,
             Hq=4, Hkv=2, D=64, dt=0, cdt=3, err=None, stream=None)
    a.update(kw)
    return lib.pa_norm_rope_store_kv(*a.values())


def test_norm_rope_store_refusals(lib):
    assert _norm(lib, dt=2) == DTYPE
    assert _norm(lib, dt=3) == DTYPE
    assert _norm(lib, cdt=1) == DTYPE                # fp16 rows, bf16 pools
    assert _norm(lib, cdt=2) == DTYPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == SHAPE
    assert _norm(lib, T=-1) == SHAPE
    assert _norm(lib, Hkv=0) == SHAPE
    assert _norm(lib, axes=0) == SHAPE
    assert _norm(lib, inter=2) == SHAPE
    assert _norm(lib, rot=80) == SHAPE
    assert _norm(lib, rot=-16) == SHAPE
    assert _norm(lib, D=60) == UNSUPPORTED
    assert _norm(lib, rot=24) == UNSUPPORTED
    assert _norm(lib, rot=8) == UNSUPPORTED
    assert _norm(lib, axes=5) == UNSUPPORTED
    big = dict(qs=4160, qos=4160, ks=2080, vs=2080)
    assert _norm(lib, D=520, **big) == UNSUPPORTED   # a row of more than a warp's 512 elements
    assert _norm(lib, T=0) == 0
    for name in ("qo", "q", "k", "v", "kc", "vc", "sm", "pos", "table", "ksc", "vsc"):
        assert _norm(lib, **{name: None}) == NULL
    assert _norm(lib, qs=248) == SHAPE
    assert _norm(lib, vs=132) == UNSUPPORTED
    assert _norm(lib, q=FAKE + 8) == UNSUPPORTED
    assert _norm(lib, qw=FAKE + 8) == UNSUPPORTED
    assert _norm(lib, kw=FAKE + 2) == UNSUPPORTED
    assert _norm(lib, ksc=FAKE + 2) == UNSUPPORTED
    assert _norm(lib, pair=bytes([0] * 31 + [1])) == SHAPE
    assert _norm(lib, nb=1 << 20, bs=1 << 12) == UNSUPPORTED  # slots beyond 32 bits


def test_norm_rope_store_refuses_overlap(lib):
    assert _norm(lib, qo=FAKE + 512) == UNSUPPORTED
    assert _norm(lib, q=1 << 25, k=FAR + 1024) == UNSUPPORTED
    assert _norm(lib, q=1 << 25, v=FAR - 1024 + 16) == UNSUPPORTED
    far = {"qo": FAKE, "q": FAKE, "qs": 512, "qos": 512, "k": FAR, "v": FAR, "ks": 512, "vs": 512}
    assert _norm(lib, **{**far, "k": FAKE + 256}) == UNSUPPORTED


def _verify(lib, **kw):
    a = dict(nxt=FAR, acc=FAKE, tokens=FAKE, probs=FAKE, ps=100, draft=FAKE, ds=100, cu=FAKE, u=FAKE, S=2, Tq=6, V=100, dt=2,
             err=None, stream=None)
    a.update(kw)
    return lib.pa_verify(*a.values())


def test_verify_refusals(lib):
    assert _verify(lib, dt=3) == DTYPE
    assert _verify(lib, S=-1) == SHAPE
    assert _verify(lib, Tq=-1) == SHAPE
    assert _verify(lib, V=0) == SHAPE
    assert _verify(lib, ps=99) == SHAPE
    assert _verify(lib, ds=99) == SHAPE
    assert _verify(lib, V=262145, ps=262145, ds=262145) == UNSUPPORTED
    assert _verify(lib, S=(1 << 24) + 1) == UNSUPPORTED
    assert _verify(lib, ps=1 << 39) == UNSUPPORTED
    assert _verify(lib, probs=FAKE + 2) == UNSUPPORTED
    assert _verify(lib, draft=FAKE + 2) == UNSUPPORTED
    assert _verify(lib, dt=0, probs=FAKE + 1) == UNSUPPORTED
    assert _verify(lib, nxt=FAKE) == UNSUPPORTED               # in place
    assert _verify(lib, nxt=FAKE + 20) == UNSUPPORTED
    assert _verify(lib, S=0) == 0
    for name in ("nxt", "acc", "tokens", "probs", "cu", "u"):
        assert _verify(lib, **{name: None}) == NULL


def _raises(error, call, *a, **kw):
    with pytest.raises(error):
        call(*a, **kw)


def test_norm_rope_store_binding_refusals():
    T, Hq, Hkv, D, nb, bs = 3, 4, 2, 64, 2, 16
    h = torch.float16

    def call(**kw):
        a = dict(q_out=torch.empty(T, Hq, D, dtype=h), q=torch.empty(T, Hq, D, dtype=h), k=torch.empty(T, Hkv, D, dtype=h),
                 v=torch.empty(T, Hkv, D, dtype=h), k_cache=torch.empty(nb, bs, Hkv, D, dtype=torch.float8_e4m3fn),
                 v_cache=torch.empty(nb, bs, Hkv, D, dtype=torch.float8_e4m3fn), slot_mapping=torch.zeros(T, dtype=torch.int32),
                 q_weight=torch.ones(D, dtype=h), k_weight=torch.ones(D, dtype=h), positions=torch.zeros(T, dtype=torch.int32),
                 cos_sin=torch.zeros(10, D), k_scale=torch.zeros(nb, Hkv, bs), v_scale=torch.zeros(nb, Hkv, bs))
        a.update(kw)
        pa.pa_norm_rope_store_kv(**a)

    for kw in (dict(q=torch.empty(T, Hq, D)), dict(k=torch.empty(T, Hkv, D, dtype=torch.bfloat16)),
               dict(v_cache=torch.empty(nb, bs, Hkv, D, dtype=h)),
               dict(k_cache=torch.empty(nb, bs, Hkv, D), v_cache=torch.empty(nb, bs, Hkv, D)),
               dict(q_weight=torch.ones(D)), dict(k_scale=torch.zeros(nb, Hkv, bs, dtype=h)), dict(slot_mapping=torch.zeros(T)),
               dict(positions=torch.zeros(T)), dict(cos_sin=torch.zeros(10, D, dtype=h)), dict(cos_sin=torch.zeros(10, 0)),
               dict(eps="a"), dict(q_weight=3)):
        _raises(TypeError, call, **kw)
    for kw in (dict(k=torch.empty(T, Hkv + 1, D, dtype=h)), dict(q_weight=torch.ones(D + 1, dtype=h)), dict(positions=None),
               dict(cos_sin=None), dict(k_scale=None), dict(v_scale=torch.zeros(nb, bs, Hkv)), dict(pair_axis=bytes(3)),
               dict(k_cache=torch.empty(nb, bs, Hkv, D, dtype=h), v_cache=torch.empty(nb, bs, Hkv, D, dtype=h)), {}):
        _raises(ValueError, call, **kw)  # the last: tensors on the CPU


def test_verify_binding_refusals():
    def call(**kw):
        a = dict(next_tokens=torch.zeros(4, dtype=torch.int32), accepted=torch.zeros(2, dtype=torch.int32),
                 tokens=torch.zeros(4, dtype=torch.int32), probs=torch.zeros(4, 10), cu_seqlens_q=torch.zeros(3, dtype=torch.int32),
                 u=torch.zeros(4))
        a.update(kw)
        pa.pa_verify(**a)

    for kw in (dict(next_tokens=torch.zeros(4, dtype=torch.int64)), dict(accepted=torch.zeros(2)), dict(tokens=torch.zeros(4)),
               dict(probs=torch.zeros(4, 10, dtype=torch.float64)), dict(cu_seqlens_q=torch.zeros(3)),
               dict(u=torch.zeros(4, dtype=torch.float64)), dict(draft_probs=torch.zeros(4, 10, dtype=torch.float16)), dict(probs=1)):
        _raises(TypeError, call, **kw)
    for kw in (dict(probs=torch.zeros(10)), dict(u=torch.zeros(5)), dict(tokens=torch.zeros(3, dtype=torch.int32)),
               dict(cu_seqlens_q=torch.zeros(4, dtype=torch.int32)), dict(draft_probs=torch.zeros(4, 9)), {}):
        _raises(ValueError, call, **kw)


def _q8(lib, **kw):
    a = dict(out=FAR, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, maxb=8, cu=FAKE, ctx=FAKE, S=2, Tq=8, max_q=4, window=0,
             Hq=4, Hkv=2, D=64, bs=16, nb=16, scale=0.125, dt=0, ws=FAKE, ws_bytes=1 << 30, err=None, stream=None)
    a.update(kw)
    return lib.pa_chunk_attn_q8(*a.values())


def test_chunk_attn_q8_refusals(lib):
    for dt in (2, 3):
        assert _q8(lib, dt=dt) == DTYPE
    for kw in (dict(S=-1), dict(Tq=-1), dict(max_q=-1), dict(window=-1), dict(bs=0), dict(nb=-1), dict(nb=0), dict(maxb=0), dict(Hq=3),
               dict(maxb=1 << 28), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _q8(lib, **kw) == SHAPE, kw
    for kw in (dict(D=80), dict(Hq=18), dict(S=65536), dict(nb=1 << 28), dict(out=FAR + 8), dict(q=FAKE + 2), dict(kc=FAKE + 8),
               dict(ks=FAKE + 4), dict(vs=FAKE + 8), dict(out=FAKE + 512)):
        assert _q8(lib, **kw) == UNSUPPORTED, kw
    for name in ("out", "q", "kc", "vc", "ks", "vs", "bt", "cu", "ctx"):
        assert _q8(lib, **{name: None}) == NULL, name
    need = pa.pa_chunk_attn_q8_workspace_size(2, 4, 2, 64)
    assert need > 0 and pa.pa_chunk_attn_q8_workspace_size(2, 4, 2, 80) == 0 and pa.pa_chunk_attn_q8_workspace_size(0, 4, 2, 64) == 0
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=FAKE + 8)):
        assert _q8(lib, **kw) == WORKSPACE, kw
    for kw in (dict(S=0), dict(Tq=0), dict(max_q=0)):
        assert _q8(lib, **kw) == 0


def test_chunk_attn_q8_binding_refusals():
    S, Tq, Hq, Hkv, D, nb, bs = 2, 5, 4, 2, 64, 3, 16
    h, e, i = torch.float16, torch.float8_e4m3fn, torch.int32

    def call(**kw):
        a = dict(out=torch.empty(Tq, Hq, D, dtype=h), q=torch.empty(Tq, Hq, D, dtype=h), k_cache=torch.empty(nb, bs, Hkv, D, dtype=e),
                 v_cache=torch.empty(nb, bs, Hkv, D, dtype=e), k_scale=torch.ones(nb, Hkv, bs), v_scale=torch.ones(nb, Hkv, bs),
                 block_tables=torch.zeros(S, 2, dtype=i), cu_seqlens_q=torch.zeros(S + 1, dtype=i),
                 context_lens=torch.zeros(S, dtype=i), max_seqlen_q=3, scale=0.1)
        a.update(kw)
        pa.pa_chunk_attn_q8(**a)

    for kw in (dict(k_cache=torch.empty(nb, bs, Hkv, D, dtype=h)), dict(v_cache=torch.empty(nb, bs, Hkv, D, dtype=torch.float8_e5m2)),
               dict(q=torch.empty(Tq, Hq, D)), dict(k_scale=torch.ones(nb, Hkv, bs, dtype=h)), dict(k_scale=None),
               dict(cu_seqlens_q=torch.zeros(S + 1)), dict(scale="x")):
        _raises(TypeError, call, **kw)
    for kw in (dict(k_scale=torch.ones(nb, bs, Hkv)), dict(v_scale=torch.ones(nb, Hkv)), dict(out=torch.empty(Tq + 1, Hq, D, dtype=h)),
               dict(cu_seqlens_q=torch.zeros(S, dtype=i)), dict(window=-1), dict(max_seqlen_q=1 << 31), {}):
        _raises(ValueError, call, **kw)

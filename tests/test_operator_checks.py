"""What the layer-step and sampling operators refuse, without a GPU: the status codes of the C entry
points and the exceptions of the binding. Every call here fails a host-side check or is an empty
no-op, so nothing is launched."""
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


def _rope(lib, **kw):
    a = dict(qo=FAR, qos=256, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, kc=FAKE, vc=FAKE, sm=FAKE, pos=FAKE,
             axes=1, pair=None, table=FAKE, max_pos=100, rot=64, inter=0, T=4, nb=8, bs=16, Hq=4, Hkv=2, D=64, dt=0,
             err=None, stream=None)
    a.update(kw)
    return lib.pa_rope_store_kv(*a.values())


def test_rope_store_refusals(lib):
    assert _rope(lib, dt=2) == DTYPE
    assert _rope(lib, T=-1) == SHAPE
    assert _rope(lib, bs=0) == SHAPE
    assert _rope(lib, Hq=0) == SHAPE
    assert _rope(lib, axes=0) == SHAPE
    assert _rope(lib, inter=2) == SHAPE
    assert _rope(lib, rot=80) == SHAPE               # wider than a head
    assert _rope(lib, D=60) == UNSUPPORTED
    assert _rope(lib, rot=24) == UNSUPPORTED
    assert _rope(lib, rot=0) == UNSUPPORTED
    assert _rope(lib, D=512, rot=272, qs=2048, qos=2048, ks=1024, vs=1024) == UNSUPPORTED
    assert _rope(lib, axes=5) == UNSUPPORTED
    assert _rope(lib, T=0) == 0                      # empty: no-op
    for name in ("qo", "q", "k", "v", "kc", "vc", "sm", "pos", "table"):
        assert _rope(lib, **{name: None}) == NULL
    assert _rope(lib, qs=248) == SHAPE               # tokens that run into each other
    assert _rope(lib, ks=0) == SHAPE
    assert _rope(lib, vs=132) == UNSUPPORTED         # tokens off the 16-byte grid
    assert _rope(lib, qos=1 << 41) == UNSUPPORTED
    assert _rope(lib, k=FAKE + 2) == UNSUPPORTED
    assert _rope(lib, table=FAKE + 4) == UNSUPPORTED
    assert _rope(lib, pair=bytes([0] * 31 + [1])) == SHAPE   # an axis that is not there


def test_rope_store_refuses_overlap(lib):
    # q_out starts inside q, covers k, or is q with another stride
    assert _rope(lib, qo=FAKE + 512) == UNSUPPORTED
    assert _rope(lib, qo=FAKE, qos=264) == UNSUPPORTED
    assert _rope(lib, q=1 << 25, k=FAR + 1024) == UNSUPPORTED
    assert _rope(lib, q=1 << 25, v=FAR - 1024 + 16) == UNSUPPORTED


def test_rope_store_in_place_refuses_keys_within_q(lib):
    # In place on q, k or v would be read from what is written: q's own rows, rows that start in one, rows that run into
    # the next token's, rows that lie beside the first token's only. (Tokens of 512 elements, of which q takes 256.)
    far = {"qo": FAKE, "q": FAKE, "qs": 512, "qos": 512, "k": FAR, "v": FAR, "ks": 512, "vs": 512}
    for name, stride in (("k", "ks"), ("v", "vs")):
        for at in (0, 128, 512 - 64, -64, 512 + 128):
            assert _rope(lib, **{**far, name: FAKE + 2 * at}) == UNSUPPORTED, at
        assert _rope(lib, **{**far, name: FAKE + 2 * 256, stride: 256}) == UNSUPPORTED


def test_pair_axis_of_sections():
    assert list(pa.rope_pair_axis([2, 3, 1])) == [0, 0, 1, 1, 1, 2]
    assert list(pa.rope_pair_axis([4, 2, 2], interleaved=True)) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert list(pa.rope_pair_axis([4, 2, 1], interleaved=True)) == [0, 1, 2, 0, 1, 0, 0]
    assert list(pa.rope_pair_axis([3])) == [0, 0, 0]
    for bad in ([], [1, 1, 1, 1, 1], [4, -1]):
        with pytest.raises(ValueError):
            pa.rope_pair_axis(bad)
    with pytest.raises(ValueError):
        pa.rope_pair_axis([1, 4, 4], interleaved=True)


def test_rope_store_binding_refusals():
    q, k = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(3, 2, 64, dtype=torch.float16)
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    idx = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(8, 64)

    def call(q_out=q, q=q, k=k, v=k, kc=pool, vc=pool, slots=idx, pos=idx, table=table, **kw):
        pa.pa_rope_store_kv(q_out, q, k, v, kc, vc, slots, pos, table, **kw)

    with pytest.raises(ValueError):                  # not on a CUDA device
        call()
    with pytest.raises(ValueError):
        call(q_out=q[:2])
    with pytest.raises(ValueError):
        call(v=k[:, :1])
    with pytest.raises(ValueError):
        call(slots=idx[:2])
    with pytest.raises(ValueError):
        call(pos=torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        call(table=table.half())
    with pytest.raises(ValueError):
        call(pair_axis=b"\0" * 31)
    with pytest.raises(ValueError):
        call(pair_axis=[0] * 32)
    with pytest.raises(TypeError):
        call(q=q.bfloat16())
    with pytest.raises(TypeError):
        call(kc=pool.float())


def _chunk(lib, **kw):
    a = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, maxb=4, cu=FAKE, ctx=FAKE, S=2, tq=8, mq=4, window=0, Hq=4,
             Hkv=2, D=64, bs=16, nb=8, scale=0.125, dt=0, ws=None, wsb=0, err=None, stream=None)
    a.update(kw)
    return lib.pa_chunk_attn(*a.values())


def test_chunk_attn_refusals(lib):
    assert _chunk(lib, dt=2) == DTYPE
    for bad in (dict(S=-1), dict(tq=-1), dict(mq=-1), dict(window=-1), dict(bs=0), dict(nb=-1), dict(maxb=-1), dict(Hq=5),
                dict(Hkv=0), dict(scale=-0.1), dict(scale=0.0), dict(scale=1e-40), dict(scale=3e38), dict(scale=float("nan")), dict(scale=float("inf")), dict(maxb=0), dict(nb=0),
                dict(maxb=1 << 30, bs=4)):
        assert _chunk(lib, **bad) == SHAPE, bad
    for bad in (dict(Hq=18), dict(D=96), dict(S=65536), dict(nb=1 << 30), dict(maxb=(1 << 27) - 1)):
        assert _chunk(lib, **bad) == UNSUPPORTED, bad
    for empty in (dict(S=0), dict(tq=0), dict(mq=0)):
        assert _chunk(lib, **empty) == 0
    for name in ("out", "q", "kc", "vc", "bt", "cu", "ctx"):
        assert _chunk(lib, **{name: None}) == NULL, name
    for name in ("out", "q", "kc", "vc"):
        assert _chunk(lib, **{name: FAKE + 8}) == UNSUPPORTED, name
    need = lib.pa_chunk_attn_workspace_size(2, 4, 2, 64)
    assert need > 0
    assert _chunk(lib) == WORKSPACE
    assert _chunk(lib, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert _chunk(lib, ws=FAKE + 8, wsb=need) == WORKSPACE
    assert lib.pa_chunk_attn_workspace_size(0, 4, 2, 64) == 0
    assert lib.pa_chunk_attn_workspace_size(2, 5, 2, 64) == 0
    assert lib.pa_chunk_attn_workspace_size(2, 4, 2, 96) == 0


def test_chunk_attn_refuses_overlap(lib):
    rows = 8 * 4 * 64 * 2
    for out, q in ((FAKE + 16, FAKE), (FAKE, FAKE + 16), (FAKE + rows - 16, FAKE), (FAKE, FAKE + rows - 16)):
        assert _chunk(lib, out=out, q=q) == UNSUPPORTED
    for out, q in ((FAKE, FAKE), (FAKE + rows, FAKE), (FAKE, FAKE + rows), (FAR, FAKE)):
        assert _chunk(lib, out=out, q=q) == WORKSPACE  # the next check


def test_chunk_attn_binding_refusals():
    q = torch.zeros(6, 4, 64, dtype=torch.float16)
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    bt, cu, ctx = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)

    def call(out=q, q=q, kc=pool, vc=pool, bt=bt, cu=cu, ctx=ctx):
        pa.pa_chunk_attn(out, q, kc, vc, bt, cu, ctx, 3, 0.125)

    with pytest.raises(ValueError):                  # not on a CUDA device
        call()
    for bad in (dict(out=q[:5]), dict(vc=pool[:1]), dict(bt=bt[:1]), dict(cu=cu[:2]), dict(ctx=ctx[None])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(out=q.float()), dict(kc=pool.bfloat16())):
        with pytest.raises(TypeError):
            call(**bad)


def _sample(lib, **kw):
    a = dict(tokens=FAKE, logits=FAKE, stride=1000, B=2, V=1000, dt=2, u=FAKE, t=FAKE, k=FAKE, p=FAKE, m=FAKE, err=None,
             stream=None)
    a.update(kw)
    return lib.pa_sample(*a.values())


def test_sample_refusals(lib):
    assert _sample(lib, dt=3) == DTYPE
    for bad in (dict(B=-1), dict(V=0), dict(stride=999)):
        assert _sample(lib, **bad) == SHAPE, bad
    for bad in (dict(V=262145, stride=262145), dict(B=(1 << 24) + 1), dict(stride=1 << 40), dict(logits=FAKE + 2),
                dict(dt=0, logits=FAKE + 1)):
        assert _sample(lib, **bad) == UNSUPPORTED, bad
    assert _sample(lib, B=0) == 0
    assert _sample(lib, tokens=None) == NULL
    assert _sample(lib, logits=None) == NULL


def test_sample_binding_refusals():
    x, t = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):                  # not on a CUDA device
        pa.pa_sample(t, x)
    with pytest.raises(ValueError):
        pa.pa_sample(t[:2], x)
    with pytest.raises(TypeError):
        pa.pa_sample(t, x.double())


def test_binding_refuses_other_types():
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    k, pool = q[:, :2].contiguous(), torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    idx, table = torch.zeros(3, dtype=torch.int32), torch.zeros(8, 64)
    rope = [q, q, k, k, pool, pool, idx, idx, table]
    for i in range(len(rope)):
        with pytest.raises(TypeError):
            pa.pa_rope_store_kv(*rope[:i], None, *rope[i + 1:])
        with pytest.raises(ValueError):              # a dimension too many
            pa.pa_rope_store_kv(*rope[:i], rope[i][None, None], *rope[i + 1:]) if i != 8 else \
                pa.pa_rope_store_kv(*rope[:3], k[None], *rope[4:])
    for i in (6, 7):
        with pytest.raises(TypeError):
            pa.pa_rope_store_kv(*rope[:i], idx.long(), *rope[i + 1:])
    with pytest.raises(TypeError):
        pa.pa_rope_store_kv(*rope, err=torch.zeros(1))
    with pytest.raises(TypeError):
        pa.pa_rope_store_kv(*rope, err=3)


def test_chunk_attn_binding_refuses_numbers():
    q, pool = torch.zeros(6, 4, 64, dtype=torch.float16), torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    bt, cu, ctx = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    args = [q, q, pool, pool, bt, cu, ctx]
    for mq, window in ((-1, 0), (1 << 31, 0), (3, -1), (3, 1 << 31)):
        with pytest.raises(ValueError):
            pa.pa_chunk_attn(*args, mq, 0.125, window)
    with pytest.raises((TypeError, OverflowError)):
        pa.pa_chunk_attn(*args, 1 << 80, 0.125)
    for mq, scale in (("3", 0.125), (3.5, 0.125), (3, "0.125")):
        with pytest.raises(TypeError):
            pa.pa_chunk_attn(*args, mq, scale)
    for i in range(len(args)):
        with pytest.raises(TypeError):
            pa.pa_chunk_attn(*args[:i], None, *args[i + 1:], 3, 0.125)
    for i in (4, 5, 6):
        with pytest.raises(TypeError):
            pa.pa_chunk_attn(*args[:i], args[i].long(), *args[i + 1:], 3, 0.125)


def test_sample_binding_refuses_settings():
    x, t = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(u=torch.zeros(2)), dict(u=torch.zeros(3).double()), dict(temperature=torch.zeros(3, 1)), dict(top_k=torch.zeros(3)),
                dict(top_p=t), dict(min_p=0.5), dict(err=torch.zeros(1))):
        with pytest.raises(TypeError):
            pa.pa_sample(t, x, **bad)
    with pytest.raises(TypeError):
        pa.pa_sample(t.long(), x)
    with pytest.raises(ValueError):
        pa.pa_sample(t, x[0])

"""The attention entry points reject bad arguments on the host before touching a GPU."""
import ctypes

import pytest

FAKE = 0x10000          # 16-byte aligned, never dereferenced: validation fails first
MISALIGNED = 0x10008


@pytest.fixture(scope="module")
def bd():
    from bit_delta_compressed_gb300 import build
    build.build()
    import bit_delta_compressed_gb300 as bd
    return bd


def cache(bd, **over):
    c = dict(k=FAKE, v=FAKE, slots=4, capacity=100, kv_heads=2, head_dim=128, stride_slot=25600, stride_token=256, stride_head=128)
    c.update(over)
    return bd.KVCacheDesc(*[c[name] for name, _ in bd.KVCacheDesc._fields_])


BAD_CACHES = [
    (dict(k=None), "BD_ERR_NULL"), (dict(v=None), "BD_ERR_NULL"), (dict(k=MISALIGNED), "BD_ERR_ALIGN"), (dict(v=MISALIGNED), "BD_ERR_ALIGN"),
    (dict(slots=0), "BD_ERR_SHAPE"), (dict(capacity=0), "BD_ERR_SHAPE"), (dict(capacity=2 ** 24 + 1), "BD_ERR_SHAPE"), (dict(kv_heads=0), "BD_ERR_SHAPE"),
    (dict(head_dim=96), "BD_ERR_SHAPE"), (dict(stride_token=0), "BD_ERR_SHAPE"), (dict(stride_slot=-8), "BD_ERR_SHAPE"), (dict(stride_head=132), "BD_ERR_ALIGN"),
    (dict(stride_slot=2 ** 39), "BD_ERR_SHAPE"), (dict(slots=2 ** 24 + 1), "BD_ERR_SHAPE"),
]


def decode(bd, c="ok", q=FAKE, stride=1024, B=3, heads=8, lens=FAKE, slots=None, window=0, sinks=0, scale=0.1, weights=None, out=FAKE, ws=FAKE, wsb=1 << 40):
    c = ctypes.byref(cache(bd)) if c == "ok" else c
    return bd.bitdelta_attn_decode(q, stride, B, heads, c, slots, lens, window, sinks, scale, weights, out, ws, wsb, None)


def prefix(bd, ids=FAKE, slots=FAKE, lens=FAKE, P=2, ws=None):
    return bd.bitdelta_attn_decode_prefix(FAKE, 1024, 3, 8, ctypes.byref(cache(bd)), None, FAKE, ids, slots, lens, P, 0, 0, 0.1, None, FAKE, ws, 1 << 40, None)


def prefill(bd, T=10, B=3, cu=FAKE, q=FAKE, ws=FAKE, wsb=1 << 40, stride=1024, sinks=0):
    return bd.bitdelta_attn_prefill(q, stride, T, B, 8, ctypes.byref(cache(bd)), None, cu, FAKE, None, None, None, 0, 0, sinks, 0.1, FAKE, ws, wsb, None)


def evict(bd, c="ok", weights=FAKE, lens=FAKE, src=FAKE, dst=FAKE, n=2, budget=50, sinks=4, recent=10, kept=None, ws=FAKE, wsb=1 << 20):
    c = ctypes.byref(cache(bd)) if c == "ok" else c
    return bd.bitdelta_cache_evict(c, weights, lens, src, dst, n, budget, sinks, recent, kept, ws, wsb, None)


@pytest.mark.parametrize("over,code", BAD_CACHES, ids=str)
def test_caches(bd, over, code):
    c = ctypes.byref(cache(bd, **over))
    assert decode(bd, c=c) == getattr(bd, code)
    assert evict(bd, c=c) == getattr(bd, code)


def test_decode_arguments(bd):
    assert decode(bd, c=None) == bd.BD_ERR_NULL
    assert decode(bd, q=None) == bd.BD_ERR_NULL
    assert decode(bd, out=None) == bd.BD_ERR_NULL
    assert decode(bd, lens=None) == bd.BD_ERR_NULL
    assert decode(bd, heads=7) == bd.BD_ERR_SHAPE                # not a multiple of the key/value heads
    assert decode(bd, heads=2 * 129, stride=1 << 20) == bd.BD_ERR_SHAPE
    assert decode(bd, heads=0) == bd.BD_ERR_SHAPE
    assert decode(bd, B=-1) == bd.BD_ERR_SHAPE
    assert decode(bd, window=-1) == bd.BD_ERR_SHAPE
    assert decode(bd, sinks=-1) == bd.BD_ERR_SHAPE
    assert decode(bd, scale=float("nan")) == bd.BD_ERR_SHAPE
    assert decode(bd, scale=float("inf")) == bd.BD_ERR_SHAPE
    assert decode(bd, stride=1016) == bd.BD_ERR_SHAPE            # rows would overlap
    assert decode(bd, stride=1028) == bd.BD_ERR_ALIGN
    assert decode(bd, q=MISALIGNED) == bd.BD_ERR_ALIGN
    assert decode(bd, lens=0x10002) == bd.BD_ERR_ALIGN
    assert decode(bd, weights=0x10002) == bd.BD_ERR_ALIGN
    assert decode(bd, ws=None) == bd.BD_ERR_WORKSPACE
    assert decode(bd, wsb=128) == bd.BD_ERR_WORKSPACE
    assert decode(bd, ws=MISALIGNED) == bd.BD_ERR_ALIGN
    assert decode(bd, B=0, q=None, out=None, lens=None, ws=None) == bd.BD_OK


def test_prefix_and_prefill_arguments(bd):
    assert prefix(bd, ids=None, ws=FAKE) == bd.BD_ERR_NULL
    assert prefix(bd, slots=None, ws=FAKE) == bd.BD_ERR_NULL
    assert prefix(bd, lens=None, ws=FAKE) == bd.BD_ERR_NULL
    assert prefix(bd, P=-1, ws=FAKE) == bd.BD_ERR_SHAPE
    assert prefix(bd, P=8193, ws=FAKE) == bd.BD_ERR_SHAPE
    assert prefix(bd, ids=0x10001, ws=FAKE) == bd.BD_ERR_ALIGN
    assert prefix(bd) == bd.BD_ERR_WORKSPACE
    assert prefill(bd, cu=None) == bd.BD_ERR_NULL
    assert prefill(bd, q=None) == bd.BD_ERR_NULL
    assert prefill(bd, T=-1) == bd.BD_ERR_SHAPE
    assert prefill(bd, sinks=-2) == bd.BD_ERR_SHAPE
    assert prefill(bd, stride=8) == bd.BD_ERR_SHAPE
    assert prefill(bd, wsb=64) == bd.BD_ERR_WORKSPACE
    assert prefill(bd, T=0, ws=None, q=None) == bd.BD_OK


def test_evict_arguments(bd):
    assert evict(bd, weights=None) == bd.BD_ERR_NULL
    assert evict(bd, lens=None) == bd.BD_ERR_NULL
    assert evict(bd, src=None) == bd.BD_ERR_NULL
    assert evict(bd, dst=None) == bd.BD_ERR_NULL
    assert evict(bd, budget=0) == bd.BD_ERR_SHAPE
    assert evict(bd, budget=101) == bd.BD_ERR_SHAPE
    assert evict(bd, sinks=41) == bd.BD_ERR_SHAPE                # sinks + recent > budget
    assert evict(bd, recent=-1) == bd.BD_ERR_SHAPE
    assert evict(bd, sinks=2 ** 62, recent=2 ** 62) == bd.BD_ERR_SHAPE
    assert evict(bd, n=-1) == bd.BD_ERR_SHAPE
    assert evict(bd, kept=0x10003) == bd.BD_ERR_ALIGN
    assert evict(bd, ws=None) == bd.BD_ERR_WORKSPACE
    assert evict(bd, wsb=8) == bd.BD_ERR_WORKSPACE
    assert evict(bd, n=0, src=None, dst=None, ws=None) == bd.BD_OK


def test_workspace_sizes(bd):
    w = bd.bitdelta_attn_workspace
    assert w(64, 64, 64, 8, 128, 0) > 0
    assert w(0, 0, 64, 8, 128, 0) > 0
    assert w(64, 64, 64, 8, 128, 4096) >= w(64, 64, 64, 8, 128, 0)
    for bad in ((-1, 1, 64, 8, 128, 0), (1, -1, 64, 8, 128, 0), (1, 1, 63, 8, 128, 0), (1, 1, 64, 0, 128, 0), (1, 1, 64, 8, 100, 0), (1, 1, 64, 8, 128, -1),
                (1, 1, 64, 8, 128, 2 ** 24 + 1), (1, 65536, 64, 8, 128, 0), (1, 1, 258, 2, 128, 0)):
        assert w(*bad) == 0
    assert bd.bitdelta_evict_workspace(3, 8, 4096) > 0
    assert bd.bitdelta_evict_workspace(3, 0, 4096) == 0
    assert bd.bitdelta_evict_workspace(3, 8, 0) == 0


def test_new_status_has_a_text(bd):
    assert "slot" in bd.status_string(bd.BD_ERR_SLOT)

"""The 4-bit cache's entry points reject bad arguments on the host before touching a GPU."""
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
    c = dict(data=FAKE, slots=4, capacity=96, kv_heads=2, head_dim=128, stride_slot=2 * 6 * 2176, stride_head=6 * 2176)
    c.update(over)
    return ctypes.byref(bd.KVCache4Desc(*[c[name] for name, _ in bd.KVCache4Desc._fields_]))


BAD_CACHES = [
    (dict(data=None), "BD_ERR_NULL"), (dict(data=MISALIGNED), "BD_ERR_ALIGN"), (dict(slots=0), "BD_ERR_SHAPE"), (dict(slots=2 ** 24 + 1), "BD_ERR_SHAPE"),
    (dict(capacity=0), "BD_ERR_SHAPE"), (dict(capacity=100), "BD_ERR_SHAPE"), (dict(capacity=2 ** 24 + 16), "BD_ERR_SHAPE"), (dict(capacity=-16), "BD_ERR_SHAPE"),
    (dict(kv_heads=0), "BD_ERR_SHAPE"), (dict(head_dim=96), "BD_ERR_SHAPE"), (dict(head_dim=32), "BD_ERR_SHAPE"), (dict(stride_slot=0), "BD_ERR_SHAPE"),
    (dict(stride_head=-16), "BD_ERR_SHAPE"), (dict(stride_slot=2 ** 40), "BD_ERR_SHAPE"), (dict(stride_head=2184), "BD_ERR_ALIGN"),
]


def move(bd, entry, c="ok", k=FAKE, k_stride=256, v=FAKE, v_stride=256, T=10, B=3, slots=None, cu=FAKE, lens=FAKE, ws=FAKE, wsb=256):
    c = cache(bd) if c == "ok" else c
    return getattr(bd, "bitdelta_cache4_" + entry)(k, k_stride, v, v_stride, T, B, c, slots, cu, lens, ws, wsb, None)


def decode(bd, c="ok", q=FAKE, stride=1024, B=3, heads=8, lens=FAKE, slots=None, window=0, sinks=0, scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40):
    c = cache(bd) if c == "ok" else c
    return bd.bitdelta_attn4_decode(q, stride, B, heads, c, slots, lens, window, sinks, scale, out, ws, wsb, None)


def prefill(bd, c="ok", q=FAKE, stride=1024, T=10, B=3, heads=8, cu=FAKE, lens=FAKE, longest=50, window=0, sinks=0, scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40):
    c = cache(bd) if c == "ok" else c
    return bd.bitdelta_attn4_prefill(q, stride, T, B, heads, c, None, cu, lens, longest, window, sinks, scale, out, ws, wsb, None)


@pytest.mark.parametrize("over,code", BAD_CACHES, ids=str)
def test_caches(bd, over, code):
    code, c = getattr(bd, code), cache(bd, **over)
    assert move(bd, "write", c=c) == code and move(bd, "read", c=c) == code
    assert decode(bd, c=c) == code and prefill(bd, c=c) == code


@pytest.mark.parametrize("entry", ["write", "read"])
def test_rows(bd, entry):
    def call(**over):
        return move(bd, entry, **over)
    assert call(c=None) == bd.BD_ERR_NULL
    assert call(k=None) == bd.BD_ERR_NULL
    assert call(v=None) == bd.BD_ERR_NULL
    assert call(lens=None) == bd.BD_ERR_NULL
    assert call(k=MISALIGNED) == bd.BD_ERR_ALIGN
    assert call(v=MISALIGNED) == bd.BD_ERR_ALIGN
    assert call(k_stride=252) == bd.BD_ERR_SHAPE              # rows would overlap
    assert call(v_stride=0) == bd.BD_ERR_SHAPE
    assert call(k_stride=260) == bd.BD_ERR_ALIGN
    assert call(v_stride=2 ** 40) == bd.BD_ERR_SHAPE
    assert call(T=-1) == bd.BD_ERR_SHAPE
    assert call(T=2 ** 30 + 1) == bd.BD_ERR_SHAPE
    assert call(B=-1) == bd.BD_ERR_SHAPE
    assert call(B=65536) == bd.BD_ERR_SHAPE
    assert call(cu=None) == bd.BD_ERR_SHAPE                   # ten rows for three requests
    assert call(lens=0x10002) == bd.BD_ERR_ALIGN
    assert call(slots=0x10001) == bd.BD_ERR_ALIGN
    assert call(cu=0x10003) == bd.BD_ERR_ALIGN
    assert call(ws=None) == bd.BD_ERR_WORKSPACE
    assert call(wsb=255) == bd.BD_ERR_WORKSPACE
    assert call(ws=MISALIGNED) == bd.BD_ERR_ALIGN
    assert call(T=0, k=None, v=None, lens=None, ws=None) == bd.BD_OK
    assert call(T=0, B=0, cu=None, k=None, v=None, lens=None, ws=None) == bd.BD_OK


@pytest.mark.parametrize("call", [decode, prefill], ids=["decode", "prefill"])
def test_attention(bd, call):
    assert call(bd, c=None) == bd.BD_ERR_NULL
    assert call(bd, q=None) == bd.BD_ERR_NULL
    assert call(bd, out=None) == bd.BD_ERR_NULL
    assert call(bd, lens=None) == bd.BD_ERR_NULL
    assert call(bd, heads=7) == bd.BD_ERR_SHAPE
    assert call(bd, heads=2 * 129, stride=1 << 20) == bd.BD_ERR_SHAPE
    assert call(bd, B=-1) == bd.BD_ERR_SHAPE
    assert call(bd, B=65536) == bd.BD_ERR_SHAPE
    assert call(bd, window=-1) == bd.BD_ERR_SHAPE
    assert call(bd, sinks=-1) == bd.BD_ERR_SHAPE
    assert call(bd, scale=float("nan")) == bd.BD_ERR_SHAPE
    assert call(bd, scale=float("inf")) == bd.BD_ERR_SHAPE
    assert call(bd, stride=1016) == bd.BD_ERR_SHAPE
    assert call(bd, stride=1028) == bd.BD_ERR_ALIGN
    assert call(bd, q=MISALIGNED) == bd.BD_ERR_ALIGN
    assert call(bd, out=MISALIGNED) == bd.BD_ERR_ALIGN
    assert call(bd, lens=0x10002) == bd.BD_ERR_ALIGN
    assert call(bd, ws=None) == bd.BD_ERR_WORKSPACE
    assert call(bd, wsb=128) == bd.BD_ERR_WORKSPACE
    assert call(bd, ws=MISALIGNED) == bd.BD_ERR_ALIGN
    assert call(bd, B=0, q=None, out=None, lens=None, ws=None) == bd.BD_OK


def test_prompts(bd):
    assert prefill(bd, cu=None) == bd.BD_ERR_NULL
    assert prefill(bd, longest=0) == bd.BD_ERR_SHAPE
    assert prefill(bd, longest=-1) == bd.BD_ERR_SHAPE
    assert prefill(bd, longest=2 ** 24 + 1) == bd.BD_ERR_SHAPE
    assert prefill(bd, T=-1) == bd.BD_ERR_SHAPE
    assert prefill(bd, wsb=bd.bitdelta_attn4_workspace(10, 3, 8, 2, 128, 50) - 1) == bd.BD_ERR_WORKSPACE
    assert prefill(bd, T=0, q=None, ws=None) == bd.BD_OK
    # a workspace for shorter requests is too small for longer ones
    assert prefill(bd, longest=96, wsb=bd.bitdelta_attn4_workspace(10, 3, 8, 2, 128, 80)) == bd.BD_ERR_WORKSPACE


def test_sizes(bd):
    assert bd.bitdelta_cache4_bytes(3, 96, 2, 128) == 3 * 6 * 2 * 2176
    assert bd.bitdelta_cache4_bytes(3, 96, 2, 64) == 3 * 6 * 2 * 1088
    for bad in ((0, 96, 2, 128), (3, 100, 2, 128), (3, 0, 2, 128), (3, 96, 0, 128), (3, 96, 2, 100), (2 ** 24 + 1, 96, 2, 128), (2 ** 24, 2 ** 24, 2 ** 31 - 1, 128)):
        assert bd.bitdelta_cache4_bytes(*bad) == 0
    w = bd.bitdelta_attn4_workspace
    assert w(64, 64, 64, 8, 128, 0) >= bd.bitdelta_attn_workspace(64, 64, 64, 8, 128, 0) > 0
    assert w(64, 2, 64, 8, 128, 1000) - w(64, 2, 64, 8, 128, 0) >= 4 * 2 * 8 * 1008 * 128
    for bad in ((-1, 1, 64, 8, 128, 0), (1, -1, 64, 8, 128, 0), (1, 1, 63, 8, 128, 0), (1, 1, 64, 0, 128, 0), (1, 1, 64, 8, 100, 0), (1, 1, 64, 8, 128, -1),
                (1, 1, 64, 8, 128, 2 ** 24 + 1), (1, 65536, 64, 8, 128, 0), (1, 65535, 64, 8, 128, 2 ** 24)):
        assert w(*bad) == 0


def test_description_is_packed_as_the_struct(bd):
    assert bd._DESC4.size == ctypes.sizeof(bd.KVCache4Desc)
    raw = bd._DESC4.pack(16, 2, 3, 4, 5, 6, 7)
    desc = bd.KVCache4Desc.from_buffer_copy(raw)
    assert [getattr(desc, name) for name, _ in desc._fields_] == [16, 2, 3, 4, 5, 6, 7]

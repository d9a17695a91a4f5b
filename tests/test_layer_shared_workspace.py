"""Caches of several layers with one workspace: ``CachedAttention(ws=...)``, and what room prompts
on a 4-bit cache ask for.  On the CPU: nothing is launched."""
import pytest
import torch

SLOTS, CAP, HQ, HK, D, TOKENS, BATCH = 4, 160, 8, 2, 64, 48, 3


@pytest.fixture(scope="module")
def bd():
    from bit_delta_compressed_gb300 import build
    build.build()
    import bit_delta_compressed_gb300 as bd
    return bd


def make(bd, **more):
    from bit_delta_compressed_gb300 import layer
    how = dict(tokens=TOKENS, batch=BATCH, device="cpu")
    return layer.CachedAttention(bd, SLOTS, CAP, HQ, HK, D, **{**how, **more})


@pytest.mark.parametrize("bits", [4, 16])
def test_one_workspace(bd, bits):
    first = make(bd, bits=bits)
    second = make(bd, bits=bits, ws=first.ws)
    assert second.ws is first.ws
    assert (second.cache if bits == 4 else second.k).data_ptr() != (first.cache if bits == 4 else first.k).data_ptr()
    assert make(bd, bits=bits).ws.data_ptr() != first.ws.data_ptr()
    # one of smaller layers may use it, and so may one of the other kind where it is large enough
    assert make(bd, bits=bits, ws=first.ws, tokens=5, batch=1).ws is first.ws
    if bits == 4:
        assert make(bd, ws=first.ws).ws is first.ws


@pytest.mark.parametrize("sizes", [dict(tokens=20000), dict(batch=400), dict(bits=4, longest=CAP, batch=BATCH + 1)], ids=str)
def test_one_that_is_too_small(bd, sizes):
    small = make(bd, bits=sizes.get("bits", 16))
    with pytest.raises(ValueError, match="workspace"):
        make(bd, ws=small.ws, **sizes)
    with pytest.raises(ValueError, match="workspace"):
        make(bd, bits=4, ws=torch.zeros(0, dtype=torch.uint8))


@pytest.mark.parametrize("slots,capacity,longest", [(128, 16384, 16384), (16, 4096, 1000), (3, 160, 1)])
def test_bytes(bd, slots, capacity, longest):
    """The cache takes 17/64 of the bf16 cache's bytes, and a workspace 4 * batch * kv_heads * longest * head_dim
    beside what attention on the bf16 cache asks for, `longest` in whole blocks."""
    hq, hk, d = 64, 8, 128
    assert bd.bitdelta_cache4_bytes(slots, capacity, hk, d) * 64 == slots * capacity * hk * d * 4 * 17
    own = bd.bitdelta_attn_workspace(256, slots, hq, hk, d, 0)
    whole = bd.bitdelta_attn4_workspace(256, slots, hq, hk, d, longest)
    room = 4 * slots * hk * -(-longest // 16) * 16 * d
    assert 0 <= whole - own - room <= 1024
    assert bd.bitdelta_attn4_workspace(256, slots, hq, hk, d, 0) == own

"""``CachedAttention(bits=4)`` hands the library's calls the lengths they need: new tokens within
their slots, and no length at all for what is not served.  On the CPU, with the calls recorded."""
import pytest
import torch

from bit_delta_compressed_gb300 import layer

SLOTS, CAP, HQ, HK, D = 4, 16, 4, 2, 64


class Recorder:
    def cache4(self, slots, capacity, kv_heads, head_dim, device):
        return torch.zeros(slots, kv_heads, capacity // 16, 17 * head_dim, dtype=torch.uint8)

    def attn4_workspace(self, tokens, batch, q_heads, kv_heads, head_dim, longest, device):
        self.longest = longest
        return torch.zeros(1)

    def cache4_write(self, k, v, cache, lens, ws, slots=None, cu_q=None):
        self.wrote = dict(k=k, v=v, lens=lens, slots=slots, cu_q=cu_q)

    def attn4_decode(self, q, cache, lens, ws, slots=None, **mask):
        self.asked = dict(q=q, lens=lens, slots=slots, **mask)
        return torch.zeros_like(q)

    def attn4_prefill(self, q, cache, cu_q, lens, ws, longest, slots=None, **mask):
        self.asked = dict(q=q, cu_q=cu_q, lens=lens, longest=longest, slots=slots, **mask)
        return torch.zeros_like(q)


def i32(values):
    return torch.tensor(values, dtype=torch.int32)


def make(lens, **more):
    c = layer.CachedAttention(Recorder(), SLOTS, CAP, HQ, HK, D, tokens=32, batch=4, window=9, sinks=2, device="cpu", bits=4, **more)
    c.lens = i32(lens)
    return c


def rows(n):
    g = torch.Generator().manual_seed(n)
    return [torch.randn(n, h * D, generator=g).to(torch.bfloat16) for h in (HQ, HK, HK)]


def test_decode():
    c = make([0, 3, CAP - 1, CAP])
    q, k, v = rows(5)
    slots = i32([2, 0, 3, -1, SLOTS])
    assert c.decode(q, k, v, slots).shape == (5, HQ * D)
    assert c.lens.tolist() == [1, 3, CAP, CAP]
    for call in (c.bd.wrote, c.bd.asked):
        # a full slot, and ones that are not there, by a length beyond the capacity
        assert call["lens"].tolist() == [CAP, 1, CAP + 1, CAP + 1, CAP + 1] and torch.equal(call["slots"], slots)
        assert call["lens"].dtype == torch.int32
    assert torch.equal(c.bd.wrote["k"], k.view(5, HK, D)) and torch.equal(c.bd.wrote["v"], v.view(5, HK, D)) and c.bd.wrote["cu_q"] is None
    assert c.bd.asked["window"] == 9 and c.bd.asked["sinks"] == 2


@pytest.mark.parametrize("cu,have,lens,after", [
    ([0, 4, 5, 5, 7], [0, 3, 1, 14], [4, 4, 1, 16], [4, 4, 1, 16]),
    ([0, 4, 5, 5, 7], [0, 3, 1, 15], [4, 4, 1, -1], [4, 4, 1, 15]),              # no room for two more
    ([0, 4, 2, 5, 7], [0, 3, 1, 2], [4, -1, -1, -1], [4, 3, 1, 2]),              # offsets that do not ascend
    ([0, 4, 5, 6, 9], [0, 3, 1, 2], [4, 4, 2, -1], [4, 4, 2, 2]),                # more rows than there are
])
def test_prefill(cu, have, lens, after):
    c = make(have)
    q, k, v = rows(7)
    slots = i32([0, 1, 2, 3])
    assert c.prefill(q, k, v, slots, i32(cu)).shape == (7, HQ * D)
    assert c.lens.tolist() == after
    for call in (c.bd.wrote, c.bd.asked):
        assert call["lens"].tolist() == lens and call["cu_q"].tolist() == cu and call["lens"].dtype == torch.int32
    assert c.bd.asked["longest"] == CAP == c.bd.longest


def test_longest():
    c = make([0, 3, 1, 12], longest=10)
    assert c.bd.longest == 10
    q, k, v = rows(9)
    c.prefill(q, k, v, i32([0, 1, 2, 3]), i32([0, 2, 2, 9, 9]))
    assert c.bd.asked["lens"].tolist() == [2, 3, 8, 12] and c.lens.tolist() == [2, 3, 8, 12]    # nothing new in the long one
    c.prefill(q, k, v, i32([0, 1, 2, 3]), i32([0, 2, 2, 5, 6]))
    assert c.bd.asked["lens"].tolist() == [4, 3, -1, -1] and c.lens.tolist() == [4, 3, 8, 12]
    c.decode(*rows(1), i32([3]))
    assert c.lens.tolist() == [4, 3, 8, 13]


def test_a_refused_call_leaves_the_lengths(monkeypatch):
    c = make([0, 3, 1, 2])
    for name in ("cache4_write", "attn4_decode", "attn4_prefill"):
        with monkeypatch.context() as m:
            def refuse(*a, **b):
                raise ValueError("refused")
            m.setattr(c.bd, name, refuse, raising=False)
            if name != "attn4_prefill":
                with pytest.raises(ValueError):
                    c.decode(*rows(2), i32([0, 3]))
            if name != "attn4_decode":
                with pytest.raises(ValueError):
                    c.prefill(*rows(3), i32([0, 3]), i32([0, 1, 3]))
        assert c.lens.tolist() == [0, 3, 1, 2]


def test_what_a_4_bit_cache_does_not_do():
    bd = Recorder()
    for wrong in (dict(bits=8), dict(bits=4, weigh=True), dict(bits=16, longest=10)):
        with pytest.raises(ValueError):
            layer.CachedAttention(bd, SLOTS, CAP, HQ, HK, D, tokens=8, batch=2, device="cpu", **wrong)
    c = make([0, 3, 1, 2])
    for prefix in (dict(prefix_ids=i32([0]), prefix_slots=i32([1])), dict(prefix_ids=i32([0])), dict(prefix_slots=i32([1]))):
        with pytest.raises(ValueError):
            c.decode(*rows(1), i32([0]), **prefix)
        with pytest.raises(ValueError):
            c.prefill(*rows(1), i32([0]), i32([0, 1]), **prefix)
    with pytest.raises(ValueError):
        c.evict(i32([0]), i32([1]), budget=2, recent=8)
    assert c.k is None and c.v is None and c.weights is None and c.lens.tolist() == [0, 3, 1, 2]

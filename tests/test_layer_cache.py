"""``CachedAttention`` appends within its cache whatever slots, lengths and row
offsets it is given: no index leaves the tensors (on a GPU that would end the
CUDA context), nothing else is overwritten, and the attention call gets what it
needs to report the error.  On the CPU, with the library's calls recorded."""
import pytest
import torch

from bit_delta_compressed_gb300 import layer

SLOTS, CAP, HQ, HK, D = 4, 6, 4, 2, 8


class Recorder:
    """The library's attention calls, as far as the layer makes them."""

    def attn_workspace(self, *sizes):
        return torch.zeros(1)

    evict_workspace = attn_workspace

    def attn_decode_prefix(self, q, k, v, lens, ids, pslots, plens, ws, slots=None, **rest):
        self.lens, self.slots, self.pslots, self.plens = lens, slots, pslots, plens
        return torch.zeros_like(q)

    def cache_evict(self, k, v, weights, lens, src, dst, budget, ws, **rest):
        self.evicted = dict(src=src, dst=dst, budget=budget, **rest)

    def attn_prefill(self, q, k, v, cu_q, lens, ws, slots=None, prefix_slots=None, prefix_lens=None, **rest):
        self.cu, self.lens, self.slots, self.pslots, self.plens = cu_q, lens, slots, prefix_slots, prefix_lens
        return torch.zeros_like(q)


def i32(values):
    return torch.tensor(values, dtype=torch.int32)


def make(lens):
    """A cache of old values, and copies that a test fills as it expects them."""
    g = torch.Generator().manual_seed(1)
    c = layer.CachedAttention(Recorder(), SLOTS, CAP, HQ, HK, D, tokens=32, batch=4, weigh=True, device="cpu")
    for t in (c.k, c.v, c.weights):
        t.copy_(torch.randn(t.shape, generator=g))
    c.lens.copy_(i32(lens))
    return c, {name: getattr(c, name).clone() for name in ("k", "v", "weights", "lens")}


def rows(n):
    g = torch.Generator().manual_seed(n)
    return [torch.randn(n, h * D, generator=g).to(torch.bfloat16) for h in (HQ, HK, HK)]


def put(want, k, v, row, slot, at):
    want["k"][slot, at], want["v"][slot, at] = k[row].view(HK, D), v[row].view(HK, D)
    want["weights"][slot, :, at] = 0


def same(c, want):
    for name, t in want.items():
        assert torch.equal(getattr(c, name), t), name


def test_decode_appends():
    c, want = make([0, 3, CAP - 1, 2])
    q, k, v = rows(3)
    assert c.decode(q, k, v, i32([2, 0, 1])).shape == (3, HQ * D)
    for row, (slot, at) in enumerate([(2, CAP - 1), (0, 0), (1, 3)]):
        put(want, k, v, row, slot, at)
    want["lens"] = i32([1, 4, CAP, 2])
    same(c, want)
    assert c.bd.lens.tolist() == [CAP, 1, 4] and c.bd.lens.dtype == torch.int32


@pytest.mark.parametrize("bad", [-1, SLOTS, 2 ** 31 - 1, -2 ** 31])
def test_decode_with_a_full_slot_and_one_out_of_range(bad):
    c, want = make([0, CAP, 2, 1])
    q, k, v = rows(4)
    slots = i32([1, bad, 2, 0])
    c.decode(q, k, v, slots)
    put(want, k, v, 2, 2, 2)
    put(want, k, v, 3, 0, 0)
    want["lens"] = i32([1, CAP, 3, 1])
    same(c, want)
    # the attention call sees a length beyond the slot, and the slot as it was given
    assert c.bd.lens[0] > CAP and c.bd.lens[2:].tolist() == [3, 1]
    assert torch.equal(c.bd.slots, slots)


def test_decode_with_nothing_to_append():
    c, want = make([CAP] * SLOTS)
    c.decode(*rows(2), i32([3, -7]))
    same(c, want)
    c.decode(*rows(0), i32([]))
    same(c, want)


@pytest.mark.parametrize("bad", [-1, SLOTS, 2 ** 31 - 1])
def test_prefix_slots_out_of_range(bad):
    c, _ = make([3, 1, 2, 5])
    c.decode(*rows(1), i32([1]), i32([0]), i32([0, bad]))
    assert c.bd.plens[0] == 3 and c.bd.pslots.tolist() == [0, bad]
    c.prefill(*rows(2), i32([1]), i32([0, 2]), i32([0]), i32([bad, 3]))
    assert c.bd.plens[1] == 5 and c.bd.pslots.tolist() == [bad, 3]


def test_prefill_appends():
    c, want = make([0, 3, 1, 2])
    q, k, v = rows(7)
    c.prefill(q, k, v, i32([3, 0, 1, 2]), i32([0, 4, 5, 5, 7]))
    for row, (slot, at) in enumerate([(3, 2), (3, 3), (3, 4), (3, 5), (0, 0), (2, 1), (2, 2)]):
        put(want, k, v, row, slot, at)
    want["lens"] = i32([1, 3, 3, 6])
    same(c, want)
    assert c.bd.lens.tolist() == [6, 1, 3, 3] and c.bd.lens.dtype == torch.int32


def test_prefill_rows_outside_every_request():
    c, want = make([0, 3, 1, 2])
    q, k, v = rows(9)
    c.prefill(q, k, v, i32([1, 0]), i32([2, 5, 6]))
    for row, (slot, at) in zip(range(2, 6), [(1, 3), (1, 4), (1, 5), (0, 0)]):
        put(want, k, v, row, slot, at)
    want["lens"] = i32([1, 6, 1, 2])
    same(c, want)
    c.prefill(q, k, v, i32([]), i32([0]))
    same(c, want)


@pytest.mark.parametrize("bad", [-1, SLOTS, 2 ** 31 - 1])
def test_prefill_with_a_prompt_too_long_and_a_slot_out_of_range(bad):
    """Neither is appended, not even in part; the others are."""
    c, want = make([0, 3, 1, 2])
    q, k, v = rows(10)
    c.prefill(q, k, v, i32([1, bad, 0]), i32([0, 4, 7, 10]))
    for row in range(3):
        put(want, k, v, 7 + row, 0, row)
    want["lens"] = i32([3, 3, 1, 2])
    same(c, want)
    assert c.bd.lens[0] == 7 and c.bd.lens[2] == 3


@pytest.mark.parametrize("cu", [[0, 2, 9, 4, 8], [0, 2, 1, 4, 8], [0, 2, -1, 4, 8], [0, 2, 2 ** 31 - 1, -2 ** 31, 8], [0, 2, -2 ** 31, 5, 8]])
def test_prefill_with_offsets_that_do_not_ascend(cu):
    """The requests before the first break are appended, those from it on are not."""
    c, want = make([0, 3, 1, 2])
    q, k, v = rows(8)
    c.prefill(q, k, v, i32([0, 1, 2, 3]), i32(cu))
    put(want, k, v, 0, 0, 0)
    put(want, k, v, 1, 0, 1)
    want["lens"] = i32([2, 3, 1, 2])
    same(c, want)
    assert c.bd.cu.tolist() == cu


def test_evict_under_a_window():
    """Kept keys move nearer: keys that had left the window would be in it again unless it lies among the recent ones."""
    for window, recent, ok in ((0, 0, True), (1, 0, True), (4, 2, False), (4, 3, True), (4, 5, True), (4, 0, False)):
        c = layer.CachedAttention(Recorder(), SLOTS, CAP, HQ, HK, D, tokens=4, batch=4, window=window, sinks=1, weigh=True, device="cpu")
        c.bd.evicted = None
        if ok:
            c.evict(i32([0]), i32([1]), 6, recent)
            assert c.bd.evicted["recent"] == recent and c.bd.evicted["sinks"] == 1
        else:
            with pytest.raises(ValueError, match="window"):
                c.evict(i32([0]), i32([1]), 6, recent)
            assert c.bd.evicted is None


def test_evict_behind_a_prefix():
    """The mask's first tokens lie in the prefix as far as it reaches: the caller says how many are own keys."""
    c = layer.CachedAttention(Recorder(), SLOTS, CAP, HQ, HK, D, tokens=4, batch=4, sinks=4, weigh=True, device="cpu")
    for sinks, kept in ((None, 4), (0, 0), (1, 1)):
        c.evict(i32([0]), i32([1]), 6, 2, sinks=sinks)
        assert c.bd.evicted["sinks"] == kept


def test_assigned_tensors_reach_the_steps():
    """A cache that is put back from a copy goes on from there."""
    c, want = make([0, 3, 1, 2])
    c.decode(*rows(2), i32([0, 1]))
    for name, t in want.items():
        setattr(c, name, t)
    c.lens += 1
    want["lens"] += 1
    q, k, v = rows(1)
    c.decode(q, k, v, i32([3]))
    put(want, k, v, 0, 3, 3)
    want["lens"] = i32([1, 4, 2, 4])
    same(c, want)


def test_refused_calls_append_nothing():
    """A step whose attention call is refused leaves the lengths as they were, so it can be made again."""
    c, want = make([0, 3, CAP, 2])

    def refuse(*args, **how):
        raise ValueError("refused")
    c.bd.attn_decode_prefix = c.bd.attn_prefill = refuse
    for step in (lambda: c.decode(*rows(3), i32([0, 2, 3])), lambda: c.decode(*rows(2), i32([-1, SLOTS])),
                 lambda: c.prefill(*rows(6), i32([3, 0, 2, 9]), i32([0, 2, 3, 5, 6]))):
        with pytest.raises(ValueError, match="refused"):
            step()
        assert torch.equal(c.lens, want["lens"])
        for b, n in enumerate(want["lens"].tolist()):
            assert torch.equal(c.k[b, :n], want["k"][b, :n]) and torch.equal(c.weights[b, :, :n], want["weights"][b, :, :n])

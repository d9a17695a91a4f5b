"""GPU: ``CachedAttention`` at the ends of its slots: what fits is served, what
does not comes out as zeros and is reported, eagerly and from a CUDA graph."""
import pytest
import torch

from bit_delta_compressed_gb300 import layer
from tests import attention_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLOTS, CAP, HQ, HK, D = 5, 40, 8, 2, 64


@pytest.fixture(scope="module")
def bd():
    return load_bd()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def make(bd, lens, **how):
    g = torch.Generator(DEV).manual_seed(sum(lens))
    c = layer.CachedAttention(bd, SLOTS, CAP, HQ, HK, D, tokens=64, batch=4, device=DEV, **how)
    c.k.copy_(torch.randn(c.k.shape, generator=g, device=DEV))
    c.v.copy_(torch.randn(c.v.shape, generator=g, device=DEV))
    c.lens.copy_(i32(lens))
    return c, g


def rows(n, g):
    return [torch.randn(n, h * D, generator=g, device=DEV).to(torch.bfloat16) for h in (HQ, HK, HK)]


def test_decode_at_the_end_of_a_slot(bd):
    """Slots with one free place, none, and of no number at all; the step after that, too."""
    c, g = make(bd, [CAP - 1, CAP, 7, 0, 12])
    slots = i32([0, 1, -1, 2])
    for step, lens in enumerate(([CAP, CAP, 8, 0, 12], [CAP, CAP, 9, 0, 12])):
        old = c.k.clone()
        q, k, v = rows(4, g)
        out = c.decode(q, k, v, slots).view(4, HQ, D)
        assert bd.device_status(c.ws) == bd.BD_ERR_SLOT
        assert c.lens.tolist() == lens
        good = [0, 3] if step == 0 else [3]
        want, bound, _ = ref.attention(q.view(4, HQ, D)[good], c.k, c.v, i32([lens[int(slots[b])] for b in good]), slots=slots[good])
        ref.assert_close(out[good], want, bound)
        assert (out[[b for b in range(4) if b not in good]] == 0).all()
        for b in good:
            s = int(slots[b])
            old[s, lens[s] - 1] = k[b].view(HK, D)
        assert torch.equal(c.k, old)


def test_prefill_beyond_the_end_of_a_slot(bd):
    c, g = make(bd, [CAP - 3, CAP - 3, 0, 5, 12])
    q, k, v = rows(30, g)
    slots, cu = i32([1, 0, SLOTS, 2]), i32([0, 3, 7, 10, 30])
    out = c.prefill(q, k, v, slots, cu).view(30, HQ, D)
    assert bd.device_status(c.ws) == bd.BD_ERR_SLOT
    assert c.lens.tolist() == [CAP - 3, CAP, 20, 5, 12]
    mine = list(range(3)) + list(range(10, 30))
    want, bound, _ = ref.attention(q.view(30, HQ, D)[mine], c.k, c.v, i32([CAP, 20]), slots=i32([1, 2]), cu_q=[0, 3, 23])
    ref.assert_close(out[mine], want, bound)
    assert (out[3:10] == 0).all()


@pytest.mark.parametrize("weigh", [False, True], ids=["", "weigh"])
def test_decode_steps_from_a_graph(bd, weigh):
    """The captured step goes on until its slot is full, then leaves it alone."""
    c, g = make(bd, [CAP - 3, 4, 0, 0, 0], weigh=weigh)
    slots = i32([0, 1])
    q, k, v = rows(2, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.decode(q, k, v, slots)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = c.decode(q, k, v, slots)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(4):
        for t, new in zip((q, k, v), rows(2, g)):
            t.copy_(new)
        graph.replay()
        full = step >= 2
        assert c.lens[:2].tolist() == [CAP if full else CAP - 1 + step, 6 + step]
        assert bd.device_status(c.ws) == (bd.BD_ERR_SLOT if full else 0)
        good = [1] if full else [0, 1]
        want, bound, _ = ref.attention(q.view(2, HQ, D)[good], c.k, c.v, c.lens[good], slots=slots[good])
        ref.assert_close(out.view(2, HQ, D)[good], want, bound)
        if full:
            assert (out[0] == 0).all()
        if weigh:
            # this step's key has what this step gave it, and the head's weights sum to the steps' number
            at = 5 + step
            _, _, (added, rel) = ref.attention(q.view(2, HQ, D)[1:], c.k, c.v, i32([at + 1]), slots=i32([1]))
            one = added[0][:, at]
            assert ((c.weights[1, :, at].double() - one).abs() <= (rel[0] + (HQ // HK + 2) * ref.F32) * one).all()
            most = (step + 2) * (HQ // HK)
            assert ((c.weights[1, :, :at + 1].double().sum(-1) - most).abs() <= 1e-3 * most).all()


@pytest.mark.parametrize("window,sinks,prefix", [(9, 0, 0), (9, 3, 0), (1, 2, 0), (9, 4, 2), (9, 2, 12), (16, 0, 20)])
def test_windowed_steps_after_an_eviction(bd, window, sinks, prefix):
    """The steps see what they would see had nothing been evicted: the mask taken over the tokens' own positions."""
    c, g = make(bd, [30, 0, 0, 0, prefix], window=window, sinks=sinks, weigh=True)
    c.weights.copy_(torch.rand(c.weights.shape, generator=g, device=DEV))
    how = (i32([0]), i32([4])) if prefix else (None, None)
    front = [(c.k[4, j].double(), c.v[4, j].double()) for j in range(prefix)]
    tokens = front + [(c.k[0, j].double(), c.v[0, j].double()) for j in range(30)]
    c.evict(i32([0]), i32([2]), budget=24, recent=window + 2)
    assert int(c.lens[2]) == 24
    for _ in range(12):
        q, k, v = rows(1, g)
        out = c.decode(q, k, v, i32([2]), *how).view(HQ, D)
        tokens.append((k.view(HK, D).double(), v.view(HK, D).double()))
        t = len(tokens) - 1
        seen = [p for p in range(t + 1) if p < sinks or p > t - window]
        kk, vv = (torch.stack([tokens[p][i] for p in seen]) for i in (0, 1))
        # the same keys in a cache of their own, all of them visible
        kc, vc = (x[None].to(torch.bfloat16) for x in (kk, vv))
        want, bound, _ = ref.attention(q.view(1, HQ, D), kc, vc, i32([len(seen)]), rounded=bool(prefix))
        ref.assert_close(out[None], want, bound)
        assert bd.device_status(c.ws) == 0


@pytest.mark.parametrize("prefix", [2, 12])
def test_eviction_behind_a_prefix_keeps_the_heaviest(bd, prefix):
    """Own keys that the mask's first tokens do not hold are kept by weight alone, and the windowed steps stay right."""
    c, g = make(bd, [30, 0, 0, 0, prefix], window=5, sinks=4, weigh=True)
    c.weights.copy_(torch.rand(c.weights.shape, generator=g, device=DEV))
    c.weights[0, :, :4] = 0                               # the first own keys are the lightest
    kept, before = max(0, 4 - prefix), c.k[0].clone()
    c.evict(i32([0]), i32([2]), budget=15, recent=6, sinks=kept)
    for h, rows_kept in enumerate(ref.evict(c.weights.cpu(), c.lens.cpu(), i32([0]).cpu(), 15, kept, 6)[0]):
        assert rows_kept[kept] >= 4
        assert torch.equal(c.k[2, :15, h], before[rows_kept, h])
    q, k, v = rows(1, g)
    out = c.decode(q, k, v, i32([2]), i32([0]), i32([4])).view(1, HQ, D)
    keys, values = (torch.cat([t[4, :min(4, prefix)], t[0, :kept], t[0, 26:30], new.view(1, HK, D)])[None]
                    for t, new in ((c.k, k), (c.v, v)))
    want, bound, _ = ref.attention(q.view(1, HQ, D), keys, values, i32([9]), rounded=True)
    ref.assert_close(out, want, bound)

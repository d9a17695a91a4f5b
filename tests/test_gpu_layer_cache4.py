"""GPU: a decoder layer whose cache is held in 4 bits: prompts, further chunks and decode steps
through ``CachedAttention(bits=4)``, by themselves and from a captured graph."""
import pytest
import torch

import workloads as wl
from bit_delta_compressed_gb300 import layer
from tests import attention_ref
from tests import cache4_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HK, D = 8, 2, 128
HIDDEN, KV, FFN = HQ * D, HK * D, 2048
SHAPES = {"q": (HIDDEN, HIDDEN), "k": (KV, HIDDEN), "v": (KV, HIDDEN), "o": (HIDDEN, HIDDEN), "gate": (FFN, HIDDEN), "up": (FFN, HIDDEN), "down": (HIDDEN, FFN)}


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 2)])
def test_layer(window, sinks):
    bd = load_bd()
    g = wl.generator(400, DEV)
    V, ids = 3, [0, 0, 2, 1]                              # the variants of the four requests
    lin = {}
    for name, (N, K) in SHAPES.items():
        bits = [torch.randint(-2 ** 31, 2 ** 31, (N, K // 32), generator=g, device=DEV, dtype=torch.int64).to(torch.int32) for _ in range(V)]
        lin[name] = {"wb": wl.base_weights(N, K, g, DEV), "alphas": 1e-3 * (1 + torch.rand(V, generator=g, device=DEV)),
                     "bits": bits, "ptrs": bd.bits_pointer_array(bits)}
    cache = layer.CachedAttention(bd, 9, 160, HQ, HK, D, tokens=128, batch=4, window=window, sinks=sinks, bits=4)
    ws = bd.linear_workspace(128, FFN, FFN, V, DEV)
    slots = i32([3, 0, 7, 5])
    before, have = cache.cache.cpu(), [0, 0, 0, 0]

    def step(counts, attend, cu):
        """A step of `counts` new tokens, and everything it left behind."""
        nonlocal before
        h = wl.activations(sum(counts), HIDDEN, g, DEV)
        bufs = {name: torch.empty((h.shape[0], SHAPES[name][0]), dtype=torch.bfloat16, device=DEV) for name in layer.NAMES}
        bd.group(i32([v for v, n in zip(ids, counts) for _ in range(n)]), V, ws)
        seen = {}

        def watched(q, k, v):
            seen.update(q=q, k=k, v=v, out=attend(q, k, v))
            return seen["out"]
        h2, parts = layer.chained_layer(bd, lin, h, V, ws, bufs, keep=True, attend=watched)
        assert bd.device_status(ws) == 0 and bd.device_status(cache.ws) == 0 and torch.isfinite(h2.float()).all()
        assert torch.equal(parts["o"][0], seen["out"])
        for b, n in enumerate(counts):
            have[b] += n
        want = ref.write(before, seen["k"].view(-1, HK, D), seen["v"].view(-1, HK, D), have, slots.tolist(), cu)
        assert torch.equal(cache.cache.cpu(), want) and cache.lens[slots.long()].tolist() == have
        before = want
        out, bound = ref.attention(seen["q"].view(-1, HQ, D), cache.cache, i32(have), slots=slots, cu_q=cu, window=window, sinks=sinks)
        attention_ref.assert_close(seen["out"].view(-1, HQ, D), out, bound)

    for counts in ([40, 7, 21, 33], [1, 0, 30, 5]):
        cu = [sum(counts[:i]) for i in range(5)]
        step(counts, lambda q, k, v: cache.prefill(q, k, v, slots, i32(cu)), cu)
    for _ in range(3):
        step([1, 1, 1, 1], lambda q, k, v: cache.decode(q, k, v, slots), None)


def test_full_slots_and_slots_that_are_not_there():
    bd = load_bd()
    g = wl.generator(401, DEV)
    cache = layer.CachedAttention(bd, 3, 32, HQ, HK, D, tokens=16, batch=4, bits=4, longest=30)
    cache.cache.copy_(torch.randint(0, 256, cache.cache.shape, generator=g, device=DEV, dtype=torch.uint8))
    cache.cache[..., 16 * D:] = 120                       # scales of 1
    cache.lens = i32([31, 32, 5])
    before = cache.cache.cpu()

    def rows(n):
        return [wl.activations(n, h * D, g, DEV) for h in (HQ, HK, HK)]

    q, k, v = rows(4)
    out = cache.decode(q, k, v, i32([1, -1, 0, 3])).view(-1, HQ, D)
    assert bd.device_status(cache.ws) == bd.BD_ERR_SLOT and cache.lens.tolist() == [32, 32, 5]
    before = ref.write(before, k[2:3].view(1, HK, D), v[2:3].view(1, HK, D), [32], [0])
    assert torch.equal(cache.cache.cpu(), before)
    want, bound = ref.attention(q[2:3].view(1, HQ, D), cache.cache, i32([32]))
    attention_ref.assert_close(out[2:3], want, bound)
    assert not out[[0, 1, 3]].any()
    # prompts: one that fits, one of a full slot, one of no slot
    q, k, v = rows(9)
    out = cache.prefill(q, k, v, i32([2, 1, 7]), i32([0, 4, 6, 9])).view(-1, HQ, D)
    assert bd.device_status(cache.ws) == bd.BD_ERR_SLOT and cache.lens.tolist() == [32, 32, 9]
    before = ref.write(before, k[:4].view(4, HK, D), v[:4].view(4, HK, D), [9], [2], [0, 4])
    assert torch.equal(cache.cache.cpu(), before)
    want, bound = ref.attention(q[:4].view(4, HQ, D), cache.cache, i32([9]), slots=[2], cu_q=[0, 4])
    attention_ref.assert_close(out[:4], want, bound)
    assert not out[4:].any()


def test_captured_steps():
    """A decode step as a graph: slots, lengths and rows change between replays."""
    bd = load_bd()
    g = wl.generator(402, DEV)
    cache = layer.CachedAttention(bd, 6, 64, HQ, HK, D, tokens=4, batch=3, window=20, sinks=1, bits=4)
    cache.lens = i32([0, 15, 16, 63, 64, 40])
    q, k, v = [wl.activations(3, h * D, g, DEV) for h in (HQ, HK, HK)]
    slots, kept = i32([0, 1, 2]), cache.lens.clone()
    cache.decode(q, k, v, slots)                          # outside the graph first
    cache.lens, graph = kept, torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = cache.decode(q, k, v, slots)
    have = kept.tolist()
    for names in ([0, 1, 2], [2, 3, 5], [3, 0, 4], [1, 2, 0]):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        slots.copy_(i32(names))
        before = cache.cache.cpu()
        graph.replay()
        served = [have[s] < 64 for s in names]
        for row, (s, ok) in enumerate(zip(names, served)):
            if ok:
                have[s] += 1
                before = ref.write(before, k[row:row + 1].view(1, HK, D), v[row:row + 1].view(1, HK, D), [have[s]], [s])
        assert cache.lens.tolist() == have and torch.equal(cache.cache.cpu(), before)
        lens = i32([have[s] if ok else 0 for s, ok in zip(names, served)])
        want, bound = ref.attention(q.view(3, HQ, D), cache.cache, lens, slots=names, window=20, sinks=1)
        attention_ref.assert_close(out.view(3, HQ, D), want, bound)
    assert bd.device_status(cache.ws) == bd.BD_ERR_SLOT

"""GPU: a decoder layer with its attention: prompts, shared prefixes, decode
steps and an eviction through one cache, each attention output checked on the
inputs it received."""
import pytest
import torch

import workloads as wl
from bit_delta_compressed_gb300 import layer
from tests import attention_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HK, D = 8, 2, 128
HIDDEN, KV, FFN = HQ * D, HK * D, 2048
SHAPES = {"q": (HIDDEN, HIDDEN), "k": (KV, HIDDEN), "v": (KV, HIDDEN), "o": (HIDDEN, HIDDEN),
          "gate": (FFN, HIDDEN), "up": (FFN, HIDDEN), "down": (HIDDEN, FFN)}


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def test_layer_with_cache():
    bd = load_bd()
    g = wl.generator(400, DEV)
    V, prompts = 3, [40, 7, 21, 33]
    ids = [0, 0, 2, 1]                                    # the variants of the four requests
    lin = {}
    for name, (N, K) in SHAPES.items():
        bits = [torch.randint(-2 ** 31, 2 ** 31, (N, K // 32), generator=g, device=DEV, dtype=torch.int64).to(torch.int32) for _ in range(V)]
        lin[name] = {"wb": wl.base_weights(N, K, g, DEV), "alphas": 1e-3 * (1 + torch.rand(V, generator=g, device=DEV)),
                     "bits": bits, "ptrs": bd.bits_pointer_array(bits)}
    cache = layer.CachedAttention(bd, 12, 160, HQ, HK, D, tokens=128, batch=4, sinks=2, weigh=True)
    ws = bd.linear_workspace(128, FFN, FFN, V, DEV)

    def step(h, variants, attend):
        M = h.shape[0]
        bufs = {name: torch.empty((M, SHAPES[name][0]), dtype=torch.bfloat16, device=DEV) for name in layer.NAMES}
        bd.group(i32(variants), V, ws)
        seen = {}

        def watched(q, k, v):
            seen["q"], seen["out"] = q, attend(q, k, v)
            return seen["out"]
        h2, parts = layer.chained_layer(bd, lin, h, V, ws, bufs, keep=True, attend=watched)
        assert bd.device_status(ws) == 0 and bd.device_status(cache.ws) == 0
        assert torch.equal(parts["o"][0], seen["out"]) and torch.isfinite(h2.float()).all()
        return seen["q"].view(M, HQ, D), seen["out"].view(M, HQ, D)

    # a prompt of variant 0 that its two requests share (slot 10), then the requests' own prompts
    q, out = step(wl.activations(50, HIDDEN, g, DEV), [0] * 50, lambda q, k, v: cache.prefill(q, k, v, i32([10]), i32([0, 50])))
    want, bound, _ = ref.attention(q, cache.k, cache.v, i32([50]), slots=[10], cu_q=[0, 50], sinks=2)
    ref.assert_close(out, want, bound)
    slots, pid, pslots = i32([3, 0, 7, 5]), i32([0, 0, -1, -1]), i32([10])
    cu = i32([sum(prompts[:i]) for i in range(5)])
    variants = [v for v, n in zip(ids, prompts) for _ in range(n)]
    q, out = step(wl.activations(sum(prompts), HIDDEN, g, DEV), variants, lambda q, k, v: cache.prefill(q, k, v, slots, cu, pid, pslots))
    how = dict(prefix_ids=pid, prefix_slots=pslots, prefix_lens=i32([50]), sinks=2)
    want, bound, _ = ref.attention(q, cache.k, cache.v, i32(prompts), slots=slots, cu_q=cu, **how)
    ref.assert_close(out, want, bound)
    # decode, evict one request into another slot, decode again
    expect = torch.zeros(4, HK, 160, dtype=torch.float64, device=DEV)
    for t in range(3):
        q, out = step(wl.activations(4, HIDDEN, g, DEV), ids, lambda q, k, v: cache.decode(q, k, v, slots, pid, pslots))
        lens = i32([n + t + 1 for n in prompts])
        want, bound, (added, _) = ref.attention(q, cache.k, cache.v, lens, slots=slots, **how)
        ref.assert_close(out, want, bound)
        for b in range(4):
            expect[b, :, :int(lens[b])] += added[b]
    got = cache.weights[slots.long()].double()
    assert ((got - expect).abs() <= 1e-4 * expect).all()
    before = cache.weights.clone()
    kept = ref.evict(before.cpu(), cache.lens.cpu(), i32([3]).cpu(), 30, 2, 8)
    cache.evict(i32([3]), i32([9]), budget=30, recent=8)
    assert int(cache.lens[9]) == 30
    for h in range(HK):
        assert torch.equal(cache.k[9, :30, h], cache.k[3, kept[0][h], h])
        assert torch.equal(cache.weights[9, h, :30], before[3, h, kept[0][h]])
    slots = i32([9, 0, 7, 5])
    q, out = step(wl.activations(4, HIDDEN, g, DEV), ids, lambda q, k, v: cache.decode(q, k, v, slots, pid, pslots))
    want, bound, _ = ref.attention(q, cache.k, cache.v, i32([31, 11, 25, 37]), slots=slots, **how)
    ref.assert_close(out, want, bound)

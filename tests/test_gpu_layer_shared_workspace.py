"""GPU: caches of several layers, 4-bit and bf16 ones, with one workspace give what each gives with its own."""
import pytest
import torch

import workloads as wl
from bit_delta_compressed_gb300 import layer
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HK, D, CAP = 16, 2, 128, 320


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("kinds", [(4, 4, 4), (4, 16, 4), (16, 4, 16)], ids=str)
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_layers(kinds, graph):
    bd = load_bd()
    g = wl.generator(90, DEV)

    def make(bits, ws=None):
        return layer.CachedAttention(bd, 6, CAP, HQ, HK, D, tokens=128, batch=4, window=100, sinks=3, bits=bits, ws=ws)

    room = make(4).ws                                       # the larger of both kinds'
    own, shared = [make(bits) for bits in kinds], [make(bits, room) for bits in kinds]
    assert all(c.ws is room for c in shared) and all(c.ws is not room for c in own)
    slots = i32([4, 0, 5, 2])

    def inputs(rows):
        return [[wl.activations(rows, h * D, g, DEV) for h in (HQ, HK, HK)] for _ in kinds]

    def check(step, x):
        for a, b in zip(step(own, x), step(shared, x)):
            assert torch.equal(a, b) and a.any()
        for a, b in zip(own, shared):
            assert torch.equal(a.lens, b.lens) and bd.device_status(a.ws) == 0 and bd.device_status(b.ws) == 0
            assert torch.equal(*((a.cache, b.cache) if a.cache is not None else (a.k, b.k)))

    for counts in ([60, 1, 40, 9], [2, 1, 3, 2], [1, 70, 1, 1]):
        cu = i32([sum(counts[:i]) for i in range(5)])
        check(lambda layers, x: [c.prefill(*y, slots, cu) for c, y in zip(layers, x)], inputs(sum(counts)))

    def decode(layers, x):
        return [c.decode(*y, slots) for c, y in zip(layers, x)]

    if not graph:
        for _ in range(3):
            check(decode, inputs(4))
        return
    x, graphs, outs = inputs(4), [], []
    check(decode, x)
    torch.cuda.synchronize()
    for layers in (own, shared):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(decode(layers, x))

    def replay(layers, fresh):
        for old, new in zip(x, fresh):
            for a, b in zip(old, new):
                a.copy_(b)
        at = 0 if layers is own else 1
        graphs[at].replay()
        return [out.clone() for out in outs[at]]

    for _ in range(3):
        check(replay, inputs(4))

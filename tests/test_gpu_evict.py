"""GPU: eviction by accumulated weight moves exactly the rows that sorting
names, for every tie, special value, budget and split."""
import math

import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bd():
    return load_bd()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def check_evict(bd, k, v, weights, lens, src, dst, budget, sinks, recent):
    n, hk = src.numel(), k.shape[2]
    k0, v0, w0, l0 = k.clone(), v.clone(), weights.clone(), lens.clone()
    kept = torch.full((n, hk, budget), -7, dtype=torch.int32, device=DEV)
    ws = bd.evict_workspace(n, hk, k.shape[1], device=DEV)
    bd.cache_evict(k, v, weights, lens, src, dst, budget, ws, sinks=sinks, recent=recent, kept=kept)
    assert bd.device_status(ws) == 0
    want = ref.evict(w0.cpu(), l0.cpu(), src.cpu(), budget, sinks, recent)
    for i in range(n):
        s, t = int(src[i]), int(dst[i])
        c = min(int(l0[s]), budget)
        assert int(lens[t]) == c
        l0[t] = c
        for h in range(hk):
            assert kept[i, h].tolist() == want[i][h] + [-1] * (budget - c)
            rows = torch.tensor(want[i][h], dtype=torch.long, device=DEV)
            k0[t, :c, h], v0[t, :c, h], w0[t, h, :c] = k0[s, rows, h], v0[s, rows, h], w0[s, h, rows]
    # everything else is as it was
    assert torch.equal(k.view(torch.int16), k0.view(torch.int16)) and torch.equal(v.view(torch.int16), v0.view(torch.int16))
    assert torch.equal(weights.view(torch.int32), w0.view(torch.int32)) and torch.equal(lens, l0)


def setup(n, capacity, hk, d, g):
    def one():
        return torch.randn(2 * n + 1, capacity, hk, d, generator=g, device=DEV).to(torch.bfloat16)
    order = torch.randperm(2 * n + 1, generator=g, device=DEV).to(torch.int32)
    return one(), one(), order[:n].contiguous(), order[n:2 * n].contiguous()


@pytest.mark.parametrize("hk,d", [(8, 128), (1, 64), (3, 128)])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (40, 4, 16), (64, 32, 32), (300, 0, 7), (513, 2, 300), (600, 0, 0)])
@pytest.mark.parametrize("kind", ["spread", "zero", "few"])
def test_evict(bd, hk, d, budget, sinks, recent, kind):
    g = torch.Generator(DEV).manual_seed(budget + hk)
    lengths = [0, 1, 2, 39, 40, 41, 255, 256, 257, 300, 301, 512, 514, 599, 600]
    n = len(lengths)
    k, v, src, dst = setup(n, 600, hk, d, g)
    lens = torch.full((2 * n + 1,), 77, dtype=torch.int32, device=DEV)
    lens[src.long()] = i32(lengths)
    w = torch.rand(2 * n + 1, hk, 600, generator=g, device=DEV).pow(8)
    if kind == "zero":
        w.zero_()
    elif kind == "few":
        w = (w * 3).round() * 0.25
        w[torch.rand(w.shape, generator=g, device=DEV) < 0.1] = -0.0
    check_evict(bd, k, v, w, lens, src, dst, budget, sinks, recent)


def test_special_weights_and_layout(bd):
    g = torch.Generator(DEV).manual_seed(3)
    n, hk, d, cap = 3, 2, 64, 700
    k, v, src, dst = setup(n, cap, hk, d, g)
    k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    lens = torch.full((2 * n + 1,), cap, dtype=torch.int32, device=DEV)
    w = torch.randn(2 * n + 1, hk, cap, generator=g, device=DEV)
    for value, share in ((math.inf, 0.1), (-math.inf, 0.2), (math.nan, 0.05), (1e-42, 0.2), (-0.0, 0.1), (0.0, 0.1)):
        w[torch.rand(w.shape, generator=g, device=DEV) < share] = value
    for budget in (20, 133, 350, 650):
        check_evict(bd, k, v, w.clone(), lens.clone(), src, dst, budget, 3, 5)


def test_long_slot_and_many_heads(bd):
    g = torch.Generator(DEV).manual_seed(5)
    k, v, src, dst = setup(1, 40000, 2, 64, g)
    w = torch.rand(3, 2, 40000, generator=g, device=DEV)
    check_evict(bd, k, v, w, i32([39999] * 3), src, dst, 30011, 4, 1000)


def test_bad_pairs_are_reported_and_left(bd):
    g = torch.Generator(DEV).manual_seed(7)
    k = torch.randn(9, 50, 2, 64, generator=g, device=DEV).to(torch.bfloat16)
    v = k.clone()
    w = torch.rand(9, 2, 50, generator=g, device=DEV)
    lens = i32([50, 50, 51, -1, 50, 50, 0, 0, 0])
    ws = bd.evict_workspace(7, 2, 50, device=DEV)
    k0, w0 = k.clone(), w.clone()
    # twice in dst, dst of one is src of another, a length out of range (twice), slots out of range (twice), a good one
    bd.cache_evict(k, v, w, lens, i32([0, 0, 2, 3, 9, 4, 5]), i32([8, 8, 6, 6, 7, -1, 0]), 10, ws)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    assert torch.equal(k, k0) and torch.equal(w, w0) and torch.equal(v, k0)
    assert lens.tolist() == [50, 50, 51, -1, 50, 50, 0, 0, 0]
    bd.cache_evict(k, v, w, lens, i32([0, 2]), i32([8, 7]), 10, ws)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    assert lens.tolist() == [50, 50, 51, -1, 50, 50, 0, 0, 10]
    assert torch.equal(k[:8], k0[:8])

"""GPU: the branches of the attention kernels that depend on how much there is to do:
few new tokens behind long caches (their keys are cut over the SMs and joined),
more requests than a thread block keeps on chip, and prefixes in other layouts."""
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


def make_cache(slots, capacity, heads, d, g, layout="token"):
    def one():
        if layout == "head":
            return torch.randn(slots, heads, capacity, d, generator=g, device=DEV, dtype=torch.bfloat16).transpose(1, 2)
        wide = torch.randn(slots, capacity, heads + (layout == "wide"), d + 8 * (layout == "wide"), generator=g, device=DEV, dtype=torch.bfloat16)
        return wide[:, :, :heads, :d]
    return one(), one()


def queries(rows, heads, d, g):
    return torch.randn(rows, heads, d, generator=g, device=DEV, dtype=torch.bfloat16) * 1.5


# own keys before the new ones, new tokens (a request of none, one of a single token, tiles that end inside a
# request), keys of the prefix that the requests name
NEW = [40, 1, 0, 130, 7]
BEFORE = [6000, 5001, 300, 2900, 0]
IDS, PREFIXES = [0, -1, 0, 1, 0], [3333, 129]
HEADS = [(64, 8, 128), (4, 4, 64), (32, 2, 64), (20, 4, 128), (128, 1, 128), (3, 3, 128)]
# a window that begins inside a block, first tokens that end inside one, of both sources
MASKS = [(0, 0), (2500, 0), (2500, 200), (4000, 3400), (1, 1700)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("prefix", [False, True], ids=["", "prefix"])
@pytest.mark.parametrize("layout", ["token", "wide"])
def test_split_prefill(bd, heads, mask, prefix, layout):
    (hq, hk, d), (window, sinks) = heads, mask
    g = torch.Generator(DEV).manual_seed(hq + window)
    n = len(NEW)
    how = dict(window=window, sinks=sinks)
    if prefix:
        how.update(prefix_ids=i32(IDS), prefix_slots=i32([n + 1, n]), prefix_lens=i32(PREFIXES))
    k, v = make_cache(n + 2, 6050, hk, d, g, layout)
    lens, cu = i32([a + b for a, b in zip(NEW, BEFORE)]), i32([sum(NEW[:i]) for i in range(n + 1)])
    slots = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    ref.hide_unseen(k, v, lens, math.nan, rows=NEW, slots=slots, **how)
    q = queries(sum(NEW), hq, d, g)
    ws = bd.attn_workspace(sum(NEW), n, hq, hk, d, device=DEV)
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device=DEV)
    bd.attn_prefill(q, k, v, cu, lens, ws, slots=slots, out=out, **how)
    want, bound, _ = ref.attention(q, k, v, lens, slots=slots, cu_q=cu, **how)
    ref.assert_close(out, want, bound)
    assert torch.equal(out, bd.attn_prefill(q, k, v, cu, lens, ws, slots=slots, **how))
    assert bd.device_status(ws) == 0


@pytest.mark.parametrize("layout", ["head", "wide"])
@pytest.mark.parametrize("heads", [(64, 8, 128), (12, 2, 64)], ids=str)
@pytest.mark.parametrize("window", [0, 333])
def test_prefix_layouts(bd, layout, heads, window):
    hq, hk, d = heads
    g = torch.Generator(DEV).manual_seed(hq + window)
    n = 7
    k, v = make_cache(n + 2, 1500, hk, d, g, layout)
    lens, how = i32([0, 1, 300, 20, 777, 128, 5]), dict(window=window, sinks=3, prefix_ids=i32([0, 0, 1, -1, 0, 1, 0]), prefix_slots=i32([n + 1, n]),
                                                        prefix_lens=i32([1500, 411]))
    ref.hide_unseen(k, v, lens, math.inf, **how)
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn_decode_prefix(q, k, v, lens, how["prefix_ids"], how["prefix_slots"], how["prefix_lens"], ws, window=window, sinks=3)
    want, bound, _ = ref.attention(q, k, v, lens, **how)
    ref.assert_close(out, want, bound)


@pytest.mark.parametrize("n", [1024, 1025, 1100, 3000])
@pytest.mark.parametrize("kind", ["short", "long at the end"])
def test_many_requests(bd, n, kind):
    """Requests beyond those that a block keeps on chip, and one of many blocks behind them."""
    g = torch.Generator(DEV).manual_seed(n)
    hq, hk, d, P = 4, 2, 64, 3
    longest = 40 if kind == "short" else 5000
    slots = i32([i % 100 for i in range(n)])
    k, v = make_cache(100 + P, longest, hk, d, g)
    lens = torch.randint(0, 41, (n,), generator=g, device=DEV, dtype=torch.int32)
    if kind != "short":
        lens[-1], lens[1020:1023] = 5000, i32([3000, 0, 1500])
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    want, bound, _ = ref.attention(q, k, v, lens, slots=slots, window=3500, sinks=2)
    ref.assert_close(bd.attn_decode(q, k, v, lens, ws, slots=slots, window=3500, sinks=2), want, bound)
    ids = torch.randint(-1, P, (n,), generator=g, device=DEV, dtype=torch.int32)
    how = dict(prefix_ids=ids, prefix_slots=i32([101, 102, 100]), prefix_lens=i32([40, 0, 33]))
    want, bound, _ = ref.attention(q, k, v, lens, slots=slots, **how)
    ref.assert_close(bd.attn_decode_prefix(q, k, v, lens, *how.values(), ws, slots=slots), want, bound)
    assert bd.device_status(ws) == 0


def test_many_requests_one_of_them_bad(bd):
    """What is out of range behind the requests kept on chip is reported, too."""
    g = torch.Generator(DEV).manual_seed(9)
    n, hq, hk, d = 1100, 4, 2, 64
    k, v = make_cache(10, 30, hk, d, g)
    lens, slots = i32([20] * n), i32([i % 10 for i in range(n)])
    lens[1090], slots[1050] = 31, 10
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn_decode(q, k, v, lens, ws, slots=slots)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    good = [b for b in range(n) if b not in (1050, 1090)]
    want, bound, _ = ref.attention(q[good], k, v, lens[good], slots=slots[good])
    ref.assert_close(out[good], want, bound)
    assert (out[[1050, 1090]] == 0).all()

"""GPU: an infinite value that a query sees makes its result infinite, two of
either sign or a NaN a NaN, in the columns that hold them and nowhere else."""
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


# what some keys' values hold, by column: (column, key from the front or the back, value)
PLANTED = [(0, 0, math.inf), (3, 5, -math.inf), (8, 2, math.inf), (8, 0, -math.inf), (17, 1, math.nan), (40, -1, math.inf), (63, -1, -math.inf), (63, 0, -math.inf)]
EXPECT = {0: math.inf, 3: -math.inf, 8: math.nan, 17: math.nan, 40: math.inf, 63: -math.inf}


def check(out, want, bound):
    """`want`: the result of the finite values; the planted columns instead hold EXPECT."""
    rows = out.double()
    for column, value in EXPECT.items():
        got = rows[..., column]
        assert bool((got.isnan() if math.isnan(value) else got == value).all()), column
        rows[..., column], want[..., column], bound[..., column] = 0.0, 0.0, 0.0
    ref.assert_close(rows, want, bound)


def plant(v, slot, length):
    for column, at, value in PLANTED:
        v[slot, at % length, :, column] = value


@pytest.mark.parametrize("heads", [(64, 8, 128), (5, 5, 64), (32, 2, 64), (24, 2, 128), (128, 1, 128)], ids=str)
@pytest.mark.parametrize("lengths", [[7, 16, 300], [6, 33, 9000]], ids=["short", "split"])
def test_decode(bd, heads, lengths):
    hq, hk, d = heads
    g = torch.Generator(DEV).manual_seed(hq + d)
    n = len(lengths)
    k, v = (torch.randn(n, max(lengths), hk, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    want, bound, _ = ref.attention(q, k, v, i32(lengths))
    for slot, length in enumerate(lengths):
        plant(v, slot, length)
    check(bd.attn_decode(q, k, v, i32(lengths), ws), want, bound)


@pytest.mark.parametrize("heads", [(64, 8, 128), (32, 2, 64)], ids=str)
def test_prefix(bd, heads):
    """In the prefix all see them; in one request's own keys that one only."""
    hq, hk, d = heads
    g = torch.Generator(DEV).manual_seed(hq)
    lens, ids = i32([40, 0, 700, 9]), i32([0, 0, 0, -1])
    k, v = (torch.randn(5, 3000, hk, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(4, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    ws = bd.attn_workspace(4, 4, hq, hk, d, device=DEV)
    how = dict(prefix_ids=ids, prefix_slots=i32([4]), prefix_lens=i32([2777]))
    want, bound, _ = ref.attention(q, k, v, lens, **how)
    for slot in (0, 4):
        clean = v.clone()
        plant(v, slot, 40 if slot == 0 else 2777)
        out = bd.attn_decode_prefix(q, k, v, lens, *how.values(), ws)
        hit = [0] if slot == 0 else [0, 1, 2]
        rest = [b for b in range(4) if b not in hit]
        check(out[hit], want[hit].clone(), bound[hit].clone())
        ref.assert_close(out[rest], want[rest], bound[rest])
        v.copy_(clean)

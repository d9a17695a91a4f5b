"""GPU: every reason for which a pair of slots is left as it is, each by itself and beside a good pair."""
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# lengths of the slots 0 .. 8; pairs (the first is good), which of them are left
LENS = [50, 50, 51, -1, -2 ** 31, 2 ** 31 - 1, 30, 0, 0]
CASES = {
    "length beyond the capacity": ([(0, 8), (2, 7)], [1]),
    "negative length": ([(0, 8), (3, 7)], [1]),
    "most negative length": ([(0, 8), (4, 7)], [1]),
    "largest length": ([(0, 8), (5, 7)], [1]),
    "source below the slots": ([(0, 8), (-1, 7)], [1]),
    "source behind the slots": ([(0, 8), (9, 7)], [1]),
    "target below the slots": ([(0, 8), (1, -1)], [1]),
    "target behind the slots": ([(0, 8), (1, 9)], [1]),
    "target is another pair's source": ([(0, 8), (1, 0)], [1]),
    "target is its own source": ([(0, 8), (1, 1)], [1]),
    "one target of two pairs": ([(0, 8), (1, 7), (6, 7)], [1, 2]),
    "nothing wrong": ([(0, 8), (6, 7)], []),
}


@pytest.mark.parametrize("case", CASES)
def test_bad_pairs(case):
    bd = load_bd()
    pairs, left = CASES[case]
    g = torch.Generator(DEV).manual_seed(7)
    k, v = (torch.randn(9, 50, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    w = torch.rand(9, 2, 50, generator=g, device=DEV)
    lens = i32(LENS)
    k0, v0, w0, l0 = k.clone(), v.clone(), w.clone(), lens.clone()
    src, dst = i32([a for a, _ in pairs]), i32([b for _, b in pairs])
    kept = torch.full((len(pairs), 2, 10), -7, dtype=torch.int32, device=DEV)
    ws = bd.evict_workspace(len(pairs), 2, 50, device=DEV)
    bd.cache_evict(k, v, w, lens, src, dst, 10, ws, sinks=1, recent=2, kept=kept)
    assert bd.device_status(ws) == (bd.BD_ERR_SLOT if left else 0)
    good = [i for i in range(len(pairs)) if i not in left]
    want = ref.evict(w0.cpu(), l0.cpu(), src[good].cpu(), 10, 1, 2)
    for i, rows in zip(good, want):
        s, t = pairs[i]
        l0[t] = 10
        for h in range(2):
            assert kept[i, h].tolist() == rows[h]
            k0[t, :10, h], v0[t, :10, h], w0[t, h, :10] = k0[s, rows[h], h], v0[s, rows[h], h], w0[s, h, rows[h]]
    for i in left:
        assert (kept[i] == -7).all()
    assert torch.equal(k, k0) and torch.equal(v, v0) and torch.equal(w, w0) and torch.equal(lens, l0)

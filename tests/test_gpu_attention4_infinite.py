"""GPU: scores on a 4-bit cache that leave 32 bits' range: a key whose score is -inf weighs nothing, and a row
of such keys alone gives zeros, by whichever kernels it is served and however its keys are split."""
import pytest
import torch

from tests import attention_ref
from tests import cache4_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bd():
    return load_bd()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


HEADS = pytest.mark.parametrize("heads", [(16, 2, 128), (4, 1, 64), (16, 1, 128), (12, 1, 64)], ids=str)


def make(bd, heads, lows, n):
    """A request whose keys are -1000 at `lows`, where a query of 2^118 scores below -2^128, and zeros elsewhere."""
    hq, hk, d = heads
    g = torch.Generator(DEV).manual_seed(n + hq)
    k = torch.zeros(n, hk, d, device=DEV, dtype=torch.bfloat16)
    k[lows] = -1000.0
    v = torch.randn(n, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
    cache = bd.cache4(1, -(-n // 16) * 16, hk, d, DEV)
    ws = bd.attn4_workspace(n, 1, hq, hk, d, longest=n, device=DEV)
    bd.cache4_write(k, v, cache, i32([n]), ws, cu_q=i32([0, n]))
    return cache, ws


def calls(bd, cache, ws, n, q):
    """(result, its rows' lengths) of one token, of few rows and of many."""
    yield bd.attn4_decode(q, cache, i32([n]), ws), [n]
    for rows in (min(n, 5), min(n, 70)):
        out = bd.attn4_prefill(q.expand(rows, -1, -1).contiguous(), cache, i32([0, rows]), i32([n]), ws, n)
        yield out, list(range(n - rows + 1, n + 1))


@HEADS
@pytest.mark.parametrize("n", [1, 40, 300, 9000])
def test_all_of_them(bd, heads, n):
    cache, ws = make(bd, heads, slice(None), n)
    q = torch.full((1, heads[0], heads[2]), 2.0 ** 118, dtype=torch.bfloat16, device=DEV)
    for out, _ in calls(bd, cache, ws, n, q):
        assert (out == 0).all()


@HEADS
@pytest.mark.parametrize("n,lows", [(40, slice(0, 20)), (300, slice(0, 200)), (300, slice(100, 300)), (9000, slice(0, 7000)), (9000, slice(3000, 9000)),
                                    (9000, slice(0, 9000, 2))], ids=str)
def test_some_of_them(bd, heads, n, lows):
    """The others score zero, and share the weight."""
    cache, ws = make(bd, heads, lows, n)
    hq, hk, d = heads
    huge = torch.arange(hq, device=DEV) % 3 != 0            # beside heads of ordinary scores
    q = torch.where(huge[:, None], 2.0 ** 118, 1.0).expand(1, hq, d).to(torch.bfloat16)
    low = torch.zeros(n, dtype=torch.bool, device=DEV)
    low[lows] = True
    v = ref.held(cache)[1][0, :n]
    for out, lengths in calls(bd, cache, ws, n, q):
        assert torch.isfinite(out.float()).all()
        rows = len(lengths)
        plain = torch.where(huge[:, None], 0.0, q).expand(rows, hq, d)
        want, bound = ref.attention(plain, cache, i32([n]), cu_q=[0, rows])
        assert ((out.double() - want).abs() <= bound)[:, ~huge].all()
        for row, length in zip(out, lengths):
            # the probabilities of the others are one power of two: f32 sums of exact terms, at most length / 16
            # steps and joins of 2^-23 each, and one rounding of the result
            seen = ~low[:length]
            share = [x[seen].sum(0) / max(1, int(seen.sum())) for x in (v[:length], v[:length].abs())]
            mean, size = (x.repeat_interleave(hq // hk, 0) for x in share)
            err = (row.double() - mean).abs()
            assert (err <= mean.abs() * 2.0 ** -8 + size * (length / 16 + 64) * 2.0 ** -23)[huge].all()

"""GPU: what a prompt call on a 4-bit cache reports goes by its arguments, not by the kernels that
serve it: of requests without rows too, and of offsets behind the last row."""
import pytest
import torch

import workloads as wl
from bit_delta_compressed_gb300 import layer
from tests import attention_ref
from tests import cache4_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HK, D, CAP = 8, 2, 128, 96
ROWS = pytest.mark.parametrize("rows", [2, 40], ids=["row by row", "tiles"])


@pytest.fixture(scope="module")
def bd():
    return load_bd()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def make(bd, seed, rows, longest=CAP):
    """Three slots, and a workspace and queries for two requests of `rows` rows."""
    g = torch.Generator(DEV).manual_seed(seed)
    cache = torch.randint(0, 256, (3, HK, CAP // 16, 17 * D), generator=g, device=DEV, dtype=torch.uint8)
    cache[..., 16 * D:] = torch.randint(88, 128, cache[..., 16 * D:].shape, generator=g, device=DEV, dtype=torch.uint8)
    q = torch.randn(2 * rows, HQ, D, generator=g, device=DEV, dtype=torch.bfloat16)
    return cache, q, bd.attn4_workspace(2 * rows, 3, HQ, HK, D, longest=longest, device=DEV)


def check(out, q, cache, mine, length, slot):
    want, bound = ref.attention(q[mine], cache, i32([length]), cu_q=[0, mine.stop - mine.start], slots=[slot])
    attention_ref.assert_close(out[mine], want, bound)


@ROWS
def test_a_long_request_without_rows(bd, rows):
    """`longest` bounds the keys of the requests that have rows: another may have as many as its slot holds."""
    cache, q, ws = make(bd, 60, rows, longest=48)
    out = bd.attn4_prefill(q, cache, i32([0, rows, rows, 2 * rows]), i32([48, CAP, 41]), ws, 48)
    check(out, q, cache, slice(0, rows), 48, 0)
    check(out, q, cache, slice(rows, 2 * rows), 41, 2)
    assert bd.device_status(ws) == 0


@ROWS
@pytest.mark.parametrize("length,slot", [(CAP + 1, 1), (-1, 1), (2 ** 31 - 1, 1), (9, -1), (9, 3), (0, 2 ** 31 - 1)])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_a_request_without_rows_that_is_out_of_range(bd, rows, length, slot, at):
    cache, q, ws = make(bd, 61, rows)
    cu, lens, slots = [0, rows, 2 * rows], [90, 77], [2, 0]
    cu.insert(at, cu[at])
    lens.insert(at, length)
    slots.insert(at, slot)
    out = torch.full_like(q, 7.0)
    bd.attn4_prefill(q, cache, i32(cu), i32(lens), ws, CAP, slots=i32(slots), out=out)
    check(out, q, cache, slice(0, rows), 90, 2)
    check(out, q, cache, slice(rows, 2 * rows), 77, 0)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT


@ROWS
@pytest.mark.parametrize("behind", [(-1, 0), (0, -1), (1, 0), (0, 1), (-2 ** 31, 2 ** 31 - 1)], ids=str)
def test_offsets_that_do_not_ascend_behind_the_last_row(bd, rows, behind):
    """All rows are the first request's; the offsets behind it are no offsets."""
    cache, q, ws = make(bd, 62, rows)
    T = 2 * rows
    cu = [0, T] + [T + x if abs(x) < 2 else x for x in behind]
    out = bd.attn4_prefill(q, cache, i32(cu), i32([85, 20, 30]), ws, CAP)
    check(out, q, cache, slice(0, T), 85, 0)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT


@ROWS
def test_layer(bd, rows):
    """A request that decode steps took beyond `longest`, and that a step of prompts names without new tokens."""
    g = wl.generator(63, DEV)
    cache = layer.CachedAttention(bd, 3, CAP, HQ, HK, D, tokens=2 * rows, batch=3, bits=4, longest=48)
    cache.cache.copy_(make(bd, 63, rows)[0])
    cache.lens = i32([1, 47, 0])
    for _ in range(3):
        cache.decode(*[wl.activations(1, h * D, g, DEV) for h in (HQ, HK, HK)], i32([1]))
    assert cache.lens.tolist() == [1, 50, 0]
    q, k, v = [wl.activations(2 * rows, h * D, g, DEV) for h in (HQ, HK, HK)]
    out = cache.prefill(q, k, v, i32([0, 1, 2]), i32([0, rows, rows, 2 * rows]))
    assert cache.lens.tolist() == [1 + rows, 50, rows]
    check(out.view(-1, HQ, D), q.view(-1, HQ, D), cache.cache, slice(0, rows), 1 + rows, 0)
    check(out.view(-1, HQ, D), q.view(-1, HQ, D), cache.cache, slice(rows, 2 * rows), rows, 2)
    assert bd.device_status(cache.ws) == 0

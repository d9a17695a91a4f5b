"""GPU: rows into a 4-bit key/value cache and out of it, against the format's definition, byte
by byte: every place of a block, ragged requests, magnitudes, layouts, and what may not be touched."""
import math

import pytest
import torch

from tests import cache4_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def bd():
    return load_bd()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def old_cache(slots, heads, tokens, d, g):
    """A cache that was used before: any numbers, and scales up to the largest."""
    cache = torch.randint(0, 256, (slots, heads, tokens // 16, 17 * d), generator=g, device=DEV, dtype=torch.uint8)
    cache[..., 16 * d:].clamp_(max=ref.CODES - 1)
    return cache


def rows(n, heads, d, g):
    return [torch.randn(n, heads, d, generator=g, device=DEV, dtype=torch.bfloat16) * (1 + 5 * torch.rand(heads, d, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2)]


def header(bd):
    return torch.zeros(256, dtype=torch.uint8, device=DEV)


def offsets(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


SHAPES = [(8, 128), (1, 128), (3, 64), (8, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_single_tokens(bd, shape):
    """One token a request, at every place of a block."""
    (heads, d), g = shape, gen(1)
    places = list(range(16)) + [31, 32, 47, 63]
    n = len(places)
    cache = old_cache(n + 1, heads, 64, d, g)
    slots = torch.randperm(n + 1, generator=g, device=DEV)[:n].to(torch.int32)
    k, v = rows(n, heads, d, g)
    ws = header(bd)
    lens = [p + 1 for p in places]
    want = ref.write(cache, k, v, lens, slots.tolist())
    bd.cache4_write(k, v, cache, i32(lens), ws, slots=slots)
    assert torch.equal(cache.cpu(), want)
    a, b = bd.cache4_read(torch.full_like(k, math.nan), torch.full_like(v, math.nan), cache, i32(lens), ws, slots=slots)
    assert torch.equal(a.double(), ref.as_held(k)) and torch.equal(b.double(), ref.as_held(v))
    assert bd.device_status(ws) == 0


RAGGED = [  # (tokens before, new tokens) of each request
    [(0, 1), (0, 16), (0, 17), (3, 1), (3, 2), (15, 1), (15, 2), (16, 16), (7, 90), (0, 0), (31, 33)],
    [(0, 300)], [(1, 299)], [(5, 0)], [(127, 1), (0, 1), (128, 129)],
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_several_tokens(bd, shape, case):
    (heads, d), g = shape, gen(2 + case)
    before, counts = zip(*RAGGED[case])
    n, T = len(counts), sum(counts)
    lens, cu = [a + b for a, b in zip(before, counts)], offsets(counts)
    cache = old_cache(n, heads, 320, d, g)
    slots = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    k, v = rows(T, heads, d, g)
    ws = header(bd)
    want = ref.write(cache, k, v, lens, slots.tolist(), cu)
    bd.cache4_write(k, v, cache, i32(lens), ws, slots=slots, cu_q=i32(cu))
    assert torch.equal(cache.cpu(), want)
    a, b = bd.cache4_read(torch.full_like(k, math.nan), torch.full_like(v, math.nan), cache, i32(lens), ws, slots=slots, cu_q=i32(cu))
    assert torch.equal(a.double(), ref.as_held(k)) and torch.equal(b.double(), ref.as_held(v))
    # whole requests, old bytes among them
    old_k, old_v = ref.held(cache)
    T, cu = sum(lens), offsets(lens)
    a, b = bd.cache4_read(*torch.zeros(2, T, heads, d, dtype=torch.bfloat16, device=DEV), cache, i32(lens), ws, slots=slots, cu_q=i32(cu))
    for i, (slot, length) in enumerate(zip(slots.tolist(), lens)):
        for got, old in ((a, old_k), (b, old_v)):
            assert torch.equal(got[cu[i]:cu[i + 1]].double(), old[slot, :length])
    assert bd.device_status(ws) == 0


def test_magnitudes(bd):
    """Zeros, ties, every power of two, saturation, and groups that are not finite."""
    g = gen(9)
    d, groups = 128, []
    for power in range(-40, 40):
        groups.append(torch.randn(32, generator=g, device=DEV) * 2.0 ** power)
    for power in (-20, -16, -13, -3, 0, 5):              # x / s an exact multiple of 1/2: ties
        groups.append((torch.arange(32, device=DEV) - 14).clamp(-14, 14) / 2 * 2.0 ** power)
        groups.append((torch.arange(32, device=DEV) - 14).clamp(-14, 14) / 2 * 2.0 ** power * 1.375)
    for top in (7 * 1.0625, 7 * 1.1875, 7 * 1.3125, 7 * 240.0, 1680.0, 1681.0, 1800.0, 1e6, 3e38):   # ties of the scale, the largest
        groups.append(torch.rand(32, generator=g, device=DEV) * top)
        groups[-1][5] = -top
    groups += [torch.zeros(32, device=DEV), -torch.zeros(32, device=DEV), torch.full((32,), 1e-40, device=DEV)]
    for bad in (math.inf, -math.inf, math.nan):
        groups.append(torch.randn(32, generator=g, device=DEV))
        groups[-1][31] = bad
    groups += [torch.randn(32, generator=g, device=DEV)] * (-len(groups) % 8)
    x = torch.stack(groups).to(torch.bfloat16).view(-1, 2, d)
    n = x.shape[0]
    y = x.flip(0).contiguous()
    cache, ws = bd.cache4(1, -(-n // 16) * 16, 2, d, DEV), header(bd)
    bd.cache4_write(x, y, cache, i32([n]), ws, cu_q=i32([0, n]))
    assert torch.equal(cache.cpu(), ref.write(torch.zeros_like(cache), x, y, [n], [0], [0, n]))
    a, b = bd.cache4_read(torch.empty_like(x), torch.empty_like(y), cache, i32([n]), ws, cu_q=i32([0, n]))
    for got, given in ((a, x), (b, y)):
        want = ref.as_held(given)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(want).any()
        assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(want))
        top = given.double().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True)
        off = (given.double() - want).unflatten(-1, (-1, 32)).abs()
        ordinary = (top >= 7 * 2.0 ** -14) & (top <= 1680)
        # s / 2, s at most half a step of 1/8 above max / 7
        assert (off <= top / 14 * (1 + 2.0 ** -4))[ordinary.expand_as(off)].all()


def test_layouts(bd):
    """Rows inside wider ones, and a cache that is part of a larger one."""
    g = gen(11)
    heads, d, counts = 3, 64, [9, 40, 1]
    T, cu, lens = sum(counts), offsets(counts), [20, 40, 33]
    wide = torch.randn(T, 2, heads + 1, d, generator=g, device=DEV, dtype=torch.bfloat16)
    k, v = wide[:, 0, :heads], wide[:, 1, 1:]
    larger = old_cache(5, heads + 2, 64, d, g)
    cache = larger[1:4, 1:heads + 1, :3]
    want = larger.cpu().clone()
    want[1:4, 1:heads + 1, :3] = ref.write(cache, k, v, lens, [2, 0, 1], cu)
    ws = header(bd)
    bd.cache4_write(k, v, cache, i32(lens), ws, slots=i32([2, 0, 1]), cu_q=i32(cu))
    assert torch.equal(larger.cpu(), want)
    out = torch.full_like(wide, 7.0)
    a, b = bd.cache4_read(out[:, 1, 1:], out[:, 0, :heads], cache, i32(lens), ws, slots=i32([2, 0, 1]), cu_q=i32(cu))
    assert torch.equal(a.double(), ref.as_held(k)) and torch.equal(b.double(), ref.as_held(v))
    assert (out[:, 1, 0] == 7).all() and (out[:, 0, heads] == 7).all()
    # one row, whose stride nobody uses; heads of one request in two caches
    k1, v1 = k[:1], v[:1]
    want = ref.write(cache.contiguous(), k1, v1, [48], [1])
    bd.cache4_write(k1, v1, cache, i32([48]), ws, slots=i32([1]))
    assert torch.equal(cache.cpu(), want) and bd.device_status(ws) == 0


def test_more_requests_than_threads(bd):
    g = gen(12)
    heads, d, n = 2, 64, 700
    counts = torch.randint(0, 4, (n,), generator=g, device=DEV).tolist()
    before = torch.randint(0, 13, (n,), generator=g, device=DEV).tolist()
    lens, cu, T = [a + b for a, b in zip(before, counts)], offsets(counts), sum(counts)
    cache, ws = old_cache(n, heads, 16, d, g), header(bd)
    k, v = rows(T, heads, d, g)
    want = ref.write(cache, k, v, lens, range(n), cu)
    bd.cache4_write(k, v, cache, i32(lens), ws, cu_q=i32(cu))
    assert torch.equal(cache.cpu(), want)
    a, b = bd.cache4_read(torch.empty_like(k), torch.empty_like(v), cache, i32(lens), ws, cu_q=i32(cu))
    assert torch.equal(a.double(), ref.as_held(k)) and torch.equal(b.double(), ref.as_held(v)) and bd.device_status(ws) == 0


BAD = [  # lens, slots, rows of each request, and which of them are served (3 slots of 32 tokens)
    ([20, 33, 9], [0, 1, 2], [2, 2, 2], [1, 0, 1]),                    # longer than the slot
    ([20, -1, 9], [0, 1, 2], [2, 2, 2], [1, 0, 1]),
    ([20, 5, 9], [0, -1, 2], [2, 2, 2], [1, 0, 1]),
    ([20, 5, 9], [0, 3, 2], [2, 2, 2], [1, 0, 1]),
    ([20, 5, 2 ** 31 - 1], [0, 1, 2 ** 31 - 1], [2, 2, 2], [1, 1, 0]),
    ([20, 5, 9], [0, 1, 2], [2, 6, 2], [1, 0, 1]),                     # more new tokens than tokens
    ([2, 0, 9], [0, 1, 2], [1, 1, 1], [1, 0, 1]),
]


@pytest.mark.parametrize("case", range(len(BAD)))
@pytest.mark.parametrize("offsets_given", [True, False])
def test_requests_out_of_range(bd, case, offsets_given):
    lens, slots, counts, served = BAD[case]
    if not offsets_given:
        counts = [1, 1, 1]
        if case == 5:
            pytest.skip("one row a request")
    g, heads, d = gen(13), 2, 64
    cache, ws, cu = old_cache(3, heads, 32, d, g), header(bd), offsets(counts)
    k, v = rows(sum(counts), heads, d, g)
    want, a, b = cache.cpu().clone(), torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    for i in range(3):
        if served[i]:
            want = ref.write(want, k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]], [lens[i]], [slots[i]], [0, counts[i]])
    how = dict(slots=i32(slots), cu_q=i32(cu) if offsets_given else None)
    bd.cache4_write(k, v, cache, i32(lens), ws, **how)
    assert torch.equal(cache.cpu(), want) and bd.device_status(ws) == bd.BD_ERR_SLOT
    bd.cache4_read(a, b, cache, i32(lens), ws, **how)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    for i in range(3):
        x, y = a[cu[i]:cu[i + 1]].double(), b[cu[i]:cu[i + 1]].double()
        if served[i]:
            assert torch.equal(x, ref.as_held(k[cu[i]:cu[i + 1]])) and torch.equal(y, ref.as_held(v[cu[i]:cu[i + 1]]))
        else:
            assert (x == 3).all() and (y == 3).all()


@pytest.mark.parametrize("cu,served", [([0, 4, 2, 8], [1, 0, 0]), ([0, 4, 4, 11], [1, 1, 0]), ([-1, 4, 6, 8], [0, 0, 0]), ([2, 4, 6, 7], [1, 1, 1]),
                                       ([0, 2 ** 31 - 1, 6, 8], [0, 0, 0]), ([0, 2, -2 ** 31, 8], [1, 0, 0]), ([3, 3, 3, 3], [1, 1, 1])], ids=str)
def test_offsets(bd, cu, served):
    """Offsets that do not ascend end the requests that are served; rows of no request are left alone."""
    g, heads, d, lens = gen(14), 2, 128, [10, 20, 30]
    cache, ws = old_cache(3, heads, 32, d, g), header(bd)
    k, v = rows(8, heads, d, g)
    want, a, b = cache.cpu().clone(), torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    put = []
    for i in range(3):
        if served[i]:
            put += range(cu[i], cu[i + 1])
            want = ref.write(want, k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]], [lens[i]], [i], [0, cu[i + 1] - cu[i]])
    code = 0 if all(served) else bd.BD_ERR_SLOT
    bd.cache4_write(k, v, cache, i32(lens), ws, cu_q=i32(cu))
    assert torch.equal(cache.cpu(), want) and bd.device_status(ws) == code
    bd.cache4_read(a, b, cache, i32(lens), ws, cu_q=i32(cu))
    assert bd.device_status(ws) == code
    for t in range(8):
        assert torch.equal(a[t].double(), ref.as_held(k[t]) if t in put else torch.full_like(k[t], 3.0).double())
        assert torch.equal(b[t].double(), ref.as_held(v[t]) if t in put else torch.full_like(v[t], 3.0).double())


def test_nothing_to_do(bd):
    cache, ws = bd.cache4(2, 32, 2, 64, DEV), header(bd)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    bd.cache4_write(none, none, cache, i32([]), ws)
    bd.cache4_read(none, none, cache, i32([5, 4]), ws, cu_q=i32([0, 0, 0]))
    assert (cache == 0).all() and bd.device_status(ws) == 0


def test_another_stream_and_a_graph(bd):
    """Calls on a stream of their own, and a captured step whose lengths and rows change between replays."""
    g, heads, d, n = gen(15), 4, 128, 5
    k, v = rows(n, heads, d, g)
    out = [torch.empty_like(k), torch.empty_like(v)]
    cache, ws, lens = bd.cache4(n, 48, heads, d, DEV), header(bd), i32([1, 15, 16, 30, 48])
    want = cache.cpu().clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        bd.cache4_write(k, v, cache, lens, ws)
        bd.cache4_read(*out, cache, lens, ws)
    stream.synchronize()
    want = ref.write(want, k, v, lens.tolist(), range(n))
    assert torch.equal(cache.cpu(), want) and torch.equal(out[0].double(), ref.as_held(k))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.cache4_write(k, v, cache, lens, ws)
        bd.cache4_read(*out, cache, lens, ws)
    for step in range(3):
        for t in (k, v):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        lens.copy_(i32([2 + step, 16, 17 + step, 31 + step, 47 - step]))
        want = ref.write(want, k, v, lens.tolist(), range(n))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache.cpu(), want) and torch.equal(out[1].double(), ref.as_held(v))
    assert bd.device_status(ws) == 0


def test_far_places(bd):
    """A cache of more than 2^32 bytes: its last tokens."""
    heads, d, tokens = 8, 128, 131072
    slots = 2 ** 32 // (heads * tokens // 16 * 17 * d) + 2
    cache, ws = torch.empty(slots, heads, tokens // 16, 17 * d, dtype=torch.uint8, device=DEV), header(bd)
    assert cache.numel() > 2 ** 32
    k, v = rows(37, heads, d, gen(16))
    for slot in (0, slots - 1):
        cache[slot, :, -3:] = 0
    how = dict(slots=i32([slots - 1]), cu_q=i32([0, 37]))
    bd.cache4_write(k, v, cache, i32([tokens]), ws, **how)
    a, b = bd.cache4_read(torch.empty_like(k), torch.empty_like(v), cache, i32([tokens]), ws, **how)
    assert torch.equal(a.double(), ref.as_held(k)) and torch.equal(b.double(), ref.as_held(v))
    assert torch.equal(cache[-1:, :, -3:].cpu(), ref.write(torch.zeros(1, heads, 3, 17 * d, dtype=torch.uint8), k, v, [48], [0], [0, 37]))
    assert (cache[0, :, -3:] == 0).all() and bd.device_status(ws) == 0

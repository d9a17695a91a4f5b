"""GPU: attention over a 4-bit cache against the definition in 64 bits, on the values that the
cache stands for, at the lengths, masks, layouts and contents where a kernel goes wrong."""
import math

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


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def make_cache(slots, tokens, heads, d, g):
    """Any numbers, and scales of ordinary values: 2^-4 to 2."""
    cache = torch.randint(0, 256, (slots, heads, tokens // 16, 17 * d), generator=g, device=DEV, dtype=torch.uint8)
    cache[..., 16 * d:] = torch.randint(11 * 8, 16 * 8, cache[..., 16 * d:].shape, generator=g, device=DEV, dtype=torch.uint8)
    return cache


def queries(rows, heads, d, g, padded=False):
    q = torch.randn(rows, heads * d + (256 if padded else 0), generator=g, device=DEV, dtype=torch.bfloat16) * 0.5
    return q[:, :heads * d].unflatten(1, (heads, d))


LENGTHS = [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511]
HEADS = [(64, 8, 128), (16, 16, 64), (20, 4, 128), (24, 2, 64), (128, 1, 128), (5, 5, 128), (36, 3, 128)]
MASKS = [(0, 0), (1, 0), (5, 1), (64, 4), (100, 70), (128, 0), (1000, 4), (3, 600), (33, 16), (32, 33)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_decode(bd, heads, mask):
    (hq, hk, d), (window, sinks) = heads, mask
    g = gen(hq * 1000 + window)
    n = len(LENGTHS)
    cache = make_cache(n + 2, 512, hk, d, g)
    slots = torch.randperm(n + 2, generator=g, device=DEV)[:n].to(torch.int32)
    lens = i32(LENGTHS)
    ref.hide_unseen(cache, lens, slots=slots, window=window, sinks=sinks)
    q = queries(n, hq, d, g)
    ws = bd.attn4_workspace(n, n, hq, hk, d, device=DEV)
    out = torch.full_like(q, math.nan)
    bd.attn4_decode(q, cache, lens, ws, slots=slots, window=window, sinks=sinks, out=out)
    want, bound = ref.attention(q, cache, lens, slots=slots, window=window, sinks=sinks)
    attention_ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


@pytest.mark.parametrize("scale", [0.2, -0.2, 0.0, 3.0])
def test_decode_layouts(bd, scale):
    """Rows of q inside wider ones, a cache that is part of a larger one, scales of either sign."""
    g = gen(5)
    n, hq, hk, d = 9, 32, 4, 64
    larger = make_cache(n + 2, 1040, hk + 1, d, g)
    cache = larger[1:n + 1, :hk]
    lens = i32([1040, 1, 0, 700, 1029, 90, 513, 128, 1024])
    ref.hide_unseen(cache, lens, window=333, sinks=2)
    q = queries(n, hq, d, g, padded=True)
    ws = bd.attn4_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn4_decode(q, cache, lens, ws, window=333, sinks=2, scale=scale)
    want, bound = ref.attention(q, cache, lens, window=333, sinks=2, scale=scale)
    attention_ref.assert_close(out, want, bound)


@pytest.mark.parametrize("heads", [(16, 2, 128), (32, 8, 64), (16, 1, 128), (32, 2, 64)], ids=str)
@pytest.mark.parametrize("batch,length", [(1, 20011), (3, 9000), (300, 40)])
def test_decode_split_and_crowded(bd, heads, batch, length):
    """One long request over the whole GPU, and more requests than it has SMs."""
    (hq, hk, d), g = heads, gen(length)
    cache = make_cache(batch, -(-length // 16) * 16, hk, d, g)
    lens = torch.randint(length // 2, length + 1, (batch,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = length
    q = queries(batch, hq, d, g)
    ws = bd.attn4_workspace(batch, batch, hq, hk, d, device=DEV)
    out = bd.attn4_decode(q, cache, lens, ws)
    want, bound = ref.attention(q, cache, lens)
    attention_ref.assert_close(out, want, bound)
    again = bd.attn4_decode(q, cache, lens, ws)
    assert torch.equal(out, again)


def test_decode_more_requests_than_a_block_keeps(bd):
    g = gen(6)
    n, hq, hk, d = 1500, 4, 1, 64
    cache = make_cache(n, 48, hk, d, g)
    lens = torch.randint(0, 49, (n,), generator=g, device=DEV, dtype=torch.int32)
    q = queries(n, hq, d, g)
    ws = bd.attn4_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn4_decode(q, cache, lens, ws, window=20, sinks=1)
    want, bound = ref.attention(q, cache, lens, window=20, sinks=1)
    attention_ref.assert_close(out, want, bound)


@pytest.mark.parametrize("rising", [True, False])
def test_peaked_scores(bd, rising):
    """Scores of several hundred, rising and falling along the keys: the running maximum moves late and far."""
    g = gen(17)
    hq, hk, d, n = 8, 1, 128, 2000
    q = torch.ones(1, hq, d, device=DEV, dtype=torch.bfloat16)
    ramp = torch.linspace(-40, 40, n, device=DEV)
    ramp = ramp if rising else ramp.flip(0)
    k = (ramp[:, None, None] + torch.randn(n, hk, d, generator=g, device=DEV)).to(torch.bfloat16)
    v = torch.randn(n, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
    cache = bd.cache4(1, n, hk, d, DEV)
    ws = bd.attn4_workspace(n, 1, hq, hk, d, longest=n, device=DEV)
    bd.cache4_write(k, v, cache, i32([n]), ws, cu_q=i32([0, n]))
    out = bd.attn4_decode(q, cache, i32([n]), ws)
    want, bound = ref.attention(q, cache, i32([n]))
    attention_ref.assert_close(out, want, bound)
    rows = q.expand(n, hq, d).contiguous()
    out = bd.attn4_prefill(rows, cache, i32([0, n]), i32([n]), ws, n)
    want, bound = ref.attention(rows, cache, i32([n]), cu_q=[0, n])
    attention_ref.assert_close(out, want, bound)


@pytest.mark.parametrize("power", [-120, -60, -15, 0, 15, 60, 100])
def test_magnitudes_of_queries(bd, power):
    """Queries far from 1 (the scale brings the scores back), one head of zeros, one with one large value."""
    g = gen(18)
    hq, hk, d = 16, 2, 128
    cache = make_cache(2, 320, hk, d, g)
    q = queries(2, hq, d, g)
    q[:, 1] = 0
    q[:, 2, 7] = 40.0
    q = (q.float() * 2.0 ** power).to(torch.bfloat16)
    lens = i32([320, 31])
    ws = bd.attn4_workspace(2, 2, hq, hk, d, device=DEV)
    out = bd.attn4_decode(q, cache, lens, ws, scale=0.1 * 2.0 ** -power)
    want, bound = ref.attention(q, cache, lens, scale=0.1 * 2.0 ** -power)
    attention_ref.assert_close(out, want, bound)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_queries_and_values_that_are_not_finite(bd, bad):
    """They reach the rows that have or see them, and no others."""
    g = gen(19)
    hq, hk, d, n = 16, 2, 128, 100
    k, v = torch.randn(2, 3 * n, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
    v[n + 40, 1, 3] = bad                                   # request 1, head 1, dims 0 to 31
    cache = bd.cache4(3, 112, hk, d, DEV)
    ws = bd.attn4_workspace(3, 3, hq, hk, d, device=DEV)
    lens = i32([n, n, n])
    bd.cache4_write(k, v, cache, lens, ws, cu_q=i32([0, n, 2 * n, 3 * n]))
    q = queries(3, hq, d, g)
    q[2, 5, 0] = bad
    out = bd.attn4_decode(q, cache, lens, ws)
    odd = torch.zeros_like(out, dtype=torch.bool)
    odd[1, 8:, :32] = True
    odd[2, 5] = True
    assert torch.equal(~torch.isfinite(out), odd)
    want, bound = ref.attention(torch.where(torch.isfinite(q), q, 0), cache, lens)
    assert ((out.double() - want).abs() <= bound)[~odd].all()


PROMPTS = [  # (tokens before, new tokens) of each request
    [(0, 1), (0, 66), (0, 131)], [(0, 0), (5, 1), (100, 40), (0, 257), (31, 2)], [(400, 16)], [(1, 511)], [(77, 128), (0, 3)],
]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", [(0, 0), (1, 0), (64, 4), (100, 130), (33, 16), (300, 700)], ids=str)
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prefill(bd, heads, mask, case):
    (hq, hk, d), (window, sinks) = heads, mask
    before, counts = zip(*PROMPTS[case])
    g, n, T = gen(hq + window + case), len(counts), sum(counts)
    cache = make_cache(n + 1, 512, hk, d, g)
    slots = torch.randperm(n + 1, generator=g, device=DEV)[:n].to(torch.int32)
    lens, cu = i32([a + b for a, b in zip(before, counts)]), i32([sum(counts[:i]) for i in range(n + 1)])
    ref.hide_unseen(cache, lens, rows=counts, slots=slots, window=window, sinks=sinks)
    q = queries(T, hq, d, g)
    longest = int(lens.max())
    ws = bd.attn4_workspace(T, n, hq, hk, d, longest=longest, device=DEV)
    ws[256:] = 255                                          # what the workspace holds is nobody's
    out = torch.full_like(q, math.nan)
    bd.attn4_prefill(q, cache, cu, lens, ws, longest, slots=slots, window=window, sinks=sinks, out=out)
    want, bound = ref.attention(q, cache, lens, cu_q=cu, slots=slots, window=window, sinks=sinks)
    attention_ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


def test_rows_of_no_request_and_a_larger_workspace(bd):
    g = gen(21)
    hq, hk, d = 8, 2, 64
    cache = make_cache(2, 64, hk, d, g)
    q = queries(12, hq, d, g)
    ws = bd.attn4_workspace(50, 9, hq, hk, d, longest=64, device=DEV)
    out = torch.full_like(q, 7.0)
    bd.attn4_prefill(q, cache, i32([3, 5, 11]), i32([40, 17]), ws, 45, out=out)
    want, bound = ref.attention(q, cache, i32([40, 17]), cu_q=[3, 5, 11])
    attention_ref.assert_close(out[3:11], want[3:11], bound[3:11])
    assert (out[:3] == 7).all() and (out[11:] == 7).all() and bd.device_status(ws) == 0


@pytest.mark.parametrize("lens,slots,served", [([20, 49, 9], [0, 1, 2], [1, 0, 1]), ([20, -1, 9], [0, 1, 2], [1, 0, 1]), ([20, 5, 9], [0, -1, 2], [1, 0, 1]),
                                               ([20, 5, 9], [0, 3, 2], [1, 0, 1]), ([20, 5, 2 ** 31 - 1], [0, 1, -2 ** 31], [1, 1, 0])], ids=str)
def test_requests_out_of_range(bd, lens, slots, served):
    g, hq, hk, d = gen(22), 8, 2, 128
    cache = make_cache(3, 48, hk, d, g)
    ws = bd.attn4_workspace(6, 3, hq, hk, d, longest=48, device=DEV)
    mine = i32([x if s else 0 for x, s in zip(lens, served)])
    at = [x if s else 0 for x, s in zip(slots, served)]
    q = queries(3, hq, d, g)
    out = bd.attn4_decode(q, cache, i32(lens), ws, slots=i32(slots))
    want, bound = ref.attention(q, cache, mine, slots=at)
    attention_ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    q = queries(6, hq, d, g)
    out = torch.full_like(q, 7.0)
    bd.attn4_prefill(q, cache, i32([0, 2, 4, 6]), i32(lens), ws, 48, slots=i32(slots), out=out)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    for b in range(3):
        rows = slice(2 * b, 2 * b + 2)
        if served[b]:
            want, bound = ref.attention(q[rows], cache, i32([lens[b]]), cu_q=[0, 2], slots=[slots[b]])
            attention_ref.assert_close(out[rows], want, bound)
        else:
            assert (out[rows] == 0).all()


def test_longer_than_the_call_allows(bd):
    g, hq, hk, d = gen(23), 8, 2, 128
    cache = make_cache(2, 64, hk, d, g)
    ws = bd.attn4_workspace(4, 2, hq, hk, d, longest=32, device=DEV)
    q = queries(4, hq, d, g)
    out = bd.attn4_prefill(q, cache, i32([0, 2, 4]), i32([33, 30]), ws, 32)
    want, bound = ref.attention(q[2:], cache, i32([30]), cu_q=[0, 2], slots=[1])
    attention_ref.assert_close(out[2:], want, bound)
    assert (out[:2] == 0).all() and bd.device_status(ws) == bd.BD_ERR_SLOT


@pytest.mark.parametrize("cu,served", [([0, 4, 2, 6], [1, 0, 0]), ([0, 2, 4, 9], [1, 1, 0]), ([-1, 2, 4, 6], [0, 0, 0])], ids=str)
def test_offsets_that_do_not_ascend(bd, cu, served):
    g, hq, hk, d = gen(24), 8, 2, 64
    cache = make_cache(3, 32, hk, d, g)
    ws = bd.attn4_workspace(6, 3, hq, hk, d, longest=32, device=DEV)
    q, lens = queries(6, hq, d, g), [20, 30, 25]
    out = torch.full_like(q, 7.0)
    bd.attn4_prefill(q, cache, i32(cu), i32(lens), ws, 32, out=out)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    for b in range(3):
        if served[b]:
            rows = slice(cu[b], cu[b + 1])
            want, bound = ref.attention(q[rows], cache, i32([lens[b]]), cu_q=[0, cu[b + 1] - cu[b]], slots=[b])
            attention_ref.assert_close(out[rows], want, bound)


def test_step_of_all_of_them_in_a_graph(bd):
    """Write, read back, decode and a prompt in one captured step, in one workspace."""
    g, hq, hk, d, n = gen(25), 16, 2, 128, 3
    cache = make_cache(n, 96, hk, d, g)
    lens, more = i32([1, 40, 90]), i32([4, 44, 94])
    cu = i32([0, 3, 6, 9])
    k, v = torch.randn(2, n, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
    k2, v2 = torch.randn(2, 3 * n, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
    q, q2 = queries(n, hq, d, g), queries(3 * n, hq, d, g)
    ws = bd.attn4_workspace(3 * n, n, hq, hk, d, longest=96, device=DEV)
    out, out2, a, b = torch.empty_like(q), torch.empty_like(q2), torch.empty_like(k), torch.empty_like(v)

    def step():
        bd.cache4_write(k, v, cache, lens, ws)
        bd.cache4_read(a, b, cache, lens, ws)
        bd.attn4_decode(q, cache, lens, ws, window=33, sinks=3, out=out)
        bd.cache4_write(k2, v2, cache, more, ws, cu_q=cu)
        bd.attn4_prefill(q2, cache, cu, more, ws, 96, window=33, sinks=3, out=out2)

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (k, v, k2, v2):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        before = cache.clone()
        lens.copy_(i32([2, 41, 70]))
        more.copy_(lens + 3)
        graph.replay()
        first = ref.write(before, k, v, lens.tolist(), range(n)).to(DEV)
        assert torch.equal(a.double(), ref.as_held(k)) and torch.equal(b.double(), ref.as_held(v))
        want, bound = ref.attention(q, first, lens, window=33, sinks=3)
        attention_ref.assert_close(out, want, bound)
        second = ref.write(first, k2, v2, more.tolist(), range(n), cu.tolist()).to(DEV)
        assert torch.equal(cache, second)
        want, bound = ref.attention(q2, second, more, cu_q=cu, window=33, sinks=3)
        attention_ref.assert_close(out2, want, bound)
    assert bd.device_status(ws) == 0


def test_far_places(bd):
    """A cache of more than 2^32 bytes: the last slot's requests."""
    hq, hk, d, tokens = 64, 8, 128, 131072
    slots = 2 ** 32 // (hk * tokens // 16 * 17 * d) + 2
    cache = torch.empty(slots, hk, tokens // 16, 17 * d, dtype=torch.uint8, device=DEV)
    g = gen(26)
    cache[-1] = make_cache(1, tokens, hk, d, g)[0]
    q, lens = queries(1, hq, d, g), i32([tokens - 3])
    ws = bd.attn4_workspace(1, 1, hq, hk, d, device=DEV)
    out = bd.attn4_decode(q, cache, lens, ws, slots=i32([slots - 1]))
    want, bound = ref.attention(q, cache[-1:], lens)
    attention_ref.assert_close(out, want, bound)


def test_requests_that_share_a_slot(bd):
    """Several requests may read one slot (at lengths of their own), in each kind of call."""
    g, hq, hk, d = gen(27), 16, 2, 128
    cache = make_cache(2, 208, hk, d, g)
    lens, slots = i32([200, 77, 200, 3, 131]), i32([1, 1, 1, 0, 1])
    ws = bd.attn4_workspace(10, 5, hq, hk, d, longest=208, device=DEV)
    q = queries(5, hq, d, g)
    want, bound = ref.attention(q, cache, lens, slots=slots)
    attention_ref.assert_close(bd.attn4_decode(q, cache, lens, ws, slots=slots), want, bound)
    q, cu = queries(10, hq, d, g), i32([0, 2, 4, 7, 8, 10])
    want, bound = ref.attention(q, cache, lens, slots=slots, cu_q=cu)
    attention_ref.assert_close(bd.attn4_prefill(q, cache, cu, lens, ws, 208, slots=slots), want, bound)
    k, v = ref.held(cache)
    a, b = bd.cache4_read(*torch.zeros(2, 10, hk, d, dtype=torch.bfloat16, device=DEV), cache, lens, ws, slots=slots, cu_q=cu)
    for i in range(5):
        r, n, s = slice(int(cu[i]), int(cu[i + 1])), int(lens[i]), int(slots[i])
        assert torch.equal(a[r].double(), k[s, n - (r.stop - r.start):n]) and torch.equal(b[r].double(), v[s, n - (r.stop - r.start):n])
    assert bd.device_status(ws) == 0


def test_two_streams_at_once(bd):
    """Calls on two streams with a workspace and a cache each, many of them under way together."""
    g, hq, hk, d, sides = gen(28), 32, 4, 128, []
    for n in (3, 5):
        cache, lens = make_cache(n, 2048, hk, d, g), torch.randint(1, 2049, (n,), generator=g, device=DEV, dtype=torch.int32)
        lens[0] = 2048
        news = [30 + 7 * i for i in range(n)]
        lens = torch.maximum(lens, i32(news))
        cu = i32([sum(news[:i]) for i in range(n + 1)])
        q, q2 = queries(n, hq, d, g), queries(sum(news), hq, d, g)
        ws = bd.attn4_workspace(sum(news), n, hq, hk, d, longest=2048, device=DEV)
        want = ref.attention(q, cache, lens), ref.attention(q2, cache, lens, cu_q=cu)
        sides.append((torch.cuda.Stream(), cache, lens, cu, q, q2, ws, want, torch.empty_like(q), torch.empty_like(q2)))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, cache, lens, cu, q, q2, ws, _, out, out2 in sides:
            with torch.cuda.stream(stream):
                bd.attn4_decode(q, cache, lens, ws, out=out)
                bd.attn4_prefill(q2, cache, cu, lens, ws, 2048, out=out2)
    torch.cuda.synchronize()
    for _, _, _, _, _, _, ws, want, out, out2 in sides:
        for got, (x, bound) in zip((out, out2), want):
            attention_ref.assert_close(got, x, bound)
        assert bd.device_status(ws) == 0


def test_prompts_longer_than_the_plan_keeps(bd):
    """More requests than the reading back and the plan keep on chip, most of one token."""
    g, hq, hk, d, n = gen(29), 8, 2, 64, 600
    cache = make_cache(n, 64, hk, d, g)
    news = [1 + (i % 37 == 5) * 9 for i in range(n)]
    lens = torch.randint(10, 65, (n,), generator=g, device=DEV, dtype=torch.int32)
    cu = torch.tensor([0] + news, device=DEV).cumsum(0).to(torch.int32)
    slots = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    q = queries(sum(news), hq, d, g)
    ref.hide_unseen(cache, lens, rows=news, slots=slots, window=17, sinks=2)
    ws = bd.attn4_workspace(sum(news), n, hq, hk, d, longest=64, device=DEV)
    out = bd.attn4_prefill(q, cache, cu, lens, ws, 64, slots=slots, window=17, sinks=2)
    want, bound = ref.attention(q, cache, lens, cu_q=cu, slots=slots, window=17, sinks=2)
    attention_ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


def test_flat_scores_over_long_requests(bd):
    """Every key weighs the same, and the result is a small mean of many values."""
    g, hq, hk, d, n = gen(30), 8, 1, 128, 40000
    cache = make_cache(2, n, hk, d, g)
    q = torch.zeros(2, hq, d, dtype=torch.bfloat16, device=DEV)
    lens = i32([n, n - 7])
    ws = bd.attn4_workspace(2, 2, hq, hk, d, device=DEV)
    out = bd.attn4_decode(q, cache, lens, ws).double()
    v = ref.held(cache)[1]
    want = torch.stack([v[i, :m].mean(0) for i, m in enumerate(lens.tolist())]).expand(2, hq, d)
    # all probabilities are the same power of two: f32 sums of them times exact values, the terms' sizes
    # added up times 2^-23 for each of at most n / 16 steps and joins, and one rounding of the result
    size = torch.stack([v[i, :m].abs().mean(0) for i, m in enumerate(lens.tolist())]).expand(2, hq, d)
    assert ((out - want).abs() <= want.abs() * 2.0 ** -8 + size * (n / 16 + 64) * 2.0 ** -23).all()


FEW = [  # (tokens before, new tokens) of each request: few enough to be served row by row
    [(0, 1)], [(300, 8)], [(0, 0), (5, 1), (100, 3), (0, 4), (300, 2)], [(47, 2), (15, 1), (500, 7), (0, 2)], [(31, 1)] * 64, [(95, 4)] * 20,
]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_few_rows(bd, heads, mask):
    (hq, hk, d), (window, sinks) = heads, mask
    for case, requests in enumerate(FEW):
        before, counts = zip(*requests)
        g, n, T = gen(hq + window + case), len(counts), sum(counts)
        cache = make_cache(n + 1, 512, hk, d, g)
        slots = torch.randperm(n + 1, generator=g, device=DEV)[:n].to(torch.int32)
        lens, cu = i32([a + b for a, b in zip(before, counts)]), i32([sum(counts[:i]) for i in range(n + 1)])
        ref.hide_unseen(cache, lens, rows=counts, slots=slots, window=window, sinks=sinks)
        q, longest = queries(T, hq, d, g), int(lens.max())
        ws = bd.attn4_workspace(T, n, hq, hk, d, longest=longest, device=DEV)
        out = torch.full_like(q, math.nan)
        bd.attn4_prefill(q, cache, cu, lens, ws, longest, slots=slots, window=window, sinks=sinks, out=out)
        assert bd.device_status(ws) == 0
        # row by row it is decode: its bound, on the keys up to the row
        rows = [(b, i) for b, c in enumerate(counts) for i in range(c)]
        at = i32([before[b] + i + 1 for b, i in rows])
        want, bound = ref.attention(q, cache, at, slots=slots[[b for b, _ in rows]], window=window, sinks=sinks)
        attention_ref.assert_close(out, want, bound, str(case))
        again = bd.attn4_prefill(q, cache, cu, lens, ws, longest, slots=slots, window=window, sinks=sinks)
        assert torch.equal(out, again)


@pytest.mark.parametrize("rows", [2, 40], ids=["row by row", "tiles"])
@pytest.mark.parametrize("lens,slots,served", [([50, 97, 49], [0, 1, 2], [1, 0, 1]), ([60, -1, 49], [0, 1, 2], [1, 0, 1]), ([60, 1, 49], [0, 1, 2], [1, 0, 1]),
                                               ([60, 45, 49], [0, -1, 2], [1, 0, 1]), ([60, 45, 49], [0, 3, 2], [1, 0, 1]),
                                               ([60, 45, 2 ** 31 - 1], [0, 1, -2 ** 31], [1, 1, 0])], ids=str)
def test_prompts_out_of_range(bd, rows, lens, slots, served):
    g, hq, hk, d = gen(31), 8, 2, 128
    cache = make_cache(3, 96, hk, d, g)
    ws = bd.attn4_workspace(3 * rows, 3, hq, hk, d, longest=96, device=DEV)
    q = queries(3 * rows + 2, hq, d, g)[1:-1]
    whole = torch.full((3 * rows + 2, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    out = bd.attn4_prefill(q, cache, i32([0, rows, 2 * rows, 3 * rows]), i32(lens), ws, 96, slots=i32(slots), out=whole[1:-1])
    assert bd.device_status(ws) == bd.BD_ERR_SLOT and (whole[0] == 7).all() and (whole[-1] == 7).all()
    for b in range(3):
        mine = slice(rows * b, rows * b + rows)
        if served[b]:
            how = dict(slots=[slots[b]] * rows) if rows == 2 else dict(slots=[slots[b]], cu_q=[0, rows])
            at = i32([lens[b] - rows + 1 + i for i in range(rows)] if rows == 2 else [lens[b]])
            want, bound = ref.attention(q[mine], cache, at, **how)
            attention_ref.assert_close(out[mine], want, bound)
        else:
            assert (out[mine] == 0).all()


@pytest.mark.parametrize("rows", [2, 40], ids=["row by row", "tiles"])
@pytest.mark.parametrize("cu,served,zeros", [([0, 2, 1, 3], [1, 0, 0], 2), ([0, 1, 2, 4], [1, 1, 0], 2), ([-1, 1, 2, 3], [0, 0, 0], 0), ([0, 0, -1, 3], [1, 0, 0], 0),
                                             ([1, 1, 2, 3], [1, 1, 1], 3), ([0, 1, 1, 2], [1, 1, 1], 3), ([0, 2 ** 30, 2, 3], [0, 0, 0], 0)], ids=str)
def test_offsets_of_prompts(bd, rows, cu, served, zeros):
    """Offsets (in `rows`): rows behind ones that do not ascend become zeros, rows of no request stay."""
    g, hq, hk, d = gen(32), 8, 2, 64
    cache, lens = make_cache(3, 128, hk, d, g), [100, 120, 90]
    cu = [x * rows if x != 2 ** 30 else x for x in cu]
    T = 3 * rows
    ws = bd.attn4_workspace(T, 3, hq, hk, d, longest=128, device=DEV)
    q = queries(T, hq, d, g)
    out = torch.full_like(q, 7.0)
    bd.attn4_prefill(q, cache, i32(cu), i32(lens), ws, 128, out=out)
    assert bd.device_status(ws) == (0 if all(served) else bd.BD_ERR_SLOT)
    put = torch.zeros(T, dtype=torch.bool, device=DEV)
    for b in range(3):
        n = cu[b + 1] - cu[b]
        if not served[b] or n == 0:
            continue
        mine = slice(cu[b], cu[b + 1])
        put[mine] = True
        want, bound = ref.attention(q[mine], cache, i32([lens[b]]), slots=[b], cu_q=[0, n])
        if rows == 2:
            want, bound = ref.attention(q[mine], cache, i32([lens[b] - n + 1 + i for i in range(n)]), slots=[b] * n)
        attention_ref.assert_close(out[mine], want, bound)
    behind = torch.arange(T, device=DEV) >= zeros * rows
    if not all(served):
        assert (out[behind] == 0).all()
        put |= behind
    assert (out[~put] == 7).all()


def test_few_rows_in_a_graph(bd):
    """A captured call of few rows whose offsets, lengths and slots change between replays."""
    g, hq, hk, d, n = gen(33), 16, 2, 128, 4
    cache = make_cache(6, 208, hk, d, g)
    q = queries(12, hq, d, g)
    cu, lens, slots = i32([0, 3, 6, 9, 12]), i32([50, 60, 70, 80]), i32([0, 1, 2, 3])
    ws = bd.attn4_workspace(12, n, hq, hk, d, longest=208, device=DEV)
    out = torch.empty_like(q)
    bd.attn4_prefill(q, cache, cu, lens, ws, 208, slots=slots, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.attn4_prefill(q, cache, cu, lens, ws, 208, slots=slots, out=out)
    for ends, sizes, places in (([0, 1, 1, 8, 12], [208, 3, 7, 130], [5, 4, 3, 2]), ([0, 12, 12, 12, 12], [100, 1, 1, 1], [1, 0, 0, 0]), ([1, 2, 3, 4, 5], [1, 1, 16, 17], [2, 2, 2, 2])):
        for t, x in ((cu, ends), (lens, sizes), (slots, places)):
            t.copy_(i32(x))
        out.fill_(7)
        graph.replay()
        rows = [(b, t) for b in range(n) for t in range(ends[b], ends[b + 1])]
        which = [t for _, t in rows]
        want, bound = ref.attention(q[which], cache, i32([sizes[b] - (ends[b + 1] - 1 - t) for b, t in rows]), slots=[places[b] for b, _ in rows])
        attention_ref.assert_close(out[which], want, bound)
        assert (out[[t for t in range(12) if t not in which]] == 7).all()
    assert bd.device_status(ws) == 0

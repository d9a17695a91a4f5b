"""GPU: attention over a key/value cache against the definition in 64 bits, at
the lengths, masks, layouts and contents where a kernel goes wrong."""
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


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def make_cache(slots, capacity, heads, d, g, layout="token"):
    """K and V as [slots, capacity, heads, d] views of several layouts."""
    def one():
        if layout == "token":
            return torch.randn(slots, capacity, heads, d, generator=g, device=DEV, dtype=torch.bfloat16)
        if layout == "head":
            return torch.randn(slots, heads, capacity, d, generator=g, device=DEV, dtype=torch.bfloat16).transpose(1, 2)
        wide = torch.randn(slots, capacity, heads + 1, d + 8, generator=g, device=DEV, dtype=torch.bfloat16)
        return wide[:, :, :heads, :d]
    return one(), one()


def queries(rows, heads, d, g, padded=False):
    q = torch.randn(rows, heads * d + (256 if padded else 0), generator=g, device=DEV, dtype=torch.bfloat16) * 1.5
    return q[:, :heads * d].unflatten(1, (heads, d))


LENGTHS = [0, 1, 2, 7, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511]
HEADS = [(64, 8, 128), (16, 16, 64), (20, 4, 128), (24, 2, 64), (128, 1, 128), (5, 5, 128)]
MASKS = [(0, 0), (1, 0), (5, 1), (64, 4), (100, 70), (128, 0), (1000, 4), (3, 600)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_decode(bd, heads, mask):
    (hq, hk, d), (window, sinks) = heads, mask
    g = gen(hq * 1000 + window)
    n = len(LENGTHS)
    k, v = make_cache(n + 2, 520, hk, d, g)
    slots = torch.randperm(n + 2, generator=g, device=DEV)[:n].to(torch.int32)
    lens = i32(LENGTHS)
    ref.hide_unseen(k, v, lens, math.nan, slots=slots, window=window, sinks=sinks)
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    out = torch.full_like(q, math.nan)
    bd.attn_decode(q, k, v, lens, ws, slots=slots, window=window, sinks=sinks, out=out)
    want, bound, _ = ref.attention(q, k, v, lens, slots=slots, window=window, sinks=sinks)
    ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


@pytest.mark.parametrize("layout", ["head", "wide"])
@pytest.mark.parametrize("fill", [math.inf, -math.inf, 3e38])
def test_decode_layouts_and_hidden_values(bd, layout, fill):
    g = gen(5)
    n, hq, hk, d = 9, 32, 4, 64
    k, v = make_cache(n, 1030, hk, d, g, layout)
    lens = i32([1030, 1, 0, 700, 1029, 90, 513, 128, 1024])
    ref.hide_unseen(k, v, lens, fill, window=333, sinks=2)
    q = queries(n, hq, d, g, padded=True)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn_decode(q, k, v, lens, ws, window=333, sinks=2, scale=0.2)
    want, bound, _ = ref.attention(q, k, v, lens, window=333, sinks=2, scale=0.2)
    ref.assert_close(out, want, bound)


@pytest.mark.parametrize("batch,length", [(1, 20011), (3, 9000), (300, 40)])
def test_decode_split_and_crowded(bd, batch, length):
    """One long request over the whole GPU, and more requests than it has SMs."""
    g = gen(length)
    hq, hk, d = 16, 2, 128
    k, v = make_cache(batch, length, hk, d, g)
    lens = torch.randint(length // 2, length + 1, (batch,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = length
    q = queries(batch, hq, d, g)
    ws = bd.attn_workspace(batch, batch, hq, hk, d, device=DEV)
    out = bd.attn_decode(q, k, v, lens, ws)
    want, bound, _ = ref.attention(q, k, v, lens)
    ref.assert_close(out, want, bound)
    again = bd.attn_decode(q, k, v, lens, ws)
    assert torch.equal(out, again)


def test_decode_peaked_scores(bd):
    """Scores of several hundred, rising and falling along the keys: the running maximum moves late and far."""
    g = gen(17)
    hq, hk, d, n = 8, 1, 128, 2000
    for rising in (True, False):
        q = torch.ones(1, hq, d, device=DEV, dtype=torch.bfloat16)
        ramp = torch.linspace(-40, 40, n, device=DEV)
        ramp = ramp if rising else ramp.flip(0)
        k = (ramp[None, :, None, None] + torch.randn(1, n, hk, d, generator=g, device=DEV)).to(torch.bfloat16)
        v = torch.randn(1, n, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
        ws = bd.attn_workspace(n, 1, hq, hk, d, device=DEV)
        out = bd.attn_decode(q, k, v, i32([n]), ws)
        want, bound, _ = ref.attention(q, k, v, i32([n]))
        ref.assert_close(out, want, bound)
        rows = q.expand(n, hq, d).contiguous()
        out = bd.attn_prefill(rows, k, v, i32([0, n]), i32([n]), ws)
        want, bound, _ = ref.attention(rows, k, v, i32([n]), cu_q=[0, n])
        ref.assert_close(out, want, bound)


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", [(0, 0), (1, 0), (64, 4), (100, 130), (300, 700)], ids=str)
def test_decode_prefix(bd, heads, mask):
    (hq, hk, d), (window, sinks) = heads, mask
    g = gen(hq + 7 * window)
    own = [0, 1, 5, 64, 128, 200, 33, 0, 17, 255, 90, 1]
    ids = [0, 0, 1, 2, -1, 0, 3, -1, 0, 1, 4, 3]
    plens = [400, 129, 0, 1, 128, 77]                          # the last one is named by nobody
    n, P = len(own), len(plens)
    k, v = make_cache(n + P, 400, hk, d, g)
    places = torch.randperm(n + P, generator=g, device=DEV).to(torch.int32)
    slots, pslots = places[:n].contiguous(), places[n:].contiguous()
    lens, ids, plens = i32(own), i32(ids), i32(plens)
    how = dict(slots=slots, window=window, sinks=sinks, prefix_ids=ids, prefix_slots=pslots, prefix_lens=plens)
    ref.hide_unseen(k, v, lens, math.nan, **how)
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws, slots=slots, window=window, sinks=sinks)
    want, bound, _ = ref.attention(q, k, v, lens, **how)
    ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


def test_decode_prefix_long(bd):
    """Prefixes long enough to be split, groups of one request and of many."""
    g = gen(23)
    hq, hk, d, n = 64, 8, 128, 60
    k, v = make_cache(n + 3, 5000, hk, d, g)
    lens = torch.randint(0, 300, (n,), generator=g, device=DEV, dtype=torch.int32)
    ids = i32([0] * 41 + [1] * 1 + [2] * 17 + [-1])[torch.randperm(n, generator=g, device=DEV)]
    pslots, plens = i32([n, n + 1, n + 2]), i32([5000, 3333, 1001])
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    out = bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws)
    want, bound, _ = ref.attention(q, k, v, lens, prefix_ids=ids, prefix_slots=pslots, prefix_lens=plens)
    ref.assert_close(out, want, bound)
    assert torch.equal(out, bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws))


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", [(0, 0), (1, 0), (40, 3), (128, 0), (200, 150)], ids=str)
@pytest.mark.parametrize("prefix", [False, True], ids=["", "prefix"])
def test_prefill(bd, heads, mask, prefix):
    (hq, hk, d), (window, sinks) = heads, mask
    g = gen(hq + 11 * window)
    new = [1, 0, 16, 33, 129, 257, 64, 5]
    before = [0, 9, 0, 300, 1, 127, 128, 700]
    n = len(new)
    how = {}
    extra = 0
    if prefix:
        extra = 3
        how = dict(prefix_ids=i32([0, 1, -1, 2, 1, 0, 2, 0]), prefix_slots=i32([n, n + 2, n + 1]), prefix_lens=i32([300, 129, 1]))
    k, v = make_cache(n + extra, 720, hk, d, g)
    lens = i32([a + b for a, b in zip(new, before)])
    cu = i32([sum(new[:i]) for i in range(n + 1)])
    slots = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    ref.hide_unseen(k, v, lens, math.nan, rows=new, slots=slots, window=window, sinks=sinks, **how)
    q = queries(sum(new), hq, d, g, padded=True)
    ws = bd.attn_workspace(sum(new), n, hq, hk, d, device=DEV)
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device=DEV)
    bd.attn_prefill(q, k, v, cu, lens, ws, slots=slots, window=window, sinks=sinks, out=out, **how)
    want, bound, _ = ref.attention(q, k, v, lens, slots=slots, cu_q=cu, window=window, sinks=sinks, **how)
    ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


@pytest.mark.parametrize("layout", ["head", "wide"])
@pytest.mark.parametrize("new,before", [(1500, 0), (40, 6000), (1, 2500), (700, 1300)])
def test_prefill_long(bd, layout, new, before):
    g = gen(new + before)
    hq, hk, d = 16, 2, 128
    n = new + before
    k, v = make_cache(2, n + 3, hk, d, g, layout)
    lens, cu, slots = i32([n]), i32([0, new]), i32([1])
    ref.hide_unseen(k, v, lens, math.nan, rows=[new], slots=slots)
    q = queries(new, hq, d, g)
    ws = bd.attn_workspace(new, 1, hq, hk, d, device=DEV)
    out = bd.attn_prefill(q, k, v, cu, lens, ws, slots=slots)
    want, bound, _ = ref.attention(q, k, v, lens, slots=slots, cu_q=cu)
    ref.assert_close(out, want, bound)
    assert torch.equal(out, bd.attn_prefill(q, k, v, cu, lens, ws, slots=slots))


def test_prefill_many_requests(bd):
    g = gen(31)
    hq, hk, d, n = 16, 4, 64, 200
    new = torch.randint(0, 60, (n,), generator=g, device=DEV, dtype=torch.int32)
    lens = new + torch.randint(0, 100, (n,), generator=g, device=DEV, dtype=torch.int32)
    cu = torch.cat([i32([0]), new.cumsum(0, dtype=torch.int32)])
    k, v = make_cache(n, 160, hk, d, g)
    q = queries(int(cu[-1]), hq, d, g)
    ws = bd.attn_workspace(q.shape[0], n, hq, hk, d, device=DEV)
    out = bd.attn_prefill(q, k, v, cu, lens, ws)
    want, bound, _ = ref.attention(q, k, v, lens, cu_q=cu)
    ref.assert_close(out, want, bound)


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", [(0, 0), (50, 3)], ids=str)
@pytest.mark.parametrize("prefix", [False, True], ids=["", "prefix"])
def test_weights(bd, heads, mask, prefix):
    (hq, hk, d), (window, sinks) = heads, mask
    g = gen(hq + 3)
    own = [0, 1, 16, 17, 300, 511, 129, 64]
    n = len(own)
    k, v = make_cache(n + 2, 512, hk, d, g)
    lens = i32(own)
    slots = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    how = {}
    if prefix:
        how = dict(prefix_ids=i32([0, 1, -1, 0, 0, 1, -1, 0]), prefix_slots=i32([n, n + 1]), prefix_lens=i32([400, 31]))
    ref.hide_unseen(k, v, lens, math.nan, slots=slots, window=window, sinks=sinks, **how)
    q = queries(n, hq, d, g)
    weights = torch.rand(n + 2, hk, 512, generator=g, device=DEV)
    start = weights.clone()
    ws = bd.attn_workspace(n, n, hq, hk, d, weigh_len=512, device=DEV)
    out = bd.attn_decode_prefix(q, k, v, lens, how.get("prefix_ids"), how.get("prefix_slots"), how.get("prefix_lens"), ws,
                                slots=slots, window=window, sinks=sinks, weights=weights)
    want, bound, (added, rel) = ref.attention(q, k, v, lens, slots=slots, window=window, sinks=sinks, **how)
    ref.assert_close(out, want, bound)
    expect = start.double()
    allow = torch.zeros_like(expect)
    for b, L in enumerate(own):
        s = int(slots[b])
        expect[s, :, :L] += added[b]
        # the sum over the group and the addition: a rounding of each partial sum
        allow[s, :, :L] = rel.get(b, 0.0) * added[b] + (hq // hk + 2) * ref.F32 * expect[s, :, :L]
    assert ((weights.double() - expect).abs() <= allow).all()


def test_out_of_range_is_reported_and_harmless(bd):
    g = gen(41)
    n, hq, hk, d = 8, 16, 2, 128
    k, v = make_cache(n, 100, hk, d, g)
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, weigh_len=100, device=DEV)
    slots = i32([0, -1, n, 3, 4, 5, 6, 2 ** 31 - 1])
    lens = i32([50, 50, 50, 101, -1, 100, -2 ** 31, 7])
    weights = torch.zeros(n, hk, 100, device=DEV)
    out = bd.attn_decode(q, k, v, lens, ws, slots=slots, weights=weights)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    ok = [0, 5]
    want, bound, _ = ref.attention(q[ok], k, v, lens[ok], slots=slots[ok])
    ref.assert_close(out[ok], want, bound)
    bad = [b for b in range(n) if b not in ok]
    assert (out[bad] == 0).all()
    assert (weights[[1, 2, 3, 4, 6, 7]] == 0).all()
    # prefix ids and the prefixes' own slots and lengths
    lens = i32([50] * n)
    ids = i32([0, 1, 2, 3, -1, -2, 4, 2 ** 31 - 1])
    out = bd.attn_decode_prefix(q, k, v, lens, ids, i32([7, n, 6, -5]), i32([60, 60, 101, 9]), ws)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    want, bound, _ = ref.attention(q[[0, 4]], k, v, lens[:2], slots=i32([0, 4]), prefix_ids=i32([0, -1]), prefix_slots=i32([7]), prefix_lens=i32([60]))
    ref.assert_close(out[[0, 4]], want, bound)
    assert (out[[1, 2, 3, 5, 6, 7]] == 0).all()
    # offsets of the query rows: beyond the rows, descending, then more new tokens than keys
    out = torch.full_like(q, 7.0)
    bd.attn_prefill(q, k, v, i32([0, 3, 9, 5, 2 ** 31 - 1]), i32([50, 50, 50, 50]), ws, out=out)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    want, bound, _ = ref.attention(q[:3], k, v, lens[:1], cu_q=[0, 3])
    ref.assert_close(out[:3], want, bound)
    assert (out[3:] == 0).all()
    out = bd.attn_prefill(q, k, v, i32([0, 8]), i32([5]), ws)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    assert (out == 0).all()


@pytest.mark.parametrize("T", [8, 700])
def test_broken_row_offsets(bd, T):
    """Offsets that come back again and again name more rows than there are: the requests
    before the first break are served, the rows from there on are zeros."""
    g = gen(59)
    B, hq, hk, d = 33, 64, 8, 128
    k, v = make_cache(B, T, hk, d, g)
    q = queries(T, hq, d, g)
    ws = bd.attn_workspace(T, B, hq, hk, d, device=DEV)
    for cu in ([0, 5] + [T, 0] * 16, [0, 5] + [T, 0, 1] * 11, [0, 5, T + 1] + [T] * 31, [0, 5, 4, -1] + [T] * 30):
        cu = i32(cu[:B + 1])
        out = torch.full_like(q, 3.0)
        bd.attn_prefill(q, k, v, cu, i32([T] * B), ws, out=out)
        assert bd.device_status(ws) == bd.BD_ERR_SLOT
        served = T if int(cu[2]) == T else 5
        ends = [0, 5, T] if served == T else [0, 5]
        want, bound, _ = ref.attention(q[:served], k, v, i32([T] * (len(ends) - 1)), cu_q=ends)
        ref.assert_close(out[:served], want, bound)
        assert (out[served:] == 0).all()


def test_offsets_past_32_bits(bd):
    """Slots, tokens and heads that lie more than 2^32 elements into the cache."""
    g = gen(43)
    hq, hk, d, cap = 8, 2, 128, 64
    base = torch.empty(5 * 2 ** 30, dtype=torch.bfloat16, device=DEV)
    v0 = 256
    for strides, slots in (((2 ** 31 + 2 ** 30, 512, 128), [0, 1]), ((2 ** 13, 2 ** 26, 128), [1, 0]), ((2 ** 16, 512, 2 ** 32), [1, 3])):
        k = base.as_strided((4 if strides[0] < 2 ** 20 else 2, cap, hk, d), strides + (1,))
        v = base.as_strided(k.shape, k.stride(), v0)
        k.copy_(torch.randn(k.shape, generator=g, device=DEV))
        v.copy_(torch.randn(k.shape, generator=g, device=DEV))
        lens = i32([64, 33])
        q = queries(2, hq, d, g)
        ws = bd.attn_workspace(2, 2, hq, hk, d, device=DEV)
        want, bound, _ = ref.attention(q, k, v, lens, slots=i32(slots))
        ref.assert_close(bd.attn_decode(q, k, v, lens, ws, slots=i32(slots)), want, bound, str(strides))
        ref.assert_close(bd.attn_prefill(q, k, v, i32([0, 1, 2]), lens, ws, slots=i32(slots)), want, bound, str(strides))


def test_streams_and_graph(bd):
    """On a stream of its own, and captured once and replayed for other lengths, slots and queries."""
    g = gen(47)
    n, hq, hk, d = 6, 32, 4, 128
    k, v = make_cache(n + 1, 900, hk, d, g)
    q, lens, slots = queries(n, hq, d, g), i32([1] * n), i32(range(n))
    ids, pslots, plens = i32([0, -1, 0, 0, -1, 0]), i32([n]), i32([640])
    ws = bd.attn_workspace(n, n, hq, hk, d, weigh_len=900, device=DEV)
    weights = torch.zeros(n + 1, hk, 900, device=DEV)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws, slots=slots, weights=weights, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws, slots=slots, weights=weights, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(3):
        q.copy_(queries(n, hq, d, g))
        lens.copy_(torch.randint(0, 901, (n,), generator=g, device=DEV, dtype=torch.int32))
        ids.copy_(i32([[0, -1][(step + i) % 2] for i in range(n)]))
        slots.copy_(torch.randperm(n, generator=g, device=DEV))
        weights.zero_()
        graph.replay()
        want, bound, (added, rel) = ref.attention(q, k, v, lens, slots=slots, prefix_ids=ids, prefix_slots=pslots, prefix_lens=plens)
        ref.assert_close(out, want, bound)
        for b, L in enumerate(lens.tolist()):
            got = weights[int(slots[b]), :, :L].double()
            assert ((got - added[b]).abs() <= (rel.get(b, 0.0) + (hq // hk + 2) * ref.F32) * added[b]).all()


def test_workspace_is_reused_across_shapes(bd):
    g = gen(53)
    ws = bd.attn_workspace(700, 70, 64, 8, 128, weigh_len=2048, device=DEV)
    for (n, hq, hk, d, L) in ((70, 64, 8, 128, 300), (1, 64, 8, 128, 2048), (33, 16, 16, 64, 100), (2, 64, 8, 128, 2000)):
        k, v = make_cache(n, L, hk, d, g)
        lens = i32([L - i % 7 for i in range(n)])
        q = queries(n, hq, d, g)
        want, bound, _ = ref.attention(q, k, v, lens)
        ref.assert_close(bd.attn_decode(q, k, v, lens, ws), want, bound)
        q = queries(7 * n, hq, d, g)
        cu = i32([7 * i for i in range(n + 1)])
        want, bound, _ = ref.attention(q, k, v, lens, cu_q=cu)
        ref.assert_close(bd.attn_prefill(q, k, v, cu, lens, ws), want, bound)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 4.0])
def test_scales(bd, scale):
    """Negative scales, and zero: the mean of what is seen."""
    g = gen(61)
    n, hq, hk, d = 5, 8, 2, 64
    k, v = make_cache(n + 1, 300, hk, d, g)
    lens, ids, pslots, plens = i32([300, 1, 129, 20, 0]), i32([0, -1, 0, -1, 0]), i32([n]), i32([131])
    how = dict(scale=scale, window=140, sinks=2)
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(300, n, hq, hk, d, device=DEV)
    want, bound, _ = ref.attention(q, k, v, lens, **how)
    ref.assert_close(bd.attn_decode(q, k, v, lens, ws, **how), want, bound)
    how.update(prefix_ids=ids, prefix_slots=pslots, prefix_lens=plens)
    want, bound, _ = ref.attention(q, k, v, lens, **how)
    ref.assert_close(bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws, scale=scale, window=140, sinks=2), want, bound)
    q, cu = queries(260, hq, d, g), i32([0, 200, 201, 250, 260, 260])
    want, bound, _ = ref.attention(q, k, v, lens, cu_q=cu, **how)
    ref.assert_close(bd.attn_prefill(q, k, v, cu, lens, ws, **how), want, bound)


def test_more_requests_than_the_plan_keeps(bd):
    """700 requests, every one with a prefix of its own or of few, in decode and prefill."""
    g = gen(67)
    n, hq, hk, d = 700, 4, 2, 64
    k, v = make_cache(2 * n, 50, hk, d, g)
    lens = torch.randint(0, 51, (n,), generator=g, device=DEV, dtype=torch.int32)
    plens = torch.randint(0, 51, (n,), generator=g, device=DEV, dtype=torch.int32)
    pslots = (n + torch.randperm(n, generator=g, device=DEV)).to(torch.int32)
    new = torch.minimum(torch.randint(0, 4, (n,), generator=g, device=DEV, dtype=torch.int32), lens)
    cu = torch.cat([i32([0]), new.cumsum(0, dtype=torch.int32)])
    ws = bd.attn_workspace(2100, n, hq, hk, d, device=DEV)
    for few in (False, True):
        ids = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        if few:
            ids = ids % 3 - 1
        how = dict(window=60, sinks=3, prefix_ids=ids, prefix_slots=pslots, prefix_lens=plens)
        q = queries(n, hq, d, g)
        want, bound, _ = ref.attention(q, k, v, lens, **how)
        ref.assert_close(bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws, window=60, sinks=3), want, bound)
        q = queries(int(cu[-1]), hq, d, g)
        want, bound, _ = ref.attention(q, k, v, lens, cu_q=cu, **how)
        ref.assert_close(bd.attn_prefill(q, k, v, cu, lens, ws, **how), want, bound)
    assert bd.device_status(ws) == 0


def test_most_prefixes(bd):
    """As many prefixes as a call takes, two of them named."""
    g = gen(71)
    n, hq, hk, d, P = 5, 8, 2, 64, 8192
    k, v = make_cache(n + 2, 90, hk, d, g)
    lens, ids = i32([7, 0, 90, 33, 1]), i32([8191, 17, 8191, -1, 17])
    pslots = torch.zeros(P, dtype=torch.int32, device=DEV)
    plens = torch.zeros(P, dtype=torch.int32, device=DEV)
    pslots[17], pslots[8191], plens[17], plens[8191] = n, n + 1, 90, 41
    q = queries(n, hq, d, g)
    ws = bd.attn_workspace(n, n, hq, hk, d, device=DEV)
    want, bound, _ = ref.attention(q, k, v, lens, prefix_ids=ids, prefix_slots=pslots, prefix_lens=plens)
    ref.assert_close(bd.attn_decode_prefix(q, k, v, lens, ids, pslots, plens, ws), want, bound)


def test_empty_calls(bd):
    k, v = make_cache(2, 10, 2, 64, gen(1))
    ws = bd.attn_workspace(1, 1, 4, 2, 64, device=DEV)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert bd.attn_decode(q, k, v, i32([]), ws).shape == (0, 4, 64)
    assert bd.attn_prefill(q, k, v, i32([0]), i32([]), ws).shape == (0, 4, 64)
    assert bd.attn_prefill(q, k, v, i32([0, 0]), i32([3]), ws).shape == (0, 4, 64)


def test_python_refusals(bd):
    k, v = make_cache(2, 10, 2, 64, gen(1))
    q, lens = queries(2, 4, 64, gen(2)), i32([3, 4])
    ws = bd.attn_workspace(2, 2, 4, 2, 64, device=DEV)
    with pytest.raises(TypeError):
        bd.attn_decode(q, k.float(), v.float(), lens, ws)
    with pytest.raises(ValueError):
        bd.attn_decode(q, k, v[:, :5], lens, ws)
    with pytest.raises(ValueError):
        bd.attn_decode(q, k, v, lens.long(), ws)
    with pytest.raises(ValueError):
        bd.attn_decode(q, k, v, i32([3]), ws)
    with pytest.raises(ValueError):
        bd.attn_decode(q.transpose(1, 2), k, v, lens, ws)
    with pytest.raises(ValueError):
        bd.attn_decode(q, k, v, lens, ws, weights=torch.zeros(2, 10, 2, device=DEV))
    with pytest.raises(ValueError):
        bd.attn_decode(q, k, v, lens, ws, out=torch.empty(2, 4, 64, device=DEV))
    with pytest.raises(ValueError):
        bd.attn_decode_prefix(q, k, v, lens, i32([0, 0]), None, None, ws)
    with pytest.raises(bd.BitDeltaError):
        bd.attn_decode(q, k, v, lens, ws, weights=torch.zeros(2, 2, 10, device=DEV), window=-1)
    with pytest.raises(bd.BitDeltaError):
        bd.attn_decode(queries(2, 5, 64, gen(3)), k, v, lens, ws)
    with pytest.raises(bd.BitDeltaError):
        bd.attn_decode(q, k, v, lens, ws[:8])
    with pytest.raises(ValueError):
        bd.cache_evict(k, v, None, lens, i32([0]), i32([1]), 5, ws)

"""GPU: prompt calls on a 4-bit cache whose requests have very different numbers of rows: a few single tokens
beside a long run of one request, many requests of few rows each, and calls at the borders between them."""
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


def make_cache(slots, tokens, heads, d, g):
    cache = torch.randint(0, 256, (slots, heads, tokens // 16, 17 * d), generator=g, device=DEV, dtype=torch.uint8)
    cache[..., 16 * d:] = torch.randint(11 * 8, 16 * 8, cache[..., 16 * d:].shape, generator=g, device=DEV, dtype=torch.uint8)
    return cache


def offsets(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def spread(n, most):
    return [1 + 7919 * i % most for i in range(n)]


CASES = {  # (tokens before, new tokens) of each request
    "one run of 9": [(300, 1), (47, 9), (0, 3), (95, 2), (1, 2), (0, 0), (31, 1)],
    "runs of 8 and 9": [(100 + i, 8 + i % 2) if i < 4 else (i, 1) for i in range(24)],
    "runs of 16 and 17": [(100 + i, 16 + i % 2) if i < 4 else (i, 1) for i in range(40)],
    "a run of many keys": [(60, 2)] * 7 + [(9000, 20)] + [(1, 1)] * 12,
    "a run among 64": [(spread(64, 400)[i], 1 if i != 37 else 193) for i in range(64)],
    "a run at the end": [(50, 0)] * 6 + [(500, 17)],
    "65 tokens": [(x, 1) for x in spread(65, 500)],
    "4 of each of 70": [(x, 4) for x in spread(70, 300)],
    "600 and two runs": [(spread(600, 90)[i], 40 if i in (3, 590) else 1) for i in range(600)],
    "1024 tokens": [(x, 1) for x in spread(1024, 60)],
    "1025 tokens": [(x, 1) for x in spread(1025, 60)],
    "200 with rows": [(20, i % 3 * (i % 7 == 0)) for i in range(1000)],
}


@pytest.mark.parametrize("heads", [(16, 2, 128), (5, 5, 64), (24, 2, 64), (36, 1, 128)], ids=str)
@pytest.mark.parametrize("mask", [(0, 0), (33, 3), (1, 0), (40, 400)], ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_uneven(bd, heads, mask, case):
    (hq, hk, d), (window, sinks) = heads, mask
    before, counts = zip(*CASES[case])
    g, n, T = torch.Generator(DEV).manual_seed(hq + window), len(counts), sum(counts)
    lens, cu = i32([a + b for a, b in zip(before, counts)]), i32(offsets(counts))
    longest = int(lens.max())
    cache = make_cache(n + 1, -(-longest // 16) * 16, hk, d, g)
    slots = torch.randperm(n + 1, generator=g, device=DEV)[:n].to(torch.int32)
    ref.hide_unseen(cache, lens, rows=counts, slots=slots, window=window, sinks=sinks)
    q = torch.randn(T, hq, d, generator=g, device=DEV, dtype=torch.bfloat16)
    ws = bd.attn4_workspace(T, n, hq, hk, d, longest=longest, device=DEV)
    ws[256:] = 255                                          # what the workspace holds is nobody's
    out = torch.full_like(q, math.nan)
    bd.attn4_prefill(q, cache, cu, lens, ws, longest, slots=slots, window=window, sinks=sinks, out=out)
    want, bound = ref.attention(q, cache, lens, cu_q=cu, slots=slots, window=window, sinks=sinks)
    attention_ref.assert_close(out, want, bound, case)
    assert bd.device_status(ws) == 0
    again = bd.attn4_prefill(q, cache, cu, lens, ws, longest, slots=slots, window=window, sinks=sinks)
    assert torch.equal(out, again)


@pytest.mark.parametrize("wrong,served", [
    (dict(slots={2: -1}), [1, 1, 0, 1, 1]), (dict(lens={1: 129}), [1, 0, 1, 1, 1]), (dict(lens={1: 20}), [1, 0, 1, 1, 1]), (dict(slots={1: 5}, lens={3: -7}), [1, 0, 1, 0, 1]),
    (dict(cu={4: 27}), [1, 1, 1, 0, 0]), (dict(cu={1: -1}), [0, 0, 0, 0, 0]), (dict(cu={2: 2}), [1, 0, 0, 0, 0]), (dict(cu={5: 2 ** 30}), [1, 1, 1, 1, 0]),
], ids=str)
def test_requests_out_of_range(bd, wrong, served):
    """Rows of requests that are not served become zeros, whichever kernels would have served them, and rows of no request stay."""
    g, hq, hk, d, n = torch.Generator(DEV).manual_seed(80), 8, 2, 128, 12
    counts = [3, 21, 4, 2, 1] + [0] * (n - 5)
    args = dict(lens=[90, 77, 128, 5, 1] + [7] * (n - 5), slots=list(range(5)) + [0] * (n - 5), cu=offsets(counts))
    T = sum(counts) + 4                                     # the last four are no request's
    for name, values in wrong.items():
        for at, x in values.items():
            args[name][at] = x
    cache = make_cache(5, 128, hk, d, g)
    q = torch.randn(T, hq, d, generator=g, device=DEV, dtype=torch.bfloat16)
    ws = bd.attn4_workspace(T, n, hq, hk, d, longest=128, device=DEV)
    out = torch.full_like(q, 7.0)
    bd.attn4_prefill(q, cache, i32(args["cu"]), i32(args["lens"]), ws, 128, slots=i32(args["slots"]), out=out)
    assert bd.device_status(ws) == bd.BD_ERR_SLOT
    ends, first = args["cu"], 0
    broken = [b for b in range(n) if not 0 <= ends[b] <= ends[b + 1] <= T]
    behind = max(0, ends[broken[0]]) if broken else sum(counts)
    for b in range(5):
        if broken and b >= broken[0]:
            break
        rows = slice(ends[b], ends[b + 1])
        if served[b]:
            want, bound = ref.attention(q[rows], cache, i32([args["lens"][b]]), cu_q=[0, rows.stop - rows.start], slots=[args["slots"][b]])
            attention_ref.assert_close(out[rows], want, bound)
        else:
            assert (out[rows] == 0).all()
    assert (out[behind:] == (0 if broken else 7)).all()


def test_in_a_graph(bd):
    """A captured call whose rows move from one request to another, from few of each to many of one and to none."""
    g, hq, hk, d, n, T = torch.Generator(DEV).manual_seed(81), 16, 2, 128, 10, 40
    cache = make_cache(n, 208, hk, d, g)
    q = torch.randn(T, hq, d, generator=g, device=DEV, dtype=torch.bfloat16)
    cu, lens, slots = i32([4 * i for i in range(n + 1)]), i32([50 + i for i in range(n)]), i32(list(range(n)))
    ws = bd.attn4_workspace(T, n, hq, hk, d, longest=208, device=DEV)
    out = torch.empty_like(q)

    def call():
        bd.attn4_prefill(q, cache, cu, lens, ws, 208, slots=slots, window=77, sinks=5, out=out)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for counts in ([4] * n, [31] + [1] * 9, [1] * 9 + [31], [0] * 5 + [40] + [0] * 4, [8, 9, 8, 9, 0, 0, 6, 0, 0, 0], [0] * n, [1] * n, [12, 12, 12] + [0] * 7):
        cu.copy_(i32(offsets(counts)))
        lens.copy_(torch.randint(40, 209, (n,), generator=g, device=DEV))
        slots.copy_(torch.randperm(n, generator=g, device=DEV))
        out.fill_(7)
        graph.replay()
        want, bound = ref.attention(q, cache, lens, cu_q=cu, slots=slots, window=77, sinks=5)
        rows = sum(counts)
        attention_ref.assert_close(out[:rows], want[:rows], bound[:rows], str(counts))
        assert (out[rows:] == 7).all()
    assert bd.device_status(ws) == 0


def test_a_step_of_drafted_tokens_beside_a_prompt(bd):
    """Written, then attended to, twice in one workspace: several tokens of many requests and a chunk of one."""
    g, hq, hk, d, n = torch.Generator(DEV).manual_seed(82), 16, 2, 64, 30
    cache = bd.cache4(n, 160, hk, d, DEV)
    cache.copy_(make_cache(n, 160, hk, d, g))
    have = [5 * i % 60 for i in range(n)]
    before = cache.cpu()
    ws = bd.attn4_workspace(120, n, hq, hk, d, longest=160, device=DEV)
    for counts in ([1 + i % 3 if i != 11 else 60 for i in range(n)], [4] * n):
        T, cu = sum(counts), offsets(counts)
        have = [a + b for a, b in zip(have, counts)]
        k, v = torch.randn(2, T, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
        q, lens = torch.randn(T, hq, d, generator=g, device=DEV, dtype=torch.bfloat16), i32(have)
        bd.cache4_write(k, v, cache, lens, ws, cu_q=i32(cu))
        out = bd.attn4_prefill(q, cache, i32(cu), lens, ws, 160, window=50, sinks=2)
        before = ref.write(before, k, v, have, range(n), cu)
        assert torch.equal(cache.cpu(), before)
        want, bound = ref.attention(q, cache, lens, cu_q=cu, window=50, sinks=2)
        attention_ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


def test_steps_that_follow_closely(bd):
    """Steps of tokens and chunks, written and attended to without a pause: what a later step writes reaches no earlier one."""
    g, hq, hk, d, n, steps = torch.Generator(DEV).manual_seed(83), 16, 2, 128, 24, 8
    cache, have = bd.cache4(n, 512, hk, d, DEV), [7 * i % 50 for i in range(n)]
    cache.copy_(make_cache(n, 512, hk, d, g))
    ws = bd.attn4_workspace(96, n, hq, hk, d, longest=512, device=DEV)
    calls = []
    for i in range(steps):
        counts = [1 + (3 * i + b) % 2 if b != 5 * i % n else 45 for b in range(n)]
        have = [a + b for a, b in zip(have, counts)]
        T = sum(counts)
        k, v = torch.randn(2, T, hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
        q = torch.randn(T, hq, d, generator=g, device=DEV, dtype=torch.bfloat16)
        calls.append((k, v, q, i32(have), i32(offsets(counts)), torch.full_like(q, math.nan)))
    torch.cuda.synchronize()
    for k, v, q, lens, cu, out in calls:
        bd.cache4_write(k, v, cache, lens, ws, cu_q=cu)
        bd.attn4_prefill(q, cache, cu, lens, ws, 512, window=60, sinks=4, out=out)
    for _, _, q, lens, cu, out in calls:
        want, bound = ref.attention(q, cache, lens, cu_q=cu, window=60, sinks=4)
        attention_ref.assert_close(out, want, bound)
    assert bd.device_status(ws) == 0


def test_two_streams_at_once(bd):
    g, hq, hk, d, sides = torch.Generator(DEV).manual_seed(84), 32, 4, 128, []
    for n, run in ((12, 30), (20, 55)):
        cache, counts = make_cache(n, 1024, hk, d, g), [1] * (n // 2) + [run] + [1] * (n - n // 2 - 1)
        lens, cu = torch.randint(60, 1025, (n,), generator=g, device=DEV, dtype=torch.int32), i32(offsets(counts))
        q = torch.randn(sum(counts), hq, d, generator=g, device=DEV, dtype=torch.bfloat16)
        ws = bd.attn4_workspace(sum(counts), n, hq, hk, d, longest=1024, device=DEV)
        sides.append((torch.cuda.Stream(), cache, lens, cu, q, ws, ref.attention(q, cache, lens, cu_q=cu), torch.empty_like(q)))
    torch.cuda.synchronize()
    for _ in range(30):
        for stream, cache, lens, cu, q, ws, _, out in sides:
            with torch.cuda.stream(stream):
                bd.attn4_prefill(q, cache, cu, lens, ws, 1024, out=out)
    torch.cuda.synchronize()
    for _, _, _, _, _, ws, (want, bound), out in sides:
        attention_ref.assert_close(out, want, bound)
        assert bd.device_status(ws) == 0

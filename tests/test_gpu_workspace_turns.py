"""GPU: attention calls give the same result whatever other entry points wrote
into the workspace before them."""
import pytest
import torch

from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def test_workspace_taken_in_turns():
    """Requests that are joined over many blocks, before and after a compression and a linear in the same workspace."""
    bd = load_bd()
    g = torch.Generator(DEV).manual_seed(5)
    n, hq, hk, d, length, N, K = 3, 16, 2, 128, 9000, 512, 1024

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)
    k, v, q = normal(n + 1, length, hk, d), normal(n + 1, length, hk, d), normal(n, hq, d)
    lens = i32([length, 4000, 8999])
    prefix = (i32([0, -1, 0]), i32([n]), i32([5000]))
    sizes = [bd.bitdelta_attn_workspace(n, n, hq, hk, d, length), bd.bitdelta_compress_workspace(N, K), bd.bitdelta_linear_workspace(8, N, K, 2)]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device=DEV)
    wb = normal(N, K)
    wf = wb + 0.01 * normal(N, K)
    x, ids = normal(8, K), i32([0, 1, 0, 1, 1, -1, 0, 1])

    def attend():
        weights = torch.zeros(n + 1, hk, length, device=DEV)
        results = []
        for call in (lambda out: bd.attn_decode(q, k, v, lens, ws, weights=weights, out=out),
                     lambda out: bd.attn_decode_prefix(q, k, v, lens, *prefix, ws, out=out)):
            results.append(torch.full_like(q, 7.0))
            call(results[-1])
        return [*results, weights]
    want = attend()
    alpha, bits = bd.compress(wf, wb, workspace=ws)
    y = bd.linear(x, ids, wb, alpha.repeat(2), [bits, bits], workspace=ws)
    for before in (lambda: bd.compress(wf, wb, workspace=ws), lambda: bd.linear(x, ids, wb, alpha.repeat(2), [bits, bits], workspace=ws)):
        for _ in range(2):
            before()
            for a, b in zip(attend(), want):
                assert torch.equal(a, b)
    assert torch.equal(bd.linear(x, ids, wb, alpha.repeat(2), [bits, bits], workspace=ws), y)
    again = bd.compress(wf, wb, workspace=ws)
    assert torch.equal(again[0], alpha) and torch.equal(again[1], bits)
    assert bd.device_status(ws) == 0

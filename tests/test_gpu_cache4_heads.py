"""GPU: rows of more than 2^31 values into a 4-bit cache and out of it."""
import pytest
import torch

from tests import cache4_ref as ref
from tests.gpu_util import load_bd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_rows_of_many_heads():
    bd = load_bd()
    d, near = 128, 9
    hk = 2 ** 31 // d + near                                # heads whose values begin at 2^31 and beyond
    g = torch.Generator(DEV).manual_seed(70)
    k, v = torch.zeros(1, hk, d, dtype=torch.bfloat16, device=DEV), torch.zeros(1, hk, d, dtype=torch.bfloat16, device=DEV)
    for t in (k, v):
        for some in (t[0, :near], t[0, -2 * near:]):
            some.copy_(torch.randn(some.shape, generator=g, device=DEV))
    cache, ws = bd.cache4(1, 16, hk, d, DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens = torch.tensor([4], dtype=torch.int32, device=DEV)
    bd.cache4_write(k, v, cache, lens, ws)
    a, b = bd.cache4_read(torch.ones_like(k), torch.ones_like(v), cache, lens, ws)
    assert bd.device_status(ws) == 0
    for x, y in ((k, a), (v, b)):
        for at in (slice(0, near), slice(hk - 2 * near, hk)):
            assert torch.equal(y[0, at].double(), ref.as_held(x[0, at]))
        assert not y[0, near:-2 * near].any()

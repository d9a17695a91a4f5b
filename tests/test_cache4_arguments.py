"""The Python entry points of the 4-bit cache refuse, before the library is called, tensors that
the kernels could not reach or would misread.  On the CPU, with stand-ins for the CUDA tensors."""
import pytest
import torch

import bit_delta_compressed_gb300 as bd
from tests.test_workspace_arguments import OnDevice, lib  # noqa: F401

S, H, N, D, B, T = 3, 2, 4, 64, 2, 5
bf16, u8 = torch.bfloat16, torch.uint8


def operands():
    return {"q": OnDevice(B, 4, D, dtype=bf16), "rows_q": OnDevice(T, 4, D, dtype=bf16), "cache": OnDevice(S, H, N, 17 * D, dtype=u8),
            "k": OnDevice(T, H, D, dtype=bf16), "v": OnDevice(T, H, D, dtype=bf16), "k1": OnDevice(B, H, D, dtype=bf16), "v1": OnDevice(B, H, D, dtype=bf16),
            "lens": OnDevice(B), "slots": OnDevice(B), "cu": OnDevice(B + 1), "out": OnDevice(B, 4, D, dtype=bf16), "rows_out": OnDevice(T, 4, D, dtype=bf16),
            "ws": OnDevice(1 << 20, dtype=u8)}


CALLS = {
    "cache4_write": (lambda o: bd.cache4_write(o["k"], o["v"], o["cache"], o["lens"], o["ws"], slots=o["slots"], cu_q=o["cu"]), "k v cache lens ws slots cu"),
    "cache4_write_one": (lambda o: bd.cache4_write(o["k1"], o["v1"], o["cache"], o["lens"], o["ws"]), "k1 v1 cache lens ws"),
    "cache4_read": (lambda o: bd.cache4_read(o["k"], o["v"], o["cache"], o["lens"], o["ws"], slots=o["slots"], cu_q=o["cu"]), "k v cache lens ws slots cu"),
    "attn4_decode": (lambda o: bd.attn4_decode(o["q"], o["cache"], o["lens"], o["ws"], slots=o["slots"], out=o["out"]), "q cache lens ws slots out"),
    "attn4_prefill": (lambda o: bd.attn4_prefill(o["rows_q"], o["cache"], o["cu"], o["lens"], o["ws"], 60, slots=o["slots"], out=o["rows_out"]),
                      "rows_q cache cu lens ws slots rows_out"),
}


@pytest.mark.parametrize("call", CALLS)
def test_devices_types_and_shapes(lib, call):  # noqa: F811
    run, names = CALLS[call]
    run(operands())
    assert lib.called == ["bitdelta_" + call.replace("_one", "")]
    for name in names.split():
        for device in (1, -1):
            o = operands()
            o[name].index, o[name].is_cuda = device, device >= 0
            with pytest.raises(ValueError):
                run(o)
        if name == "ws":
            continue
        o = operands()
        t = o[name]
        o[name] = OnDevice(*t.shape, dtype=torch.float16)
        with pytest.raises((TypeError, ValueError)):
            run(o)
        o[name] = OnDevice(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype)
        if name != "lens":          # (the number of requests: the others then do not fit it)
            with pytest.raises(ValueError):
                run(o)
    o = operands()
    o["ws"] = OnDevice(1 << 20, dtype=u8, contiguous=False)
    with pytest.raises(ValueError):
        run(o)
    assert len(lib.called) == 1


def strided(t, *stride):
    t.meta = torch.empty_strided(t.shape, stride, dtype=t.dtype, device="meta")
    return t


def test_strides(lib):  # noqa: F811
    run = CALLS["cache4_write"][0]
    W = 17 * D
    for wrong in ((H * N * W, N * W, 2 * W, 1), (H * N * W * 2, N * W * 2, W * 2, 2)):      # blocks with gaps between and inside
        o = operands()
        strided(o["cache"], *wrong)
        with pytest.raises(ValueError):
            run(o)
    for name in ("k", "v"):
        for wrong in ((H * D * 2, D * 2, 1), (H * D * 2, D * 2, 2)):
            o = operands()
            strided(o[name], *wrong)
            with pytest.raises(ValueError):
                run(o)
    o = operands()
    strided(o["cache"], 10 * N * W, 3 * N * W, W, 1)
    strided(o["k"], 1024, D, 1)
    run(o)
    assert lib.args[1] == 1024 and lib.args[3] == H * D
    desc = bd.KVCache4Desc.from_buffer_copy(lib.args[6])
    assert [getattr(desc, n) for n, _ in desc._fields_] == [1 << 20, S, 16 * N, H, D, 10 * N * W, 3 * N * W]


def test_rows_and_requests(lib):  # noqa: F811
    o = operands()
    with pytest.raises(ValueError):
        bd.cache4_write(o["k"], o["v"], o["cache"], o["lens"], o["ws"])                     # five rows, two requests
    with pytest.raises(ValueError):
        bd.cache4_write(o["k"], o["v1"], o["cache"], o["lens"], o["ws"], cu_q=o["cu"])
    with pytest.raises(ValueError):
        bd.attn4_decode(o["q"], OnDevice(S, H, N, 17 * 96, dtype=u8), o["lens"], o["ws"])
    with pytest.raises(ValueError):
        bd.attn4_decode(o["q"], OnDevice(S, H, N, 17 * 128, dtype=u8), o["lens"], o["ws"])  # q's head_dim is another
    with pytest.raises(TypeError):
        bd.attn4_decode(o["q"], OnDevice(S, H, N, 17 * D, dtype=torch.int8), o["lens"], o["ws"])
    assert not lib.called


@pytest.mark.parametrize("given,passed", [(0, 0), (7, 7), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 5, -1)])
def test_masks_beyond_32_bits(lib, given, passed):  # noqa: F811
    o = operands()
    for mask in (dict(window=given, sinks=3), dict(window=3, sinks=given)):
        want = [passed if x == given else x for x in mask.values()]
        bd.attn4_decode(o["q"], o["cache"], o["lens"], o["ws"], out=o["out"], **mask)
        assert list(lib.args[7:9]) == want
        bd.attn4_prefill(o["rows_q"], o["cache"], o["cu"], o["lens"], o["ws"], 60, out=o["rows_out"], **mask)
        assert list(lib.args[10:12]) == want


def test_empty_caches_of_no_size():
    with pytest.raises(bd.BitDeltaError):
        bd.cache4(2, 100, 2, 64)
    with pytest.raises(bd.BitDeltaError):
        bd.cache4(0, 96, 2, 64)
    cache = bd.cache4(2, 96, 3, 64, device="cpu")
    assert cache.shape == (2, 3, 6, 17 * 64) and not cache.any()
    with pytest.raises(bd.BitDeltaError):
        bd.attn4_workspace(4, 2, 8, 3, 64)
    assert bd.attn4_workspace(4, 2, 6, 3, 64, longest=20, device="cpu").dtype == torch.uint8

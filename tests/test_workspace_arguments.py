"""The Python entry points refuse, before the library is called, a workspace
and other tensors that the kernels could not reach: on the CPU, on another
device, or with gaps.  On the CPU, with stand-ins for the CUDA tensors."""
import pytest
import torch

import bit_delta_compressed_gb300 as bd


class OnDevice:
    """A CUDA tensor as far as the bindings look at one."""

    def __init__(self, *shape, dtype=torch.int32, device=0, contiguous=True):
        self.meta = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self.index, self.whole = self.meta.shape, dtype, device, contiguous
        self.is_cuda, self.device = True, torch.device("cuda", device)

    def stride(self, *i):
        return self.meta.stride(*i)

    def dim(self):
        return self.meta.dim()

    def numel(self):
        return self.meta.numel()

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.whole

    def data_ptr(self):
        return 1 << 20


class Library:
    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        def call(*args):
            self.called.append(name)
            self.args = args
            return bd.BD_OK
        return call


@pytest.fixture()
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(bd, "get_lib", lambda: lib)
    monkeypatch.setattr(bd, "_stream", lambda stream=None: 0)
    return lib


S, C, H, D, B, V = 3, 10, 2, 64, 2, 2
bf16, f32 = torch.bfloat16, torch.float32


def operands():
    return {"q": OnDevice(B, 4, D, dtype=bf16), "k": OnDevice(S, C, H, D, dtype=bf16), "v": OnDevice(S, C, H, D, dtype=bf16),
            "lens": OnDevice(B), "slots": OnDevice(B), "ids": OnDevice(B), "pslots": OnDevice(1), "plens": OnDevice(1), "cu": OnDevice(B + 1),
            "out": OnDevice(B, 4, D, dtype=bf16), "weights": OnDevice(S, H, C, dtype=f32), "all_lens": OnDevice(S),
            "src": OnDevice(1), "dst": OnDevice(1), "kept": OnDevice(1, H, 5), "ws": OnDevice(1 << 20, dtype=torch.uint8)}


CALLS = {
    "attn_decode": (lambda o: bd.attn_decode(o["q"], o["k"], o["v"], o["lens"], o["ws"], slots=o["slots"], weights=o["weights"], out=o["out"]),
                    "q k v lens ws slots weights out"),
    "attn_decode_prefix": (lambda o: bd.attn_decode_prefix(o["q"], o["k"], o["v"], o["lens"], o["ids"], o["pslots"], o["plens"], o["ws"], out=o["out"]),
                           "q k v lens ids pslots plens ws out"),
    "attn_prefill": (lambda o: bd.attn_prefill(o["q"], o["k"], o["v"], o["cu"], o["lens"], o["ws"], out=o["out"]), "q k v cu lens ws out"),
    "cache_evict": (lambda o: bd.cache_evict(o["k"], o["v"], o["weights"], o["all_lens"], o["src"], o["dst"], 5, o["ws"], kept=o["kept"]),
                    "k v weights all_lens src dst ws kept"),
}


@pytest.mark.parametrize("call", CALLS)
def test_attention_calls(lib, call):
    run, names = CALLS[call]
    run(operands())
    assert lib.called == ["bitdelta_" + call]
    for name in names.split():
        for wrong in (dict(device=1), dict(device=-1)):
            o = operands()
            o[name].index = wrong["device"]
            o[name].is_cuda = wrong["device"] >= 0
            with pytest.raises(ValueError):
                run(o)
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8), OnDevice(1 << 20, dtype=torch.uint8, contiguous=False)):
        with pytest.raises(ValueError):
            run({**operands(), "ws": ws})
    assert len(lib.called) == 1


@pytest.mark.parametrize("given,passed", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                          (10 ** 30, 2 ** 31 - 1), (-1, -1), (-2 ** 32, -1), (-2 ** 32 + 5, -1)])
def test_masks_beyond_32_bits(lib, given, passed):
    """A window or a number of first tokens that the C ABI's int32 does not hold is not cut down to its low bits."""
    o = operands()
    for mask in (dict(window=given, sinks=3), dict(window=3, sinks=given)):
        want = [passed if x == given else x for x in mask.values()]
        bd.attn_decode(o["q"], o["k"], o["v"], o["lens"], o["ws"], out=o["out"], **mask)
        assert list(lib.args[7:9]) == want
        bd.attn_decode_prefix(o["q"], o["k"], o["v"], o["lens"], o["ids"], o["pslots"], o["plens"], o["ws"], out=o["out"], **mask)
        assert list(lib.args[11:13]) == want
        bd.attn_prefill(o["q"], o["k"], o["v"], o["cu"], o["lens"], o["ws"], out=o["out"], **mask)
        assert list(lib.args[13:15]) == want


M, N, K = 4, 32, 64
LINEAR = {
    "compress": lambda ws: bd.compress(OnDevice(N, K, dtype=bf16), OnDevice(N, K, dtype=bf16), workspace=ws, alpha_out=OnDevice(1, dtype=f32), bits_out=OnDevice(N, K // 32)),
    "linear": lambda ws: bd.linear(OnDevice(M, K, dtype=bf16), OnDevice(M), OnDevice(N, K, dtype=bf16), OnDevice(V, dtype=f32), [OnDevice(N, K // 32)] * V,
                                   workspace=ws, out=OnDevice(M, N, dtype=f32)),
    "linear_rows": lambda ws: bd.linear_rows(OnDevice(M, K, dtype=bf16), OnDevice(M), OnDevice(N, K, dtype=bf16), OnDevice(V, N, dtype=f32), [OnDevice(N, K // 32)] * V,
                                             workspace=ws, out=OnDevice(M, N, dtype=f32)),
    "group": lambda ws: bd.group(OnDevice(M), V, ws),
    "linear_grouped": lambda ws: bd.linear_grouped(OnDevice(M, K, dtype=bf16), OnDevice(N, K, dtype=bf16), OnDevice(V, dtype=f32),
                                                   bd.bits_pointer_array([OnDevice(N, K // 32)] * V), V, OnDevice(M, N, dtype=bf16), ws),
}


@pytest.mark.parametrize("call", LINEAR)
def test_linear_and_compress_calls(lib, call):
    LINEAR[call](OnDevice(1 << 20, dtype=torch.uint8))
    assert len(lib.called) == 1
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8), OnDevice(1 << 20, dtype=torch.uint8, device=1), OnDevice(1 << 20, dtype=torch.uint8, contiguous=False)):
        with pytest.raises(ValueError):
            LINEAR[call](ws)
    assert len(lib.called) == 1

"""Sizes and row strides past the ints of the C ABI are refused: ctypes would
cut them to their low 32 bits, and the call would take other rows."""
import ctypes

import pytest
import torch

import latency_skinny_bf16_gb300 as sk

FAR = (1 << 32) + 64          # its low 32 bits are a good stride
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Fake:
    """Stands for a CUDA tensor; nothing of it is read."""
    is_cuda, device, nbytes = True, torch.device("cuda", 0), 1 << 40

    def __init__(self, shape, dtype, ld=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        st = [1]
        for s in reversed(shape[1:]):
            st.insert(0, st[0] * s)
        if ld is not None:
            st[len(shape) - 2] = ld
        self._stride = tuple(st)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 40


class Stream:
    cuda_stream = 0


def test_ctypes_cuts_without_a_word():
    assert ctypes.c_int(FAR).value == 64


def pairs(T=8, k=4, dtype=I32, ld=None):
    return Fake((T, k), dtype, ld)


CALLS = {
    "ids' stride": lambda: sk.expert_dispatch(pairs(ld=FAR), 16, pos=pairs(), order=Fake((32,), I32), offsets=Fake((17,), I32)),
    "tokens": lambda: sk.expert_dispatch(pairs(1 << 32, 1), 16, pos=pairs(1 << 32, 1), order=Fake((1 << 32,), I32),
                                         offsets=Fake((17,), I32)),
    "num_experts": lambda: sk.expert_dispatch(pairs(), FAR, pos=pairs(), order=Fake((32,), I32), offsets=Fake((FAR + 1,), I32)),
    "x's stride": lambda: sk.expert_dispatch(pairs(), 16, x=Fake((8, 64), BF16, FAR), xs=Fake((32, 64), BF16), pos=pairs(),
                                             order=Fake((32,), I32), offsets=Fake((17,), I32)),
    "ys' stride": lambda: sk.expert_combine(Fake((32, 64), BF16, FAR), pairs(), out=Fake((8, 64), BF16)),
    "pos": lambda: sk.expert_combine(Fake((32, 64), BF16), pairs(8, FAR), out=Fake((8, 64), BF16)),
    "weights' stride": lambda: sk.expert_combine(Fake((32, 64), BF16), pairs(), pairs(dtype=F32, ld=FAR), out=Fake((8, 64), BF16)),
    "dy's stride": lambda: sk.expert_combine_grad(Fake((8, 64), BF16, FAR), Fake((32, 64), BF16), pairs(), dys=Fake((32, 64), BF16),
                                                  dweights=pairs(dtype=F32)),
    "w's stride": lambda: sk.experts_gemm(Fake((32, 64), BF16), Fake((5,), I32), Fake((4, 48, 64), BF16, FAR),
                                          out=Fake((32, 48), BF16)),
    "a's stride": lambda: sk.lora_gemm(Fake((8, 64), BF16), Fake((48, 64), BF16), Fake((4, 16, 64), BF16, FAR),
                                       Fake((4, 48, 16), BF16), Fake((8,), I32), out=Fake((8, 48), F32), workspace=Fake((1,), F32)),
    "workspace": lambda: sk.lora_workspace(FAR, 48, 16, F32),
    "gemm": lambda: sk.gemm(Fake((8, 64), BF16, FAR), Fake((48, 64), BF16), out=Fake((8, 48), F32), stream=Stream),
    "gemm's rows": lambda: sk.gemm(Fake((FAR, 64), BF16), Fake((48, 64), BF16), out=Fake((FAR, 48), F32), stream=Stream),
    "router_topk": lambda: sk.router_topk(Fake((8, 64), F32, FAR), 4, weights=pairs(dtype=F32), ids=pairs(), stream=Stream),
    "rmsnorm_gemm": lambda: sk.rmsnorm_gemm(Fake((8, 64), BF16), Fake((64,), BF16), 1e-6, Fake((48, 64), BF16, FAR),
                                            out=Fake((8, 48), F32), xn=Fake((8, 64), BF16), stream=Stream),
}


@pytest.mark.parametrize("call", CALLS)
def test_refused(call, monkeypatch):
    class Library:
        def __getattr__(self, name):
            def reached(*a):
                raise AssertionError(f"{name} was called")
            return reached
    monkeypatch.setattr(sk, "_lib", Library())
    monkeypatch.setattr(sk.experts, "_loaded", Library())
    monkeypatch.setattr(sk.experts, "_import_torch", lambda: None)
    monkeypatch.setattr(sk.experts, "torch", torch)
    monkeypatch.setattr(sk.experts, "_current", lambda device: 0)
    with pytest.raises(ValueError, match="past 2147483647"):
        CALLS[call]()

"""Calls of the operators for a few tokens and of the junction with tensors or a stream of another GPU: refused before
anything reaches the library, whose kernels run on the current device.  On stand-ins for tensors: no GPU is needed."""
import contextlib
import types

import pytest
import torch

import mxfp8_block_scaled_03_gb300 as mx

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
T, K, N, H, F, E, k = 3, 256, 128, 256, 128, 2, 2


class Tensor:
    """What the wrappers look at in a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), torch.device("cuda", device)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20


class Library:
    """Notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 4096

        def call(*a):
            self.calls.append(name)
            return mx.OK
        return call


@pytest.fixture
def library(monkeypatch):
    """A library that only counts, two GPUs of which 0 is current, and streams that select their device."""
    lib, current = Library(), [0]

    @contextlib.contextmanager
    def stream_context(stream):
        before, current[0] = current[0], stream.device.index
        try:
            yield
        finally:
            current[0] = before
    monkeypatch.setattr(mx, "lib", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    for name in ("empty", "empty_like"):
        def make(like, *a, dtype=None, device=None, **kw):
            shape, dev = (like.shape, like.device) if isinstance(like, Tensor) else (
                (like,) if isinstance(like, int) else like, device)
            return Tensor(dtype or getattr(like, "dtype", None), *shape, device=dev.index)
        monkeypatch.setattr(torch, name, make)
    return lib


def matvec(nv):
    w = [Tensor(U8, N, K // 2 if nv else K), Tensor(U8, mx._sf_mma_bytes(nv, N, K))] + ([Tensor(F32, 1)] if nv else [])
    t = dict(x=Tensor(BF16, T, K), w=w, out=Tensor(BF16, T, N), workspace=Tensor(U8, 4096))
    f = (lambda x, w, **kw: mx.nvfp4_matvec(x, w, **kw)) if nv else (lambda x, w, **kw: mx.mxfp8_matvec(x, *w, **kw))
    return f, t


def layer(nv):
    per = 2 if nv else 1

    def w(M, K):
        return [Tensor(U8, M, K // per), Tensor(U8, mx._sf_mma_bytes(nv, M, K))] + ([Tensor(F32, 1)] if nv else [])
    t = dict(x=Tensor(BF16, T, H), experts=Tensor(I32, T, k), gates=Tensor(F32, T, k), w1=w(E * 2 * F, H), w2=w(E * H, F),
             out=Tensor(BF16, T, H), workspace=Tensor(U8, 4096))
    if nv:
        return mx.nvfp4_moe_decode_fwd, t
    return (lambda x, experts, gates, w1, w2, **kw: mx.moe_decode_fwd(x, experts, gates, *w1, *w2, **kw)), t


def norm_fwd():
    t = dict(y=Tensor(BF16, T, H), res=Tensor(F32, T, H), w_post=Tensor(F32, H), gate=Tensor(F32, T, 1),
             w_pre=Tensor(F32, H), out=[Tensor(F32, T, H), Tensor(BF16, T, H), Tensor(F32, 2, T)])
    return mx.residual_norm_fwd, t


def norm_bwd():
    t = dict(dn=Tensor(BF16, T, H), dres_out=Tensor(F32, T, H), y=Tensor(BF16, T, H), res_out=Tensor(F32, T, H),
             stats=Tensor(F32, 2, T), w_post=Tensor(F32, H), gate=Tensor(F32, H), w_pre=Tensor(F32, H),
             workspace=Tensor(U8, 4096))
    return mx.residual_norm_bwd, t


CALLS = {"mxfp8_matvec": lambda: matvec(False), "nvfp4_matvec": lambda: matvec(True),
         "moe_decode_fwd": lambda: layer(False), "nvfp4_moe_decode_fwd": lambda: layer(True),
         "residual_norm_fwd": norm_fwd, "residual_norm_bwd": norm_bwd}


def flat(t):
    return [z for v in t.values() for z in (v if isinstance(v, list) else [v])]


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_the_current_device_are_taken(library, name):
    f, t = CALLS[name]()
    f(**t)
    assert library.calls == [name]


@pytest.mark.parametrize("name", CALLS)
def test_one_tensor_elsewhere_is_refused(library, name):
    f, t = CALLS[name]()
    for z in flat(t):
        z.device = torch.device("cuda", 1)
        with pytest.raises(ValueError):
            f(**t)
        z.device = torch.device("cuda", 0)
    assert library.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_all_tensors_on_a_device_that_is_not_current_are_refused(library, name):
    f, t = CALLS[name]()
    for z in flat(t):
        z.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        f(**t)
    assert library.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(library, name):
    f, t = CALLS[name]()
    with pytest.raises(ValueError):
        f(**t, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    assert library.calls == []
    f(**t, stream=types.SimpleNamespace(device=torch.device("cuda", 0)))
    for z in flat(t):      # the tensors' own stream makes their device the current one
        z.device = torch.device("cuda", 1)
    f(**t, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    assert library.calls == [name, name]

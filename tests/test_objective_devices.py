"""The router's and the cross entropy's calls with tensors or a stream of another GPU, and with wrong types and shapes:
refused before anything reaches the library.  On stand-ins for tensors: no GPU is needed."""
import types

import pytest
import torch

import mxfp8_block_scaled_03_gb300 as mx
from tests.test_decode_devices import Tensor, flat, library  # noqa: F401  (a fixture)

BF16, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
T, E, k, H, V = 6, 16, 3, 64, 100


def route_fwd():
    t = dict(logits=Tensor(BF16, T, E), token_mask=Tensor(torch.bool, T), workspace=Tensor(U8, 4096),
             out=[Tensor(I32, T, k), Tensor(F32, T, k), Tensor(F32, T), Tensor(I32, E + 1), Tensor(F32, E), Tensor(F32, 2)])
    return (lambda **kw: mx.moe_route_fwd(k=k, **kw)), t


def route_bwd():
    t = dict(logits=Tensor(F32, T, E), experts=Tensor(I32, T, k), gates=Tensor(F32, T, k), lse=Tensor(F32, T),
             counts=Tensor(I32, E + 1), dgates=Tensor(F32, T * k), dlosses=Tensor(F32, 2), row_of_slot=Tensor(I32, T, k),
             dprob_sum=Tensor(F32, E), out=Tensor(F32, T, E))
    return mx.moe_route_bwd, t


def lce_fwd():
    t = dict(x=Tensor(BF16, T, H), w=Tensor(BF16, V, H), targets=Tensor(I64, T), out=[Tensor(F32, T), Tensor(F32, T)],
             workspace=Tensor(U8, 4096))
    return mx.linear_cross_entropy_fwd, t


def lce_bwd():
    t = dict(dloss=Tensor(F32, T), x=Tensor(BF16, T, H), w=Tensor(BF16, V, H), targets=Tensor(I32, T), lse=Tensor(F32, T),
             dlse=Tensor(F32, T), out=[Tensor(BF16, T, H), Tensor(BF16, V, H)], workspace=Tensor(U8, 4096))
    return mx.linear_cross_entropy_bwd, t


CALLS = {"moe_route_fwd": route_fwd, "moe_route_bwd": route_bwd, "linear_cross_entropy_fwd": lce_fwd,
         "linear_cross_entropy_bwd": lce_bwd}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_the_current_device_are_taken(library, name):  # noqa: F811
    f, t = CALLS[name]()
    f(**t)
    for optional in ("out", "workspace", "token_mask", "dlse", "dprob_sum", "dlosses"):
        t.pop(optional, None)
    f(**t)
    assert library.calls == [name, name]


@pytest.mark.parametrize("name", CALLS)
def test_one_tensor_elsewhere_is_refused(library, name):  # noqa: F811
    f, t = CALLS[name]()
    for z in flat(t):
        z.device = torch.device("cuda", 1)
        with pytest.raises(ValueError):
            f(**t)
        z.device = torch.device("cuda", 0)
    assert library.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_wrong_types_and_shapes_are_refused(library, name):  # noqa: F811
    f, t = CALLS[name]()
    for z in flat(t):
        if z is t.get("workspace"):
            continue
        dtype, shape = z.dtype, z.shape
        z.dtype = torch.float64
        with pytest.raises(ValueError):
            f(**t)
        z.dtype, z.shape = dtype, torch.Size((*shape[:-1], shape[-1] + 1))
        with pytest.raises(ValueError):
            f(**t)
        z.shape = shape
    assert library.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(library, name):  # noqa: F811
    f, t = CALLS[name]()
    with pytest.raises(ValueError):
        f(**t, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    assert library.calls == []
    f(**t, stream=types.SimpleNamespace(device=torch.device("cuda", 0)))
    for z in flat(t):      # the tensors' own stream makes their device the current one
        z.device = torch.device("cuda", 1)
    f(**t, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    assert library.calls == [name, name]


def test_rows_without_gradients_are_refused(library):  # noqa: F811
    f, t = route_bwd()
    t["dgates"] = None
    with pytest.raises(ValueError):
        f(**t)

"""Outputs that are not as many as the call returns, and tensors with another number of dimensions: refused with ValueError
before anything reaches the library.  On stand-ins for tensors."""
import pytest
import torch

from tests.test_decode_devices import Tensor, library  # noqa: F401  (a fixture)
from tests.test_objective_devices import CALLS, F32


@pytest.mark.parametrize("name", [n for n in CALLS if n != "moe_route_bwd"])
@pytest.mark.parametrize("change", [lambda o: o[:-1], lambda o: [*o, Tensor(F32, 4)], lambda o: []])
def test_another_number_of_outputs_is_refused(library, name, change):  # noqa: F811
    f, t = CALLS[name]()
    t["out"] = change(list(t["out"]))
    with pytest.raises(ValueError):
        f(**t)
    assert library.calls == []


@pytest.mark.parametrize("name,which", [("moe_route_fwd", "logits"), ("moe_route_bwd", "logits"), ("moe_route_bwd", "experts"),
                                        ("linear_cross_entropy_fwd", "x"), ("linear_cross_entropy_fwd", "w"),
                                        ("linear_cross_entropy_bwd", "w"), ("linear_cross_entropy_bwd", "targets")])
def test_another_number_of_dimensions_is_refused(library, name, which):  # noqa: F811
    f, t = CALLS[name]()
    shape = t[which].shape
    for other in ((), (shape.numel(),) if len(shape) > 1 else (1, shape[0]), (*shape, 1)):
        t[which].shape = torch.Size(other)
        with pytest.raises(ValueError):
            f(**t)
    assert library.calls == []

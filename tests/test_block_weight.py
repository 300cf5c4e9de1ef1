"""A BlockWeight's tensors do not change under the addresses that it holds. On
the CPU: no device memory is touched."""

import pytest

from quantized_weight_skinny_amd import prompt_api as qp


@pytest.mark.parametrize("name", ["codes", "scales", "device", "n", "k", "_fields"])
def test_what_the_addresses_belong_to_is_not_replaced(name):
    w = qp.BlockWeight.__new__(qp.BlockWeight)
    setattr(w, name, 1)   # as its constructor does
    with pytest.raises(AttributeError, match="does not change"):
        setattr(w, name, 2)
    assert getattr(w, name) == 1
    w.label = "gate_up"   # anything else is the caller's
    w.label = "down"

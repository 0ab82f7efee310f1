"""smoke() calls every operator of the training step (read from its source; no GPU)."""
import inspect

import pytest

import __graft_entry__ as entry


@pytest.mark.parametrize("name", ["fp8_rmsnorm_quant", "fp8_rmsnorm_backward", "fp8_swiglu_quant", "fp8_swiglu_backward", "fp8_quant_grouped_t",
                                  "fp8_blockscaled_grouped_wgrad", "fp8_grad_norm", "fp8_grad_clip"])
def test_smoke_calls(name):
    assert "_smoke_train(" in inspect.getsource(entry.smoke)
    assert f"fb.{name}(" in inspect.getsource(entry._smoke_train)

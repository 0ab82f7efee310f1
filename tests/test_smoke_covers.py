"""smoke() calls every operator of the package's hot paths (read from its source; no GPU)."""
import inspect

import pytest

import __graft_entry__ as entry


@pytest.mark.parametrize("name", ["fp8_quant_act_1x128", "fp8_blockscaled_gemm", "fp8_kv_append", "fp8_kv_attention", "fp8_moe_route",
                                  "fp8_moe_route_backward", "fp8_moe_dispatch"])
def test_smoke_calls(name):
    source = inspect.getsource(entry.smoke) + inspect.getsource(getattr(entry, "_smoke_decoder", entry.smoke))
    assert f"fb.{name}(" in source

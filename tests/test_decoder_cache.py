"""A KVCache's tensors are fixed, and their storages are read at each call (no GPU: nothing is launched)."""
import types

import pytest

import fp8_block_scaled_05_amd as fb

torch = pytest.importorskip("torch")


def _tensors(device="cpu"):
    return [torch.zeros(8, 2, 16, 64, dtype=torch.uint8, device=device) for _ in range(2)] + [torch.ones(8, 2, device=device) for _ in range(2)]


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "args", "other"])
def test_tensors_cannot_be_replaced(name):
    """A call would go on with the memory of a replaced tensor, which may be given away by then."""
    cache = fb.KVCache.__new__(fb.KVCache)             # a whole one needs the GPU
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1))


def _append(tensors):
    rows = [torch.zeros(5, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2)]
    i32 = [torch.zeros(n, dtype=torch.int32) for n in (3, 2)] + [torch.zeros(2, 4, dtype=torch.int32)]
    fb.fp8_kv_append(*rows, types.SimpleNamespace(args=tuple(tensors)), *i32, 4)


@pytest.mark.parametrize("at,change,error,match", [
    (0, lambda t: t[:7], ValueError, "shape"), (1, lambda t: t.view(torch.int8), TypeError, "v must be"),
    (2, lambda t: t.double(), TypeError, "k_scale must be"), (3, lambda t: t[:, :1], ValueError, "v_scale has shape"),
    (0, lambda t: t[0], ValueError, "k must be"), (0, lambda t: t.transpose(2, 3).contiguous().transpose(2, 3), ValueError, "contiguous"),
    (3, lambda t: None, TypeError, "v_scale must be a tensor"), (0, lambda t: t, ValueError, "GPU")])
def test_tensors_are_read_at_each_call(at, change, error, match):
    t = _tensors()
    t[at] = change(t[at])
    with pytest.raises(error, match=match):
        _append(t)


def test_a_resized_tensor_is_refused():
    t = _tensors()
    t[1].resize_(4, 2, 16, 64)
    with pytest.raises(ValueError, match="v has shape"):
        _append(t)
    with pytest.raises(TypeError, match="KVCache"):
        _append(t[:3])

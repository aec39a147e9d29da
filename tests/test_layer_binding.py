"""The bindings of a layer's other serving steps with tensors that have no memory (no GPU): what they hand to the library, call after call."""
import pytest
import torch

F16 = torch.float16


@pytest.fixture
def layer(monkeypatch):
    """The module with its device checks and its launches taken out; `calls` are the descriptors that would have been launched."""
    from hadamard_rotated_codebook_gb300 import build
    build.build()
    from hadamard_rotated_codebook_gb300 import layer as mod
    mod.calls = []
    monkeypatch.setattr(mod, "_dev", lambda *a: None)
    monkeypatch.setattr(mod, "_i32", lambda *a: 16)
    monkeypatch.setattr(mod, "_call", lambda dev, fn, desc: mod.calls.append(desc))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)  # the index of their device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: t.device.index)
    mod._lora_bytes.clear()
    yield mod
    mod._lora_bytes.clear()
    del mod.calls


def _new(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_a_refused_call_leaves_no_size_behind(layer):
    """A call that the library refuses (a matrix without outputs; too many adapters) does not decide the workspace of a later one of the same
    tokens, requests, inputs and rank."""
    def call(out, adapters=2):
        n, n_in, rank = 3, 64, 8
        layer.cq_lora_add([_new(n, out)], _new(n, n_in), [_new(adapters, rank, n_in, dtype=F16)], [_new(adapters, out, rank, dtype=F16)],
                          _new(2, dtype=torch.int32), _new(3, dtype=torch.int32))
        return layer.calls[-1].workspace_bytes

    need = call(32)
    assert need >= 3 * 16 * 4
    for refused in ((0,), (32, 2 ** 30)):
        layer._lora_bytes.clear()
        assert call(*refused) == 0  # what is wrong with it is the library's to say
        assert call(32) == need


def test_norm_widths_that_leave_32_bits_are_refused(layer):
    """The library's sizes are 32 bits wide: a row of 2^32 + 64 elements is not one of 64."""
    for width in (2 ** 32 + 64, 2 ** 31, 2 ** 33):
        with pytest.raises(ValueError, match="32 bits"):
            layer.cq_block_norm(_new(1, width, dtype=F16))
    assert not layer.calls
    layer.cq_block_norm(_new(1, 64, dtype=F16))
    assert layer.calls[-1].width == 64


def test_ranks_that_leave_32_bits_are_refused(layer):
    rank = 2 ** 32 + 8
    with pytest.raises(ValueError, match="32 bits"):
        layer.cq_lora_add([_new(1, 4)], _new(1, 8), [_new(1, rank, 8, dtype=F16)], [_new(1, 4, rank, dtype=F16)], _new(1, dtype=torch.int32),
                          _new(2, dtype=torch.int32))

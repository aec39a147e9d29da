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

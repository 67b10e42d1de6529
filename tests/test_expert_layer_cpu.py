"""fp8_expert_layer: where it makes what lies between its steps. On the CPU, with the device `meta`
in the place of the GPU's and nothing launched."""
import contextlib

import pytest
import torch

import fp8_quantized_paged_store_gb300 as kvq


@pytest.fixture
def calls(monkeypatch):
    """(name, tensors) of every call of the library."""
    seen, tensors = [], []

    def note(name, args):
        tensors.append([t for t, *_ in args])
        return 0

    monkeypatch.setattr(kvq, "_tensors", note)
    monkeypatch.setattr(kvq, "_call", lambda name, *_: seen.append((name, tensors[-1])))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: t.device.type == "meta"), raising=False)
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: t)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, pin_memory=False, **k: empty(*a, **k))
    return seen


def arguments(tokens=5):
    def on(*shape, dtype=torch.uint8):
        return torch.empty(shape, dtype=dtype, device="meta")
    f32 = torch.float32
    return dict(x=on(tokens, 256), x_scales=on(tokens, 2, dtype=f32), gate_up=on(8, 256, 256), gate_up_scales=on(8, 2, 2, dtype=f32),
                down=on(8, 256, 128), down_scales=on(8, 2, 1, dtype=f32), top_k=2, status=on(1, dtype=torch.int32))


def test_what_lies_between_the_steps_is_made_on_the_device(calls):
    """Logits may lie in page-locked host memory; what is made of them may not: nothing keeps a block
    of host memory from its next user while the kernels read it."""
    kvq.fp8_expert_layer(logits=torch.zeros(5, 8), **arguments())
    assert [name for name, _ in calls] == ["route_experts", "sort_by_expert", "fp8_expert_gated_matmul",
                                           "fp8_expert_matmul", "combine_experts"]
    host = [(name, t.shape) for name, tensors in calls for t in tensors if not t.is_cuda]
    assert host == [("route_experts", (5, 8))]


def test_a_stream_of_another_device_is_refused_before_anything_runs(calls, monkeypatch):
    class Stream:
        device = torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(TypeError):
        kvq.fp8_expert_layer(logits=torch.zeros(5, 8), stream=Stream(), **arguments())
    assert not calls

"""Calls on tensors of a GPU that is not the current one, with the library and torch's device
calls replaced (no GPU needed): each entry point is called while the tensors' GPU is current,
with a stream of that GPU, and the caller's current GPU stays what it was."""
import ctypes

import pytest
import torch

from lora_rank_adapter_gb300 import binding, training

F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


class Far:
    """As much of a tensor on cuda:1 as the bindings look at."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, *shape, dtype=F32):
        self.like = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype = self.like.shape, dtype
        for name in ("dim", "numel", "stride", "is_contiguous", "element_size"):
            setattr(self, name, getattr(self.like, name))

    def get_device(self):
        return 1

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        pass


class Stream:
    def __init__(self, device):
        self.device_index, self.cuda_stream = device, 0x700 + device


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs, GPU 0 current: a list of (entry point, GPU current at the call, stream)."""
    state, calls = {"current": 0}, []

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *_):
            state["current"] = self.before

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                if name.endswith("_size"):
                    return 4096
                # the stream is the last argument
                calls.append((name, state["current"], args[-1]))
                return 0
            return entry

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x500 + d, raising=False)
    for module in (binding, training):
        monkeypatch.setattr(module, "lib", lambda: Library())
    monkeypatch.setattr(training, "_bytes", lambda size, device, stream: Far(size, dtype=torch.uint8))
    monkeypatch.setattr(training, "_workspace_size", lambda *a: 4096)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(d))
    monkeypatch.setattr(binding, "workspace", lambda *a, **k: Far(4096, dtype=torch.uint8))
    return state, calls


def _training_calls():
    T, V, P = 6, 40, 1
    x, lab, v = Far(T, V), Far(T, dtype=I64), Far(T)
    cu, ref, pair, loss, metrics = Far(3, dtype=I32), Far(2), Far(1), Far(1), Far(3)
    plan = lambda **k: training.lora_adamw_plan([Far(8)], [Far(8)], [Far(8)], [Far(8)], **k)  # noqa: E731
    return {
        "lora_token_logps": lambda **k: training.lora_token_logps(x, lab, v, **k),
        "lora_token_logps_backward": lambda **k: training.lora_token_logps_backward(x, lab, Far(T, 2), v, Far(T, V), **k),
        "lora_preference_loss": lambda **k: training.lora_preference_loss(x, lab, cu, ref, 0.1, v, Far(2 * P), pair, loss,
                                                                         dlogits=Far(T, V), **k),
        "lora_policy_loss": lambda **k: training.lora_policy_loss(x, lab, v, v, None, Far(T), metrics, **k),
        "lora_scale_gradient": lambda **k: training.lora_scale_gradient(x, loss, **k),
        "lora_adamw_build": plan,
        "lora_grad_norm": lambda **k: training.lora_grad_norm(plan(), 1.0, Far(2), **k),
        "lora_adamw": lambda **k: training.lora_adamw(plan(), 1e-3, 1, **k),
    }


def _adapter_calls():
    M, K, L, r, S, R = 16, 24, 32, 8, 3, 8
    X, A, B, Y, h, dY = Far(M, K), Far(K, r), Far(r, L), Far(M, L), Far(M, r), Far(M, L)
    dX, dA, dB = Far(M, K), Far(K, r), Far(r, L)
    slots, ranks, scal = Far(M, dtype=I32), Far(S, dtype=I32), Far(S)
    a, b, y, hm = Far(S, R, K, dtype=BF16), Far(S, L, R, dtype=BF16), Far(M, L, dtype=BF16), Far(M, R)
    x, ga, ids = Far(M, K, dtype=BF16), Far(S, R, 50, dtype=BF16), Far(M, dtype=I64)
    return {
        "lora_forward": lambda **k: binding.lora_forward(X, A, B, Y, 1.0, **k),
        "lora_forward_h": lambda **k: binding.lora_forward_h(X, A, B, Y, 1.0, h, **k),
        "lora_backward": lambda **k: binding.lora_backward(X, dY, A, B, h, 1.0, dX, dA, dB, **k),
        "lora_backward_ex": lambda **k: binding.lora_backward_ex(X, dY, A, B, h, 1.0, dX, dA, dB, **k),
        "lora_backward_dx_da": lambda **k: binding.lora_backward_dx_da(X, dY, A, B, 1.0, dX, dA, **k),
        "lora_backward_db": lambda **k: binding.lora_backward_db(X, A, dY, 1.0, dB, **k),
        "lora_group_by_slot": lambda **k: binding.lora_group_by_slot(slots, ranks, R, slots, slots, slots, **k),
        "lora_shrink": lambda **k: binding.lora_shrink(x, a, slots, ranks, R, hm, **k),
        "lora_expand": lambda **k: binding.lora_expand(hm, b, slots, ranks, scal, y, [L], R, **k),
        "lora_apply_linear": lambda **k: binding.lora_apply_linear(x, a, b, slots, ranks, scal, y, [L], R, **k),
        "lora_gather_shrink": lambda **k: binding.lora_gather_shrink(ids, ga, slots, ranks, R, hm, **k),
    }


CALLS = {**_training_calls(), **_adapter_calls()}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_tensors_gpu_is_current_during_the_call(gpus, name):
    state, calls = gpus
    address = lambda s: s.value if isinstance(s, ctypes.c_void_p) else s  # noqa: E731
    for here in (0, 1):
        state["current"] = here
        CALLS[name]()
        assert state["current"] == here
        entry, current, stream = calls[-1]
        assert entry == name and current == 1 and address(stream) == 0x501
        CALLS[name](stream=Stream(1))
        assert calls[-1][1] == 1 and address(calls[-1][2]) == 0x701


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_stream_of_another_gpu_is_refused(gpus, name):
    _, calls = gpus
    with pytest.raises(ValueError, match="cuda:0"):
        CALLS[name](stream=Stream(0))
    assert all(entry != name for entry, _, _ in calls)


def test_a_schedule_is_built_on_the_slots_gpu(gpus, monkeypatch):
    _, calls = gpus
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **{**k, "device": "cpu"}))
    binding.lora_build_schedule(Far(5, dtype=I32), Far(3, dtype=I32), 8)
    assert calls[-1][:2] == ("lora_build_schedule", 1)


def test_tensors_off_the_gpu_are_refused(gpus):
    _, calls = gpus
    X = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        binding.lora_forward(X, torch.zeros(8, 2), torch.zeros(2, 8), X, 1.0)
    assert not calls

"""A plan's table, which the binding allocates on the stream of the build: a call on another
stream is told to the allocator, which else hands the memory out while a kernel there still
reads addresses from it (the library and the streams replaced, no GPU needed)."""
import pytest
import torch

from lora_rank_adapter_gb300 import torch_ops, training
from tests.test_other_gpu_host import Far, Stream, gpus  # noqa: F401


@pytest.fixture
def tables(gpus, monkeypatch):  # noqa: F811
    """The streams recorded for each table made, and the current stream (of GPU 1)."""
    made, current = [], {"stream": Stream(1)}
    current["stream"].cuda_stream = 0x501

    def table(size, device, stream):
        t = Far(size, dtype=torch.uint8)
        recorded = []
        t.record_stream = lambda s: recorded.append(s.cuda_stream)
        made.append(recorded)
        return t

    monkeypatch.setattr(training, "_bytes", table)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current["stream"])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current["stream"].cuda_stream, raising=False)
    return made, current


def _plan(**k):
    return training.lora_adamw_plan([Far(8)], [Far(8)], [Far(8)], [Far(8)], **k)


def test_calls_on_the_plans_own_stream_record_nothing(tables):
    made, _ = tables
    plan = _plan()
    training.lora_grad_norm(plan, 1.0, Far(2))
    training.lora_adamw(plan, 1e-3, 1)
    side = Stream(1)
    other = _plan(stream=side)
    training.lora_adamw(other, 1e-3, 1, stream=side)
    assert made == [[], []]


def test_calls_on_other_streams_are_recorded_once_each(tables):
    made, current = tables
    plan, side = _plan(), Stream(1)
    for _ in range(2):
        training.lora_grad_norm(plan, 1.0, Far(2), stream=side)
        training.lora_adamw(plan, 1e-3, 1, stream=side)
    assert made == [[0x701]]
    # the current stream has changed since the build
    current["stream"] = Stream(1)
    current["stream"].cuda_stream = 0x888
    training.lora_adamw(plan, 1e-3, 1)
    training.lora_adamw(plan, 1e-3, 2)
    assert made == [[0x701, 0x888]]


@pytest.mark.gpu
def test_steps_on_changing_streams():
    """Gradients that move, so new plans, on a stream of their own and on the default one in turn,
    while the default stream's freed memory is written over: equal to steps on one stream."""
    dev = "cuda:0"
    torch.cuda.set_device(0)
    g = torch.Generator().manual_seed(0)
    begin = [torch.randn(300, 200, generator=g) for _ in range(20)]
    grads = [[torch.randn(300, 200, generator=g).to(dev) for _ in begin] for _ in range(3)]

    def run(streams):
        params = [t.to(dev).requires_grad_() for t in begin]
        opt = torch_ops.AdamW(params, lr=1e-2, max_norm=1.0)
        for k in range(12):
            s = streams[k % len(streams)]
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for p, v in zip(params, grads[k // 4]):
                    p.grad = v.clone() if k % 2 else v
                opt.step()
                opt.zero_grad()
            torch.cuda.current_stream().wait_stream(s)
            junk = [torch.full((4096,), 0x7F, dtype=torch.uint8, device=dev) for _ in range(32)]
            del junk
        torch.cuda.synchronize()
        return params

    side = torch.cuda.Stream()
    one = run([torch.cuda.current_stream()])
    for p, q in zip(one, run([side, torch.cuda.current_stream()])):
        assert torch.equal(p, q)

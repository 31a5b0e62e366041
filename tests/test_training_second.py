"""Second derivatives through the losses: they raise, none is taken for zero."""
import pytest
import torch

from lora_rank_adapter_gb300 import torch_ops, training

DEV = "cuda:0"
LABELS = [1, 0, 4, 2, 2, 1]


def _formula(logits):
    """The mean negative log-probability, and its gradient with respect to the logits."""
    logp = torch.log_softmax(logits, 1)
    labels = torch.tensor(LABELS, device=logits.device)
    d = (logp.exp() - torch.nn.functional.one_hot(labels, logits.shape[1])) / len(LABELS)
    return -logp.gather(1, labels[:, None]).mean(), d


def _losses(device):
    labels = torch.tensor(LABELS, device=device)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device=device)
    return {"preference": lambda x: torch_ops.preference_loss(x, labels, cu)[0],
            "policy": lambda x: torch_ops.policy_loss(x, labels, None, torch.ones(6, device=device))[0]}


def _check(loss, device):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(6, 3, generator=g).to(device)
    W = torch.randn(3, 7, generator=g).to(device).requires_grad_()
    (dW,) = torch.autograd.grad(loss(torch.tanh(x @ W)), W, create_graph=True)
    (first,) = torch.autograd.grad(loss(torch.tanh(x @ W)), W)
    assert torch.equal(dW.detach(), first) and not first.requires_grad
    with pytest.raises(RuntimeError, match="second derivatives|no autograd formula"):
        torch.autograd.grad(dW.square().sum(), W)


@pytest.mark.parametrize("which", ["preference", "policy"])
def test_second_derivatives_raise(which, monkeypatch):
    """The kernels replaced by the formula, on the CPU."""
    def op(n_outputs):
        def made(logits, *args):
            with torch.no_grad():
                loss, d = _formula(logits)
            empty = torch.zeros(3)
            return [loss, empty, empty, empty, d] if n_outputs == 5 else [loss.expand(3).clone(), empty, d]
        return made

    monkeypatch.setattr(torch_ops, "preference_loss_op", op(5))
    monkeypatch.setattr(torch_ops, "policy_loss_op", op(3))
    monkeypatch.setattr(training, "lora_scale_gradient", lambda d, f: d.mul_(f))
    _check(_losses("cpu")[which], "cpu")


@pytest.mark.parametrize("which", ["preference", "policy"])
def test_no_gradient_is_made_where_none_is_wanted(which, monkeypatch):
    """Under no_grad, logits that require a gradient themselves take no second pass and no memory."""
    wanted = []

    def op(logits, *args):
        wanted.append(args[-1])
        empty = torch.zeros(3)
        return [torch.zeros(()), empty, empty, empty, empty] if which == "preference" else [empty, empty, empty]

    monkeypatch.setattr(torch_ops, which + "_loss_op", op)
    x = torch.zeros(6, 7, requires_grad=True)
    loss = _losses("cpu")[which]
    with torch.no_grad():
        loss(x)
    loss(x.detach())
    loss(x)
    assert wanted == [False, False, True]


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["preference", "policy", "logps", "linear"])
def test_second_derivatives_raise_on_the_gpu(which):
    torch.cuda.set_device(0)
    labels = torch.tensor(LABELS, device=DEV)
    A, B = torch.ones(8, 2, device=DEV), torch.ones(2, 8, device=DEV)

    def linear(y):
        y = torch.nn.functional.pad(y, (0, 1))
        return torch_ops.lora_linear(y, A, B, torch.zeros_like(y), 1.0).square().sum()

    losses = {**_losses(DEV), "logps": lambda x: torch_ops.token_logps(x, labels).sum(), "linear": linear}
    _check(losses[which], DEV)

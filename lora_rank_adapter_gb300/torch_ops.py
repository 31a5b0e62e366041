"""PyTorch integration of liblora.so: custom ops and autograd.

The multi-adapter ops are registered as torch.library custom ops so that
torch.compile sees each as one opaque node, as the mstar page
"mstar.engine.resources.lora.ops" describes for its own ops: `expand_`,
`apply_linear_` and `forward_` add into their output in place and declare it
(mutates_args), so functionalization keeps every read of it ordered around the
add.  Each op has a fake (shape-only) implementation that runs without a GPU and
a CUDA implementation that calls the C ABI; there is no CPU kernel.

`LoraLinearFn` / `lora_linear` is an autograd.Function over the single-adapter
ops (NeMo AutoModel page "nemo_automodel.components._peft.lora_kernel":
lora_forward_wrapper, lora_da_dx_update_wrapper, lora_db_update_wrapper), on
the fused pair forward_h_ / backward_ex:
    out = base + scale * (x @ A) @ B
with gradients dx = scale * dout @ B^T @ A^T, dA = scale * x^T @ (dout @ B^T),
dB = scale * (x @ A)^T @ dout and dbase = dout.

`token_logps`, `preference_loss` and `policy_loss` are the differentiable forms of the
loss operators of `training`, and `AdamW` an optimizer on lora_grad_norm / lora_adamw:
    loss, pair_loss, seq_logps = preference_loss(logits, labels, cu_seqlens, ref_logps, beta=0.1)
    loss.backward(); optimizer.step()
The losses form their gradient with the forward pass, while a row is at hand; the
backward pass multiplies it by the incoming gradient in place (no pass over it when
that is 1; a bf16 gradient is rounded once more unless that is a power of two) and
hands it on, so it can be taken once and has no gradient of its own: second
derivatives (create_graph) through a loss raise.  That pass is Python, so
torch.compile runs the two losses outside its graph (fullgraph=True refuses them);
token_logps is two opaque nodes.
"""
from typing import List, Optional, Sequence

import torch

from . import binding, training

NS = "lora_gb300"


def _slots_list(out_slices: Sequence[int]) -> List[int]:
    return [int(v) for v in out_slices]


# ----------------------------------------------------------------------------- multi adapter
@torch.library.custom_op(f"{NS}::shrink", mutates_args=(), device_types="cuda")
def shrink(x: torch.Tensor, a: torch.Tensor, slots: torch.Tensor, ranks: torch.Tensor,
           max_rank: int, num_slices: int) -> torch.Tensor:
    """h[t, i*R + j] = x[t] . a[slot(t), i*R + j] (fp32; unspecified past the rank)."""
    h = torch.zeros((x.shape[0], num_slices * max_rank), dtype=torch.float32, device=x.device)
    binding.lora_shrink(x, a, slots, ranks, max_rank, h, num_slices=num_slices)
    return h


@shrink.register_fake
def _(x, a, slots, ranks, max_rank, num_slices):
    return x.new_empty((x.shape[0], num_slices * max_rank), dtype=torch.float32)


@torch.library.custom_op(f"{NS}::expand_", mutates_args=("y",), device_types="cuda")
def expand_(y: torch.Tensor, h: torch.Tensor, b: torch.Tensor, slots: torch.Tensor, ranks: torch.Tensor,
            scalings: torch.Tensor, out_slices: List[int], max_rank: int) -> None:
    """y[t, slice i] += scalings[slot] * h[t, slice i] @ b[slot, slice i]^T, in place."""
    binding.lora_expand(h, b, slots, ranks, scalings, y, _slots_list(out_slices), max_rank)


@expand_.register_fake
def _(y, h, b, slots, ranks, scalings, out_slices, max_rank):
    return None


@torch.library.custom_op(f"{NS}::apply_linear_", mutates_args=("y",), device_types="cuda")
def apply_linear_(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, slots: torch.Tensor,
                  ranks: torch.Tensor, scalings: torch.Tensor, out_slices: List[int], max_rank: int) -> None:
    """Shrink then expand into y, in place."""
    binding.lora_apply_linear(x, a, b, slots, ranks, scalings, y, _slots_list(out_slices), max_rank)


@apply_linear_.register_fake
def _(y, x, a, b, slots, ranks, scalings, out_slices, max_rank):
    return None


@torch.library.custom_op(f"{NS}::gather_shrink", mutates_args=(), device_types="cuda")
def gather_shrink(ids: torch.Tensor, a: torch.Tensor, slots: torch.Tensor, ranks: torch.Tensor,
                  max_rank: int) -> torch.Tensor:
    """h[t, j] = a[slot(t), j, ids[t]] for j < rank; zeros for ids outside [0, V)."""
    h = torch.zeros((ids.shape[0], max_rank), dtype=torch.float32, device=ids.device)
    binding.lora_gather_shrink(ids, a, slots, ranks, max_rank, h)
    return h


@gather_shrink.register_fake
def _(ids, a, slots, ranks, max_rank):
    return a.new_empty((ids.shape[0], max_rank), dtype=torch.float32)


# ----------------------------------------------------------------------------- single adapter
@torch.library.custom_op(f"{NS}::forward_", mutates_args=("y",), device_types="cuda")
def forward_(y: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: float) -> None:
    """y += scale * (x @ A) @ B, in place."""
    binding.lora_forward(x, A, B, y, scale)


@forward_.register_fake
def _(y, x, A, B, scale):
    return None


@torch.library.custom_op(f"{NS}::backward", mutates_args=(), device_types="cuda")
def backward(x: torch.Tensor, dout: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
             scale: float) -> List[torch.Tensor]:
    """(dx, dA, dB) of out = base + scale * (x @ A) @ B; dA and dB in fp32."""
    dx = torch.empty_like(x)
    dA = torch.empty(A.shape, dtype=torch.float32, device=x.device)
    dB = torch.empty(B.shape, dtype=torch.float32, device=x.device)
    binding.lora_backward_dx_da(x, dout, A, B, scale, dx, dA)
    binding.lora_backward_db(x, A, dout, scale, dB)
    return [dx, dA, dB]


@backward.register_fake
def _(x, dout, A, B, scale):
    return [torch.empty_like(x), A.new_empty(A.shape, dtype=torch.float32),
            B.new_empty(B.shape, dtype=torch.float32)]


@torch.library.custom_op(f"{NS}::forward_h_", mutates_args=("y",), device_types="cuda")
def forward_h_(y: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: float) -> torch.Tensor:
    """y += scale * (x @ A) @ B in place; returns h = x @ A (fp32) for backward_ex."""
    h = torch.empty((x.shape[0], A.shape[1]), dtype=torch.float32, device=x.device)
    binding.lora_forward_h(x, A, B, y, scale, h)
    return h


@forward_h_.register_fake
def _(y, x, A, B, scale):
    return x.new_empty((x.shape[0], A.shape[1]), dtype=torch.float32)


@torch.library.custom_op(f"{NS}::backward_ex", mutates_args=(), device_types="cuda")
def backward_ex(x: torch.Tensor, dout: torch.Tensor, A: torch.Tensor, B: torch.Tensor, h: torch.Tensor,
                scale: float, grads_in_input_dtype: bool) -> List[torch.Tensor]:
    """(dx, dA, dB) in one call from the h that forward_h_ saved (x is read
    once); dA and dB in x's dtype when grads_in_input_dtype, else fp32."""
    gdt = x.dtype if grads_in_input_dtype else torch.float32
    dx = torch.empty_like(x)
    dA = torch.empty(A.shape, dtype=gdt, device=x.device)
    dB = torch.empty(B.shape, dtype=gdt, device=x.device)
    flags = binding.BWD_GRAD_INPUT_DTYPE if grads_in_input_dtype else 0
    binding.lora_backward_ex(x, dout, A, B, h, scale, dx, dA, dB, flags=flags)
    return [dx, dA, dB]


@backward_ex.register_fake
def _(x, dout, A, B, h, scale, grads_in_input_dtype):
    gdt = x.dtype if grads_in_input_dtype else torch.float32
    return [torch.empty_like(x), A.new_empty(A.shape, dtype=gdt), B.new_empty(B.shape, dtype=gdt)]


class LoraLinearFn(torch.autograd.Function):
    """out = base + scale * (x @ A) @ B on the GPU kernels: the forward saves
    h = x @ A, and the backward computes dx, dA and dB in one call from it (x is
    read once), returning dA and dB in the parameters' dtype (rounded once from
    the fp32 sums)."""

    @staticmethod
    def forward(ctx, x, A, B, base, scale):
        out = base.clone()
        h = forward_h_(out, x, A, B, float(scale))
        ctx.save_for_backward(x, A, B, h)
        ctx.scale = float(scale)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, A, B, h = ctx.saved_tensors
        in_dtype = A.dtype == x.dtype and B.dtype == x.dtype
        dx, dA, dB = backward_ex(x, dout.contiguous(), A, B, h, ctx.scale, in_dtype)
        return dx, dA.to(A.dtype), dB.to(B.dtype), dout, None


def lora_linear(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, base: torch.Tensor, scale: float):
    """Differentiable out = base + scale * (x @ A) @ B (x [M,K], A [K,r], B [r,L], base [M,L])."""
    return LoraLinearFn.apply(x, A, B, base, scale)


# ----------------------------------------------------------------------------- losses over logits
@torch.library.custom_op(f"{NS}::token_logps", mutates_args=(), device_types="cuda")
def token_logps_op(logits: torch.Tensor, labels: torch.Tensor, temperature: float) -> List[torch.Tensor]:
    """(logps, stats): the labels' log-probabilities, and what their gradient needs."""
    T = logits.shape[0]
    logps = torch.empty(T, dtype=torch.float32, device=logits.device)
    stats = torch.empty((T, 2), dtype=torch.float32, device=logits.device)
    training.lora_token_logps(logits, labels, logps, temperature=temperature, stats=stats)
    return [logps, stats]


@token_logps_op.register_fake
def _(logits, labels, temperature):
    T = logits.shape[0]
    return [logits.new_empty((T,), dtype=torch.float32), logits.new_empty((T, 2), dtype=torch.float32)]


@torch.library.custom_op(f"{NS}::token_logps_backward", mutates_args=(), device_types="cuda")
def token_logps_backward_op(logits: torch.Tensor, labels: torch.Tensor, stats: torch.Tensor, dlogps: torch.Tensor,
                            temperature: float) -> torch.Tensor:
    """dlogits from the log-probabilities' gradient."""
    dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    training.lora_token_logps_backward(logits, labels, stats, dlogps, dlogits, temperature=temperature)
    return dlogits


@token_logps_backward_op.register_fake
def _(logits, labels, stats, dlogps, temperature):
    return logits.new_empty(logits.shape)


@torch.library.custom_op(f"{NS}::preference_loss", mutates_args=(), device_types="cuda")
def preference_loss_op(logits: torch.Tensor, labels: torch.Tensor, cu_seqlens: torch.Tensor,
                       ref_logps: Optional[torch.Tensor], beta: float, kind: str, label_smoothing: float,
                       length_normalize: bool, temperature: float, with_gradient: bool) -> List[torch.Tensor]:
    """(loss [], pair_loss [P], seq_logps [2P], token_logps [T], dlogits: empty without a gradient)."""
    T, P, f32 = logits.shape[0], cu_seqlens.numel() // 2, torch.float32
    dev = logits.device
    loss, pair = torch.empty((), dtype=f32, device=dev), torch.empty(P, dtype=f32, device=dev)
    seq, tok = torch.empty(2 * P, dtype=f32, device=dev), torch.empty(T, dtype=f32, device=dev)
    d = torch.empty(logits.shape if with_gradient else (0, 0), dtype=logits.dtype, device=dev)
    training.lora_preference_loss(logits, labels, cu_seqlens, ref_logps, beta, tok, seq, pair, loss,
                                  dlogits=d if with_gradient else None, kind=kind, label_smoothing=label_smoothing,
                                  length_normalize=length_normalize, temperature=temperature)
    return [loss, pair, seq, tok, d]


@preference_loss_op.register_fake
def _(logits, labels, cu_seqlens, ref_logps, beta, kind, label_smoothing, length_normalize, temperature,
      with_gradient):
    T, P = logits.shape[0], cu_seqlens.numel() // 2
    new = lambda *shape: logits.new_empty(shape, dtype=torch.float32)  # noqa: E731
    return [new(), new(P), new(2 * P), new(T), logits.new_empty(logits.shape if with_gradient else (0, 0))]


@torch.library.custom_op(f"{NS}::policy_loss", mutates_args=(), device_types="cuda")
def policy_loss_op(logits: torch.Tensor, labels: torch.Tensor, old_logps: Optional[torch.Tensor],
                   advantages: torch.Tensor, weights: Optional[torch.Tensor], ref_logps: Optional[torch.Tensor],
                   clip_low: float, clip_high: float, kl_beta: float, temperature: float,
                   with_gradient: bool) -> List[torch.Tensor]:
    """(metrics [3]: loss, weighted KL, weight of the clipped tokens; token_logps [T]; dlogits)."""
    T, dev = logits.shape[0], logits.device
    metrics = torch.empty(3, dtype=torch.float32, device=dev)
    tok = torch.empty(T, dtype=torch.float32, device=dev)
    d = torch.empty(logits.shape if with_gradient else (0, 0), dtype=logits.dtype, device=dev)
    training.lora_policy_loss(logits, labels, old_logps, advantages, weights, tok, metrics, ref_logps=ref_logps,
                              dlogits=d if with_gradient else None, clip_low=clip_low, clip_high=clip_high,
                              kl_beta=kl_beta, temperature=temperature)
    return [metrics, tok, d]


@policy_loss_op.register_fake
def _(logits, labels, old_logps, advantages, weights, ref_logps, clip_low, clip_high, kl_beta, temperature,
      with_gradient):
    T = logits.shape[0]
    return [logits.new_empty((3,), dtype=torch.float32), logits.new_empty((T,), dtype=torch.float32),
            logits.new_empty(logits.shape if with_gradient else (0, 0))]


class TokenLogpsFn(torch.autograd.Function):
    """logps[t] = log_softmax(logits[t] / temperature)[labels[t]]."""

    @staticmethod
    def forward(ctx, logits, labels, temperature):
        logps, stats = token_logps_op(logits, labels, temperature)
        ctx.save_for_backward(logits, labels, stats)
        ctx.temperature = temperature
        return logps

    @staticmethod
    def backward(ctx, dlogps):
        logits, labels, stats = ctx.saved_tensors
        return token_logps_backward_op(logits, labels, stats, dlogps.contiguous(), ctx.temperature), None, None


def _anchor(logits):
    """A tensor of no elements with the logits' history: it keeps the way back to them open and
    not their memory.  None where no gradient is wanted."""
    return logits[:0].clone() if logits.requires_grad and torch.is_grad_enabled() else None


class _NoSecondFn(torch.autograd.Function):
    """The tensor itself as if made from the logits, by a node that refuses to be gone back
    through.  (A tensor without a history would be a constant to second derivatives.)"""

    @staticmethod
    def forward(ctx, d, anchor):
        return d.detach()

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("this loss has no second derivatives: its gradient is made with its forward pass")


def _hand_on(ctx, dloss):
    """The gradient that the forward pass made, times the loss's own: once."""
    if ctx.dlogits is None:
        raise RuntimeError("the gradient of this loss is made once, with its forward pass, and has been taken")
    d, ctx.dlogits = ctx.dlogits, None
    training.lora_scale_gradient(d, dloss.float().reshape(1))
    if torch.is_grad_enabled():              # create_graph
        d = _NoSecondFn.apply(d, *ctx.saved_tensors)
    return d


class PreferenceLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, anchor, *args):
        loss, pair, seq, tok, d = preference_loss_op(logits, *args, anchor is not None)
        ctx.save_for_backward(anchor)
        ctx.dlogits = d if anchor is not None else None
        ctx.mark_non_differentiable(pair, seq, tok)
        return loss, pair, seq, tok

    @staticmethod
    def backward(ctx, dloss, *_):
        return (_hand_on(ctx, dloss),) + (None,) * 9


class PolicyLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, anchor, *args):
        metrics, tok, d = policy_loss_op(logits, *args, anchor is not None)
        ctx.save_for_backward(anchor)
        ctx.dlogits = d if anchor is not None else None
        loss = metrics[0].clone()
        ctx.mark_non_differentiable(metrics, tok)
        return loss, metrics, tok

    @staticmethod
    def backward(ctx, dloss, *_):
        return (_hand_on(ctx, dloss),) + (None,) * 10


def token_logps(logits: torch.Tensor, labels: torch.Tensor, temperature: float = 1.0) -> torch.Tensor:
    """Differentiable log-probabilities [T] of labels [T] (int64; 0 where a label is outside
    [0, V)) under logits [T, V]."""
    return TokenLogpsFn.apply(logits, labels, float(temperature))


def preference_loss(logits, labels, cu_seqlens, ref_logps=None, beta=0.1, kind="sigmoid", label_smoothing=0.0,
                    length_normalize=False, temperature=1.0):
    """(loss, pair_loss [P], seq_logps [2P]) of P pairs of packed sequences, pair p preferring
    sequence p to sequence P + p; the loss is differentiable in the logits."""
    loss, pair, seq, _ = PreferenceLossFn.apply(logits, _anchor(logits), labels, cu_seqlens, ref_logps, float(beta),
                                                kind, float(label_smoothing), bool(length_normalize),
                                                float(temperature))
    return loss, pair, seq


def policy_loss(logits, labels, old_logps, advantages, weights=None, ref_logps=None, clip_low=0.2, clip_high=0.2,
                kl_beta=0.0, temperature=1.0):
    """(loss, metrics [3], token_logps [T]) of the clipped policy loss with a KL term; the loss
    is differentiable in the logits."""
    return PolicyLossFn.apply(logits, _anchor(logits), labels, old_logps, advantages, weights, ref_logps,
                              float(clip_low), float(clip_high), float(kl_beta), float(temperature))


# ----------------------------------------------------------------------------- optimizer
class AdamW:
    """AdamW over an adapter's tensors (all of one dtype), one launch a step.

    state_bits: 32, or 8 for e4m3 states with a scale for each 256 elements, rounded at
    random (reproducibly) so that they follow their gradients over any number of steps.
    masters: keep fp32 copies that the step updates (for bf16 parameters whose updates are
    smaller than their rounding).  max_norm: clip the gradients' global norm to it; `norm` then holds
    (norm, factor) of the last step.  Parameters without a gradient sit a step out: each
    has its own count of steps, which its bias corrections go by (one launch for each
    count there is)."""

    def __init__(self, params, lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32, masters=False,
                 max_norm=None):
        self.params = tuple(params)
        if len({id(p) for p in self.params}) != len(self.params):
            raise ValueError("a parameter is given twice: both of its updates would be under way at once")
        if state_bits not in (8, 32):
            raise ValueError("state_bits has to be 8 or 32")
        self.lr, self.betas, self.eps, self.weight_decay, self.max_norm = lr, betas, eps, weight_decay, max_norm
        self.step_count = 0                  # of the steps taken
        self._behind = {}                    # by parameter: how many of them it sat out
        self._plan, self._groups, self._laid_out = None, None, None
        self.norm = torch.zeros(2, device=self.params[0].device) if max_norm is not None and self.params else None
        zeros = lambda p, dt: torch.zeros_like(p, dtype=dt, requires_grad=False)  # noqa: E731
        dt = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        # the plans hold these tensors' addresses: tuples, since none of them may be replaced
        self.exp_avg = tuple(zeros(p, dt) for p in self.params)
        self.exp_avg_sq = tuple(zeros(p, dt) for p in self.params)
        scales = lambda: tuple(torch.zeros(-(-p.numel() // training.ADAMW_BLOCK), device=p.device)  # noqa: E731
                               for p in self.params)
        self.exp_avg_scale = scales() if state_bits == 8 else None
        self.exp_avg_sq_scale = scales() if state_bits == 8 else None
        self.masters = tuple(p.detach().float().clone(memory_format=torch.preserve_format) for p in self.params) \
            if masters else None

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def _states(self):
        return {k: v for k, v in (("exp_avg", self.exp_avg), ("exp_avg_sq", self.exp_avg_sq),
                                  ("exp_avg_scale", self.exp_avg_scale),
                                  ("exp_avg_sq_scale", self.exp_avg_sq_scale), ("masters", self.masters))
                if v is not None}

    def _steps(self):
        """The count of steps; of each parameter, where they differ."""
        counts = [self.step_count - self._behind.get(i, 0) for i in range(len(self.params))]
        return self.step_count if not any(self._behind.values()) else counts

    def state_dict(self):
        """The step count (a list of each parameter's, where they differ) and copies of the states."""
        return {"step": self._steps(), **{k: [t.clone() for t in v] for k, v in self._states().items()}}

    @torch.no_grad()
    def load_state_dict(self, state):
        """Takes over what state_dict() of an optimizer with the same parameters and options gave.
        8-bit codes have to lie in memory as the parameter does: a scale belongs to 256 of them
        in that order."""
        mine = self._states()
        if set(state) != set(mine) | {"step"} or any(len(state[k]) != len(v) for k, v in mine.items()) or \
                isinstance(state["step"], (list, tuple)) and len(state["step"]) != len(self.params):
            raise ValueError("the state is of another optimizer: other options or other parameters")
        for k, v in mine.items():
            for t, u in zip(v, state[k]):
                if t.shape != u.shape or t.dtype != u.dtype:
                    raise ValueError(f"{k} is of another shape or type")
                if t.dtype == torch.float8_e4m3fn and any(a != b for n, a, b in zip(t.shape, t.stride(), u.stride())
                                                          if n > 1):
                    raise ValueError(f"{k} holds 8-bit codes of another memory layout")
        for k, v in mine.items():
            for t, u in zip(v, state[k]):
                t.copy_(u)
        step = state["step"]
        counts = [int(c) for c in step] if isinstance(step, (list, tuple)) else [int(step)] * len(self.params)
        self.step_count = max(counts, default=0)
        self._behind = {i: self.step_count - c for i, c in enumerate(counts) if c != self.step_count}

    @torch.no_grad()
    def step(self):
        """One step from the parameters' .grad; the tensors' addresses are laid out again when a
        gradient has moved."""
        at = [i for i, p in enumerate(self.params) if p.grad is not None]
        if not at:
            return
        # a gradient laid out otherwise than its parameter is brought to the parameter's layout
        grads = [g if g.stride() == p.stride() else torch.empty_like(p, dtype=g.dtype).copy_(g)
                 for p, g in ((self.params[i], self.params[i].grad) for i in at)]
        laid_out = [(i, g.data_ptr(), g.dtype, g.stride(), self.params[i].data_ptr()) for i, g in zip(at, grads)]
        missed = [self._behind.get(i, 0) for i in at] if self._behind else None
        if self._laid_out != (laid_out, missed):
            self._laid_out = None
            self._lay_out(at, grads, missed)
            self._laid_out = (laid_out, missed)
        self.step_count += 1
        if len(at) < len(self.params):
            for i in set(range(len(self.params))).difference(at):
                self._behind[i] = self._behind.get(i, 0) + 1
        if self.max_norm is not None:
            training.lora_grad_norm(self._plan, self.max_norm, self.norm)
        for behind, plan in self._groups:
            training.lora_adamw(plan, self.lr, self.step_count - behind, self.betas[0], self.betas[1], self.eps,
                                self.weight_decay, grad_factor=None if self.max_norm is None else self.norm[1:])

    def _lay_out(self, at, grads, missed):
        """The plans of the parameters `at`: of all of them for the norm, and of those with the
        same count of steps for the step."""
        def plan(of):
            pick = lambda v: None if v is None else [v[at[k]] for k in of]  # noqa: E731
            made = training.lora_adamw_plan([self.params[at[k]].detach() for k in of], [grads[k] for k in of],
                                            pick(self.exp_avg), pick(self.exp_avg_sq), masters=pick(self.masters),
                                            exp_avg_scales=pick(self.exp_avg_scale),
                                            exp_avg_sq_scales=pick(self.exp_avg_sq_scale),
                                            stochastic=self.exp_avg_scale is not None)
            made.tensors = None              # gradients are not kept alive beyond the step that uses them
            return made

        counts = sorted(set(missed)) if missed else [0]
        everything = range(len(at))
        self._plan = plan(everything) if len(counts) == 1 or self.max_norm is not None else None
        self._groups = [(counts[0], self._plan)] if len(counts) == 1 else \
            [(c, plan([k for k in everything if missed[k] == c])) for c in counts]

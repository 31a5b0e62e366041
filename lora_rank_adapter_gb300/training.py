"""Thin Python binding of the training operators (include/lora_train.h): the
log-probabilities of labels, the preference loss and the clipped policy loss with
their gradients, and the AdamW step over an adapter's many tensors.

Like `binding`, each function has the name of the C entry point it calls, takes
torch tensors that already live on the GPU, checks and marshals them, allocates
the workspace the C side asks for and passes the current CUDA stream of the tensors'
GPU, whichever GPU is current; outputs are tensors of the caller.  All arithmetic
runs in the library's CUDA kernels.

    from lora_rank_adapter_gb300 import training
    training.lora_preference_loss(logits, labels, cu_seqlens, ref_logps, 0.1,
                                  token_logps, seq_logps, pair_loss, loss, dlogits=dlogits)
    plan = training.lora_adamw_plan(params, grads, exp_avg, exp_avg_sq)   # once
    training.lora_grad_norm(plan, 1.0, norm)                              # each step
    training.lora_adamw(plan, lr=1e-4, step=k, grad_factor=norm[1:])

`torch_ops` holds the differentiable forms.
"""
import ctypes
import functools

import torch

from . import binding
from .binding import _check, _dtype, _entry, _raw_stream

TRAIN_EXPORTS = ["lora_train_workspace_size", "lora_token_logps", "lora_token_logps_backward",
                 "lora_preference_loss", "lora_policy_loss", "lora_scale_gradient", "lora_adamw_table_size",
                 "lora_adamw_build", "lora_grad_norm", "lora_adamw"]
TRAIN_PREFERENCE_LOSS, TRAIN_POLICY_LOSS = 0, 1
PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
PREF_LENGTH_NORMALIZE = 1
ADAMW_STATE_8BIT, ADAMW_MASTER, ADAMW_STOCHASTIC = 1, 2, 16
ADAMW_BLOCK, ADAMW_CHUNK = 256, 2048
POLICY_HELD_BYTES = 768 << 10      # rows up to here need no workspace in lora_policy_loss


class AdamWTensor(ctypes.Structure):
    """lora_adamw_tensor_t: the device addresses of one tensor and its size."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("master", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class AdamWPlanStruct(ctypes.Structure):
    """lora_adamw_plan_t."""
    _fields_ = [("table", ctypes.c_void_p), ("chunks", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class AdamWHyper(ctypes.Structure):
    """lora_adamw_hyper_t."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


_lib = None


def lib():
    """The loaded liblora.so with the signatures of include/lora_train.h."""
    global _lib
    if _lib is not None:
        return _lib
    L = binding.lib()
    i32, i64, u32, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
    P, sz = ctypes.c_void_p, ctypes.c_size_t
    TP, PP, HP = ctypes.POINTER(AdamWTensor), ctypes.POINTER(AdamWPlanStruct), ctypes.POINTER(AdamWHyper)
    sig = {
        "lora_train_workspace_size": (sz, [i32, i64, i64]),
        "lora_token_logps": (i32, [i32, i64, i64, P, i64, P, f32, P, P, P]),
        "lora_token_logps_backward": (i32, [i32, i64, i64, P, i64, P, f32, P, P, P, i64, P]),
        "lora_preference_loss": (i32, [i32, i64, i64, i32, P, i64, P, P, P, i32, f32, f32, u32, f32, P, P, P, P,
                                       P, i64, f32, P, sz, P]),
        "lora_policy_loss": (i32, [i32, i64, i64, P, i64, P, P, P, P, P, f32, f32, f32, f32, P, P, P, i64, f32,
                                   P, sz, P]),
        "lora_scale_gradient": (i32, [i32, i64, i64, P, i64, P, P]),
        "lora_adamw_table_size": (sz, [TP, i32]),
        "lora_adamw_build": (i32, [TP, i32, i32, i32, u32, P, sz, PP, P]),
        "lora_grad_norm": (i32, [PP, f32, P, P]),
        "lora_adamw": (i32, [PP, HP, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _refuse(t, n, dtype, name, device):
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} has to be {dtype} on cuda:{device}, not {t.dtype} on {t.device}")
    raise ValueError(f"{name} has to hold {n} contiguous elements, not {tuple(t.shape)} of strides {t.stride()}")


def _vector(t, n, dtype, name, device):
    """The address of a contiguous tensor of n elements on GPU `device` (its number)."""
    if t.dtype is not dtype or t.get_device() != device or t.numel() != n or not t.is_contiguous():
        _refuse(t, n, dtype, name, device)
    return t.data_ptr()


def _optional(t, n, dtype, name, device):
    return None if t is None else _vector(t, n, dtype, name, device)


def _matrix(x, name):
    """(rows, columns, address, row stride) of a [T, V] tensor with unit column stride."""
    if x.dim() != 2:
        raise ValueError(f"{name} have to be [T, V]")
    if not x.is_cuda:
        raise ValueError(f"{name} have to be on a GPU")
    T, V = x.shape
    ld, unit = x.stride()
    if unit != 1 and V > 1 and T > 0:
        raise ValueError(f"{name} need unit column stride")
    return T, V, x.data_ptr(), ld if T > 1 else max(V, 1)


def _rows(logits, labels):
    T, V, x, ld = _matrix(logits, "logits")
    device = logits.get_device()
    return T, V, x, ld, _vector(labels, T, torch.int64, "labels", device), device


def _gradient(dlogits, logits):
    """(address, row stride) of the gradient of the logits."""
    if dlogits is None:
        return None, 0
    if dlogits.shape != logits.shape or dlogits.dtype is not logits.dtype or dlogits.device != logits.device:
        raise ValueError("dlogits have to be like the logits")
    return _matrix(dlogits, "dlogits")[2:]


@functools.lru_cache(maxsize=1024)
def _workspace_size(op, n, m):
    return lib().lora_train_workspace_size(op, n, m)


def _bytes(size, device, stream):
    """`size` bytes of device memory, in the order of `stream` (None: the current one):
    what the allocator hands out may be in use until the work before it is done."""
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def train_workspace(op, n, m=0, device="cuda", stream=None):
    """A uint8 workspace of lora_train_workspace_size() bytes (None when zero) on
    `device`, for work on `stream`."""
    size = _workspace_size(op, n, m)
    return _bytes(size, device, stream) if size else None


def _workspace(ws, op, n, m, device, stream):
    if ws is None:
        ws = train_workspace(op, n, m, device, stream)
    elif ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws has to be one stretch of memory on cuda:{device}, not {ws.device}, strides {ws.stride()}")
    return ws, (0 if ws is None else ws.data_ptr()), (0 if ws is None else ws.numel() * ws.element_size())


# ----------------------------------------------------------------------------- log-probabilities and losses
def lora_token_logps(logits, labels, logps, temperature=1.0, stats=None, stream=None):
    """logps[t] = log_softmax(logits[t] / temperature)[labels[t]] (fp32; 0 where the
    label is outside [0, V)).  stats: fp32 [T, 2] for lora_token_logps_backward."""
    T, V, x, ld, lab, dev = _rows(logits, labels)
    f32 = torch.float32
    entry = _entry(lib().lora_token_logps, dev)
    st = entry(_dtype(logits), T, V, x, ld, lab, temperature, _vector(logps, T, f32, "logps", dev),
               _optional(stats, 2 * T, f32, "stats", dev), _raw_stream(stream, dev))
    _check(st, "lora_token_logps")
    return logps


def lora_token_logps_backward(logits, labels, stats, dlogps, dlogits, temperature=1.0, stream=None):
    """dlogits of lora_token_logps from its stats and the log-probabilities' gradient
    dlogps (fp32 [T]); dlogits may be the logits themselves."""
    T, V, x, ld, lab, dev = _rows(logits, labels)
    f32 = torch.float32
    if dlogits is None:
        raise ValueError("dlogits are missing")
    d, ldd = _gradient(dlogits, logits)
    entry = _entry(lib().lora_token_logps_backward, dev)
    st = entry(_dtype(logits), T, V, x, ld, lab, temperature, _vector(stats, 2 * T, f32, "stats", dev),
               _vector(dlogps, T, f32, "dlogps", dev), d, ldd, _raw_stream(stream, dev))
    _check(st, "lora_token_logps_backward")
    return dlogits


def lora_preference_loss(logits, labels, cu_seqlens, ref_logps, beta, token_logps, seq_logps, pair_loss, loss,
                         dlogits=None, kind="sigmoid", label_smoothing=0.0, length_normalize=False, temperature=1.0,
                         grad_scale=1.0, ws=None, stream=None):
    """The paired log-ratio loss over packed sequences (int32 cu_seqlens [2P + 1]; pair p
    prefers sequence p to sequence P + p); with dlogits also its gradient.  ref_logps
    [2P] or None; token_logps [T], seq_logps [2P], pair_loss [P] and loss [1] are written."""
    T, V, x, ld, lab, dev = _rows(logits, labels)
    f32 = torch.float32
    if kind not in PREFERENCE_KINDS:
        raise ValueError(f"kind has to be one of {sorted(PREFERENCE_KINDS)}")
    n = cu_seqlens.numel()
    if n % 2 != 1:
        raise ValueError("cu_seqlens have to hold 2 P + 1 offsets")
    P = n // 2
    d, ldd = _gradient(dlogits, logits)
    ws, w, wn = _workspace(ws, TRAIN_PREFERENCE_LOSS, T, P, dev, stream)
    entry = _entry(lib().lora_preference_loss, dev)
    st = entry(_dtype(logits), T, V, P, x, ld, lab, _vector(cu_seqlens, n, torch.int32, "cu_seqlens", dev),
               _optional(ref_logps, 2 * P, f32, "ref_logps", dev), PREFERENCE_KINDS[kind], beta, label_smoothing,
               PREF_LENGTH_NORMALIZE if length_normalize else 0, temperature,
               _vector(token_logps, T, f32, "token_logps", dev), _vector(seq_logps, 2 * P, f32, "seq_logps", dev),
               _vector(pair_loss, P, f32, "pair_loss", dev), _vector(loss, 1, f32, "loss", dev), d, ldd, grad_scale,
               w, wn, _raw_stream(stream, dev))
    _check(st, "lora_preference_loss")
    return loss


def lora_policy_loss(logits, labels, old_logps, advantages, weights, token_logps, metrics, ref_logps=None,
                     dlogits=None, clip_low=0.2, clip_high=0.2, kl_beta=0.0, temperature=1.0, grad_scale=1.0,
                     ws=None, stream=None):
    """The clipped policy loss with a KL term, summed with the tokens' weights (None: 1);
    with dlogits also its gradient.  old_logps, ref_logps: fp32 [T] or None.  token_logps
    [T] and metrics [3] (loss, weighted KL, weight of the clipped tokens) are written."""
    T, V, x, ld, lab, dev = _rows(logits, labels)
    f32 = torch.float32
    d, ldd = _gradient(dlogits, logits)
    if d is None or V * logits.element_size() <= POLICY_HELD_BYTES:      # no workspace
        w = wn = 0
    else:
        ws, w, wn = _workspace(ws, TRAIN_POLICY_LOSS, T, V * logits.element_size(), dev, stream)
    entry = _entry(lib().lora_policy_loss, dev)
    st = entry(_dtype(logits), T, V, x, ld, lab, _optional(old_logps, T, f32, "old_logps", dev),
               _optional(ref_logps, T, f32, "ref_logps", dev), _vector(advantages, T, f32, "advantages", dev),
               _optional(weights, T, f32, "weights", dev), clip_low, clip_high, kl_beta, temperature,
               _vector(token_logps, T, f32, "token_logps", dev), _vector(metrics, 3, f32, "metrics", dev), d, ldd,
               grad_scale, w, wn, _raw_stream(stream, dev))
    _check(st, "lora_policy_loss")
    return metrics


def lora_scale_gradient(x, factor, stream=None):
    """x *= factor (fp32 device scalar) in place for a [T, V] gradient; no pass over x when it is 1."""
    T, V, p, ld = _matrix(x, "gradients")
    dev = x.get_device()
    entry = _entry(lib().lora_scale_gradient, dev)
    st = entry(_dtype(x), T, V, p, ld, _vector(factor, 1, torch.float32, "factor", dev), _raw_stream(stream, dev))
    _check(st, "lora_scale_gradient")
    return x


# ----------------------------------------------------------------------------- optimizer
class AdamWPlan:
    """The addresses of an optimizer's tensors, laid out once on the device.  Holds
    the tensors; build it again when one of them is replaced.  Its calls belong on one
    stream, or one after the other."""

    def __init__(self, struct, table, tensors, stream):
        self.struct, self.table, self.tensors = struct, table, tensors
        self.ref = ctypes.byref(struct)
        self.device, self.chunks = table.get_device(), int(struct.chunks)
        self.streams = {stream}              # the addresses of those that the table's memory waits for

    def used_on(self, stream):
        """The address of the stream of a call (None: the current one).  The table's memory is
        not handed out again before the work on that stream is done, whichever stream it is."""
        raw = torch._C._cuda_getCurrentRawStream(self.device) if stream is None else _raw_stream(stream, self.device)
        if raw not in self.streams:
            self.table.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
            self.streams.add(raw)
        return raw


def _expect(ok, what):
    if not ok:
        raise ValueError(what)


def _dense(t):
    """Whether the elements fill one stretch of memory in some order of the axes."""
    if t.numel() == 0:
        return True
    want = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda x: (x[1], x[0])):
        if size == 1:
            continue
        if stride != want:
            return False
        want *= size
    return True


def lora_adamw_plan(params, grads, exp_avg, exp_avg_sq, masters=None, exp_avg_scales=None, exp_avg_sq_scales=None,
                    stream=None, stochastic=False):
    """Lays out the tensors of lora_grad_norm and lora_adamw.  params and grads: lists of
    bf16 or fp32 tensors (one dtype each).  States in 32 bits: fp32 tensors.  States in 8
    bits: float8_e4m3fn (or uint8) codes of the same shape, with fp32 scales
    [ceil(numel / 256)] in exp_avg_scales / exp_avg_sq_scales (exp_avg_sq then holds the
    square root of the second moment).  masters: fp32 copies that the step updates, the
    parameters being their rounding.  A tensor, its gradient, states and master share one
    dense layout.  stochastic: 8-bit states are rounded at random (reproducibly, by step
    and place), without which they stop following their gradients over some thousand steps."""
    n = len(params)
    s8 = exp_avg_scales is not None
    _expect(s8 == (exp_avg_sq_scales is not None), "8-bit states need both lists of scales")
    _expect(s8 or not stochastic, "stochastic rounding is for 8-bit states")
    lists = {"grads": grads, "exp_avg": exp_avg, "exp_avg_sq": exp_avg_sq, "masters": masters,
             "exp_avg_scales": exp_avg_scales, "exp_avg_sq_scales": exp_avg_sq_scales}
    for name, values in lists.items():
        _expect(values is None or len(values) == n, f"{name} has to hold one tensor for each of the {n} params")
    device = params[0].device if n else torch.device("cuda", torch.cuda.current_device())
    _expect(device.type == "cuda", "params have to be on a GPU")
    state = (torch.float8_e4m3fn, torch.uint8) if s8 else (torch.float32,)
    kinds = {"grads": None, "exp_avg": state, "exp_avg_sq": state, "masters": (torch.float32,)}
    table_in = (AdamWTensor * max(n, 1))()
    for i, p in enumerate(params):
        _expect(p.dtype == params[0].dtype and p.device == device, "params have to share dtype and device")
        _expect(_dense(p), "params have to be dense")
        for name, allowed in kinds.items():
            if lists[name] is None:
                continue
            t = lists[name][i]
            allowed = allowed or (grads[0].dtype,)
            if t.dtype not in allowed or t.device != device:
                raise ValueError(f"{name}[{i}] has to be {allowed[0]} on {device}")
            if t.shape != p.shape or not (t.stride() == p.stride() or (t.is_contiguous() and p.is_contiguous())):
                raise ValueError(f"{name}[{i}] has to have its parameter's shape and strides")
        for name in ("exp_avg_scales", "exp_avg_sq_scales"):
            if s8:
                _vector(lists[name][i], -(-p.numel() // ADAMW_BLOCK), torch.float32, name, device.index)
        addr = lambda values: values[i].data_ptr() if values is not None and p.numel() else None  # noqa: E731
        table_in[i] = AdamWTensor(addr(params), addr(grads), addr(exp_avg), addr(exp_avg_sq), addr(exp_avg_scales),
                                  addr(exp_avg_sq_scales), addr(masters), p.numel())
    flags = (ADAMW_STATE_8BIT if s8 else 0) | (ADAMW_MASTER if masters is not None else 0) | \
        (ADAMW_STOCHASTIC if stochastic else 0)
    size = lib().lora_adamw_table_size(table_in, n)
    table = _bytes(size, device, stream)
    struct = AdamWPlanStruct()
    raw = _raw_stream(stream, device.index)
    entry = _entry(lib().lora_adamw_build, device.index)
    st = entry(table_in, n, _dtype(params[0]) if n else binding.LORA_F32, _dtype(grads[0]) if n else binding.LORA_F32,
               flags, table.data_ptr(), table.numel(), ctypes.byref(struct), raw)
    _check(st, "lora_adamw_build")
    return AdamWPlan(struct, table, (list(params), {k: list(v) for k, v in lists.items() if v is not None}), raw)


def lora_grad_norm(plan, max_norm, out, stream=None):
    """out[0] = the 2-norm of all gradients, out[1] = min(1, max_norm / (norm + 1e-6)) (fp32 [2])."""
    entry = _entry(lib().lora_grad_norm, plan.device)
    st = entry(plan.ref, max_norm, _vector(out, 2, torch.float32, "out", plan.device), plan.used_on(stream))
    _check(st, "lora_grad_norm")
    return out


def lora_adamw(plan, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_factor=None, stream=None):
    """One AdamW step over the plan's tensors; step counts from 1.  grad_factor: fp32
    device scalar that the gradients are multiplied by (lora_grad_norm's out[1:])."""
    hyper = AdamWHyper(lr, beta1, beta2, eps, weight_decay, step)
    entry = _entry(lib().lora_adamw, plan.device)
    st = entry(plan.ref, ctypes.byref(hyper), _optional(grad_factor, 1, torch.float32, "grad_factor", plan.device),
               plan.used_on(stream))
    _check(st, "lora_adamw")

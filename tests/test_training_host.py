"""The training operators of liblora.so on the host: every entry point of
include/lora_train.h is exported, and bad arguments are refused before anything
is launched (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from lora_rank_adapter_gb300 import training as T
from tests._util import ROOT

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: every call below fails validation or has nothing to do
ODD2 = ctypes.c_void_p(0x10002)      # aligned for bf16 only
ODD1 = ctypes.c_void_p(0x10001)
NULL = ctypes.c_void_p(0)
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return T.lib()


def test_every_declared_symbol_is_exported(L):
    with open(os.path.join(ROOT, "include", "lora_train.h")) as f:
        declared = re.findall(r"^LORA_API\s+[\w\s\*]+?\b(lora_\w+)\s*\(", f.read(), re.M)
    assert sorted(declared) == sorted(T.TRAIN_EXPORTS) and len(set(declared)) == len(declared)
    for name in declared:
        assert hasattr(L, name), name


ROWS = {"dt": 1, "T": 6, "V": 33, "x": FAKE, "ld": 33, "lab": FAKE, "temp": 1.0}
BAD_ROWS = [({"dt": 5}, UNSUPPORTED), ({"T": -1}, INVALID), ({"V": -1}, INVALID), ({"T": 1 << 31}, INVALID),
            ({"x": NULL}, INVALID), ({"x": ODD1}, ALIGNMENT), ({"dt": 0, "x": ODD2}, ALIGNMENT), ({"ld": 32}, INVALID),
            ({"lab": NULL}, INVALID), ({"lab": ctypes.c_void_p(0x10004)}, ALIGNMENT), ({"temp": 0.0}, INVALID),
            ({"temp": -1.0}, INVALID), ({"temp": NAN}, INVALID), ({"temp": INF}, INVALID)]


def logps(L, out=FAKE, stats=NULL, **k):
    k = {**ROWS, **k}
    return L.lora_token_logps(k["dt"], k["T"], k["V"], k["x"], k["ld"], k["lab"], k["temp"], out, stats, NULL)


def logps_bwd(L, stats=FAKE, g=FAKE, d=FAKE, ldd=33, **k):
    k = {**ROWS, **k}
    return L.lora_token_logps_backward(k["dt"], k["T"], k["V"], k["x"], k["ld"], k["lab"], k["temp"], stats, g, d, ldd,
                                       NULL)


def pref(L, P=2, cu=FAKE, ref=FAKE, kind=0, beta=0.1, eps=0.0, flags=0, tok=FAKE, seq=FAKE, pair=FAKE, loss=FAKE,
         d=NULL, ldd=0, gs=1.0, ws=NULL, wsb=0, **k):
    k = {**ROWS, **k}
    return L.lora_preference_loss(k["dt"], k["T"], k["V"], P, k["x"], k["ld"], k["lab"], cu, ref, kind, beta, eps,
                                  flags, k["temp"], tok, seq, pair, loss, d, ldd, gs, ws, wsb, NULL)


def policy(L, old=FAKE, ref=NULL, adv=FAKE, w=NULL, lo=0.2, hi=0.2, kl=0.0, tok=ctypes.c_void_p(0x20000), met=FAKE, d=NULL, ldd=0, gs=1.0,
           ws=NULL, wsb=0, **k):
    k = {**ROWS, **k}
    return L.lora_policy_loss(k["dt"], k["T"], k["V"], k["x"], k["ld"], k["lab"], old, ref, adv, w, lo, hi, kl,
                              k["temp"], tok, met, d, ldd, gs, ws, wsb, NULL)


@pytest.mark.parametrize("change,status", BAD_ROWS)
def test_rows_are_checked_by_every_loss_operator(L, change, status):
    for call in (logps, logps_bwd, pref, policy):
        assert call(L, **change) == status, call.__name__


def test_vocabulary_limit(L):
    for call in (logps, logps_bwd, pref, policy):
        assert call(L, V=(1 << 30) + 1, ld=1 << 31) == UNSUPPORTED, call.__name__


def test_token_logps_arguments(L):
    assert logps(L, out=NULL) == INVALID
    assert logps(L, out=ODD2) == ALIGNMENT
    assert logps(L, stats=ctypes.c_void_p(0x10004)) == ALIGNMENT      # pairs of floats
    assert logps(L, T=0, out=NULL, x=NULL, lab=NULL) == OK
    assert logps_bwd(L, d=NULL) == INVALID
    assert logps_bwd(L, stats=NULL) == INVALID
    assert logps_bwd(L, g=NULL) == INVALID
    assert logps_bwd(L, ldd=32) == INVALID
    assert logps_bwd(L, d=ODD1) == ALIGNMENT
    assert logps_bwd(L, x=FAKE, d=FAKE, ldd=40) == INVALID            # in place needs the logits' own stride
    assert logps_bwd(L, T=0, x=NULL, d=NULL, stats=NULL, g=NULL, lab=NULL) == OK


def test_preference_arguments(L):
    for change, status in [({"P": -1}, INVALID), ({"kind": 3}, UNSUPPORTED), ({"beta": 0.0}, INVALID),
                           ({"beta": NAN}, INVALID), ({"eps": -0.1}, INVALID), ({"eps": 1.5}, INVALID),
                           ({"flags": 2}, INVALID), ({"cu": NULL}, INVALID),
                           ({"cu": ODD2}, ALIGNMENT), ({"tok": NULL}, INVALID), ({"seq": NULL}, INVALID),
                           ({"pair": NULL}, INVALID), ({"loss": NULL}, INVALID), ({"ref": ODD2}, ALIGNMENT),
                           ({"d": FAKE, "ldd": 5}, INVALID), ({"gs": INF}, INVALID)]:
        assert pref(L, **change) == status, change
    need = L.lora_train_workspace_size(T.TRAIN_PREFERENCE_LOSS, 6, 2)
    assert need > 0
    assert pref(L) == WORKSPACE
    assert pref(L, eps=0.1, kind=1) == WORKSPACE          # smoothing belongs to the sigmoid loss; the others pass it by
    assert pref(L, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert pref(L, ws=ctypes.c_void_p(0x10080), wsb=need) == WORKSPACE


def test_policy_arguments(L):
    for change, status in [({"adv": NULL}, INVALID), ({"tok": NULL}, INVALID), ({"met": NULL}, INVALID),
                           ({"old": ODD2}, ALIGNMENT), ({"ref": ODD2}, ALIGNMENT), ({"w": ODD2}, ALIGNMENT),
                           ({"met": ODD2}, ALIGNMENT),
                           ({"lo": -0.1}, INVALID), ({"lo": 1.1}, INVALID), ({"hi": -1.0}, INVALID),
                           ({"hi": INF}, INVALID), ({"kl": NAN}, INVALID), ({"kl": -1.0}, INVALID),
                           ({"gs": NAN}, INVALID), ({"d": FAKE, "ldd": 3}, INVALID)]:
        assert policy(L, **change) == status, change
    assert policy(L, tok=FAKE, old=FAKE) == INVALID                   # an output that is an input
    # rows held on chip need no workspace; longer ones do, for a gradient
    size = L.lora_train_workspace_size
    assert size(T.TRAIN_POLICY_LOSS, 6, T.POLICY_HELD_BYTES) == 0
    need = size(T.TRAIN_POLICY_LOSS, 6, T.POLICY_HELD_BYTES + 1)
    assert need > 0 and size(T.TRAIN_POLICY_LOSS, 6, 0) == need
    V = T.POLICY_HELD_BYTES // 2 + 1
    long = dict(V=V, ld=V, d=ctypes.c_void_p(0x30000), ldd=V)
    assert policy(L, **long) == WORKSPACE
    assert policy(L, ws=FAKE, wsb=need - 1, **long) == WORKSPACE


def test_scale_gradient_arguments(L):
    f = lambda dt=1, n=4, v=9, x=FAKE, ld=9, s=FAKE: L.lora_scale_gradient(dt, n, v, x, ld, s, NULL)  # noqa: E731
    assert f(dt=4) == UNSUPPORTED
    assert f(n=-1) == INVALID
    assert f(ld=8) == INVALID
    assert f(x=NULL) == INVALID
    assert f(s=NULL) == INVALID
    assert f(x=ODD1) == ALIGNMENT
    assert f(n=0, x=NULL, s=NULL) == OK


def _tensors(*numels, **k):
    a = {"p": 0x10000, "g": 0x20000, "m": 0x30000, "v": 0x40000, "ms": 0x50000, "vs": 0x60000, "w": 0x70000, **k}
    return (T.AdamWTensor * max(len(numels), 1))(
        *[T.AdamWTensor(a["p"], a["g"], a["m"], a["v"], a["ms"], a["vs"], a["w"], n) for n in numels])


def build(L, tensors, n=1, pd=0, gd=0, flags=0, table=FAKE, size=0, plan=True):
    made = T.AdamWPlanStruct()
    return L.lora_adamw_build(tensors, n, pd, gd, flags, table, size, ctypes.byref(made) if plan else None, NULL)


def test_adamw_build_arguments(L):
    t = _tensors(5000)
    size = L.lora_adamw_table_size
    assert size(t, 1) >= 3 * 64 and size(_tensors(2048, 0, 1), 3) > 2 * 64
    assert size(_tensors(2048 * 1000), 1) - size(_tensors(2048 * 100), 1) == 900 * 64
    assert L.lora_adamw_table_size(t, -1) == 0 and L.lora_adamw_table_size(None, 1) == 0
    assert L.lora_adamw_table_size(_tensors(-1), 1) == 0
    assert build(L, t, plan=False) == INVALID
    assert build(L, t, pd=7) == UNSUPPORTED
    assert build(L, t, gd=7) == UNSUPPORTED
    assert build(L, t, flags=4) == INVALID
    assert build(L, _tensors(-5)) == INVALID
    assert build(L, None, n=2) == INVALID
    for name in ("p", "g", "m", "v"):
        assert build(L, _tensors(10, **{name: 0})) == INVALID, name
    assert build(L, _tensors(10, p=0x10002)) == ALIGNMENT                    # fp32 at 2 bytes
    assert build(L, _tensors(10, p=0x10002), pd=1) == WORKSPACE              # bf16: passes on to the next check
    assert build(L, _tensors(10, ms=0, vs=0)) == WORKSPACE                   # no scales wanted in 32 bits
    assert build(L, _tensors(10, ms=0), flags=T.ADAMW_STATE_8BIT) == INVALID
    assert build(L, _tensors(10, m=0x30001), flags=T.ADAMW_STATE_8BIT) == WORKSPACE
    assert build(L, _tensors(10, w=0), flags=T.ADAMW_MASTER) == INVALID
    assert build(L, t, size=size(t, 1) - 1) == WORKSPACE
    assert build(L, t, table=ctypes.c_void_p(0x10040), size=1 << 20) == WORKSPACE
    assert build(L, _tensors(0), table=NULL, size=1 << 20) == WORKSPACE       # even of nothing


def test_adamw_step_arguments(L):
    plan = T.AdamWPlanStruct(0x10000, 4, 0, 0, 0, 0)
    P = ctypes.byref
    good = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
    step = lambda p=plan, f=NULL, **k: L.lora_adamw(P(p), P(T.AdamWHyper(**{**good, **k})), f, NULL)  # noqa: E731
    for bad in ({"step": 0}, {"lr": -1.0}, {"lr": NAN}, {"beta1": 1.0}, {"beta2": 1.0}, {"beta1": -0.1},
                {"eps": -1e-9}, {"weight_decay": INF}):
        assert step(**bad) == INVALID, bad
    assert step(f=ODD2) == ALIGNMENT
    assert L.lora_adamw(P(plan), None, NULL, NULL) == INVALID
    assert step(T.AdamWPlanStruct(0, 4, 0, 0, 0, 0)) == INVALID
    assert step(T.AdamWPlanStruct(0x10000, -1, 0, 0, 0, 0)) == INVALID
    assert step(T.AdamWPlanStruct(0x10000, 4, 9, 0, 0, 0)) == UNSUPPORTED
    assert step(T.AdamWPlanStruct(0x10000, 4, 0, 0, 8, 0)) == INVALID
    assert step(T.AdamWPlanStruct(0, 0, 0, 0, 0, 0)) == INVALID              # never built
    assert step(T.AdamWPlanStruct(0x10000, 0, 0, 0, 0, 0)) == OK             # a plan of nothing
    norm = lambda p=plan, m=1.0, out=FAKE: L.lora_grad_norm(P(p), m, out, NULL)  # noqa: E731
    assert norm(m=-1.0) == INVALID
    assert norm(m=NAN) == INVALID
    assert norm(out=NULL) == INVALID
    assert norm(out=ODD2) == ALIGNMENT
    assert norm(T.AdamWPlanStruct(0x10001, 4, 0, 0, 0, 0)) == INVALID
    assert L.lora_grad_norm(None, 1.0, FAKE, NULL) == INVALID


def test_python_binding_refuses_what_it_cannot_pass_on():
    x, lab = torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        T.lora_token_logps(x, lab, torch.zeros(3))
    with pytest.raises(ValueError, match="T, V"):
        T.lora_token_logps(x[0], lab, torch.zeros(3))
    with pytest.raises(ValueError, match="GPU"):
        T.lora_adamw_plan([x], [x], [x], [x])
    with pytest.raises(ValueError, match="one tensor"):
        T.lora_adamw_plan([x], [], [x], [x])
    with pytest.raises(ValueError, match="both"):
        T.lora_adamw_plan([x], [x], [x], [x], exp_avg_scales=[x])
    assert T._dense(torch.zeros(4, 6).t()) and T._dense(torch.zeros(4, 1, 6)) and T._dense(torch.zeros(3, 4, 5).transpose(0, 2))
    assert not T._dense(torch.zeros(4, 6)[:, :5]) and not T._dense(torch.zeros(1, 6).expand(4, 6))

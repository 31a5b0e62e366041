"""lora_top_logps, its gradient and lora_distill_loss on the host: bad arguments are refused before
anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from lora_rank_adapter_gb300 import training as T
from tests.test_other_gpu_host import Far, gpus  # noqa: F401
from tests.test_training_host import ALIGNMENT, FAKE, INF, INVALID, NAN, NULL, ODD1, ODD2, OK, UNSUPPORTED

FAR = ctypes.c_void_p(0x20000)
ROWS = {"dt": 1, "T": 6, "V": 33, "K": 4, "x": FAKE, "ld": 33, "temp": 1.0}


@pytest.fixture(scope="module")
def L():
    _build.build()
    return T.lib()


def top(L, lab=FAKE, lp=FAKE, H=NULL, ids=FAKE, out=FAKE, rest=NULL, stats=NULL, **k):
    k = {**ROWS, **k}
    return L.lora_top_logps(k["dt"], k["T"], k["V"], k["K"], k["x"], k["ld"], lab, k["temp"], lp, H, ids, out, rest, stats,
                            NULL)


def back(L, lab=FAKE, ids=FAKE, stats=FAKE, H=FAKE, gl=FAKE, gh=FAKE, gt=FAKE, d=FAR, ldd=33, **k):
    k = {**ROWS, **k}
    return L.lora_top_logps_backward(k["dt"], k["T"], k["V"], k["K"], k["x"], k["ld"], lab, ids, k["temp"], stats, H, gl, gh,
                                     gt, d, ldd, NULL)


def distill(L, ids=FAKE, q=FAKE, rest=NULL, w=NULL, kind=0, row=FAR, loss=ctypes.c_void_p(0x30000), d=NULL, ldd=0, gs=1.0, **k):
    k = {**ROWS, **k}
    return L.lora_distill_loss(k["dt"], k["T"], k["V"], k["K"], k["x"], k["ld"], ids, q, rest, w, kind, k["temp"], row,
                               loss, d, ldd, gs, NULL)


@pytest.mark.parametrize("change,status", [
    ({"dt": 5}, UNSUPPORTED), ({"T": -1}, INVALID), ({"V": -1}, INVALID), ({"T": 1 << 31}, INVALID), ({"x": NULL}, INVALID),
    ({"x": ODD1}, ALIGNMENT), ({"dt": 0, "x": ODD2}, ALIGNMENT), ({"ld": 32}, INVALID), ({"temp": 0.0}, INVALID),
    ({"temp": -1.0}, INVALID), ({"temp": NAN}, INVALID), ({"temp": INF}, INVALID), ({"temp": 1e-39}, INVALID),
    ({"V": (1 << 30) + 1, "ld": 1 << 31}, UNSUPPORTED), ({"K": -1}, INVALID), ({"K": 129}, UNSUPPORTED),
    ({"ids": ctypes.c_void_p(0x10004)}, ALIGNMENT)])
def test_rows_and_lists_are_checked(L, change, status):
    for call in (top, back, distill):
        assert call(L, **change) == status, call.__name__


def test_top_arguments(L):
    for change, status in [({"lab": NULL}, INVALID), ({"lp": NULL}, INVALID), ({"ids": NULL}, INVALID), ({"out": NULL}, INVALID),
                           ({"lab": ODD2}, ALIGNMENT), ({"lp": ODD2}, ALIGNMENT), ({"H": ODD2}, ALIGNMENT),
                           ({"out": ODD2}, ALIGNMENT), ({"rest": ODD2}, ALIGNMENT),
                           ({"stats": ctypes.c_void_p(0x10004)}, ALIGNMENT)]:
        assert top(L, **change) == status, change
    assert top(L, T=0, x=NULL, lab=NULL, lp=NULL, ids=NULL, out=NULL) == OK


def test_backward_arguments(L):
    for change, status in [({"d": NULL}, INVALID), ({"stats": NULL}, INVALID), ({"lab": NULL}, INVALID), ({"H": NULL}, INVALID),
                           ({"ids": NULL}, INVALID), ({"ldd": 32}, INVALID), ({"d": ODD1}, ALIGNMENT),
                           ({"d": FAKE, "ldd": 40}, INVALID),      # in place needs the logits' own stride
                           ({"gl": ODD2}, ALIGNMENT), ({"gh": ODD2}, ALIGNMENT), ({"gt": ODD2}, ALIGNMENT),
                           ({"H": ODD2}, ALIGNMENT), ({"stats": ctypes.c_void_p(0x10004)}, ALIGNMENT)]:
        assert back(L, **change) == status, change
    assert back(L, T=0, x=NULL, lab=NULL, ids=NULL, stats=NULL, H=NULL, gl=NULL, gh=NULL, gt=NULL, d=NULL) == OK


def test_distill_arguments(L):
    for change, status in [({"K": 0}, INVALID), ({"kind": 2}, UNSUPPORTED), ({"ids": NULL}, INVALID), ({"q": NULL}, INVALID),
                           ({"row": NULL}, INVALID), ({"loss": NULL}, INVALID), ({"q": ODD2}, ALIGNMENT),
                           ({"rest": ODD2}, ALIGNMENT), ({"w": ODD2}, ALIGNMENT), ({"row": ODD2}, ALIGNMENT),
                           ({"loss": ODD2}, ALIGNMENT), ({"gs": NAN}, INVALID), ({"gs": INF}, INVALID),
                           ({"d": FAR, "ldd": 5}, INVALID), ({"d": FAKE, "ldd": 40}, INVALID), ({"d": ODD1, "ldd": 33}, ALIGNMENT),
                           ({"row": FAKE, "w": FAKE}, INVALID), ({"loss": FAR}, INVALID), ({"row": FAKE, "q": FAKE}, INVALID),
                           ({"row": FAR, "rest": FAR}, INVALID)]:
        assert distill(L, **change) == status, change


def test_row_losses_share_no_place_with_what_is_read(L):
    """Parts of the rows' losses (24 bytes from FAR on) within an input or around the loss."""
    far = FAR.value
    at = lambda offset: ctypes.c_void_p(far + offset)  # noqa: E731
    for name, size in (("ids", 6 * 4 * 8), ("q", 6 * 4 * 4), ("rest", 24), ("w", 24), ("loss", 4)):
        for offset in (8 - size, 16):
            assert distill(L, **{name: at(offset)}) == INVALID, (name, offset)


def test_binding_refuses_tensors_that_do_not_belong(gpus):
    """What the binding itself refuses, by tensors that only say where they are."""
    _, calls = gpus
    x, v, m, ids = Far(6, 40), Far(6), Far(6, 4), Far(6, 4, dtype=torch.int64)
    lab = Far(6, dtype=torch.int64)
    for bad in (lambda: T.lora_top_logps(x, ids, m, labels=lab), lambda: T.lora_top_logps(x, ids, m, logps=v),
                lambda: T.lora_top_logps(x, Far(24, dtype=torch.int64), m),
                lambda: T.lora_top_logps_backward(x, Far(6, 2), None),
                lambda: T.lora_top_logps_backward(x, Far(6, 2), x, dlogps=v),
                lambda: T.lora_top_logps_backward(x, Far(6, 2), x, dentropy=v),
                lambda: T.lora_top_logps_backward(x, Far(6, 2), x, dtop_logps=m),
                lambda: T.lora_distill_loss(x, ids, m, v, Far(1), kind="both"),
                lambda: T.lora_distill_loss(x, Far(24, dtype=torch.int64), m, v, Far(1))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: T.lora_top_logps(x, Far(6, 4), m), lambda: T.lora_top_logps(x, ids, Far(6, 5)),
                lambda: T.lora_top_logps(x, ids, m, entropy=Far(5)), lambda: T.lora_top_logps(x, ids, m, stats=v),
                lambda: T.lora_distill_loss(x, ids, Far(5, 4), v, Far(1)),
                lambda: T.lora_distill_loss(x, ids, m, v, Far(1), dlogits=Far(6, 41)),
                lambda: T.lora_distill_loss(x, ids, m, v, Far(1), weights=Far(6, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            bad()
    assert calls == []


def test_calls_run_on_their_tensors_gpu(gpus):
    state, calls = gpus
    x, v, m, ids, lab = Far(6, 40), Far(6), Far(6, 4), Far(6, 4, dtype=torch.int64), Far(6, dtype=torch.int64)
    T.lora_top_logps(x, ids, m, labels=lab, logps=v, entropy=v, rest_logps=v, stats=Far(6, 2))
    T.lora_top_logps_backward(x, Far(6, 2), x, labels=lab, top_ids=ids, entropy=v, dlogps=v, dentropy=v, dtop_logps=m)
    T.lora_distill_loss(x, ids, m, v, Far(1), rest_logps=v, weights=v, dlogits=x, kind="reverse")
    assert [c[0] for c in calls] == ["lora_top_logps", "lora_top_logps_backward", "lora_distill_loss"]
    assert all(c[1] == 1 and c[2] == 0x501 for c in calls) and state["current"] == 0

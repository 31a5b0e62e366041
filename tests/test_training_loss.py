"""The loss operators against plain implementations in 64 bits: log-probabilities of
labels, preference loss and clipped policy loss, with their gradients.

Tolerances.  logp = (x - m)/temp - ln S in fp32: the product and the logarithm are
rounded to 2^-24 of values up to about |logp| + 12, the terms of S have a relative
error near 2^-22 (the exponential) and S is summed in a tree, so |error| <=
4e-6 max(1, |logp|).  A probability has the relative error of its exponential and of
S, below 4e-6, so an element of dlogits in row t is off by at most 4e-6 |c_t| for the
exact coefficient c_t, plus what c_t itself is off by, plus one rounding (2^-9
relative, 2^-8 allowed) in bf16."""
import math

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from lora_rank_adapter_gb300 import training

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 4e-6
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)


def make(T, V, dtype, seed=0, pad=0, first=0, ignored=0.2):
    """Logits inside a wider buffer of sentinels (first columns before, pad after), labels, some of them ignored."""
    g = torch.Generator().manual_seed(seed)
    full = torch.full((T, first + V + pad), 77.0)
    full[:, first:first + V] = torch.randn(T, V, generator=g) * 3
    full = full.to(dtype).to(DEV)
    labels = torch.randint(0, V, (T,), generator=g)
    labels[torch.rand(T, generator=g) < ignored] = -100
    return full, full[:, first:first + V], labels.to(DEV)


def oracle_logps(x, labels, temp=1.0):
    """(logp, p, ok) in 64 bits on the CPU."""
    z = x.double().cpu() / temp
    if x.shape[1]:
        z = z - z.amax(1, keepdim=True)      # exact; a huge common part would swallow ln V
    lab = labels.cpu()
    ok = (lab >= 0) & (lab < x.shape[1])
    rows = torch.arange(len(lab))
    lse = torch.logsumexp(z, 1) if x.shape[1] else torch.zeros(len(lab))
    logp = torch.zeros(len(lab), dtype=torch.float64)
    logp[ok] = (z[rows, lab.clamp(0, max(0, x.shape[1] - 1))] - lse)[ok]
    p = (z - lse[:, None]).exp()
    return logp, p, ok


def oracle_dlogits(p, labels, ok, coef, temp=1.0):
    d = -p * coef[:, None] / temp
    rows = torch.arange(len(ok))[ok]
    d[rows, labels.cpu()[ok]] += coef[ok] / temp
    d[~ok] = 0
    return d


def check_logps(got, want):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= EPS * want.abs().clamp(min=1)).all()), float(err.max())


def check_dlogits(got, want, coef, slack, temp=1.0):
    """slack: what each row's coefficient may be off by."""
    rounding = 2.0 ** -8 * want.abs() if got.dtype == BF16 else 0.0
    err = (got.double().cpu() - want).abs()
    bound = ((EPS * coef.abs() + slack) / temp)[:, None] + rounding + 1e-30
    assert bool((err <= bound).all()), float((err / bound).max())


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 255), (7, 1001), (2, 2049), (3, 8192), (2, 32003), (1, 128256)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", SIZES)
def test_token_logps_and_gradient(T, V, dtype):
    for pad, first, temp in ((0, 0, 1.0), (3, 1, 0.7), (8, 8, 1.6)):
        full, x, labels = make(T, V, dtype, seed=V, pad=pad, first=first)
        logps = torch.full((T,), 5.0, device=DEV)
        stats = torch.empty((T, 2), device=DEV)
        training.lora_token_logps(x, labels, logps, temperature=temp, stats=stats)
        want, p, ok = oracle_logps(x, labels, temp)
        check_logps(logps, want)
        coef = torch.randn(T, generator=torch.Generator().manual_seed(1))
        out = torch.full_like(full, 55.0)
        d = out[:, first:first + V]
        training.lora_token_logps_backward(x, labels, stats, coef.to(DEV), d, temperature=temp)
        check_dlogits(d, oracle_dlogits(p, labels, ok, coef.double(), temp), coef.double(), 0.0, temp)
        assert bool((out[:, :first] == 55).all()) and bool((out[:, first + V:] == 55).all())
        # other alignment of the gradient than of the logits, then in place
        other = torch.full((T, V + 5), 55.0, dtype=dtype, device=DEV)
        training.lora_token_logps_backward(x, labels, stats, coef.to(DEV), other[:, 3:3 + V], temperature=temp)
        assert torch.equal(other[:, 3:3 + V], d) and bool((other[:, :3] == 55).all())
        assert bool((other[:, 3 + V:] == 55).all())
        training.lora_token_logps_backward(x, labels, stats, coef.to(DEV), x, temperature=temp)
        assert torch.equal(x, d)
        assert bool((full[:, :first] == 77).all()) and bool((full[:, first + V:] == 77).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 4099, 70000])
def test_rows_with_masks_infinities_and_nan(V, dtype):
    _, x, labels = make(12, V, dtype, seed=3, ignored=0.0)
    low, inf, nan = torch.finfo(dtype).min, math.inf, math.nan
    labels[:] = torch.arange(12, device=DEV) % 5
    x[0, 5:] = -inf                 # most of the row masked out
    x[1, 5:] = low
    x[2, :] = low                   # nothing left, by the lowest value: uniform
    x[3, :] = -inf                  # nothing left, by minus infinity: NaN, as 0 / 0
    x[4, 7] = inf
    x[5, 7] = nan
    x[6, int(labels[6])] = -inf     # the label itself masked: logp -inf
    x[7, :] = nan
    labels[7] = -100                # not looked at
    x[8, :] = inf
    labels[8] = V
    x[9, :-1] = -inf                # one column left, and it is the label
    labels[9] = V - 1
    x[10, :] = torch.finfo(dtype).max      # equal and huge: uniform
    want, p, ok = oracle_logps(x, labels)
    logps, stats = torch.empty(12, device=DEV), torch.empty((12, 2), device=DEV)
    training.lora_token_logps(x, labels, logps, stats=stats)
    got = logps.double().cpu()
    for t in (3, 4, 5):
        assert math.isnan(got[t]), t
    assert got[6] == -inf and got[7] == 0 and got[8] == 0 and got[9] == 0
    fine = torch.tensor([0, 1, 2, 9, 10, 11])
    check_logps(logps[fine.to(DEV)], want[fine])
    assert abs(got[2] + math.log(V)) < 1e-5 and abs(got[10] + math.log(V)) < 1e-5
    for in_place in (False, True):
        d = x if in_place else torch.empty_like(x)
        one = torch.ones(12, device=DEV)
        training.lora_token_logps_backward(x, labels, stats, one, d)
        assert bool((d[7] == 0).all()) and bool((d[8] == 0).all())
        for t in (3, 4, 5):
            assert bool(d[t].isnan().any()), t
        rows = torch.tensor([0, 1, 2, 6, 9, 10, 11])
        check_dlogits(d[rows.to(DEV)], oracle_dlogits(p, labels, ok, torch.ones(12, dtype=torch.float64))[rows],
                      torch.ones(7, dtype=torch.float64), 0.0)


def run_preference(x, labels, cu, ref, beta=0.2, **k):
    T, P = x.shape[0], len(cu) // 2
    out = {"tok": torch.full((T,), 9.0, device=DEV), "seq": torch.full((2 * P,), 9.0, device=DEV),
           "pair": torch.full((P,), 9.0, device=DEV), "loss": torch.full((1,), 9.0, device=DEV)}
    d, grad = k.pop("d", None), k.pop("grad", True)
    if d is None and grad:
        d = torch.full(x.shape, 3.0, dtype=x.dtype, device=DEV)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    training.lora_preference_loss(x, labels, cu, None if ref is None else ref.to(DEV), beta, out["tok"], out["seq"],
                                  out["pair"], out["loss"], dlogits=d, **k)
    out["d"] = d
    return out


def oracle_preference(x, labels, cu, ref, beta=0.2, kind="sigmoid", label_smoothing=0.0, length_normalize=False,
                      temperature=1.0, grad_scale=1.0):
    logp, p, ok = oracle_logps(x, labels, temperature)
    T, P = len(logp), len(cu) // 2
    z = logp.clone().requires_grad_(True)
    S, off = [], []
    for i in range(2 * P):
        lo, hi = min(max(cu[i], 0), T), min(max(cu[i + 1], 0), T)
        n = max(1, int(ok[lo:hi].sum())) if length_normalize else 1
        S.append(z[lo:hi][ok[lo:hi]].sum() / n if hi > lo else z.sum() * 0)
        off.append(float((EPS * logp[lo:hi].abs().clamp(min=1) * ok[lo:hi]).sum()) / n + 2e-7 * abs(float(S[-1].detach())))
    pair, coef_off = [], torch.zeros(T, dtype=torch.float64)
    for i in range(P):
        d = S[i] - S[P + i] - (0 if ref is None else float(ref[i]) - float(ref[P + i]))
        delta = off[i] + off[P + i] + 1e-6 * (abs(float(d.detach())) + 1)
        if kind == "sigmoid":
            h = beta * d
            pair.append(-(1 - label_smoothing) * torch.nn.functional.logsigmoid(h)
                        - label_smoothing * torch.nn.functional.logsigmoid(-h))
            curve = beta * beta / 4
        elif kind == "hinge":
            pair.append(torch.clamp(1 - beta * d, min=0))
            curve = 0.0
        else:
            pair.append((d - 1 / (2 * beta)) ** 2)
            curve = 2.0
        for j in (i, P + i):
            lo, hi = min(max(cu[j], 0), T), min(max(cu[j + 1], 0), T)
            n = max(1, int(ok[lo:hi].sum())) if length_normalize else 1
            coef_off[lo:hi] = curve * delta / P / n
    loss = torch.stack(pair).mean() if P else z.sum() * 0
    (coef,) = torch.autograd.grad(loss, z)
    coef = coef * grad_scale
    return {"logp": logp, "seq": torch.tensor([float(v.detach()) for v in S], dtype=torch.float64), "off": torch.tensor(off),
            "pair": torch.tensor([float(v.detach()) for v in pair], dtype=torch.float64), "loss": float(loss.detach()), "coef": coef,
            "coef_off": coef_off * abs(grad_scale) + 2e-6 * coef.abs(),
            "d": oracle_dlogits(p, labels, ok, coef, temperature), "temp": temperature}


def check_preference(got, want):
    check_logps(got["tok"], want["logp"])
    assert bool(((got["seq"].double().cpu() - want["seq"]).abs() <= want["off"] + 1e-7).all())
    P = len(want["pair"])
    scale = 1 + want["pair"].abs()
    slope = 1.0 + 4 * want["pair"].abs().sqrt()          # at most |dl/dd| for every kind at these beta
    tol = slope * (want["off"][:P] + want["off"][P:] + 2e-6 * (1 + want["seq"].abs().max() if P else 0)) + 1e-6 * scale
    assert bool(((got["pair"].double().cpu() - want["pair"]).abs() <= tol).all())
    assert abs(float(got["loss"]) - want["loss"]) <= (float(tol.max()) if P else 0.0)
    if got["d"] is not None:
        check_dlogits(got["d"], want["d"], want["coef"], want["coef_off"], want["temp"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,opts", [("sigmoid", {}), ("sigmoid", {"label_smoothing": 0.2, "temperature": 0.8}),
                                       ("hinge", {"grad_scale": 0.25, "label_smoothing": 0.1}), ("ipo", {"length_normalize": True}),
                                       ("sigmoid", {"length_normalize": True, "temperature": 1.4})])
def test_preference_loss(kind, opts, dtype):
    for V, cu, pad in ((61, [0, 4, 9, 9, 16], 0), (1003, [0, 30, 31], 1), (8200, [0, 1, 2, 3, 4, 5, 20], 8)):
        T = cu[-1] + 3               # three rows in no sequence
        full, x, labels = make(T, V, dtype, seed=V, pad=pad)
        ref = torch.randn(len(cu) - 1, generator=torch.Generator().manual_seed(2)) * 2
        if kind == "ipo":            # the target 1 / (2 beta) apart
            ref = ref * 0.1
        for r in (ref, None):
            got = run_preference(x, labels, cu, r, kind=kind, **opts)
            check_preference(got, oracle_preference(x, labels, cu, r, kind=kind, **opts))
        assert bool((got["d"][cu[-1]:] == 0).all())
        again = run_preference(x, labels, cu, r, kind=kind, **opts)
        for k in got:
            assert torch.equal(got[k], again[k]), k
        forward = run_preference(x, labels, cu, r, kind=kind, grad=False, **opts)
        for k in ("tok", "seq", "pair", "loss"):
            assert torch.equal(got[k], forward[k]), k
        copy = full.clone()[:, :V]
        placed = run_preference(copy, labels, cu, r, kind=kind, d=copy, **opts)
        assert torch.equal(placed["d"], got["d"])


def test_preference_loss_of_empty_and_ignored_sequences():
    _, x, labels = make(10, 50, F32, seed=1, ignored=0.0)
    labels[4:8] = -1                                    # pair 1's chosen sequence is ignored whole
    cu = [0, 4, 8, 10, 10]                              # and its rejected one is empty
    got = run_preference(x, labels, cu, None, length_normalize=True)
    check_preference(got, oracle_preference(x, labels, cu, None, length_normalize=True))
    assert float(got["seq"][1]) == 0 and float(got["seq"][3]) == 0
    assert abs(float(got["pair"][1]) - math.log(2)) < 1e-6
    assert bool((got["d"][4:8] == 0).all())
    # no pair, no row, offsets past the end
    got = run_preference(x, labels, [0], None)
    assert float(got["loss"]) == 0 and bool((got["d"] == 0).all())
    got = run_preference(x[:0], labels[:0], [0, 0, 0], None)
    assert abs(float(got["loss"]) - math.log(2)) < 1e-6
    cu = [-5, 4, 99]
    check_preference(run_preference(x, labels, cu, None), oracle_preference(x, labels, cu, None))


def run_policy(x, labels, old, adv, w, ref=None, d=None, grad=True, **k):
    T = x.shape[0]
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out = {"tok": torch.full((T,), 9.0, device=DEV), "metrics": torch.full((3,), 9.0, device=DEV)}
    if d is None and grad:
        d = torch.full(x.shape, 3.0, dtype=x.dtype, device=DEV)
    training.lora_policy_loss(x, labels, dev(old), dev(adv), dev(w), out["tok"], out["metrics"], ref_logps=dev(ref),
                              dlogits=d, **k)
    out["d"] = d
    return out


def check_policy(got, x, labels, old, adv, w, ref, clip_low=0.2, clip_high=0.2, kl_beta=0.0, temperature=1.0,
                 grad_scale=1.0):
    logp, p, ok = oracle_logps(x, labels, temperature)
    check_logps(got["tok"], logp)
    T = len(logp)
    adv = adv.double()
    weight = torch.where(ok, torch.ones(T, dtype=torch.float64) if w is None else w.double(), 0.0)
    ratio = (logp - (logp if old is None else old.double())).exp()
    lo, hi = 1 - clip_low, 1 + clip_high
    pg = -torch.minimum(ratio * adv, ratio.clamp(lo, hi) * adv)
    clipped = ((adv > 0) & (ratio > hi)) | ((adv < 0) & (ratio < lo))
    coef = torch.where(clipped, 0.0, -adv * ratio)
    gap = torch.zeros(T, dtype=torch.float64) if ref is None else ref.double() - logp
    kl = torch.expm1(gap) - gap
    coef = (coef - kl_beta * torch.expm1(gap)) * weight * grad_scale
    coef = torch.where(ok, coef, 0.0)
    off = EPS * logp.abs().clamp(min=1) + 1e-6           # logp, and the exponentials' own rounding
    slack = weight.abs() * (adv.abs() * ratio + kl_beta * gap.exp()) * off * abs(grad_scale)
    tol = float((weight.abs() * (adv.abs() * ratio + (kl_beta + 1) * (gap.exp() + 1 + gap.abs())) * off).sum()) + 1e-6
    want = [float((weight * (pg + kl_beta * kl)).sum()), float((weight * kl).sum()), float((weight * clipped).sum())]
    for i in range(3):
        assert abs(float(got["metrics"][i]) - want[i]) <= tol + 1e-6 * abs(want[i]), (i, float(got["metrics"][i]), want)
    if got["d"] is not None:
        check_dlogits(got["d"], oracle_dlogits(p, labels, ok, coef, temperature), coef, slack + 2e-6 * coef.abs(),
                      temperature)


def policy_inputs(x, labels, seed, temperature=1.0, spread=0.4, bounds=(0.8, 1.2)):
    g = torch.Generator().manual_seed(seed)
    T = x.shape[0]
    logp, _, _ = oracle_logps(x, labels, temperature)
    r = torch.exp(spread * torch.randn(T, generator=g, dtype=torch.float64))
    for b in bounds:                 # off the clip bounds, where the gradient jumps
        r = torch.where((r - b).abs() < 1e-3, r * 0.99, r)
    return ((logp - r.log()).float(), torch.randn(T, generator=g), torch.rand(T, generator=g),
            (logp + 0.3 * torch.randn(T, generator=g, dtype=torch.float64)).float())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,pad", [(1, 1, 0), (9, 63, 0), (40, 1025, 3), (6, 32003, 0), (17, 8192, 8),
                                     (300, 515, 0), (3, 128256, 0), (2, 250001, 0)])
def test_policy_loss(T, V, pad, dtype):
    for temp in (1.0, 0.8):
        full, x, labels = make(T, V, dtype, seed=T, pad=pad)
        old, adv, w, ref = policy_inputs(x, labels, T, temp)
        for k in (dict(), dict(ref=ref, kl_beta=0.1), dict(grad_scale=-2.0)):
            ref_k = k.pop("ref", None)
            got = run_policy(x, labels, old, adv, w, ref=ref_k, temperature=temp, **k)
            check_policy(got, x, labels, old, adv, w, ref_k, temperature=temp, **k)
        again = run_policy(x, labels, old, adv, w, temperature=temp, grad_scale=-2.0)
        for n in got:
            assert torch.equal(got[n], again[n]), n
        forward = run_policy(x, labels, old, adv, w, grad=False, temperature=temp)
        for n in ("tok", "metrics"):
            assert torch.equal(got[n], forward[n]), n
        copy = full.clone()[:, :V]
        placed = run_policy(copy, labels, old, adv, w, d=copy, temperature=temp, grad_scale=-2.0)
        assert torch.equal(placed["d"], got["d"])


@pytest.mark.parametrize("dtype,V", [(BF16, 17001), (F32, 9004), (BF16, 600), (F32, 60001)])
@pytest.mark.parametrize("T", [33, 76, 100, 152, 200, 310, 700])
def test_every_cut_of_the_rows(T, V, dtype):
    """Row counts and sizes on both sides of every rule by which rows are cut over blocks."""
    _, x, labels = make(T, V, dtype, seed=T, pad=1)
    logps, stats = torch.empty(T, device=DEV), torch.empty((T, 2), device=DEV)
    training.lora_token_logps(x, labels, logps, stats=stats)
    want, p, ok = oracle_logps(x, labels)
    check_logps(logps, want)
    coef = torch.randn(T, generator=torch.Generator().manual_seed(3))
    d = torch.empty_like(x)
    training.lora_token_logps_backward(x, labels, stats, coef.to(DEV), d)
    check_dlogits(d, oracle_dlogits(p, labels, ok, coef.double()), coef.double(), 0.0)
    old, adv, w, ref = policy_inputs(x, labels, T)
    check_policy(run_policy(x, labels, old, adv, w, ref=ref, kl_beta=0.1), x, labels, old, adv, w, ref, kl_beta=0.1)
    cu = [0, T // 5, T // 2, T // 2, T - 1]
    check_preference(run_preference(x, labels, cu, None), oracle_preference(x, labels, cu, None))


def test_policy_loss_defaults_and_ignored_rows():
    _, x, labels = make(70, 500, F32, seed=8, ignored=0.5)
    old, adv, w, ref = policy_inputs(x, labels, 1)
    got = run_policy(x, labels, None, adv, None)
    check_policy(got, x, labels, None, adv, None, None)
    x[labels < 0] = math.nan          # ignored rows are not read, their other values neither used
    clean = run_policy(x, labels, old, adv, w, ref=ref, kl_beta=0.2)
    for t in (old, adv, w, ref):
        t[(labels < 0).cpu()] = math.nan
    dirty = run_policy(x, labels, old, adv, w, ref=ref, kl_beta=0.2)
    for k in clean:
        assert torch.equal(clean[k], dirty[k]), k
    assert bool((dirty["d"][labels < 0] == 0).all())
    labels[:] = -1
    got = run_policy(x, labels, old, adv, w)
    assert bool((got["metrics"] == 0).all()) and bool((got["d"] == 0).all()) and bool((got["tok"] == 0).all())
    empty = run_policy(x[:0], labels[:0], old[:0], adv[:0], w[:0])
    assert bool((empty["metrics"] == 0).all())


@pytest.mark.parametrize("op", ["preference", "policy"])
def test_gradient_against_differences(op):
    """Central differences of the loss along random directions, in fp32: the loss has an
    error of some 1e-6, the step is 2e-2 in each of V logits of unit-norm directions."""
    T, V, cu = 12, 40, [0, 2, 6, 9, 12]
    _, x, labels = make(T, V, F32, seed=4, ignored=0.1)
    old, adv, w, ref = policy_inputs(x, labels, 3, spread=0.05)
    seq_ref = torch.tensor([-20.0, -30.0, -25.0, -24.0])

    def loss(z, d=None):
        if op == "preference":
            got = run_preference(z, labels, cu, seq_ref, beta=0.1, label_smoothing=0.1, grad=False, d=d)
            return float(got["loss"])
        return float(run_policy(z, labels, old, adv, w, ref=ref, kl_beta=0.3, d=d, grad=False)["metrics"][0])

    d = torch.empty_like(x)
    loss(x, d)
    g = torch.Generator().manual_seed(5)
    h = 2e-2
    for _ in range(6):
        u = torch.randn(T, V, generator=g)
        u = (u / u.norm()).to(DEV)
        step = h * math.sqrt(T)
        slope = (loss(x + step * u) - loss(x - step * u)) / (2 * step)
        want = float((d.double() * u.double()).sum())
        assert abs(slope - want) <= 2e-3 * float(d.norm()) + 4e-5, (slope, want)


def test_many_short_rows_and_labels_out_of_range():
    """More rows than any grid holds at once; labels far outside the vocabulary."""
    T, V = 70001, 5
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, V, generator=g).to(DEV)
    labels = torch.randint(-3, 9, (T,), generator=g)
    labels[::1000] = 2 ** 40
    labels[1::1000] = -2 ** 40
    labels[2::1000] = 2 ** 32 + 1              # its low 32 bits are a valid label
    labels = labels.to(DEV)
    logps, stats = torch.empty(T, device=DEV), torch.empty((T, 2), device=DEV)
    training.lora_token_logps(x, labels, logps, stats=stats)
    want, p, ok = oracle_logps(x, labels)
    check_logps(logps, want)
    assert bool((logps[(~ok).to(DEV)] == 0).all())
    d = torch.empty_like(x)
    one = torch.ones(T, device=DEV)
    training.lora_token_logps_backward(x, labels, stats, one, d)
    check_dlogits(d, oracle_dlogits(p, labels, ok, torch.ones(T, dtype=torch.float64)), torch.ones(T, dtype=torch.float64), 0.0)
    for shape in ((T, V), (40, 9001)):         # the same labels where a row takes a block or a cluster
        lab = torch.full((shape[0],), 2 ** 32 + 1, device=DEV)
        out = run_policy(torch.randn(shape, device=DEV), lab, None, torch.ones(shape[0]), None)
        assert bool((out["d"] == 0).all()) and bool((out["metrics"] == 0).all())


def test_preference_with_an_impossible_answer():
    """A label that is masked out has log-probability minus infinity: as the rejected
    sequence's it leaves loss 0 and no slope, as the chosen one's an infinite loss."""
    _, x, labels = make(8, 60, F32, seed=2, ignored=0.0)
    x[6, int(labels[6])] = -math.inf
    got = run_preference(x, labels, [0, 4, 8], None)
    assert float(got["loss"]) == 0 and float(got["seq"][1]) == -math.inf
    assert bool((got["d"] == 0).all())
    x[2, int(labels[2])], x[6, int(labels[6])] = -math.inf, 0.0
    got = run_preference(x, labels, [0, 4, 8], None)
    assert float(got["loss"]) == math.inf and bool(got["d"].isfinite().all())


def test_in_a_graph():
    """Captured once and replayed on new values: no host sync, no state left behind."""
    _, x, labels = make(40, 3001, BF16, seed=5)
    old, adv, w, _ = policy_inputs(x, labels, 2)
    old, adv, w = old.to(DEV), adv.to(DEV), w.to(DEV)
    cu = torch.tensor([0, 10, 25, 30, 40], dtype=torch.int32, device=DEV)
    tok, met, d = torch.empty(40, device=DEV), torch.empty(3, device=DEV), torch.empty_like(x)
    tok2, seq, pair, loss = (torch.empty(n, device=DEV) for n in (40, 4, 2, 1))
    d2, p = torch.empty_like(x), x.float()
    m, v, norm = torch.zeros_like(p), torch.zeros_like(p), torch.empty(2, device=DEV)
    plan = training.lora_adamw_plan([p], [d], [m], [v])

    def step():
        training.lora_policy_loss(x, labels, old, adv, w, tok, met, dlogits=d)
        training.lora_preference_loss(x, labels, cu, None, 0.1, tok2, seq, pair, loss, dlogits=d2)
        training.lora_grad_norm(plan, 0.1, norm)
        training.lora_adamw(plan, lr=1e-2, step=1, grad_factor=norm[1:])

    outs = (tok, met, d, tok2, seq, pair, loss, d2, p, m, v, norm)
    start = [t.clone() for t in outs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        for t, b in zip(outs, start):
            t.copy_(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        s.synchronize()
        for change in (1.0, 0.5):
            for t, b in zip(outs, start):
                t.copy_(b)
            x.mul_(change)
            step()
            s.synchronize()
            want = [t.clone() for t in outs]
            for t, b in zip(outs, start):
                t.copy_(b)
            graph.replay()
            s.synchronize()
            for t, b in zip(outs, want):
                assert torch.equal(t, b)


def test_offsets_past_32_bits():
    """Rows 2^30 + 8 elements apart: element offsets and byte offsets pass 32 bits."""
    ld, V, T = (1 << 30) + 8, 1000, 4
    _, small, labels = make(T, V, BF16, seed=6, ignored=0.0)
    flat = torch.empty(3 * ld + V, dtype=BF16, device=DEV)
    x = torch.as_strided(flat, (T, V), (ld, 1))
    x.copy_(small)
    old, adv, w, _ = policy_inputs(small, labels, 2)
    want = run_policy(small, labels, old, adv, w)
    got = run_policy(x, labels, old, adv, w, d=x)
    for k in ("tok", "metrics", "d"):
        assert torch.equal(got[k], want[k]), k
    x.copy_(small)
    got = run_preference(x, labels, [0, 2, 4], None, d=x)
    want = run_preference(small, labels, [0, 2, 4], None)
    assert torch.equal(got["d"], want["d"]) and torch.equal(got["loss"], want["loss"])


def test_on_another_stream():
    _, x, labels = make(200, 5000, BF16, seed=7)
    old, adv, w, _ = policy_inputs(x, labels, 2)
    want = run_policy(x, labels, old, adv, w)
    want_p = run_preference(x, labels, [0, 90, 200], None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, got_p = [], []
    with torch.cuda.stream(s):
        for _ in range(3):
            got.append(run_policy(x, labels, old, adv, w))
            got_p.append(run_preference(x, labels, [0, 90, 200], None))
    s.synchronize()
    for a, b in zip(got, got_p):
        assert all(torch.equal(a[k], want[k]) for k in want)
        assert all(torch.equal(b[k], want_p[k]) for k in want_p)
    # a stream by argument
    logps = torch.empty(200, device=DEV)
    pair, seq, loss = torch.empty(1, device=DEV), torch.empty(2, device=DEV), torch.empty(1, device=DEV)
    cu = torch.tensor([0, 90, 200], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for _ in range(5):
        # the current stream keeps the block that the call's workspace must not be busy
        busy = torch.empty(1 << 26, device=DEV)
        for _ in range(20):
            busy.mul_(1.0001)
        junk = torch.full((8192,), 7, dtype=torch.uint8, device=DEV)
        del junk
        loss.zero_()
        s.wait_stream(torch.cuda.current_stream())
        training.lora_preference_loss(x, labels, cu, None, 0.2, logps, seq, pair, loss, stream=s)
        s.synchronize()
        assert torch.equal(loss, want_p["loss"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_gradient(dtype):
    for T, V, pad, first in ((1, 1, 0, 0), (5, 1003, 2, 1), (3, 4096, 8, 0)):
        full, x, _ = make(T, V, dtype, seed=9, pad=pad, first=first)
        want = (x.float() * 0.3).to(dtype)
        same = x.clone()
        training.lora_scale_gradient(x, torch.ones(1, device=DEV))
        assert torch.equal(x, same)
        training.lora_scale_gradient(x, torch.full((1,), 0.3, device=DEV))
        assert torch.equal(x, want)
        assert bool((full[:, :first] == 77).all()) and bool((full[:, first + V:] == 77).all())


def test_refusals():
    _, x, labels = make(4, 8, BF16)
    logps = torch.empty(4, device=DEV)
    for bad in (dict(logits=x.half()), dict(logits=x.t()), dict(labels=labels.int()), dict(labels=labels[:3]),
                dict(logps=logps.double()), dict(logps=torch.empty(4)), dict(temperature=0.0),
                dict(stats=torch.empty(4, device=DEV))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            training.lora_token_logps(**{**dict(logits=x, labels=labels, logps=logps), **bad})
    with pytest.raises(ValueError):
        run_preference(x, labels, [0, 2], None)
    with pytest.raises(ValueError):
        run_preference(x, labels, [0, 2, 4], None, kind="other")
    with pytest.raises(ValueError):
        run_preference(x, labels, [0, 2, 4], None, d=torch.empty(4, 9, dtype=BF16, device=DEV))
    with pytest.raises(RuntimeError):
        run_preference(x, labels, [0, 2, 4], None, ws=torch.empty(256, dtype=torch.uint8, device=DEV))

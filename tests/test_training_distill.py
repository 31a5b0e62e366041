"""The distillation loss from a teacher's record of its most probable tokens, and its gradient, against
a plain implementation in 64 bits.

Tolerances.  ln p of a token or of the rest is off by 4e-6 (1 + |ln p|) (an exponential's 2^-22, its
argument's roundings, sums in a tree, a logarithm), p relatively by as much, and q by 4e-6 (1 + |ln q|)
likewise.  With g = ln p - ln q of a token or of the rest:
    forward loss      sum q 4e-6 (2 + |ln p| + |ln q|) (1 + |g|)
    reverse loss      sum p 4e-6 (2 + |ln p| + |ln q|) (1 + |g|)
    forward gradient  4e-6 (p Q (2 + |ln p|) + q (2 + |ln q|)); outside the list q = q_r p / p_r and both logarithms
                      of the token's share in the rest too: 4e-6 (2 + |ln p| + |ln p_r| + |ln q_r|) (p Q + q_r p / p_r)
    reverse gradient  p 4e-6 (2 + |ln p| + |ln q|) (1 + |g| + |L|) + p (the loss's own)
all times |weight| / temperature, and a rounding of 2^-8 relative in bf16 (2^-24 in fp32)."""
import math

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from lora_rank_adapter_gb300 import training

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 4e-6
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan
FORMS = [("forward", True), ("forward", False), ("reverse", True), ("reverse", False)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)


def make(T, V, K, dtype, seed=0, pad=0, first=0, temp=1.0, near=0.7):
    """Student's logits inside a wider buffer of sentinels, and a teacher's record near them."""
    g = torch.Generator().manual_seed(seed)
    full = torch.full((T, first + V + pad), 77.0)
    full[:, first:first + V] = torch.randn(T, V, generator=g) * 3
    full = full.to(dtype).to(DEV)
    x = full[:, first:first + V]
    z = torch.log_softmax(x.double().cpu() / temp + near * torch.randn(T, V, generator=g), 1)
    n = min(K, V)
    top, ids = z.topk(n, 1)
    rest = z.scatter(1, ids, -INF).logsumexp(1)
    if n < K:
        ids = torch.cat([ids, torch.full((T, K - n), -1)], 1)
        top = torch.cat([top, torch.full((T, K - n), -INF)], 1)
    w = torch.rand(T, generator=g) + 0.5
    return full, x, ids.to(DEV), top.float().to(DEV), rest.float().to(DEV), w.to(DEV)


def call(x, ids, top, rest, w, kind, d=None, temp=1.0, scale=1.0, stream=None):
    T = x.shape[0]
    row, loss = torch.full((T,), 5.0, device=DEV), torch.full((1,), 5.0, device=DEV)
    training.lora_distill_loss(x, ids, top, row, loss, rest_logps=rest, weights=w, dlogits=d, kind=kind, temperature=temp,
                               grad_scale=scale, stream=stream)
    return row, loss


def oracle(x, ids, top, rest, w, kind, temp=1.0, scale=1.0):
    """{row, loss, d} with the tolerances of each, in 64 bits on the CPU, row by row as the header says."""
    x, ids, top = x.double().cpu(), ids.cpu(), top.double().cpu()
    T, V = x.shape
    w = torch.ones(T, dtype=torch.float64) if w is None else w.double().cpu()
    row, tol = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    d, dtol = torch.zeros(T, V, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    for t in range(T):
        seen = {}
        for i, lq in zip(ids[t].tolist(), top[t].tolist()):
            if 0 <= i < V and i not in seen:
                seen[i] = lq
        if not seen or w[t] == 0:
            continue
        at, lnq = torch.tensor(list(seen)), torch.tensor(list(seen.values()), dtype=torch.float64)
        z = x[t] / temp
        z = z - z.max()
        lnp = z - z.logsumexp(0)
        p = lnp.exp()
        others = torch.ones(V, dtype=torch.bool)
        others[at] = False
        lj, pj, q = lnp[at], p[at], lnq.exp()
        ln_pr = lnp[others].logsumexp(0) if others.any() else torch.tensor(-INF, dtype=torch.float64)
        if rest is not None:
            lj, lnq = torch.cat([lj, ln_pr[None]]), torch.cat([lnq, rest[t].double().cpu()[None]])
            pj, q = lj.exp(), lnq.exp()
        gap = torch.where(lj == lnq, 0.0, lj - lnq)
        m = q if kind == "forward" else pj
        gap = torch.where(m == 0, 0.0, gap)
        L = (m * gap).sum() * (-1 if kind == "forward" else 1)
        weight = 2 + torch.where(m == 0, 0.0, lj.abs() + lnq.abs())
        row[t], tol[t] = L, EPS * (m * weight * (1 + gap.abs())).sum() + 1e-12
        c = float(w[t]) * scale / temp
        n, lnp0 = len(at), torch.where(p > 0, lnp.abs(), 0.0)
        g, gt = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.float64)
        if kind == "forward":
            Q = q.sum()
            g, gt = p * Q, EPS * p * Q * (2 + lnp0)
            g[at] -= q[:n]
            gt[at] += EPS * q[:n] * (2 + torch.where(q[:n] == 0, 0.0, lnq[:n].abs()))
            if rest is not None and q[n] > 0 and others.any():
                share = torch.where(others, (lnp - ln_pr).exp() * q[n], 0.0)
                g -= share
                gt += torch.where(others, EPS * (2 + lnp0 + ln_pr.abs() + lnq[n].abs()) * (p * Q + share), 0.0)
        else:
            P = pj.sum()
            if rest is not None:
                a = torch.full((V,), float(gap[n]), dtype=torch.float64)
                a[at] = gap[:n]
                g = p * (a - L)
            else:
                a = torch.zeros(V, dtype=torch.float64)
                a[at] = gap[:n] + 1
                g = p * (a - L - P)
            size = torch.full((V,), float(weight.max()), dtype=torch.float64)
            gt = p * (EPS * (size + lnp0) * (2 + a.abs() + L.abs()) + tol[t])
        d[t], dtol[t] = c * g, abs(c) * gt
    return {"row": row, "row_tol": tol, "loss": (w * row).sum(), "loss_tol": (w.abs() * tol).sum() + 1e-7 * (w * row).abs().sum(),
            "d": d, "d_tol": dtol}


def close(got, want, bound):
    got = got.double().cpu()
    err = torch.where(got == want, 0.0, (got - want).abs())
    assert bool((err <= bound).all()), (float((err / bound).max()), got.flatten()[:4], want.flatten()[:4])


def check(row, loss, d, want):
    close(row, want["row"], want["row_tol"])
    close(loss[0], want["loss"], want["loss_tol"])
    if d is not None:
        close(d, want["d"], want["d_tol"] + (2.0 ** -8 if d.dtype == BF16 else 2.0 ** -23) * want["d"].abs() + 1e-30)


SIZES = [(1, 1, 1), (3, 2, 5), (2, 7, 3), (5, 8, 8), (4, 9, 2), (3, 255, 128), (40, 300, 64), (7, 1001, 20), (2, 2049, 1),
         (3, 8192, 128), (2, 32003, 17), (1, 128256, 20), (160, 17001, 64), (90, 20001, 100), (3, 450000, 30), (2, 300001, 9)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,K", SIZES)
def test_sizes_strides_and_forms(T, V, K, dtype):
    for n, (kind, with_rest) in enumerate(FORMS):
        pad, first, temp = [(0, 0, 1.0), (3, 1, 0.7), (8, 8, 1.6), (1, 0, 1.0)][n]
        full, x, ids, top, rest, w = make(T, V, K, dtype, seed=V + K, pad=pad, first=first, temp=temp)
        rest = rest if with_rest else None
        want = oracle(x, ids, top, rest, w, kind, temp, 0.5)
        row, loss = call(x, ids, top, rest, w, kind, temp=temp)
        check(row, loss, None, want)
        out = torch.full_like(full, 55.0)
        d = out[:, first:first + V]
        row, loss = call(x, ids, top, rest, w, kind, d, temp, 0.5)
        check(row, loss, d, want)
        assert bool((out[:, :first] == 55).all()) and bool((out[:, first + V:] == 55).all())
        other = torch.full((T, V + 5), 55.0, dtype=dtype, device=DEV)      # at another alignment
        call(x, ids, top, rest, w, kind, other[:, 3:3 + V], temp, 0.5)
        assert torch.equal(other[:, 3:3 + V], d)
        assert bool((other[:, :3] == 55).all()) and bool((other[:, 3 + V:] == 55).all())
        again = call(x, ids, top, rest, w, kind, x, temp, 0.5)             # in place
        assert torch.equal(x, d) and torch.equal(again[0], row) and torch.equal(again[1], loss)
        assert bool((full[:, :first] == 77).all()) and bool((full[:, first + V:] == 77).all())


@pytest.mark.parametrize("kind,with_rest", FORMS)
@pytest.mark.parametrize("V", [200, 30001, 128256])
def test_ignored_rows_short_lists_and_repeated_tokens(V, kind, with_rest):
    T, K = 12, 40
    _, x, ids, top, rest, w = make(T, V, K, BF16, seed=5)
    x[1], x[2] = NAN, NAN
    w[1] = 0.0                       # not looked at
    ids[2] = -1
    ids[3, 7:] = -1                  # shorter lists, holes in them
    ids[4, ::2] = V + 3
    ids[5, 10:20] = ids[5, 0:10]     # listed again: the first counts
    ids[6, :] = ids[6, 0].clone()
    ids[7] = torch.arange(K)         # the row's first tokens, and its last ones
    ids[8] = V - 1 - torch.arange(K)
    ids[9] = torch.arange(K) * 8 % V
    rest = rest if with_rest else None
    d = torch.empty_like(x)
    row, loss = call(x, ids, top, rest, w, kind, d)
    check(row, loss, d, oracle(x, ids, top, rest, w, kind))
    assert row[1] == 0 and row[2] == 0 and bool(d[[1, 2]].eq(0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [60, 9001, 100000])
def test_sure_models(V, dtype):
    """Student and teacher leave next to nothing outside the list: the rest is summed by itself."""
    T, K = 6, 3
    _, x, ids, top, rest, w = make(T, V, K, dtype, seed=6)
    x -= 3
    for t in range(T):
        x[t, ids[t, 0]] = 10.0 + 5 * t      # a rest of e^-13 to e^-38 times what is in it
    rest = torch.linspace(-40, -3, T).to(DEV)
    for kind in ("forward", "reverse"):
        d = torch.empty_like(x)
        row, loss = call(x, ids, top, rest, w, kind, d)
        check(row, loss, d, oracle(x, ids, top, rest, w, kind))


@pytest.mark.parametrize("V", [60, 20001])
def test_masks_and_infinities(V):
    K = 5
    _, x, ids, top, rest, w = make(8, V, K, F32, seed=8)
    ids[:] = torch.arange(K)
    x[0, K:] = -INF                  # the student gives nothing to the rest
    rest[0] = -INF                   # nor does the teacher
    x[1, K:] = torch.finfo(F32).min
    x[2, 3] = -INF                   # a listed token that the student masks and the teacher does not
    x[3, 2] = -INF
    top[3, 2] = -INF                 # both mask it
    x[4, :] = -INF                   # no distribution
    x[5, V - 1] = NAN
    x[6, 1] = INF
    rest[1] = -INF
    for kind, with_rest in FORMS:
        d = torch.empty_like(x)
        r = rest if with_rest else None
        row, _ = call(x, ids, top, r, w, kind, d)
        want = oracle(x[[0, 1, 3, 7]], ids[[0, 1, 3, 7]], top[[0, 1, 3, 7]], None if r is None else r[[0, 1, 3, 7]],
                      w[[0, 1, 3, 7]], kind)
        close(row[[0, 1, 3, 7]], want["row"], want["row_tol"])
        close(d[[0, 1, 3, 7]], want["d"], want["d_tol"] + 2.0 ** -23 * want["d"].abs() + 1e-30)
        assert bool(d[[0, 1], K:].eq(0).all())
        if kind == "forward":
            assert row[2] == INF and bool(d[2].isfinite().all())
        else:
            assert bool(row[2].isfinite())
        for t in (4, 5, 6):
            assert math.isnan(row[t]) and bool(d[t].isnan().any()), t


@pytest.mark.parametrize("V", [60, 9001, 40001])
@pytest.mark.parametrize("temp", [1e-3, 0.02, 50.0, 1e20, 3e37])
def test_far_temperatures(V, temp):
    """Students of one token, and uniform ones with masks: all but zero and all but equal probabilities."""
    T, K = 4, 6
    _, x, ids, _, _, w = make(T, V, K, F32, seed=12)
    x[1, V - 20:] = -INF
    top = torch.log_softmax(torch.randn(T, K + 1, generator=torch.Generator().manual_seed(5)), 1).to(DEV)
    top, rest = top[:, :K].contiguous(), top[:, K].contiguous()
    for kind in ("forward", "reverse"):
        d = torch.empty_like(x)
        row, loss = call(x, ids, top, rest, w, kind, d, temp)
        check(row, loss, d, oracle(x, ids, top, rest, w, kind, temp))


def test_gradient_against_differences():
    T, V, K, temp = 2, 19, 4, 1.3
    _, x, ids, top, rest, w = make(T, V, K, F32, seed=9, temp=temp)
    for kind, with_rest in FORMS:
        r = rest if with_rest else None
        d = torch.empty_like(x)
        call(x, ids, top, r, w, kind, d, temp)
        value = lambda z: float(oracle(z, ids, top, r, w, kind, temp)["loss"])  # noqa: E731
        x64, step = x.double().cpu(), 1e-5
        for t in range(T):
            for v in range(V):
                up, down = x64.clone(), x64.clone()
                up[t, v] += step
                down[t, v] -= step
                # third derivatives (below 10 here) / 6 step^2, rounding 1e-15 / step; the kernel 4e-6 (2 + 12) (1 + 3)
                assert abs(float(d[t, v]) - (value(up) - value(down)) / (2 * step)) <= 2.5e-4, (kind, t, v)


def test_record_of_the_model_itself_has_no_loss():
    """A record that lora_top_logps made of the same logits: no divergence, and the record is what distillation takes."""
    T, V, K = 20, 50001, 64
    _, x, *_ = make(T, V, 1, BF16, seed=10)
    ids = torch.empty((T, K), dtype=torch.int64, device=DEV)
    top, rest = torch.empty((T, K), device=DEV), torch.empty(T, device=DEV)
    for temp in (1.0, 0.6):
        training.lora_top_logps(x, ids, top, rest_logps=rest, temperature=temp)
        for kind in ("forward", "reverse"):
            d = torch.empty_like(x)
            row, loss = call(x, ids, top, rest, None, kind, d, temp)
            # each bucket's ln p is off by 4e-6 (1 + |ln p|) on both sides, at most 4e-6 * 30 here
            assert float(row.abs().max()) <= 2.4e-4 and float(d.abs().max()) <= 2.4e-4
            check(row, loss, d, oracle(x, ids, top, rest, None, kind, temp))


@pytest.mark.parametrize("T,V,dtype", [(700, 70001, BF16), (1500, 20000, BF16), (600, 40002, F32), (4000, 300, F32),
                                       (3000, 4000, BF16), (2000, 15001, BF16)])
def test_many_rows_in_place(T, V, dtype):
    g = torch.Generator(DEV).manual_seed(T)
    x = (torch.randn((T, V), generator=g, device=DEV) * 3).to(dtype)
    K = 33
    ids = torch.randint(0, V, (T, K), generator=g, device=DEV)
    top = torch.log_softmax(torch.randn((T, K + 1), generator=g, device=DEV), 1)
    top, rest = top[:, :K].contiguous(), top[:, K].contiguous()
    w = torch.rand(T, generator=g, device=DEV)
    w[::5] = 0.0
    ids[3::7] = -1
    d = torch.empty_like(x)
    row, loss = call(x, ids, top, rest, w, "forward", d)
    some = torch.arange(0, T, 97, device=DEV)
    want = oracle(x[some], ids[some], top[some], rest[some], w[some], "forward")
    close(row[some], want["row"], want["row_tol"])
    close(d[some], want["d"], want["d_tol"] + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * want["d"].abs() + 1e-30)
    for _ in range(3):
        copy = x.clone()
        again = call(copy, ids, top, rest, w, "forward", copy)
        assert torch.equal(copy, d) and torch.equal(again[0], row) and torch.equal(again[1], loss)


@pytest.mark.parametrize("V,dtype", [(70001, BF16), (128256, BF16), (130000, F32)])
def test_long_runs_of_ignored_rows(V, dtype):
    """Clusters that come for thousands of rows, all but a few of them ignored, alone and in runs."""
    g = torch.Generator(DEV).manual_seed(7)
    T, K, live = 3000, 5, 40
    x = torch.full((T, V), NAN, dtype=dtype, device=DEV)
    ids = torch.randint(0, V, (T, K), generator=g, device=DEV)
    top = torch.log_softmax(torch.randn((T, K + 1), generator=g, device=DEV), 1)[:, :K].contiguous()
    w = torch.zeros(T, device=DEV)
    rows = torch.cat([torch.randperm(T, generator=g, device=DEV)[:live], torch.arange(1500, 1520, device=DEV)]).unique()
    x[rows] = (torch.randn((len(rows), V), generator=g, device=DEV) * 3).to(dtype)
    w[rows] = 0.5
    d = torch.full_like(x, 3.0)
    for _ in range(3):
        row, loss = call(x, ids, top, None, w, "forward", d)
    some = rows[::9]
    want = oracle(x[some], ids[some], top[some], None, w[some], "forward")
    close(row[some], want["row"], want["row_tol"])
    close(d[some], want["d"], want["d_tol"] + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * want["d"].abs() + 1e-30)
    off = torch.ones(T, dtype=torch.bool, device=DEV)
    off[rows] = False
    assert bool(row[off].eq(0).all()) and not bool(d[off].any()) and bool(row[rows].ne(0).all())
    # every row once: the loss is their sum
    close(loss[0], (w.double() * row.double()).sum().cpu(), 1e-6 * float((w * row).abs().sum()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 7, 8, 17, 40, 257, 1901, 4099, 20011, 52003, 450003])
def test_gradients_at_any_offset(V, dtype):
    """Rows of the gradient at every offset within 16 bytes to those of the logits: the same values, and nothing beside them."""
    T, K = 3, 6
    _, x, ids, top, rest, w = make(T, V, K, dtype, seed=V, pad=1, first=2)
    ids[1] = torch.tensor([0, V - 1, V // 2, 1, V - 2, V // 2 + 1], device=DEV)     # the ends too
    d = torch.empty_like(x)                                                          # rows as the logits' up to a shift
    call(x, ids, top, rest, w, "forward", d)
    check(*call(x, ids, top, rest, w, "forward"), d, oracle(x, ids, top, rest, w, "forward"))
    for first in range(16 // x.element_size()):
        out = torch.full((T, V + 16), 55.0, dtype=dtype, device=DEV)
        call(x, ids, top, rest, w, "forward", out[:, first:first + V])
        assert torch.equal(out[:, first:first + V], d), first
        assert bool((out[:, :first] == 55).all()) and bool((out[:, first + V:] == 55).all())


def test_results_that_lie_beside_the_inputs():
    """One buffer of weights, row losses, the loss and the rest, with no gap between them."""
    T, V, K = 37, 500, 9
    _, x, ids, top, rest, w = make(T, V, K, F32, seed=3)
    for kind in ("forward", "reverse"):
        want = call(x, ids, top, rest, w, kind)
        buf = torch.cat([w, torch.full((T + 1,), 5.0, device=DEV), rest])
        row, loss = buf[T:2 * T], buf[2 * T:2 * T + 1]
        training.lora_distill_loss(x, ids, top, row, loss, rest_logps=buf[2 * T + 1:], weights=buf[:T], kind=kind)
        assert torch.equal(row, want[0]) and torch.equal(loss, want[1])
        assert torch.equal(buf[:T], w) and torch.equal(buf[2 * T + 1:], rest)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 9001, 40001])
def test_rows_far_apart(V, dtype):
    """Offsets of rows and of their gradients beyond 2^31 elements."""
    T, K, ld = 3, 12, (1 << 30) + 8
    _, x, ids, top, rest, w = make(T, V, K, dtype, seed=V)
    d = torch.empty_like(x)
    want = call(x, ids, top, rest, w, "forward", d)
    far = torch.empty(2 * ld + V, dtype=dtype, device=DEV).as_strided((T, V), (ld, 1))
    far.copy_(x)
    row, loss = call(far, ids, top, rest, w, "forward")
    check(row, loss, None, oracle(x, ids, top, rest, w, "forward"))
    got = call(far, ids, top, rest, w, "forward", far)
    check(*got, far, oracle(x, ids, top, rest, w, "forward"))
    check(*want, d, oracle(x, ids, top, rest, w, "forward"))


@pytest.mark.parametrize("V,dtype", [(140003, F32), (210001, F32), (420001, BF16)])
def test_many_rows_of_a_long_vocabulary(V, dtype):
    """One block a row, of more rounds than the word that says in which of them a listed token is met."""
    T, K = 80, 128
    _, x, ids, top, rest, w = make(T, V, K, dtype, seed=V)
    ids[:, ::5] = torch.arange(V - 26, V, device=DEV)           # the same tokens late in each row, some twice
    want = oracle(x, ids, top, rest, w, "reverse")
    row, loss = call(x, ids, top, rest, w, "reverse")
    check(row, loss, None, want)
    d = torch.empty_like(x)
    row, loss = call(x, ids, top, rest, w, "reverse", d)
    check(row, loss, d, want)


def test_two_streams_and_a_graph():
    _, x, ids, top, rest, w = make(30, 32003, 20, BF16, seed=1)
    _, y, ids2, top2, rest2, w2 = make(3, 128256, 64, F32, seed=2)
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    want = call(x, ids, top, rest, w, "forward", dx), call(y, ids2, top2, None, None, "reverse", dy)
    first = dx.clone(), dy.clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got = call(x, ids, top, rest, w, "forward", dx, stream=a), call(y, ids2, top2, None, None, "reverse", dy, stream=b)
        torch.cuda.synchronize()
        assert all(torch.equal(g, h) for p, q in zip(got, want) for g, h in zip(p, q))
        assert torch.equal(dx, first[0]) and torch.equal(dy, first[1])
    row, loss = torch.empty(30, device=DEV), torch.empty(1, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        training.lora_distill_loss(x, ids, top, row, loss, rest_logps=rest, weights=w, dlogits=dx)
    dx.zero_()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, first[0]) and torch.equal(row, want[0][0]) and torch.equal(loss, want[0][1])


def test_no_rows():
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    row, loss = call(e(0, 100), torch.empty((0, 5), dtype=torch.int64, device=DEV), e(0, 5), None, None, "forward")
    assert float(loss) == 0.0

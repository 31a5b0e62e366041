"""Log-probabilities with entropy and the most probable tokens, and their gradient, against plain
implementations in 64 bits.

Tolerances, u = (x - m) / temperature.  An exponential has a relative error of 2^-22 of its own
and 3 * 2^-24 |u| from the three roundings of its argument, below 2^-22 (1 + |u|); sums of positive
terms in a tree of short chains are off by 4e-6 of themselves, the logarithm and the last
differences by some 2^-24 of values up to |result| + 12.  So, with p's relative error
e_v = 4e-6 + 2^-22 (1 + |u_v|):
    logps, top_logps, rest_logps    4e-6 max(1, |value|), twice that for the rest (two sums)
    entropy = ln S - sum e u / S    2^-22 sum p (1 + |u|) (1 + |u| + H) + 4e-6 (1 + H)
    gradient                        e_v p_v (|G| + |h| (|ln p_v| + H + 1)) + 4e-6 (own gradients), / temperature,
                                    and a rounding of 2^-8 relative in bf16
Ids are exact."""
import math

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from lora_rank_adapter_gb300 import training

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS, HALF = 4e-6, 2.0 ** -22
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


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


def call(x, K, labels=None, temp=1.0, stream=None):
    T = x.shape[0]
    full = lambda *s, v=5.0: torch.full(s, v, device=DEV)  # noqa: E731
    out = {"ids": torch.full((T, K), 12345, dtype=torch.int64, device=DEV), "top": full(T, K), "H": full(T),
           "rest": full(T), "stats": full(T, 2), "logps": full(T) if labels is not None else None}
    training.lora_top_logps(x, out["ids"], out["top"], labels=labels, logps=out["logps"], entropy=out["H"],
                            rest_logps=out["rest"], stats=out["stats"], temperature=temp, stream=stream)
    return out


def oracle(x, K, labels=None, temp=1.0):
    """In 64 bits on the CPU; rows that are ignored as the header says."""
    x = x.double().cpu()
    T, V = x.shape
    z = x / temp
    z = z - z.amax(1, keepdim=True)
    lnp = z - z.logsumexp(1, keepdim=True)
    p = lnp.exp()
    H = torch.special.entr(p).sum(1)
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :K]
    ids = torch.full((T, K), -1)
    top = torch.full((T, K), -INF, dtype=torch.float64)
    ids[:, :order.shape[1]] = order
    top[:, :order.shape[1]] = lnp.gather(1, order)
    ids[top == -INF] = -1
    listed = torch.zeros_like(p, dtype=torch.bool).scatter_(1, order, True)
    rest = lnp.masked_fill(listed, -INF).logsumexp(1)
    ok = torch.ones(T, dtype=torch.bool)
    out = {"p": p, "lnp": lnp, "u": z, "H": H, "ids": ids, "top": top, "rest": rest, "ok": ok}
    if labels is not None:
        lab = labels.cpu()
        ok = (lab >= 0) & (lab < V)
        out["logps"] = torch.where(ok, lnp.gather(1, lab.clamp(0, V - 1)[:, None])[:, 0], 0.0)
        out["ok"] = ok
        ids[~ok], top[~ok] = -1, -INF
        out["H"], out["rest"] = torch.where(ok, H, 0.0), torch.where(ok, rest, 0.0)
    return out


def close(got, want, bound):
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    err = torch.where(same, 0.0, (got - want).abs())
    assert bool((err <= bound).all()), (float((err / bound).max()), got.flatten()[:4], want.flatten()[:4])


def check(got, want, rows=slice(None)):
    w = {k: v[rows] for k, v in want.items()}
    g = {k: v[rows] if v is not None else None for k, v in got.items()}
    assert torch.equal(g["ids"].cpu(), w["ids"])
    close(g["top"], w["top"], EPS * w["top"].abs().clamp(1, 1e30))
    if g["logps"] is not None:
        close(g["logps"], w["logps"], EPS * w["logps"].abs().clamp(1, 1e30))
    u = w["u"].abs()
    bound = HALF * torch.where(w["p"] > 0, w["p"] * (1 + u) * (1 + u + w["H"][:, None]), 0.0).sum(1) + EPS * (1 + w["H"])
    close(g["H"], w["H"], bound)
    close(g["rest"], w["rest"], 2 * EPS * w["rest"].abs().clamp(1, 1e30))


SIZES = [(1, 1, 1), (3, 2, 5), (2, 7, 0), (5, 8, 3), (4, 9, 9), (3, 255, 128), (40, 300, 64), (7, 1001, 20), (2, 2049, 1),
         (3, 8192, 128), (2, 32003, 17), (1, 128256, 20), (160, 32000, 64), (90, 50001, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,K", SIZES)
def test_sizes_strides_and_temperatures(T, V, K, dtype):
    for pad, first, temp in ((0, 0, 1.0), (3, 1, 0.7), (8, 8, 1.6)):
        full, x, labels = make(T, V, dtype, seed=V + K, pad=pad, first=first)
        before = full.clone()
        want = oracle(x, K, labels, temp)
        check(call(x, K, labels, temp), want)
        if pad:
            check(call(x, K, None, temp), oracle(x, K, None, temp))
        assert torch.equal(full, before)


def test_results_that_are_not_wanted():
    _, x, labels = make(5, 3001, BF16)
    want = call(x, 7, labels)
    ids, top = torch.empty((5, 7), dtype=torch.int64, device=DEV), torch.empty((5, 7), device=DEV)
    training.lora_top_logps(x, ids, top)
    all_rows = call(x, 7)
    assert torch.equal(ids, all_rows["ids"]) and torch.equal(top, all_rows["top"])
    H = torch.empty(5, device=DEV)
    none = torch.empty((5, 0), dtype=torch.int64, device=DEV), torch.empty((5, 0), device=DEV)
    training.lora_top_logps(x, *none, labels=labels, logps=torch.empty(5, device=DEV), entropy=H)
    close(H, want["H"].double().cpu(), 2 * EPS * 12)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("V", [500, 40000, 128256])
def test_rows_in_any_order(T, V, dtype):
    """Rows whose largest values come where the search for them expects the fewest: ascending, descending,
    constant, in steps, all of them in one stretch or one column of the pieces, masked by the lowest value."""
    i = torch.arange(V, dtype=torch.float64)
    kinds = [i / V * 20, -i / V * 20, torch.full_like(i, 1.5), torch.zeros_like(i), (i // (V // 7)) * 1.0,
             torch.where(i > V - 700, i - V + 720, 0.1 * (i % 13)), torch.where(i % 8 == 3, i / V, -3.0 - (i % 5)),
             torch.where(i % 1000 == 7, 2.0, float(torch.finfo(dtype).min)), torch.where(i < 4, 9.0 + i, -INF),
             torch.where(i % 2 == 0, 0.0, -0.0), torch.where(i == V - 1, 30.0, i / V),
             torch.where(i < V // 2, -float("inf"), -i / V)]
    x = torch.stack([kinds[t % len(kinds)] for t in range(T)]).to(dtype).to(DEV)
    for K in (1, 20, 128):
        rows = slice(0, min(T, len(kinds)))
        got, want = call(x, K), oracle(x[rows], K)
        check({k: v[rows] if v is not None else None for k, v in got.items()}, want)
        for t in range(len(kinds), T):      # the same row gives the same anywhere
            assert torch.equal(got["ids"][t], got["ids"][t % len(kinds)])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 4099, 70000])
def test_masks_infinities_and_nan(V, dtype):
    _, x, _ = make(12, V, dtype, seed=3)
    labels = torch.arange(12, device=DEV) % 5
    low = torch.finfo(dtype).min
    x[0, 5:] = -INF                 # most of the row masked out: fewer alternatives than asked for
    x[1, 5:] = low
    x[2, :] = low                   # nothing left, by the lowest value: uniform
    x[3, :] = -INF                  # nothing left, by minus infinity: NaN, as 0 / 0
    x[4, 7] = INF
    x[5, 7] = NAN
    x[6, int(labels[6])] = -INF     # the label itself masked: logp -inf
    x[7, :] = NAN
    labels[7] = -100                # not looked at
    x[8, :] = INF
    labels[8] = V
    x[9, :-1] = -INF                # one column left, and it is the label
    labels[9] = V - 1
    x[10, :] = torch.finfo(dtype).max      # equal and huge: uniform
    x[11, ::3], x[11, 1::3], x[11, 2::3] = low, -INF, low * 0.75      # nothing but masks of three kinds
    K = 9
    got, want = call(x, K, labels), oracle(x, K, labels)
    check(got, want, torch.tensor([0, 1, 2, 6, 7, 8, 9, 10, 11]))
    for t in (3, 4, 5):
        assert bool((got["ids"][t] == -1).all()) and bool(got["top"][t].isnan().all())
        assert all(math.isnan(got[k][t]) for k in ("logps", "H", "rest"))
    assert got["ids"][0].tolist()[5:] == [-1] * 4 and got["logps"][6] == -INF
    one = torch.ones(12, device=DEV)
    for in_place in (False, True):
        d = x.clone() if in_place else torch.empty_like(x)
        training.lora_top_logps_backward(d if in_place else x, got["stats"], d, labels=labels, top_ids=got["ids"],
                                         entropy=got["H"], dlogps=one, dentropy=one, dtop_logps=one[:, None].repeat(1, K))
        assert bool(d[[7, 8]].eq(0).all()) and bool(d[[3, 4, 5]].isnan().any(1).all())
        assert bool(d[[0, 1, 2, 6, 9, 10, 11]].isfinite().all())
        assert bool(d[0, 5:].eq(0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temp", [1e-3, 0.02, 50.0, 1e20, 3e37])
def test_far_temperatures(dtype, temp):
    """Rows whose exponentials are all but one zero, and rows that are all but uniform, masks among them."""
    _, x, labels = make(6, 3001, dtype, seed=12)
    x[1::2, 5::7] = -INF
    x[2, 9::11] = torch.finfo(dtype).min
    x[4] *= 1e30
    x[5, 1000:] = -INF
    check(call(x, 20, labels, temp), oracle(x, 20, labels, temp))


def oracle_gradient(w, x, labels, ids, gl, gh, gt, temp):
    """(gradient, its tolerance before the last rounding)"""
    T, V = x.shape
    own, size = torch.zeros(T, V, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    G = torch.zeros(T, dtype=torch.float64)
    if gl is not None:
        lab, g = labels.cpu().clamp(0, V - 1)[:, None], torch.where(w["ok"], gl.double().cpu(), 0.0)[:, None]
        own.scatter_add_(1, lab, g)
        size.scatter_add_(1, lab, g.abs())
        G += g[:, 0]
    if gt is not None:
        i = ids.cpu()
        g = torch.where((i >= 0) & (i < V) & w["ok"][:, None], gt.double().cpu(), 0.0)
        own.scatter_add_(1, i.clamp(0, V - 1), g)
        size.scatter_add_(1, i.clamp(0, V - 1), g.abs())
        G += g.sum(1)
    h = torch.zeros(T, dtype=torch.float64) if gh is None else torch.where(w["ok"], gh.double().cpu(), 0.0)
    lnp = torch.where(w["p"] > 0, w["lnp"], 0.0)
    d = own - w["p"] * (G[:, None] + h[:, None] * (lnp + w["H"][:, None]))
    d[~w["ok"]] = 0
    e = EPS + HALF * (1 + torch.where(w["p"] > 0, w["u"].abs(), 0.0))
    mass = size.sum(1)[:, None] + h.abs()[:, None] * (lnp.abs() + w["H"][:, None] + 1)
    return d / temp, (e * w["p"] * mass + EPS * size) / temp


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,K", [s for s in SIZES if s[0] < 100])
def test_gradient(T, V, K, dtype):
    g = torch.Generator().manual_seed(K)
    for pad, first, temp, use in ((0, 0, 1.0, "lht"), (3, 1, 0.7, "lt"), (8, 8, 1.6, "h"), (1, 0, 1.0, "l")):
        full, x, labels = make(T, V, dtype, seed=V + K, pad=pad, first=first)
        got, w = call(x, K, labels, temp), oracle(x, K, labels, temp)
        gl = torch.randn(T, generator=g).to(DEV) if "l" in use else None
        gh = torch.randn(T, generator=g).to(DEV) if "h" in use else None
        gt = torch.randn(T, K, generator=g).to(DEV) if "t" in use else None
        args = dict(labels=labels, top_ids=got["ids"], entropy=got["H"], dlogps=gl, dentropy=gh, dtop_logps=gt,
                    temperature=temp)
        out = torch.full_like(full, 55.0)
        d = out[:, first:first + V]
        training.lora_top_logps_backward(x, got["stats"], d, **args)
        want, tol = oracle_gradient(w, x, labels, got["ids"], gl, gh, gt, temp)
        rounding = 2.0 ** -8 * want.abs() if dtype == BF16 else 2.0 ** -24 * want.abs()
        close(d, want, tol + rounding + 1e-30)
        assert bool((out[:, :first] == 55).all()) and bool((out[:, first + V:] == 55).all())
        other = torch.full((T, V + 5), 55.0, dtype=dtype, device=DEV)      # at another alignment
        training.lora_top_logps_backward(x, got["stats"], other[:, 3:3 + V], **args)
        assert torch.equal(other[:, 3:3 + V], d)
        assert bool((other[:, :3] == 55).all()) and bool((other[:, 3 + V:] == 55).all())
        training.lora_top_logps_backward(x, got["stats"], x, **args)       # in place
        assert torch.equal(x, d)
        assert bool((full[:, :first] == 77).all()) and bool((full[:, first + V:] == 77).all())


def test_gradient_of_any_ids():
    """Repeated ids add up, ids outside the row have no gradient, and the label may be one of them."""
    T, V, K = 6, 3001, 12
    _, x, labels = make(T, V, F32, ignored=0.0)
    got, w = call(x, K, labels), oracle(x, K, labels)
    ids = torch.randint(0, 7, (T, K), generator=torch.Generator().manual_seed(1))
    ids[:, 3] = V - 1
    ids[:, 4] = V - 1
    ids[1, 5], ids[2, 6], ids[3] = V, -5, -1
    labels[:3] = 2
    ids = ids.to(DEV)
    gt = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(DEV)
    gl = torch.randn(T, generator=torch.Generator().manual_seed(3)).to(DEV)
    d = torch.empty_like(x)
    got = call(x, K, labels)
    training.lora_top_logps_backward(x, got["stats"], d, labels=labels, top_ids=ids, dlogps=gl, dtop_logps=gt)
    want, tol = oracle_gradient(oracle(x, K, labels), x, labels, ids, gl, None, gt, 1.0)
    close(d, want, tol + 2.0 ** -24 * want.abs() + 1e-30)


def test_gradient_against_differences():
    """Central differences of the formula in 64 bits, of a weighted sum of all results."""
    T, V, K, temp = 2, 23, 4, 1.3
    _, x, labels = make(T, V, F32, seed=9, ignored=0.0)
    got = call(x, K, labels, temp)
    g = torch.Generator().manual_seed(4)
    gl, gh, gt = torch.randn(T, generator=g), torch.randn(T, generator=g), torch.randn(T, K, generator=g)
    d = torch.empty_like(x)
    training.lora_top_logps_backward(x, got["stats"], d, labels=labels, top_ids=got["ids"], entropy=got["H"],
                                     dlogps=gl.to(DEV), dentropy=gh.to(DEV), dtop_logps=gt.to(DEV), temperature=temp)
    ids, lab = got["ids"].cpu(), labels.cpu()

    def value(z):
        lnp = torch.log_softmax(z / temp, 1)
        H = -(lnp.exp() * lnp).sum(1)
        return (gl * lnp.gather(1, lab[:, None])[:, 0] + gh * H).sum() + (gt * lnp.gather(1, ids)).sum()

    x64, step = x.double().cpu(), 1e-5
    for t in range(T):
        for v in range(V):
            up, down = x64.clone(), x64.clone()
            up[t, v] += step
            down[t, v] -= step
            slope = float(value(up) - value(down)) / (2 * step)
            # the difference: third derivatives (below 10 here) / 6 step^2 and rounding 1e-15 / step; the kernel: 4e-6
            assert abs(float(d[t, v]) - slope) <= 2e-5, (t, v)


def test_rows_without_incoming_gradient_are_not_read():
    T, V, K = 5, 9001, 6
    _, x, labels = make(T, V, BF16, ignored=0.0)
    got = call(x, K, labels)
    gl, gh, gt = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV), torch.zeros((T, K), device=DEV)
    gt[1, 3] = 1.0
    x[0], x[2] = NAN, NAN
    d = torch.full_like(x, 3.0)
    training.lora_top_logps_backward(x, got["stats"], d, labels=labels, top_ids=got["ids"], entropy=got["H"], dlogps=gl,
                                     dentropy=gh, dtop_logps=gt)
    assert bool(d[[0, 2, 3, 4]].eq(0).all()) and bool(d[1].ne(0).any()) and bool(d.isfinite().all())


def test_repeated_calls_agree_and_streams_do_not_meet():
    _, x, labels = make(300, 50001, BF16, seed=1)
    _, y, other = make(2, 128256, F32, seed=2)
    first, second = call(x, 64, labels), call(y, 100, other)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = call(x, 64, labels, stream=a), call(y, 100, other, stream=b)
        torch.cuda.synchronize()
        for g, w in zip(got, (first, second)):
            for k in w:
                assert torch.equal(g[k], w[k]), k


def test_captured_and_replayed():
    T, V, K = 9, 32003, 20
    _, x, labels = make(T, V, BF16)
    out = call(x, K, labels)
    one = torch.ones(T, device=DEV)
    d = torch.empty_like(x)

    def both():
        training.lora_top_logps(x, out["ids"], out["top"], labels=labels, logps=out["logps"], entropy=out["H"],
                                rest_logps=out["rest"], stats=out["stats"])
        training.lora_top_logps_backward(x, out["stats"], d, labels=labels, top_ids=out["ids"], entropy=out["H"],
                                         dlogps=one, dentropy=one, dtop_logps=out["top"])
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    _, fresh, _ = make(T, V, BF16, seed=77)
    x.copy_(fresh)
    graph.replay()
    torch.cuda.synchronize()
    replayed = {k: v.clone() for k, v in out.items()}, d.clone()
    both()
    for k, v in out.items():
        assert torch.equal(v, replayed[0][k]), k
    assert torch.equal(d, replayed[1])
    check(out, oracle(x, K, labels))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(3, 1), (3, 7), (2, 17), (3, 40), (2, 1901), (2, 20011), (400, 9001)])
def test_gradients_at_any_offset(T, V, dtype):
    """Rows of the gradient at every offset within 16 bytes to those of the logits: the same values, and nothing beside them."""
    K = 6
    _, x, labels = make(T, V, dtype, seed=V, pad=1, first=2)
    near = call(x, K, labels)
    g, gt = torch.randn(T, device=DEV), torch.randn(T, K, device=DEV)
    back = lambda d: training.lora_top_logps_backward(  # noqa: E731
        x, near["stats"], d, labels=labels, top_ids=near["ids"], entropy=near["H"], dlogps=g, dentropy=g, dtop_logps=gt)
    d = torch.full((T, V + 3), 55.0, dtype=dtype, device=DEV)[:, 2:2 + V]      # at the logits' own offsets
    back(d)
    for first in range(16 // x.element_size()):
        out = torch.full((T, V + 16), 55.0, dtype=dtype, device=DEV)
        back(out[:, first:first + V])
        assert torch.equal(out[:, first:first + V], d), first
        assert bool((out[:, :first] == 55).all()) and bool((out[:, first + V:] == 55).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 40001])
def test_rows_far_apart(V, dtype):
    """Offsets of rows and of their gradients beyond 2^31 elements."""
    T, K, ld = 3, 12, (1 << 30) + 8
    _, x, labels = make(T, V, dtype, seed=V, ignored=0.0)
    far = torch.empty(2 * ld + V, dtype=dtype, device=DEV).as_strided((T, V), (ld, 1))
    far.copy_(x)
    out = call(far, K, labels)
    check(out, oracle(x, K, labels))
    near = call(x, K, labels)
    g = torch.randn(T, device=DEV)
    d = torch.empty_like(x)
    training.lora_top_logps_backward(x, near["stats"], d, labels=labels, entropy=near["H"], dlogps=g, dentropy=g)
    training.lora_top_logps_backward(far, near["stats"], far, labels=labels, entropy=near["H"], dlogps=g, dentropy=g)
    assert torch.equal(far, d)


@pytest.mark.parametrize("V,dtype", [(9001, BF16), (16000, F32), (30011, F32), (64001, BF16)])
def test_many_rows(V, dtype):
    """More rows than the device holds large blocks twice: random, ascending ones, and ones of one value but for some."""
    T = 1000
    _, x, labels = make(T, V, dtype, seed=V, pad=1)
    x[10] = torch.arange(V, device=DEV) / V
    x[11], x[12] = x[10].flip(0), x[10] * 100
    x[13] = 1.0
    x[14, 5:] = -INF
    x[15] = torch.linspace(-4, 4, V, device=DEV) + x[16] / 3
    for K in (1, 20, 48, 49):
        check(call(x, K, labels), oracle(x, K, labels))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2, 160])
def test_long_vocabulary(T, dtype):
    _, x, labels = make(T, 500003 if T > 2 else 1000003, dtype, seed=T, ignored=0.0)
    check(call(x, 128, labels), oracle(x, 128, labels))


def test_no_rows_and_no_columns():
    call(torch.empty((0, 100), device=DEV), 5, torch.empty(0, dtype=torch.int64, device=DEV))
    out = call(torch.empty((3, 0), device=DEV), 5)
    assert bool(out["ids"].eq(-1).all()) and bool(out["H"].isnan().all())
    out = call(torch.empty((3, 0), device=DEV), 5, torch.zeros(3, dtype=torch.int64, device=DEV))
    assert bool(out["ids"].eq(-1).all()) and bool(out["H"].eq(0).all())

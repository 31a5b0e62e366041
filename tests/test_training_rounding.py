"""8-bit optimizer states over thousands of steps: rounded at random, m and u = sqrt(v) follow
their gradients, where rounding to nearest leaves them at their place in the block; and the
rounding itself, bit for bit against the same steps in torch."""
import ctypes

import pytest
import torch

from lora_rank_adapter_gb300 import _build, torch_ops, training
from tests.test_training_adamw import BF16, F32, HYPER, blocks, cpu, dequantize, make, sentinels_hold

DEV = "cuda:0"
A, B, M32 = 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF
SIZES = [1, 7, 255, 256, 257, 2047, 2048, 2049, 0, 5000, 40000]


# ----------------------------------------------------------------------------- the rounding in torch
def times(x, c):
    """x * c modulo 2^32, x an int64 tensor or a number below 2^32."""
    return ((x & 0xFFFF) * c + (((x >> 16) * c & 0xFFFF) << 16)) & M32


def mix(x):
    x = x ^ (x >> 16)
    x = times(x, A)
    x = x ^ (x >> 15)
    x = times(x, B)
    x = x ^ (x >> 16)
    x = times(x, A)
    return x ^ (x >> 15)


def bits(step, first_chunk, n):
    """The 32 bits of each of n elements of a tensor whose first chunk has this number."""
    i = torch.arange(n, dtype=torch.int64)
    key = mix((mix((step + mix(step >> 32)) & M32) + first_chunk + i // training.ADAMW_CHUNK) & M32)
    x = times((key + i % training.ADAMW_CHUNK) & M32, A)
    x = x ^ (x >> 15)
    x = times(x, B)
    return x ^ (x >> 16)


def to_code(q, r):
    base = torch.where(q.abs() < 2.0 ** -6, torch.copysign(torch.full_like(q, 2.0 ** -6), q), 0.0)
    t = ((q + base).view(torch.int32).long() & M32) + 16 * r + 8 & 0xFFF00000
    t = torch.where(t >= 2 ** 31, t - 2 ** 32, t).to(torch.int32).view(F32)
    return (t - base).clamp(-448.0, 448.0)


def quantize(x, r, least=0.0):
    """(codes, scales) of a tensor from its 16-bit numbers r."""
    n = x.numel()
    top = blocks(x).abs().amax(1).clamp(min=1e-30)
    q = blocks(x) * torch.div(torch.full_like(top, 448.0), top)[:, None]
    q = to_code(q.reshape(-1)[:n], r)
    if least:
        q = torch.where(x > 0, q.clamp(min=least), q)
    return q.to(torch.float8_e4m3fn), top * (1 / 448.0)


def test_the_rounding_is_unbiased_and_between_neighbours():
    """Every value of [0, 448] goes to one of the two e4m3 values around it, up with the probability
    of its place between them: over all 2^16 numbers the mean is the value to 2^-17 of their
    distance (numbers are centred), plus 2^-20 for the 20 bits of the place."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    r = torch.arange(65536, dtype=torch.int64)
    g = torch.Generator().manual_seed(0)
    for k in range(126):
        lo, hi = codes[k], codes[k + 1]
        for f in [0.0] + torch.rand(3, generator=g).tolist():
            q = lo + (hi - lo) * f
            for sign in (1.0, -1.0):
                out = to_code(torch.full((65536,), float(q) * sign), r) * sign
                assert bool(((out == lo) | (out == hi)).all()) and (f > 0 or bool((out == lo).all()))
                got = (out.double() - float(lo)) / float(hi - lo)
                assert abs(float(got.mean()) - float((q - lo) / (hi - lo))) <= 2.0 ** -17 + 2.0 ** -19
    assert bool((to_code(torch.full((65536,), 448.0001), r) == 448).all())
    # the numbers: both halves spread evenly, and unlike from step to step
    x = torch.stack([bits(s, 0, 8192) for s in range(1, 60)])
    for half in (x & 0xFFFF, x >> 16):
        u = half.double() / 65536 - 0.5
        n = u.numel()
        assert abs(float(u.mean())) < 5 / (12 * n) ** 0.5
        for a, b in ((u[1:], u[:-1]), (u[:, 1:], u[:, :-1]), (u[:, 256:], u[:, :-256]), (u[:, 2048:], u[:, :-2048])):
            assert abs(float((a * b).mean()) * 12) < 5 / a.numel() ** 0.5


def test_the_flag_belongs_to_8_bit_states():
    _build.build()
    L = training.lib()
    t = (training.AdamWTensor * 1)(training.AdamWTensor(0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0, 10))

    def build(flags):
        made = training.AdamWPlanStruct()
        return L.lora_adamw_build(t, 1, 0, 0, flags, ctypes.c_void_p(0x10000), 0, ctypes.byref(made), None)

    assert build(training.ADAMW_STOCHASTIC) == 1                                       # invalid
    assert build(training.ADAMW_STOCHASTIC | training.ADAMW_STATE_8BIT) == 4           # passes on to the workspace
    plan = training.AdamWPlanStruct(0x10000, 4, 0, 0, training.ADAMW_STOCHASTIC, 0)
    hyper = training.AdamWHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    assert L.lora_adamw(ctypes.byref(plan), ctypes.byref(hyper), None, None) == 1
    with pytest.raises(ValueError, match="8-bit"):
        x = torch.zeros(4)
        training.lora_adamw_plan([x], [x], [x], [x], stochastic=True)


# ----------------------------------------------------------------------------- on the GPU
def _plan(s):
    return training.lora_adamw_plan(s["p"], s["g"], s["m"], s["v"], masters=s["w"] or None, exp_avg_scales=s["ms"],
                                    exp_avg_sq_scales=s["vs"], stochastic=True)


@pytest.mark.gpu
@pytest.mark.parametrize("param,grad,master", [(F32, F32, False), (BF16, F32, True), (BF16, BF16, False),
                                               (F32, BF16, False), (BF16, BF16, True)])
@pytest.mark.parametrize("offset", [0, 3, 8])
def test_codes_bit_for_bit(param, grad, master, offset):
    torch.cuda.set_device(0)
    s = make(SIZES, param, grad, 8, master, offset)
    plan = _plan(s)
    factor = 0.37
    f = torch.full((1,), factor, device=DEV)
    for step in (1, 2, 50, 2 ** 33 + 5):
        before = cpu(s)
        training.lora_adamw(plan, step=step, grad_factor=f, **HYPER)
        after = cpu(s)
        chunk = 0
        for i, n in enumerate(SIZES):
            g = before["g"][i].float() * torch.tensor(factor, dtype=F32)
            m = dequantize(before["m"][i], before["ms"][i])
            u = dequantize(before["v"][i], before["vs"][i])
            m = m * HYPER["beta1"] + g * (1 - HYPER["beta1"])
            v = (u * u) * HYPER["beta2"] + (g * g) * (1 - HYPER["beta2"])
            r = bits(step, chunk, n)
            chunk += -(-n // training.ADAMW_CHUNK)
            for q, scale, x, low, least in (("m", "ms", m, r & 0xFFFF, 0.0), ("v", "vs", v.sqrt(), r >> 16, 2.0 ** -9)):
                want_q, want_s = quantize(x, low, least)
                assert torch.equal(after[q][i].float(), want_q.float()), (step, n, q)
                assert torch.equal(after[scale][i], want_s), (step, n, scale)
    sentinels_hold(s)


@pytest.mark.gpu
def test_nan_and_infinity_make_the_block_nan():
    torch.cuda.set_device(0)
    for bad in (float("nan"), float("inf")):
        s = make([1024], F32, F32, 8, False)
        s["g"][0][300] = bad
        training.lora_adamw(_plan(s), step=3, **HYPER)
        after = cpu(s)
        for q, scale in (("m", "ms"), ("v", "vs")):
            x = dequantize(after[q][0], after[scale][0])
            assert not bool(x[256:512].isfinite().any()) and bool(x[:256].isfinite().all()) and bool(x[512:].isfinite().all())


def _follow(gradient, steps, betas, n=64 * 256):
    """The optimizer's (m, u) and the exact ones after some thousand steps."""
    torch.cuda.set_device(0)
    p = torch.zeros(n, device=DEV, requires_grad=True)
    p.grad = torch.zeros(n, device=DEV)
    opt = torch_ops.AdamW([p], lr=0.0, betas=betas, weight_decay=0.0, state_bits=8)
    m, v = (torch.zeros(n, device=DEV, dtype=torch.float64) for _ in range(2))
    gen = torch.Generator(DEV).manual_seed(0)
    for t in range(1, steps + 1):
        gradient(t, p.grad, gen)
        g = p.grad.double()
        m.mul_(betas[0]).add_(g, alpha=1 - betas[0])
        v.mul_(betas[1]).addcmul_(g, g, value=1 - betas[1])
        opt.step()
    value = lambda q, s: q[0].float().view(-1, 256).double() * s[0].double()[:, None]  # noqa: E731
    return (value(opt.exp_avg, opt.exp_avg_scale).view(-1), value(opt.exp_avg_sq, opt.exp_avg_sq_scale).view(-1), m,
            v.sqrt())


def _one_outlier(t, g, gen):
    g.normal_(generator=gen)
    if t == 300:
        g[::256] = 300.0


def _half_shrinks(t, g, gen):
    g.normal_(generator=gen)
    if t > 1000:
        g.view(-1, 256)[:, :128] /= 20.0


@pytest.mark.gpu
@pytest.mark.parametrize("gradient,steps", [(_one_outlier, 6000), (_half_shrinks, 10000)])
def test_u_follows_its_own_gradients(gradient, steps):
    """An element's u scatters about its value: a step moves it by some d = 0.0005 of itself, which
    the rounding makes a move of up to w = 1/8 with probability d / w (variance w d), and the
    average over 1 / 0.001 steps takes it back, so the relative variance is at most w d / 0.002 =
    0.177^2.  The median over 16384 elements lies within 5 % (a skewed scatter moves it by less
    than 0.177^2), and 1 % of them are off by more than three deviations at most."""
    _, u, _, want = _follow(gradient, steps, (0.9, 0.999))
    u, want = u.view(-1, 256)[:, 1:], want.view(-1, 256)[:, 1:]      # the outlier's own elements aside
    for part in (slice(0, 127), slice(127, 255)):
        ratio = (u / want)[:, part].flatten()
        low, mid, high = (float(ratio.quantile(q)) for q in (0.01, 0.5, 0.99))
        assert 0.95 < mid < 1.05 and low > 0.55 and high < 1.75, (low, mid, high)


@pytest.mark.gpu
def test_m_follows_its_own_gradients():
    """Gradients that halve in half of a block, beta1 = 0.99: m comes to lie on one of the two codes
    around its value, at most 1/8 of it apart."""
    def gradient(t, g, gen):
        g.fill_(1.0)
        if t > 500:
            g.view(-1, 256)[:, :128] = 0.47

    m, _, want, _ = _follow(gradient, 3000, (0.99, 0.999))
    assert float(((m - want).abs() / want).max()) <= 0.126

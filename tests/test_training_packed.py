"""Large tensors packed without padding, so off every 16-byte boundary: element by element, the
step and the norm give what they give on aligned tensors, bit for bit (the same values go to the
same lanes), and the norm of packed gradients to the rounding of its sums."""
import math

import pytest
import torch

from lora_rank_adapter_gb300 import _build, training

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SIZES = [1000003, 4099, 2500001, 1, 777777]


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    torch.cuda.set_device(0)


def _lay(values, dtype, packed):
    """The values in tensors of their own, or one after the other behind one odd element."""
    if not packed:
        return [v.to(dtype).to(DEV) for v in values], None
    flat = torch.full((1 + sum(v.numel() for v in values) + 5,), 3.0).to(dtype).to(DEV)
    views, at = [], 1
    for v in values:
        views.append(flat[at:at + v.numel()])
        views[-1].copy_(v.to(dtype))
        at += v.numel()
    return views, flat


@pytest.mark.parametrize("param,grad,master", [(F32, F32, False), (BF16, F32, True), (BF16, BF16, False)])
@pytest.mark.parametrize("bits,stochastic", [(32, False), (8, False), (8, True)])
def test_packed_as_aligned(param, grad, master, bits, stochastic):
    g = torch.Generator().manual_seed(0)
    rand = lambda scale: [torch.randn(n, generator=g) * scale for n in SIZES]  # noqa: E731
    values = {"p": rand(0.05), "g": rand(1e-2), "m": rand(1e-3), "v": [t.abs() for t in rand(1e-2)]}
    results = []
    for packed in (False, True):
        state = F32 if bits == 32 else E4M3
        s, flats = {}, []
        for k, dt in (("p", param), ("g", grad), ("m", state), ("v", state)) + ((("w", F32),) if master else ()):
            scale = 100.0 if bits == 8 and k in "mv" else 1.0
            s[k], flat = _lay([t * scale for t in values["p" if k == "w" else k]], dt, packed)
            flats.append(flat)
        scales = [[torch.full((-(-n // 256),), 1e-2, device=DEV) for n in SIZES] for _ in range(2)] if bits == 8 else [None] * 2
        plan = training.lora_adamw_plan(s["p"], s["g"], s["m"], s["v"], masters=s.get("w"), exp_avg_scales=scales[0],
                                        exp_avg_sq_scales=scales[1], stochastic=stochastic)
        norm = torch.empty(2, device=DEV)
        for step in (1, 2):
            training.lora_grad_norm(plan, 1.0, norm)
            training.lora_adamw(plan, lr=1e-2, step=step, grad_factor=norm[1:])
        want = math.sqrt(sum(float(t.double().square().sum()) for t in s["g"]))
        assert abs(float(norm[0]) - want) <= 2.0 ** -21 * want
        for flat in flats:
            if flat is not None:
                assert float(flat[0]) == 3.0 and bool((flat[-5:].float() == 3.0).all())
        results.append(sum((s[k] for k in s if k != "g"), []) + [norm] + sum((x or [] for x in scales), []))
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.clone().view(torch.uint8))

"""What is measured of the training operators beside the adapter product: the log-probabilities of
labels with their gradient, the preference loss and the clipped policy loss with theirs, and the
AdamW step over an adapter's many tensors with states in 32 or in 8 bits.

`own` chooses between the plain form of an operator (elementary torch operations in 32 bits) and the
calls that a user makes of lora_rank_adapter_gb300.training; both take the state that prepare() makes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 256            # elements of an 8-bit state that share one scale
TOP = 448.0            # largest e4m3 value
LEAST = 2.0 ** -9      # smallest positive e4m3 value
TINY = 1e-30           # a block's largest magnitude counts as at least this
ADAM = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
MODULES = "4096x4096,4096x1024,4096x1024,4096x4096,4096x14336,4096x14336,14336x4096"   # in x out of one layer


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a few answer tokens of one sequence scored in fp32, with a vocabulary of odd size (latency counts)
        {"name": "logps_few", "op": "logps", "T": 7, "V": 32003, "type": "f32", "grad": False, "temperature": 0.7,
         "prompt": 0.0, "stride_pad": 0, "masked": 3},
        # a supervised step: prompts ignored, gradient of every token's log-probability, padded vocabulary columns
        {"name": "logps_supervised", "op": "logps", "T": 4096, "V": 128256, "type": "bf16", "grad": True,
         "temperature": 1.0, "prompt": 0.4, "stride_pad": 0, "masked": 56},
        # one pair of short answers
        {"name": "preference_one_pair", "op": "preference", "P": 1, "length": 24, "V": 32000, "type": "bf16",
         "kind": "sigmoid", "smoothing": 0.0, "normalize": False, "temperature": 1.0, "prompt": 0.3, "stride_pad": 0,
         "masked": 0, "lengths": 1},
        # four ragged pairs in fp32, rows of odd size and so off every 16-byte boundary, length-normalised
        {"name": "preference_ragged_f32", "op": "preference", "P": 4, "length": 190, "V": 50001, "type": "f32",
         "kind": "ipo", "smoothing": 0.0, "normalize": True, "temperature": 1.0, "prompt": 0.25, "stride_pad": 0,
         "masked": 0, "lengths": 2},
        # a full batch of eight pairs of about 512 tokens over a large vocabulary
        {"name": "preference_batch", "op": "preference", "P": 8, "length": 512, "V": 128256, "type": "bf16",
         "kind": "sigmoid", "smoothing": 0.1, "normalize": False, "temperature": 1.0, "prompt": 0.3, "stride_pad": 0,
         "masked": 0, "lengths": 3},
        # a short rollout: one answer of 48 tokens
        {"name": "policy_short", "op": "policy", "B": 1, "length": 48, "V": 128256, "type": "bf16", "temperature": 1.0,
         "kl": 0.04, "prompt": 0.0, "stride_pad": 0, "masked": 0, "lengths": 4},
        # ragged rollouts in fp32 with padded rows, no KL term, sampled at a temperature
        {"name": "policy_ragged_f32", "op": "policy", "B": 6, "length": 333, "V": 32001, "type": "f32",
         "temperature": 0.8, "kl": 0.0, "prompt": 0.2, "stride_pad": 7, "masked": 1, "lengths": 5},
        # a group of sixteen rollouts of about 512 tokens over a large vocabulary
        {"name": "policy_group", "op": "policy", "B": 16, "length": 512, "V": 128256, "type": "bf16",
         "temperature": 1.0, "kl": 0.04, "prompt": 0.2, "stride_pad": 0, "masked": 0, "lengths": 6},
        # one adapted layer of odd sizes packed without padding, fp32 throughout, with clipping
        {"name": "adamw32_one_layer", "op": "adamw", "bits": 32, "layers": 1, "rank": 8, "modules": "512x512,511x515",
         "param": "f32", "grad": "f32", "master": False, "clip": True, "pad": 1},
        # every linear of 32 layers at rank 64: bf16 adapters with fp32 masters, fp32 gradients, clipping
        {"name": "adamw32_all_layers", "op": "adamw", "bits": 32, "layers": 32, "rank": 64, "modules": MODULES,
         "param": "bf16", "grad": "f32", "master": True, "clip": True, "pad": 256},
        # two layers of odd sizes with states in 8 bits
        {"name": "adamw8_odd", "op": "adamw", "bits": 8, "layers": 2, "rank": 16, "modules": "4096x4096,1000x1023",
         "param": "f32", "grad": "f32", "master": False, "clip": False, "pad": 256},
        # every linear of 32 layers at rank 64, bf16 adapters and gradients, states in 8 bits
        {"name": "adamw8_all_layers", "op": "adamw", "bits": 8, "layers": 32, "rank": 64, "modules": MODULES,
         "param": "bf16", "grad": "bf16", "master": False, "clip": False, "pad": 256},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logps", "preference", "policy", "adamw"])
    if op == "adamw":
        bits = rng.choice([32, 8])
        dims = [rng.choice([_log_int(rng, 64, 16384) | 1, 64 * (_log_int(rng, 1, 224) | 1)]) for _ in range(4)]
        case = {"op": op, "bits": bits, "layers": _log_int(rng, 1, 32), "rank": _log_int(rng, 1, 128),
                "modules": "%dx%d,%dx%d" % tuple(dims), "param": rng.choice(["bf16", "f32"]),
                "grad": rng.choice(["bf16", "f32"]), "master": rng.random() < 0.3,
                "clip": bits == 32 and rng.random() < 0.5, "pad": 256 if bits == 8 else rng.choice([1, 256])}
        while work(case)["bytes"] > 4e9 and case["rank"] > 1:
            case["rank"] //= 2
        return case
    kind = rng.choice(["bf16", "bf16", "f32"])
    V = rng.choice([_log_int(rng, 250, 131071) | 1, 64 * (_log_int(rng, 4, 2047) | 1), 128256])
    most = int(1.9e9 // (V * (2 if kind == "bf16" else 4)))   # rows
    case = {"op": op, "V": V, "type": kind, "temperature": rng.choice([1.0, 1.0, 0.7, 1.3]),
            "prompt": rng.choice([0.0, 0.2, 0.5]), "stride_pad": rng.choice([0, 0, 5, 64]),
            "masked": rng.choice([0, 0, 1, 17])}
    if op == "logps":
        case.update(T=_log_int(rng, 1, min(most, 8192)) | 1, grad=rng.random() < 0.5)
    elif op == "preference":
        P = _log_int(rng, 1, 16)
        case.update(P=P, length=_log_int(rng, 2, max(2, min(1024, most // (4 * P)))),
                    kind=rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"]), smoothing=rng.choice([0.0, 0.1]),
                    normalize=rng.random() < 0.3, lengths=rng.randrange(1000))
    else:
        B = _log_int(rng, 1, 32)
        case.update(B=B, length=_log_int(rng, 2, max(2, min(1024, most // (2 * B)))), kl=rng.choice([0.0, 0.04]),
                    lengths=rng.randrange(1000))
    return case


def _sequences(case):
    """Lengths of the packed sequences and of their prompts, whose tokens are ignored: by the case alone."""
    rng = random.Random(case["lengths"])
    n = 2 * case["P"] if case["op"] == "preference" else case["B"]
    lens = [max(1, int(case["length"] * rng.uniform(0.4, 1.6))) for _ in range(n)]
    return lens, [int(case["prompt"] * k) for k in lens]


def _rows(case):
    """(rows of logits, rows whose label counts)"""
    if case["op"] == "logps":
        ignored = int(case["prompt"] * case["T"])
        return case["T"], case["T"] - ignored
    lens, prompts = _sequences(case)
    return sum(lens), sum(lens) - sum(prompts)


def _numels(case):
    found = []
    for _ in range(case["layers"]):
        for m in case["modules"].split(","):
            k, l = (int(v) for v in m.split("x"))
            found += [(case["rank"], k), (l, case["rank"])]
    return found


def work(case):
    if case["op"] == "adamw":
        n = sum(a * b for a, b in _numels(case))
        p, g = (2 if case[k] == "bf16" else 4 for k in ("param", "grad"))
        per = (8 + p if case["master"] else 2 * p) + g + (16 if case["bits"] == 32 else 4 + 16.0 / BLOCK)
        return {"bytes": n * per, "flops": 16.0 * n}
    T, valid = _rows(case)
    e, V = (2 if case["type"] == "bf16" else 4), case["V"]
    grad = case["op"] != "logps" or case["grad"]
    b = valid * V * e + T * 12.0
    if grad:
        b += T * V * float(e)
    if case["op"] == "policy":
        b += T * 16.0
    return {"bytes": float(b), "flops": valid * V * (10.0 if grad else 5.0)}


# ------------------------------------------------------------------------------------------- inputs
def _logits(case, T, gen):
    """Logits as a model gives them: the label a few units above a spread of 2, some columns masked out."""
    V, dt = case["V"], TYPES[case["type"]]
    full = torch.empty((T, V + case["stride_pad"]), dtype=dt, device=DEV)
    full.normal_(0.0, 2.0, generator=gen)
    x = full[:, :V]
    labels = torch.randint(0, V - case["masked"], (T,), generator=gen, device=DEV)
    lift = (math.log(V) + 1.0 + 2.0 * torch.randn((T, 1), generator=gen, device=DEV)).to(dt)
    x.scatter_add_(1, labels[:, None], lift)
    if case["masked"]:      # half of the masked columns at the type's lowest value, half at minus infinity
        k = case["masked"]
        x[:, V - k:] = torch.finfo(dt).min
        x[:, V - k // 2:] = -math.inf
    return x, labels


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    return _prepare_adamw(case, gen) if case["op"] == "adamw" else _prepare_loss(case, gen)


def _prepare_loss(case, gen):
    T, valid = _rows(case)
    x, labels = _logits(case, T, gen)
    s = {"case": case, "logits": x, "logps": torch.empty(T, device=DEV)}
    if case["op"] == "logps":
        labels[:T - valid] = -100
        s["labels"] = labels
        if case["grad"]:
            s["dlogps"] = -torch.rand(T, generator=gen, device=DEV) / max(1, valid)
            s["stats"] = torch.empty((T, 2), device=DEV)
            s["dlogits"] = torch.empty_like(x)
        return s
    lens, prompts = _sequences(case)
    cu = [0]
    for k in lens:
        cu.append(cu[-1] + k)
    ignored = torch.zeros(T, dtype=torch.bool)
    for start, k in zip(cu, prompts):
        ignored[start:start + k] = True
    labels[ignored.to(DEV)] = -100
    s.update(labels=labels, longest=max(lens), dlogits=torch.empty_like(x),
             cu=torch.tensor(cu, dtype=torch.int32, device=DEV))
    valid_rows = (labels >= 0).nonzero()[:, 0]
    near = torch.zeros(T, device=DEV)        # about the model's own log-probabilities
    for rows in valid_rows.split(1024):
        near[rows] = _logp_rows(x[rows], labels[rows], case["temperature"])[0]
    if case["op"] == "preference":
        P = case["P"]
        S = _by_sequence(near, s["cu"], s["longest"])
        n = _by_sequence((labels >= 0).float(), s["cu"], s["longest"]).clamp(min=1)
        ref = S / n if case["normalize"] else S
        s.update(ref=ref + torch.randn(2 * P, generator=gen, device=DEV) * (0.3 if case["normalize"] else 3.0),
                 seq_logps=torch.empty(2 * P, device=DEV), pair_loss=torch.empty(P, device=DEV),
                 loss=torch.empty(1, device=DEV), beta=0.1)
    else:
        # The policy moved a little since the rollout. The gradient jumps where the ratio meets a clip bound:
        # ratios stay off the two bounds by a thousandth, so that the last bit of a sum decides none of them.
        r = torch.exp(0.15 * torch.randn(T, generator=gen, device=DEV))
        for bound in (0.8, 1.28):
            r = torch.where((r - bound).abs() < 2e-3, r * 0.99, r)
        lens_t = torch.tensor(lens, dtype=torch.float32, device=DEV).repeat_interleave(torch.tensor(lens, device=DEV))
        s.update(old=near - r.log(), ref=near + 0.3 * torch.randn(T, generator=gen, device=DEV),
                 adv=torch.randn(len(lens), generator=gen, device=DEV).repeat_interleave(torch.tensor(lens, device=DEV)),
                 weights=1.0 / (lens_t * len(lens)), metrics=torch.empty(3, device=DEV), clip_low=0.2, clip_high=0.28)
    return s


def _quantize(x, least=0.0):
    """(codes, scales) of a [blocks, BLOCK] fp32 tensor; `least`: what a positive value rounds to at the least."""
    top = x.abs().amax(1).clamp(min=TINY)
    q = x * torch.div(torch.full_like(top, TOP), top)[:, None]
    if least:
        q = torch.where(x > 0, q.clamp(min=least), q)
    return q.to(torch.float8_e4m3fn), top * (1.0 / TOP)


def _prepare_adamw(case, gen):
    shapes, at, n = _numels(case), [], 0
    for a, b in shapes:
        at.append(n)
        n += -(-(a * b) // case["pad"]) * case["pad"]
    # one flat buffer for each kind, as trainers keep them; the tensors are views, any padding between them is zero
    real = torch.zeros(n, dtype=torch.bool)
    if case["pad"] == 1:
        real[:] = True
    else:
        for (a, b), o in zip(shapes, at):
            real[o:o + a * b] = True
    real = real.to(DEV)

    def fill(scale, dtype=torch.float32):
        return torch.where(real, torch.empty(n, device=DEV).normal_(0.0, scale, generator=gen), 0.0).to(dtype)

    views = lambda flat: [flat[o:o + a * b].view(a, b) for (a, b), o in zip(shapes, at)]  # noqa: E731
    s = {"case": case, "step": 100, "flat": {}}
    master = fill(0.02)
    f = s["flat"]
    f["p"] = master.to(TYPES[case["param"]])
    f["g"] = fill(1e-3, TYPES[case["grad"]])
    f["g"] *= torch.where(torch.rand(n, generator=gen, device=DEV) < 0.01, 30.0, 1.0).to(f["g"].dtype)
    m, u = fill(1e-4), fill(3e-4).abs()
    if case["master"]:
        f["master"] = master
    if case["bits"] == 32:
        f["m"], f["v"] = m, u * u
        names = ("m", "v")
    else:
        f["m"], f["m_scale"] = _quantize(m.view(-1, BLOCK))
        f["v"], f["v_scale"] = _quantize(u.view(-1, BLOCK), LEAST)
        f["m"], f["v"] = f["m"].view(-1), f["v"].view(-1)
        names = ("m", "v")
    del m, u
    s["factor"] = torch.full((1,), 0.37, device=DEV)        # what the gradients are scaled by where the step does not clip
    s["norm"] = torch.empty(2, device=DEV)
    s["tensors"] = {k: views(f[k]) for k in ("p", "g") + names + (("master",) if case["master"] else ())}
    if case["bits"] == 8:
        for k in ("m_scale", "v_scale"):
            s["tensors"][k] = [f[k][o // BLOCK:o // BLOCK + -(-(a * b) // BLOCK)] for (a, b), o in zip(shapes, at)]
    if own:
        from lora_rank_adapter_gb300 import training
        t = s["tensors"]
        s["plan"] = training.lora_adamw_plan(t["p"], t["g"], t["m"], t["v"], masters=t.get("master"),
                                             exp_avg_scales=t.get("m_scale"), exp_avg_sq_scales=t.get("v_scale"))
    return s


# ------------------------------------------------------------------------------------------- plain forms
def _logp_rows(logits, labels, temperature):
    x = logits.float()
    if temperature != 1.0:
        x = x / temperature
    top = x.amax(1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    ok = (labels >= 0) & (labels < logits.shape[1])
    at = torch.where(ok, labels, 0)[:, None]
    logp = (x.gather(1, at) - top - total.log())[:, 0]
    return torch.where(ok, logp, 0.0), e, total, ok, at


def _dlogits(e, total, ok, at, dlogp, temperature, dtype):
    c = torch.where(ok, dlogp, 0.0)[:, None]
    if temperature != 1.0:
        c = c / temperature
    d = e * (-c / total)
    return d.scatter_add_(1, at, c).to(dtype)


def _by_sequence(values, cu, longest):
    at = cu[:-1, None].long() + torch.arange(longest, device=cu.device)
    inside = at < cu[1:, None]
    return torch.where(inside, values[torch.where(inside, at, 0)], 0.0).sum(1)


def _log_sigmoid(h):
    return torch.clamp(h, max=0.0) - torch.log1p(torch.exp(-h.abs()))


def _plain_preference(s):
    case, P = s["case"], s["case"]["P"]
    logp, e, total, ok, at = _logp_rows(s["logits"], s["labels"], case["temperature"])
    S = _by_sequence(logp, s["cu"], s["longest"])
    n = torch.ones_like(S)
    if case["normalize"]:
        n = _by_sequence(ok.float(), s["cu"], s["longest"]).clamp(min=1)
        S = S / n
    d = (S[:P] - S[P:]) - (s["ref"][:P] - s["ref"][P:])
    beta, eps = s["beta"], case["smoothing"]
    if case["kind"] == "sigmoid":
        h = beta * d
        pair = -(1 - eps) * _log_sigmoid(h) - eps * _log_sigmoid(-h)
        slope = beta * (1 / (1 + torch.exp(-h)) - (1 - eps))
    elif case["kind"] == "hinge":
        pair = torch.clamp(1 - beta * d, min=0.0)
        slope = torch.where(1 - beta * d > 0, -beta, 0.0)
    else:
        pair = (d - 0.5 / beta) ** 2
        slope = 2 * (d - 0.5 / beta)
    each = torch.cat([slope, -slope]) / P / n
    seq = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(logp.numel(), device=DEV, dtype=torch.int32), right=True)
    dl = _dlogits(e, total, ok, at, each[seq], case["temperature"], s["logits"].dtype)
    return {"loss": pair.mean()[None], "pair_loss": pair, "seq_logps": S, "logps": logp, "dlogits": dl}


def _plain_policy(s):
    case = s["case"]
    logp, e, total, ok, at = _logp_rows(s["logits"], s["labels"], case["temperature"])
    r = torch.exp(logp - s["old"])
    lo, hi = 1 - s["clip_low"], 1 + s["clip_high"]
    adv, w = s["adv"], torch.where(ok, s["weights"], 0.0)
    pg = -torch.minimum(r * adv, torch.clamp(r, lo, hi) * adv)
    clipped = ((adv > 0) & (r > hi)) | ((adv < 0) & (r < lo))
    c = torch.where(clipped, 0.0, -adv * r)
    kl = torch.zeros_like(pg)
    if case["kl"]:
        d = s["ref"] - logp
        kl = torch.exp(d) - d - 1
        c = c + case["kl"] * (1 - torch.exp(d))
    dl = _dlogits(e, total, ok, at, w * c, case["temperature"], s["logits"].dtype)
    metrics = torch.stack([(w * (pg + case["kl"] * kl)).sum(), (w * kl).sum(), (w * clipped.float()).sum()])
    return {"metrics": metrics, "logps": logp, "dlogits": dl}


def _plain_adamw(s):
    case, f, a = s["case"], s["flat"], ADAM
    s["step"] += 1
    g = f["g"].float()
    if case["clip"]:
        norm = (g * g).sum().sqrt()
        s["norm"][0] = norm
        s["norm"][1] = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
        g = g * s["norm"][1]
    else:
        g = g * s["factor"][0]
    bc1, bc2 = 1 - a["beta1"] ** s["step"], 1 - a["beta2"] ** s["step"]
    if case["bits"] == 32:
        m, v = f["m"], f["v"]
    else:
        m = (f["m"].float().view(-1, BLOCK) * f["m_scale"][:, None]).view(-1)
        v = (f["v"].float().view(-1, BLOCK) * f["v_scale"][:, None]).view(-1)
        v = v * v
    m = m * a["beta1"] + g * (1 - a["beta1"])
    v = v * a["beta2"] + (g * g) * (1 - a["beta2"])
    u = v.sqrt()
    p = f["master"] if case["master"] else f["p"].float()
    p = p * (1 - a["lr"] * a["weight_decay"]) - (a["lr"] / bc1) * (m / (u * (1 / math.sqrt(bc2)) + a["eps"]))
    f["p"].copy_(p)
    if case["master"]:
        f["master"].copy_(p)
    if case["bits"] == 32:
        f["m"].copy_(m)
        f["v"].copy_(v)
    else:
        q, scale = _quantize(m.view(-1, BLOCK))
        f["m"].copy_(q.view(-1))
        f["m_scale"].copy_(scale)
        q, scale = _quantize(u.view(-1, BLOCK), LEAST)
        f["v"].copy_(q.view(-1))
        f["v_scale"].copy_(scale)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = {k: v for k, v in s["flat"].items() if k != "g"}
    if s["case"]["clip"]:
        out["norm"] = s["norm"]
    return out


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "adamw":
            return _plain_adamw(state)
        if case["op"] == "preference":
            return _plain_preference(state)
        if case["op"] == "policy":
            return _plain_policy(state)
        logp, e, total, ok, at = _logp_rows(state["logits"], state["labels"], case["temperature"])
        if not case["grad"]:
            return {"logps": logp}
        return {"logps": logp, "dlogits": _dlogits(e, total, ok, at, state["dlogps"], case["temperature"],
                                                   state["logits"].dtype)}
    from lora_rank_adapter_gb300 import training
    s = state
    if case["op"] == "adamw":
        s["step"] += 1
        factor = s["factor"]
        if case["clip"]:
            training.lora_grad_norm(s["plan"], 1.0, s["norm"])
            factor = s["norm"][1:]
        training.lora_adamw(s["plan"], step=s["step"], grad_factor=factor, **ADAM)
        return _adamw_outputs(s)
    if case["op"] == "logps":
        training.lora_token_logps(s["logits"], s["labels"], s["logps"], temperature=case["temperature"],
                                  stats=s.get("stats"))
        if not case["grad"]:
            return {"logps": s["logps"]}
        training.lora_token_logps_backward(s["logits"], s["labels"], s["stats"], s["dlogps"], s["dlogits"],
                                           temperature=case["temperature"])
        return {"logps": s["logps"], "dlogits": s["dlogits"]}
    if case["op"] == "preference":
        training.lora_preference_loss(s["logits"], s["labels"], s["cu"], s["ref"], s["beta"], s["logps"],
                                      s["seq_logps"], s["pair_loss"], s["loss"], dlogits=s["dlogits"],
                                      kind=case["kind"], label_smoothing=case["smoothing"],
                                      length_normalize=case["normalize"], temperature=case["temperature"])
        return {"loss": s["loss"], "pair_loss": s["pair_loss"], "seq_logps": s["seq_logps"], "logps": s["logps"],
                "dlogits": s["dlogits"]}
    training.lora_policy_loss(s["logits"], s["labels"], s["old"], s["adv"], s["weights"], s["logps"], s["metrics"],
                              ref_logps=s["ref"] if case["kl"] else None, dlogits=s["dlogits"],
                              clip_low=s["clip_low"], clip_high=s["clip_high"], kl_beta=case["kl"],
                              temperature=case["temperature"])
    return {"metrics": s["metrics"], "logps": s["logps"], "dlogits": s["dlogits"]}


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_loss(s)


def _exact_loss(s):
    case, x, labels = s["case"], s["logits"], s["labels"]
    T, V = x.shape
    temp = case["temperature"]
    ok = ((labels >= 0) & (labels < V)).tolist()
    spans = [(i, min(i + 512, T)) for i in range(0, T, 512)]
    logp, lse = torch.zeros(T, dtype=torch.float64, device=DEV), torch.zeros(T, dtype=torch.float64, device=DEV)
    keep = torch.tensor(ok, device=DEV)
    for i, j in spans:
        z = x[i:j].double() / temp
        lse[i:j] = torch.logsumexp(z, 1)
        picked = z[torch.arange(j - i, device=DEV), labels[i:j].clamp(0, V - 1)]
        logp[i:j] = torch.where(keep[i:j], picked - lse[i:j], torch.zeros_like(picked))
    out = {"logps": logp}
    if case["op"] == "logps":
        if not case["grad"]:
            return out
        coef = s["dlogps"].double()
    elif case["op"] == "preference":
        P, cu = case["P"], s["cu"].tolist()
        S, n = [], []
        for i in range(2 * P):
            count = sum(ok[cu[i]:cu[i + 1]])
            n.append(max(1, count) if case["normalize"] else 1)
            S.append(float(logp[cu[i]:cu[i + 1]].sum()) / n[-1])
        ref, beta, eps = s["ref"].double().tolist(), s["beta"], case["smoothing"]
        pair, coef = [], torch.zeros(T, dtype=torch.float64, device=DEV)
        for p in range(P):
            d = (S[p] - S[P + p]) - (ref[p] - ref[P + p])
            if case["kind"] == "sigmoid":
                soft = lambda h: math.log1p(math.exp(-h)) if h > 0 else math.log1p(math.exp(h)) - h  # noqa: E731
                pair.append((1 - eps) * soft(beta * d) + eps * soft(-beta * d))
                slope = beta * (eps / (1 + math.exp(-beta * d)) - (1 - eps) / (1 + math.exp(beta * d)))
            elif case["kind"] == "hinge":
                pair.append(max(0.0, 1 - beta * d))
                slope = -beta if beta * d < 1 else 0.0
            else:
                pair.append((d - 1 / (2 * beta)) ** 2)
                slope = 2 * (d - 1 / (2 * beta))
            coef[cu[p]:cu[p + 1]] = slope / P / n[p]
            coef[cu[P + p]:cu[P + p + 1]] = -slope / P / n[P + p]
        as64 = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
        out.update(loss=as64([sum(pair) / P]), pair_loss=as64(pair), seq_logps=as64(S))
    else:
        w = torch.where(keep, s["weights"].double(), 0.0)
        adv, lo, hi, kl = s["adv"].double(), 1 - s["clip_low"], 1 + s["clip_high"], case["kl"]
        ratio = (logp - s["old"].double()).exp()
        free = torch.where(adv >= 0, ratio <= hi, ratio >= lo)
        bounded = torch.where(adv >= 0, ratio.clamp(max=hi), ratio.clamp(min=lo))
        coef, gap = -adv * ratio * free, s["ref"].double() - logp
        div = torch.expm1(gap) - gap if kl else torch.zeros_like(gap)
        if kl:
            coef = coef - kl * torch.expm1(gap)
        coef = coef * w
        out["metrics"] = torch.stack([(w * (kl * div - adv * bounded)).sum(), (w * div).sum(), (w * ~free).sum()])
    d = torch.zeros((T, V), dtype=torch.float64, device=DEV)
    for i, j in spans:
        soft = torch.exp(x[i:j].double() / temp - lse[i:j, None])
        c = torch.where(keep[i:j], coef[i:j], torch.zeros_like(coef[i:j])) / temp
        d[i:j] = -c[:, None] * soft
        d[torch.arange(i, j, device=DEV), labels[i:j].clamp(0, V - 1)] += c
    out["dlogits"] = d
    return out


def _e4m3(x):
    """The nearest value of sign, 4 exponent bits and 3 of mantissa, halves to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_adamw(s):
    case, a = s["case"], ADAM
    f = {k: v.double() for k, v in s["flat"].items()}
    step, out = s["step"] + 1, {}
    factor = 0.0
    if case["clip"]:
        norm = f["g"].square().sum().sqrt()
        factor = torch.clamp(1 / (norm + 1e-6), max=1)
        out["norm"] = torch.stack([norm, factor])
    else:
        factor = s["factor"].double()[0]
    g = f["g"] * factor
    if case["bits"] == 32:
        m, v = f["m"], f["v"]
    else:
        m = (f["m"].view(-1, BLOCK) * f["m_scale"][:, None]).view(-1)
        v = (f["v"].view(-1, BLOCK) * f["v_scale"][:, None]).view(-1).square()
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * g.square()
    denom = (v / (1 - a["beta2"] ** step)).sqrt() + a["eps"]
    p = f["master"] if case["master"] else f["p"]
    p = p - a["lr"] * a["weight_decay"] * p - a["lr"] * (m / (1 - a["beta1"] ** step)) / denom
    out["p"] = p
    if case["master"]:
        out["master"] = p
    if case["bits"] == 32:
        out.update(m=m, v=v)
        return out
    for name, x, least in (("m", m, 0.0), ("v", v.sqrt(), LEAST)):
        x = x.view(-1, BLOCK)
        top = x.abs().amax(1).clamp(min=TINY)
        q = x * (TOP / top)[:, None]
        if least:
            q = torch.where((x > 0) & (q < least), torch.full_like(q, least), q)
        out[name], out[name + "_scale"] = _e4m3(q).view(-1), top / TOP
    return out

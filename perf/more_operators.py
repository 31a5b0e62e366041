"""What is measured of the operators that record a model's most probable tokens and train on such a record:
log-probabilities of given tokens with entropy and top alternatives (lora_top_logps), their gradient, and
the distillation loss from a teacher's top tokens with its gradient (lora_distill_loss).

`own` chooses between the plain form of an operator (elementary torch operations in 32 bits) and the
calls that a user makes of lora_rank_adapter_gb300.training; both take the state that prepare() makes.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST = 1.6e9           # bytes of a drawn case's logits


# ------------------------------------------------------------------------------------------- cases
def _top(name, **more):
    case = {"name": name, "op": "top", "type": "bf16", "temperature": 1.0, "labels": True, "prompt": 0.0, "masked": 0,
            "allowed": 0, "stride_pad": 0, "grad": False}
    return {**case, **more}


def _distill(name, **more):
    case = {"name": name, "op": "distill", "type": "bf16", "temperature": 1.0, "kind": "forward", "rest": True,
            "ignored": 0.0, "masked": 0, "stride_pad": 0, "grad": True}
    return {**case, **more}


def listed():
    return [
        # one decoded token of one request with its alternatives (latency counts)
        _top("top_one_token", T=1, V=128256, K=20),
        # a decode batch in fp32, sampled at a temperature, some columns of the vocabulary masked out
        _top("top_decode_f32", T=48, V=32003, K=5, type="f32", temperature=0.7, masked=17),
        # a decode batch whose output is held to a grammar: a handful of tokens is allowed in each row
        _top("top_constrained", T=97, V=128256, K=20, allowed=11),
        # scoring a prompt: one alternative beside each token, odd rows off every 16-byte boundary, a third ignored
        _top("top_prompt_f32", T=2049, V=50001, K=1, type="f32", prompt=0.3),
        # the record of a teacher over a batch of sequences: no labels, 64 tokens a row
        _top("top_teacher", T=4096, V=128256, K=64, labels=False),
        # a policy step's entropy bonus: log-probabilities, entropies and their gradient
        _top("top_entropy_step", T=2731, V=128256, K=8, prompt=0.2, grad=True),
        # gradient through the alternatives too, in fp32 with rows of odd size and stride
        _top("top_step_f32", T=333, V=32001, K=17, type="f32", temperature=1.3, stride_pad=6, masked=3, grad=True),
        # a short answer distilled from eight tokens a row, without the rest
        _distill("distill_short", T=24, V=32000, K=8, rest=False),
        # many rows of a small vocabulary of odd size
        _distill("distill_small_vocabulary", T=8192, V=4099, K=16, ignored=0.1),
        # the student's divergence from its teacher in fp32 (reverse), ragged, at a temperature
        _distill("distill_reverse_f32", T=1501, V=50001, K=32, type="f32", kind="reverse", temperature=0.8, ignored=0.2,
                 masked=5, stride_pad=7),
        # evaluation: no gradient, the longest list
        _distill("distill_evaluate", T=2048, V=128256, K=128, grad=False, kind="reverse"),
        # a full batch of sequences over a large vocabulary, prompts ignored
        _distill("distill_batch", T=6001, V=128256, K=64, ignored=0.25),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["bf16", "bf16", "f32"])
    V = rng.choice([_log_int(rng, 300, 131071) | 1, 64 * (_log_int(rng, 5, 2047) | 1), 128256])
    most = int(MOST // (V * (2 if kind == "bf16" else 4)))
    common = {"T": _log_int(rng, 1, min(most, 8192)), "V": V, "K": _log_int(rng, 1, 128), "type": kind,
              "temperature": rng.choice([1.0, 1.0, 0.7, 1.3]), "masked": rng.choice([0, 0, 1, 17]),
              "stride_pad": rng.choice([0, 0, 5, 64]), "grad": rng.random() < 0.6}
    if rng.random() < 0.5:
        case = _top("", **common)
        case.update(labels=rng.random() < 0.7, allowed=0 if case["grad"] else rng.choice([0, 0, 0, 0, 11]))
        case["prompt"] = rng.choice([0.0, 0.2, 0.5]) if case["labels"] else 0.0
    else:
        case = _distill("", **common)
        case.update(kind=rng.choice(["forward", "forward", "reverse"]), rest=rng.random() < 0.6,
                    ignored=rng.choice([0.0, 0.2, 0.5]))
    del case["name"]
    return case


def _valid(case):
    return case["T"] - int((case["prompt"] if case["op"] == "top" else case["ignored"]) * case["T"])


def work(case):
    T, V, K, valid = case["T"], case["V"], case["K"], _valid(case)
    e = 2 if case["type"] == "bf16" else 4
    b = valid * V * float(e)
    if case["grad"]:
        b += T * V * float(e)
    if case["op"] == "top":
        b += T * (K * 12.0 + 8.0)                        # ids, log-probabilities, entropy, rest
        b += T * 12.0 if case["labels"] else 0.0         # label and its log-probability
        if case["grad"]:
            b += T * (4.0 * K + 8.0)
    else:
        b += T * (K * 12.0 + 8.0 + (4.0 if case["rest"] else 0.0))
    return {"bytes": b, "flops": valid * V * (12.0 if case["grad"] else 6.0)}


# ------------------------------------------------------------------------------------------- inputs
def _logits(case, gen):
    """Logits as a model gives them: the label a few units above a spread of 2, some columns masked out."""
    T, V, dt = case["T"], case["V"], TYPES[case["type"]]
    full = torch.empty((T, V + case["stride_pad"]), dtype=dt, device=DEV)
    full.normal_(0.0, 2.0, generator=gen)
    x = full[:, :V]
    labels = torch.randint(0, V - case["masked"], (T,), generator=gen, device=DEV)
    lift = (math.log(V) + 1.0 + 2.0 * torch.randn((T, 1), generator=gen, device=DEV)).to(dt)
    x.scatter_add_(1, labels[:, None], lift)
    k = case["masked"]
    if k:                   # half of the masked columns at the type's lowest value, half at minus infinity
        x[:, V - k:] = torch.finfo(dt).min
        x[:, V - k // 2:] = -math.inf
    if case.get("allowed"):
        at = torch.randint(0, V - k, (T, case["allowed"]), generator=gen, device=DEV)
        at[:, 0] = labels
        kept = x.gather(1, at)
        x.fill_(-math.inf)
        x.scatter_(1, at, kept)
    return x, labels


def _record(x, case, gen):
    """A teacher's most probable tokens: near the student, but not the same."""
    T, K, V = case["T"], case["K"], case["V"]
    ids = torch.empty((T, K), dtype=torch.int64, device=DEV)
    logps, rest = torch.empty((T, K), device=DEV), torch.empty(T, device=DEV)
    for i in range(0, T, 1024):
        z = x[i:i + 1024].float() / case["temperature"]
        z += 0.5 * torch.randn(z.shape, generator=gen, device=DEV)
        z -= z.logsumexp(1, keepdim=True)
        logps[i:i + 1024], ids[i:i + 1024] = z.topk(K, 1)
        z.scatter_(1, ids[i:i + 1024], -math.inf)
        rest[i:i + 1024] = z.logsumexp(1)
    # some rows were recorded with half as many tokens (the others' mass is not known then: it stays out of the rest)
    few = torch.rand(T, generator=gen, device=DEV) < 0.1
    ids[few, (K + 1) // 2:] = -1
    return ids, logps, rest


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    T, K = case["T"], case["K"]
    x, labels = _logits(case, gen)
    valid = _valid(case)
    f32 = lambda *shape: torch.empty(shape, device=DEV)  # noqa: E731
    s = {"case": case, "logits": x}
    if case["op"] == "top":
        labels[:T - valid] = -100
        s.update(labels=labels if case["labels"] else None, logps=f32(T) if case["labels"] else None, entropy=f32(T),
                 top_ids=torch.empty((T, K), dtype=torch.int64, device=DEV), top_logps=f32(T, K), rest=f32(T))
        if case["grad"]:
            s["dlogps"] = torch.randn(T, generator=gen, device=DEV) / T if case["labels"] else None
            s["dentropy"] = -0.01 * (1 + torch.rand(T, generator=gen, device=DEV)) / T
            s["dtop"] = 0.1 * torch.randn((T, K), generator=gen, device=DEV) / (T * K)
            s.update(stats=f32(T, 2), dlogits=torch.empty_like(x))
        return s
    ids, logps, rest = _record(x, case, gen)
    weights = torch.full((T,), 1.0 / max(1, valid), device=DEV)
    off = torch.randperm(T, generator=gen, device=DEV)[:T - valid]
    weights[off[::2]] = 0.0             # half of the ignored rows by their weight, half by an empty list
    ids[off[1::2]] = -1
    s.update(ids=ids, teacher=logps, rest=rest if case["rest"] else None, weights=weights, row_loss=f32(T), loss=f32(1))
    s["dlogits"] = torch.empty_like(x) if case["grad"] else None
    return s


# ------------------------------------------------------------------------------------------- plain forms
def _softmax(logits, temperature):
    """(z, its largest, exp(z - largest), their sum)"""
    z = logits.float()
    if temperature != 1.0:
        z = z / temperature
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    return z, top, e, e.sum(1, keepdim=True)


def _largest(logits, K):
    """Places of a row's K largest values, ties to the lowest place: keys that order by value, then by place."""
    bits = (logits.float() + 0.0).view(torch.int32)
    key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() << 32
    key |= 0xFFFFFFFF - torch.arange(logits.shape[1], device=DEV)
    return 0xFFFFFFFF - (key.topk(K, 1)[0] & 0xFFFFFFFF)


def _plain_top(s):
    case, x, labels = s["case"], s["logits"], s["labels"]
    T, V = x.shape
    z, top, e, total = _softmax(x, case["temperature"])
    ids = _largest(x, case["K"])
    log_total = total.log()
    lnp = z - top - log_total
    p = e / total
    entropy = -torch.where(p > 0, p * lnp, 0.0).sum(1)
    top_logps = lnp.gather(1, ids)
    rest = e.scatter(1, ids, 0.0).sum(1).log() - log_total[:, 0]
    ids = torch.where(top_logps == -math.inf, -1, ids)
    out = {"entropy": entropy, "top_ids": ids, "top_logps": top_logps, "rest": rest}
    ok = torch.ones(T, dtype=torch.bool, device=DEV)
    if labels is not None:
        ok = (labels >= 0) & (labels < V)
        at = torch.where(ok, labels, 0)[:, None]
        out = {"entropy": torch.where(ok, entropy, 0.0), "top_ids": torch.where(ok[:, None], ids, -1),
               "top_logps": torch.where(ok[:, None], top_logps, -math.inf), "rest": torch.where(ok, rest, 0.0),
               "logps": torch.where(ok, lnp.gather(1, at)[:, 0], 0.0)}
    if not case["grad"]:
        return out
    there = (ids >= 0) & ok[:, None]
    g = torch.where(there, s["dtop"], 0.0)
    gH = torch.where(ok, s["dentropy"], 0.0)[:, None]
    total_g = g.sum(1, keepdim=True)
    if labels is not None:
        gl = torch.where(ok, s["dlogps"], 0.0)[:, None]
        total_g = total_g + gl
    d = -p * (total_g + gH * torch.where(p > 0, lnp + entropy[:, None], 0.0))
    d = torch.where(ok[:, None], d, 0.0)
    d.scatter_add_(1, torch.where(there, ids, 0), g)
    if labels is not None:
        d.scatter_add_(1, at, gl)
    out["dlogits"] = (d / case["temperature"]).to(x.dtype)
    return out


def _plain_distill(s):
    case, x, ids = s["case"], s["logits"], s["ids"]
    z, top, e, total = _softmax(x, case["temperature"])
    log_total = total.log()
    there = (ids >= 0) & (ids < x.shape[1])
    ok = there.any(1) & (s["weights"] != 0)
    at = torch.where(there, ids, torch.where(there[:, :1], ids[:, :1], 0))   # the first entry is there wherever one is
    lnp = z.gather(1, at) - top - log_total
    p = lnp.exp()
    lnq = s["teacher"]
    q = torch.where(there, lnq.exp(), 0.0)
    forward = case["kind"] == "forward"
    gap = lnp - lnq
    terms = torch.where(there, -q * gap if forward else torch.where(p > 0, p * gap, 0.0), 0.0)
    L = terms.sum(1, keepdim=True)
    Q = q.sum(1, keepdim=True)
    P = torch.where(there, p, 0.0).sum(1, keepdim=True)
    e = e.scatter_(1, at, 0.0)                                   # of the tokens that are not listed
    rest = e.sum(1, keepdim=True)
    pr = rest / total
    if case["rest"]:
        lnqr = s["rest"][:, None]
        gap_r = rest.log() - log_total - lnqr
        qr = lnqr.exp()
        if forward:
            L = L - torch.where(qr > 0, qr * gap_r, 0.0)
            Q = Q + qr
            f = (Q * pr - qr) / rest
        else:
            L = L + torch.where(pr > 0, pr * gap_r, 0.0)
            f = (gap_r - L) / total
    else:
        f = Q / total if forward else -(L + P) / total
    row_loss = torch.where(ok, L[:, 0], 0.0)
    out = {"row_loss": row_loss, "loss": (s["weights"] * row_loss).sum()[None]}
    if not case["grad"]:
        return out
    if forward:
        dj = p * Q - q
    elif case["rest"]:
        dj = p * (gap - L)
    else:
        dj = p * (gap + 1 - L - P)
    c = torch.where(ok, s["weights"], 0.0)[:, None] / case["temperature"]
    d = torch.where(ok[:, None], e * torch.where(rest > 0, f * c, 0.0), 0.0)
    d.scatter_add_(1, at, torch.where(there & ok[:, None], dj * c, 0.0))
    out["dlogits"] = d.to(x.dtype)
    return out


def run(state):
    s, case = state, state["case"]
    if not own:
        return _plain_top(s) if case["op"] == "top" else _plain_distill(s)
    from lora_rank_adapter_gb300 import training
    if case["op"] == "top":
        training.lora_top_logps(s["logits"], s["top_ids"], s["top_logps"], labels=s["labels"], logps=s["logps"],
                                entropy=s["entropy"], rest_logps=s["rest"], stats=s.get("stats"),
                                temperature=case["temperature"])
        out = {k: s[k] for k in ("entropy", "top_ids", "top_logps", "rest")}
        if case["labels"]:
            out["logps"] = s["logps"]
        if case["grad"]:
            training.lora_top_logps_backward(s["logits"], s["stats"], s["dlogits"], labels=s["labels"],
                                             top_ids=s["top_ids"], entropy=s["entropy"], dlogps=s["dlogps"],
                                             dentropy=s["dentropy"], dtop_logps=s["dtop"],
                                             temperature=case["temperature"])
            out["dlogits"] = s["dlogits"]
        return out
    training.lora_distill_loss(s["logits"], s["ids"], s["teacher"], s["row_loss"], s["loss"], rest_logps=s["rest"],
                               weights=s["weights"], dlogits=s["dlogits"], kind=case["kind"],
                               temperature=case["temperature"])
    out = {"row_loss": s["row_loss"], "loss": s["loss"]}
    if case["grad"]:
        out["dlogits"] = s["dlogits"]
    return out


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    rows = [(_exact_top if case["op"] == "top" else _exact_distill)(s, slice(i, min(i + 256, case["T"])))
            for i in range(0, case["T"], 256)]
    out = {k: torch.cat([r[k] for r in rows]) for k in rows[0]}
    if case["op"] == "distill":
        out["loss"] = out["loss"].sum(0, keepdim=True)
    return out


def _exact_top(s, rows):
    case, x = s["case"], s["logits"][rows]
    n, V = x.shape
    logp = torch.log_softmax(x.double() / case["temperature"], 1)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :case["K"]]
    counts = torch.ones(n, dtype=torch.bool, device=DEV)
    out = {}
    if s["labels"] is not None:
        label = s["labels"][rows]
        counts = (label >= 0) & (label < V)
        out["logps"] = logp[torch.arange(n, device=DEV), label.clamp(0, V - 1)].masked_fill(~counts, 0.0)
    p = logp.exp()
    H = torch.special.entr(p).sum(1)
    chosen = torch.zeros_like(p, dtype=torch.bool).scatter_(1, order, True)
    best = logp.gather(1, order)
    absent = best.isinf() | ~counts[:, None]
    out["entropy"] = H.masked_fill(~counts, 0.0)
    out["top_ids"] = order.masked_fill(absent, -1)
    out["top_logps"] = best.masked_fill(absent, -math.inf)
    out["rest"] = logp.masked_fill(chosen, -math.inf).logsumexp(1).masked_fill(~counts, 0.0)
    if case["grad"]:
        # the vector of incoming gradients times the Jacobian of log p, then of the softmax
        g = torch.zeros_like(p)
        g.scatter_add_(1, order, s["dtop"][rows].double().masked_fill(absent, 0.0))
        if s["labels"] is not None:
            g[torch.arange(n, device=DEV), label.clamp(0, V - 1)] += s["dlogps"][rows].double()
        g = g - p * g.sum(1, keepdim=True)
        g -= s["dentropy"][rows].double()[:, None] * (p * H[:, None] - torch.special.entr(p))
        out["dlogits"] = (g / case["temperature"]).masked_fill(~counts[:, None], 0.0)
    return out


def _exact_distill(s, rows):
    """From the divergence of two distributions over buckets: each listed token, and all others together."""
    case, x, ids = s["case"], s["logits"][rows], s["ids"][rows]
    n, V = x.shape
    w = s["weights"][rows].double()
    here = (ids >= 0) & (ids < V)
    counts = here.any(1) & (w != 0)
    logp = torch.log_softmax(x.double() / case["temperature"], 1)
    bucket = torch.zeros((n, V + 1), dtype=torch.bool, device=DEV)
    bucket.scatter_(1, torch.where(here, ids, V), True)
    bucket = bucket[:, :V]
    a = torch.cat([logp, torch.full((n, 1), -math.inf, dtype=torch.float64, device=DEV)], 1)
    a = a.gather(1, torch.where(here, ids, V))
    b = s["teacher"][rows].double().masked_fill(~here, -math.inf)
    if case["rest"]:
        a = torch.cat([a, logp.masked_fill(bucket, -math.inf).logsumexp(1, keepdim=True)], 1)
        b = torch.cat([b, s["rest"][rows].double()[:, None]], 1)
    log_ratio = torch.where(b == -math.inf, torch.zeros_like(b), b - a)
    if case["kind"] == "forward":
        L = (b.exp() * log_ratio).masked_fill(b == -math.inf, 0.0).sum(1)
        by_bucket = -b.exp()                              # d L / d (ln p of the bucket)
    else:
        L = -(a.exp() * log_ratio).masked_fill(a == -math.inf, 0.0).sum(1)
        by_bucket = a.exp() * (1 - log_ratio)
        by_bucket = by_bucket.masked_fill((a == -math.inf) | (b == -math.inf), 0.0)
    L = L.masked_fill(~counts, 0.0)
    out = {"row_loss": L, "loss": (w * L).sum()[None]}
    if case["grad"]:
        p = logp.exp()
        d = torch.zeros((n, V + 1), dtype=torch.float64, device=DEV)
        K = case["K"]
        d.scatter_add_(1, torch.where(here, ids, V), by_bucket[:, :K].masked_fill(~here, 0.0))
        d = d[:, :V]
        if case["rest"]:
            within = (logp - a[:, K:]).exp().masked_fill(bucket, 0.0)      # a token's share of its bucket
            d += within * by_bucket[:, K:]
        d -= p * by_bucket.sum(1, keepdim=True)
        out["dlogits"] = (d * (w / case["temperature"])[:, None]).masked_fill(~counts[:, None], 0.0)
    return out

"""Cases of the post-training losses of the output layer, with their plain forms.

Five operators, in the order in which a trainer meets them:

  clipped_policy            clipped policy loss with a KL term on per-token log-probabilities
  policy_loss               the same loss on given logits, with its gradient to the logits
  policy_forward_backward   the same loss through the LM head (hidden states and weight), with dX and dW
  distill_topk              distillation from a teacher's top logits on given student logits
  distill_forward_backward  the same loss through the LM head, with dX and dW

``run`` computes the plain form (elementary torch operations) where ``own`` is
false and calls the package where it is true.  ``exact`` differentiates the
definition in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one short answer's tokens: a latency-bound call between two passes of a head
        {"name": "policy_rows_short", "op": "policy_rows", "n": 512, "kl": 0.0, "masked": 0.1},
        # the tokens of a whole rollout batch at once
        {"name": "policy_rows_batch", "op": "policy_rows", "n": 1048576, "kl": 0.05, "masked": 0.3},
        # scoring a handful of tokens on a small vocabulary: latency
        {"name": "policy_logits_few", "op": "policy_logits", "n": 4, "v": 4096, "dtype": "fp32", "pad": 0,
         "kl": 0.05, "ent": 0.0, "temp": 1.0, "masked": 0.0},
        # a micro-batch sampled at a temperature, odd vocabulary in rows of a padded buffer
        {"name": "policy_logits_odd", "op": "policy_logits", "n": 1023, "v": 50021, "dtype": "fp16", "pad": 43,
         "kl": 0.04, "ent": 0.01, "temp": 0.7, "masked": 0.2},
        # a training micro-batch on a large vocabulary, entropy bonus and KL on
        {"name": "policy_logits_batch", "op": "policy_logits", "n": 4096, "v": 128256, "dtype": "bf16", "pad": 0,
         "kl": 0.02, "ent": 0.001, "temp": 1.0, "masked": 0.25},
        # a few positions against a short teacher list: latency
        {"name": "distill_logits_few", "op": "distill_logits", "n": 16, "v": 4096, "dtype": "fp32", "pad": 0, "k": 8,
         "temp": 1.0, "ce": 0.0, "masked": 0.0},
        # softened distillation mixed with the hard labels (two softmaxes of one row)
        {"name": "distill_logits_soft", "op": "distill_logits", "n": 777, "v": 32064, "dtype": "fp16", "pad": 0, "k": 50,
         "temp": 2.0, "ce": 0.5, "masked": 0.1},
        # a training micro-batch on the largest vocabulary
        {"name": "distill_logits_batch", "op": "distill_logits", "n": 2048, "v": 256000, "dtype": "bf16", "pad": 0,
         "k": 64, "temp": 1.0, "ce": 0.0, "masked": 0.25},
        # the package's smallest head
        {"name": "policy_head_small", "op": "policy_head", "n": 256, "h": 256, "v": 4096, "kl": 0.05, "masked": 0.1},
        # a policy step of a large head
        {"name": "policy_head_large", "op": "policy_head", "n": 2048, "h": 4096, "v": 128256, "kl": 0.02, "masked": 0.25},
        # a small head with sizes that end inside every tile
        {"name": "distill_head_small", "op": "distill_head", "n": 300, "h": 264, "v": 5003, "k": 16, "temp": 2.0,
         "ce": 0.0, "masked": 0.1},
        # a distillation step of a head with the largest vocabulary
        {"name": "distill_head_large", "op": "distill_head", "n": 2048, "h": 2304, "v": 256000, "k": 64, "temp": 1.0,
         "ce": 0.25, "masked": 0.25},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy_rows", "policy_logits", "distill_logits", "policy_head", "distill_head"])
    c = {"op": op}
    if op == "policy_rows":
        c["n"] = _log_uniform(rng, 1, 1048576)
    elif op in ("policy_logits", "distill_logits"):
        c["dtype"] = rng.choice(list(DTYPES))
        c["v"] = _log_uniform(rng, 100, 256000)
        most = 4096 * 128256 * 2 // DTYPES[c["dtype"]].itemsize
        c["n"] = _log_uniform(rng, 1, max(1, min(16384, most // c["v"])))
        c["pad"] = rng.choice([0, 0, rng.randint(1, 64)])
    else:
        c["h"] = 8 * _log_uniform(rng, 8, 512)
        c["v"] = _log_uniform(rng, 200, 256000)
        c["n"] = _log_uniform(rng, 1, max(1, min(8192, 2048 * 4096 * 128256 // (c["h"] * c["v"]))))
    c["masked"] = rng.choice([0.0, rng.uniform(0.02, 0.6)])
    if op.startswith("policy"):
        c["kl"] = rng.choice([0.0, rng.uniform(0.01, 0.1)])
        if op == "policy_logits":
            c["ent"] = rng.choice([0.0, rng.uniform(0.0005, 0.01)])
            c["temp"] = rng.choice([1.0, rng.uniform(0.6, 1.4)])
    else:
        c["k"] = min(c["v"], _log_uniform(rng, 1, 256))
        c["temp"] = rng.choice([1.0, rng.uniform(1.2, 4.0)])
        c["ce"] = rng.choice([0.0, rng.uniform(0.1, 0.9)])
        if op == "distill_head" and c["temp"] != 1.0:
            c["ce"] = 0.0  # through the head the hard labels are mixed in at temperature 1 only
    return c


# ------------------------------------------------------------------ inputs --

CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _mask(y, share, g):
    """A masked prompt in front and scattered masked rows behind it."""
    n = y.numel()
    y[: int(0.5 * share * n)] = IGNORE
    y[torch.rand(n, device="cuda", generator=g) < 0.5 * share] = IGNORE


def _policy_inputs(s, lp, g):
    """Rollout-time and reference log-probabilities around the current ones, and
    one advantage per answer.  Log-ratios within 2e-3 of a clip border are moved
    off it: on which side of a border such a value falls is rounding."""
    n = lp.numel()
    delta = 0.15 * torch.randn(n, device="cuda", generator=g)
    for b in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
        delta = torch.where((delta - b).abs() < 2e-3, b + 4e-3, delta)
    s["old_logp"] = lp - delta
    s["ref_logp"] = lp - 0.2 * torch.randn(n, device="cuda", generator=g) if s["case"]["kl"] else None
    answers = torch.randn(8, device="cuda", generator=g)
    s["advantages"] = answers[torch.arange(n, device="cuda") * 8 // n].contiguous()


def _logits(c, g):
    buf = torch.randn(c["n"], c["v"] + c["pad"], device="cuda", generator=g).mul_(2.0).to(DTYPES[c["dtype"]])
    return buf[:, : c["v"]]


def _sample(x, g):
    """One token per row of softmax(x), by exponential races."""
    return (x - torch.empty_like(x).exponential_(generator=g).log_()).argmax(1).to(torch.int32)


def _teacher(s, z, g):
    """The K largest logits of a teacher near the student that favours low ids
    (frequent tokens); some rows hold fewer entries (id -1)."""
    c = s["case"]
    n, v, k = c["n"], c["v"], c["k"]
    u = torch.randn(n, v, device="cuda", generator=g).add_(z)
    u -= 0.3 * torch.log(torch.arange(1, v + 1, device="cuda", dtype=torch.float32))
    top, ids = torch.topk(u, k, dim=1)
    short = (torch.rand(n, device="cuda", generator=g) < 0.1)[:, None] & (torch.arange(k, device="cuda") > k // 2)
    s["teacher_ids"] = torch.where(short, -1, ids).to(torch.int32)
    s["teacher_logits"] = top.to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    n = c["n"]
    if c["op"] == "policy_rows":
        lp = -1.5 * torch.empty(n, device="cuda").exponential_(generator=g)
        s["row_loss"] = -lp
        s["y"] = torch.randint(0, 32064, (n,), device="cuda", generator=g, dtype=torch.int32)
        _mask(s["y"], c["masked"], g)
        _policy_inputs(s, lp, g)
        return s
    if c["op"].endswith("head"):
        s["X"] = torch.randn(n, c["h"], device="cuda", generator=g).to(torch.bfloat16)
        s["W"] = torch.randn(c["v"], c["h"], device="cuda", generator=g).mul_(0.02).to(torch.bfloat16)
        z = (s["X"] @ s["W"].T).float()
    else:
        s["logits"] = _logits(c, g)
        z = s["logits"].float()
    if c["op"].startswith("policy"):
        x = z / c.get("temp", 1.0)
        s["y"] = _sample(x, g)
        lp = x.gather(1, s["y"].long()[:, None])[:, 0] - torch.logsumexp(x, 1)
        _mask(s["y"], c["masked"], g)
        _policy_inputs(s, lp, g)
    else:
        s["y"] = _sample(z, g)
        _mask(s["y"], c["masked"], g)
        _teacher(s, z, g)
    return s


# -------------------------------------------------------------- plain forms --


def _mean_weight(valid):
    return valid.double() / valid.sum().clamp(min=1)


def _policy_rows(s, lp, valid):
    """Per row and in 64 bits: the policy loss without its entropy term, its
    derivative by the row's log-probability, and the KL estimate."""
    c = s["case"]
    old, adv = s["old_logp"].double(), s["advantages"].double()
    r = torch.exp(lp - old)
    clipped = torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH)
    loss = -torch.minimum(r * adv, clipped * adv)
    active = torch.where(adv >= 0, r <= 1 + CLIP_HIGH, r >= 1 - CLIP_LOW)
    d = torch.where(active, -adv * r, 0.0)
    kl = torch.zeros_like(lp)
    if s["ref_logp"] is not None:
        q = s["ref_logp"].double() - lp
        kl = torch.exp(q) - q - 1
        loss = loss + c["kl"] * kl
        d = d + c["kl"] * (1 - torch.exp(q))
    zero = torch.zeros((), dtype=torch.float64, device=lp.device)
    return torch.where(valid, loss, zero), torch.where(valid, d, zero), torch.where(valid, kl, zero)


def _softmax_parts(x):
    """Shifted logits, their exponentials and the row sums (64 bits)."""
    m = x.amax(1, keepdim=True)
    xm = (x - m).clamp_(min=-1e4)
    e = torch.exp(xm)
    l = e.sum(1, dtype=torch.float64)
    return m[:, 0].double(), xm, e, l


def _plain_policy_rows(s):
    valid = s["y"] != IGNORE
    loss, d, kl = _policy_rows(s, -s["row_loss"].double(), valid)
    w = _mean_weight(valid)
    return (loss * w).sum()[None], loss.float(), kl.float(), (-d * w).float()


def _plain_policy_logits(s):
    c = s["case"]
    valid = s["y"] != IGNORE
    yc = torch.where(valid, s["y"], 0).long()
    x = s["logits"].float() / c["temp"]
    m, xm, e, l = _softmax_parts(x)
    log_l = torch.log(l)
    lp = x.gather(1, yc[:, None])[:, 0].double() - m - log_l
    ent = log_l - (e * xm).sum(1, dtype=torch.float64) / l
    loss, d, kl = _policy_rows(s, lp, valid)
    w = _mean_weight(valid)
    zero = torch.zeros((), dtype=torch.float64, device=lp.device)
    lp, ent = torch.where(valid, lp, zero), torch.where(valid, ent, zero)
    total = ((loss - c["ent"] * ent) * w).sum()[None]
    p = e / l.float()[:, None]
    cw = c["ent"] * w
    a = (-d * w + cw * (ent - log_l)).float()
    grad = p * (a[:, None] + cw.float()[:, None] * xm)
    grad.scatter_add_(1, yc[:, None], (d * w).float()[:, None])
    grad = torch.where(valid[:, None], grad / c["temp"], 0.0)
    return total.float(), lp.float(), ent.float(), kl.float(), grad.to(s["logits"].dtype)


def _distill_logit_grad(s, z):
    """Row losses (64 bits) and the gradient to the logits, in 32 bits."""
    c = s["case"]
    t, ce = c["temp"], c["ce"]
    valid = s["y"] != IGNORE
    yc = torch.where(valid, s["y"], 0).long()
    w = _mean_weight(valid)
    there = s["teacher_ids"] >= 0
    ids = torch.where(there, s["teacher_ids"], 0).long()
    u = torch.where(there, s["teacher_logits"].double() / t, -math.inf)
    top = u.amax(1, keepdim=True)
    q = torch.exp(u - top)
    log_q = u - top - torch.log(q.sum(1, keepdim=True))
    q = torch.exp(log_q)
    x = z / t
    m, _, e, l = _softmax_parts(x)
    lse = m + torch.log(l)
    log_p = x.gather(1, ids).double() - lse[:, None]
    rows = torch.where(there, q * (torch.where(there, log_q, 0.0) - log_p), 0.0).sum(1)
    grad = e / l.float()[:, None]
    grad.scatter_add_(1, ids, -q.float())
    grad = grad / t
    if ce:
        m, _, e, l = _softmax_parts(z)
        rows = rows + ce * (m + torch.log(l) - z.gather(1, yc[:, None])[:, 0].double())
        grad = grad + ce * e / l.float()[:, None]
        grad.scatter_add_(1, yc[:, None], torch.full_like(grad[:, :1], -ce))
    rows = torch.where(valid, rows, 0.0)
    return (rows * w).sum()[None].float(), rows.float(), torch.where(valid[:, None], grad * w.float()[:, None], 0.0)


def _plain_distill_logits(s):
    loss, rows, grad = _distill_logit_grad(s, s["logits"].float())
    return loss, rows, grad.to(s["logits"].dtype)


def _plain_policy_head(s):
    X, W = s["X"].float(), s["W"].float()
    valid = s["y"] != IGNORE
    yc = torch.where(valid, s["y"], 0).long()
    z = X @ W.T
    m, _, e, l = _softmax_parts(z)
    lp = z.gather(1, yc[:, None])[:, 0].double() - m - torch.log(l)
    loss, d, _ = _policy_rows(s, lp, valid)
    w = _mean_weight(valid)
    a = (d * w).float()
    grad = e * (-a / l.float())[:, None]
    grad.scatter_add_(1, yc[:, None], a[:, None])
    lp = torch.where(valid, lp, 0.0)
    dX, dW = grad @ W, grad.T @ X
    return (loss * w).sum()[None].float(), lp.float(), dX.to(torch.bfloat16), dW.to(torch.bfloat16)


def _plain_distill_head(s):
    X, W = s["X"].float(), s["W"].float()
    loss, rows, grad = _distill_logit_grad(s, X @ W.T)
    return loss, rows, (grad @ W).to(torch.bfloat16), (grad.T @ X).to(torch.bfloat16)


PLAIN = {"policy_rows": _plain_policy_rows, "policy_logits": _plain_policy_logits, "policy_head": _plain_policy_head,
         "distill_logits": _plain_distill_logits, "distill_head": _plain_distill_head}


# ------------------------------------------------------------ the package's --


def _own(s):
    import lm_head_linear_03_b200 as F
    c = s["case"]
    if c["op"].startswith("policy"):
        kw = {"ref_logp": s["ref_logp"], "clip_low": CLIP_LOW, "clip_high": CLIP_HIGH, "kl_coef": c["kl"]}
        if c["op"] == "policy_rows":
            loss, rows, kl, weight, _ = F.clipped_policy(s["row_loss"], s["y"], s["old_logp"], s["advantages"], **kw)
            return loss, rows, kl, weight
        if c["op"] == "policy_logits":
            loss, _, logp, ent, kl, grad = F.policy_loss(s["logits"], s["y"], s["old_logp"], s["advantages"],
                                                         entropy_coef=c["ent"], temperature=c["temp"], **kw)
            return loss, logp, ent, kl, grad
        loss, _, logp, dX, dW = F.policy_forward_backward(s["X"], s["W"], s["y"], s["old_logp"], s["advantages"], **kw)
        return loss, logp, dX, dW
    kw = {"temperature": c["temp"], "ce_weight": c["ce"], "row_loss": True}
    if c["op"] == "distill_logits":
        loss, _, rows, grad = F.distill_topk(s["logits"], s["y"], s["teacher_ids"], s["teacher_logits"], **kw)
        return loss, rows, grad
    loss, _, rows, dX, dW = F.distill_forward_backward(s["X"], s["W"], s["y"], s["teacher_ids"], s["teacher_logits"], **kw)
    return loss, rows, dX, dW


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact --


def _exact_policy(s, lp, entropy, valid):
    """The scalar loss, the rows' losses and KL estimates of log-probabilities lp (64 bits)."""
    c = s["case"]
    r = (lp - s["old_logp"].double()).exp()
    adv = s["advantages"].double()
    rows = -torch.min(r * adv, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
    kl = torch.zeros_like(lp)
    if s["ref_logp"] is not None:
        gap = s["ref_logp"].double() - lp
        kl = gap.exp() - gap - 1
        rows = rows + c["kl"] * kl
    if entropy is not None:
        rows = rows - c["ent"] * entropy
    keep = valid.double()
    return (rows * keep).sum() / max(1.0, keep.sum().item()), rows * keep, kl * keep


def _exact_distill(s, z):
    c = s["case"]
    valid = s["y"] != IGNORE
    keep = valid.double()
    ids = s["teacher_ids"].long()
    u = (s["teacher_logits"].double() / c["temp"]).masked_fill(ids < 0, -math.inf)
    log_q = torch.log_softmax(u, 1).masked_fill(ids < 0, 0.0)
    q = torch.softmax(u, 1)
    log_p = torch.log_softmax(z / c["temp"], 1).gather(1, ids.clamp(min=0))
    rows = (q * (log_q - log_p)).sum(1)
    if c["ce"]:
        yc = torch.where(valid, s["y"], 0).long()
        rows = rows - c["ce"] * torch.log_softmax(z, 1).gather(1, yc[:, None])[:, 0]
    return (rows * keep).sum() / max(1.0, keep.sum().item()), rows * keep


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    valid = s["y"] != IGNORE
    yc = torch.where(valid, s["y"], 0).long()
    if c["op"] == "policy_rows":
        l = s["row_loss"].double().requires_grad_(True)
        loss, rows, kl = _exact_policy(s, -l, None, valid)
        (w,) = torch.autograd.grad(loss, l)
        return loss.detach()[None], rows.detach(), kl.detach(), w
    if c["op"].endswith("head"):
        leaves = [s["X"].double().requires_grad_(True), s["W"].double().requires_grad_(True)]
        z = leaves[0] @ leaves[1].T
    else:
        leaves = [s["logits"].double().requires_grad_(True)]
        z = leaves[0]
    if c["op"].startswith("distill"):
        loss, rows = _exact_distill(s, z)
        return (loss.detach()[None], rows.detach(), *torch.autograd.grad(loss, leaves))
    logp = torch.log_softmax(z / c.get("temp", 1.0), 1)
    lp = logp.gather(1, yc[:, None])[:, 0]
    entropy = -(logp.exp() * logp).sum(1) if c["op"] == "policy_logits" else None
    loss, _, kl = _exact_policy(s, lp, entropy, valid)
    grads = torch.autograd.grad(loss, leaves)
    lp = lp.detach() * valid
    if c["op"] == "policy_logits":
        return loss.detach()[None], lp, entropy.detach() * valid, kl.detach(), *grads
    return (loss.detach()[None], lp, *grads)


# -------------------------------------------------------------------- work --


def work(case):
    c = case
    n = c["n"]
    if c["op"] == "policy_rows":  # row loss, target, old, advantage (and reference) in; row loss, KL and weight out
        return {"bytes": n * (16 + 12 + (4 if c["kl"] else 0)), "flops": 20 * n}
    rows = n * (20 if c["op"].startswith("policy") else 8 + 6 * c["k"])  # per-row vectors in and out
    if c["op"].endswith("logits"):  # the logits once, their gradient once
        return {"bytes": 2 * n * c["v"] * DTYPES[c["dtype"]].itemsize + rows, "flops": 6 * n * c["v"]}
    # X, W once, dX, dW once; the three products of the unfused head
    return {"bytes": 4 * c["h"] * (n + c["v"]) + rows, "flops": 6 * n * c["h"] * c["v"]}

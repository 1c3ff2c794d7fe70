"""The losses at the vocabulary: what is measured of them, and their plain forms.

Two operators, reached through ``zero_sharded_optimizer_gb300.losses``:

- ``xent``: softmax cross entropy of ``hidden @ weight.T`` against labels, with
  the gradients of ``hidden`` and ``weight``;
- ``distill``: distillation from a teacher's top logits (a Kullback-Leibler
  divergence at a temperature), alone or mixed with the cross entropy, with the
  same gradients.

A case names the operator ("op"), whether the gradient is taken ("grad"), the
token count T, vocabulary V and width D, the storage type, the share of rows
without a target, the extra row stride of both matrices, the reduction of the
loss and, for distillation, K, the temperature and the mixing weight.
"""

import math

import torch

own = False

IGNORE = -100


def _case(name, op, grad, T, V, D, dtype="bf16", masked=0.0, pad=0, reduction="mean", K=0,
          tau=1.0, alpha=1.0, labels=True, ragged=False):
    return {"name": name, "op": op, "grad": grad, "T": T, "V": V, "D": D, "dtype": dtype,
            "masked": masked, "pad": pad, "reduction": reduction, "K": K, "tau": tau,
            "alpha": alpha, "labels": labels, "ragged": ragged}


def listed():
    return [
        # The log-probability of one next token (GPT-2-small's head): all latency and one read of W.
        _case("xent one token", "xent", False, 1, 50257, 768, reduction="none"),
        # Perplexity of a validation batch, 16 contexts of 1024.
        _case("xent evaluation", "xent", False, 16384, 50257, 768, reduction="none"),
        # A unit test's model or a first experiment: everything is latency. Odd in every size.
        _case("xent tiny fp32", "xent", True, 37, 1009, 96, "f32"),
        # A training micro-batch of GPT-2-small: 8 contexts of 1024 in the mixed mode.
        _case("xent gpt2 step", "xent", True, 8192, 50257, 768),
        # Fine-tuning on answers only: 60 % of the rows are prompt, and every row has its own weight.
        _case("xent answers only", "xent", True, 4096, 32000, 2048, masked=0.6, reduction="none"),
        # A wide model with a large vocabulary: the largest products.
        _case("xent large", "xent", True, 4096, 131072, 4096),
        # The full-precision mode of the optimizer, two contexts of 1024, a summed loss.
        _case("xent fp32 step", "xent", True, 2048, 50257, 768, "f32", reduction="sum"),
        # Rows that no 16-byte boundary fits: an odd width inside a wider buffer, an odd token count.
        _case("xent odd strides", "xent", True, 999, 50257, 771, masked=0.1, pad=5),
        # Distillation into GPT-2-small, mixed with its own cross entropy.
        _case("distill gpt2 step", "distill", True, 4096, 50257, 768, K=64, tau=2.0, alpha=0.5),
        # Distillation alone, from short and ragged lists of the teacher's candidates.
        _case("distill ragged", "distill", True, 2048, 32000, 1024, K=20, tau=1.0, labels=False,
              masked=0.05, ragged=True),
        # The divergence from the teacher on a short held-out text.
        _case("distill evaluation", "distill", False, 129, 50257, 768, K=8, tau=1.0,
              labels=False, reduction="none"),
        # A small full-precision student, many candidates, a high temperature.
        _case("distill fp32", "distill", True, 333, 10007, 512, "f32", K=100, tau=3.0, alpha=0.7),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = 4096 * 131072 * 4096 // 4
    while True:
        T, V, D = log_int(1, 16384), log_int(1000, 131072), log_int(64, 4096)
        if rng.random() < 0.5:      # half of the widths are what models have, half are anything
            D = max(64, D // 64 * 64)
        if T * V * D <= most and D != 3072:
            break
    op = rng.choice(["xent", "distill"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    masked = rng.choice([0.0, 0.0, 0.1, 0.6])
    pad = rng.choice([0, 0, 0, 1, 8])
    reduction = rng.choice(["mean", "sum", "none"])
    c = _case("", op, rng.random() < 0.75, T, V, D, dtype, masked, pad, reduction)
    if op == "distill":
        c.update(K=log_int(1, 128), tau=rng.choice([1.0, 2.0, 4.0]), labels=rng.random() < 0.5,
                 ragged=rng.random() < 0.5)
        c["alpha"] = rng.choice([0.3, 0.5, 0.9]) if c["labels"] else 1.0
    del c["name"]
    return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _matrix(rows, cols, pad, dtype, values):
    """``values`` inside a buffer of wider rows (pad = 0: contiguous)."""
    if pad == 0:
        return values.to(dtype)
    wide = torch.zeros(rows, cols + pad, dtype=dtype, device=values.device)
    wide[:, :cols] = values
    return wide[:, :cols]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    T, V, D, dt = case["T"], case["V"], case["D"], _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    # Rows of the head of length about 0.6 (GPT-2's 0.02 a value at its width), and hidden
    # states that favour their label by some logits, more for some tokens than for others.
    w = normal(V, D).mul_(0.6 / math.sqrt(D))
    labels = (uniform(T) * math.log(V)).exp().long().sub_(1).clamp_(0, V - 1)  # frequent ids are low
    favour = 9.0 * uniform(T)
    h = normal(T, D) + (favour / 0.36).unsqueeze(1) * w[labels]
    state = {"case": dict(case), "weight": _matrix(V, D, case["pad"], dt, w),
             "hidden": _matrix(T, D, case["pad"], dt, h)}
    del w, h
    gone = uniform(T) < case["masked"]
    state["labels"] = torch.where(gone, IGNORE, labels) if case["labels"] else None
    if case["op"] == "distill":
        K = min(case["K"], V // 2)
        step = max(1, V // (K + 1))
        jump = 1 + (uniform(T, K) * (step - 1)).long()
        jump[:, 0] = 0
        ids = (labels.unsqueeze(1) + jump.cumsum(1)) % V      # the label first, all distinct
        rank = torch.arange(K, device=dev, dtype=torch.float32)
        logits = 8.0 - 1.5 * torch.log1p(rank) + 0.5 * normal(T, K)
        if case["ragged"]:
            ids[uniform(T, K) < 0.3] = -1                     # an absent candidate
        ids[gone] = -1
        state["ids"], state["teacher"] = ids, logits
    # The gradient of the total with respect to each row's loss, where the caller has one.
    state["dloss"] = (0.5 + uniform(T)) / T if case["reduction"] == "none" and case["grad"] else None
    return state


def _run_own(s):
    from zero_sharded_optimizer_gb300 import losses
    c = s["case"]
    if c["op"] == "xent":
        args = (s["hidden"], s["weight"], s["labels"])
        more = {"ignore_index": IGNORE}
        forward, step = losses.xent_forward, losses.xent_step
    else:
        args = (s["hidden"], s["weight"], s["ids"], s["teacher"])
        more = {"temperature": c["tau"], "labels": s["labels"], "alpha": c["alpha"],
                "ignore_index": IGNORE}
        forward, step = losses.distill_forward, losses.distill_step
    if not c["grad"]:
        r = forward(*args, reduction=c["reduction"], **more)
    else:
        r = step(*args, reduction=c["reduction"], dloss=s["dloss"], **more)
    out = {"loss": r.loss}
    if c["reduction"] != "none":
        out["reduced"] = r.reduced
    if c["grad"]:
        out["dhidden"], out["dweight"] = r.dhidden, r.dweight
    return out


def run(state):
    if own:
        return _run_own(state)
    c, dt = state["case"], _dtype(state["case"])
    h, w = state["hidden"].float(), state["weight"].float()
    T = h.shape[0]
    z = h @ w.t()
    loss = torch.zeros(T, device=h.device)
    valid = torch.zeros(T, dtype=torch.bool, device=h.device)
    parts = []     # (row factor, softmax, ids, what is taken from them)
    ce, kd = (1.0, 0.0) if c["op"] == "xent" else (1.0 - c["alpha"], c["alpha"])
    if state["labels"] is not None:
        y = state["labels"]
        has = y != IGNORE
        valid |= has
        at = torch.where(has, y, 0).unsqueeze(1)
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - top)
        total = e.sum(1, keepdim=True)
        lse = top + torch.log(total)
        loss = loss + torch.where(has, ce * (lse - z.gather(1, at)).squeeze(1), 0.0)
        parts.append((torch.where(has, ce, 0.0), e.div_(total), at, torch.ones_like(at, dtype=torch.float32)))
    if c["op"] == "distill":
        tau, ids = c["tau"], state["ids"]
        there = ids >= 0
        some = there.any(1)
        valid |= some
        at = torch.where(there, ids, 0)
        t = torch.where(there, state["teacher"] / tau, -math.inf)
        t = t - torch.where(some, t.amax(1), 0.0).unsqueeze(1)
        q = torch.where(there, torch.exp(t), 0.0)
        q = q / torch.where(some, q.sum(1), 1.0).unsqueeze(1)
        zt = z / tau
        top = zt.amax(1, keepdim=True)
        e = torch.exp(zt.sub_(top))
        total = e.sum(1, keepdim=True)
        lse = top + torch.log(total)
        logq = torch.log(torch.where(q > 0, q, 1.0))
        kl = (q * (logq - z.gather(1, at) / tau + lse)).sum(1)
        loss = loss + torch.where(some, kd * tau * tau * kl, 0.0)
        parts.append((torch.where(some, kd * tau, 0.0), e.div_(total), at, q))
    out = {"loss": loss}
    count = valid.sum().clamp(min=1)
    if c["reduction"] != "none":
        out["reduced"] = loss.sum() / count if c["reduction"] == "mean" else loss.sum()
    if c["grad"]:
        del z
        row = torch.ones(T, device=h.device)
        if c["reduction"] == "mean":
            row = row / count
        elif c["reduction"] == "none":
            row = state["dloss"]
        g = None
        for factor, p, at, q in parts:
            p.scatter_add_(1, at, -q)
            p.mul_((factor * row).unsqueeze(1))
            g = p if g is None else g.add_(p)
        out["dhidden"] = (g @ w).to(dt)
        out["dweight"] = (g.t() @ h).to(dt)
    return out


def work(case):
    T, V, D = case["T"], case["V"], case["D"]
    rows = T * (1.0 - case["masked"])
    size = 2 if case["dtype"] == "bf16" else 4
    sparse = 8 * T * (1 if case["labels"] else 0) + 12 * T * case["K"]
    read = size * (rows * D + V * D) + sparse
    if not case["grad"]:
        return {"bytes": read + 4 * T, "flops": 2.0 * rows * V * D}
    # The logits, and the two products of their gradient.
    return {"bytes": read + 4 * T + size * (T * D + V * D), "flops": 6.0 * rows * V * D}


def exact(case, seed):
    """The definition in 64 bits: losses from log-sum-exp, gradients by
    differentiating them, a block of rows at a time."""
    T, V, D = case["T"], case["V"], case["D"]
    if (6.0 if case["grad"] else 2.0) * T * V * D > 1.4e13:
        return None
    s = prepare(case, seed)
    w = s["weight"].double().requires_grad_(case["grad"])
    hidden = s["hidden"].double()
    y, ids = s["labels"], s.get("ids")
    xent = case["op"] == "xent"
    counted = (y != IGNORE) if y is not None else torch.zeros(T, dtype=torch.bool, device=w.device)
    if not xent:
        counted = counted | (ids >= 0).any(1)
    rows = {"none": s["dloss"], "sum": torch.ones(T, device=w.device),
            "mean": torch.ones(T, device=w.device, dtype=torch.float64) / max(1, int(counted.sum()))}
    factor = rows[case["reduction"]]
    losses, dhidden, dweight = [], [], torch.zeros_like(w) if case["grad"] else None
    for a in range(0, T, 1024):
        b = min(T, a + 1024)
        h = hidden[a:b].clone().requires_grad_(case["grad"])
        z = h @ w.T
        value = torch.zeros(b - a, dtype=torch.float64, device=w.device)
        if y is not None:
            r = torch.nonzero(y[a:b] != IGNORE).squeeze(1)
            part = torch.logsumexp(z[r], 1) - z[r, y[a:b][r]]
            value = value.index_add(0, r, part * (1.0 if xent else 1.0 - case["alpha"]))
        if not xent:
            tau = case["tau"]
            r = torch.nonzero((ids[a:b] >= 0).any(1)).squeeze(1)
            i = ids[a:b][r]
            u = (s["teacher"][a:b][r].double() / tau).masked_fill(i < 0, -math.inf)
            logq = u - torch.logsumexp(u, 1, keepdim=True)
            logp = z[r].gather(1, i.clamp(min=0)) / tau - torch.logsumexp(z[r] / tau, 1, keepdim=True)
            terms = torch.exp(logq) * (logq.masked_fill(i < 0, 0.0) - logp)
            value = value.index_add(0, r, case["alpha"] * tau * tau * terms.sum(1))
        losses.append(value.detach())
        if case["grad"]:
            gh, gw = torch.autograd.grad((value * factor[a:b]).sum(), (h, w))
            dhidden.append(gh)
            dweight += gw
        del z
    loss = torch.cat(losses)
    out = {"loss": loss}
    if case["reduction"] != "none":
        out["reduced"] = (loss * (rows["mean"] if case["reduction"] == "mean" else 1.0)).sum()
    if case["grad"]:
        out["dhidden"], out["dweight"] = torch.cat(dhidden), dweight
    return out

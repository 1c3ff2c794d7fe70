"""What stands around the head of a tied-embedding model: what is measured, and the plain forms.

Four operators:

- ``lookup``: rows of the embedding by token id, scaled
  (``zero_sharded_optimizer_gb300.embedding``);
- ``scatter``: the embedding's gradient, the scaled sum of the rows of equal id
  in float32, rounded once (the same module);
- ``policy``: the clipped policy loss with a term that keeps it near a
  reference, from hidden states and the head's weight, with the gradients of
  both (``zero_sharded_optimizer_gb300.losses``);
- ``preference``: the loss of pairs of a preferred and a rejected sequence, from
  the same, with the same gradients (the same module).

A case names the operator ("op") and the sizes: T tokens, a vocabulary of V,
width D, the storage type and the extra row stride of every matrix ("pad"). The
two losses have the share of rows without a target, the reduction and whether
the gradients are taken ("grad"); a policy case the share of its sequences whose
advantage is zero ("still"), the bounds of the ratio and the reference's weight;
a preference case the number of pairs and the options of its loss.
"""

import math

import torch

own = False

IGNORE = -100


def _case(name, op, T, V, D, dtype="bf16", pad=0, **more):
    c = {"name": name, "op": op, "T": T, "V": V, "D": D, "dtype": dtype, "pad": pad}
    if op in ("lookup", "scatter"):
        c.update(scale=1.0, gone=0.0)
    else:
        c.update(grad=True, masked=0.0, reduction="mean")
    if op == "policy":
        c.update(still=0.0, low=0.2, high=0.2, kl=0.0)
    if op == "preference":
        c.update(pairs=1, kind="sigmoid", beta=0.1, smoothing=0.0, margin=0.0, average=False, nll=0.0,
                 reference=True)
    c.update(more)
    return c


def listed():
    return [
        # The next token of a sequence that is generated: all latency.
        _case("lookup one token", "lookup", 1, 50257, 768),
        # A large batch of a wide model, scaled as its embedding is: all traffic.
        _case("lookup large", "lookup", 131072, 131072, 4096, scale=64.0),
        # A unit test's model, odd in every size, some ids outside the vocabulary.
        _case("scatter tiny fp32", "scatter", 37, 1009, 97, "f32", pad=3, scale=0.5, gone=0.1),
        # A training micro-batch of GPT-2-small: 8 contexts of 1024 in the mixed mode.
        _case("scatter gpt2", "scatter", 8192, 50257, 768),
        # The large batch's gradient.
        _case("scatter large", "scatter", 131072, 131072, 4096, scale=64.0),
        # A first experiment in full precision: everything is latency.
        _case("policy tiny fp32", "policy", 37, 1009, 96, "f32", kl=0.05),
        # A micro-batch of sampled answers for GPT-2-small; a quarter of the groups had equal rewards.
        _case("policy gpt2 step", "policy", 8192, 50257, 768, still=0.25, high=0.28),
        # Answers behind prompts that carry no loss, each token with its own weight, kept near a reference.
        _case("policy answers only", "policy", 4096, 32000, 2048, masked=0.4, kl=0.02, reduction="none"),
        # Two short pairs in rows that no 16-byte boundary fits.
        _case("preference tiny", "preference", 61, 1009, 99, pad=5, pairs=2, masked=0.3, smoothing=0.1),
        # A micro-batch of pairs for GPT-2-small, prompts masked, with a share of the preferred answers' own loss.
        _case("preference gpt2 step", "preference", 8192, 50257, 768, pairs=16, masked=0.3, nll=0.2),
        # A wide model with a large vocabulary: few long pairs, a squared loss of the mean log-probabilities.
        _case("preference large", "preference", 4096, 131072, 4096, pairs=4, masked=0.1, kind="squared", beta=1.0,
              margin=0.5, average=True),
        # Held-out pairs in full precision: the loss alone, for each pair.
        _case("preference evaluation", "preference", 2048, 50257, 768, "f32", grad=False, pairs=8, masked=0.3,
              reduction="none"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["lookup", "scatter", "policy", "preference"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    pad = rng.choice([0, 0, 0, 1, 8])
    rows = op in ("lookup", "scatter")
    while True:
        T, V, D = log_int(1, 262144 if rows else 16384), log_int(1000, 131072), log_int(64, 4096)
        if rng.random() < 0.5:      # half of the widths are what models have, half are anything
            D = max(64, D // 64 * 64)
        if rows and (T + V) * D * (2 if dtype == "f32" else 1) <= 2 * 131072 * 4096:
            break
        if not rows and T >= 4 and T * V * D <= 4096 * 131072 * 4096 // 4:
            break
    c = _case("", op, T, V, D, dtype, pad)
    if rows:
        c.update(scale=rng.choice([1.0, 1.0, 0.3, math.sqrt(D)]), gone=rng.choice([0.0, 0.0, 0.1]))
    else:
        c.update(grad=rng.random() < 0.75, masked=rng.choice([0.0, 0.1, 0.3, 0.6]),
                 reduction=rng.choice(["mean", "sum", "none"]))
    if op == "policy":
        c.update(still=rng.choice([0.0, 0.0, 0.25, 0.5]), low=rng.choice([0.1, 0.2]), high=rng.choice([0.2, 0.28]),
                 kl=rng.choice([0.0, 0.02, 0.1]))
    if op == "preference":
        c.update(pairs=min(log_int(1, 64), T // 4), average=rng.random() < 0.3, nll=rng.choice([0.0, 0.0, 0.2]))
        c["reference"] = not c["average"] or rng.random() < 0.5     # sums without one differ by the lengths
        if rng.random() < 0.75:
            c.update(beta=rng.choice([0.05, 0.1, 0.5]), smoothing=rng.choice([0.0, 0.1]),
                     margin=rng.choice([0.0, 0.5]))
        else:
            c.update(kind="squared", beta=0.1, margin=0.5)
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


def _logps(hidden, weight, labels):
    """The labels' log-probabilities, 2048 rows at a time (0 without a label)."""
    w, out = weight.float(), []
    for a in range(0, hidden.shape[0], 2048):
        z, y = hidden[a:a + 2048].float() @ w.t(), labels[a:a + 2048]
        x = z.gather(1, y.clamp(min=0).unsqueeze(1)).squeeze(1) - torch.logsumexp(z, 1)
        out.append(torch.where(y >= 0, x, 0.0))
    return torch.cat(out)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    op, T, V, D, pad, dt = case["op"], case["T"], case["V"], case["D"], case["pad"], _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    state = {"case": dict(case)}
    # Frequent ids are low, as in a vocabulary in order of frequency.
    tokens = (uniform(T) * math.log(V)).exp().long().sub_(1).clamp_(0, V - 1)
    if op in ("lookup", "scatter"):
        state["ids"] = torch.where(uniform(T) < case["gone"], -1, tokens)
        if op == "lookup":
            state["weight"] = _matrix(V, D, pad, dt, normal(V, D).mul_(0.6 / math.sqrt(D)))
        else:
            state["dout"] = _matrix(T, D, pad, dt, normal(T, D).mul_(1.0 / math.sqrt(T)))
        return state
    # Rows of the head of length about 0.6 (GPT-2's 0.02 a value at its width), and hidden
    # states that favour their label by some logits, more for some tokens than for others.
    w = normal(V, D).mul_(0.6 / math.sqrt(D))
    favour = 9.0 * uniform(T)
    h = normal(T, D) + (favour / 0.36).unsqueeze(1) * w[tokens]
    state["weight"], state["hidden"] = _matrix(V, D, pad, dt, w), _matrix(T, D, pad, dt, h)
    del w, h
    labels = torch.where(uniform(T) < case["masked"], IGNORE, tokens)
    grad = case["grad"] and case["reduction"] == "none"
    if op == "policy":
        state["labels"] = labels
        logps = _logps(state["hidden"], state["weight"], labels)
        # The policy has moved since the tokens were sampled; no ratio lies on a bound.
        moved = 0.15 * normal(T)
        for bound in (1.0 - case["low"], 1.0 + case["high"]):
            moved = torch.where((moved.exp() - bound).abs() < 2e-3, moved + 0.01, moved)
        state["old_logps"] = logps - moved
        # One advantage for each answer of about 64 tokens, a little different from token to token.
        answer = torch.arange(T, device=dev) // 64
        each = normal(T)
        still = (uniform(T) < case["still"])[answer]
        state["advantages"] = torch.where(still, 0.0, each[answer] + 0.1 * normal(T))
        state["ref_logps"] = logps - 0.2 * normal(T) if case["kl"] else None
        state["dloss"] = (0.5 + uniform(T)) / T if grad else None
        return state
    # Preferred sequences first, then the rejected, of ragged lengths.
    P = case["pairs"]
    share = 0.5 + uniform(2 * P).double()
    ends = (share.cumsum(0) / share.sum() * T).long()
    ends[-1] = T
    state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), ends])
    # A sequence begins with its prompt, which carries no loss.
    seq = torch.searchsorted(ends, torch.arange(T, device=dev), right=True)
    begin, end = state["offsets"][seq], ends[seq]
    inside = (torch.arange(T, device=dev) - begin).double() / (end - begin).double()
    state["labels"] = torch.where(inside < case["masked"], IGNORE, tokens)
    state["ref_logps"] = None
    if case["reference"]:
        logps = _logps(state["hidden"], state["weight"], state["labels"])
        sums = torch.zeros(2 * P, dtype=torch.float64, device=dev).index_add_(0, seq, logps.double())
        moved = normal(2 * P).double()
        if case["average"]:
            count = torch.zeros_like(sums).index_add_(0, seq, (state["labels"] >= 0).double())
            state["ref_logps"] = (sums / count.clamp(min=1) - 0.2 * moved).float()
        else:
            state["ref_logps"] = (sums - 8.0 * moved).float()
    state["dloss"] = (0.5 + uniform(P)) / P if grad else None
    return state


def _run_own(s):
    c = s["case"]
    if c["op"] == "lookup":
        from zero_sharded_optimizer_gb300 import embedding
        return {"out": embedding.embedding_forward(s["ids"], s["weight"], scale=c["scale"])}
    if c["op"] == "scatter":
        from zero_sharded_optimizer_gb300 import embedding
        return {"dweight": embedding.embedding_backward(s["ids"], s["dout"], c["V"], scale=c["scale"])}
    from zero_sharded_optimizer_gb300 import losses
    if c["op"] == "policy":
        args = (s["hidden"], s["weight"], s["labels"], s["old_logps"], s["advantages"])
        more = {"ref_logps": s["ref_logps"], "clip": (c["low"], c["high"]), "kl_weight": c["kl"]}
        forward, step = losses.policy_forward, losses.policy_step
    else:
        args = (s["hidden"], s["weight"], s["labels"], s["offsets"])
        more = {"ref_logps": s["ref_logps"], "kind": c["kind"], "beta": c["beta"], "smoothing": c["smoothing"],
                "margin": c["margin"], "average": c["average"], "nll_weight": c["nll"]}
        forward, step = losses.preference_forward, losses.preference_step
    if c["grad"]:
        r = step(*args, reduction=c["reduction"], dloss=s["dloss"], ignore_index=IGNORE, **more)
    else:
        r = forward(*args, reduction=c["reduction"], ignore_index=IGNORE, **more)
    out = {"loss": r.loss, "logps": r.logps}
    if c["reduction"] != "none":
        out["reduced"] = r.reduced
    if c["grad"]:
        out["dhidden"], out["dweight"] = r.dhidden, r.dweight
    return out


def run(state):
    if own:
        return _run_own(state)
    c, dt = state["case"], _dtype(state["case"])
    if c["op"] == "lookup":
        there = state["ids"] >= 0
        rows = state["weight"][torch.where(there, state["ids"], 0)].float() * c["scale"]
        return {"out": torch.where(there.unsqueeze(1), rows, 0.0).to(dt)}
    if c["op"] == "scatter":
        there = state["ids"] >= 0
        rows = torch.where(there.unsqueeze(1), state["dout"].float(), 0.0)
        total = torch.zeros(c["V"], c["D"], device=rows.device)
        total.index_add_(0, torch.where(there, state["ids"], 0), rows)
        return {"dweight": (total * c["scale"]).to(dt)}
    h, w, y = state["hidden"].float(), state["weight"].float(), state["labels"]
    has = y != IGNORE
    at = torch.where(has, y, 0).unsqueeze(1)
    z = h @ w.t()
    top = z.amax(1, keepdim=True)
    chosen = z.gather(1, at)
    p = torch.exp(z.sub_(top))
    total = p.sum(1, keepdim=True)
    logps = torch.where(has, (chosen - top - torch.log(total)).squeeze(1), 0.0)
    if c["op"] == "policy":
        adv = state["advantages"]
        ratio = torch.exp(logps - state["old_logps"])
        bounded = ratio.clamp(1.0 - c["low"], 1.0 + c["high"])
        loss = torch.where(has, torch.maximum(-adv * ratio, -adv * bounded), 0.0)
        slope = torch.where(-adv * ratio >= -adv * bounded, -adv * ratio, 0.0)    # by the log-probability
        if c["kl"]:
            d = state["ref_logps"] - logps
            loss = loss + torch.where(has, c["kl"] * (torch.exp(d) - d - 1.0), 0.0)
            slope = slope + c["kl"] * (1.0 - torch.exp(d))
        count = has.sum().clamp(min=1)
        out = {"loss": loss, "logps": logps}
    else:
        P, offsets = c["pairs"], state["offsets"]
        rows = torch.arange(c["T"], device=h.device)
        seq = (rows.unsqueeze(1) >= offsets[1:]).sum(1)
        zero = torch.zeros(2 * P, dtype=torch.float64, device=h.device)
        n = zero.index_add(0, seq, has.double())
        sums = zero.index_add(0, seq, logps.double())
        mean = sums / n.clamp(min=1)
        x = mean if c["average"] else sums
        if state["ref_logps"] is not None:
            x = x - state["ref_logps"]
        u = c["beta"] * (x[:P] - x[P:]) - c["margin"]
        if c["kind"] == "sigmoid":
            away = torch.log1p(torch.exp(-u.abs()))
            loss = (1.0 - c["smoothing"]) * ((-u).clamp(min=0) + away) + c["smoothing"] * (u.clamp(min=0) + away)
            du = c["smoothing"] - 1.0 / (1.0 + torch.exp(u))
        else:
            loss, du = u * u, 2.0 * u
        some = (n[:P] + n[P:]) > 0
        loss = torch.where(some, loss - c["nll"] * mean[:P], 0.0).float()
        per = torch.cat([du, -du]) * c["beta"]
        if c["average"]:
            per = per / n.clamp(min=1)
        per[:P] -= c["nll"] / n[:P].clamp(min=1)
        if state["dloss"] is not None:
            per = per * torch.cat([state["dloss"], state["dloss"]])
        slope = per.float()[seq]
        count = some.sum().clamp(min=1)
        out = {"loss": loss, "logps": sums.float()}
    if c["reduction"] != "none":
        out["reduced"] = loss.sum() / count if c["reduction"] == "mean" else loss.sum()
    if c["grad"]:
        if c["reduction"] == "mean":
            slope = slope / count
        elif c["reduction"] == "none" and c["op"] == "policy":
            slope = slope * state["dloss"]
        slope = torch.where(has, slope, 0.0)
        p.div_(total).scatter_add_(1, at, torch.full_like(total, -1.0))
        p.mul_(-slope.unsqueeze(1))
        out["dhidden"] = (p @ w).to(dt)
        out["dweight"] = (p.t() @ h).to(dt)
    return out


def work(case):
    T, V, D = case["T"], case["V"], case["D"]
    size = 2 if case["dtype"] == "bf16" else 4
    rows = min(T, V)       # the distinct rows of the table, at most
    if case["op"] == "lookup":
        return {"bytes": 8 * T + size * D * (rows + T), "flops": float(T * D)}
    if case["op"] == "scatter":
        return {"bytes": 8 * T + size * D * (T + V), "flops": float(T * D)}
    rows = T * (1.0 - case["masked"])
    read = size * (rows * D + V * D) + 8 * T
    read += 12 * T if case["op"] == "policy" else 32 * case["pairs"]
    flops, written = 2.0 * rows * V * D, 8 * T
    if case["grad"]:        # the two products of the logits' gradient, for the rows that have one
        flops += 4.0 * rows * (1.0 - case.get("still", 0.0) * (not case.get("kl", 0.0))) * V * D
        written += size * (T * D + V * D)
    return {"bytes": read + written, "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits: log-probabilities from log-sum-exp, gradients by
    differentiating the losses, a block of rows at a time."""
    T, V, D, op = case["T"], case["V"], case["D"], case["op"]
    if op in ("policy", "preference") and (6.0 if case["grad"] else 2.0) * T * V * D > 1.2e13:
        return None
    s = prepare(case, seed)
    if op in ("lookup", "scatter"):
        if max(T, V) * D > 1 << 29:
            return None
        kept = torch.nonzero((s["ids"] >= 0) & (s["ids"] < V)).squeeze(1)
        if op == "lookup":
            out = torch.zeros(T, D, dtype=torch.float64, device=s["ids"].device)
            out[kept] = torch.index_select(s["weight"], 0, s["ids"][kept]).double()
            return {"out": out * case["scale"]}
        out = torch.zeros(V, D, dtype=torch.float64, device=s["ids"].device)
        out.index_put_((s["ids"][kept],), s["dout"][kept].double() * case["scale"], accumulate=True)
        return {"dweight": out}
    w, y = s["weight"].double(), s["labels"]
    blocks = [(a, min(T, a + 1024)) for a in range(0, T, 1024)]
    kept = torch.nonzero((y >= 0) & (y < V)).squeeze(1)
    lse = torch.zeros(T, dtype=torch.float64, device=w.device)
    logps = torch.zeros_like(lse)
    for a, b in blocks:
        z = s["hidden"][a:b].double() @ w.T
        lse[a:b] = torch.logsumexp(z, 1)
        r = torch.nonzero((y[a:b] >= 0) & (y[a:b] < V)).squeeze(1)
        logps[a + r] = z[r, y[a:b][r]] - lse[a + r]
        del z
    logps.requires_grad_()
    if op == "policy":
        l = logps[kept]
        ratio, adv = torch.exp(l - s["old_logps"][kept].double()), s["advantages"][kept].double()
        gain = torch.minimum(ratio * adv, torch.clamp(ratio, 1.0 - case["low"], 1.0 + case["high"]) * adv)
        each = -gain
        if case["kl"]:
            d = s["ref_logps"][kept].double() - l
            each = each + case["kl"] * (torch.expm1(d) - d)
        loss = torch.zeros_like(lse).index_put((kept,), each)
        count = max(1, len(kept))
        shown = logps.detach()
    else:
        P, ends = case["pairs"], s["offsets"].tolist()
        sums, count, n = [], 0, []
        for i in range(2 * P):
            inside = kept[(kept >= ends[i]) & (kept < ends[i + 1])]
            sums.append(logps[inside].sum())
            n.append(len(inside))
        each = []
        for i in range(P):
            a, b = sums[i], sums[P + i]
            if case["average"]:
                a, b = a / max(1, n[i]), b / max(1, n[P + i])
            if s["ref_logps"] is not None:
                a, b = a - s["ref_logps"][i].double(), b - s["ref_logps"][P + i].double()
            u = case["beta"] * (a - b) - case["margin"]
            if case["kind"] == "sigmoid":
                value = -(1.0 - case["smoothing"]) * torch.nn.functional.logsigmoid(u) \
                    - case["smoothing"] * torch.nn.functional.logsigmoid(-u)
            else:
                value = u.square()
            value = value - case["nll"] * sums[i] / max(1, n[i])
            each.append(value if n[i] + n[P + i] else value * 0.0)
            count += n[i] + n[P + i] > 0
        loss, count, shown = torch.stack(each), max(1, count), torch.stack(sums).detach()
    share = {"none": s["dloss"], "sum": 1.0, "mean": 1.0 / count}[case["reduction"]]
    out = {"loss": loss.detach(), "logps": shown}
    if case["reduction"] != "none":
        out["reduced"] = (loss.detach() * share).sum()
    if case["grad"]:
        slope = torch.autograd.grad((loss * share).sum(), logps)[0]
        out["dhidden"] = torch.zeros(T, D, dtype=torch.float64, device=w.device)
        out["dweight"] = torch.zeros_like(w)
        for a, b in blocks:
            r = a + torch.nonzero(slope[a:b]).squeeze(1)
            if not len(r):
                continue
            h = s["hidden"][r].double()
            g = torch.exp(h @ w.T - lse[r].unsqueeze(1))
            g[torch.arange(len(r), device=w.device), y[r]] -= 1.0
            g *= -slope[r].unsqueeze(1)
            out["dhidden"][r] = g @ w
            out["dweight"] += g.T @ h
            del g
    return out

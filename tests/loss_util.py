"""The vocabulary losses in 64 bits, and how far a kernel may be from them.

``reference`` writes the definition out (softmax by exponentials, gradients by
their formulas); ``bounds`` derives, value by value, the error that the stated
arithmetic allows:

- a logit is a sum of D products of stored values in fp32, in any order and
  with truncating adders: |dz| <= 2 D 2^-24 * sum_k |h_k w_k| (the fp32 mode
  drops products below 2^-24 of the value: one more 2^-22 of the same sum);
- a softmax value is off by a factor exp(2 |dz|) and a few fp32 roundings of
  its argument and value: 2 |dz| + 2^-20 (1 + |z - lse| 2^-2) of itself;
- the gradient of a logit is rounded once to bf16 (2^-8 of itself; up to 256
  rows a second bf16 value keeps what that left over, 2^-16; the fp32 mode
  keeps 2^-21), and the sums of products with it are in fp32;
- the result is rounded to its type.
"""

import math

import torch

IGNORE = -100


def reference(hidden, weight, labels=None, ids=None, logits=None, tau=1.0, alpha=1.0,
              ignore_index=IGNORE, reduction="mean", dloss=None, grad_scale=1.0):
    """Dict of float64 results; the rows without a target are left out of every product."""
    dev = hidden.device
    T, V = hidden.shape[0], weight.shape[0]
    w = weight.double()
    valid = torch.zeros(T, dtype=torch.bool, device=dev)
    ce, kd = (1.0, 0.0) if ids is None else (1.0 - alpha, alpha * tau)
    has_y = torch.zeros_like(valid)
    if labels is not None:
        has_y = (labels != ignore_index) & (labels >= 0) & (labels < V)
        valid = valid | has_y
    has_t = torch.zeros_like(valid)
    if ids is not None:
        there = (ids >= 0) & (ids < V) & (logits.double() != -math.inf)
        has_t = there.any(1)
        valid = valid | has_t
    h = torch.where(valid.unsqueeze(1), hidden.double(), 0.0)
    z = h @ w.T
    absz = h.abs() @ w.abs().T
    loss = torch.zeros(T, dtype=torch.float64, device=dev)
    g = torch.zeros(T, V, dtype=torch.float64, device=dev)
    size = torch.zeros_like(g)      # the same with every term positive
    out = {"valid": valid, "absz": absz.amax(1) if T and V else absz.sum(1)}
    if labels is not None:
        lse = torch.logsumexp(z, 1)
        at = torch.where(has_y, labels, 0).unsqueeze(1)
        loss = loss + torch.where(has_y, ce * (lse - z.gather(1, at)[:, 0]), 0.0)
        p = torch.exp(z - lse.unsqueeze(1)) * (ce * has_y).unsqueeze(1)
        hot = torch.zeros_like(g).scatter_add_(1, at, (ce * has_y).double().unsqueeze(1))
        g, size = g + p - hot, size + p + hot
        out["lse"] = torch.where(valid, lse, 0.0)
    if ids is not None:
        u = torch.where(there, logits.double() / tau, -math.inf)
        # from the row's maximum: beside a maximum of the type's lowest value log K would be lost
        u = u - torch.where(has_t, u.amax(1), 0.0).unsqueeze(1)
        total = torch.where(has_t, torch.exp(u).sum(1), 1.0).unsqueeze(1)
        q = torch.exp(u) / total
        logq = torch.where(q > 0, u - torch.log(total), 0.0)
        lse = torch.logsumexp(z / tau, 1)
        at = torch.where(there, ids, 0)
        kl = (q * (logq - z.gather(1, at) / tau + lse.unsqueeze(1))).sum(1)
        loss = loss + torch.where(has_t, alpha * tau * tau * kl, 0.0)
        p = torch.exp(z / tau - lse.unsqueeze(1)) * (kd * has_t).unsqueeze(1)
        hot = torch.zeros_like(g).scatter_add_(1, at, kd * q)
        g, size = g + p - hot, size + p + hot
        out["lse_tau"] = torch.where(valid, lse, 0.0)
    count = max(1, int(valid.sum()))
    out["loss"] = loss
    out["share"] = 1.0 / count if reduction == "mean" else 1.0   # of a row's loss in the reduced one
    out["reduced"] = {"none": None, "sum": loss.sum(), "mean": loss.sum() / count}[reduction]
    row = torch.ones(T, dtype=torch.float64, device=dev)
    if reduction == "none":
        row = torch.where(valid, dloss.double(), 0.0) if dloss is not None else row
    else:
        row = row * (float(dloss) if dloss is not None else 1.0)
    if reduction == "mean":
        row = row / count
    row = row * grad_scale
    g, size = g * row.unsqueeze(1), size * row.abs().unsqueeze(1)
    out.update(g=g, size=size, h=h, w=w, dhidden=g @ w, dweight=g.T @ h)
    return out


def bounds(r, dtype, parts=1):
    """Elementwise error allowed of loss, dhidden and dweight; `parts`: bf16 values that the
    gradient of a logit is kept in, each rounding to nearest what the one before left over."""
    T, V = r["g"].shape
    D = r["w"].shape[1]
    f32 = dtype == torch.float32
    unit = 2.0 ** -24 if f32 else 2.0 ** -8
    dz = (2 * D * 2.0 ** -24 + (2.0 ** -22 if f32 else 0.0)) * r["absz"]
    loss = 4 * dz + 2.0 ** -20 * (1 + r["absz"]) + 2.0 ** -22 * r["loss"].abs()
    g = r["g"].abs() * (2.0 ** -21 if f32 else 2.0 ** (-8 * parts)) + \
        r["size"] * (2 * dz + 2.0 ** -20 * (1 + r["absz"] / 4)).unsqueeze(1)
    dh = g @ r["w"].abs() + 2 * V * 2.0 ** -24 * (r["g"].abs() @ r["w"].abs())
    dw = g.T @ r["h"].abs() + 2 * T * 2.0 ** -24 * (r["g"].abs().T @ r["h"].abs())
    tiny = 2.0 ** -126
    return {"loss": loss + tiny,
            "dhidden": dh * 1.01 + unit * 1.01 * r["dhidden"].abs() + tiny,
            "dweight": dw * 1.01 + unit * 1.01 * r["dweight"].abs() + tiny}


def check(got, r, dtype, what="", parts=1):
    """``got``: a losses.Losses; fields that are None are not checked."""
    b = bounds(r, dtype, parts)
    for name in ("loss", "dhidden", "dweight"):
        x = getattr(got, name)
        if x is None:
            continue
        x = x.double().reshape(r[name].shape)
        off = (x - r[name]).abs()
        bad = ~(off <= b[name])
        if bad.any():
            i = int(torch.argmax((off / b[name]).nan_to_num(nan=math.inf).flatten()))
            raise AssertionError(
                f"{what} {name}: {int(bad.sum())} of {x.numel()} outside their bounds; worst at {i}: "
                f"got {float(x.flatten()[i])!r}, exact {float(r[name].flatten()[i])!r}, "
                f"bound {float(b[name].flatten()[i]):.3g}")
    if got.reduced is not None:
        total = float(b["loss"].sum()) * r["share"]
        assert abs(float(got.reduced) - float(r["reduced"])) <= total + 2.0 ** -22 * abs(float(r["reduced"])) + 1e-30, what

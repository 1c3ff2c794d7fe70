"""The policy and the preference loss in 64 bits, and how far a kernel may be
from them (loss_util's bounds of a logit, carried on):

- a log-probability is off by e = 4 dz + 2^-20 (1 + sum |h w|) + 2^-22 |l|, dz
  the bound of a logit, as the cross entropy is;
- a policy loss changes with it by no more than its steepest slope nearby,
  L = |A| r e^e + |c| (e^(d + e) + 1), and its slope by as much again;
- a sequence's sum is off by the sum of its rows' e, u by |beta| times two such;
  the sigmoid loss changes by at most |u's error| and its derivative by a
  quarter of that, the squared loss by (2 |u| + error) error, its derivative by
  twice the error; the preferred sequence's own loss by its rows' mean e;
- the stored slope and the losses are rounded to fp32;
- a slope that is off makes the whole of its row's gradient off in proportion.
"""

import math

import torch

from loss_util import IGNORE

__all__ = ["IGNORE", "policy", "preference", "check"]


def _rows(hidden, weight, labels, ignore_index, dtype):
    V, D = weight.shape
    has = (labels != ignore_index) & (labels >= 0) & (labels < V)
    h, w = torch.where(has.unsqueeze(1), hidden.double(), 0.0), weight.double()
    z, absz = h @ w.T, (h.abs() @ w.abs().T).amax(1)
    lse = torch.logsumexp(z, 1)
    at = torch.where(has, labels, 0)
    l = torch.where(has, z.gather(1, at.unsqueeze(1))[:, 0] - lse, 0.0)
    p = torch.exp(z - lse.unsqueeze(1))
    hot = torch.zeros_like(p).scatter_(1, at.unsqueeze(1), 1.0)
    dz = (2 * D * 2.0 ** -24 + (2.0 ** -22 if dtype == torch.float32 else 0.0)) * absz
    e = torch.where(has, 4 * dz + 2.0 ** -20 * (1 + absz) + 2.0 ** -22 * l.abs(), 0.0)
    return dict(has=has, h=h, w=w, absz=absz, lse=torch.where(has, lse, 0.0), l=l, p=p, hot=hot, dz=dz, e=e)


def _gradients(r, slope, slope_error, factor, factor_error=0.0):
    """Adds the gradients of slopes (times `factor`, one or for each row) to `r`."""
    s, se = slope * factor, slope_error * abs(factor) + factor_error * abs(slope)
    r["g"] = s.unsqueeze(1) * (r["hot"] - r["p"])
    r["size"] = s.abs().unsqueeze(1) * (r["hot"] + r["p"])
    r["slope_error"] = se.unsqueeze(1) * (r["hot"] + r["p"])
    r["dhidden"], r["dweight"] = r["g"] @ r["w"], r["g"].T @ r["h"]
    return r


def policy(hidden, weight, labels, old, adv, ref=None, clip=(0.2, 0.2), kl=0.0, reduction="mean", dloss=None,
           grad_scale=1.0, ignore_index=IGNORE):
    r = _rows(hidden, weight, labels, ignore_index, hidden.dtype)
    has, l, e = r["has"], r["l"], r["e"]
    A = torch.where(has, adv.double(), 0.0)
    ratio = torch.where(has & (A != 0), torch.exp(l - torch.where(has, old.double(), 0.0)), 1.0)
    held = ratio.clamp(1 - clip[0], 1 + clip[1])
    loss = torch.maximum(-A * ratio, -A * held)
    slope = torch.where(-A * ratio >= -A * held, -A * ratio, 0.0)
    steep = A.abs() * ratio * torch.exp(e)
    if kl:
        d = torch.where(has, ref.double() - l, 0.0)
        loss, slope = loss + kl * (torch.expm1(d) - d), slope - kl * torch.expm1(d)
        steep = steep + abs(kl) * (torch.exp(d + e) + 1)
    r["loss"], r["loss_error"] = torch.where(has, loss, 0.0), steep * e + 2.0 ** -22 * (loss.abs() + steep)
    r["logps"], r["logps_error"] = l, e
    slope = torch.where(has, slope, 0.0)
    slope_error = torch.where(has & (slope != 0), steep * e + 2.0 ** -22 * (slope.abs() + steep), 0.0)
    r["slopes"], r["slopes_error"] = slope, slope_error
    count = max(1, int(has.sum()))
    r["count"] = count if reduction == "mean" else 1
    if reduction == "none":
        factor = torch.where(has, dloss.double(), 0.0) if dloss is not None else torch.ones_like(l)
    else:
        factor = torch.full_like(l, (float(dloss) if dloss is not None else 1.0) / r["count"])
    return _gradients(r, slope, slope_error, factor * grad_scale)


def preference(hidden, weight, labels, bounds, ref=None, kind="sigmoid", beta=0.1, smoothing=0.0, margin=0.0,
               average=False, nll=0.0, reduction="mean", dloss=None, grad_scale=1.0, ignore_index=IGNORE):
    """`bounds`: the 2 P + 1 offsets as a list."""
    r = _rows(hidden, weight, labels, ignore_index, hidden.dtype)
    has, l, e = r["has"], r["l"], r["e"]
    P, dev = len(bounds) // 2, l.device
    n = [int(has[a:b].sum()) for a, b in zip(bounds, bounds[1:])]
    S = [float(l[a:b].sum()) for a, b in zip(bounds, bounds[1:])]
    E = [float(e[a:b].sum()) for a, b in zip(bounds, bounds[1:])]
    loss, loss_error, slopes, slopes_error = [], [], [0.0] * (2 * P), [0.0] * (2 * P)
    for i in range(P):
        c, j = i, P + i
        if n[c] + n[j] == 0:
            loss.append(0.0)
            loss_error.append(0.0)
            continue
        share = [1.0 / max(1, n[k]) if average else 1.0 for k in (c, j)]
        x = [S[k] * f - (float(ref[k]) if ref is not None else 0.0) for k, f in zip((c, j), share)]
        u = beta * (x[0] - x[1]) - margin
        du = abs(beta) * (E[c] * share[0] + E[j] * share[1])
        if kind == "sigmoid":
            soft = max(-u, 0.0) + math.log1p(math.exp(-abs(u)))     # log(1 + e^-u)
            value = (1 - smoothing) * soft + smoothing * (soft + u)
            down = math.exp(-soft - u) if u > -700 else 1.0          # sigmoid(-u)
            turn, off, turn_off = smoothing - down, du, du / 4
        else:
            value, turn, off, turn_off = u * u, 2 * u, (2 * abs(u) + du) * du, 2 * du
        mean = 1.0 / max(1, n[c])
        loss.append(value - nll * S[c] * mean)
        loss_error.append(off + abs(nll) * E[c] * mean + 2.0 ** -22 * (abs(value) + abs(nll * S[c] * mean)))
        for k, f, sign in ((c, share[0], 1), (j, share[1], -1)):
            if n[k]:
                own = nll * mean if sign > 0 else 0.0
                slopes[k] = sign * turn * beta * f - own
                slopes_error[k] = turn_off * abs(beta) * f + 2.0 ** -22 * (abs(turn * beta * f) + abs(own))
    def double(x):
        return torch.tensor(x, dtype=torch.float64, device=dev)

    r["loss"], r["loss_error"] = double(loss), double(loss_error)
    r["logps"], r["logps_error"] = double(S), double(E) + 2.0 ** -24 * double(S).abs()
    r["slopes"], r["slopes_error"] = double(slopes), double(slopes_error)
    r["counts"] = torch.tensor(n, dtype=torch.int32, device=dev)
    some = sum(1 for i in range(P) if n[i] + n[P + i])
    r["count"] = max(1, some) if reduction == "mean" else 1
    row, row_error, factor = torch.zeros_like(l), torch.zeros_like(l), torch.zeros_like(l)
    for k, (a, b) in enumerate(zip(bounds, bounds[1:])):
        row[a:b], row_error[a:b] = slopes[k], slopes_error[k]
        if reduction == "none":
            factor[a:b] = float(dloss[k % P]) if dloss is not None and n[k % P] + n[k % P + P] else 1.0
        else:
            factor[a:b] = (float(dloss) if dloss is not None else 1.0) / r["count"]
    zero = torch.zeros_like(l)
    return _gradients(r, torch.where(has, row, zero), torch.where(has, row_error, zero), factor * grad_scale)


def check(got, r, dtype, what="", parts=1):
    """``got``: a losses.LogpLosses; fields that are None are not checked."""
    f32 = dtype == torch.float32
    unit = 2.0 ** -24 if f32 else 2.0 ** -8
    bound = {name: 1.01 * r[name + "_error"] + 2.0 ** -23 * r[name].abs() for name in ("loss", "logps", "slopes")}
    T, V, D = r["h"].shape[0], *r["w"].shape
    g = r["g"].abs() * (2.0 ** -21 if f32 else 2.0 ** (-8 * parts)) + r["slope_error"] + \
        r["size"] * (2 * r["dz"] + 2.0 ** -20 * (1 + r["absz"] / 4)).unsqueeze(1)
    size = r["g"].abs() + g
    bound["dhidden"] = g @ r["w"].abs() + 2 * V * 2.0 ** -24 * (size @ r["w"].abs())
    bound["dweight"] = g.T @ r["h"].abs() + 2 * T * 2.0 ** -24 * (size.T @ r["h"].abs())
    for name in ("dhidden", "dweight"):
        bound[name] = 1.01 * (bound[name] + unit * (r[name].abs() + bound[name]))
    for name, b in bound.items():
        x = getattr(got, name)
        if x is None or (got.loss is None and name == "slopes"):
            continue
        x = x.double().reshape(r[name].shape)
        off = (x - r[name]).abs()
        bad = ~(off <= b + 2.0 ** -126)
        if bad.any():
            i = int(torch.argmax((off / b).nan_to_num(nan=math.inf).flatten()))
            raise AssertionError(
                f"{what} {name}: {int(bad.sum())} of {x.numel()} outside their bounds; worst at {i}: "
                f"got {float(x.flatten()[i])!r}, exact {float(r[name].flatten()[i])!r}, "
                f"bound {float(b.flatten()[i]):.3g}")
    if got.row_logps is not None and got.loss is not None:
        off = (got.row_logps.double().flatten() - r["l"]).abs()
        assert bool((off <= 1.01 * r["e"] + 2.0 ** -23 * r["l"].abs()).all()), f"{what} row_logps"
    if got.counts is not None:
        assert torch.equal(got.counts, r["counts"]), what
    if got.reduced is not None:
        want = float(r["loss"].sum()) / r["count"]
        total = float(bound["loss"].sum()) / r["count"]
        assert abs(float(got.reduced) - want) <= 1.01 * total + 2.0 ** -22 * abs(want) + 1e-30, what

"""Float64 definitions of the layer norm, the gated linear recurrence and the
projected cross entropy, and of their gradients, in plain torch operations
(any device).

TEST INFRASTRUCTURE ONLY, like ``oracle.py``: it shares nothing with the HIP
library.  The gradients are written from the formulas; the tests pin them
against central differences of the forwards.
"""
from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().to(torch.float64)


# ---- layer norm ------------------------------------------------------------

def layer_norm(x, weight=None, bias=None, eps=1e-5):
    x, weight, bias = f64(x), f64(weight), f64(bias)
    mean = x.mean(-1)
    rstd = ((x - mean[..., None]).square().mean(-1) + eps).rsqrt()
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_grad(dy, x, mean, rstd, weight=None):
    dy, x, mean, rstd, weight = map(f64, (dy, x, mean, rstd, weight))
    xhat = (x - mean[..., None]) * rstd[..., None]
    e = dy if weight is None else dy * weight
    dx = rstd[..., None] * (e - e.mean(-1, keepdim=True) - xhat * (e * xhat).mean(-1, keepdim=True))
    rows = tuple(range(x.dim() - 1))
    return {"dx": dx, "dweight": (dy * xhat).sum(rows) if rows else dy * xhat,
            "dbias": dy.sum(rows) if rows else dy.clone()}


# ---- gated linear recurrence -------------------------------------------------

def softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def gates(r, i, lam, scale):
    """log a, a, m = sqrt(1 - a^2), sigmoid(r), sigmoid(i)."""
    sr, si = torch.sigmoid(f64(r)), torch.sigmoid(f64(i))
    la = -scale * softplus(f64(lam)) * sr
    return la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), sr, si


def gated_recurrence(x, r, i, lam, scale=8.0, h0=None):
    x = f64(x)
    _, a, m, _, si = gates(r, i, lam, scale)
    batch, steps, dim = x.shape
    h = x.new_zeros(batch, dim) if h0 is None else f64(h0).clone()
    y = torch.empty_like(x)
    for t in range(steps):
        h = a[:, t] * h + m[:, t] * si[:, t] * x[:, t]
        y[:, t] = h
    return y, h


def gated_recurrence_grad(x, r, i, lam, y, dy, scale=8.0, h0=None, dh_last=None):
    """Gradients as a function of the stored outputs ``y``."""
    x, y, dy, lam64 = f64(x), f64(y), f64(dy), f64(lam)
    la, a, m, sr, si = gates(r, i, lam, scale)
    batch, steps, dim = x.shape
    carry = x.new_zeros(batch, dim) if dh_last is None else f64(dh_last).clone()
    g = torch.empty_like(x)
    for t in range(steps - 1, -1, -1):
        g[:, t] = dy[:, t] + carry
        carry = a[:, t] * g[:, t]
    start = x.new_zeros(batch, 1, dim) if h0 is None else f64(h0)[:, None]
    before = torch.cat([start, y[:, :-1]], 1) if steps else y
    # d log a: through a (da = g h_{t-1}) and through m (dm/dlog a = -a^2 / m)
    q = torch.where(m > 0, la / m, torch.zeros_like(m))
    w = g * before * a * la - g * si * x * a * a * q
    sp = softplus(lam64)
    ratio = torch.where(sp > 0, torch.sigmoid(lam64) / sp, torch.ones_like(sp))
    return {"dx": g * m * si, "dr": w * (1 - sr), "di": g * m * si * x * (1 - si),
            "dlam": w.sum((0, 1)) * ratio, "dh0": carry, "g": g, "w": w}


# ---- cross entropy of a projection ---------------------------------------------

def linear_cross_entropy(hidden, weight, targets, ignore_index=-100):
    logits = f64(hidden) @ f64(weight).t()
    lse = torch.logsumexp(logits, -1)
    live = targets != ignore_index
    valid = (targets >= 0) & (targets < weight.shape[0])
    at = torch.where(valid, targets, torch.zeros_like(targets))
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    loss = torch.where(valid, loss, torch.full_like(loss, float("nan")))
    return torch.where(live, loss, torch.zeros_like(loss)), lse


def linear_cross_entropy_grad(hidden, weight, targets, lse, dloss, ignore_index=-100):
    live = (targets != ignore_index)[:, None]
    h = torch.where(live, f64(hidden), torch.zeros((), dtype=torch.float64, device=hidden.device))
    w = f64(weight)
    p = torch.exp(h @ w.t() - f64(lse)[:, None])
    valid = (targets >= 0) & (targets < weight.shape[0])
    hit = torch.arange(weight.shape[0], device=targets.device)[None] == targets[:, None]
    p = (p - hit.to(p.dtype)) * torch.where(valid, f64(dloss), torch.full_like(f64(dloss), float("nan")))[:, None]
    p = torch.where(live, p, torch.zeros_like(p))
    return {"dhidden": p @ w, "dweight": p.t() @ h, "p": p}

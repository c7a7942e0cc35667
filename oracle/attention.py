"""Float64 definitions of the norm of queries and keys with their rotation, of
linear attention with a decay per head, of the selection of beams and of the
reordering of states, and of their gradients, in plain torch operations (any
device).

TEST INFRASTRUCTURE ONLY, like ``oracle.py``: it shares nothing with the HIP
library.  The recurrences are walked step by step as they are written; the
tests pin the gradients against central differences of the forwards.
"""
from __future__ import annotations

import math

import torch

from oracle.layers import f64


# ---- norm of a head with its rotation --------------------------------------------

def angles(positions, rotary, base):
    j = torch.arange(rotary // 2, dtype=torch.float64, device=positions.device)
    return positions.to(torch.float64)[..., None] * base ** (-2.0 * j / max(rotary, 1))


def rotate(n, a, rotary):
    """Turns value j < rotary / 2 with value j + rotary / 2 by a[..., None, j]."""
    half = rotary // 2
    c, s = torch.cos(a)[..., None, :], torch.sin(a)[..., None, :]
    x, y = n[..., :half], n[..., half:2 * half]
    return torch.cat([x * c - y * s, y * c + x * s, n[..., rotary:]], -1)


def head_norm_rotary(x, positions, weight=None, base=10000.0, eps=1e-6, rotary=None):
    x, weight = f64(x), f64(weight)
    rotary = x.shape[-1] // 2 * 2 if rotary is None else rotary
    n = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return rotate(n if weight is None else n * weight, angles(positions, rotary, base), rotary)


def head_norm_rotary_grad(dy, x, positions, weight=None, base=10000.0, eps=1e-6, rotary=None):
    dy, x, weight = f64(dy), f64(x), f64(weight)
    rotary = x.shape[-1] // 2 * 2 if rotary is None else rotary
    dn = rotate(dy, -angles(positions, rotary, base), rotary)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    e = dn if weight is None else dn * weight
    dx = r * (e - x * r.square() * (e * x).mean(-1, keepdim=True))
    return {"dx": dx, "dweight": (dn * x * r).flatten(0, -2).sum(0)}


# ---- linear attention ------------------------------------------------------------

def linear_attention(q, k, v, log_decay, scale=1.0, h0=None):
    """q, k (batch, L, heads, key), v (batch, L, heads, value)."""
    q, k, v, log_decay, h0 = map(f64, (q, k, v, log_decay, h0))
    batch, steps, heads, key = q.shape
    state = q.new_zeros(batch, heads, key, v.shape[-1]) if h0 is None else h0.clone()
    gate = torch.exp(log_decay)[:, None, None]
    o = torch.zeros_like(v)
    for t in range(steps):
        state = gate * state + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * (q[:, t, :, :, None] * state).sum(-2)
    return o, state


def linear_attention_grad(q, k, v, log_decay, do, scale=1.0, h0=None, dh_last=None):
    q, k, v, log_decay, do, h0, dh_last = map(f64, (q, k, v, log_decay, do, h0, dh_last))
    batch, steps, heads, key = q.shape
    zero = q.new_zeros(batch, heads, key, v.shape[-1])
    gate = torch.exp(log_decay)[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    state = zero if h0 is None else h0
    for t in range(steps):
        state = gate * state + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * (state * do[:, t, :, None, :]).sum(-1)
    back = zero if dh_last is None else dh_last      # gate R_{t+1}, at the end dh_last
    for t in reversed(range(steps)):
        r = back + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = (r * v[:, t, :, None, :]).sum(-1)
        dv[:, t] = (r * k[:, t, :, :, None]).sum(-2)
        back = gate * r
    return {"dq": dq, "dk": dk, "dv": dv, "dh0": back}


def packed(f, rows, cu_seqlens, states):
    """f over every sequence of packed rows: rows and results (total, ...), a
    dict of (seqs, ...) or None states by name; the results joined, 0 in rows
    of no sequence.  f takes (1, L, ...) rows and (1, ...) states and returns a
    tuple, states last."""
    ends = cu_seqlens.tolist()
    parts = []
    for b, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        parts.append(f(*[t[None, lo:hi] for t in rows],
                       **{n: None if s is None else s[b:b + 1] for n, s in states.items()}))
    out = []
    for j in range(len(parts[0]) - 1):
        like = parts[0][j]
        whole = like.new_zeros(rows[0].shape[0], *like.shape[2:])
        for (lo, hi), p in zip(zip(ends[:-1], ends[1:]), parts):
            whole[lo:hi] = p[j][0]
        out.append(whole)
    return (*out, torch.cat([p[-1] for p in parts]))


# ---- beams -------------------------------------------------------------------------

def beam_values(logits, scores):
    """scores + log softmax, -inf for the words of a beam without values.  The
    exponentials are summed exactly, so that equal beams have equal values."""
    logits, scores = f64(logits), f64(scores)
    top = logits.amax(-1, keepdim=True)
    sums = [math.fsum(row) if all(map(math.isfinite, row)) else float("nan")
            for row in (logits - top).exp().flatten(0, -2).tolist()]
    lse = torch.tensor(sums, dtype=torch.float64, device=logits.device).view(top.shape).log() + top
    value = scores[..., None] + (logits - lse)
    live = torch.isfinite(lse) & torch.isfinite(scores)[..., None]
    return torch.where(live, value, torch.full_like(value, float("-inf")))


def beam_select(logits, scores, count):
    """By value, equal ones of one beam by logit, then by j * vocab + v."""
    value = beam_values(logits, scores)
    live = (value > float("-inf")).any(-1, keepdim=True)
    vocab = logits.shape[-1]
    order = torch.where(live, f64(logits), torch.zeros_like(value)).sort(dim=-1, descending=True, stable=True).indices
    at = (order + vocab * torch.arange(logits.shape[1], device=logits.device)[:, None]).flatten(1)
    best, by_value = torch.sort(value.flatten(1).gather(1, at), dim=1, descending=True, stable=True)
    at = at.gather(1, by_value)[:, :count]
    return best[:, :count], at % vocab, at // vocab


def state_reorder(state, origins):
    beams = origins.shape[1]
    own = torch.arange(beams, device=origins.device).expand_as(origins)
    origins = torch.where((origins >= 0) & (origins < beams), origins, own)
    return state[torch.arange(origins.shape[0], device=origins.device)[:, None], origins]

"""Cases of the training and decoding operators that stand around the scans:
layer norm, the gated linear recurrence and the softmax cross entropy of a
vocabulary projection, each with its gradient.

``listed()`` gives the cases, ``draw(rng)`` one more of the same ranges,
``prepare`` the tensors a program holds before the call, ``run`` one call and
its outputs, ``work`` the bytes and operations no implementation can do
without, ``exact`` the outputs from the definitions in 64 bits.  With ``own``
false ``run`` evaluates the definitions with elementary torch operations in
float32; with ``own`` true it calls the library.

Definitions (float32 parameters; activations x, r, i, y ... in one dtype):

  layer norm, per row of D values
    y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
  gated linear recurrence, per batch and channel
    log a_t = -c softplus(lam) sigmoid(r_t)
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t
  cross entropy of a projection onto V words, per token
    l = W hidden,  lse = log sum_v exp l_v,  loss = lse - l_target
"""
import math

import torch

own = False

EPS = 1e-5       # of the layer norm
SCALE = 8.0      # c of the recurrence
IGNORE = -100    # target of a token without a loss
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of 64 sequences: the norm in front of a layer
        {"name": "norm_tokens_bf16", "op": "norm_fwd", "rows": 64, "dim": 2560, "io": "bf16"},
        # the norm of a float32 model over ragged rows whose width is odd
        {"name": "norm_odd_f32", "op": "norm_fwd", "rows": 4099, "dim": 1001, "io": "f32"},
        # backward of the norm over one training micro-batch (2 x 4096 tokens)
        {"name": "norm_layer_bwd_bf16", "op": "norm_bwd", "rows": 8192, "dim": 2560, "io": "bf16"},
        # one decode step of a few sequences, where the call's latency counts
        {"name": "recurrence_step_bf16", "op": "rec_step", "batch": 8, "dim": 5120, "io": "bf16"},
        # the recurrence of a training micro-batch, forward
        {"name": "recurrence_layer_bf16", "op": "rec_fwd", "batch": 2, "seqlen": 4096,
         "dim": 5120, "io": "bf16", "h0": False},
        # its backward
        {"name": "recurrence_layer_bwd_bf16", "op": "rec_bwd", "batch": 2, "seqlen": 4096,
         "dim": 5120, "io": "bf16", "h0": False},
        # one sequence of a million steps on few channels, continued from a state
        {"name": "recurrence_million_bf16", "op": "rec_fwd", "batch": 1, "seqlen": 1 << 20,
         "dim": 256, "io": "bf16", "h0": True},
        # backward of a float32 model at odd sizes, continued from a state
        {"name": "recurrence_ragged_bwd_f32", "op": "rec_bwd", "batch": 3, "seqlen": 1537,
         "dim": 769, "io": "f32", "h0": True},
        # scoring a few tokens: the vocabulary's weight is read once
        {"name": "loss_tokens_bf16", "op": "loss_fwd", "tokens": 16, "dim": 2560,
         "vocab": 50021, "io": "bf16"},
        # the loss of a training micro-batch over an odd vocabulary, forward
        {"name": "loss_layer_bf16", "op": "loss_fwd", "tokens": 8192, "dim": 2560,
         "vocab": 50021, "io": "bf16"},
        # its backward: gradients of the hidden states and of the weight
        {"name": "loss_layer_bwd_bf16", "op": "loss_bwd", "tokens": 8192, "dim": 2560,
         "vocab": 50021, "io": "bf16"},
        # backward of a small float32 model at odd sizes
        {"name": "loss_ragged_bwd_f32", "op": "loss_bwd", "tokens": 517, "dim": 769,
         "vocab": 32003, "io": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _ragged(rng, n):
    """n, or a near size that is a multiple of nothing in particular."""
    return n if rng.random() < 0.3 else max(1, n - rng.randrange(0, max(1, n // 16) + 1))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "rec_step", "rec_fwd", "rec_bwd", "loss_fwd", "loss_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        dim = _ragged(rng, _log_uniform(rng, 32, 8192))
        rows = _ragged(rng, _log_uniform(rng, 1, max(1, min(16384, (1 << 24) // dim))))
        return {"op": op, "rows": rows, "dim": dim, "io": io}
    if op == "rec_step":
        return {"op": op, "batch": _log_uniform(rng, 1, 256),
                "dim": _ragged(rng, _log_uniform(rng, 64, 8192)), "io": io}
    if op.startswith("rec"):
        most = (1 << 27) if op == "rec_fwd" else (1 << 25)
        dim = _ragged(rng, _log_uniform(rng, 64, 5120))
        batch = rng.randint(1, 4)
        seqlen = _ragged(rng, _log_uniform(rng, 1, min(1 << 20, most // (dim * batch))))
        return {"op": op, "batch": batch, "seqlen": seqlen, "dim": dim, "io": io,
                "h0": rng.random() < 0.5}
    dim = _ragged(rng, _log_uniform(rng, 64, 2560))
    vocab = _ragged(rng, _log_uniform(rng, 1000, 65536))
    most = (1 << 39) if io == "bf16" else (1 << 34)
    tokens = _ragged(rng, _log_uniform(rng, 1, max(1, min(8192, most // (dim * vocab)))))
    return {"op": op, "tokens": tokens, "dim": dim, "vocab": vocab, "io": io}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    io = DTYPES[case["io"]]

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dtype)

    def uniform(*shape, lo, hi):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo

    op = case["op"]
    s = {"op": op}
    if op.startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        # a residual stream: rows of different sizes, off zero
        s["x"] = (normal(rows, dim) * uniform(rows, 1, lo=0.5, hi=3.0) + normal(rows, 1, std=0.5)).to(io)
        s["weight"] = normal(dim, mean=1.0, std=0.2)
        s["bias"] = normal(dim, std=0.2)
        if op == "norm_bwd":
            s["dy"] = normal(rows, dim, dtype=io)
            x = s["x"].double()
            mean = x.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(-1) + EPS).rsqrt().float()
        return s
    if op.startswith("rec"):
        batch, dim = case["batch"], case["dim"]
        shape = (batch, dim) if op == "rec_step" else (batch, case["seqlen"], dim)
        for name in ("x", "r", "i"):
            s[name] = normal(*shape, dtype=io)
        # the slowest decay of a channel lies between 0.9 and 0.999 a step
        s["lam"] = torch.log(torch.expm1(-torch.log(uniform(dim, lo=0.9, hi=0.999)) / SCALE))
        if op == "rec_step":
            s["state"] = normal(batch, dim)
            return s
        s["h0"] = normal(batch, dim) if case["h0"] else None
        if op == "rec_bwd":
            s["y"] = _scan(*_coefficients(s["x"], s["r"], s["i"], s["lam"])[:2], s["h0"]).to(io)
            s["dy"] = normal(*shape, dtype=io)
            s["dh_last"] = normal(batch, dim) if case["h0"] else None
        return s
    tokens, dim, vocab = case["tokens"], case["dim"], case["vocab"]
    s["hidden"] = normal(tokens, dim, dtype=io)
    s["weight"] = normal(vocab, dim, dtype=io, std=2.0 / math.sqrt(dim))
    s["targets"] = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    # about one token in sixteen is padding
    s["targets"][torch.rand(tokens, generator=g, device="cuda") < 1.0 / 16] = IGNORE
    if op == "loss_bwd":
        s["lse"] = torch.logsumexp(s["hidden"].float() @ s["weight"].float().t(), -1)
        # gradient of the mean over the tokens that have a loss
        s["dloss"] = torch.full((tokens,), 1.0 / max(1, int((s["targets"] != IGNORE).sum())), device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------

def run(state):
    return (_library if own else _plain)(state)


def _library(s):
    import selective_state_space_05_amd as mssm
    op = s["op"]
    if op == "norm_fwd":
        return mssm.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS)
    if op == "norm_bwd":
        return mssm.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "rec_step":
        y = mssm.gated_recurrence_update(s["state"], s["x"], s["r"], s["i"], s["lam"], SCALE)
        return y, s["state"]
    if op == "rec_fwd":
        return mssm.gated_recurrence_fwd(s["x"], s["r"], s["i"], s["lam"], SCALE, h0=s["h0"])
    if op == "rec_bwd":
        return mssm.gated_recurrence_bwd(s["x"], s["r"], s["i"], s["lam"], s["y"], s["dy"], SCALE,
                                         h0=s["h0"], dh_last=s["dh_last"])
    if op == "loss_fwd":
        return mssm.linear_cross_entropy_fwd(s["hidden"], s["weight"], s["targets"], IGNORE)
    return mssm.linear_cross_entropy_bwd(s["hidden"], s["weight"], s["targets"], s["lse"], s["dloss"], IGNORE)


def _coefficients(x, r, i, lam):
    """a_t, the input term, and the pieces the backward needs, in float32."""
    sr, si = torch.sigmoid(r.float()), torch.sigmoid(i.float())
    # log(1 + e^lam) in 64 bits: for lam far below zero 1 + e^lam loses e^lam
    sp = torch.log1p(torch.exp(lam.double())).float()
    la = -SCALE * sp * sr
    m = torch.sqrt(-torch.expm1(2.0 * la))
    return torch.exp(la), m * si * x.float(), la, m, sr, si


def _scan(a, b, h0):
    """h_t = a_t h_{t-1} + b_t along dim 1 by doubling the span of the terms."""
    if h0 is not None and a.shape[1]:
        b = torch.cat([(b[:, :1] + a[:, :1] * h0[:, None]), b[:, 1:]], 1)
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(-1)
        rstd = ((x - mean[:, None]).square().mean(-1) + EPS).rsqrt()
        y = (x - mean[:, None]) * rstd[:, None] * s["weight"] + s["bias"]
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        wdy = dy * s["weight"]
        dx = (wdy - wdy.mean(-1, keepdim=True) - xhat * (wdy * xhat).mean(-1, keepdim=True)) * rstd
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    if op == "rec_step":
        a, b = _coefficients(s["x"], s["r"], s["i"], s["lam"])[:2]
        s["state"].mul_(a).add_(b)
        return s["state"].to(s["x"].dtype), s["state"]
    if op == "rec_fwd":
        a, b = _coefficients(s["x"], s["r"], s["i"], s["lam"])[:2]
        h = _scan(a, b, s["h0"])
        return h.to(s["x"].dtype), h[:, -1].clone()
    if op == "rec_bwd":
        io = s["x"].dtype
        a, b, la, m, sr, si = _coefficients(s["x"], s["r"], s["i"], s["lam"])
        dy = s["dy"].float()
        if s["dh_last"] is not None:
            dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dh_last"][:, None]], 1)
        # g_t = dy_t + a_{t+1} g_{t+1}: the same recurrence from the end
        later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        g = _scan(later.flip(1), dy.flip(1), None).flip(1)
        h0 = torch.zeros_like(g[:, 0]) if s["h0"] is None else s["h0"]
        before = torch.cat([h0[:, None], s["y"].float()[:, :-1]], 1)
        u = si * s["x"].float()
        # dlog a = da a - dm a^2 / m; its product with log a stays finite as a -> 1
        w = g * before * a * la - g * u * a * a * torch.where(m > 0, la / m, torch.zeros_like(m))
        sp = torch.log1p(torch.exp(s["lam"].double())).float()
        return {"dx": (g * m * si).to(io), "dr": (w * (1.0 - sr)).to(io),
                "di": (g * b * (1.0 - si)).to(io),
                "dlam": w.sum((0, 1)) * torch.sigmoid(s["lam"]) / sp,
                "dh0": a[:, 0] * g[:, 0]}
    hidden, weight = s["hidden"].float(), s["weight"].float()
    logits = hidden @ weight.t()
    live = s["targets"] != IGNORE
    at = torch.where(live, s["targets"], torch.zeros_like(s["targets"]))[:, None]
    if op == "loss_fwd":
        top = logits.max(-1, keepdim=True).values
        lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(-1))
        loss = lse - logits.gather(1, at)[:, 0]
        return torch.where(live, loss, torch.zeros_like(loss)), lse
    p = torch.exp(logits - s["lse"][:, None])
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    p = torch.where(live[:, None], p * s["dloss"][:, None], torch.zeros_like(p))
    return {"dhidden": (p @ weight).to(s["hidden"].dtype), "dweight": (p.t() @ hidden).to(s["weight"].dtype)}


# ---- bytes and operations ----------------------------------------------------

def work(case):
    e = 4 if case["io"] == "f32" else 2
    op = case["op"]
    if op.startswith("norm"):
        n, rows, dim = case["rows"] * case["dim"], case["rows"], case["dim"]
        if op == "norm_fwd":   # x, weight, bias -> y, mean, rstd
            return {"bytes": 2 * n * e + 8 * dim + 8 * rows, "flops": 8 * n}
        # dy, x, mean, rstd, weight -> dx, dweight, dbias
        return {"bytes": 3 * n * e + 12 * dim + 8 * rows, "flops": 14 * n}
    if op.startswith("rec"):
        bd = case["batch"] * case["dim"]
        if op == "rec_step":   # x, r, i, lam, state -> y, state
            return {"bytes": 4 * bd * e + 8 * bd + 4 * case["dim"], "flops": 20 * bd}
        n = bd * case["seqlen"]
        if op == "rec_fwd":    # x, r, i, lam, h0 -> y, h_last
            return {"bytes": 4 * n * e + 4 * bd * (2 if case["h0"] else 1) + 4 * case["dim"], "flops": 20 * n}
        # x, r, i, y, dy, lam, h0, dh_last -> dx, dr, di, dlam, dh0
        return {"bytes": 8 * n * e + 4 * bd * (3 if case["h0"] else 1) + 8 * case["dim"], "flops": 40 * n}
    t, d, v = case["tokens"], case["dim"], case["vocab"]
    if op == "loss_fwd":       # hidden, weight, targets -> loss, lse
        return {"bytes": (t * d + v * d) * e + 16 * t, "flops": 2 * t * v * d}
    # hidden, weight, targets, lse, dloss -> dhidden, dweight; the logits are formed again
    return {"bytes": 2 * (t * d + v * d) * e + 16 * t, "flops": 6 * t * v * d}


# ---- the definitions in 64 bits ----------------------------------------------

def _walk(a, b, h):
    """States of h_t = a_t h_{t-1} + b_t from h: (batch, steps, dim) in 64
    bits, walked step by step in stretches that run side by side."""
    batch, steps, dim = a.shape
    if steps == 0:
        return b
    width = max(1, math.isqrt(steps))
    count = -(-steps // width)
    out = torch.zeros((batch, count * width, dim), dtype=torch.float64, device=a.device)
    decay = torch.ones_like(out)
    out[:, :steps], decay[:, :steps] = b, a
    out, decay = out.view(batch, count, width, dim), decay.view(batch, count, width, dim)
    for j in range(1, width):
        out[:, :, j] += decay[:, :, j] * out[:, :, j - 1]
        decay[:, :, j] *= decay[:, :, j - 1]
    for k in range(count):
        out[:, k] += decay[:, k] * h[:, None]
        h = out[:, k, -1]
    return out.view(batch, count * width, dim)[:, :steps]


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op.startswith("norm"):
        x, w = s["x"], s["weight"]
        dim = x.shape[1]
        if op == "norm_fwd":
            mean = x.sum(1) / dim
            rstd = 1.0 / torch.sqrt((x - mean.view(-1, 1)).pow(2).sum(1) / dim + EPS)
            return (x - mean.view(-1, 1)) * rstd.view(-1, 1) * w + s["bias"], mean, rstd
        z = (x - s["mean"].view(-1, 1)) * s["rstd"].view(-1, 1)
        e = s["dy"] * w
        dx = s["rstd"].view(-1, 1) * (e - e.sum(1, True) / dim - z * ((e * z).sum(1, True) / dim))
        return {"dx": dx, "dweight": (s["dy"] * z).sum(0), "dbias": s["dy"].sum(0)}
    if op.startswith("rec"):
        soft = torch.where(s["lam"] > 30, s["lam"], torch.log1p(s["lam"].exp()))
        gr, gi = 1 / (1 + torch.exp(-s["r"])), 1 / (1 + torch.exp(-s["i"]))
        rate = -SCALE * soft * gr
        a, m = rate.exp(), (-torch.expm1(2 * rate)).sqrt()
        if op == "rec_step":
            h = a * s["state"] + m * gi * s["x"]
            return h, h
        start = torch.zeros_like(s["x"][:, 0]) if s["h0"] is None else s["h0"]
        if op == "rec_fwd":
            h = _walk(a, m * gi * s["x"], start)
            return h, h[:, -1]
        g = s["dy"].clone()
        if s["dh_last"] is not None:
            g[:, -1] += s["dh_last"]
        steps = g.shape[1]
        back = torch.arange(steps - 1, -1, -1, device=g.device)
        nxt = torch.zeros_like(a)
        nxt[:, 1:] = a[:, 1:][:, torch.arange(steps - 2, -1, -1, device=g.device)]
        g = _walk(nxt, g[:, back], torch.zeros_like(start))[:, back]
        prev = s["y"].roll(1, 1)
        prev[:, 0] = start
        da, dm = g * prev, g * gi * s["x"]
        drate = da * a - dm * torch.where(m > 0, a * a / m, torch.zeros_like(m))
        return {"dx": g * m * gi, "dr": drate * rate * (1 - gr), "di": g * m * s["x"] * gi * (1 - gi),
                "dlam": (drate * gr).sum((0, 1)) * (-SCALE) / (1 + torch.exp(-s["lam"])),
                "dh0": a[:, 0] * g[:, 0]}
    hidden, weight, targets = s["hidden"], s["weight"], s["targets"]
    tokens, vocab = hidden.shape[0], weight.shape[0]
    loss, lse = hidden.new_zeros(tokens), hidden.new_zeros(tokens)
    dh, dw = torch.zeros_like(hidden), torch.zeros_like(weight)
    words = torch.arange(vocab, device=targets.device)
    for t0 in range(0, tokens, 1024):      # some tokens at a time
        t1 = min(tokens, t0 + 1024)
        h, live = hidden[t0:t1], targets[t0:t1] != IGNORE
        logits = torch.mm(h, weight.t())
        hit = words[None, :] == targets[t0:t1, None]
        if op == "loss_fwd":
            lse[t0:t1] = torch.logsumexp(logits, 1)
            loss[t0:t1] = torch.where(live, lse[t0:t1] - (logits * hit).sum(1), loss[t0:t1])
            continue
        p = (logits - s["lse"][t0:t1, None]).exp() - hit.double()
        p *= (s["dloss"][t0:t1] * live)[:, None]
        dh[t0:t1] = torch.mm(p, weight)
        dw += torch.mm(p.t(), h)
    return (loss, lse) if op == "loss_fwd" else {"dhidden": dh, "dweight": dw}

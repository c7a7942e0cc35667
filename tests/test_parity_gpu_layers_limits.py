"""GPU parity of the layer norm, the gated linear recurrence and the projected
cross entropy at the ends of their ranges: sizes at which a further level of
their kernels begins, gates and decays next to their limits, infinite logits.
Needs an MI355X; marked ``gpu``.

The bounds are those of test_parity_gpu_layers.py, or derived where they stand."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import test_parity_gpu_layers as base  # noqa: E402
from oracle import layers  # noqa: E402
from test_parity_gpu_layers import IO, dev, mssm, randn, within  # noqa: E402,F401  (two fixtures among them)

pytestmark = pytest.mark.gpu
U32 = base.U32


def announce(*what):
    print("[limits]", *what, flush=True)


# ---- gated linear recurrence: more groups of channels than 2^25 ------------------

def test_gated_recurrence_more_than_2_25_groups(dev, mssm):
    """A group of channels is one sequence here (dim 1), and a second segment
    makes the groups exchange: what a group publishes lies past 2^31 entries.
    7.5 GB each for the inputs (one buffer for the three) and the output, 86 GB
    of workspace."""
    batch, steps = (1 << 25) + 64, 111
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GiB of free memory")
    announce("recurrence", batch, "groups")
    x = torch.empty(batch, steps, 1, dtype=torch.bfloat16, device=dev)
    for k in range(0, batch, 1 << 22):
        x[k:k + (1 << 22)].normal_()
    lam = torch.full((1,), -6.0, device=dev)
    y, last = mssm.gated_recurrence_fwd(x, x, x, lam, 8.0)
    for first in (0, (1 << 24) - 32, (1 << 25) - 64, 1 << 25):
        xs, ys = x[first:first + 64], y[first:first + 64]
        yo, lo = layers.gated_recurrence(xs, xs, xs, lam, 8.0)
        bound = base.rec_forward_bound(xs, xs, xs, lam, yo, None)
        within(last[first:first + 64], lo, bound[:, -1] + 1e-30, "h_last")
        within(ys, yo, bound + base.half_step(yo, ys) * 1.01, "y")
    del x, y, xs, ys
    torch.cuda.empty_cache()


# ---- gated linear recurrence: gates that are almost closed, decays that are fast --

FLUSH, STEP = 2.0 ** -126, 2.0 ** -149   # smallest normal and subnormal float32


def gate_bounds(r, lam, scale=8.0):
    """log a, a, m, sigmoid(r) in float64 and how far the float32 ones are off.

    sigmoid: the exponent's rounding times |r| and three operations; a hardware
    reciprocal gives 0 for a result below FLUSH.  softplus, its product with the
    scale and log a round to a multiple of STEP where they are subnormal.  a: the
    rounding of 1 + (a - 1) or, below log a = -0.35, an exponential whose argument
    is rounded twice.  m is a root: off by half its radicand's relative error or,
    where that is large, by the root of its error."""
    la, a, m, sr, _ = layers.gates(r, r, lam, scale)
    rate = scale * layers.softplus(lam.double())
    d_la = la.abs() * (3 * r.double().abs() + 24) * U32 + torch.where(sr < 2 * FLUSH, rate * FLUSH, 0 * la)
    d_la = d_la + scale * 2 * STEP * sr + STEP
    far = a * (d_la + (3 * la.abs() + 8) * U32) + FLUSH
    d_a = torch.where(la < -0.34, far, d_la + 2 * U32)
    d_em = 2 * a * a * (d_la + (3 * la.abs() + 8) * U32 * (la < -0.34)) + 8 * U32 * m * m + 2 * STEP
    d_m = torch.minimum(d_em.sqrt(), d_em / m.clamp(min=1e-300)) + 4 * U32 * m
    return la, a, m, sr, d_la, d_a, d_m


def walk_back(a, dy, d_a, dh_last):
    """g_t = dy_t + a_{t+1} g_{t+1}: bounds of its error and of its size, and of
    what leaves the first step (test_gated_recurrence_backward's)."""
    e = torch.zeros_like(a[:, 0])
    size = e if dh_last is None else dh_last.double().abs()
    d_g, g_size = torch.empty_like(a), torch.empty_like(a)
    for t in range(a.shape[1] - 1, -1, -1):
        size = dy[:, t].double().abs() + size
        e = e + 2 * U32 * size
        d_g[:, t], g_size[:, t] = e, size
        e = a[:, t] * e + 2 * (d_a[:, t] + U32 * a[:, t]) * size
        size = a[:, t] * size
    return d_g, e + U32 * size


def check_gates_forward(mssm, x, r, i, lam, h0):
    _, a, m, _, _, d_a, d_m = gate_bounds(r, lam)
    si, ax = torch.sigmoid(i.double()), x.double().abs()
    b = m * si * ax
    d_b = si * ax * d_m + b * (3 * i.double().abs() + 20) * U32
    e = torch.zeros_like(a[:, 0])
    size = e if h0 is None else h0.double().abs()
    bound = torch.empty_like(a)
    for t in range(a.shape[1]):
        new = a[:, t] * size + b[:, t]
        e = a[:, t] * e + 2 * ((d_a[:, t] + U32 * a[:, t]) * size + d_b[:, t] + 2 * U32 * new)
        size = new
        bound[:, t] = e
    y, last = mssm.gated_recurrence_fwd(x, r, i, lam, 8.0, h0=h0)
    yo, lo = layers.gated_recurrence(x, r, i, lam, 8.0, h0)
    within(last, lo, bound[:, -1] + FLUSH, "h_last")
    within(y, yo, bound + base.half_step(yo, y) * 1.01, "y")


def check_gates_backward(mssm, x, r, i, lam, h0, dh_last, names=("dx", "di", "dr", "dh0", "dlam")):
    y = layers.gated_recurrence(x, r, i, lam, 8.0, h0)[0].to(x.dtype)
    dy = randn(x.device, *x.shape, seed=11, dtype=x.dtype)
    got = mssm.gated_recurrence_bwd(x, r, i, lam, y, dy, 8.0, h0=h0, dh_last=dh_last)
    want = layers.gated_recurrence_grad(x, r, i, lam, y, dy, 8.0, h0, dh_last)
    _, a, _, _, _, d_a, _ = gate_bounds(r, lam)
    d_g, d_h0 = walk_back(a, dy, d_a, dh_last)
    within_grads(got, want, x, r, i, lam, y, h0, d_g, d_h0, names)
    return got


def within_grads(got, want, x, r, i, lam, y, h0, d_g, d_h0, names=("dx", "di", "dr", "dh0", "dlam")):
    """d_g, d_h0: how far g and what leaves the first step are off."""
    la, a, m, sr, d_la, d_a, d_m = gate_bounds(r, lam)
    si, ax = torch.sigmoid(i.double()), x.double().abs()
    g = want["g"].abs()
    rel_s = (3 * i.double().abs() + 12) * U32
    d_gm = d_g * m + g * d_m + 2 * U32 * g * m
    start = torch.zeros_like(a[:, :1]) if h0 is None else h0.double()[:, None]
    before = torch.cat([start, y.double()[:, :-1]], 1).abs()
    # w = a g log a (h_{t-1} - u a / m), u = sigmoid(i) x.  log a / m is about the
    # root of -log a / 2.  a g log a may round to a multiple of STEP, and 1 / m
    # reaches at most 2^74.
    u = si * ax
    q = torch.where(m > 0, la / m, 0 * m).abs()
    d_q = torch.minimum(d_la.sqrt(), 1.1 * q * d_la / la.abs().clamp(min=1e-300)) + 10 * U32 * q
    one, two = a * la.abs() * before, a * a * u * q
    inverse = (1 / m.clamp(min=2.0 ** -74))
    d_w = (d_g * (one + two) + g * (a * before * d_la + a * a * u * d_q + d_a * (before * la.abs() + 2 * a * u * q)
                                    + (one + two) * (rel_s + 10 * U32)) + STEP * (before + u * a * inverse))
    bounds = {"dx": si * d_gm + g * m * si * rel_s,
              "di": u * (1 - si) * d_gm + g * m * u * ((1 - si) * (rel_s + 2 * U32) + si * rel_s + U32),
              "dr": d_w * (1 - sr) + want["w"].abs() * (sr * (3 * r.double().abs() + 24) * U32 + 2 * U32),
              "dh0": d_h0 + FLUSH}
    ratio = torch.sigmoid(lam.double()) / layers.softplus(lam.double())
    n = (a.shape[0] * a.shape[1] + 16) * U32
    bounds["dlam"] = ratio * (d_w.sum((0, 1)) + n * want["w"].abs().sum((0, 1))) + want["dlam"].abs() * 16 * U32 + FLUSH
    for key in names:
        extra = base.half_step(want[key], got[key]) * 1.01 if key in ("dx", "di", "dr") else 0
        within(got[key], want[key], bounds[key] + extra, key)


CLOSED = [0.0, -70.0, -80.0, -83.0, -85.0, -86.0, -86.5, -87.0, -87.5, -88.0, -95.0, -104.0]


def closed_inputs(dev, steps, value, io):
    shape = (2, steps, 66)
    x, i = (randn(dev, *shape, seed=k, dtype=IO[io]) for k in (1, 2))
    return x, torch.full(shape, value, device=dev, dtype=IO[io]), i, torch.linspace(-100.0, -2.0, 66, device=dev)


@pytest.mark.parametrize("value", CLOSED)
@pytest.mark.parametrize("steps", [5, 300])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_recurrence_almost_closed_gates(dev, mssm, value, steps, io):
    """1 - a^2 through the subnormals down to 0: what little enters and every
    gradient keep float32's relative precision as far as log a itself does."""
    announce("almost closed", value, steps, io)
    x, r, i, lam = closed_inputs(dev, steps, value, io)
    check_gates_forward(mssm, x, r, i, lam, None)
    got = check_gates_backward(mssm, x, r, i, lam, None, randn(dev, 2, 66, seed=12), ("dx", "di", "dr", "dh0"))
    assert torch.isfinite(got["dlam"]).all()


@pytest.mark.parametrize("log_a", [-0.3, -0.36, -1.0, -5.0, -8.0, -12.0, -17.0, -25.0, -40.0, -60.0])
@pytest.mark.parametrize("steps", [5, 300])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_recurrence_fast_decays(dev, mssm, log_a, steps, io):
    """A decay far below one keeps its relative precision: it is a factor of
    dr, dlam and dh0.  log a lies around the value given."""
    announce("fast decays", log_a, steps, io)
    shape = (2, steps, 66)
    x, i, r = (randn(dev, *shape, seed=k, dtype=IO[io], scale=s) for k, s in ((1, 1.0), (2, 1.0), (3, 0.2)))
    lam = torch.full((66,), -log_a / 4, dtype=torch.float64, device=dev).expm1().log().float()
    h0, dh_last = randn(dev, 2, 66, seed=4), randn(dev, 2, 66, seed=12)
    check_gates_forward(mssm, x, r, i, lam, h0)
    check_gates_backward(mssm, x, r, i, lam, h0, dh_last)


@pytest.mark.parametrize("steps", [5, 300])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_recurrence_lam_far_out(dev, mssm, steps, io):
    """dlam's factor sigmoid(lam) / softplus(lam), where both leave float32's
    range (below -87 and -104) and where it is steep."""
    announce("lam far out", steps, io)
    shape = (2, steps, 130)
    x, i, r = (randn(dev, *shape, seed=k, dtype=IO[io]) for k in (1, 2, 3))
    lam = torch.linspace(-100.0, 29.0, 130, device=dev)
    check_gates_backward(mssm, x, r, i, lam, randn(dev, 2, 130, seed=4), randn(dev, 2, 130, seed=12))


# ---- projected cross entropy: logits without bounds -------------------------------

def far_logit_inputs(dev, io, tokens):
    """Words 50 and 51 have logits around -3e38 and, in float32, -infinity (sums
    of finite products); the other words' are of order one."""
    hidden, weight, targets = base.loss_inputs(dev, (tokens, 72, 300), io)
    hidden[:, 0], hidden[:, 1] = 1.0, 1.0
    weight[50:52] = 0
    weight[50, 0] = weight[51, 0] = weight[51, 1] = -3e38
    targets = torch.where((targets == 50) | (targets == 51), 7, targets)
    return hidden, weight, targets


@pytest.mark.parametrize("tokens", [20, 150])
def test_linear_cross_entropy_words_far_below(dev, mssm, tokens):
    """A word whose logit is very negative or overflows to -infinity has p = 0: it
    adds nothing to any gradient and its own is 0.  The other words and the hidden
    states keep the bounds of the call without these words."""
    announce("words far below", tokens)
    hidden, weight, targets = far_logit_inputs(dev, "f32", tokens)
    keep = torch.ones(300, dtype=torch.bool, device=dev)
    keep[50:52] = False
    fewer = targets - 2 * ((targets > 51).long())
    _, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    _, want_lse = layers.linear_cross_entropy(hidden, weight[keep], fewer)
    d = base.logit_bound(hidden, weight[keep]).amax(1) + 400 * U32 + 4 * U32 * want_lse.abs()
    within(lse, want_lse, d, "lse")
    dloss = randn(dev, tokens, seed=3)
    got = mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss)
    want = layers.linear_cross_entropy_grad(hidden, weight[keep], fewer, lse, dloss)
    bh, bw = base.loss_grad_bounds(hidden, weight[keep], lse, dloss, want, U32)
    within(got["dhidden"], want["dhidden"], bh + base.half_step(want["dhidden"], hidden) * 1.01, "dhidden")
    within(got["dweight"][keep], want["dweight"], bw + base.half_step(want["dweight"], weight) * 1.01, "dweight")
    assert (got["dweight"][50:52] == 0).all()


@pytest.mark.parametrize("tokens", [20, 150])
@pytest.mark.parametrize("vocab", [3, 300, 20000])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_infinite_logits(dev, mssm, tokens, vocab, io):
    """A logit of infinity makes lse and the loss of another word infinite and its
    own word's NaN; one of -infinity is as if the word were not there; a token
    whose logits all are has lse -infinity."""
    announce("infinite logits", tokens, vocab, io)
    hidden, weight, targets = base.loss_inputs(dev, (tokens, 72, vocab), io)
    targets[targets == -100] = 0
    weight[1] = 0
    weight[1, 0] = float("inf")
    hidden[:, 0] = torch.where(torch.arange(tokens, device=dev) % 2 == 0, 1.0, -1.0)
    targets[:4] = torch.tensor([1, 0, 2, 0], device=dev)
    loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    lo, so = layers.linear_cross_entropy(hidden, weight, targets)
    up = hidden[:, 0] > 0
    assert (lse[up] == float("inf")).all() and (so[up] == float("inf")).all()
    assert torch.equal(torch.isnan(loss), torch.isnan(lo)) and torch.isnan(loss[0])
    assert (loss[up & (targets != 1)] == float("inf")).all()
    fine = ~up & (targets != 1)
    finite = weight.clone()
    finite[1] = 0
    logits = hidden.double() @ finite.double().t()
    d = base.logit_bound(hidden, finite).amax(1) + (vocab + 16 + 2 * (logits.amax(1) - logits.amin(1))) * U32
    d = d + 4 * U32 * torch.where(fine, so.abs(), 0)
    within(lse[fine], so[fine], d[fine], "lse")
    within(loss[fine], lo[fine], (2 * d + 2 * U32 * (so.abs() + logits.abs().amax(1)))[fine], "loss")
    assert (loss[~up & (targets == 1)] == float("inf")).all()
    weight[:] = 0
    weight[:, 0] = float("inf")
    loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    assert (lse[up] == float("inf")).all() and (lse[~up] == -float("inf")).all() and torch.isnan(loss).all()


# ---- layer norm: very wide rows --------------------------------------------------

@pytest.mark.parametrize("dim", [(1 << 25) + 21, (1 << 27) + 5])
def test_layer_norm_backward_of_millions_of_columns(dev, mssm, dim):
    """The columns' sums are added by more workgroups than one dimension of their
    grid holds (from 2^27 columns on more threads than one could)."""
    base.test_layer_norm_backward(dev, mssm, (2, dim), "bf16")
    torch.cuda.empty_cache()


def test_layer_norm_without_columns(dev, mssm):
    """The mean of no values is NaN; nothing that memory held before is returned."""
    for io in IO.values():
        torch.full((5,), 3.0, device=dev)    # freed: what an unwritten result would hold
        y, mean, rstd = mssm.layer_norm_fwd(torch.empty(5, 0, dtype=io, device=dev))
        assert y.shape == (5, 0) and mean.shape == rstd.shape == (5,)
        assert torch.isnan(mean).all() and torch.isnan(rstd).all()
        g = mssm.layer_norm_bwd(y, y.clone(), mean, rstd)
        assert g["dx"].shape == (5, 0) and g["dweight"].shape == g["dbias"].shape == (0,)


# ---- gated linear recurrence: more segments than one published state covers --------

def walk(a, b, start):
    """s_t = a_t s_{t-1} + b_t along dim 1 in 64 bits: stretches side by side, then
    what enters each."""
    batch, steps, dim = a.shape
    width = 512
    count = -(-steps // width)
    s = torch.zeros(batch, count * width, dim, dtype=torch.float64, device=a.device)
    p = torch.ones_like(s)
    s[:, :steps], p[:, :steps] = b, a
    s, p = s.view(batch, count, width, dim), p.view(batch, count, width, dim)
    for k in range(1, width):
        s[:, :, k] += p[:, :, k] * s[:, :, k - 1]
        p[:, :, k] *= p[:, :, k - 1]
    for k in range(count):
        s[:, k] += p[:, k] * start[:, None]
        start = s[:, k, -1]
    return s.view(batch, -1, dim)[:, :steps]


def before_of(s, start):
    return torch.cat([start[:, None], s[:, :-1]], 1)


# io, dim, steps, steps of a span of 512 segments forward
SPANS = [("bf16", 2, 200003, 512 * 176), ("f32", 3, 120007, 512 * 110), ("bf16", 3, 120007, 512 * 110)]


def span_inputs(dev, io, dim, steps, span):
    """Decays that remember most of a span, and inputs of one sign that swell and
    fade over part of one: a state that is missing, late or of another span shows,
    and the bound, relative to sums of magnitudes, is relative to the states."""
    t = torch.arange(steps, device=dev, dtype=torch.float64)[None, :, None]
    phase = torch.arange(dim, device=dev, dtype=torch.float64)[None, None]
    swell = (1 + 0.9 * torch.sin(t * (6.28 / (0.6 * span)) + phase)).float()
    x, dy = (randn(dev, 2, steps, dim, seed=k).abs().mul(swell).to(IO[io]) for k in (1, 5))
    i = randn(dev, 2, steps, dim, seed=2, dtype=IO[io])
    r = randn(dev, 2, steps, dim, seed=3, dtype=IO[io], scale=0.2)
    lam = torch.full((dim,), 2 / (0.7 * span) / 8, dtype=torch.float64, device=dev).expm1().log().float()
    return x, r, i, lam, dy


@pytest.mark.parametrize("io,dim,steps,span", SPANS)
def test_gated_recurrence_forward_over_spans(dev, mssm, io, dim, steps, span):
    announce("spans fwd", io, dim, steps)
    assert steps > 2 * span
    x, r, i, lam, _ = span_inputs(dev, io, dim, steps, span)
    h0 = randn(dev, 2, dim, seed=4).abs() * 300
    y, last = mssm.gated_recurrence_fwd(x, r, i, lam, 8.0, h0=h0)
    _, a, m, _, _, d_a, d_m = gate_bounds(r, lam)
    si = torch.sigmoid(i.double())
    b = m * si * x.double()
    d_b = si * x.double() * d_m + b * (3 * i.double().abs() + 20) * U32
    yo = walk(a, b, h0.double())
    bound = walk(a, 2 * ((d_a + U32 * a) * before_of(yo, h0.double()) + d_b + 2 * U32 * yo), 0 * h0.double())
    assert (bound / yo).max() < 0.1
    within(last, yo[:, -1], bound[:, -1], "h_last")
    within(y, yo, bound + base.half_step(yo, y) * 1.01, "y")


@pytest.mark.parametrize("io,dim,steps,span", SPANS)
def test_gated_recurrence_backward_over_spans(dev, mssm, io, dim, steps, span):
    """The backward's segments are shorter: three spans and more."""
    announce("spans bwd", io, dim, steps)
    x, r, i, lam, dy = span_inputs(dev, io, dim, steps, span)
    h0, dh_last = randn(dev, 2, dim, seed=4).abs() * 300, randn(dev, 2, dim, seed=6).abs() * 1e4
    la, a, m, sr, _, d_a, _ = gate_bounds(r, lam)
    si, X = torch.sigmoid(i.double()), x.double()
    y = walk(a, m * si * X, h0.double()).to(IO[io])
    got = mssm.gated_recurrence_bwd(x, r, i, lam, y, dy, 8.0, h0=h0, dh_last=dh_last)
    # from the end, the carry G' = a (dy + G): everything is positive, so that
    # sizes are the values
    back = lambda v: v.flip(1)  # noqa: E731
    out = walk(back(a), back(a * dy.double()), dh_last.double())
    carry = before_of(out, dh_last.double())
    g = dy.double() + back(carry)
    # an error that enters at a step: of the sum, then of its product with the decay
    e = walk(back(a), back(a) * 2 * U32 * back(g) + 2 * (back(d_a) + U32 * back(a)) * back(g), 0 * dh_last.double())
    d_g = back(before_of(e, 0 * dh_last.double())) + 2 * U32 * g
    assert (d_g / g).max() < 0.1
    before = before_of(y.double(), h0.double())
    w = g * before * a * la - g * si * X * a * a * la / m
    lam64 = lam.double()
    want = {"g": g, "w": w, "dx": g * m * si, "dr": w * (1 - sr), "di": g * m * si * X * (1 - si), "dh0": out[:, -1],
            "dlam": w.sum((0, 1)) * torch.sigmoid(lam64) / layers.softplus(lam64)}
    within_grads(got, want, x, r, i, lam, y, h0, d_g, e[:, -1] + 2 * U32 * out[:, -1])


# ---- layer norm: every group of lanes goes over several rows -----------------------

@pytest.mark.parametrize("shape", [(70001, 5), (70001, 40), (40009, 128), (20011, 250), (9001, 513), (6145, 2560),
                                   (6149, 2048), (2100, 2600), (1100, 9999), (600, 12001)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_layer_norm_rows_in_turn(dev, mssm, shape, io):
    """Rows held by 8 to 1024 lanes, at least two of them and mostly three or more
    in turn in each direction, the last turn not full; the bounds are those of the
    other sizes."""
    announce("norm rows in turn", shape, io)
    base.test_layer_norm_forward(dev, mssm, shape, io)
    base.test_layer_norm_backward(dev, mssm, shape, io)


# ---- projected cross entropy: several pieces of the vocabulary, rows copied ---------

@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_forward_over_copied_pieces(dev, mssm, io):
    """An odd width: weight is copied to aligned rows in two pieces of the
    vocabulary (52224 words, then 7789), with targets at both pieces' ends."""
    tokens, dim, vocab = 40, 2557, 60013
    announce("loss fwd, copied pieces", io)
    hidden, weight, targets = base.loss_inputs(dev, (tokens, dim, vocab), io)
    targets[:8] = torch.tensor([0, 1, 52222, 52223, 52224, 52225, vocab - 2, vocab - 1], device=dev)
    loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    lo, so = layers.linear_cross_entropy(hidden, weight, targets)
    logits = hidden.double() @ weight.double().t()
    # as test_linear_cross_entropy_forward
    d = base.logit_bound(hidden, weight).amax(1) + (vocab + 16 + 2 * (logits.amax(1) - logits.amin(1))) * U32
    d = d + 4 * U32 * so.abs()
    within(lse, so, d, "lse")
    within(loss, lo, 2 * d + 2 * U32 * (so.abs() + logits.abs().amax(1)), "loss")
    assert (loss[targets == -100] == 0).all()


@pytest.mark.parametrize("shape", [(4099, 41, 40001), (2500, 33, 60000)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_backward_over_copied_pieces(dev, mssm, shape, io):
    """The backward with copied rows over pieces of which the last is shorter."""
    announce("loss bwd, copied pieces", shape, io)
    base.test_linear_cross_entropy_backward(dev, mssm, shape, io)
    torch.cuda.empty_cache()

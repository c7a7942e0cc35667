"""GPU parity of the layer norm, the gated linear recurrence and the projected
cross entropy against their float64 definitions.  Needs an MI355X; marked
``gpu``.

Every tolerance is a bound per element that follows from the roundings: a
float32 operation is off by at most U32 = 2^-24 of its result, a hardware
exponential, logarithm, reciprocal or square root by 2 U32, a stored bfloat16 by
2^-8 of its value (half a step), and a float32 sum of n terms, in whatever
order, by n U32 times the sum of their magnitudes."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from oracle import layers  # noqa: E402

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_05_amd
    return selective_state_space_05_amd


def announce(*what):
    print("[layers]", *what, flush=True)


def randn(dev, *shape, seed=0, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).to(dev)


def half_step(t, like):
    """Half a step of the dtype of `like` at the values t."""
    return t.abs() * (torch.finfo(like.dtype).eps / 2) + torch.finfo(like.dtype).tiny


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g where %.3g is allowed" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(bound.expand_as(err)[bad].max()))


# ---- layer norm --------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 63), (7, 64), (3, 65), (1000, 40), (9, 512), (33, 769),
               (2, 2560), (300, 1001), (5, 4097), (3, 8192), (2, 16391), (2, 40007)]


def norm_bounds(x, w, b, mean, rstd):
    """Bounds of mean, rstd and y (before y's own rounding)."""
    dim = x.shape[-1]
    n = dim + 8
    ax = x.abs()
    d_mean = (n * U32) * ax.mean(-1)
    # the variance sums (x - mu)^2 of a shifted mu: its own square on top
    var = (x - mean[:, None]).square().mean(-1)
    dev_ = (x - mean[:, None]).abs()
    d_var = (n + 4) * U32 * var + d_mean.square() + 2 * (U32 * (ax.amax(-1) + mean.abs()) + d_mean) * dev_.mean(-1)
    d_rstd = rstd * (0.5 * d_var * rstd.square() + 8 * U32)
    w = torch.ones_like(x[0]) if w is None else w.double()
    ab = torch.zeros_like(w) if b is None else b.double().abs()
    d_diff = d_mean[:, None] + U32 * (ax + mean.abs()[:, None]) + d_var[:, None] * 0
    xhat = dev_ * rstd[:, None]
    d_y = w.abs() * (d_diff * rstd[:, None] + dev_ * d_rstd[:, None] + 4 * U32 * xhat) + 2 * U32 * (xhat * w.abs() + ab)
    return d_mean, d_rstd, d_y


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_layer_norm_forward(dev, mssm, shape, io):
    announce("norm fwd", shape, io)
    rows, dim = shape
    x = randn(dev, rows, dim, seed=dim, dtype=IO[io], scale=2.0, shift=0.7)
    for affine in (True, False):
        w = randn(dev, dim, seed=1, shift=1.0, scale=0.3) if affine else None
        b = randn(dev, dim, seed=2) if affine else None
        y, mean, rstd = mssm.layer_norm_fwd(x, w, b, 1e-5)
        yo, mo, ro = layers.layer_norm(x, w, b, 1e-5)
        d_mean, d_rstd, d_y = norm_bounds(x.double(), w, b, mo, ro)
        within(mean, mo, d_mean, "mean")
        within(rstd, ro, d_rstd, "rstd")
        within(y, yo, d_y + half_step(yo, y) * 1.01, "y")


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_layer_norm_backward(dev, mssm, shape, io):
    announce("norm bwd", shape, io)
    rows, dim = shape
    x = randn(dev, rows, dim, seed=dim, dtype=IO[io], scale=2.0, shift=0.7)
    dy = randn(dev, rows, dim, seed=dim + 1, dtype=IO[io])
    w = randn(dev, dim, seed=1, shift=1.0, scale=0.3)
    _, mo, ro = layers.layer_norm(x, w, None, 1e-5)
    mean, rstd = mo.float(), ro.float()
    for weight in (w, None):
        g = mssm.layer_norm_bwd(dy, x, mean, rstd, weight)
        want = layers.layer_norm_grad(dy, x, mean, rstd, weight)
        X, D, R = x.double(), dy.double(), rstd.double()[:, None]
        xhat = (X - mean.double()[:, None]) * R
        # xhat is off by the rounding of the difference and of the product
        d_xhat = (U32 * (X - mean.double()[:, None]).abs()) * R + 2 * U32 * xhat.abs()
        e = D if weight is None else D * weight.double()
        n = (dim + 8) * U32
        d_m0 = n * e.abs().mean(-1, keepdim=True)
        d_m1 = n * (e * xhat).abs().mean(-1, keepdim=True) + (e.abs() * d_xhat).mean(-1, keepdim=True)
        m0, m1 = e.mean(-1, keepdim=True), (e * xhat).mean(-1, keepdim=True)
        size = e.abs() + m0.abs() + (xhat * m1).abs()
        d_dx = R * (d_m0 + xhat.abs() * d_m1 + d_xhat * m1.abs() + 6 * U32 * size)
        within(g["dx"], want["dx"], d_dx + half_step(want["dx"], g["dx"]) * 1.01, "dx")
        nr = (rows + 8) * U32
        within(g["dweight"], want["dweight"], nr * (D * xhat).abs().sum(0) + (D.abs() * d_xhat).sum(0), "dweight")
        within(g["dbias"], want["dbias"], nr * D.abs().sum(0) + 1e-30, "dbias")


def test_layer_norm_unaligned_rows_and_higher_rank(dev, mssm):
    """Rows that start at any element, tensors of rank 1 and 3, and outputs
    next to memory that must not be touched."""
    announce("norm unaligned")
    for io in IO.values():
        for off in (1, 3):
            buf = randn(dev, 3 * 129 + 8, seed=off, dtype=io)
            x = buf[off:off + 3 * 129].view(3, 129)
            guard = torch.full((3 * 129 + 8,), 7.0, dtype=io, device=dev)
            out = guard[off:off + 3 * 129].view(3, 129)
            y, _, _ = mssm.layer_norm_fwd(x, out=out)
            assert torch.equal(y, mssm.layer_norm_fwd(x.clone())[0])
            assert (guard[:off] == 7).all() and (guard[off + 3 * 129:] == 7).all()
    x = randn(dev, 2, 3, 40, seed=5)
    y, mean, _ = mssm.layer_norm_fwd(x)
    assert mean.shape == (2, 3)
    assert torch.equal(y, mssm.layer_norm_fwd(x.view(6, 40))[0].view(2, 3, 40))
    assert mssm.layer_norm_fwd(x[0, 0])[1].shape == ()


def test_layer_norm_special_rows(dev, mssm):
    """A constant row has zero variance; a row with a NaN or an infinity is NaN
    and leaves the others alone; no rows give zero weight gradients."""
    announce("norm special rows")
    x = randn(dev, 4, 300, seed=9)
    x[0] = 3.0
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y, mean, rstd = mssm.layer_norm_fwd(x, eps=1e-5)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and torch.isnan(y[2]).any()
    assert torch.equal(y[3], mssm.layer_norm_fwd(x[3:4].clone())[0][0])
    g = mssm.layer_norm_bwd(x[:0], x[:0], mean[:0], rstd[:0])
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all() and g["dx"].shape == (0, 300)


def test_layer_norm_gradient_is_the_difference_quotient(dev, mssm):
    """Along a direction: <dx, d> equals the central difference of <y, dy> of
    the float64 forward, whose error at step 1e-6 is below 1e-6 of the scale."""
    announce("norm differences")
    x, dy = randn(dev, 6, 96, seed=1), randn(dev, 6, 96, seed=2)
    d = randn(dev, 6, 96, seed=3).double()
    _, mean, rstd = mssm.layer_norm_fwd(x)
    g = mssm.layer_norm_bwd(dy, x, mean, rstd)
    f = lambda s: (layers.layer_norm(x.double() + s * d)[0] * dy.double()).sum()  # noqa: E731
    quotient = (f(1e-6) - f(-1e-6)) / 2e-6
    got = (g["dx"].double() * d).sum()
    scale = (g["dx"].double() * d).abs().sum()
    assert abs(got - quotient) <= scale * 1e-5


def test_layer_norm_repeats_bit_for_bit(dev, mssm):
    announce("norm repeat")
    x, dy = randn(dev, 3000, 513, seed=1, dtype=torch.bfloat16), randn(dev, 3000, 513, seed=2, dtype=torch.bfloat16)
    _, mean, rstd = mssm.layer_norm_fwd(x)
    a, b = (mssm.layer_norm_bwd(dy, x, mean, rstd) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)


# ---- gated linear recurrence ---------------------------------------------------

REC_SHAPES = [(1, 1, 1), (2, 1, 64), (1, 2, 3), (3, 5, 2), (1, 17, 65), (2, 33, 63), (1, 127, 129), (2, 130, 64),
              (1, 257, 70), (3, 300, 37), (1, 1025, 130), (2, 2049, 31), (1, 9001, 34), (1, 33000, 3)]


def rec_inputs(dev, shape, io, h0, seed=0):
    batch, steps, dim = shape
    x, r, i = (randn(dev, *shape, seed=seed + k + steps, dtype=IO[io]) for k in range(3))
    lam = randn(dev, dim, seed=seed + 7, scale=2.0, shift=-4.0)
    return x, r, i, lam, (randn(dev, batch, dim, seed=seed + 8) if h0 else None)


def rec_coefficient_bounds(x, r, i, lam):
    """Bounds of the computed a and input term b.  sigmoid: the exponent's
    rounding times |r|, then three operations; log a: softplus (4) and two
    products; a - 1: at most eight operations, or an exponential whose
    argument's rounding counts; m: half of its radicand's relative error."""
    la, a, m, sr, si = layers.gates(r, i, lam, 8.0)
    rel_la = (3 * r.double().abs() + 24) * U32
    d_p = la.abs() * a * rel_la + (8 * U32) * (1 - a) + 2 * U32 * la.abs() * a
    d_a = d_p + U32
    d_p = d_p + torch.where(la < -0.3, 2 * U32 * torch.ones_like(a), torch.zeros_like(a))
    p = 1 - a
    d_b = m * si * x.double().abs() * (0.5 * (d_p / p.clamp(min=1e-300)).clamp(max=1.0) * 2
                                       + (3 * i.double().abs() + 20) * U32)
    return la, a, m, sr, si, d_a, d_b


def rec_forward_bound(x, r, i, lam, y, h0):
    """Bound of every state: errors enter at each step and decay with it.  The
    states' carries pass as products of decays, each off by d_a + U32: twice
    the step's own error covers that association."""
    _, a, _, _, _, d_a, d_b = rec_coefficient_bounds(x, r, i, lam)
    e = torch.zeros_like(y[:, 0])
    out = torch.empty_like(y)
    prev = torch.zeros_like(y[:, 0]) if h0 is None else h0.double().abs()
    size = prev.clone()    # sum of magnitudes: what an intermediate state may reach
    b = layers.gates(r, i, lam, 8.0)
    b = b[2] * b[4] * x.double().abs()
    for t in range(y.shape[1]):
        new = a[:, t] * size + b[:, t]
        e = a[:, t] * e + 2 * ((d_a[:, t] + U32) * size + d_b[:, t] + 2 * U32 * new)
        size = new
        out[:, t] = e
    return out


@pytest.mark.parametrize("shape", REC_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("h0", [False, True])
def test_gated_recurrence_forward(dev, mssm, shape, io, h0):
    announce("recurrence fwd", shape, io, h0)
    x, r, i, lam, start = rec_inputs(dev, shape, io, h0)
    y, last = mssm.gated_recurrence_fwd(x, r, i, lam, 8.0, h0=start)
    yo, lo = layers.gated_recurrence(x, r, i, lam, 8.0, start)
    bound = rec_forward_bound(x, r, i, lam, yo, start)
    within(last, lo, bound[:, -1] + 1e-30, "h_last")
    within(y, yo, bound + half_step(yo, y) * 1.01, "y")


@pytest.mark.parametrize("shape", REC_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("h0", [False, True])
def test_gated_recurrence_backward(dev, mssm, shape, io, h0):
    announce("recurrence bwd", shape, io, h0)
    batch, steps, dim = shape
    x, r, i, lam, start = rec_inputs(dev, shape, io, h0)
    y = layers.gated_recurrence(x, r, i, lam, 8.0, start)[0].to(IO[io])
    dy = randn(dev, *shape, seed=11, dtype=IO[io])
    dhl = randn(dev, batch, dim, seed=12) if h0 else None
    got = mssm.gated_recurrence_bwd(x, r, i, lam, y, dy, 8.0, h0=start, dh_last=dhl)
    want = layers.gated_recurrence_grad(x, r, i, lam, y, dy, 8.0, start, dhl)
    la, a, m, sr, si, d_a, d_b = rec_coefficient_bounds(x, r, i, lam)
    # g runs the recurrence from the end: its error likewise
    e = torch.zeros_like(a[:, 0])
    size = torch.zeros_like(a[:, 0]) if dhl is None else dhl.double().abs()
    d_g, g_size = torch.empty_like(a), torch.empty_like(a)
    for t in range(steps - 1, -1, -1):
        size = dy[:, t].double().abs() + size
        e = e + 2 * U32 * size
        d_g[:, t], g_size[:, t] = e, size
        e = a[:, t] * e + 2 * (d_a[:, t] + U32) * size
        size = a[:, t] * size
    g = want["g"].abs()
    ax = x.double().abs()
    rel_m = 0.5 * (d_a / (1 - a).clamp(min=1e-300)).clamp(max=2.0) + 8 * U32
    # above -0.35, a - 1 is formed without the rounding of a
    rel_m = torch.where(la > -0.3, (3 * r.double().abs() + 32) * U32, rel_m)
    rel_s = (3 * i.double().abs() + 8) * U32
    dx = m * si
    within(got["dx"], want["dx"], d_g * dx + g * dx * (rel_m + rel_s + 4 * U32)
           + half_step(want["dx"], got["dx"]) * 1.01, "dx")
    ddi = m * si * ax * (1 - si)
    # 1 - sigmoid: its absolute error is sigmoid's plus one rounding
    within(got["di"], want["di"], d_g * ddi + g * ddi * (rel_m + rel_s + 4 * U32)
           + g * m * si * ax * (si * rel_s + U32) + half_step(want["di"], got["di"]) * 1.01, "di")
    start64 = torch.zeros_like(a[:, :1]) if start is None else start.double()[:, None]
    before = torch.cat([start64, y.double()[:, :-1]], 1).abs()
    q = torch.where(m > 0, la / m, torch.zeros_like(m)).abs()
    one = before * a * la.abs()
    two = si * ax * a * a * q
    rel_la = (3 * r.double().abs() + 24) * U32
    d_w = d_g * (one + two) + g * (one * (rel_la + 6 * U32) + two * (rel_la + rel_m + rel_s + 10 * U32)
                                   + (before * la.abs() + 2 * si * ax * a * q) * d_a)
    within(got["dr"], want["dr"], d_w * (1 - sr) + want["w"].abs() * (sr * rel_la + 2 * U32)
           + half_step(want["dr"], got["dr"]) * 1.01, "dr")
    ratio = torch.sigmoid(lam.double()) / layers.softplus(lam.double())
    n = (batch * steps + 16) * U32
    within(got["dlam"], want["dlam"], ratio * (d_w.sum((0, 1)) + n * want["w"].abs().sum((0, 1)))
           + want["dlam"].abs() * 16 * U32 + 1e-30, "dlam")
    within(got["dh0"], want["dh0"], e + U32 * g_size[:, 0] + 1e-30, "dh0")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_recurrence_update_equals_one_step(dev, mssm, io):
    announce("recurrence update", io)
    for batch, dim in [(1, 1), (3, 65), (8, 512), (5, 1001)]:
        x, r, i, lam, state = rec_inputs(dev, (batch, 1, dim), io, True)
        y, last = mssm.gated_recurrence_fwd(x, r, i, lam, h0=state)
        got = mssm.gated_recurrence_update(state, x[:, 0].contiguous(), r[:, 0].contiguous(),
                                           i[:, 0].contiguous(), lam)
        assert torch.equal(got, y[:, 0]) and torch.equal(state, last)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gated_recurrence_in_pieces_and_in_place(dev, mssm, io):
    """A sequence in pieces, the state advanced in place (h0 the h_out buffer):
    both stay within the bound of the whole."""
    announce("recurrence pieces", io)
    x, r, i, lam, start = rec_inputs(dev, (2, 1500, 70), io, True)
    state, ys = start.clone(), []
    for lo, hi in ((0, 1), (1, 700), (700, 1500)):
        y, h = mssm.gated_recurrence_fwd(x[:, lo:hi].contiguous(), r[:, lo:hi].contiguous(),
                                         i[:, lo:hi].contiguous(), lam, h0=state, h_out=state)
        assert h.data_ptr() == state.data_ptr()
        ys.append(y)
    yo, lo_ = layers.gated_recurrence(x, r, i, lam, 8.0, start)
    bound = rec_forward_bound(x, r, i, lam, yo, start)
    within(torch.cat(ys, 1), yo, bound + half_step(yo, ys[0]) * 1.01, "y")
    within(state, lo_, bound[:, -1], "state")


def test_gated_recurrence_empty_sequence(dev, mssm):
    announce("recurrence L=0")
    x = torch.empty(2, 0, 5, device=dev)
    lam, h0 = randn(dev, 5), randn(dev, 2, 5, seed=1)
    y, h = mssm.gated_recurrence_fwd(x, x.clone(), x.clone(), lam, h0=h0)
    assert y.shape == (2, 0, 5) and torch.equal(h, h0)
    assert (mssm.gated_recurrence_fwd(x, x.clone(), x.clone(), lam)[1] == 0).all()
    g = mssm.gated_recurrence_bwd(x, x.clone(), x.clone(), lam, x.clone(), x.clone(), h0=h0, dh_last=h0.clone())
    assert torch.equal(g["dh0"], h0) and (g["dlam"] == 0).all()


def test_gated_recurrence_saturated_gates(dev, mssm):
    """Closed gates keep the state bit for bit; open ones drop it; infinite
    gate inputs and lam far out give finite outputs and gradients."""
    announce("recurrence saturated")
    shape = (2, 300, 66)
    x, _, i, lam, h0 = rec_inputs(dev, shape, "f32", True)
    for value in (-2000.0, -float("inf")):
        r = torch.full(shape, value, device=dev)
        y, last = mssm.gated_recurrence_fwd(x, r, i, lam, h0=h0)
        assert torch.equal(last, h0) and torch.equal(y, h0[:, None].expand(shape))
        g = mssm.gated_recurrence_bwd(x, r, i, lam, y, x.clone(), h0=h0)
        assert all(torch.isfinite(v).all() for v in g.values()) and (g["dr"] == 0).all()
    r = torch.full(shape, float("inf"), device=dev)
    lam = torch.full((66,), 60.0, device=dev)
    lam[0] = -200.0
    y, last = mssm.gated_recurrence_fwd(x, r, i, lam, h0=h0)
    want = torch.sigmoid(i.double()) * x.double()
    within(y[:, :, 1:], want[:, :, 1:], want[:, :, 1:].abs() * (3 * i.double().abs()[:, :, 1:] + 16) * U32 + 1e-37,
           "open gates")
    assert torch.equal(last[:, 0], h0[:, 0])
    g = mssm.gated_recurrence_bwd(x, r, i, lam, y, x.clone(), h0=h0)
    assert all(torch.isfinite(v).all() for v in g.values())


def test_gated_recurrence_keeps_infinities_in_their_channel(dev, mssm):
    announce("recurrence inf")
    shape = (1, 400, 70)
    x, r, i, lam, _ = rec_inputs(dev, shape, "f32", False)
    clean = mssm.gated_recurrence_fwd(x, r, i, lam)[0]
    x[0, 200, 13], x[0, 100, 40] = float("inf"), float("nan")
    y = mssm.gated_recurrence_fwd(x, r, i, lam)[0]
    keep = [c for c in range(70) if c not in (13, 40)]
    assert torch.equal(y[:, :, keep], clean[:, :, keep])
    assert torch.equal(y[0, :200, 13], clean[0, :200, 13]) and torch.isinf(y[0, 200:, 13]).all()
    assert torch.equal(y[0, :100, 40], clean[0, :100, 40]) and torch.isnan(y[0, 100:, 40]).all()


def test_gated_recurrence_repeats_bit_for_bit(dev, mssm):
    announce("recurrence repeat")
    x, r, i, lam, h0 = rec_inputs(dev, (1, 20011, 200), "bf16", True)
    runs = []
    for _ in range(3):
        y, h = mssm.gated_recurrence_fwd(x, r, i, lam, h0=h0)
        runs.append([y, h] + list(mssm.gated_recurrence_bwd(x, r, i, lam, y, x.clone(), h0=h0).values()))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_gated_recurrence_unaligned(dev, mssm):
    """Tensors that start at any element, outputs next to guards."""
    announce("recurrence unaligned")
    for io in IO.values():
        shape, n = (2, 70, 33), 2 * 70 * 33
        bufs = [randn(dev, n + 8, seed=k, dtype=io) for k in range(3)]
        lam = randn(dev, 33, shift=-4.0)
        for off in (1, 3):
            x, r, i = (b[off:off + n].view(shape) for b in bufs)
            guard = torch.full((n + 8,), 7.0, dtype=io, device=dev)
            y, h = mssm.gated_recurrence_fwd(x, r, i, lam, out=guard[off:off + n].view(shape))
            yc, hc = mssm.gated_recurrence_fwd(x.clone(), r.clone(), i.clone(), lam)
            assert torch.equal(y, yc) and torch.equal(h, hc)
            assert (guard[:off] == 7).all() and (guard[off + n:] == 7).all()


def test_gated_recurrence_gradient_is_the_difference_quotient(dev, mssm):
    """Along a direction of r and of lam, against the float64 forward at step
    1e-6; the gradient reads y in float32, off by 1e-6 of the scale at most."""
    announce("recurrence differences")
    x, r, i, lam, h0 = rec_inputs(dev, (2, 60, 20), "f32", True)
    dy = randn(dev, 2, 60, 20, seed=21)
    y, _ = mssm.gated_recurrence_fwd(x, r, i, lam, h0=h0)
    g = mssm.gated_recurrence_bwd(x, r, i, lam, y, dy, h0=h0)
    dr, dl = randn(dev, 2, 60, 20, seed=22).double(), randn(dev, 20, seed=23).double()
    f = lambda s, u: (layers.gated_recurrence(x, r.double() + s * dr, i, lam.double() + u * dl, 8.0, h0)[0]  # noqa: E731
                      * dy.double()).sum()
    for key, d, q in (("dr", dr, (f(1e-6, 0) - f(-1e-6, 0)) / 2e-6), ("dlam", dl, (f(0, 1e-6) - f(0, -1e-6)) / 2e-6)):
        terms = g[key].double() * d
        assert abs(terms.sum() - q) <= 1e-5 * terms.abs().sum(), key


# ---- projected cross entropy ----------------------------------------------------

LOSS_SHAPES = [(1, 1, 1), (1, 8, 1000), (5, 7, 3), (16, 64, 333), (130, 72, 517), (64, 136, 129), (257, 129, 1111),
               (300, 256, 2050), (513, 40, 700), (33, 2561, 300)]


def loss_inputs(dev, shape, io, seed=0):
    tokens, dim, vocab = shape
    hidden = randn(dev, tokens, dim, seed=seed + dim, dtype=IO[io])
    weight = randn(dev, vocab, dim, seed=seed + vocab, dtype=IO[io], scale=2.0 / math.sqrt(dim))
    g = torch.Generator().manual_seed(seed + tokens)
    targets = torch.randint(0, vocab, (tokens,), generator=g)
    if tokens > 2:
        targets[tokens // 2] = -100
        targets[0], targets[-1] = vocab - 1, 0
    return hidden, weight, targets.to(dev)


def logit_bound(hidden, weight):
    """Sums of dim products, exact in float32 (bf16) or rounded (float32)."""
    return (hidden.shape[1] + 2) * U32 * (hidden.double().abs() @ weight.double().abs().t())


@pytest.mark.parametrize("shape", LOSS_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_forward(dev, mssm, shape, io):
    announce("loss fwd", shape, io)
    hidden, weight, targets = loss_inputs(dev, shape, io)
    loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    lo, so = layers.linear_cross_entropy(hidden, weight, targets)
    logits = hidden.double() @ weight.double().t()
    # the sum of exponentials: their arguments' roundings, and vocab additions
    d = logit_bound(hidden, weight).amax(1) + (shape[2] + 16 + 2 * (logits.amax(1) - logits.amin(1))) * U32
    d = d + 4 * U32 * so.abs()
    within(lse, so, d, "lse")
    within(loss, lo, 2 * d + 2 * U32 * (so.abs() + logits.abs().amax(1)), "loss")
    assert (loss[targets == -100] == 0).all()


def loss_grad_bounds(hidden, weight, lse, dloss, want, step):
    """p is off by its exponent's error and rounds once to the I/O dtype (half
    a step, `step`); the gradients' sums over words or tokens add theirs."""
    h, w, p = hidden.double().abs(), weight.double().abs(), want["p"].abs()
    soft = torch.exp(hidden.double() @ weight.double().t() - lse.double()[:, None]) * dloss.double().abs()[:, None]
    d_l = logit_bound(hidden, weight) + 8 * U32 * (1 + (hidden.double() @ weight.double().t()).abs()
                                                   + lse.double().abs()[:, None])
    d_p = soft * (d_l + 4 * U32) + p * (step + 2 * U32)
    d_p[want["p"] == 0] = 0
    return (d_p @ w + (weight.shape[0] + 8) * U32 * (p @ w),
            d_p.t() @ h + (hidden.shape[0] + 8) * U32 * (p.t() @ h))


@pytest.mark.parametrize("shape", LOSS_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_backward(dev, mssm, shape, io):
    announce("loss bwd", shape, io)
    hidden, weight, targets = loss_inputs(dev, shape, io)
    lse = layers.linear_cross_entropy(hidden, weight, targets)[1].float()
    dloss = randn(dev, shape[0], seed=3)
    got = mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss)
    want = layers.linear_cross_entropy_grad(hidden, weight, targets, lse, dloss)
    bh, bw = loss_grad_bounds(hidden, weight, lse, dloss, want, torch.finfo(IO[io]).eps / 2)
    within(got["dhidden"], want["dhidden"], bh + half_step(want["dhidden"], hidden) * 1.01, "dhidden")
    within(got["dweight"], want["dweight"], bw + half_step(want["dweight"], weight) * 1.01, "dweight")
    assert (got["dhidden"][targets == -100] == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_over_several_pieces(dev, mssm, io):
    """More tokens times words than one piece of the vocabulary holds, with a
    ragged last piece; float64 on the GPU."""
    shape = (4099, 40, 40001)
    announce("loss pieces", shape, io)
    hidden, weight, targets = loss_inputs(dev, shape, io)
    loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    lo, so = layers.linear_cross_entropy(hidden, weight, targets)
    d = logit_bound(hidden, weight).amax(1) + (shape[2] + 64) * U32 + 4 * U32 * so.abs()
    within(lse, so, d, "lse")
    within(loss, lo, 2 * d + 64 * U32, "loss")
    dloss = randn(dev, shape[0], seed=3)
    got = mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss)
    want = layers.linear_cross_entropy_grad(hidden, weight, targets, lse, dloss)
    bh, bw = loss_grad_bounds(hidden, weight, lse, dloss, want, torch.finfo(IO[io]).eps / 2)
    within(got["dhidden"], want["dhidden"], bh + half_step(want["dhidden"], hidden) * 1.01, "dhidden")
    within(got["dweight"], want["dweight"], bw + half_step(want["dweight"], weight) * 1.01, "dweight")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_masked_tokens_hold_anything(dev, mssm, io):
    """Ignored tokens may hold NaN and infinities, in hidden, lse and dloss:
    nothing of them reaches a gradient; all tokens ignored gives zeros."""
    announce("loss masked", io)
    hidden, weight, targets = loss_inputs(dev, (70, 72, 300), io)
    dloss = randn(dev, 70, seed=3)
    lse = layers.linear_cross_entropy(hidden, weight, targets)[1].float()
    skip = torch.arange(70, device=dev) % 3 == 1
    targets[skip] = -100
    clean_h = hidden.clone()
    clean_h[skip] = 0
    clean = mssm.linear_cross_entropy_bwd(clean_h, weight, targets, lse, dloss)
    hidden[skip], lse[skip], dloss[skip] = float("nan"), float("inf"), float("nan")
    hidden[1] = float("inf")
    loss, _ = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    assert (loss[skip] == 0).all() and torch.isfinite(loss).all()
    got = mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss)
    assert torch.equal(got["dhidden"], clean["dhidden"]) and torch.equal(got["dweight"], clean["dweight"])
    targets[:] = -100
    got = mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss)
    assert (got["dhidden"] == 0).all() and (got["dweight"] == 0).all()


def test_linear_cross_entropy_bad_targets_and_other_ignore_index(dev, mssm):
    """A target outside the vocabulary gives NaN for its token alone; any value
    may be the ignored one."""
    announce("loss bad targets")
    hidden, weight, targets = loss_inputs(dev, (40, 64, 200), "bf16")
    targets[targets == -100] = 5
    good, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    bad = targets.clone()
    bad[3], bad[7], bad[11] = 200, -1, 1 << 40
    loss, _ = mssm.linear_cross_entropy_fwd(hidden, weight, bad)
    odd = torch.zeros(40, dtype=torch.bool, device=dev)
    odd[[3, 7, 11]] = True
    assert torch.isnan(loss[odd]).all() and torch.equal(loss[~odd], good[~odd])
    dloss = torch.ones(40, device=dev)
    g = mssm.linear_cross_entropy_bwd(hidden, weight, bad, lse, dloss)
    assert torch.isnan(g["dhidden"][odd]).all() and torch.isfinite(g["dhidden"][~odd]).all()
    bad[3], bad[7], bad[11] = 9, 9, 9
    loss, _ = mssm.linear_cross_entropy_fwd(hidden, weight, bad, ignore_index=9)
    assert (loss[bad == 9] == 0).all()


def test_linear_cross_entropy_large_logits(dev, mssm):
    """Logits of thousands of either sign neither overflow nor vanish."""
    announce("loss large logits")
    hidden, weight, targets = loss_inputs(dev, (50, 64, 400), "f32")
    hidden *= 500.0
    loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    lo, so = layers.linear_cross_entropy(hidden, weight, targets)
    d = logit_bound(hidden, weight).amax(1) + 500 * U32 + 8 * U32 * so.abs()
    within(lse, so, d, "lse")
    within(loss, lo, 2 * d + 8 * U32 * so.abs(), "loss")


def test_linear_cross_entropy_unaligned_and_empty(dev, mssm):
    announce("loss unaligned")
    for io in IO.values():
        hb, wb = randn(dev, 20 * 64 + 8, seed=1, dtype=io), randn(dev, 90 * 64 + 8, seed=2, dtype=io)
        targets = torch.arange(20, device=dev)
        h, w = hb[1:1 + 20 * 64].view(20, 64), wb[3:3 + 90 * 64].view(90, 64)
        loss, lse = mssm.linear_cross_entropy_fwd(h, w, targets)
        lc, sc = mssm.linear_cross_entropy_fwd(h.clone(), w.clone(), targets)
        assert torch.equal(loss, lc) and torch.equal(lse, sc)
        dl = torch.ones(20, device=dev)
        a = mssm.linear_cross_entropy_bwd(h, w, targets, lse, dl)
        b = mssm.linear_cross_entropy_bwd(h.clone(), w.clone(), targets, lse, dl)
        assert torch.equal(a["dhidden"], b["dhidden"]) and torch.equal(a["dweight"], b["dweight"])
        loss, lse = mssm.linear_cross_entropy_fwd(h[:0], w, targets[:0])
        assert loss.shape == (0,)
        g = mssm.linear_cross_entropy_bwd(h[:0], w, targets[:0], lse, dl[:0])
        assert (g["dweight"] == 0).all()


def test_linear_cross_entropy_gradient_is_the_difference_quotient(dev, mssm):
    announce("loss differences")
    hidden, weight, targets = loss_inputs(dev, (30, 48, 150), "f32")
    dloss = randn(dev, 30, seed=4)
    _, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
    g = mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse, dloss)
    dh, dw = randn(dev, 30, 48, seed=5).double(), randn(dev, 150, 48, seed=6).double()
    f = lambda s, u: (layers.linear_cross_entropy(hidden.double() + s * dh, weight.double() + u * dw, targets)[0]  # noqa: E731
                      * dloss.double()).sum()
    for key, d, q in (("dhidden", dh, (f(1e-6, 0) - f(-1e-6, 0)) / 2e-6),
                      ("dweight", dw, (f(0, 1e-6) - f(0, -1e-6)) / 2e-6)):
        terms = g[key].double() * d
        assert abs(terms.sum() - q) <= 1e-5 * terms.abs().sum(), key


def test_linear_cross_entropy_repeats_bit_for_bit(dev, mssm):
    announce("loss repeat")
    hidden, weight, targets = loss_inputs(dev, (513, 264, 3001), "bf16")
    runs = []
    for _ in range(2):
        loss, lse = mssm.linear_cross_entropy_fwd(hidden, weight, targets)
        runs.append([loss, lse] + list(mssm.linear_cross_entropy_bwd(hidden, weight, targets, lse,
                                                                     torch.ones_like(loss)).values()))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ---- streams and graphs ----------------------------------------------------------

def everything(mssm, t):
    y, mean, rstd = mssm.layer_norm_fwd(t["x"], t["w"])
    g = mssm.layer_norm_bwd(t["dy"], t["x"], mean, rstd, t["w"])
    h, last = mssm.gated_recurrence_fwd(t["x"], t["r"], t["i"], t["lam"])
    gr = mssm.gated_recurrence_bwd(t["x"], t["r"], t["i"], t["lam"], h, t["dy"])
    flat = h.view(-1, h.shape[-1])
    loss, lse = mssm.linear_cross_entropy_fwd(flat, t["vocab"], t["targets"])
    gl = mssm.linear_cross_entropy_bwd(flat, t["vocab"], t["targets"], lse, t["dloss"])
    return [y, mean, rstd, h, last, loss, lse] + [v for d in (g, gr, gl) for v in d.values()]


def together_inputs(dev, seed):
    shape = (2, 600, 72)
    t = {k: randn(dev, *shape, seed=seed + n, dtype=torch.bfloat16) for n, k in enumerate(("x", "r", "i", "dy"))}
    t["w"], t["lam"] = randn(dev, 72, seed=seed + 5), randn(dev, 72, seed=seed + 6, shift=-4.0)
    t["vocab"] = randn(dev, 999, 72, seed=seed + 7, dtype=torch.bfloat16, scale=0.2)
    t["targets"] = torch.arange(1200, device=dev) % 999
    t["dloss"] = torch.full((1200,), 1.0 / 1200, device=dev)
    return t


def test_layers_on_another_stream(dev, mssm):
    announce("layers on another stream")
    t = together_inputs(dev, 50)
    want = everything(mssm, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = everything(mssm, t)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layers_in_a_graph(dev, mssm):
    """Captured once, replayed on new values with eager work in between: every
    replay equals the eager result."""
    announce("layers in a graph")
    t = together_inputs(dev, 60)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        everything(mssm, t)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything(mssm, t)
    for k in range(4):
        for key, v in together_inputs(dev, 70 + k).items():
            t[key].copy_(v)
        want = [v.clone() for v in everything(mssm, t)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


# ---- sizes at which another kernel or tile takes over ---------------------------

@pytest.mark.parametrize("shape", [(700, 2600), (520, 6001), (3, 9999), (2, 12001), (2, 16384), (2, 20011), (2, 24577)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_layer_norm_wide_rows(dev, mssm, shape, io):
    """Rows held by several waves, with more rows than workgroups, and rows that
    no workgroup holds; the bounds are those of the other sizes."""
    test_layer_norm_forward(dev, mssm, shape, io)
    test_layer_norm_backward(dev, mssm, shape, io)


@pytest.mark.parametrize("shape", [(600, 264, 25001), (24, 136, 20000), (17, 2560, 130), (200, 72, 33000)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_cross_entropy_tiles(dev, mssm, shape, io):
    """The largest tiles, the narrow ones and those between, with ends that no
    tile divides; the bounds are those of the other sizes."""
    test_linear_cross_entropy_forward(dev, mssm, shape, io)
    test_linear_cross_entropy_backward(dev, mssm, shape, io)

"""The float64 definitions of the layer norm, the gated linear recurrence and
the projected cross entropy: gradients against central differences of the
forwards, and the properties that follow from the definitions.  CPU only."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from oracle import layers  # noqa: E402

STEP = 1e-5
# central differences of functions of order 1 with third derivatives of order
# 10: STEP^2 * 10 / 6 truncation plus 2^-52 / STEP rounding, both below 1e-9
# times the terms summed
TOL = 1e-7


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g, dtype=torch.float64) * scale


def directional(f, args, key, direction):
    """d/ds f(args with args[key] + s direction) at 0."""
    up, down = dict(args), dict(args)
    up[key] = args[key] + STEP * direction
    down[key] = args[key] - STEP * direction
    return (f(**up) - f(**down)) / (2 * STEP)


def check(f, args, grads):
    for k, (key, grad) in enumerate(grads.items()):
        d = rand(*args[key].shape, seed=100 + k)
        got = directional(f, args, key, d)
        want = (grad * d).sum()
        assert abs(got - want) <= TOL * (1 + abs(want)), (key, float(got), float(want))


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 32)])
def test_layer_norm_gradient(rows, dim):
    x, w, b, dy = rand(rows, dim), rand(dim, seed=1), rand(dim, seed=2), rand(rows, dim, seed=3)

    def f(x, w, b):
        return (layers.layer_norm(x, w, b)[0] * dy).sum()

    _, mean, rstd = layers.layer_norm(x, w, b)
    g = layers.layer_norm_grad(dy, x, mean, rstd, w)
    if dim > 1:   # at dim 1 the output does not depend on x: 0 = 0 up to rstd ~ 300
        check(f, dict(x=x, w=w, b=b), {"x": g["dx"], "w": g["dweight"], "b": g["dbias"]})
    else:
        check(f, dict(x=x, w=w, b=b), {"w": g["dweight"], "b": g["dbias"]})
        assert g["dx"].abs().max() < 1e-9


@pytest.mark.parametrize("h0", [False, True])
def test_gated_recurrence_gradient(h0):
    batch, steps, dim = 2, 9, 5
    a = dict(x=rand(batch, steps, dim), r=rand(batch, steps, dim, seed=1), i=rand(batch, steps, dim, seed=2),
             lam=rand(dim, seed=3) - 1.0, h0=rand(batch, dim, seed=4))
    dy, dhl = rand(batch, steps, dim, seed=5), rand(batch, dim, seed=6)

    def f(x, r, i, lam, h0):
        y, hl = layers.gated_recurrence(x, r, i, lam, 8.0, h0)
        return (y * dy).sum() + (hl * dhl).sum()

    if not h0:
        a["h0"] = torch.zeros(batch, dim, dtype=torch.float64)
    y, _ = layers.gated_recurrence(a["x"], a["r"], a["i"], a["lam"], 8.0, a["h0"])
    g = layers.gated_recurrence_grad(a["x"], a["r"], a["i"], a["lam"], y, dy, 8.0, a["h0"], dhl)
    check(f, a, {"x": g["dx"], "r": g["dr"], "i": g["di"], "lam": g["dlam"], "h0": g["dh0"]})


def test_gated_recurrence_saturated_gates_stay_finite():
    """r -> -inf closes the gate: a = 1, the state stays, every gradient is
    finite; r large lets the state go."""
    x, i, y = rand(1, 3, 2), rand(1, 3, 2, seed=1), rand(1, 3, 2, seed=2)
    r = torch.full((1, 3, 2), -2000.0, dtype=torch.float64)
    lam = torch.tensor([-3.0, 0.5], dtype=torch.float64)
    h0 = rand(1, 2, seed=3)
    out, last = layers.gated_recurrence(x, r, i, lam, 8.0, h0)
    assert torch.equal(last, h0)
    g = layers.gated_recurrence_grad(x, r, i, lam, y, rand(1, 3, 2, seed=4), 8.0, h0)
    assert all(torch.isfinite(v).all() for v in g.values())
    assert g["dr"].abs().max() == 0


def test_gated_recurrence_pieces_equal_whole():
    x, r, i, lam = rand(2, 11, 3), rand(2, 11, 3, seed=1), rand(2, 11, 3, seed=2), rand(3, seed=3)
    y, h = layers.gated_recurrence(x, r, i, lam)
    y0, h0 = layers.gated_recurrence(x[:, :4], r[:, :4], i[:, :4], lam)
    y1, h1 = layers.gated_recurrence(x[:, 4:], r[:, 4:], i[:, 4:], lam, h0=h0)
    # torch's vectorised exp and log1p round a value differently by its place
    # in the vector: at most eight roundings of 2^-53 a step over 11 steps of
    # states below 8
    assert h.abs().max() < 8
    tol = 11 * 8 * 8 * 2.0 ** -53
    assert (torch.cat([y0, y1], 1) - y).abs().max() <= tol and (h1 - h).abs().max() <= tol


@pytest.mark.parametrize("tokens,dim,vocab", [(1, 1, 1), (4, 3, 7), (6, 5, 20)])
def test_linear_cross_entropy_gradient(tokens, dim, vocab):
    g = torch.Generator().manual_seed(tokens)
    targets = torch.randint(0, vocab, (tokens,), generator=g)
    if tokens > 1:
        targets[1] = -100
    dl = rand(tokens, seed=9)
    a = dict(hidden=rand(tokens, dim), weight=rand(vocab, dim, seed=1))

    def f(hidden, weight):
        return (layers.linear_cross_entropy(hidden, weight, targets)[0] * dl).sum()

    _, lse = layers.linear_cross_entropy(a["hidden"], a["weight"], targets)
    grad = layers.linear_cross_entropy_grad(a["hidden"], a["weight"], targets, lse, dl)
    check(f, a, {"hidden": grad["dhidden"], "weight": grad["dweight"]})


def test_linear_cross_entropy_against_library():
    h, w = rand(7, 4), rand(9, 4, seed=1)
    t = torch.tensor([0, 8, -100, 3, 3, -100, 5])
    loss, _ = layers.linear_cross_entropy(h, w, t)
    ref = torch.nn.functional.cross_entropy(h @ w.t(), t, reduction="none")
    assert torch.allclose(loss, ref, rtol=1e-13, atol=1e-13)

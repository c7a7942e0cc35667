"""Pins of the float64 definitions in oracle/attention.py: closed forms, torch's
own float64 functions, and central differences of the forwards.  CPU."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from oracle import attention as A  # noqa: E402


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def difference(f, x, step=1e-5):
    """Directional central difference of f at x, and the direction."""
    d = randn(*x.shape, seed=99)
    return (f(x + step * d) - f(x - step * d)) / (2 * step), d


@pytest.mark.parametrize("dim,rotary", [(8, 8), (7, 4), (6, 0), (5, 2)])
def test_head_norm_rotary(dim, rotary):
    x, w, pos = randn(4, 3, dim), randn(dim, seed=1), torch.tensor([0, 1, 17, -5])
    y = A.head_norm_rotary(x, pos, w, 100.0, 1e-6, rotary)
    n = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
    assert torch.equal(y[0][..., rotary:], n[0][..., rotary:]) or torch.allclose(y[0], n[0], atol=1e-15)
    assert torch.allclose(y.norm(dim=-1), n.norm(dim=-1))       # turns keep lengths
    for j in range(rotary // 2):
        z = torch.complex(n[..., j], n[..., j + rotary // 2])
        z = z * torch.exp(1j * pos[:, None] * 100.0 ** (-2 * j / rotary))
        assert torch.allclose(y[..., j], z.real) and torch.allclose(y[..., j + rotary // 2], z.imag)


def test_rotated_products_depend_on_the_distance():
    q, k = randn(1, 1, 16), randn(1, 1, 16, seed=1)
    def at(p, r):
        return (A.rotate(q, A.angles(torch.tensor([p]), 16, 1e4), 16) * A.rotate(k, A.angles(torch.tensor([r]), 16, 1e4), 16)).sum()
    assert math.isclose(at(1000, 990), at(20, 10), rel_tol=1e-9)


@pytest.mark.parametrize("weighted", [True, False])
def test_head_norm_rotary_gradient(weighted):
    x, pos, dy = randn(3, 2, 6), torch.tensor([0, 4, 9]), randn(3, 2, 6, seed=2)
    w = randn(6, seed=1) if weighted else None
    g = A.head_norm_rotary_grad(dy, x, pos, w, 50.0, 1e-3, 4)
    num, d = difference(lambda v: (A.head_norm_rotary(v, pos, w, 50.0, 1e-3, 4) * dy).sum(), x)
    assert math.isclose(num, (g["dx"] * d).sum(), rel_tol=1e-7)
    w = torch.ones(6, dtype=torch.float64) if w is None else w
    num, d = difference(lambda v: (A.head_norm_rotary(x, pos, v, 50.0, 1e-3, 4) * dy).sum(), w)
    assert math.isclose(num, (g["dweight"] * d).sum(), rel_tol=1e-7)


def attention_inputs(batch=2, steps=7, heads=3, key=4, value=5):
    return (randn(batch, steps, heads, key), randn(batch, steps, heads, key, seed=1),
            randn(batch, steps, heads, value, seed=2), -randn(heads, seed=3).abs(),
            randn(batch, heads, key, value, seed=4))


def test_linear_attention_is_the_masked_product():
    q, k, v, ld, h0 = attention_inputs()
    o, last = A.linear_attention(q, k, v, ld, 0.5, h0)
    t = torch.arange(7, dtype=torch.float64)
    mask = torch.tril(torch.exp(ld[:, None, None] * (t[:, None] - t)))
    p = torch.einsum("bihd,bjhd->bhij", q, k) * mask
    want = torch.einsum("bhij,bjhd->bihd", p, v)
    want += torch.exp(ld * (t[:, None] + 1))[None, :, :, None] * torch.einsum("bihk,bhkv->bihv", q, h0)
    assert torch.allclose(o, 0.5 * want)
    w = torch.exp(ld * (6 - t[:, None]))
    assert torch.allclose(last, torch.einsum("bjhk,bjhv,jh->bhkv", k, v, w) + torch.exp(7 * ld)[:, None, None] * h0)


def test_linear_attention_in_pieces_and_without_decay():
    q, k, v, ld, h0 = attention_inputs()
    o, last = A.linear_attention(q, k, v, ld, 1.0, h0)
    a, mid = A.linear_attention(q[:, :3], k[:, :3], v[:, :3], ld, 1.0, h0)
    b, end = A.linear_attention(q[:, 3:], k[:, 3:], v[:, 3:], ld, 1.0, mid)
    assert torch.allclose(torch.cat([a, b], 1), o) and torch.allclose(end, last)
    flat = A.linear_attention(q, k, v, torch.zeros(3))[1]
    assert torch.allclose(flat, torch.einsum("bjhk,bjhv->bhkv", k, v))


@pytest.mark.parametrize("which", ["dq", "dk", "dv", "dh0"])
def test_linear_attention_gradient(which):
    q, k, v, ld, h0 = attention_inputs()
    do, dlast = randn(*v.shape, seed=5), randn(*h0.shape, seed=6)
    g = A.linear_attention_grad(q, k, v, ld, do, 0.7, h0, dlast)
    ins = {"dq": q, "dk": k, "dv": v, "dh0": h0}

    def loss(x):
        a = {**ins, which: x}
        o, last = A.linear_attention(a["dq"], a["dk"], a["dv"], ld, 0.7, a["dh0"])
        return (o * do).sum() + (last * dlast).sum()

    num, d = difference(loss, ins[which])
    assert math.isclose(num, (g[which] * d).sum(), rel_tol=1e-7)


def test_packed_is_each_sequence_by_itself():
    q, k, v, ld, _ = attention_inputs(batch=1, steps=9)
    h0 = randn(4, 3, 4, 5, seed=8)
    cu = torch.tensor([1, 4, 4, 8, 8])
    o, last = A.packed(lambda a, b, c, h0: A.linear_attention(a, b, c, ld, 1.0, h0), (q[0], k[0], v[0]), cu, {"h0": h0})
    assert o[0].abs().max() == 0 and o[8].abs().max() == 0
    assert torch.equal(last[1], h0[1]) and torch.equal(last[3], h0[3])
    want, end = A.linear_attention(q[:, 4:8], k[:, 4:8], v[:, 4:8], ld, 1.0, h0[2:3])
    assert torch.equal(o[4:8], want[0]) and torch.equal(last[2], end[0])


def test_beam_select():
    logits, scores = randn(2, 3, 11), randn(2, 3, seed=1)
    scores[0, 1] = float("-inf")
    logits[1, 2] = float("-inf")
    logits[1, 0, 4] = float("-inf")
    best, tokens, beams = A.beam_select(logits, scores, 33)
    for b in range(2):
        p = scores[b][:, None] + torch.log_softmax(logits[b], -1)
        p = torch.where(p.isnan(), torch.full_like(p, float("-inf")), p)
        order = sorted(range(33), key=lambda i: (-p.flatten()[i].item(), i))
        assert (beams[b] * 11 + tokens[b]).tolist() == order
        live = best[b].isfinite()
        assert torch.allclose(best[b][live], p.flatten()[order][live]) and (best[b][~live] == float("-inf")).all()


def test_state_reorder():
    s = torch.arange(12).view(2, 3, 2)
    got = A.state_reorder(s, torch.tensor([[2, 0, 0], [1, 5, -1]]))
    assert got.tolist() == [[[4, 5], [0, 1], [0, 1]], [[8, 9], [8, 9], [10, 11]]]


def test_beam_select_orders_merged_values_by_their_logits():
    """Values that float64 cannot tell apart: by beam, then by logit, then by word."""
    logits = torch.tensor([[[1.0, 3.0, 2.0, 3.0], [9.0, 8.0, 7.0, 10.0]]])
    best, tokens, beams = A.beam_select(logits, torch.tensor([[-1e30, -1e30]]), 6)
    assert tokens[0].tolist() == [1, 3, 2, 0, 3, 0] and beams[0].tolist() == [0, 0, 0, 0, 1, 1]
    assert (best == torch.tensor(-1e30).double()).all()
    tokens = A.beam_select(logits, torch.tensor([[float("-inf")] * 2]), 6)[1]
    assert tokens[0].tolist() == [0, 1, 2, 3, 0, 1]


def test_terms_that_hold_a_float32():
    """A value as the sum of roundings to bfloat16, each of what those before left: one is
    off by 1.7e-3 in the root mean square, two by 2.7e-6, three by less than float32 is."""
    x = randn(1 << 16).float()
    left, off = x.clone(), []
    for _ in range(3):
        left = left - left.to(torch.bfloat16).float()      # exact in float32
        off.append((left.norm() / x.norm()).item())
    assert 1.6e-3 < off[0] < 1.8e-3 and 2e-6 < off[1] < 3.5e-6 and off[2] < 2 ** -24 / 3
    # a bound of 16 roundings of a float32 tells two terms from three
    assert off[1] > 2 * 16 * 2 ** -24 > 16 * 2 ** -24 > 100 * off[2]

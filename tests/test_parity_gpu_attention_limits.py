"""Linear attention, its norm and the beam search's operators at the edges of what
their entry points allow.  Needs an MI355X; marked ``gpu``."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from oracle import attention as A  # noqa: E402
from test_parity_gpu_attention import (D_TURN, IO, NINF, U32, attention_inputs, dev, half_step, mssm,  # noqa: E402,F401
                                       pair_size, randn, rms, within)   # (fixtures among them)

pytestmark = pytest.mark.gpu


def announce(*what):
    print("[attention limits]", *what, flush=True)


# ---- states advanced in place ----------------------------------------------------------

@pytest.mark.parametrize("shape", [(1, 3873, 20, 128, 128), (2, 700, 3, 40, 72), (3, 300, 1, 16, 24), (1, 2050, 2, 200, 130)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_states_in_place_over_several_segments(dev, mssm, shape, io):
    """The workgroup that writes the final state is not the one that reads the initial one:
    a state advanced in place is what a separate output holds, bit for bit."""
    announce("in place", shape, io)
    b, _, h, key, value = shape
    x = attention_inputs(dev, shape, io)
    h0 = randn(dev, b, h, key, value, seed=5, scale=3.0)
    want, end = mssm.linear_attention_fwd(**x, h0=h0)
    for _ in range(3):
        state = h0.clone()
        o, back = mssm.linear_attention_fwd(**x, h0=state, h_out=state)
        assert back is state and torch.equal(o, want) and torch.equal(state, end)


@pytest.mark.parametrize("longest", [None, 3959, 64])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_packed_states_in_place_over_several_segments(dev, mssm, io, longest):
    """The same with more workgroups than the device holds at once, with sequences of no
    step and of one among them."""
    announce("packed in place", io, longest)
    lengths = [1159, 684, 2298, 416, 0, 3959, 3723, 1, 1896, 2072, 2788]
    cu = torch.tensor([0] + lengths, device=dev).cumsum(0)
    total, n = sum(lengths), len(lengths)
    x = attention_inputs(dev, (1, total, 8, 128, 128), io)
    rows = (x["q"][0], x["k"][0], x["v"][0])
    h0 = randn(dev, n, 8, 128, 128, seed=5, scale=3.0)
    want, end = mssm.linear_attention_fwd(*rows, x["log_decay"], h0=h0, cu_seqlens=cu, max_seqlen=longest)
    assert torch.equal(end[4], h0[4])
    for _ in range(3):
        state = h0.clone()
        o, _ = mssm.linear_attention_fwd(*rows, x["log_decay"], h0=state, h_out=state, cu_seqlens=cu, max_seqlen=longest)
        assert torch.equal(o, want) and torch.equal(state, end)


def test_states_in_place_in_a_replayed_graph(dev, mssm):
    """Every replay continues from where the one before it ended."""
    announce("in place graph")
    x = attention_inputs(dev, (2, 700, 2, 64, 64), "bf16")
    h0 = randn(dev, 2, 2, 64, 64, seed=5)
    state = h0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mssm.linear_attention_fwd(**x, h0=state, h_out=state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = mssm.linear_attention_fwd(**x, h0=state, h_out=state)
    state.copy_(h0)
    want = h0
    for turn in range(4):
        graph.replay()
        wo, want = mssm.linear_attention_fwd(**x, h0=want)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(state, want), turn


# ---- beams whose values merge -----------------------------------------------------------

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("beams,vocab,count", [(1, 300, 5), (3, 5000, 16), (2, 12345, 64), (32, 4097, 64), (4, 9, 30)])
def test_beam_select_values_that_float64_merges(dev, mssm, io, beams, vocab, count):
    """Mask scores that swallow every logit, and logits that vanish beside lse: words of a
    beam still rank by their logits, and none of the best is left out on the way."""
    announce("merged values", io, beams, vocab, count)
    scores = torch.tensor([-1e30, torch.finfo(torch.float32).min, 3e38, 0.0, -1e15, -1e30, 0.0], device=dev)[:, None].repeat(1, beams)
    # 2^42 apart where float64 holds multiples of 1/8 .. 1 and lse is off by 1e-6 at most
    scores[4] -= torch.arange(beams, device=dev) * 2.0 ** 42
    scores[5, 1:] = NINF
    logits = randn(dev, len(scores), beams, vocab, seed=beams, dtype=IO[io], scale=3.0)
    logits[3] *= 2.0 ** -70
    logits[3, 1:] = NINF                                   # lse beside which the logits vanish, once
    logits[6] = logits[6] * 2.0 ** -80
    logits[6] = logits[6, :1]                              # and in beams that are alike
    logits[0, 0, vocab // 2:] = -4.0                       # equal logits among them
    best, tokens, origins = mssm.beam_select(logits, scores, count)
    want, wt, wb = A.beam_select(logits, scores, count)
    assert torch.equal(origins, wb) and torch.equal(tokens, wt)
    live = want.isfinite()
    assert torch.equal(best.isfinite(), live)
    err = (best.double() - want).abs()[live]
    # lse to 1e-5 (sums of up to 12345 exponentials), the score's rounding and the output's
    assert (err <= 1e-5 + 2 * want[live].abs() * U32).all()


def test_beam_select_of_the_most_entries(dev, mssm):
    """One entry more is refused: 2^23 - 1 entries of one beam and three words."""
    announce("most entries")
    batch = (1 << 23) - 1
    g = torch.Generator(device=dev).manual_seed(1)
    logits = torch.randn(batch, 1, 3, generator=g, device=dev)
    best, tokens, origins = mssm.beam_select(logits, torch.zeros(batch, 1, device=dev), 2)
    want, at = logits[:, 0].double().log_softmax(-1).sort(dim=-1, descending=True, stable=True)
    assert torch.equal(tokens, at[:, :2]) and not origins.any()
    # float32 sums of three exponentials and the output's rounding of values up to 20
    assert (best.double() - want[:, :2]).abs().max() <= 40 * U32
    with pytest.raises(mssm.MssmError, match="2\\^23"):
        mssm.beam_select(torch.empty(1 << 23, 1, 1, device=dev), torch.zeros(1 << 23, 1, device=dev))


# ---- how near the values are -----------------------------------------------------------

# every number of key blocks and of waves, whole vectors and not, one segment and several
NEAR_SHAPES = [(1, 900, 2, 128, 128), (2, 200, 2, 64, 40), (1, 430, 3, 72, 200), (1, 300, 2, 33, 57), (1, 200, 2, 96, 64),
               (1, 260, 1, 192, 256), (1, 170, 2, 256, 192), (1, 1500, 1, 120, 130)]


@pytest.mark.parametrize("shape", NEAR_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_is_off_by_its_storage_alone(dev, mssm, shape, io):
    """States and their gradients are float32 sums; what enters matrix products in bfloat16
    is split so that outputs and gradients are off by their own rounding and no more.

    In the root mean square of the relative error.  States: the three terms that a
    float32 is split into leave 2^-27, so what is left are float32 roundings with random
    signs: an exponential, its argument, a factor a chunk and a few hundred sums, 16 U32.
    (Two terms leave the square of a bfloat16's storage, 2.7e-6, as the next test shows.)
    Outputs: two terms leave 2^-18 at most.  A value c that is off by a of the exact w is
    stored within |round(c) - c| of itself, whose root mean square is that of w to a, and
    is off by a more: 2 a beside the storage of w."""
    announce("near", shape, io)
    b, _, h, key, value = shape
    x = attention_inputs(dev, shape, io)
    h0, dlast = randn(dev, b, h, key, value, seed=5, scale=3.0), randn(dev, b, h, key, value, seed=6)
    do = randn(dev, *x["v"].shape, seed=9, dtype=IO[io])
    scale = key ** -0.5
    o, last = mssm.linear_attention_fwd(**x, scale=scale, h0=h0)
    g = mssm.linear_attention_bwd(**x, do=do, scale=scale, h0=h0, dh_last=dlast)
    wo, wl = A.linear_attention(**x, scale=scale, h0=h0)
    wg = A.linear_attention_grad(**x, do=do, scale=scale, h0=h0, dh_last=dlast)
    off = (2.0 ** -18 if io == "bf16" else 0.0) + 16 * U32
    for what, got, want in [("o", o, wo)] + [(n, g[n], wg[n]) for n in ("dq", "dk", "dv")]:
        assert rms(got, want) <= rms(want.to(got.dtype), want) + 2 * off, what
    for what, got, want in (("h_last", last, wl), ("dh0", g["dh0"], wg["dh0"])):
        assert rms(got, want) <= 16 * U32, what


# ---- norms of very large and very small values -----------------------------------------

@pytest.mark.parametrize("scale,eps", [(2.0 ** 100, 1e-6), (2.0 ** 66, 1e-6), (2.0 ** 60, 0.0), (2.0 ** -44, 0.0), (2.0 ** -50, 0.0),
                                       (2.0 ** -80, 0.0), (2.0 ** -80, 2.0 ** -160), (2.0 ** -100, 0.0), (2.0 ** -100, 1e-6)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rotary", [(128, 128), (256, 64), (24, 8), (7, 4)])
def test_qk_norm_rotary_beyond_the_range_of_squares(dev, mssm, scale, eps, io, dim, rotary):
    """Heads whose sum of squares float32 cannot hold, beside ordinary ones, forward and
    backward; bounds as for ordinary ones, since a power of two costs nothing."""
    announce("norm range", scale, eps, io, dim, rotary)
    pos = torch.arange(9, device=dev)
    x = randn(dev, 9, 3, dim, seed=1)
    x[:, 0] *= scale
    x[4:, 2] *= scale
    x = x.to(IO[io])
    w = randn(dev, dim, seed=2, shift=1.0, scale=0.3)
    dy = randn(dev, 9, 3, dim, seed=3, dtype=IO[io])
    got = mssm.qk_norm_rotary_fwd(x, x.clone(), pos, w, None, eps=eps, rotary_dim=rotary)
    g = mssm.qk_norm_rotary_bwd(dy, dy.clone(), x, x.clone(), pos, w, None, eps=eps, rotary_dim=rotary)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    X = x.double()
    r = (X.square().mean(-1, keepdim=True) + eps).rsqrt()
    for y, n, wt in ((got[0], "q", w), (got[1], "k", None)):
        want = A.head_norm_rotary(x, pos, wt, 1e4, eps, rotary)
        bound = pair_size(A.head_norm_rotary(x, pos, wt, 1e4, eps, 0), rotary) * ((dim / 2 + 12) * U32 + D_TURN)
        within(y, want, bound + half_step(want, y) * 1.01, n)
        want = A.head_norm_rotary_grad(dy, x, pos, wt, 1e4, eps, rotary)
        dn = pair_size(dy.double(), rotary)
        e = dn if wt is None else dn * wt.double().abs()
        rel_n, rel_r = D_TURN + 4 * U32, (dim / 2 + 6) * U32
        c = r.square() * (e * X.abs()).mean(-1, keepdim=True)
        bound = r * (e * (rel_n + rel_r + 4 * U32) + X.abs() * c * (rel_n + 3 * rel_r + (dim + 10) * U32))
        within(g["d" + n], want["dx"], bound + half_step(want["dx"], g["d" + n]) * 1.01, "d" + n)
        size = (dn * X.abs() * r).flatten(0, -2).sum(0)
        within(g["d%s_weight" % n], want["dweight"], size * (rel_n + rel_r + 40 * U32) + 1e-30, n + " weight")


def test_beam_select_refuses_a_huge_count_without_allocating_for_it(dev, mssm):
    announce("huge count")
    logits, scores = randn(dev, 2, 3, 50), randn(dev, 2, 3)
    for count in (10 ** 13, 65, 151, 0, -1, -10 ** 13):
        with pytest.raises(mssm.MssmError, match="count"):
            mssm.beam_select(logits, scores, count)


@pytest.mark.parametrize("positions", [1 << 6, 1 << 12, 1 << 20])
@pytest.mark.parametrize("rotary", [2, 64, 256])
def test_qk_norm_rotary_turns_to_a_step_of_float32(dev, mssm, positions, rotary):
    """Heads of ones and zeros whose norm is exactly 1 show the cosines and sines
    themselves: the functions are good to a step (U32 from 1/2 on), the turn by what the
    fraction's rounding left adds half of one; angles are float64."""
    announce("turns", positions, rotary)
    g = torch.Generator().manual_seed(positions + rotary)
    pos = torch.randint(0, positions, (4000,), generator=g).to(dev)
    x = torch.zeros(4000, 1, rotary, device=dev)
    x[..., :rotary // 2] = 1.0
    y = mssm.qk_norm_rotary_fwd(x, x.clone(), pos, eps=0.5)[0]
    a = A.angles(pos, rotary, 1e4)
    want = torch.cat([a.cos(), a.sin()], -1)[:, None]
    within(y, want, torch.full_like(want, 1.5 * U32 + 2.0 ** -30), "turn")

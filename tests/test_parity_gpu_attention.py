"""GPU parity of the norm of queries and keys with their rotation, of linear
attention with a decay per head and of the beam search's operators against
their float64 definitions.  Needs an MI355X; marked ``gpu``.

Every tolerance is a bound per element that follows from the roundings: a
float32 operation is off by at most U32 = 2^-24 of its result, a hardware
exponential, root or reciprocal by 2 U32, a stored bfloat16 by 2^-8 of its value
(half a step), and a float32 sum of n terms, in whatever order, by n U32 times
the sum of their magnitudes."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from oracle import attention as A  # noqa: E402

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
NINF = float("-inf")


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
    print("[attention]", *what, flush=True)


def randn(dev, *shape, seed=0, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).to(dev)


def half_step(t, like):
    """Half a step of the dtype of `like` at the values t."""
    return t.abs() * (torch.finfo(like.dtype).eps / 2) + torch.finfo(like.dtype).tiny


def within(got, want, bound, what):
    assert got.shape == want.shape, what
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g where %.3g is allowed" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(bound.expand_as(err)[bad].max()))


# ---- norm with rotation ------------------------------------------------------------

# (tokens, q heads, k heads, dim, rotary): vectors and single elements, every number of
# lanes a head, one and two slots a lane, several tokens a workgroup
NORM_SHAPES = [(1, 1, 1, 1, 0), (3, 2, 1, 2, 2), (5, 3, 2, 7, 4), (2, 1, 4, 16, 16), (9, 4, 4, 64, 64), (7, 20, 5, 128, 128),
               (33, 3, 3, 128, 64), (6, 2, 2, 96, 32), (4, 5, 1, 80, 40), (5, 2, 2, 81, 80), (3, 2, 3, 200, 50),
               (4, 2, 2, 256, 256), (11, 1, 2, 255, 254), (4097, 3, 1, 32, 32), (5000, 2, 2, 24, 16), (4, 0, 3, 64, 64),
               (4, 3, 0, 64, 64)]


def norm_inputs(dev, shape, io, seed=0):
    tokens, qh, kh, dim, _ = shape
    g = torch.Generator().manual_seed(seed + 5)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g).to(dev)
    pos[::3] = torch.arange(pos[::3].numel(), device=dev)
    return (randn(dev, tokens, qh, dim, seed=seed, dtype=IO[io], scale=2.0), randn(dev, tokens, kh, dim, seed=seed + 1, dtype=IO[io], scale=0.1),
            pos, randn(dev, dim, seed=seed + 2, shift=1.0, scale=0.3), randn(dev, dim, seed=seed + 3, shift=1.0, scale=0.3))


def pair_size(n, rotary):
    """|value| + |the value it is turned with|."""
    half = rotary // 2
    a = n.abs()
    s = a[..., :half] + a[..., half:rotary]
    return torch.cat([s, s, a[..., rotary:]], -1)


# A sine or cosine: the fraction of a turn is stored in float32 (half of it at most: 2^-26
# off), which 2 pi turns into an angle; the function itself is good to 4 U32; the float64
# angle of a position below 2^20 is good to 2^20 * 2^-50 / (2 pi) turns.
D_TURN = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32) + 4 * U32


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_qk_norm_rotary_forward(dev, mssm, shape, io):
    announce("norm fwd", shape, io)
    q, k, pos, wq, wk = norm_inputs(dev, shape, io)
    dim, rotary = shape[3:]
    for weighted in (True, False):
        got = mssm.qk_norm_rotary_fwd(q, k, pos, wq if weighted else None, wk if weighted else None, rotary_dim=rotary)
        for g, x, w, what in zip(got, (q, k), (wq, wk), "qk"):
            w = w if weighted else None
            want = A.head_norm_rotary(x, pos, w, 1e4, 1e-6, rotary)
            n = A.head_norm_rotary(x, pos, w, 1e4, 1e-6, 0)
            # 1 / sqrt of a sum of dim squares, two products, the turn's two
            bound = pair_size(n, rotary) * ((dim / 2 + 12) * U32 + D_TURN)
            within(g, want, bound + half_step(want, g) * 1.01, what)


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_qk_norm_rotary_backward(dev, mssm, shape, io):
    announce("norm bwd", shape, io)
    q, k, pos, wq, wk = norm_inputs(dev, shape, io)
    dim, rotary = shape[3:]
    dq, dk = randn(dev, *q.shape, seed=7, dtype=IO[io]), randn(dev, *k.shape, seed=8, dtype=IO[io])
    for weighted in (True, False):
        got = mssm.qk_norm_rotary_bwd(dq, dk, q, k, pos, wq if weighted else None, wk if weighted else None, rotary_dim=rotary)
        for n, x, dy, w in (("q", q, dq, wq), ("k", k, dk, wk)):
            w = w if weighted else None
            want = A.head_norm_rotary_grad(dy, x, pos, w, 1e4, 1e-6, rotary)
            if x.numel() == 0:
                assert got["d%s_weight" % n].abs().max() == 0
                continue
            X = x.double()
            r = (X.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            dn = pair_size(dy.double(), rotary)          # bounds |dn|
            e = dn if w is None else dn * w.double().abs()
            rel_n, rel_r = D_TURN + 4 * U32, (dim / 2 + 6) * U32
            c = r.square() * (e * X.abs()).mean(-1, keepdim=True)
            bound = r * (e * (rel_n + rel_r + 4 * U32) + X.abs() * c * (rel_n + 3 * rel_r + (dim + 10) * U32))
            within(got["d" + n], want["dx"], bound + half_step(want["dx"], got["d" + n]) * 1.01, "d" + n)
            size = (dn * X.abs() * r).flatten(0, -2).sum(0)
            rows = x.shape[0] * x.shape[1]
            within(got["d%s_weight" % n], want["dweight"], size * (rel_n + rel_r + (rows + 10) * U32) + 1e-30, n + " weight")


def test_qk_norm_rotary_special_rows(dev, mssm):
    """Rows of zeros, of infinity and NaN stay by themselves; negative positions; higher rank."""
    announce("norm special")
    x = randn(dev, 2, 3, 2, 32, seed=1)
    x[0, 0, 0] = 0.0
    x[0, 1, 1, 5] = float("nan")
    pos = torch.tensor([[-3, 0, 5], [1 << 40, -(1 << 31), 7]], device=dev)
    q, k = mssm.qk_norm_rotary_fwd(x, x.clone(), pos)
    assert torch.equal(q.isnan(), k.isnan()) and q.isnan().sum() == 32 and q[0, 1, 1].isnan().all()
    assert (q[0, 0, 0] == 0).all()
    want = A.head_norm_rotary(x[0, 2], pos[0, 2].expand(1)[0], None)
    within(q[0, 2], want, torch.full_like(want, 1e-5), "position 5")
    want = A.head_norm_rotary(x[0], pos[0])[0]
    within(q[0, 0], want, torch.full_like(want, 1e-5), "position -3")


def test_qk_norm_rotary_unaligned(dev, mssm):
    """Tensors that start at any element, next to memory that is not touched."""
    announce("norm unaligned")
    for io in IO.values():
        for off in (1, 3):
            n = 5 * 2 * 64
            buf = randn(dev, n + 8, seed=off, dtype=io)
            x = buf[off:off + n].view(5, 2, 64)
            pos = torch.arange(5, device=dev)
            a = mssm.qk_norm_rotary_fwd(x, x, pos)[0]
            b = mssm.qk_norm_rotary_fwd(x.clone(), x.clone(), pos)[0]
            assert torch.equal(a, b)


def test_qk_norm_rotary_gradient_is_the_difference_quotient(dev, mssm):
    announce("norm difference")
    q, k, pos, wq, wk = norm_inputs(dev, (6, 2, 3, 20, 12), "f32")
    dq, dk = randn(dev, *q.shape, seed=3), randn(dev, *k.shape, seed=4)
    g = mssm.qk_norm_rotary_bwd(dq, dk, q, k, pos, wq, wk, rotary_dim=12)
    for name, at in (("dq", 0), ("dk", 1), ("dq_weight", 2), ("dk_weight", 3)):
        ins = [q.double(), k.double(), wq.double(), wk.double()]
        d = randn(dev, *ins[at].shape, seed=9).double()

        def loss(step):
            a = list(ins)
            a[at] = a[at] + step * d
            return ((A.head_norm_rotary(a[0], pos, a[2], rotary=12) * dq.double()).sum()
                    + (A.head_norm_rotary(a[1], pos, a[3], rotary=12) * dk.double()).sum()).item()

        num = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # float32 gradients: (values + roundings) U32 of the terms' sizes
        terms = (g[name].double() * d).abs().sum().item()
        assert abs(num - (g[name].double() * d).sum().item()) <= 1e-5 * terms, name


# ---- linear attention ----------------------------------------------------------------

# (batch, steps, heads, key, value): one step to several chunks, ragged ones, every shape
# of a workgroup, widths that are no multiple of anything, several slices of values
ATTENTION_SHAPES = [(1, 1, 1, 1, 1), (2, 1, 3, 16, 8), (1, 31, 2, 5, 3), (2, 33, 2, 64, 64), (1, 64, 3, 40, 33),
                    (3, 65, 1, 64, 128), (2, 129, 2, 128, 128), (1, 200, 2, 72, 100), (1, 130, 1, 256, 64),
                    (1, 70, 2, 128, 200), (1, 150, 1, 200, 256), (2, 97, 1, 129, 65), (1, 100, 2, 63, 130)]
# several segments of a sequence
LONG_SHAPES = [(1, 700, 1, 64, 64), (1, 1025, 2, 16, 24), (2, 519, 1, 130, 20)]


def attention_inputs(dev, shape, io, seed=0):
    b, n, h, key, value = shape
    ld = -torch.rand(h, generator=torch.Generator().manual_seed(seed)).mul(3).exp().sub(1).mul(0.02)
    ld[-1] = -0.003
    return {"q": randn(dev, b, n, h, key, seed=seed + 1, dtype=IO[io]), "k": randn(dev, b, n, h, key, seed=seed + 2, dtype=IO[io]),
            "v": randn(dev, b, n, h, value, seed=seed + 3, dtype=IO[io]), "log_decay": ld.to(dev)}


def attention_sizes(x, scale, h0):
    """The operator on magnitudes: what the terms of every output add up to."""
    return A.linear_attention(x["q"].abs(), x["k"].abs(), x["v"].abs(), x["log_decay"], abs(scale), None if h0 is None else h0.abs())


def output_factor(io, steps, key):
    """Relative error of a sum of terms on its way: products and sums in float32 (those of
    a chunk, of the width, and of the chunks in turn), decays of up to `steps` steps
    (an exponent of at most 88 off by U32, an exponential, one factor a chunk); in
    bfloat16 also the rounding of either the decayed product or the state, and the two
    roundings of the state's terms."""
    f32 = (2 * key + 3 * 64 + 4 * (steps // 32 + 2) + 100) * U32
    return f32 + (U16 * (1 + U16) + U16 * U16 if io == "bf16" else 0.0)


def state_factor(io, steps):
    return (3 * 64 + 4 * (steps // 32 + 2) + 100) * U32 + (U16 * U16 if io == "bf16" else 0.0)


def rms(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# Two roundings to bfloat16 of relative size 2^-8 at most, 2^-8 / sqrt(3) in the root mean
# square where values are spread evenly over a step, less over all steps: one on the way,
# one in the output.  Terms whose sum they enter are as large as that sum is in the root
# mean square, since their signs are independent.
RMS = {"f32": 4e-6, "bf16": U16 * math.sqrt(2 / 3)}


def check_attention(mssm, x, io, scale, h0, dlast, seed=0):
    steps, key, value = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    o, last = mssm.linear_attention_fwd(**x, scale=scale, h0=h0)
    want, end = A.linear_attention(**x, scale=scale, h0=h0)
    size, states = attention_sizes(x, scale, h0)
    within(o, want, size * output_factor(io, steps, key) + half_step(want, o) * 1.01, "o")
    within(last, end, states * state_factor(io, steps), "h_last")
    if o.numel() > 2000:
        assert rms(o, want) <= RMS[io] * 1.1
    do = randn(o.device, *o.shape, seed=seed + 9, dtype=o.dtype)
    g = mssm.linear_attention_bwd(**x, do=do, scale=scale, h0=h0, dh_last=dlast)
    w = A.linear_attention_grad(**x, do=do, scale=scale, h0=h0, dh_last=dlast)
    ax = {n: t.abs() for n, t in x.items() if n != "log_decay"}
    s = A.linear_attention_grad(**ax, log_decay=x["log_decay"], do=do.abs(), scale=abs(scale), h0=None if h0 is None else h0.abs(),
                                dh_last=None if dlast is None else dlast.abs())
    for n, width in (("dq", value), ("dk", value), ("dv", key)):
        within(g[n], w[n], s[n] * output_factor(io, steps, width) + half_step(w[n], g[n]) * 1.01, n)
        if w[n].numel() > 2000:
            assert rms(g[n], w[n]) <= RMS[io] * 1.1, n
    within(g["dh0"], w["dh0"], s["dh0"] * state_factor(io, steps), "dh0")


@pytest.mark.parametrize("shape", ATTENTION_SHAPES + LONG_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("states", [False, True])
def test_linear_attention(dev, mssm, shape, io, states):
    announce("attention", shape, io, states)
    b, _, h, key, value = shape
    x = attention_inputs(dev, shape, io)
    h0 = randn(dev, b, h, key, value, seed=5, scale=3.0) if states else None
    dlast = randn(dev, b, h, key, value, seed=6) if states else None
    check_attention(mssm, x, io, key ** -0.5, h0, dlast)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, -1e-6, -5.0, -60.0, NINF])
def test_linear_attention_decays(dev, mssm, io, decay):
    """No decay at all, slow and fast ones, and one that forgets every step at once."""
    announce("attention decay", io, decay)
    shape = (1, 200, 2, 24, 40)
    x = attention_inputs(dev, shape, io)
    x["log_decay"] = torch.tensor([decay, -0.01], device=dev)
    h0, dlast = (randn(dev, 1, 2, 24, 40, seed=s) for s in (5, 6))
    check_attention(mssm, x, io, 1.0, h0, dlast)


CU = {"ragged": ([0, 0, 1, 38, 38, 300, 428], 428), "covered in part": ([3, 70, 70, 190], 200), "one": ([0, 77], 77),
      "none in it": ([4, 4, 4], 9)}


@pytest.mark.parametrize("which", CU)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("longest", [None, 1, 1000])
def test_linear_attention_packed(dev, mssm, which, io, longest):
    """Sequences of different lengths, empty ones, rows of no sequence, and any estimate
    of the longest one."""
    announce("packed", which, io, longest)
    ends, total = CU[which]
    cu, n = torch.tensor(ends, device=dev), len(ends) - 1
    x = attention_inputs(dev, (1, total, 2, 48, 20), io)
    rows = (x["q"][0], x["k"][0], x["v"][0])
    h0, dlast = (randn(dev, n, 2, 48, 20, seed=s) for s in (5, 6))
    o, last = mssm.linear_attention_fwd(*rows, x["log_decay"], 0.2, h0=h0, cu_seqlens=cu, max_seqlen=longest)
    f = lambda q, k, v, h0: A.linear_attention(q, k, v, x["log_decay"], 0.2, h0)  # noqa: E731
    want, end = A.packed(f, rows, cu, {"h0": h0})
    size, states = A.packed(f, tuple(t.abs() for t in rows), cu, {"h0": h0.abs()})
    within(o, want, size * output_factor(io, total, 48) + half_step(want, o) * 1.01, "o")
    within(last, end, states * state_factor(io, total), "h_last")
    out = torch.full_like(o, 7.0)
    mssm.linear_attention_fwd(*rows, x["log_decay"], 0.2, h0=h0, cu_seqlens=cu, max_seqlen=longest, out=out)
    assert torch.equal(out, o) and (o[ends[-1]:] == 0).all() and (o[:ends[0]] == 0).all()
    do = randn(dev, *o.shape, seed=9, dtype=o.dtype)
    g = mssm.linear_attention_bwd(*rows, x["log_decay"], do, 0.2, h0=h0, dh_last=dlast, cu_seqlens=cu, max_seqlen=longest)

    def grad(q, k, v, do, h0, dh_last):
        r = A.linear_attention_grad(q, k, v, x["log_decay"], do, 0.2, h0, dh_last)
        return r["dq"], r["dk"], r["dv"], r["dh0"]

    want = A.packed(grad, (*rows, do), cu, {"h0": h0, "dh_last": dlast})
    size = A.packed(grad, tuple(t.abs() for t in (*rows, do)), cu, {"h0": h0.abs(), "dh_last": dlast.abs()})
    for n, w, s, width in zip(("dq", "dk", "dv"), want, size, (20, 20, 48)):
        within(g[n], w, s * output_factor(io, total, width) + half_step(w, g[n]) * 1.01, n)
    within(g["dh0"], want[3], size[3] * state_factor(io, total), "dh0")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_offsets_outside_the_rows(dev, mssm, io):
    """Offsets that fall or lead outside are held to the rows: nothing else is read or
    written, and the sequences that are in order come out right."""
    announce("bad offsets", io)
    x = attention_inputs(dev, (1, 90, 1, 16, 16), io)
    rows = (x["q"][0], x["k"][0], x["v"][0])
    guard = torch.full((90 + 64, 1, 16), 7.0, dtype=IO[io], device=dev)
    out = guard[32:122]
    cu = torch.tensor([-5, 40, 20, 60, 1 << 40], device=dev)
    o, last = mssm.linear_attention_fwd(*rows, x["log_decay"], cu_seqlens=cu, out=out)
    assert (guard[:32] == 7).all() and (guard[122:] == 7).all()
    want, end = mssm.linear_attention_fwd(*(t[None, :40].contiguous() for t in rows), x["log_decay"])
    assert torch.equal(last[0], end[0]) and torch.equal(last[1], torch.zeros_like(last[1]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_update_is_one_step(dev, mssm, io):
    announce("update", io)
    for b, h, key, value in [(1, 1, 1, 1), (2, 3, 16, 8), (3, 2, 128, 128), (40, 8, 64, 64), (2, 2, 33, 30), (70, 4, 20, 256),
                             (2, 3, 256, 255)]:
        x = attention_inputs(dev, (b, 1, h, key, value), io)
        for ld in (x["log_decay"], torch.full_like(x["log_decay"], NINF)):
            x["log_decay"] = ld
            h0 = randn(dev, b, h, key, value, seed=5)
            want, end = A.linear_attention(**x, scale=0.3, h0=h0)
            size, states = attention_sizes(x, 0.3, h0)
            state = h0.clone()
            o = mssm.linear_attention_update(state, x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["log_decay"], 0.3)
            within(o, want[:, 0], size[:, 0] * (key + 10) * U32 + half_step(want[:, 0], o) * 1.01, "o")
            within(state, end, states * 8 * U32, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_in_pieces_and_in_place(dev, mssm, io):
    """A sequence in pieces, states passed on in place, then steps of one token."""
    announce("pieces", io)
    shape = (2, 150, 2, 32, 48)
    x = attention_inputs(dev, shape, io)
    want, end = A.linear_attention(**x)
    size, states = attention_sizes(x, 1.0, None)
    state = torch.zeros(2, 2, 32, 48, device=dev)
    parts = []
    for lo, hi in ((0, 64), (64, 65), (65, 140)):
        part = {n: t[:, lo:hi].contiguous() if n != "log_decay" else t for n, t in x.items()}
        o, back = mssm.linear_attention_fwd(**part, h0=state, h_out=state)
        assert back is state
        parts.append(o)
    for t in range(140, 150):
        parts.append(mssm.linear_attention_update(state, *(x[n][:, t].contiguous() for n in "qkv"), x["log_decay"])[:, None])
    o = torch.cat(parts, 1)
    within(o, want, size * output_factor(io, 150, 32) + half_step(want, o) * 1.01, "o")
    within(state, end, states * state_factor(io, 150), "state")
    assert mssm.linear_attention_fwd(**x, return_last_state=False)[1] is None


def test_linear_attention_empty(dev, mssm):
    announce("empty")
    q, v = torch.zeros(2, 0, 3, 8, device=dev), torch.zeros(2, 0, 3, 4, device=dev)
    ld, h0 = torch.zeros(3, device=dev), randn(dev, 2, 3, 8, 4)
    o, last = mssm.linear_attention_fwd(q, q, v, ld, h0=h0)
    assert o.shape == v.shape and torch.equal(last, h0)
    g = mssm.linear_attention_bwd(q, q, v, ld, v, dh_last=h0)
    assert torch.equal(g["dh0"], h0) and g["dq"].shape == q.shape
    assert mssm.linear_attention_fwd(q, q, v, ld)[1].abs().max() == 0
    rows = torch.ones(5, 3, 8, device=dev)
    o, last = mssm.linear_attention_fwd(rows, rows, rows, ld, cu_seqlens=torch.zeros(1, dtype=torch.int64, device=dev))
    assert (o == 0).all() and last.shape == (0, 3, 8, 8)
    g = mssm.linear_attention_bwd(rows, rows, rows, ld, rows, cu_seqlens=torch.zeros(1, dtype=torch.int64, device=dev))
    assert (g["dq"] == 0).all() and (g["dk"] == 0).all() and (g["dv"] == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), NINF, float("nan")])
def test_linear_attention_keeps_what_is_not_finite_behind(dev, mssm, io, bad):
    """An infinite or NaN value reaches its own column from its own step on, a query its
    own outputs, a key what follows: no output before them, no other sequence or head."""
    announce("not finite", io, bad)
    shape = (2, 150, 2, 40, 70)
    clean = attention_inputs(dev, shape, io)
    o, last = mssm.linear_attention_fwd(**clean)
    at = 37
    for name, col in (("v", 5), ("q", 3), ("k", 2), ("all", 0)):
        x = {n: t.clone() for n, t in clean.items()}
        for n in ("q", "k", "v") if name == "all" else (name,):
            x[n][0, at, 1, col] = bad
        got, end = mssm.linear_attention_fwd(**x)
        keep = torch.ones_like(o, dtype=torch.bool)
        if name == "v":
            keep[0, at:, 1, col] = False
        elif name == "q":
            keep[0, at, 1] = False
        else:
            keep[0, at:, 1] = False
        # a chunk walked step by step rounds its sums otherwise
        size = attention_sizes(clean, 1.0, None)[0]
        bound = 2 * size * output_factor(io, 150, 40) + 2 * half_step(o.double(), o)
        within(torch.where(keep, got, o), o.double(), bound, name)
        assert not got[~keep].isfinite().any()
        assert end[1].isfinite().all() and end[0, 0].isfinite().all()
    do = randn(dev, *o.shape, seed=9, dtype=o.dtype)
    g = mssm.linear_attention_bwd(**clean, do=do)
    d = do.clone()
    d[0, at, 1, 4] = bad
    h = mssm.linear_attention_bwd(**clean, do=d)
    s = A.linear_attention_grad(**{n: t.abs() for n, t in clean.items() if n != "log_decay"}, log_decay=clean["log_decay"], do=do.abs())
    keep = {n: torch.ones_like(t, dtype=torch.bool) for n, t in g.items()}
    keep["dq"][0, at, 1] = False
    keep["dk"][0, :at + 1, 1] = False
    keep["dv"][0, :at + 1, 1, 4] = False
    for n in ("dq", "dk", "dv"):
        bound = 2 * s[n] * output_factor(io, 150, 70) + 2 * half_step(g[n].double(), g[n])
        within(torch.where(keep[n], h[n], g[n]), g[n].double(), bound, n)
        assert not h[n][~keep[n]].isfinite().any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_unaligned(dev, mssm, io):
    """Rows that start at any element, outputs next to memory that is not touched."""
    announce("unaligned", io)
    for off in (1, 3):
        shape = (1, 70, 2, 24, 24)
        n = 70 * 2 * 24
        bufs = {name: randn(dev, n + 8, seed=i, dtype=IO[io]) for i, name in enumerate("qkv")}
        x = {name: b[off:off + n].view(1, 70, 2, 24) for name, b in bufs.items()}
        x["log_decay"] = torch.tensor([-0.1, -0.01], device=dev)
        guard = torch.full((n + 8,), 7.0, dtype=IO[io], device=dev)
        o = mssm.linear_attention_fwd(**x, out=guard[off:off + n].view(1, 70, 2, 24))[0]
        assert (guard[:off] == 7).all() and (guard[off + n:] == 7).all(), shape
        assert torch.equal(o, mssm.linear_attention_fwd(**{a: t.clone() for a, t in x.items()})[0])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_repeats_bit_for_bit(dev, mssm, io):
    announce("repeat", io)
    x = attention_inputs(dev, (2, 900, 2, 64, 96), io)
    do = randn(dev, *x["v"].shape, seed=9, dtype=IO[io])
    first = (*mssm.linear_attention_fwd(**x), *mssm.linear_attention_bwd(**x, do=do).values())
    for _ in range(3):
        again = (*mssm.linear_attention_fwd(**x), *mssm.linear_attention_bwd(**x, do=do).values())
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("which", ["dq", "dk", "dv", "dh0"])
def test_linear_attention_gradient_is_the_difference_quotient(dev, mssm, which):
    announce("difference", which)
    x = attention_inputs(dev, (2, 45, 2, 6, 7), "f32")
    h0, dlast, do = randn(dev, 2, 2, 6, 7, seed=5), randn(dev, 2, 2, 6, 7, seed=6), randn(dev, 2, 45, 2, 7, seed=7)
    g = mssm.linear_attention_bwd(**x, do=do, scale=0.5, h0=h0, dh_last=dlast)[which].double()
    ins = {"dq": x["q"], "dk": x["k"], "dv": x["v"], "dh0": h0}
    d = randn(dev, *ins[which].shape, seed=8).double()

    def loss(step):
        a = {n: t.double() for n, t in ins.items()}
        a[which] = a[which] + step * d
        o, last = A.linear_attention(a["dq"], a["dk"], a["dv"], x["log_decay"], 0.5, a["dh0"])
        return ((o * do.double()).sum() + (last * dlast.double()).sum()).item()

    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(num - (g * d).sum().item()) <= 1e-5 * (g * d).abs().sum().item()


# ---- beams -----------------------------------------------------------------------------

# (batch, beams, vocab, count): several pieces of a vocabulary, fewer words than a wave has
# lanes, every candidate asked for, the limits
BEAM_SHAPES = [(1, 1, 1, 1), (2, 1, 5, 5), (3, 4, 7, 20), (1, 2, 63, 3), (2, 3, 64, 64), (1, 4, 1000, 8), (2, 5, 4095, 10),
               (3, 2, 4097, 4), (1, 32, 9001, 64), (4, 8, 50021, 16), (1, 3, 131101, 6), (2, 16, 300, 32)]


def beam_inputs(dev, shape, io, seed=0):
    batch, beams, vocab, _ = shape
    logits = randn(dev, batch, beams, vocab, seed=seed, dtype=IO[io], scale=3.0)
    return logits, randn(dev, batch, beams, seed=seed + 1, shift=-9.0)


def check_beams(mssm, logits, scores, count):
    """Values that two orders of the same float64 comparison can tell apart: those of
    different beams differ by the error of lse, vocab U32 at most."""
    best, tokens, beams = mssm.beam_select(logits, scores, count)
    want, wt, wb = A.beam_select(logits, scores, count)
    vocab = logits.shape[-1]
    assert torch.equal(beams, wb) and torch.equal(tokens, wt)
    live = want.isfinite()
    assert torch.equal(best.isfinite(), live) and (best[~live] == NINF).all()
    err = (best.double() - want).abs()[live]
    # lse: an exponential and its argument (off by U32 of at most 100), a sum of vocab terms
    bound = (100 + 10 + math.sqrt(vocab)) * U32 + half_step(want[live], best) * 1.01
    assert (err <= bound).all(), err.max()


@pytest.mark.parametrize("shape", BEAM_SHAPES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_beam_select(dev, mssm, shape, io):
    announce("beams", shape, io)
    logits, scores = beam_inputs(dev, shape, io)
    check_beams(mssm, logits, scores, shape[3])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_beam_select_ties_and_masks(dev, mssm, io):
    """Equal logits, equal beams, forbidden words, beams without a value."""
    announce("ties", io)
    for vocab, count in ((9, 12), (5000, 40), (12345, 64)):
        logits, scores = beam_inputs(dev, (6, 3, vocab, count), io)
        logits[0] = 0.5                                        # all words alike
        scores[0] = -1.0
        logits[1] = logits[1, :1]                              # all beams alike
        scores[1] = -2.0
        scores[2, 1:] = NINF                                   # the first step of a search
        logits[3, :, 2:] = NINF                                # few words allowed
        logits[4, 0] = NINF                                    # a beam without any
        scores[4, 2] = NINF
        logits[5] = (logits[5].float() * 0.5).round() * 2      # many equal ones
        check_beams(mssm, logits, scores, count)
        best = mssm.beam_select(logits, torch.full_like(scores, NINF), count)
        assert (best[0] == NINF).all() and torch.equal(best[1][0] + best[2][0] * vocab, torch.arange(count, device=dev))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_beam_select_not_finite(dev, mssm, io):
    """NaN, +infinity and the type's lowest value stay in their beam."""
    announce("beams not finite", io)
    logits, scores = beam_inputs(dev, (4, 3, 6000, 8), io)
    logits[0, 0, 17] = float("nan")
    logits[1, 1, 5000] = float("inf")
    scores[2, 0], scores[2, 2] = float("nan"), float("inf")
    logits[3, :, 100:] = torch.finfo(IO[io]).min
    check_beams(mssm, logits, scores, 8)


def test_beam_select_unaligned_and_empty(dev, mssm):
    announce("beams unaligned")
    for io in IO.values():
        buf = randn(dev, 2 * 3 * 501 + 8, seed=1, dtype=io)
        for off in (1, 3):
            logits = buf[off:off + 2 * 3 * 501].view(2, 3, 501)
            check_beams(mssm, logits, randn(dev, 2, 3), 5)
        best, tokens, beams = mssm.beam_select(torch.zeros(0, 3, 10, dtype=io, device=dev), torch.zeros(0, 3, device=dev))
        assert best.shape == tokens.shape == beams.shape == (0, 3)
    with pytest.raises(mssm.MssmError):
        mssm.beam_select(logits, torch.zeros(2, 3, device=dev), 0)
    with pytest.raises(mssm.MssmError):
        mssm.beam_select(logits, torch.zeros(2, 3, device=dev), 65)


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 13, 16, 32])
def test_state_reorder(dev, mssm, beams):
    """Permutations, copies of one beam, beams that stay, and origins outside; every size of
    a moved piece; memory around the states is not touched."""
    announce("reorder", beams)
    g = torch.Generator().manual_seed(beams)
    for batch in (1, 3):
        states = [randn(dev, batch, beams, 3, 40, 4), randn(dev, batch, beams, 7, dtype=torch.bfloat16),
                  torch.randint(0, 1 << 40, (batch, beams, 5), generator=g).to(dev),
                  torch.randint(0, 200, (batch, beams, 11), generator=g).to(torch.uint8).to(dev),
                  torch.zeros(batch, beams, 0, device=dev), randn(dev, batch, beams)]
        guard = torch.full((batch * beams * 9 + 7,), 7.0, device=dev)
        part = guard[3:3 + batch * beams * 9].view(batch, beams, 9)
        part.copy_(randn(dev, batch, beams, 9, seed=4))
        states.append(part)
        for origins in (torch.stack([torch.randperm(beams, generator=g) for _ in range(batch)]),
                        torch.randint(0, beams, (batch, beams), generator=g), torch.zeros(batch, beams, dtype=torch.int64),
                        torch.arange(beams).repeat(batch, 1), torch.randint(-3, beams + 3, (batch, beams), generator=g)):
            origins = origins.to(dev)
            want = [A.state_reorder(s.clone(), origins) for s in states]
            assert mssm.state_reorder(states, origins) is states
            assert all(torch.equal(a, b) for a, b in zip(states, want))
        assert (guard[:3] == 7).all() and (guard[-4:] == 7).all()


def test_state_reorder_many_states(dev, mssm):
    """More states than one launch holds; one tensor by itself; none."""
    announce("reorder many")
    states = [randn(dev, 2, 3, 10 + i, seed=i) for i in range(75)]
    origins = torch.tensor([[1, 2, 0], [2, 2, 2]], device=dev)
    want = [A.state_reorder(s.clone(), origins) for s in states]
    mssm.state_reorder(states, origins)
    assert all(torch.equal(a, b) for a, b in zip(states, want))
    one = randn(dev, 2, 3, 4)
    want = A.state_reorder(one.clone(), origins)
    assert mssm.state_reorder(one, origins) is one and torch.equal(one, want)
    assert mssm.state_reorder([], origins) == []
    with pytest.raises(ValueError, match="batch, beams"):
        mssm.state_reorder([one[:1]], origins)
    with pytest.raises(mssm.MssmError, match="overlaps"):
        mssm.state_reorder([one, one], origins)


# ---- together ----------------------------------------------------------------------------

def layer(mssm, t):
    """A layer on a prompt, its backward, and a step of beam search on its states."""
    q, k = mssm.qk_norm_rotary_fwd(t["q"], t["k"], t["pos"], t["wq"], t["wk"])
    o, state = mssm.linear_attention_fwd(q, k, t["v"], t["ld"], 0.1)
    g = mssm.linear_attention_bwd(q, k, t["v"], t["ld"], t["do"], 0.1)
    n = mssm.qk_norm_rotary_bwd(g["dq"], g["dk"], t["q"], t["k"], t["pos"], t["wq"], t["wk"])
    step = mssm.linear_attention_update(state, q[:, -1].contiguous(), k[:, -1].contiguous(), t["v"][:, 0].contiguous(), t["ld"], 0.1)
    beams = state.view(2, 2, *state.shape[1:])
    logits = step.flatten(1).view(2, 2, -1)
    best, words, origins = mssm.beam_select(logits, t["scores"], 2)
    mssm.state_reorder([beams], origins)
    return [o, state, g["dv"], *n.values(), step, best, words, origins]


def layer_inputs(dev, seed):
    shape = (4, 600, 3, 32)
    return {"q": randn(dev, *shape, seed=seed, dtype=torch.bfloat16), "k": randn(dev, *shape, seed=seed + 1, dtype=torch.bfloat16),
            "v": randn(dev, *shape, seed=seed + 2, dtype=torch.bfloat16), "do": randn(dev, *shape, seed=seed + 3, dtype=torch.bfloat16),
            "pos": torch.arange(600, device=dev).repeat(4, 1), "wq": randn(dev, 32, seed=seed + 4, shift=1.0),
            "wk": randn(dev, 32, seed=seed + 5, shift=1.0), "ld": torch.tensor([-0.2, -0.03, -0.004], device=dev),
            "scores": randn(dev, 2, 2, seed=seed + 6)}


def test_together(dev, mssm):
    """Prompt, gradients, a step and a selection against the definitions."""
    announce("together")
    t = layer_inputs(dev, 0)
    q, k = mssm.qk_norm_rotary_fwd(t["q"], t["k"], t["pos"], t["wq"], t["wk"])
    o, state, dv, dq, dk, dwq, dwk, step, best, words, origins = layer(mssm, t)
    wo, ws = A.linear_attention(q, k, t["v"], t["ld"], 0.1)
    assert rms(o, wo) <= RMS["bf16"] * 1.1
    w1, ws = A.linear_attention(q[:, -1:], k[:, -1:], t["v"][:, :1], t["ld"], 0.1, ws)
    assert rms(step, w1[:, 0]) <= U16
    wb, ww, wi = A.beam_select(step.flatten(1).view(2, 2, -1), t["scores"], 2)
    assert torch.equal(words, ww) and torch.equal(origins, wi)
    ws = A.state_reorder(ws.view(2, 2, *ws.shape[1:]), wi).view(state.shape)
    assert rms(state, ws) <= 1e-4
    g = mssm.linear_attention_bwd(q, k, t["v"], t["ld"], t["do"], 0.1)
    wg = A.linear_attention_grad(q, k, t["v"], t["ld"], t["do"], 0.1)
    for got, n, x, w in ((dq, "dq", t["q"], t["wq"]), (dk, "dk", t["k"], t["wk"])):
        assert rms(g[n], wg[n]) <= RMS["bf16"] * 1.1
        want = A.head_norm_rotary_grad(g[n], x, t["pos"], w)
        assert rms(got, want["dx"]) <= U16
    assert rms(dv, wg["dv"]) <= RMS["bf16"] * 1.1


def test_on_another_stream(dev, mssm):
    announce("stream")
    t = layer_inputs(dev, 3)
    want = layer(mssm, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer(mssm, t)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_in_a_graph(dev, mssm):
    """Captured once, replayed with eager calls of the same operators in between, on
    inputs that change."""
    announce("graph")
    t = layer_inputs(dev, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(mssm, t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(mssm, t)
    for turn in range(4):
        other = layer_inputs(dev, 20 + turn)
        for n in t:
            t[n].copy_(other[n])
        graph.replay()
        want = layer(mssm, other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_two_streams_at_once(dev, mssm):
    """The same calls on two streams, with nothing shared but inputs."""
    announce("two streams")
    a, b = layer_inputs(dev, 40), layer_inputs(dev, 50)
    wa, wb = layer(mssm, a), layer(mssm, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = layer(mssm, a)
        with torch.cuda.stream(s2):
            gb = layer(mssm, b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ga, wa)) and all(torch.equal(x, y) for x, y in zip(gb, wb))

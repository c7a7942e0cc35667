"""Cases of the linear attention layer and of decoding by beams: the norm of
queries and keys with their rotation, linear attention with a decay per head,
the selection of beams over a vocabulary and the reordering of their states.

``listed()`` gives the cases, ``draw(rng)`` one more of the same ranges,
``prepare`` the tensors a program holds before the call, ``run`` one call and
its outputs, ``work`` the bytes and operations no implementation can do
without, ``exact`` the outputs from the definitions in 64 bits.  With ``own``
false ``run`` evaluates the definitions with elementary torch operations in
float32 (angles of positions and the values that beams are chosen by in
float64); with ``own`` true it calls the library.

Definitions (activations in one dtype, states and weights float32):

  norm and rotation, per token at position p and head of D values
    n = x rsqrt(mean(x^2) + eps) w
    y_j = n_j cos a_j - n_{j+R/2} sin a_j,  y_{j+R/2} = n_{j+R/2} cos a_j + n_j sin a_j,
    a_j = p base^(-2j/R) for j < R/2;  values from R on stay as they are
  linear attention, per sequence and head
    S_t = e^log_decay S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
  selection, per batch entry, over beams j and words v
    value = score_j + logit_{j,v} - log sum_v exp logit_{j,v}   (NaN counts as -inf)
    the `count` largest, ties to the lowest j V + v
  reorder, in place:  row (b, j) <- row (b, origin[b, j])
"""
import math

import torch

own = False

BASE, EPS = 10000.0, 1e-6    # of the rotation and the norm
CHUNK = 256                  # steps that the plain form's attention takes at a time
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # queries and keys of one decode step of eight sequences
        {"name": "norm_step_bf16", "op": "norm_fwd", "tokens": 8, "q_heads": 20, "k_heads": 20,
         "dim": 128, "rotary": 128, "far": 1 << 14, "io": "bf16"},
        # a float32 model with odd head counts, half of each head rotated, far positions
        {"name": "norm_odd_f32", "op": "norm_fwd", "tokens": 1031, "q_heads": 9, "k_heads": 3,
         "dim": 80, "rotary": 40, "far": 1 << 20, "io": "f32"},
        # backward of the norm and rotation over one training micro-batch (2 x 4096 tokens)
        {"name": "norm_layer_bwd_bf16", "op": "norm_bwd", "tokens": 8192, "q_heads": 20,
         "k_heads": 20, "dim": 128, "rotary": 128, "far": 4096, "io": "bf16"},
        # one decode step of one sequence, where the call's latency counts
        {"name": "attention_step_one_bf16", "op": "attn_step", "batch": 1, "heads": 20,
         "key": 128, "value": 128, "io": "bf16"},
        # one decode step of 64 sequences: their states are read and written
        {"name": "attention_step_bf16", "op": "attn_step", "batch": 64, "heads": 20,
         "key": 128, "value": 128, "io": "bf16"},
        # the attention of a training micro-batch, forward
        {"name": "attention_layer_bf16", "op": "attn_fwd", "batch": 2, "seqlen": 4096,
         "heads": 20, "key": 128, "value": 128, "io": "bf16", "packed": False, "h0": False},
        # its backward
        {"name": "attention_layer_bwd_bf16", "op": "attn_bwd", "batch": 2, "seqlen": 4096,
         "heads": 20, "key": 128, "value": 128, "io": "bf16", "packed": False, "h0": False},
        # one long prompt on few heads, continued from a state
        {"name": "attention_long_bf16", "op": "attn_fwd", "batch": 1, "seqlen": 1 << 17,
         "heads": 4, "key": 128, "value": 128, "io": "bf16", "packed": False, "h0": True},
        # backward of a small float32 model over packed sequences of any length, odd sizes
        {"name": "attention_packed_bwd_f32", "op": "attn_bwd", "batch": 7, "seqlen": 431,
         "heads": 5, "key": 80, "value": 72, "io": "f32", "packed": True, "h0": True},
        # a step of one beam search, twice as many candidates as beams
        {"name": "beams_one_bf16", "op": "beam", "batch": 1, "beams": 4, "vocab": 50021,
         "count": 8, "io": "bf16"},
        # a step of a batch of searches with wide beams
        {"name": "beams_batch_f32", "op": "beam", "batch": 16, "beams": 8, "vocab": 50021,
         "count": 16, "io": "f32"},
        # the states of two layers and the words so far, half of the beams replaced
        {"name": "reorder_bf16", "op": "reorder", "batch": 16, "beams": 4, "moved": 2,
         "layers": 2, "heads": 20, "key": 128, "value": 128, "words": 257},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _ragged(rng, n):
    """n, or a near size that is a multiple of nothing in particular."""
    return n if rng.random() < 0.3 else max(1, n - rng.randrange(0, max(1, n // 16) + 1))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "attn_step", "attn_fwd", "attn_bwd", "beam", "reorder"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        dim = rng.choice([64, 128, rng.randint(16, 256)])
        k_heads = _log_uniform(rng, 1, 24)
        q_heads = k_heads * rng.choice([1, 1, 2, 4])
        tokens = _ragged(rng, _log_uniform(rng, 1, max(1, min(1 << 16, (1 << 24) // (dim * q_heads)))))
        return {"op": op, "tokens": tokens, "q_heads": q_heads, "k_heads": k_heads, "dim": dim,
                "rotary": rng.choice([dim // 2 * 2, dim // 4 * 2, 0]), "far": _log_uniform(rng, 1024, 1 << 20),
                "io": io}
    if op == "beam":
        beams = rng.randint(1, 16)
        vocab = _ragged(rng, _log_uniform(rng, 1000, 1 << 17))
        return {"op": op, "batch": _log_uniform(rng, 1, max(1, (1 << 22) // (beams * vocab))), "beams": beams,
                "vocab": vocab, "count": rng.choice([beams, 2 * beams]), "io": io}
    key, value = (rng.choice([64, 128, rng.randint(16, 256)]) for _ in range(2))
    heads = _log_uniform(rng, 1, 40)
    if op == "reorder":
        beams = rng.randint(2, 16)
        most = (1 << 26) // (beams * heads * key * value)
        return {"op": op, "batch": _log_uniform(rng, 1, max(1, min(32, most))), "beams": beams,
                "moved": rng.randint(1, beams), "layers": rng.randint(1, 3), "heads": heads,
                "key": key, "value": value, "words": _log_uniform(rng, 1, 4000)}
    if op == "attn_step":
        return {"op": op, "batch": _log_uniform(rng, 1, max(1, min(256, (1 << 24) // (heads * key * value)))),
                "heads": heads, "key": key, "value": value, "io": io}
    most = (1 << 30) if io == "bf16" else (1 << 27)
    batch = rng.randint(1, 8)
    seqlen = _ragged(rng, _log_uniform(rng, 1, max(1, min(1 << 17, most // (batch * heads * max(key, 64) * max(value, 64))))))
    return {"op": op, "batch": batch, "seqlen": seqlen, "heads": heads, "key": key, "value": value,
            "io": io, "packed": rng.random() < 0.4, "h0": rng.random() < 0.5}


# ---- inputs ------------------------------------------------------------------

def _lengths(case, seed):
    """Lengths of packed sequences, batch * seqlen in all: ragged, some of
    them empty."""
    g = torch.Generator()
    g.manual_seed(seed)
    total = case["batch"] * case["seqlen"]
    share = torch.rand(case["batch"], generator=g) + 0.01
    share[torch.rand(case["batch"], generator=g) < 0.15] = 0.0
    lengths = [int(total * v / max(1e-6, float(share.sum()))) for v in share.tolist()]
    lengths[0] += total - sum(lengths)
    return lengths


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dtype)

    op = case["op"]
    s = {"op": op}
    if op == "reorder":
        batch, beams = case["batch"], case["beams"]
        s["states"] = [normal(batch, beams, case["heads"], case["key"], case["value"])
                       for _ in range(case["layers"])]
        s["states"].append(torch.randint(0, 50021, (batch, beams, case["words"]), generator=g, device="cuda"))
        # `moved` beams of every entry continue another one, the others themselves
        order = torch.rand(batch, beams, generator=g, device="cuda").argsort(1)[:, :case["moved"]]
        origins = torch.arange(beams, device="cuda").repeat(batch, 1)
        shift = torch.randint(1, beams, (batch, case["moved"]), generator=g, device="cuda")
        s["origins"] = origins.scatter(1, order, (order + shift) % beams)
        return s
    io = DTYPES[case["io"]]
    if op.startswith("norm"):
        t, d = case["tokens"], case["dim"]
        s["rotary"] = case["rotary"]
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda")
        for name, heads in (("q", case["q_heads"]), ("k", case["k_heads"])):
            # projections: heads of different sizes
            size = torch.rand(1, heads, 1, generator=g, device="cuda") * 2.5 + 0.5
            s[name] = (normal(t, heads, d) * size).to(io)
            s[name + "_weight"] = normal(d, mean=1.0, std=0.2)
            if op == "norm_bwd":
                s["d" + name] = normal(t, heads, d, dtype=io)
        return s
    if op == "beam":
        batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
        s["count"] = case["count"]
        logits = normal(batch, beams, vocab, std=3.0)
        # about one word in a hundred is forbidden
        logits[torch.rand(batch, beams, vocab, generator=g, device="cuda") < 0.01] = float("-inf")
        s["logits"] = logits.to(io)
        s["scores"] = normal(batch, beams, mean=-20.0, std=2.0).sort(1, descending=True).values
        return s
    heads, key, value = case["heads"], case["key"], case["value"]
    # decays a step from 1 - 1/32 to 1 - 1/512 over the heads
    s["log_decay"] = torch.log1p(-torch.exp(-torch.linspace(math.log(32), math.log(512), heads,
                                                            device="cuda", dtype=torch.float64))).float()
    s["scale"] = key ** -0.5
    if op == "attn_step":
        batch = case["batch"]
        s["q"], s["k"] = normal(batch, heads, key, dtype=io), normal(batch, heads, key, dtype=io)
        s["v"] = normal(batch, heads, value, dtype=io)
        s["state"] = normal(batch, heads, key, value, std=4.0)
        return s
    batch = case["batch"]
    shape = (batch, case["seqlen"])
    s["cu_seqlens"], s["longest"] = None, case["seqlen"]
    if case["packed"]:
        lengths = _lengths(case, seed)
        ends = [sum(lengths[:j]) for j in range(batch + 1)]
        s["cu_seqlens"] = torch.tensor(ends, device="cuda")
        s["longest"] = max(lengths)
        shape = (ends[-1],)
    s["q"], s["k"] = normal(*shape, heads, key, dtype=io), normal(*shape, heads, key, dtype=io)
    s["v"] = normal(*shape, heads, value, dtype=io)
    s["h0"] = normal(batch, heads, key, value, std=4.0) if case["h0"] else None
    if op == "attn_bwd":
        s["do"] = normal(*shape, heads, value, dtype=io)
        s["dh_last"] = normal(batch, heads, key, value, std=0.2) if case["h0"] else None
    return s


# ---- one pass ----------------------------------------------------------------

def run(state):
    return (_library if own else _plain)(state)


def _library(s):
    import selective_state_space_05_amd as mssm
    op = s["op"]
    if op == "norm_fwd":
        return mssm.qk_norm_rotary_fwd(s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"],
                                       base=BASE, eps=EPS, rotary_dim=s["rotary"])
    if op == "norm_bwd":
        return mssm.qk_norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["q_weight"],
                                       s["k_weight"], base=BASE, eps=EPS, rotary_dim=s["rotary"])
    if op == "attn_step":
        o = mssm.linear_attention_update(s["state"], s["q"], s["k"], s["v"], s["log_decay"], s["scale"])
        return o, s["state"]
    if op == "attn_fwd":
        return mssm.linear_attention_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], h0=s["h0"],
                                         cu_seqlens=s["cu_seqlens"], max_seqlen=s["longest"])
    if op == "attn_bwd":
        return mssm.linear_attention_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], s["scale"],
                                         h0=s["h0"], dh_last=s["dh_last"], cu_seqlens=s["cu_seqlens"],
                                         max_seqlen=s["longest"])
    if op == "beam":
        return mssm.beam_select(s["logits"], s["scores"], s["count"])
    mssm.state_reorder(s["states"], s["origins"])
    return s["states"]


def _rotate(n, cos, sin, rotary):
    half = rotary // 2
    a, b, rest = n[..., :half], n[..., half:rotary], n[..., rotary:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _angles(positions, rotary):
    """cos and sin of every token's angles, the angles in float64."""
    rate = BASE ** (-2.0 * torch.arange(rotary // 2, device=positions.device, dtype=torch.float64) / max(1, rotary))
    a = positions.double()[:, None, None] * rate
    return torch.cos(a).float(), torch.sin(a).float()


def _norm_grad(dy, x, w, cos, sin, rotary):
    x32, dn = x.float(), _rotate(dy.float(), cos, -sin, rotary)
    r = (x32.square().mean(-1, keepdim=True) + EPS).rsqrt()
    e = dn * w
    dx = r * (e - x32 * r * (e * x32 * r).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dn * x32 * r).sum((0, 1))


def _attend(q, k, v, log_decay, first, early, lengths):
    """o_i = sum_{j <= i} g^(i-j) (q_i . k_j) v_j + g^(i+early) q_i first over
    (batch, heads, steps, width), g = e^log_decay, and the state behind the
    last step, g^n first + sum_j g^(n-early-j) k_j v_j^T with n steps in all."""
    batch, heads, steps, key = q.shape
    ld = log_decay[None, :, None]
    n = max(1, -(-steps // CHUNK))
    at = torch.arange(n * CHUNK, device=q.device)
    tail = torch.exp(ld * (lengths[:, None] - early - at[None, :steps])[:, None].clamp(min=0).float())
    live = (at[None, :steps] < lengths[:, None])[:, None]
    weighted = k * torch.where(live, tail, torch.zeros_like(tail))[..., None]
    last = weighted.transpose(2, 3).contiguous() @ v
    if first is not None:
        last = last + torch.exp(ld * lengths[:, None, None].float())[..., None] * first

    def cut(t):
        t = torch.nn.functional.pad(t, (0, 0, 0, n * CHUNK - steps))
        return t.reshape(batch, heads, n, CHUNK, t.shape[-1])

    q, k, v = cut(q), cut(k), cut(v)
    i = at[:CHUNK].float()
    gap = i[:, None] - i
    inside = torch.where(gap >= 0, torch.exp(ld[..., None] * gap.clamp(min=0)), torch.zeros_like(gap))
    p = (q @ k.transpose(3, 4).contiguous()) * inside[:, :, None]
    o = p @ v
    local = (k * torch.exp(ld * (CHUNK - early - i))[:, :, None, :, None]).transpose(3, 4).contiguous() @ v
    chunks = at[:n].float()
    back = chunks[:, None] - 1 - chunks
    carry = torch.where(back >= 0, torch.exp(ld[..., None] * CHUNK * back.clamp(min=0)), torch.zeros_like(back))
    entering = (carry @ local.reshape(batch, heads, n, -1)).reshape(local.shape)
    if first is not None:
        entering = entering + torch.exp(ld * CHUNK * chunks)[..., None, None] * first[:, :, None]
    o = o + torch.exp(ld * (i + early))[:, :, None, :, None] * (q @ entering)
    return o.reshape(batch, heads, n * CHUNK, -1)[:, :, :steps], last


def _plain_attention(s):
    cu, longest = s["cu_seqlens"], s["longest"]
    q = s["q"]
    if cu is None:
        lengths = torch.full((q.shape[0],), longest, device=q.device)
    else:
        lengths = cu[1:] - cu[:-1]
        steps = torch.arange(longest, device=q.device)
        at = (cu[:-1, None] + steps).clamp(max=max(0, q.shape[0] - 1))
        turned = (cu[1:, None] - 1 - steps).clamp(min=0)
        live = (steps < lengths[:, None])[..., None, None]
        rows = torch.repeat_interleave(torch.arange(cu.shape[0] - 1, device=q.device), lengths, output_size=q.shape[0])
        offset = torch.arange(q.shape[0], device=q.device) - cu[:-1][rows]

    def spread(t, back=False):       # -> (sequences, heads, steps, width), in time or against it
        t = t.float()
        if cu is not None:
            t = t[turned if back else at] * live if t.shape[0] else t.new_zeros(live.shape[:2] + t.shape[1:])
        elif back:
            t = t.flip(1)
        return t.transpose(1, 2).contiguous()

    def gather(t, like, back=False):
        t = t.transpose(1, 2)
        if cu is not None:
            t = t[rows, (lengths[rows] - 1 - offset) if back else offset]
        elif back:
            t = t.flip(1)
        return t.to(like.dtype).contiguous()

    k, v, ld, scale = s["k"], s["v"], s["log_decay"], s["scale"]
    gate = torch.exp(ld)[:, None, None]
    first = None if s["h0"] is None else s["h0"]
    if s["op"] == "attn_fwd":
        o, last = _attend(spread(q) * scale, spread(k), spread(v), ld, first, 1, lengths)
        return gather(o, v), last
    do, dlast = s["do"], s["dh_last"]
    turn = None if first is None else first.transpose(2, 3).contiguous()
    dq = _attend(spread(do) * scale, spread(v), spread(k), ld, turn, 1, lengths)[0]
    turn = None if dlast is None else dlast.transpose(2, 3).contiguous()
    dk = _attend(spread(v, True), spread(do, True), spread(q, True) * scale, ld, turn, 0, lengths)[0]
    dv, dfirst = _attend(spread(k, True), spread(q, True) * scale, spread(do, True), ld, dlast, 0, lengths)
    return {"dq": gather(dq, q), "dk": gather(dk, k, True), "dv": gather(dv, v, True), "dh0": dfirst}


def _plain(s):
    op = s["op"]
    if op == "reorder":
        at = torch.arange(s["origins"].shape[0], device=s["origins"].device)[:, None]
        return [t.copy_(t[at, s["origins"]]) for t in s["states"]]
    if op.startswith("norm"):
        cos, sin = _angles(s["positions"], s["rotary"])
        if op == "norm_bwd":
            dq, dqw = _norm_grad(s["dq"], s["q"], s["q_weight"], cos, sin, s["rotary"])
            dk, dkw = _norm_grad(s["dk"], s["k"], s["k_weight"], cos, sin, s["rotary"])
            return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
        q, k = s["q"].float(), s["k"].float()
        q = q * (q.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["q_weight"]
        k = k * (k.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["k_weight"]
        return (_rotate(q, cos, sin, s["rotary"]).to(s["q"].dtype),
                _rotate(k, cos, sin, s["rotary"]).to(s["k"].dtype))
    if op == "attn_step":
        k, v = s["k"].float(), s["v"].float()
        s["state"].mul_(torch.exp(s["log_decay"])[:, None, None]).add_(k[..., :, None] * v[..., None, :])
        o = (s["q"].float()[..., :, None] * s["state"]).sum(-2) * s["scale"]
        return o.to(s["v"].dtype), s["state"]
    if op == "beam":
        logits, n = s["logits"].double(), s["count"]
        top = logits.amax(-1, keepdim=True)
        lse = top + torch.log(torch.exp(logits - top).sum(-1, keepdim=True))
        value = (s["scores"].double()[..., None] + (logits - lse)).flatten(1)
        value = torch.where(value.isnan(), torch.full_like(value, float("-inf")), value)
        best, at = torch.sort(value, dim=1, descending=True, stable=True)
        vocab = logits.shape[2]
        return best[:, :n].float(), at[:, :n] % vocab, at[:, :n] // vocab
    return _plain_attention(s)


# ---- bytes and operations ----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "reorder":      # the moved rows, read and written
        row = case["layers"] * case["heads"] * case["key"] * case["value"] * 4 + case["words"] * 8
        return {"bytes": 2 * case["batch"] * case["moved"] * row, "flops": 0}
    e = 4 if case["io"] == "f32" else 2
    if op.startswith("norm"):
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        if op == "norm_fwd":     # q, k, positions, weights -> q, k
            return {"bytes": 2 * n * e + 8 * case["tokens"] + 8 * case["dim"], "flops": 8 * n}
        # dq, dk, q, k, positions, weights -> dq, dk, dweights
        return {"bytes": 3 * n * e + 8 * case["tokens"] + 16 * case["dim"], "flops": 16 * n}
    if op == "beam":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * e, "flops": 4 * n}
    bh, key, value = case["batch"] * case["heads"], case["key"], case["value"]
    if op == "attn_step":        # q, k, v, state -> o, state
        return {"bytes": bh * (8 * key * value + 2 * (key + value) * e), "flops": 5 * bh * key * value}
    n, states = bh * case["seqlen"], 4 * bh * key * value
    if op == "attn_fwd":         # q, k, v, h0 -> o, h_last
        return {"bytes": 2 * n * (key + value) * e + states * (2 if case["h0"] else 1), "flops": 4 * n * key * value}
    # q, k, v, do, h0, dh_last -> dq, dk, dv, dh0
    return {"bytes": n * (4 * key + 3 * value) * e + states * (3 if case["h0"] else 1),
            "flops": 10 * n * key * value}


# ---- the definitions in 64 bits ----------------------------------------------

def _runs(s, case):
    """(first, behind the last) row of every sequence of the flattened rows."""
    if s["cu_seqlens"] is None:
        return [(b * case["seqlen"], (b + 1) * case["seqlen"]) for b in range(case["batch"])]
    cu = s["cu_seqlens"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_sequence(q, k, v, do, ld, scale, h, dh):
    """One sequence, (steps, heads, width) in 64 bits, 128 steps at a time
    through the state in front of each stretch."""
    steps, width = q.shape[0], 128
    o, dq, dk, dv = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    heads_first = [t.permute(1, 0, 2) for t in ((q, k, v) if do is None else (q, k, v, do))]

    def part(a, b):
        n = b - a
        i = torch.arange(n, device=q.device, dtype=torch.float64)
        mask = torch.tril(torch.exp(ld[:, None, None] * (i[:, None] - i).clamp(min=0)))
        return (mask, [torch.exp(ld[:, None] * x)[..., None] for x in (i + 1, n - 1 - i)],
                torch.exp(ld * n)[:, None, None], [t[:, a:b].contiguous() for t in heads_first])

    for a in range(0, steps, width):
        mask, (front, back), whole, (qa, ka, va, *rest) = part(a, min(steps, a + width))
        if do is None:
            r = torch.bmm(torch.bmm(qa, ka.mT.contiguous()) * mask, va) + front * torch.bmm(qa, h)
            o[a:a + width] = scale * r.permute(1, 0, 2)
        else:
            r = torch.bmm(torch.bmm(rest[0], va.mT.contiguous()) * mask, ka) + front * torch.bmm(rest[0], h.mT.contiguous())
            dq[a:a + width] = scale * r.permute(1, 0, 2)
        h = whole * h + torch.bmm((ka * back).mT.contiguous(), va)
    if do is None:
        return o, h
    decay = torch.exp(ld)[:, None, None]
    dh = dh / decay                      # so that every stretch decays it by its own steps
    for a in reversed(range(0, steps, width)):
        mask, (front, back), whole, (qa, ka, va, da) = part(a, min(steps, a + width))
        down = mask.mT.contiguous()      # of later steps i on j <= i
        rest = back * decay              # g^(n-j) from behind the stretch
        dk[a:a + width] = (scale * torch.bmm(torch.bmm(va, da.mT.contiguous()) * down, qa)
                           + rest * torch.bmm(va, dh.mT.contiguous())).permute(1, 0, 2)
        dv[a:a + width] = (scale * torch.bmm(torch.bmm(ka, qa.mT.contiguous()) * down, da)
                           + rest * torch.bmm(ka, dh)).permute(1, 0, 2)
        dh = whole * dh + scale * torch.bmm((qa * front / decay).mT.contiguous(), da)
    return dq, dk, dv, dh * decay


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "reorder":
        picked = []
        for t in s["states"]:
            rows = [[t[b, int(j)] for j in s["origins"][b]] for b in range(t.shape[0])]
            picked.append(torch.stack([torch.stack(r) for r in rows]).to(torch.float64 if t.is_floating_point() else t.dtype))
        return picked
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op.startswith("norm"):
        half, d = case["rotary"] // 2, case["dim"]
        turn = torch.zeros(case["tokens"], 1, d, dtype=torch.complex128, device="cuda") + 1
        if half:
            rate = torch.exp(-math.log(BASE) * torch.arange(half, device="cuda", dtype=torch.float64) / half)
            turn[:, 0, :half] = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                                            s["positions"].double().view(-1, 1) * rate)

        def spin(t, by):                 # pairs as complex numbers
            t = t.clone()
            z = torch.complex(t[..., :half].contiguous(), t[..., half:2 * half].contiguous()) * by[..., :half]
            t[..., :half], t[..., half:2 * half] = z.real, z.imag
            return t

        out = {}
        for n in ("q", "k"):
            x, w = s[n], s[n + "_weight"]
            r = 1 / torch.sqrt(x.pow(2).sum(-1, True) / d + EPS)
            if op == "norm_fwd":
                out[n] = spin(x * r * w, turn)
                continue
            dn = spin(s["d" + n], turn.conj())
            e = dn * w
            out["d" + n] = e * r - x * r.pow(3) * ((e * x).sum(-1, True) / d)
            out["d" + n + "_weight"] = (dn * (x * r)).sum(1).sum(0)
        if op == "norm_fwd":
            return out["q"], out["k"]
        return {n: out[n] for n in ("dq", "dk", "dq_weight", "dk_weight")}
    if op == "attn_step":
        h = torch.exp(s["log_decay"]).view(1, -1, 1, 1) * s["state"] + s["k"].unsqueeze(3) * s["v"].unsqueeze(2)
        return (s["q"].unsqueeze(3) * h).sum(2) * s["scale"], h
    if op == "beam":
        batch, beams, vocab = s["logits"].shape
        p = s["scores"].unsqueeze(2) + torch.log_softmax(s["logits"], 2)
        flat = torch.where(p != p, torch.full_like(p, float("-inf")), p).view(batch, beams * vocab)
        words = []
        for _ in range(case["count"]):   # the largest, the first of equal ones, again and again
            top = flat.amax(1, keepdim=True)
            at = (flat == top).int().argmax(1, keepdim=True)
            words.append((top, at))
            flat = flat.scatter(1, at, float("-inf"))
        value, at = torch.cat([w[0] for w in words], 1), torch.cat([w[1] for w in words], 1)
        return value, at % vocab, torch.div(at, vocab, rounding_mode="floor")
    heads = case["heads"]
    rows = {n: s[n].reshape(-1, heads, s[n].shape[-1]) for n in ("q", "k", "v", "do") if n in s}
    zero = torch.zeros(heads, case["key"], case["value"], dtype=torch.float64, device="cuda")
    parts = []
    for b, (lo, hi) in enumerate(_runs(s, case)):
        do = rows["do"][lo:hi] if op == "attn_bwd" else None
        parts.append(_exact_sequence(
            rows["q"][lo:hi], rows["k"][lo:hi], rows["v"][lo:hi], do, s["log_decay"], s["scale"],
            zero if s["h0"] is None else s["h0"][b],
            zero if op == "attn_fwd" or s["dh_last"] is None else s["dh_last"][b]))
    joined = [torch.cat([p[j] for p in parts]) for j in range(len(parts[0]) - 1)]
    ends = torch.stack([p[-1] for p in parts])
    if op == "attn_fwd":
        return joined[0].view(s["v"].shape), ends
    return {"dq": joined[0].view(s["q"].shape), "dk": joined[1].view(s["k"].shape),
            "dv": joined[2].view(s["v"].shape), "dh0": ends}

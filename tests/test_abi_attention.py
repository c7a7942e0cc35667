"""Refusals of the norm-with-rotation, linear-attention and beam-search entry
points: the C ABI rejects every invalid call before touching the HIP runtime,
and the binding rejects what the C ABI cannot see.  No GPU; pointers are fake
non-null addresses that validation never dereferences."""
from __future__ import annotations

import ctypes

import pytest

from selective_state_space_05_amd import _lib
from test_abi import L, fake  # noqa: F401  (L is the library fixture)

INVALID, UNSUPPORTED = _lib.MSSM_ERR_INVALID_ARG, _lib.MSSM_ERR_UNSUPPORTED


def call(L, fn, names, scalars, *last, **ptrs):
    p = {n: fake(8 * k + 1) for k, n in enumerate(names) if n not in scalars}
    p.update(scalars)
    p.update(ptrs)
    return getattr(L, "mssm_" + fn)(*[p[n] for n in names], *last, None)


def norm(L, fn, names, tokens=4, q_heads=2, k_heads=3, dim=8, rotary=6, io=0, param=0, **kw):
    scalars = dict(base=kw.pop("base", 1e4), eps=kw.pop("eps", 1e-6), workspace=kw.pop("workspace", None),
                   bytes=kw.pop("bytes", 0))
    return call(L, fn, names, scalars, _lib.HeadNormDims(tokens, q_heads, k_heads, dim, rotary),
                _lib.DTypes(io, param), **kw)


def norm_fwd(L, **kw):
    return norm(L, "qk_norm_rotary_fwd", ["q", "k", "positions", "q_weight", "k_weight", "base", "eps", "q_out",
                                          "k_out"], **kw)


def norm_bwd(L, **kw):
    return norm(L, "qk_norm_rotary_bwd", ["dq_out", "dk_out", "q", "k", "positions", "q_weight", "k_weight", "base",
                                          "eps", "dq", "dk", "dq_weight", "dk_weight", "workspace", "bytes"], **kw)


def attention(L, fn, names, seqs=2, seqlen=5, total=None, heads=3, key=4, value=6, io=0, param=0, **kw):
    scalars = dict(scale=kw.pop("scale", 1.0), workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0),
                   cu_seqlens=kw.pop("cu_seqlens", None))
    total = seqs * seqlen if total is None else total
    return call(L, fn, names, scalars, _lib.AttentionDims(seqs, seqlen, total, heads, key, value),
                _lib.DTypes(io, param), **kw)


def attn_fwd(L, **kw):
    return attention(L, "linear_attention_fwd", ["q", "k", "v", "log_decay", "scale", "h0", "cu_seqlens", "o",
                                                 "h_last", "workspace", "bytes"], **kw)


def attn_bwd(L, **kw):
    return attention(L, "linear_attention_bwd", ["q", "k", "v", "log_decay", "scale", "h0", "cu_seqlens", "d_o",
                                                 "dh_last", "dq", "dk", "dv", "dh0", "workspace", "bytes"], **kw)


def attn_step(L, **kw):
    return attention(L, "linear_attention_update", ["state", "q", "k", "v", "log_decay", "scale", "o"], **kw)


def beam(L, batch=2, beams=3, vocab=10, count=4, io=0, param=0, **kw):
    scalars = dict(workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0))
    return call(L, "beam_select", ["logits", "scores", "out_scores", "out_tokens", "out_beams", "workspace", "bytes"],
                scalars, _lib.BeamDims(batch, beams, vocab, count), _lib.DTypes(io, param), **kw)


def reorder(L, states=None, rows=(32, 8), batch=2, beams=3, origins=fake(500), count=None):
    states = [fake(1), fake(64)] if states is None else states
    n = len(states)
    return L.mssm_state_reorder((ctypes.c_void_p * n)(*states), (ctypes.c_int64 * n)(*rows), n if count is None else count,
                                origins, _lib.BeamDims(batch, beams, 1, 1), None)


CALLS = {"norm_fwd": norm_fwd, "norm_bwd": norm_bwd, "attn_fwd": attn_fwd, "attn_bwd": attn_bwd,
         "attn_step": attn_step, "beam": beam}
REQUIRED = {"norm_fwd": ["q", "k", "positions", "q_out", "k_out"],
            "norm_bwd": ["dq_out", "dk_out", "q", "k", "positions", "dq", "dk"],
            "attn_fwd": ["q", "k", "v", "log_decay", "o"],
            "attn_bwd": ["q", "k", "v", "log_decay", "d_o", "dq", "dk", "dv"],
            "attn_step": ["state", "q", "k", "v", "log_decay", "o"],
            "beam": ["logits", "scores", "out_scores", "out_tokens", "out_beams"]}
# (output, overlapping operand)
OVERLAPS = {"norm_fwd": [("q_out", "q"), ("k_out", "k"), ("q_out", "k_out"), ("k_out", "positions"), ("q_out", "k_weight")],
            "norm_bwd": [("dq", "dq_out"), ("dk", "q"), ("dq", "dk"), ("dq_weight", "dk_weight"), ("dk_weight", "k")],
            "attn_fwd": [("o", "q"), ("o", "v"), ("h_last", "log_decay"), ("o", "h_last"), ("h_last", "h0"), ("o", "h0")],
            "attn_bwd": [("dq", "q"), ("dk", "v"), ("dv", "d_o"), ("dh0", "dh_last"), ("dq", "dk"), ("dh0", "h0"),
                         ("dv", "log_decay")],
            "attn_step": [("state", "q"), ("o", "v"), ("o", "state"), ("state", "log_decay")],
            "beam": [("out_scores", "scores"), ("out_tokens", "logits"), ("out_tokens", "out_beams")]}


@pytest.mark.parametrize("op,name", [(o, n) for o in CALLS for n in REQUIRED[o]])
def test_null_required_pointer(L, op, name):
    assert CALLS[op](L, **{name: None}) == INVALID
    assert name.encode() in L.mssm_last_error()


@pytest.mark.parametrize("op,out,other", [(o, a, b) for o in CALLS for a, b in OVERLAPS[o]])
def test_overlap(L, op, out, other):
    at = fake(900)
    assert CALLS[op](L, **{out: at + 4, other: at}) == INVALID
    assert b"overlap" in L.mssm_last_error()


def test_overlap_with_packed_offsets(L):
    at = fake(900)
    assert attn_fwd(L, cu_seqlens=at, o=at + 8) == INVALID and b"overlap" in L.mssm_last_error()
    assert attn_bwd(L, cu_seqlens=at, dh0=at + 8) == INVALID and b"overlap" in L.mssm_last_error()


@pytest.mark.parametrize("op", CALLS)
def test_dtypes(L, op):
    assert CALLS[op](L, io=2) == INVALID
    assert CALLS[op](L, param=3) == INVALID
    assert CALLS[op](L, param=_lib.MSSM_BF16) == UNSUPPORTED


SIZES = {"norm_fwd": ["tokens", "q_heads", "k_heads", "dim", "rotary"], "attn_fwd": ["seqs", "seqlen", "heads", "key", "value"],
         "attn_step": ["seqs", "heads", "key", "value"], "beam": ["batch", "beams", "vocab", "count"]}
SIZES["norm_bwd"], SIZES["attn_bwd"] = SIZES["norm_fwd"], SIZES["attn_fwd"]


@pytest.mark.parametrize("op,key", [(o, k) for o in CALLS for k in SIZES[o]])
def test_negative_and_huge_sizes(L, op, key):
    assert CALLS[op](L, **{key: -1}) == INVALID
    assert CALLS[op](L, **{key: 1 << 40}) in (INVALID, UNSUPPORTED)
    assert CALLS[op](L, **{key: (1 << 62) + 1}) in (INVALID, UNSUPPORTED)
    assert L.mssm_last_error()


def test_sizes_out_of_the_operators_ranges(L):
    for op in ("norm_fwd", "norm_bwd"):
        assert CALLS[op](L, dim=0, rotary=0) == INVALID
        assert CALLS[op](L, rotary=5) == INVALID and b"rotary" in L.mssm_last_error()
        assert CALLS[op](L, rotary=10) == INVALID
        assert CALLS[op](L, dim=257) == UNSUPPORTED
    for op in ("attn_fwd", "attn_bwd", "attn_step"):
        for key in ("key", "value"):
            assert CALLS[op](L, **{key: 0}) == INVALID
            assert CALLS[op](L, **{key: 257}) == UNSUPPORTED
        assert CALLS[op](L, seqs=1 << 10, heads=1 << 10) == UNSUPPORTED
    assert attn_fwd(L, total=11) == INVALID and b"total" in L.mssm_last_error()
    assert attn_bwd(L, total=1 << 31, cu_seqlens=fake(700)) == UNSUPPORTED
    for key in ("beams", "vocab", "count"):
        assert beam(L, **{key: 0}) == INVALID
    assert beam(L, count=31) == INVALID and b"count" in L.mssm_last_error()
    assert beam(L, beams=33) == UNSUPPORTED
    assert beam(L, count=65, vocab=100) == UNSUPPORTED
    assert beam(L, batch=1 << 20, vocab=1 << 20) == UNSUPPORTED
    assert beam(L, batch=1 << 24, vocab=64) == UNSUPPORTED
    assert beam(L, batch=1 << 20, beams=16, vocab=64) == UNSUPPORTED


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0, 0.0])
def test_host_scalars(L, bad):
    for op in ("norm_fwd", "norm_bwd"):
        assert CALLS[op](L, base=bad) == INVALID
        if bad != 0.0:
            assert CALLS[op](L, eps=bad) == INVALID
    if bad not in (-1.0, 0.0):
        for op in ("attn_fwd", "attn_bwd", "attn_step"):
            assert CALLS[op](L, scale=bad) == INVALID


def test_empty_calls_need_no_gpu(L):
    for f, kw in [(norm_fwd, dict(tokens=0)), (norm_fwd, dict(q_heads=0, k_heads=0)), (attn_fwd, dict(heads=0)),
                  (attn_bwd, dict(heads=0)), (attn_step, dict(seqs=0)), (beam, dict(batch=0)),
                  (attn_fwd, dict(seqs=0)), (attn_fwd, dict(seqlen=0, h_last=None)), (attn_bwd, dict(seqlen=0, dh0=None))]:
        assert f(L, **kw) == _lib.MSSM_OK, (f, kw, L.mssm_last_error())
    assert norm_bwd(L, tokens=0, dq_weight=None, dk_weight=None) == _lib.MSSM_OK
    assert reorder(L, states=[], rows=[]) == _lib.MSSM_OK
    assert reorder(L, batch=0) == _lib.MSSM_OK


def test_state_reorder_refusals(L):
    assert reorder(L, origins=None) == INVALID and b"origins" in L.mssm_last_error()
    assert reorder(L, states=[fake(1), None]) == INVALID and b"states[1]" in L.mssm_last_error()
    assert reorder(L, rows=[32, -1]) == INVALID
    assert reorder(L, count=-1) == INVALID
    assert reorder(L, states=[fake(1), fake(1) + 64]) == INVALID and b"overlaps states[0]" in L.mssm_last_error()
    assert reorder(L, states=[fake(500), fake(64)]) == INVALID and b"origins" in L.mssm_last_error()
    assert reorder(L, beams=0) == INVALID
    assert reorder(L, beams=33) == UNSUPPORTED
    assert reorder(L, rows=[1 << 62, 8]) in (INVALID, UNSUPPORTED)
    assert reorder(L, rows=[1 << 39, 8], batch=1 << 10) == UNSUPPORTED
    n = ctypes.POINTER(ctypes.c_int64)()
    assert L.mssm_state_reorder((ctypes.c_void_p * 1)(fake(1)), n, 1, fake(9), _lib.BeamDims(1, 1, 1, 1), None) == INVALID
    p = ctypes.POINTER(ctypes.c_void_p)()
    assert L.mssm_state_reorder(p, (ctypes.c_int64 * 1)(4), 1, fake(9), _lib.BeamDims(1, 1, 1, 1), None) == INVALID


def queries(L, io):
    """(call, sizes, its workspace, an input to overlap) where one is needed."""
    dt = _lib.DTypes(io, 0)
    return [(norm_bwd, dict(tokens=300), L.mssm_qk_norm_rotary_bwd_workspace(_lib.HeadNormDims(300, 2, 3, 8, 6), dt), "q"),
            (attn_fwd, dict(seqlen=5000), L.mssm_linear_attention_workspace(_lib.AttentionDims(2, 5000, 10000, 3, 4, 6), dt, 0), "k"),
            (attn_bwd, dict(seqlen=5000), L.mssm_linear_attention_workspace(_lib.AttentionDims(2, 5000, 10000, 3, 4, 6), dt, 1), "d_o"),
            (beam, {}, L.mssm_beam_select_workspace(_lib.BeamDims(2, 3, 10, 4), dt), "logits")]


@pytest.mark.parametrize("io", [0, 1])
def test_workspace_refusals(L, io):
    for f, sizes, need, operand in queries(L, io):
        assert need > 0 and need % 4 == 0
        at = fake(1 << 20) // 256 * 256
        assert f(L, io=io, workspace=at, bytes=need - 1, **sizes) == INVALID and b"smaller" in L.mssm_last_error()
        assert f(L, io=io, workspace=at, bytes=-1, **sizes) == INVALID
        assert f(L, io=io, workspace=at + 16, bytes=need, **sizes) == INVALID and b"aligned" in L.mssm_last_error()
        assert f(L, io=io, workspace=at, bytes=need, **{operand: at}, **sizes) == INVALID
        assert b"overlap" in L.mssm_last_error()


def test_workspace_queries_refuse_what_the_calls_refuse(L):
    dt, bad = _lib.DTypes(0, 0), _lib.DTypes(7, 0)
    assert L.mssm_qk_norm_rotary_bwd_workspace(_lib.HeadNormDims(1, 1, 1, 300, 0), dt) == -1 and L.mssm_last_error()
    assert L.mssm_qk_norm_rotary_bwd_workspace(_lib.HeadNormDims(1, 1, 1, 8, 0), bad) == -1
    assert L.mssm_linear_attention_workspace(_lib.AttentionDims(1, 1, 1, 1, 300, 1), dt, 0) == -1
    assert L.mssm_linear_attention_workspace(_lib.AttentionDims(-1, 1, 1, 1, 3, 1), dt, 1) == -1
    assert L.mssm_linear_attention_workspace(_lib.AttentionDims(1, 0, 0, 1, 3, 1), dt, 1) == 0
    assert L.mssm_beam_select_workspace(_lib.BeamDims(1, 1, 3, 4), dt) == -1


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import selective_state_space_05_amd as mssm
    x, n = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, dtype=torch.int64)
    for f, args in [(mssm.qk_norm_rotary_fwd, (x, x, n)), (mssm.qk_norm_rotary_bwd, (x, x, x, x, n)),
                    (mssm.linear_attention_fwd, (x, x, x, torch.zeros(4))),
                    (mssm.linear_attention_bwd, (x, x, x, torch.zeros(4), x)),
                    (mssm.linear_attention_update, (x, x[0], x[0], x[0], torch.zeros(4))),
                    (mssm.beam_select, (x[0], x[0, 0])), (mssm.state_reorder, ([x], n))]:
        with pytest.raises(ValueError, match="GPU"):
            f(*args)
        with pytest.raises(TypeError):
            f(*([None] * len(args)))

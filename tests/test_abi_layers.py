"""Refusals of the layer-norm, gated-recurrence and cross-entropy entry points:
the C ABI rejects every invalid call before touching the HIP runtime, and the
binding rejects what the C ABI cannot see.  No GPU; pointers are fake non-null
addresses that validation never dereferences."""
from __future__ import annotations

import pytest

from selective_state_space_05_amd import _lib
from test_abi import L, fake  # noqa: F401  (L is the library fixture)

INVALID, UNSUPPORTED = _lib.MSSM_ERR_INVALID_ARG, _lib.MSSM_ERR_UNSUPPORTED


def call(L, fn, names, scalars, dims, io=0, param=0, **ptrs):
    p = {n: fake(2 * k + 1) for k, n in enumerate(names) if n not in scalars}
    p.update(scalars)
    p.update(ptrs)
    return getattr(L, "mssm_" + fn)(*[p[n] for n in names], dims, _lib.DTypes(io, param), None)


def norm_fwd(L, rows=4, dim=8, io=0, param=0, **kw):
    return call(L, "layer_norm_fwd", ["x", "weight", "bias", "eps", "y", "mean", "rstd"],
                dict(eps=kw.pop("eps", 1e-5)), _lib.NormDims(rows, dim), io, param, **kw)


def norm_bwd(L, rows=4, dim=8, io=0, param=0, **kw):
    return call(L, "layer_norm_bwd", ["dy", "x", "mean", "rstd", "weight", "dx", "dweight", "dbias", "workspace", "bytes"],
                dict(workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0)),
                _lib.NormDims(rows, dim), io, param, **kw)


def rec_fwd(L, batch=2, seqlen=5, dim=8, io=0, param=0, **kw):
    return call(L, "gated_recurrence_fwd", ["x", "r", "i", "lam", "scale", "h0", "y", "h_last", "workspace", "bytes"],
                dict(scale=kw.pop("scale", 8.0), workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0)), _lib.RecurrenceDims(batch, seqlen, dim), io, param, **kw)


def rec_bwd(L, batch=2, seqlen=5, dim=8, io=0, param=0, **kw):
    return call(L, "gated_recurrence_bwd",
                ["x", "r", "i", "lam", "scale", "h0", "y", "dy", "dh_last", "dx", "dr", "di", "dlam", "dh0",
                 "workspace", "bytes"],
                dict(scale=kw.pop("scale", 8.0), workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0)), _lib.RecurrenceDims(batch, seqlen, dim), io, param, **kw)


def rec_step(L, batch=2, seqlen=1, dim=8, io=0, param=0, **kw):
    return call(L, "gated_recurrence_update", ["state", "x", "r", "i", "lam", "scale", "y"],
                dict(scale=kw.pop("scale", 8.0)), _lib.RecurrenceDims(batch, seqlen, dim), io, param, **kw)


def loss_fwd(L, tokens=4, dim=8, vocab=10, io=0, param=0, **kw):
    return call(L, "linear_cross_entropy_fwd", ["hidden", "weight", "targets", "ignore", "loss", "lse", "workspace", "bytes"],
                dict(ignore=-100, workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0)), _lib.LossDims(tokens, dim, vocab), io, param, **kw)


def loss_bwd(L, tokens=4, dim=8, vocab=10, io=0, param=0, **kw):
    return call(L, "linear_cross_entropy_bwd",
                ["hidden", "weight", "targets", "ignore", "lse", "dloss", "dhidden", "dweight", "workspace", "bytes"],
                dict(ignore=-100, workspace=kw.pop("workspace", None), bytes=kw.pop("bytes", 0)), _lib.LossDims(tokens, dim, vocab), io, param, **kw)


CALLS = {"norm_fwd": norm_fwd, "norm_bwd": norm_bwd, "rec_fwd": rec_fwd, "rec_bwd": rec_bwd,
         "rec_step": rec_step, "loss_fwd": loss_fwd, "loss_bwd": loss_bwd}
REQUIRED = {"norm_fwd": ["x", "y"], "norm_bwd": ["dy", "x", "mean", "rstd", "dx"],
            "rec_fwd": ["x", "r", "i", "lam", "y"],
            "rec_bwd": ["x", "r", "i", "lam", "y", "dy", "dx", "dr", "di"],
            "rec_step": ["state", "x", "r", "i", "lam", "y"],
            "loss_fwd": ["hidden", "weight", "targets", "loss"],
            "loss_bwd": ["hidden", "weight", "targets", "lse", "dloss", "dhidden", "dweight"]}
# (output, overlapping operand)
OVERLAPS = {"norm_fwd": [("y", "x"), ("mean", "rstd"), ("y", "weight"), ("rstd", "bias")],
            "norm_bwd": [("dx", "dy"), ("dx", "x"), ("dweight", "dbias"), ("dbias", "weight"), ("dweight", "mean")],
            "rec_fwd": [("y", "x"), ("y", "r"), ("h_last", "lam"), ("y", "h_last"), ("y", "h0")],
            "rec_bwd": [("dx", "x"), ("dr", "di"), ("dlam", "lam"), ("dh0", "h0"), ("dh0", "dh_last"),
                        ("dx", "dy"), ("di", "y")],
            "rec_step": [("y", "x"), ("state", "x"), ("y", "state"), ("state", "lam")],
            "loss_fwd": [("loss", "lse"), ("loss", "targets"), ("lse", "hidden"), ("loss", "weight")],
            "loss_bwd": [("dhidden", "hidden"), ("dweight", "weight"), ("dhidden", "dweight"),
                         ("dweight", "lse"), ("dhidden", "dloss")]}


@pytest.mark.parametrize("op,name", [(o, n) for o in CALLS for n in REQUIRED[o]])
def test_null_required_pointer(L, op, name):
    assert CALLS[op](L, **{name: None}) == INVALID
    assert name.encode() in L.mssm_last_error()


@pytest.mark.parametrize("op,out,other", [(o, a, b) for o in CALLS for a, b in OVERLAPS[o]])
def test_overlap(L, op, out, other):
    at = fake(900)
    assert CALLS[op](L, **{out: at + 4, other: at}) == INVALID
    assert b"overlap" in L.mssm_last_error()


@pytest.mark.parametrize("op", CALLS)
def test_dtypes(L, op):
    assert CALLS[op](L, io=2) == INVALID
    assert CALLS[op](L, param=3) == INVALID
    assert CALLS[op](L, param=_lib.MSSM_BF16) == UNSUPPORTED


@pytest.mark.parametrize("op,key", [(o, k) for o in CALLS for k in
                                    (["rows", "dim"] if o.startswith("norm") else
                                     ["batch", "dim"] + (["seqlen"] if o != "rec_step" else [])
                                     if o.startswith("rec") else ["tokens", "dim", "vocab"])])
def test_negative_and_huge_sizes(L, op, key):
    assert CALLS[op](L, **{key: -1}) == INVALID
    assert CALLS[op](L, **{key: 1 << 40}) in (INVALID, UNSUPPORTED)
    assert L.mssm_last_error()


@pytest.mark.parametrize("op", ["loss_fwd", "loss_bwd"])
@pytest.mark.parametrize("key", ["dim", "vocab"])
def test_loss_needs_a_width_and_a_vocabulary(L, op, key):
    assert CALLS[op](L, **{key: 0}) == INVALID


@pytest.mark.parametrize("bad", [-1.0, float("nan"), float("inf")])
def test_host_scalars(L, bad):
    assert norm_fwd(L, eps=bad) == INVALID
    for op in ("rec_fwd", "rec_bwd", "rec_step"):
        assert CALLS[op](L, scale=bad) == INVALID


def test_empty_calls_need_no_gpu(L):
    for op, kw in [("norm_fwd", dict(rows=0)), ("norm_fwd", dict(dim=0)), ("norm_bwd", dict(dim=0)),
                   ("rec_fwd", dict(batch=0)), ("rec_fwd", dict(dim=0)), ("rec_step", dict(batch=0)),
                   ("loss_fwd", dict(tokens=0))]:
        assert CALLS[op](L, **kw) == _lib.MSSM_OK, (op, L.mssm_last_error())
    assert norm_bwd(L, rows=0, dweight=None, dbias=None) == _lib.MSSM_OK
    assert rec_bwd(L, batch=0, dlam=None, dh0=None) == _lib.MSSM_OK
    assert rec_fwd(L, seqlen=0, h_last=None) == _lib.MSSM_OK


def queries(L, io=0):
    """(call, sizes, its workspace, an input to overlap) where one is needed."""
    dt = _lib.DTypes(io, 0)
    return [(norm_bwd, dict(rows=300, dim=40), L.mssm_layer_norm_bwd_workspace(_lib.NormDims(300, 40), dt), "dy"),
            (rec_fwd, dict(seqlen=3000), L.mssm_gated_recurrence_workspace(_lib.RecurrenceDims(2, 3000, 8), dt, 0), "x"),
            (rec_bwd, dict(seqlen=3000), L.mssm_gated_recurrence_workspace(_lib.RecurrenceDims(2, 3000, 8), dt, 1), "y"),
            (loss_fwd, dict(tokens=40), L.mssm_linear_cross_entropy_workspace(_lib.LossDims(40, 8, 10), dt, 0, 1), "hidden"),
            (loss_bwd, dict(tokens=40), L.mssm_linear_cross_entropy_workspace(_lib.LossDims(40, 8, 10), dt, 1, 1), "weight")]


@pytest.mark.parametrize("io", [0, 1])
def test_workspace_refusals(L, io):
    for f, sizes, need, operand in queries(L, io):
        assert need > 0 and need % 4 == 0
        at = fake(800) // 256 * 256
        assert f(L, io=io, workspace=at, bytes=need - 1, **sizes) == INVALID and b"smaller" in L.mssm_last_error()
        assert f(L, io=io, workspace=at, bytes=-1, **sizes) == INVALID
        assert f(L, io=io, workspace=at + 16, bytes=need, **sizes) == INVALID and b"aligned" in L.mssm_last_error()
        assert f(L, io=io, workspace=at, bytes=need, **{operand: at}, **sizes) == INVALID
        assert b"overlap" in L.mssm_last_error()


def test_workspace_queries_refuse_what_the_calls_refuse(L):
    dt, bad = _lib.DTypes(0, 0), _lib.DTypes(7, 0)
    assert L.mssm_layer_norm_bwd_workspace(_lib.NormDims(-1, 4), dt) == -1 and L.mssm_last_error()
    assert L.mssm_layer_norm_bwd_workspace(_lib.NormDims(1, 4), bad) == -1
    assert L.mssm_gated_recurrence_workspace(_lib.RecurrenceDims(1, 1 << 40, 4), dt, 0) == -1
    assert L.mssm_gated_recurrence_workspace(_lib.RecurrenceDims(1, 9, 1 << 21), dt, 1) == -1
    assert L.mssm_linear_cross_entropy_workspace(_lib.LossDims(1, 0, 4), dt, 0, 1) == -1
    assert L.mssm_gated_recurrence_workspace(_lib.RecurrenceDims(1, 0, 4), dt, 1) == 0
    assert L.mssm_linear_cross_entropy_workspace(_lib.LossDims(0, 4, 4), dt, 1, 1) == 0


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import selective_state_space_05_amd as mssm
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="GPU"):
        mssm.layer_norm_fwd(x)
    with pytest.raises(ValueError, match="GPU"):
        mssm.gated_recurrence_fwd(x, x, x, torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        mssm.linear_cross_entropy_fwd(x[0], x[1], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        mssm.layer_norm_fwd(None)

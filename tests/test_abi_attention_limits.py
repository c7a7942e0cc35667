"""What the workspaces of the attention and beam-search entry points have room for, and
refusals at the edges of their ranges.  No GPU."""
from __future__ import annotations

import pytest

from selective_state_space_05_amd import _lib
from test_abi import L, fake  # noqa: F401  (L is the library fixture)
from test_abi_attention import attn_bwd, attn_fwd, beam, norm_fwd, reorder


@pytest.mark.parametrize("io", [0, 1])
def test_workspace_holds_a_state_for_every_segment(L, io):
    """256 steps of one head are two segments of 128.  Forward: a state in front of each,
    the first one's for a call whose h0 is its h_last; backward: two in front of the second."""
    dt, state = _lib.DTypes(io, 0), 2 * 3 * 16 * 24 * 4
    dims = _lib.AttentionDims(2, 256, 512, 3, 16, 24)
    assert L.mssm_linear_attention_workspace(dims, dt, 0) == 2 * state
    assert L.mssm_linear_attention_workspace(dims, dt, 1) == 2 * state
    at = fake(1 << 20) // 256 * 256
    assert attn_fwd(L, io=io, seqlen=256, heads=3, key=16, value=24, workspace=at, bytes=state) == _lib.MSSM_ERR_INVALID_ARG
    assert b"smaller" in L.mssm_last_error()
    one = _lib.AttentionDims(2, 100, 200, 3, 16, 24)                # one segment
    assert L.mssm_linear_attention_workspace(one, dt, 0) == 0


def test_selection_refuses_more_entries_than_its_second_launch_takes(L):
    """That launch has 512 threads an entry, and a launch is below 2^32 threads."""
    dt = _lib.DTypes(0, 0)
    assert L.mssm_beam_select_workspace(_lib.BeamDims((1 << 23) - 1, 1, 64, 4), dt) > 0
    for batch in (1 << 23, (1 << 24) - 1):
        assert beam(L, batch=batch, beams=1, vocab=64) == _lib.MSSM_ERR_UNSUPPORTED and b"batch" in L.mssm_last_error()
        assert L.mssm_beam_select_workspace(_lib.BeamDims(batch, 1, 64, 4), dt) == -1
    # the reordering's launch has 256 threads an entry and state
    assert reorder(L, batch=1 << 24, rows=[16, 16]) == _lib.MSSM_ERR_UNSUPPORTED
    assert reorder(L, batch=1 << 23, rows=[4097, 16]) == _lib.MSSM_ERR_UNSUPPORTED


@pytest.mark.parametrize("packed", [False, True])
def test_overlaps_are_refused_without_steps_too(L, packed):
    """What an empty sequence copies or clears may not lie on an input either."""
    at = fake(900)
    sizes = dict(seqlen=0, cu_seqlens=fake(950) if packed else None)
    for f, out, inputs in ((attn_fwd, "h_last", ["log_decay", "h0"]), (attn_bwd, "dh0", ["log_decay", "h0", "dh_last"])):
        for name in inputs + ["cu_seqlens"] * packed:
            assert f(L, **{**sizes, out: at + 4, name: at}) == _lib.MSSM_ERR_INVALID_ARG, (out, name)
            assert b"overlap" in L.mssm_last_error()
    assert attn_bwd(L, **sizes, dh0=at, dh_last=at) == _lib.MSSM_ERR_INVALID_ARG
    assert attn_bwd(L, **sizes, dh0=at, h0=at) == _lib.MSSM_ERR_INVALID_ARG
    assert attn_fwd(L, **sizes, h0=at, h_last=at) == _lib.MSSM_OK          # already there


def test_norm_refuses_what_its_indices_do_not_hold(L):
    for sizes in (dict(tokens=1, q_heads=1 << 23), dict(tokens=1, k_heads=1 << 23), dict(tokens=1 << 31, q_heads=0, k_heads=0),
                  dict(tokens=1 << 20, q_heads=1 << 11)):
        assert norm_fwd(L, **sizes) == _lib.MSSM_ERR_UNSUPPORTED, sizes


def test_binding_and_header_agree_on_the_most_candidates():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mssm.h")).read()
    assert int(re.search(r"#define MSSM_MAX_BEAM_COUNT (\d+)", src).group(1)) == _lib.MAX_BEAM_COUNT

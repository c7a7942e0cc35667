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

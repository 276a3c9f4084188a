"""What the serving calls' contracts say of rows, paths, memory and sizes that
no ordinary step reaches: nodes that are not there, whatever stands in their q;
indices that point outside; streams of the caller's; sizes beyond 32 bits."""
import pytest
import torch

import rope_period_truncated_b200 as wp
from test_gpu_tree import Case, _i32

pytestmark = pytest.mark.gpu

INF = float("inf")


def _unused(c, kind):
    """Writes into the q rows of nodes that are not there."""
    for b, n in enumerate(c.nodes):
        q = c.q[b, n:]
        q.zero_()
        if kind == "one":
            q[..., 5] = 3e38
        elif kind == "all":
            q[:] = 3e38
        elif kind == "inf":
            q[..., 0] = INF
        elif kind == "minus":
            q[..., 17] = -INF
        elif kind == "large":
            q.copy_(torch.linspace(-40, 40, q.numel()).reshape(q.shape))
        elif kind == "nan":
            q[:, ::2] = float("nan")


# few rows: a CTA per unit; whole units of a line of tiles; parts of units. Many rows: one split; several.
ABSENT = [(64, 4, 2, 5, [40, 0, 333, 128], [3, 1, 5, 2], 0),
          (128, 8, 2, 6, [100, 64, 5] * 40 + [700], [6, 2, 1] * 40 + [4], 16),
          (128, 8, 2, 8, [2500, 900, 1300], [7, 8, 1], 64),
          (64, 4, 1, 20, [120, 200], [11, 19], 0),
          (128, 8, 2, 21, [1500, 2300], [20, 3], 16)]


@pytest.mark.parametrize("kind", ["one", "all", "inf", "minus", "nan"])
@pytest.mark.parametrize("d,Hq,Hkv,T,lens,nodes,P", ABSENT)
def test_absent_nodes_are_zero(d, Hq, Hkv, T, lens, nodes, P, kind):
    """Whatever their q holds: a finite value whose products overflow, infinities, NaN."""
    c = Case(d + T, d, Hq, Hkv, T, lens, nodes, P, False)
    _unused(c, kind)
    o, lse = c.run([40, 2 ** 31 - 1, 300, 70] * (d // 64))
    for b, n in enumerate(nodes):
        assert (o[b, n:] == 0).all() and (lse[b, :, n:] == -INF).all(), f"sequence {b}"
        assert torch.isfinite(o[b, :n].float()).all() and torch.isfinite(lse[b, :, :n]).all(), f"sequence {b}"
    assert wp.wp_device_status() == 0

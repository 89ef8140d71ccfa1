"""Group norm with rows of no positions (GPU): they add nothing to the gradients of weight and bias, whatever eps is.

With eps = 0 such a row's 1 / sqrt(var + eps) is an infinity, which must stay in its place in ``stats``.
Tolerances as in test_groupnorm_gpu."""
import numpy as np
import pytest

import channel_oracle as ref
from gpu_helpers import say, torch_dev
from test_groupnorm_gpu import make, r64, run, within

pytestmark = pytest.mark.gpu


# B, L, C, groups, type, silu: groups that stay in a block's registers, and (the last three) groups that do not
@pytest.mark.parametrize("case", [
    (4, 60, 64, 4, "bf16", True), (3, 200, 32, 2, "f32", False), (5, 2000, 64, 2, "bf16", False),
    (3, 50, 30, 3, "f32", True), (2, 40, 7, 1, "bf16", False), (3, 3000, 128, 1, "f32", True),
], ids=str)
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rows_of_no_positions(case, eps):
    torch = torch_dev()
    B, L, C, groups, t, silu = case
    say("[gnorm] empty rows %s eps %g" % (case, eps))
    p = make(torch, B, L, C, t, t, seed=L)
    p["lengths"] = torch.full((B,), L, dtype=torch.int32, device="cuda")
    p["lengths"][0], p["lengths"][B - 1] = 0, L // 2
    if B > 3:
        p["lengths"][2] = -5
    exp = ref.groupnorm(r64(p["x"]), r64(p["w"]), r64(p["b"]), groups, float(np.float32(eps)), silu,
                        p["lengths"].cpu().numpy(), r64(p["dy"]))
    got = run(torch, p, groups, silu, lengths=True, eps=eps)
    for k in ("y", "dx", "dweight", "dbias"):
        within(k, got[k], exp[k])
    assert (got["dx"][0] == 0).all() and (got["y"][0] == 0).all()


@pytest.mark.parametrize("C,groups", [(64, 4), (30, 3)])
@pytest.mark.parametrize("L", [0, 9])
def test_no_positions_at_all(C, groups, L):
    torch = torch_dev()
    from selective_state_space_88_amd import scan

    say("[gnorm] no positions: %d channels, L %d" % (C, L))
    e = torch.full((3, L, C), 2.0, device="cuda")
    w = torch.ones(C, device="cuda")
    lengths = torch.zeros(3, dtype=torch.int32, device="cuda")
    stats = torch.full((3, groups, 3), 4.0, device="cuda")
    y = scan.groupnorm_fwd(e, w, groups=groups, eps=0.0, stats=stats, lengths=lengths)
    d = scan.groupnorm_bwd(e, e, w, stats, bias=w, groups=groups, lengths=lengths)
    torch.cuda.synchronize()
    assert (y == 0).all() and (d["dx"] == 0).all()
    assert (d["dweight"] == 0).all() and (d["dbias"] == 0).all()
    assert (stats[..., :2] == 0).all() and torch.isinf(stats[..., 2]).all()

"""Linear attention (GPU) with infinities and NaN in single tokens: what the recurrence keeps finite
stays finite and right (nothing flows back to earlier tokens, into other heads or other columns), and
what it makes infinite or NaN is not finite.

Bounds where finite: those of test_linattn_gpu.py, with the sums of absolute terms taken without the
token's non-finite features.
"""
import numpy as np
import pytest

import block_oracle as ref
from gpu_helpers import say, torch_dev
from test_linattn_gpu import H2, args64, make, run

pytestmark = pytest.mark.gpu


def check(torch, p, dtype, label):
    got = run(torch, p)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.linattn(*args64(p, True))
    clean = {n: (t.clone().nan_to_num(0.0, 0.0, 0.0) if t is not None and t.is_floating_point() and n != "log_decay"
                 else t) for n, t in p.items() if n != "scale"}
    mag = ref.linattn_scale(*args64(clean, True))
    K, V, L = p["q"].shape[-1], p["v"].shape[-1], p["q"].shape[1]
    bad = []
    for n in want:
        y, w, m = got[n].double().cpu().numpy(), want[n], mag[n]
        live = np.isfinite(w)
        tol = (K + V + 3 * L + 32) * 2.0 ** -24 * m
        if dtype == "bf16":
            tol = tol + (2.0 ** -24 * m if n in ("s_final", "ds_init") else 2.0 ** -14 * m)
        if dtype == "bf16" and n not in ("s_final", "ds_init"):
            tol = tol + H2 * np.abs(np.where(live, w, 0)) * (1 + 2.0 ** -6)
        off = np.abs(np.where(live, y - np.where(live, w, 0), 0))
        if np.isfinite(y[~live]).any():
            bad.append("%s: %d of %d non-finite values came out finite" % (n, np.isfinite(y[~live]).sum(), (~live).sum()))
        if not (off <= tol + 1e-30).all():
            bad.append("%s: %d of %d finite values are wrong, %d of them not finite" % (
                n, (~(off <= tol + 1e-30)).sum(), live.sum(), (~np.isfinite(y[live])).sum()))
    say("[linattn] non-finite %s %s: %s" % (label, dtype, bad or "as the recurrence"))
    assert not bad, bad


WHERE = [("v", 40, 5), ("v", 0, 0), ("v", 99, 30), ("k", 40, 3), ("k", 63, 0), ("q", 17, 2), ("do", 70, 11), ("do", 5, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", WHERE, ids=str)
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("V", [48, 128])
def test_one_feature_of_one_token(dtype, where, value, V):
    torch = torch_dev()
    name, t, e = where
    p = make(torch, 9, 2, 100, 3, 3, 3, 3, 24, V, dtype, state=True, decay=[-0.01, -0.2, 0.0])
    p[name][1, t, 1, e] = float(value)
    check(torch, p, dtype, "%s %s V=%d" % (where, value, V))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (200, 40), (40, 200)])
def test_in_a_long_row(dtype, K, V):
    """A row that is cut into segments: later segments' states carry it, earlier ones' do not."""
    torch = torch_dev()
    p = make(torch, 10, 1, 700, 2, 2, 2, 2, K, V, dtype, state=True, decay=[-0.01, -0.03])
    p["v"][0, 333, 1, 7] = float("nan")
    p["do"][0, 400, 0, 9] = float("inf")
    check(torch, p, dtype, "long row")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_feature_reads_it(dtype):
    """Shared heads: a NaN in a shared value head reaches the heads that share it only."""
    torch = torch_dev()
    p = make(torch, 11, 2, 70, 4, 4, 2, 2, 16, 32, dtype, state=True, decay=[-0.01, -0.02, -0.04, -0.08])
    p["v"][0, 66, 1, 0] = float("nan")
    check(torch, p, dtype, "shared heads")

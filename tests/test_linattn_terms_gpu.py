"""Linear attention (GPU): products keep f32 accuracy relative to their terms, also where the terms
cancel.  bf16 inputs are exact and the state is f32, so what is left when two terms of opposite sign
meet is right to the roundings of f32, and the output is rounded once.

Bound, per output, in half-steps of f32 (U) of the sum of absolute terms: a score is a sum of K
products (K), the decay's power is off by 3 and meets two scales (2); the weighted value or score is
split without loss and its products are added (3 parts, one rounding each, and the addition of the two
terms: 4); a state passes 4 a chunk, is read in K products (K) and scaled (2); the end.  In all
(2 K + 16 + 4 chunks) U, chunks = ceil(L / 32) + 1; a bf16 output 2^-8 of itself on top.
"""
import numpy as np
import pytest

import block_oracle as ref
from gpu_helpers import say, torch_dev
from test_linattn_gpu import args64, make, run

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DECAYS = [-2.0 ** -12, -2.0 ** -9, -0.002, -0.01]


def check(label, got, p, dtype):
    K, L = p["q"].shape[-1], p["q"].shape[1]
    want, mag = ref.linattn(*args64(p, True)), ref.linattn_scale(*args64(p, True))
    bound = (2 * K + 16 + 4 * (-(-L // 32) + 1)) * U
    ratios = {}
    for n in want:
        tol = bound * mag[n] + 1e-30
        if dtype == "bf16" and n not in ("s_final", "ds_init"):
            tol = tol + 2.0 ** -8 * np.abs(want[n])
        y = got[n].double().cpu().numpy()
        ratios[n] = float((np.abs(y - want[n]) / tol).max())
    say("[linattn] %s %s: of the bound %s" % (label, dtype, {n: round(r, 3) for n, r in ratios.items()}))
    assert max(ratios.values()) <= 1, ratios


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L", [(16, 2), (16, 40), (16, 65), (16, 130), (1, 400)])
@pytest.mark.parametrize("V", [48, 128])
def test_two_tokens_cancel(dtype, B, L, V):
    """Two tokens with one key and opposite values, read (and, for the gradients, fed back) by the last
    two tokens with one query and opposite gradients: what is left is the decay between neighbours."""
    torch = torch_dev()
    p = make(torch, 3 + L, B, L, 4, 4, 4, 4, 8, V, dtype, decay=DECAYS)
    last = max(L - 2, 0)
    for n, live in (("k", (0, 1)), ("v", (0, 1)), ("q", (last, L - 1)), ("do", (last, L - 1))):
        x = p[n].clone()
        p[n].zero_()
        first, second = live
        p[n][:, first] = x[:, first]
        p[n][:, second] = -x[:, first] if n in ("v", "do") else x[:, first]
    check("two tokens %d x %d, V = %d" % (B, L, V), run(torch, p), p, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [48, 128])
def test_two_rows_of_the_state_cancel(dtype, V):
    """A state whose first two rows are nearly opposite, read by a query that adds them; the gradient's
    state alike, read by the keys (dv) and, for its first two columns, by the values (dk)."""
    torch = torch_dev()
    p = make(torch, 5, 16, 3, 4, 4, 4, 4, 8, V, dtype, state=True, decay=DECAYS)
    for n in ("q", "k", "v", "do"):
        p[n].zero_()
    p["q"][..., :2] = 1.5
    p["k"][..., :2] = 0.75
    p["do"][..., :2] = 1.25
    p["v"][..., :2] = 0.5
    for s in ("s_init", "ds_final"):
        x = p[s]
        x[:, :, 2:] = 0
        x[:, :, 1] = -x[:, :, 0] * (1 + 2.0 ** -15)
        x[..., 1] = -x[..., 0] * (1 + 2.0 ** -14)
    check("two rows, V = %d" % V, run(torch, p), p, dtype)

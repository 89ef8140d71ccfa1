"""Linear attention (GPU) where a bound by the sum of absolute terms says nothing: what is left of a
decayed state, element by element, against the float64 recurrence.
"""
import numpy as np
import pytest

from gpu_helpers import say, torch_dev
from test_linattn_gpu import args64, dev, make, run

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of f32


def worst(got, want, tol):
    """Largest |got - want| / tol over the elements; every one of them finite."""
    y = got.double().cpu().numpy()
    assert np.isfinite(y).all()
    return float((np.abs(y - want) / tol).max())


# ------------------------------------------------------------------ what is left of a decayed state

# from hardly any decay to e^-80 over the row, on both sides of lam = 1/2 for a token and for a chunk
DECAYS = [0.0, -2.0 ** -14, -0.003, -0.01, -0.0108, -0.011, -0.021, -0.022, -0.05, -0.1, -0.15, -0.2, -0.25, -0.5]
# tokens; a walk of several chunks (f32: 32, bf16: 64), rows cut into segments, lengths that end inside
# a chunk; batches that fill the chip (not cut)
LEFT = [(1, 1, 1), (1, 33, 1), (1, 64, 1), (2, 150, 1), (1, 300, 1), (120, 150, 1), (2, 100, 3)]


@pytest.mark.parametrize("case", LEFT, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_a_decay_leaves(case, dtype):
    """Tokens whose keys (whose queries, for the gradient) are zero add nothing, so the state after L of
    them is lam^L s_init, and o_t = scale lam^(t+1) q_t . s_init; the gradient's state alike.  To a few
    roundings of the value itself: a factor is off by 3 U at most (exp or expm1 and one addition) and its
    product by one more, 4 U for every chunk of at least 32 tokens or segment of at least 64, below
    (3 (L / 32 + L / 64 + 2) + 8) U.  One feature of q is not zero, so o has one term."""
    torch = torch_dev()
    B, L, seed = case
    H, K, V = len(DECAYS), 24, 40
    p = make(torch, seed, B, L, H, H, H, H, K, V, dtype, state=True, decay=DECAYS)
    for n in ("k", "q"):
        p[n].zero_()
    want_state = lambda s: np.exp(np.array(DECAYS, dtype=np.float32).astype(np.float64) * L)[None, :, None, None] * s
    tol = (3 * (L // 32 + L // 64 + 2) + 8) * U
    got = run(torch, p)
    for name, s in (("s_final", "s_init"), ("ds_init", "ds_final")):
        want = want_state(p[s].double().numpy())
        w = worst(got[name], want, tol * np.abs(want) + 1e-36)
        say("[linattn] left %s %s %s: worst %.3f of the tolerance" % (case, dtype, name, w))
        assert w <= 1, (case, name, w)
    # read by one feature
    p["q"][..., 3] = 1.5
    got = run(torch, p, grads=False)
    t = np.arange(1, L + 1)
    lam = np.exp(np.array(DECAYS, dtype=np.float32).astype(np.float64)[None, :] * t[:, None])   # [L, H]
    want = 0.25 * 1.5 * lam[None, :, :, None] * p["s_init"].double().numpy()[:, None, :, 3]
    # two factors more (scale, and the state's parts in bf16: 2 U), one rounding of the output
    tol_o = (tol + 8 * U + (2.0 ** -8 if dtype == "bf16" else 0)) * np.abs(want) + 1e-36
    w = worst(got["o"], want, tol_o)
    say("[linattn] left %s %s o: worst %.3f of the tolerance" % (case, dtype, w))
    assert w <= 1, (case, w)


@pytest.mark.parametrize("V", [40, 64, 7])
def test_what_a_decay_leaves_of_a_step(V):
    """The same for one token: exp and one product, 4 half-steps of the value."""
    torch = torch_dev()
    from selective_state_space_88_amd import scan

    decays = DECAYS + [-0.6931, -0.6932, -1.0, -5.0, -10.0, -16.0, -20.0, -40.0, -80.0]
    H, K = len(decays), 33
    p = make(torch, 2, 3, 1, H, H, H, H, K, V, "f32", state=True, decay=decays)
    d = dev(p)
    d["k"].zero_()
    q = torch.zeros_like(d["q"][:, 0])
    q[..., 5] = 2.0
    out = torch.empty_like(d["s_init"])
    o = scan.linattn_step(q, d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["s_init"], scale=0.5, s_out=out)
    torch.cuda.synchronize()
    lam = np.exp(np.array(decays, dtype=np.float32).astype(np.float64))
    want = lam[None, :, None, None] * p["s_init"].double().numpy()
    w = worst(out, want, 4 * U * np.abs(want) + 1e-40)
    wo = worst(o, want[:, :, 5], 6 * U * np.abs(want[:, :, 5]) + 1e-40)
    say("[linattn] left of a step: worst %.3f, o %.3f of the tolerance" % (w, wo))
    assert w <= 1 and wo <= 1, (w, wo)

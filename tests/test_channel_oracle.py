"""The 64-bit references of the gated recurrence and the group norm against differences (CPU)."""
import numpy as np
import pytest

import channel_oracle as ref


def slope(f, v, at, e):
    p, q = v.copy(), v.copy()
    p[at] += e
    q[at] -= e
    return (f(p) - f(q)) / (2 * e)


@pytest.mark.parametrize("mix", ["none", "leak", "unit"])
@pytest.mark.parametrize("with_rate", [False, True])
def test_gatedrec_gradients(mix, with_rate):
    r = np.random.default_rng(5)
    B, L, C = 2, 19, 3
    x, g, i, dh = (r.standard_normal((B, L, C)) for _ in range(4))
    rate = 0.05 + r.random(C) if with_rate else None
    lengths, starts = np.array([19, 11]), (r.random((B, L)) < 0.15).astype(np.int32)
    s0, ds = r.standard_normal((B, C)), r.standard_normal((B, C))

    def loss(x=x, g=g, i=i, rate=rate, s0=s0):
        o = ref.gatedrec(x, g, i, rate, mix, lengths, starts, s0)
        return (o["h"][0] * dh).sum() + (o["s_final"][0] * ds).sum()

    got = ref.gatedrec(x, g, i, rate, mix, lengths, starts, s0, dh, ds)
    # central differences: an error of e^2 (1e-10) and 1e-16 / e times the loss
    for name, v, d in (("x", x, "dx"), ("g", g, "dg"), ("i", i, "di"), ("rate", rate, "drate"), ("s0", s0, "ds_init")):
        if v is None:
            continue
        for k in r.choice(v.size, min(v.size, 12), replace=False):
            at = np.unravel_index(k, v.shape)
            want = slope(lambda q: loss(**{name: q}), v, at, 1e-5)
            assert abs(got[d][0][at] - want) < 1e-7 * (1 + abs(want)), (name, at)
    assert (got["dx"][0][1, 11:] == 0).all() and (got["h"][0][1, 11:] == 0).all()


@pytest.mark.parametrize("silu", [False, True])
def test_groupnorm_gradients(silu):
    r = np.random.default_rng(6)
    B, L, C, G = 2, 9, 6, 2
    x, dy = r.standard_normal((B, L, C)) + 1, r.standard_normal((B, L, C))
    w, bias = 1 + 0.3 * r.standard_normal(C), r.standard_normal(C)
    lengths = np.array([9, 5])

    def loss(x=x, w=w, bias=bias):
        return (ref.groupnorm(x, w, bias, G, 1e-5, silu, lengths)["y"][0] * dy).sum()

    got = ref.groupnorm(x, w, bias, G, 1e-5, silu, lengths, dy)
    for name, v, d in (("x", x, "dx"), ("w", w, "dweight"), ("bias", bias, "dbias")):
        for k in r.choice(v.size, min(v.size, 12), replace=False):
            at = np.unravel_index(k, v.shape)
            want = slope(lambda q: loss(**{name: q}), v, at, 1e-5)
            assert abs(got[d][0][at] - want) < 1e-7 * (1 + abs(want)), (name, at)
    one = ref.groupnorm(x[:, :1, :1], w[:1], bias[:1], 1, 1e-5, silu, None, dy[:, :1, :1])
    assert (one["dx"][0] == 0).all()

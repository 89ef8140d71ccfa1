"""Group norm over bf16 values that are nearly all equal (GPU): the deviation of a group may be far below the spacing
of its values, and what the mean's rounding to f32 left is then as large as the deviations themselves.

Bounds, with u = 2^-24, for the f32 arithmetic of a first mean m and the deviations around it: m is a sum of f32
values off by at most 150 u |mean|, the values' deviations from it are exact, or rounded by u of themselves, and the
rest of the mean is their sum: off by 150 u of their mean size, which is mean |c| + |m - mean| at most.  The
variance is the mean of their squares (150 u) less the rest's square: off by 155 u (var + (m - mean)^2)."""
import numpy as np
import pytest

from gpu_helpers import say, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def reference(x, dy, w, groups, eps):
    B, L, C = x.shape
    xg = x.reshape(B, L, groups, C // groups)
    mean = xg.mean((1, 3), keepdims=True)
    c = xg - mean
    var = (c * c).mean((1, 3), keepdims=True)
    inv = 1 / np.sqrt(var + eps)
    first = 150 * U * np.abs(mean)
    off_mean = 150 * U * (np.abs(c).mean((1, 3), keepdims=True) + first) + 2.0 ** -47 * np.abs(mean)
    rel = 0.5 * 155 * U * (var + first ** 2) / (var + eps) + 4 * U
    flat = lambda v: np.broadcast_to(v, xg.shape).reshape(B, L, C)
    n = flat(c * inv)
    off_n = flat(inv * (off_mean + 3 * U * np.abs(c))) + np.abs(n) * flat(rel)
    out = dict(y=(n * w, np.abs(w) * off_n + 4 * U * np.abs(n * w)))
    out["dbias"] = (dy.sum((0, 1)), 150 * U * np.abs(dy).sum((0, 1)))
    off_w = np.abs(dy) * off_n + 150 * U * np.abs(dy * n)
    out["dweight"] = ((dy * n).sum((0, 1)), off_w.sum((0, 1)))
    d = dy * w
    of = lambda v: flat(v.reshape(xg.shape).mean((1, 3), keepdims=True))
    m0, m1 = of(d), of(d * n)
    off0, off1 = of(152 * U * np.abs(d)), of(np.abs(d) * off_n + 152 * U * np.abs(d * n))
    size = np.abs(d) + np.abs(m0) + np.abs(n * m1)
    iv = flat(inv)
    out["dx"] = (iv * (d - m0 - n * m1),
                 iv * (2 * U * np.abs(d) + off0 + np.abs(n) * off1 + off_n * np.abs(m1) + 5 * U * size) + flat(rel) * iv * size)
    return out


def within(name, got, want):
    value, bound = want
    y = got.double().cpu().numpy()
    tol = bound + np.abs(value) * (2.0 ** -8 if got.element_size() == 2 else 2.0 ** -24) + 1e-30
    d = np.abs(y - value)
    say("[gnorm] %s: worst %.3f of the tolerance" % (name, float((d / tol).max())))
    assert np.isfinite(y).all() and (d <= tol).all(), name


# L, C, groups (the last one too large for a block's registers), the common value and the other ones
@pytest.mark.parametrize("L,C,groups", [(4096, 32, 2), (300, 64, 2), (1024, 128, 2), (20000, 16, 1)])
@pytest.mark.parametrize("common,other", [(3008.0, 3024.0), (1.0, 1.0078125), (-200.0, 40.0)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_nearly_constant(L, C, groups, common, other, out):
    torch = torch_dev()
    from selective_state_space_88_amd import scan

    say("[gnorm] %d x %d, %d groups: %g and %g, %s" % (L, C, groups, common, other, out))
    gen = torch.Generator().manual_seed(L)
    x = torch.full((2, L, C), common)
    size = C // groups
    for b in range(2):
        for g in range(groups):
            for k in range(1 + 2 * b):   # one value of each group is another one, or three
                x[b, (7 + 31 * k + g) % L, g * size + (k + g) % size] = other
    x = x.to(torch.bfloat16)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[out]
    dy = torch.randn(2, L, C, generator=gen).to(dt)
    w = 1 + 0.3 * torch.randn(C, generator=gen)
    exp = reference(x.double().numpy(), dy.double().numpy(), w.double().numpy(), groups, float(np.float32(1e-5)))
    x, dy, w = x.cuda(), dy.cuda(), w.cuda()
    stats = torch.empty(2, groups, 3, device="cuda")
    y = scan.groupnorm_fwd(x, w, groups=groups, stats=stats, out_dtype=dt)
    d = scan.groupnorm_bwd(dy, x, w, stats, bias=w, groups=groups)
    torch.cuda.synchronize()
    within("y", y, exp["y"])
    for k in ("dx", "dweight", "dbias"):
        within(k, d[k], exp[k])

"""64-bit references of the gated linear recurrence and the group norm, on the CPU in numpy, each with a
bound on what f32 arithmetic may add.

Written from the definitions: the recurrence and its gradient token by token, the norm over a row's
positions at once.  Bounds, with u = 2^-24 (a rounding to nearest) and the hardware exp2, reciprocal and
square root at 2 u:

  sigmoid(z): the exponent's rounding |z| u, exp2 2 u, the sum u, the reciprocal 2 u: (|z| + 5) u, and
  (2 |z| + 8) u for 1 - sigmoid formed as e sigmoid.  With a rate, l = -rate sigmoid(g) is off by
  (|g| + 6) u; 1 - e^l by the polynomial's seven roundings and 5e-8 < u more, or, from 1 - e^l >= 0.22
  on, by the sum's (3 u of at most 1) / 0.22 < 14 u: gate = (2 |g| + 30) u covers every form.
  So a is off by gate min(1 - a, a (1 + |l|)): its 1 - a and itself are both that exact.
  b = w s x: gate + (|i| + 13) u of its size.
  The recurrence: every token adds at most 3 u of the sum of its terms' sizes (the rounded a, the sum, the
  join of pieces), and what is there passes on times a.

The gradients follow the same rules through the chain rule's products.
"""
import numpy as np

U = 2.0 ** -24


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def gates(g, i, rate, mix):
    """a, 1 - a, w, s, sigmoid(g) and the gate's bound, each [B, L, C]."""
    sg = sigmoid(g)
    if rate is None:
        a, m, size = sg, sigmoid(-g), 1.0
    else:
        log_a = -rate * sg
        a, m, size = np.exp(log_a), -np.expm1(log_a), 1.0 + np.abs(log_a)
    w = np.ones_like(a) if mix == "none" else m if mix == "leak" else np.sqrt(m * (2.0 - m))
    s = np.ones_like(a) if i is None else sigmoid(i)
    gate = (2 * np.abs(g) + 30) * U
    return a, m, w, s, sg, gate, gate * np.minimum(m, a * size)


def gatedrec(x, g, i=None, rate=None, mix="none", lengths=None, starts=None, s_init=None, dh=None, ds_final=None):
    """Dict of name -> (value, bound): h, s_final, marks and, with dh, dx, dg, di, drate, ds_init."""
    B, L, C = x.shape
    a, m, w, s, sg, gate, off_a = gates(g, i, rate, mix)
    size_i = 0.0 if i is None else np.abs(i)
    b = w * s * x
    off_b = np.abs(b) * (gate + (size_i + 13) * U)
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    fresh = np.zeros((B, L), bool) if starts is None else starts != 0
    h, off_h = np.zeros((B, L, C)), np.zeros((B, L, C))
    before, off_before = np.zeros((B, L, C)), np.zeros((B, L, C))
    marks, off_marks = np.zeros((B, -(-L // 16), C)), np.zeros((B, -(-L // 16), C))
    state = np.zeros((B, C)) if s_init is None else s_init.astype(np.float64).copy()
    off, size = np.zeros((B, C)), np.abs(state)
    for t in range(L):
        live = (t < n)[:, None]
        if t % 16 == 0:
            marks[:, t // 16], off_marks[:, t // 16] = state, off
        f = fresh[:, t, None]
        prev, off_prev, size_prev = (np.where(f, 0.0, v) for v in (state, off, size))
        before[:, t], off_before[:, t] = prev, off_prev
        new = a[:, t] * prev + b[:, t]
        new_size = a[:, t] * size_prev + np.abs(b[:, t])
        new_off = a[:, t] * off_prev + off_a[:, t] * size_prev + off_b[:, t] + 3 * U * new_size
        h[:, t], off_h[:, t] = np.where(live, new, 0.0), np.where(live, new_off, 0.0)
        state, off, size = (np.where(live, p, q) for p, q in ((new, state), (new_off, off), (new_size, size)))
    out = dict(h=(h, off_h), s_final=(state, off), marks=(marks, off_marks))
    if dh is None:
        return out
    D = np.zeros((B, C)) if ds_final is None else ds_final.astype(np.float64).copy()
    off, size = np.zeros((B, C)), np.abs(D)
    G, off_G = np.zeros((B, L, C)), np.zeros((B, L, C))
    for t in range(L - 1, -1, -1):
        live = (t < n)[:, None]
        new = dh[:, t] + D
        new_size = np.abs(dh[:, t]) + size
        new_off = off + 3 * U * new_size
        G[:, t], off_G[:, t] = np.where(live, new, 0.0), np.where(live, new_off, 0.0)
        f = fresh[:, t, None]
        D2, off2, size2 = (np.where(f, 0.0, v) for v in (a[:, t] * new, a[:, t] * new_off + off_a[:, t] * new_size,
                                                         a[:, t] * new_size))
        D, off, size = (np.where(live, p, q) for p, q in ((D2, D), (off2, off), (size2, size)))
    out["ds_init"] = (D, off)
    gs = gate + (size_i + 16) * U           # every product of w, s and their slopes
    aG = np.abs(G)
    out["dx"] = (G * w * s, off_G * w * s + aG * w * s * gs)
    slope = s * (1.0 - s) if i is None else s * sigmoid(-i)
    out["di"] = (G * w * x * slope, (off_G + aG * 2 * gs) * np.abs(w * x * slope))
    with np.errstate(divide="ignore", invalid="ignore"):
        dw = np.zeros_like(a) if mix == "none" else -np.ones_like(a) if mix == "leak" else np.where(w > 0, -a / w, 0.0)
    part = s * x * dw
    to_a = before + part
    off_to_a = off_before + np.abs(part) * 2 * gs + 2 * U * (np.abs(before) + np.abs(part))
    da = G * to_a
    off_da = off_G * np.abs(to_a) + aG * off_to_a
    if rate is None:
        k = a * m
        out["dg"] = (da * k, (off_da + np.abs(da) * 2 * gs) * k)
    else:
        k = a * rate * sg * sigmoid(-g)
        out["dg"] = (-da * k, (off_da + np.abs(da) * 3 * gs) * k)
        each, off_each = da * a * sg, (off_da + np.abs(da) * 3 * gs) * a * sg
        rows = B * L
        out["drate"] = (-each.sum((0, 1)), off_each.sum((0, 1)) + min(rows, 4096) * U * np.abs(each).sum((0, 1)))
    return out


def groupnorm(x, w, bias, groups, eps, silu, lengths=None, dy=None):
    """Dict of name -> (value, bound): y, mean, inv and, with dy, dx, dweight, dbias.

    Sums: at most 64 + 32 f32 additions around a value K of the channel (the rest in 64 bits), or, where a
    group stays on chip, 128 + 22 around its mean; K is off the mean by at most the largest deviation d: the
    mean is off by 150 u (mean |x - m| + d), the variance by 450 u (std + d)^2."""
    B, L, C = x.shape
    S = C // groups
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    z = lambda: np.zeros((B, L, C))
    out = dict(y=(z(), z()), mean=(np.zeros((B, groups)), np.zeros((B, groups))),
               inv=(np.full((B, groups), 1 / np.sqrt(eps) if eps else np.inf), np.full((B, groups), 0.0)))
    if dy is not None:
        out.update(dx=(z(), z()), dweight=(np.zeros(C), np.zeros(C)), dbias=(np.zeros(C), np.zeros(C)))
    bb = np.zeros(C) if bias is None else bias
    for b in range(B):
        N = n[b] * S
        if N == 0:
            continue
        xg = x[b, :n[b]].reshape(n[b], groups, S)
        mean = xg.mean((0, 2), keepdims=True)
        c = xg - mean
        var = (c * c).mean((0, 2), keepdims=True)
        inv = 1.0 / np.sqrt(var + eps)
        d = np.abs(c).max((0, 2), keepdims=True)
        off_mean = 150 * U * (np.abs(c).mean((0, 2), keepdims=True) + d)
        rel = 225 * U * (np.sqrt(var) + d) ** 2 / (var + eps) + 4 * U
        unit = c * inv
        off_n = inv * (off_mean + 3 * U * np.abs(c)) + np.abs(unit) * rel
        flat = lambda v: np.broadcast_to(v, (n[b], groups, S)).reshape(n[b], C)
        unit, off_n = flat(unit), flat(off_n)
        u = unit * w + bb
        off_u = np.abs(w) * off_n + 4 * U * (np.abs(unit * w) + np.abs(bb))
        sg = sigmoid(u)
        y = u * sg if silu else u
        out["y"][0][b, :n[b]] = y
        out["y"][1][b, :n[b]] = 1.1 * off_u + (np.abs(y) * (np.abs(u) + 8) * U if silu else 0)
        out["mean"][0][b], out["mean"][1][b] = mean[0, :, 0], off_mean[0, :, 0] + 2.0 ** -47 * np.abs(mean[0, :, 0])
        out["inv"][0][b], out["inv"][1][b] = inv[0, :, 0], (inv * rel)[0, :, 0]
        if dy is None:
            continue
        g = dy[b, :n[b]]
        du, off_du = g.copy(), np.zeros_like(g)
        if silu:
            act = sg + u * sg * sigmoid(-u)
            du = g * act
            # the slope's own slope is at most 1/2; its terms sg, u sg (1 - sg) round with the sigmoid
            off_du = np.abs(g) * (0.5 * off_u + (np.abs(act) + 1) * (np.abs(u) + 12) * U)
        out["dbias"][0][:] += du.sum(0)
        out["dbias"][1][:] += (off_du + 150 * U * np.abs(du)).sum(0)
        out["dweight"][0][:] += (du * unit).sum(0)
        off_w = off_du * np.abs(unit) + np.abs(du) * off_n + 150 * U * np.abs(du * unit)
        out["dweight"][1][:] += off_w.sum(0)
        dn, off_dn = du * w, off_du * np.abs(w) + 2 * U * np.abs(du * w)
        mean_of = lambda v: flat(v.reshape(n[b], groups, S).mean((0, 2), keepdims=True))
        m0, m1 = mean_of(dn), mean_of(dn * unit)
        off0 = mean_of(off_dn + 150 * U * np.abs(dn))
        off1 = mean_of(off_dn * np.abs(unit) + np.abs(dn) * off_n + 150 * U * np.abs(dn * unit))
        iv = flat(inv)
        size = np.abs(dn) + np.abs(m0) + np.abs(unit * m1)
        out["dx"][0][b, :n[b]] = iv * (dn - m0 - unit * m1)
        out["dx"][1][b, :n[b]] = iv * (off_dn + off0 + np.abs(unit) * off1 + off_n * np.abs(m1) + 5 * U * size) + \
            flat(rel) * iv * size
    return out

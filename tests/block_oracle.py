"""64-bit references of linear attention, rotary positions and the norms, on the CPU in numpy.

Written from the definitions: the recurrence token by token, the rotation as a complex product,
the gradients by the chain rule.  ``linattn`` also returns, for each output, the sum of the
absolute values of its terms: the scale of its rounding errors.
"""
import numpy as np


def heads_of(x, H):
    """[B, L, heads, D] -> [B, L, H, D], head h reading h // (H // heads)."""
    return np.repeat(x, H // x.shape[2], axis=2)


def share(dx, heads):
    B, L, H, D = dx.shape
    return dx.reshape(B, L, heads, H // heads, D).sum(3)


def linattn(q, k, v, log_decay, scale, lengths=None, s_init=None, do=None, ds_final=None):
    """Dict of o, s_final and (with do) dq, dk, dv, ds_init in float64; absent inputs are None."""
    B, L, Hq, K = q.shape
    H, V = log_decay.shape[0], v.shape[-1]
    Hk, Hv = k.shape[2], v.shape[2]
    with np.errstate(over="ignore"):
        lam = np.exp(log_decay.astype(np.float64))
    q, k, v = heads_of(q, H), heads_of(k, H), heads_of(v, H)
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    o = np.zeros((B, L, H, V))
    s_final = np.zeros((B, H, K, V))
    grads = do is not None
    dq, dk, dv = np.zeros((B, L, H, K)), np.zeros((B, L, H, K)), np.zeros((B, L, H, V))
    ds_init = np.zeros((B, H, K, V))
    for b in range(B):
        S = np.zeros((H, K, V)) if s_init is None else s_init[b].astype(np.float64).copy()
        for t in range(n[b]):
            S = lam[:, None, None] * S + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], S)
            if grads:
                dq[b, t] = scale * np.einsum("hkv,hv->hk", S, do[b, t])
        s_final[b] = S
        if grads:
            G = np.zeros((H, K, V)) if ds_final is None else ds_final[b].astype(np.float64).copy()
            for t in range(n[b] - 1, -1, -1):
                G = G + scale * q[b, t, :, :, None] * do[b, t, :, None, :]
                dk[b, t] = np.einsum("hkv,hv->hk", G, v[b, t])
                dv[b, t] = np.einsum("hkv,hk->hv", G, k[b, t])
                G = lam[:, None, None] * G
            ds_init[b] = G
    out = dict(o=o, s_final=s_final)
    if grads:
        out.update(dq=share(dq, Hq), dk=share(dk, Hk), dv=share(dv, Hv), ds_init=ds_init)
    return out


def linattn_scale(q, k, v, log_decay, scale, lengths=None, s_init=None, do=None, ds_final=None):
    """linattn on absolute values: what its rounding errors are relative to."""
    a = lambda x: None if x is None else np.abs(x)
    return linattn(a(q), a(k), a(v), log_decay, abs(scale), lengths, a(s_init), a(do), a(ds_final))


def rope(x, pos, inv_freq, amp=1.0, interleaved=False, inverse=False):
    n = inv_freq.shape[0]
    angle = pos.astype(np.float64)[..., None] * inv_freq.astype(np.float64)
    turn = (np.exp((-1j if inverse else 1j) * angle) * amp)[:, :, None]
    y = x.astype(np.float64).copy()
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if interleaved else (y[..., :n], y[..., n:2 * n])
    w = (a + 1j * b) * turn
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = w.real, w.imag
    else:
        y[..., :n], y[..., n:2 * n] = w.real, w.imag
    return y


def _norm(t, groups, eps):
    tg = t.reshape(*t.shape[:-1], groups, -1)
    rms = np.sqrt((tg ** 2).mean(-1, keepdims=True) + eps)
    unit = tg / rms

    def back(d):
        d = d.reshape(tg.shape)
        return ((d - unit * (d * unit).mean(-1, keepdims=True)) / rms).reshape(t.shape)

    return unit.reshape(t.shape), back


def addnorm(x, residual, w, alpha, eps):
    s = alpha * x + (0.0 if residual is None else residual)
    return _norm(s, 1, eps)[0] * w, s


def addnorm_bwd(dy, s, w, dsum, alpha, eps):
    unit, back = _norm(s, 1, eps)
    d = back(dy * w) + (0.0 if dsum is None else dsum)
    return dict(dresidual=d, dx=alpha * d, dweight=(dy * unit).reshape(-1, s.shape[-1]).sum(0))


def _sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def gatenorm(x, z, w, groups, gate_first, eps):
    gate = 1.0 if z is None else z * _sigmoid(z)
    return _norm(x * gate, groups, eps)[0] * w if gate_first else _norm(x, groups, eps)[0] * w * gate


def gatenorm_bwd(dy, x, z, w, groups, gate_first, eps):
    sg = 1.0 if z is None else _sigmoid(z)
    gate = 1.0 if z is None else z * sg
    before, after = (gate, 1.0) if gate_first else (1.0, gate)
    unit, back = _norm(x * before, groups, eps)
    d = back(dy * after * w)
    out = dict(dx=d * before, dweight=(dy * after * unit).reshape(-1, x.shape[-1]).sum(0), dz=None)
    if z is not None:
        out["dz"] = (d * x if gate_first else dy * unit * w) * (sg + z * sg * (1.0 - sg))
    return out

"""fp64 reference of the constant-decay linear attention, its gradients and draft trees.

Plain token by token (node by node) evaluation in numpy, from the definitions:

    S_t = lam_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t               (decay rule)
    S_i = alpha_i (I - beta_i k_i k_i^T) S_p + beta_i k_i v_i^T      (delta rule, node i below p)

Arrays are [B, T, H, 128] as in the library; shared QK heads are contiguous groups.
Each function has a majorant beside it: the same sums over absolute values, which bounds
what roundings inside the sums can do to a result, whatever the signs.
"""
import numpy as np


def _np(x):
    return None if x is None else np.asarray(x.double().cpu().numpy() if hasattr(x, "cpu") else x, dtype=np.float64)


def _rep(x, Hv):
    return np.repeat(x, Hv // x.shape[2], axis=2)


def decay_forward(q, k, v, decay, S0=None):
    """(o [B, T, Hv, dv], S_T [B, Hv, dk, dv])."""
    q, k, v, decay, S0 = _np(q), _np(k), _np(v), _np(decay), _np(S0)
    B, T, Hv, dv = v.shape
    q, k = _rep(q, Hv), _rep(k, Hv)
    S = np.zeros((B, Hv, q.shape[-1], dv)) if S0 is None else S0.copy()
    o = np.zeros_like(v)
    for t in range(T):
        S = decay[None, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = np.einsum("bhij,bhi->bhj", S, q[:, t])
    return o, S


def decay_backward(q, k, v, decay, S0, dO, dS_final):
    """Gradients (dq, dk, dv, dS0) of <dO, o> + <dS_final, S_T>."""
    q, k, v, decay, S0, dO, dS = (_np(x) for x in (q, k, v, decay, S0, dO, dS_final))
    B, T, Hv, dv_ = v.shape
    Hqk, dk_ = q.shape[2], q.shape[3]
    qr, kr = _rep(q, Hv), _rep(k, Hv)
    S = np.zeros((B, Hv, dk_, dv_)) if S0 is None else S0.copy()
    lam = decay[None, :, None, None]
    dq, dk, dv = np.zeros_like(qr), np.zeros_like(kr), np.zeros_like(v)
    for t in range(T):
        S = lam * S + kr[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = np.einsum("bhij,bhj->bhi", S, dO[:, t])
    G = np.zeros((B, Hv, dk_, dv_)) if dS is None else dS.copy()      # dL/dS_t before token t's read-out
    for t in range(T - 1, -1, -1):
        G = G + qr[:, t, :, :, None] * dO[:, t, :, None, :]
        dk[:, t] = np.einsum("bhij,bhj->bhi", G, v[:, t])
        dv[:, t] = np.einsum("bhij,bhi->bhj", G, kr[:, t])
        G = lam * G
    share = lambda x: x.reshape(B, T, Hqk, Hv // Hqk, dk_).sum(3)  # noqa: E731
    return share(dq), share(dk), dv, G


def _abs(*xs):
    return tuple(None if x is None else np.abs(_np(x)) for x in xs)


def decay_forward_majorant(q, k, v, decay, S0=None):
    return decay_forward(*_abs(q, k, v, decay, S0))


def decay_backward_majorant(q, k, v, decay, S0, dO, dS_final):
    return decay_backward(*_abs(q, k, v, decay, S0, dO, dS_final))


def tree_alive(parents):
    """alive[b][i]: node i is not padding (parents in [0, i) or -1 all the way up)."""
    p = np.asarray(parents)
    alive = np.zeros(p.shape, dtype=bool)
    for b in range(p.shape[0]):
        for i in range(p.shape[1]):
            alive[b, i] = p[b, i] == -1 or (0 <= p[b, i] < i and alive[b, p[b, i]])
    return alive


def tree(q, k, v, parents, S, alpha=None, beta=None, decay=None, majorant=False):
    """Outputs and states of every node: (o [B, n, Hv, dv], S_nodes [B, n, Hv, dk, dv], alive).

    S [B, Hv, dk, dv]: the cached states.  Delta rule with alpha, beta [B, n, Hv], decay rule
    with decay [Hv].  majorant: sums of absolute values."""
    q, k, v, S, alpha, beta, decay = (_np(x) for x in (q, k, v, S, alpha, beta, decay))
    if majorant:
        q, k, v, S, alpha, beta, decay = _abs(q, k, v, S, alpha, beta, decay)
    p = np.asarray(parents)
    B, n, Hv, dv = v.shape
    k = _rep(k, Hv)
    q = None if q is None else _rep(q, Hv)
    alive = tree_alive(p)
    states = np.zeros((B, n) + S.shape[1:])
    o = np.zeros_like(v)
    for b in range(B):
        for i in range(n):
            if not alive[b, i]:
                continue
            P = S[b] if p[b, i] < 0 else states[b, p[b, i]]
            ki, vi = k[b, i], v[b, i]
            if decay is not None:
                new = decay[:, None, None] * P + ki[:, :, None] * vi[:, None, :]
            else:
                a, be = alpha[b, i][:, None], beta[b, i][:, None]
                w = a * np.einsum("hij,hi->hj", P, ki)
                u = be * (vi + w if majorant else vi - w)
                new = a[:, :, None] * P + ki[:, :, None] * u[:, None, :]
            states[b, i] = new
            if q is not None:
                o[b, i] = np.einsum("hij,hi->hj", new, q[b, i])
    return o, states, alive


QMAX = {"int8": 127.0, "e4m3": 448.0}
TINY = 1e-30


def e4m3_values():
    """The non-negative finite values of the e4m3 format, in code order 0 .. 126."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def round_e4m3(y):
    """Nearest e4m3 value, ties to the even code."""
    vals = e4m3_values()
    a = np.abs(y)
    hi = np.clip(np.searchsorted(vals, a), 0, len(vals) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - vals[lo], vals[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(a >= vals[-1], len(vals) - 1, pick)
    return np.copysign(vals[pick], y)


def quantise_rows(S, fmt):
    """(codes' values, scales) of rows S [..., 128]: every 32-bit rounding done from 64 bits."""
    x = np.asarray(S, dtype=np.float64)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        bad = ~np.isfinite(x).all(-1)
        zero = ~bad & (top < TINY)
        inv = np.float32(QMAX[fmt] / top).astype(np.float64)
        y = np.float32(x * inv[..., None]).astype(np.float64)
        y = np.where((bad | zero)[..., None], 0.0, y)
        c = np.clip(np.rint(y), -QMAX[fmt], QMAX[fmt]) if fmt == "int8" else round_e4m3(y)
        scale = np.float32(top / QMAX[fmt])
    scale = np.where(zero, np.float32(0), np.where(bad, np.float32(np.nan), scale))
    return c, scale

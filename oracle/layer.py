"""fp64 definitions of the layer operators around the attention, in numpy:
rotary embedding, linear layer, differential attention.  Shares no code with
the CUDA path; `diff_attention` also returns how far 16-bit probabilities may
move each output."""
import math

import numpy as np


def rotary(x, pos, freqs, axis=None, half=False, parts=1, scale=1.0, inverse=False):
    """x [B, S, H, d], pos [B, S] or (with axis, the axis of each pair) [B, S, 3]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    n, R = x.shape[-1] // parts, 2 * len(freqs)
    sign = -1.0 if inverse else 1.0
    for part in range(parts):
        for p, w in enumerate(freqs):
            t = np.asarray(pos if axis is None else pos[..., axis[p]], np.float64) * w
            c, s = scale * np.cos(t)[..., None], sign * scale * np.sin(t)[..., None]
            i, j = (p, p + R // 2) if half else (2 * p, 2 * p + 1)
            i, j = part * n + i, part * n + j
            y[..., i] = x[..., i] * c - x[..., j] * s
            y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def activation(y, name):
    if name == "gelu":
        return y * 0.5 * np.vectorize(math.erfc)(-y / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * y * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
    if name == "silu":
        return y / (1.0 + np.exp(-y))
    return np.maximum(y, 0.0) if name == "relu" else y


def linear(x, w, bias=None, act="none", residual=None):
    y = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    y = activation(y, act)
    return y if residual is None else y + np.asarray(residual, np.float64)


def diff_attention(q, k, v, lam, lambda_init, norm_w=None, eps=1e-5, allowed=None, scale=None, u=0.0):
    """q [B, H, S_q, d], k and v [B, H_kv, S_kv, d], allowed bool [B, S_kv].

    Returns (o [B, S_q, H, d], lse [2, B, H, S_q], bound): bound is the first
    order change of o when every probability moves by a factor of at most
    1 + u.  What masked keys hold is never read."""
    q, k, v, lam = (np.asarray(t, np.float64) for t in (q, k, v, lam))
    B, H, S_q, d = q.shape
    G = H // k.shape[1]
    scale = 1.0 / math.sqrt(d // 2) if scale is None else scale
    o, bound = np.zeros((B, S_q, H, d)), np.zeros((B, S_q, H, d))
    lse = np.full((2, B, H, S_q), -np.inf)
    for b in range(B):
        keep = np.arange(k.shape[2]) if allowed is None else np.flatnonzero(allowed[b])
        if not len(keep):
            continue
        for h in range(H):
            kk, vv = k[b, h // G][keep], v[b, h // G][keep]
            lh = math.exp(lam[0, h] @ lam[1, h]) - math.exp(lam[2, h] @ lam[3, h]) + lambda_init
            for m, f in ((0, 1.0), (1, -lh)):
                ch = slice(m * d // 2, (m + 1) * d // 2)
                t = q[b, h][:, ch] @ kk[:, ch].T * scale
                mx = t.max(-1, keepdims=True)
                e = np.exp(t - mx)
                l = e.sum(-1, keepdims=True)
                lse[m, b, h] = (mx + np.log(l))[:, 0]
                o[b, :, h] += f * (e / l) @ vv
                bound[b, :, h] += u * abs(f) * (e / l) @ np.abs(vv)
    if norm_w is not None:
        ms = (o * o).mean(-1, keepdims=True)
        r = (1.0 - lambda_init) / np.sqrt(ms + eps)
        turn = np.sqrt((bound * bound).mean(-1, keepdims=True) / (ms + eps))     # relative change of 1 / rms
        bound = r * np.abs(norm_w) * (bound + np.abs(o) * turn)
        o = o * r * np.asarray(norm_w, np.float64)
    return o, lse, bound

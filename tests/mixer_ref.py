"""Float64 references of the gated linear recurrence and of the query/key norm,
written from their definitions (token by token, one pair at a time), with the
sums of absolute values that bound their rounding errors."""
from __future__ import annotations

import numpy as np

# half a step, relative to the value
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def recurrence(q, k, v, g, scale, state=None, lengths=None):
    """q, k [B, N, H, dk], v [B, N, H, dv], g [B, N, H] (float64).  Returns o, the
    final state, and both computed from absolute values."""
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    n = np.full(B, N) if lengths is None else np.clip(lengths, 0, N)
    S = np.zeros((B, H, dk, dv)) if state is None else state.copy()
    A = np.abs(S)
    o, oa = np.zeros((B, N, H, dv)), np.zeros((B, N, H, dv))
    for b in range(B):
        for t in range(int(n[b])):
            a = np.exp(g[b, t])[:, None, None]
            S[b] = a * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            A[b] = a * A[b] + np.abs(k[b, t])[:, :, None] * np.abs(v[b, t])[:, None, :]
            o[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], S[b])
            oa[b, t] = abs(scale) * np.einsum("hk,hkv->hv", np.abs(q[b, t]), A[b])
    return o, S, oa, A


def recurrence_grad(do, q, k, v, g, scale, state=None, lengths=None, d_final=None):
    """Gradients (dq, dk, dv, dg, dS_0) by the definition, the states of every token kept."""
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    n = np.full(B, N) if lengths is None else np.clip(lengths, 0, N)
    dq, dk_, dv_ = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg, d0 = np.zeros(g.shape), np.zeros((B, H, dk, dv))
    for b in range(B):
        S = np.zeros((int(n[b]) + 1, H, dk, dv))
        if state is not None:
            S[0] = state[b]
        for t in range(int(n[b])):
            S[t + 1] = np.exp(g[b, t])[:, None, None] * S[t] + k[b, t][:, :, None] * v[b, t][:, None, :]
        dS = np.zeros((H, dk, dv)) if d_final is None else d_final[b].copy()
        for t in range(int(n[b]) - 1, -1, -1):
            dS = dS + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dq[b, t] = scale * np.einsum("hkv,hv->hk", S[t + 1], do[b, t])
            dk_[b, t] = np.einsum("hkv,hv->hk", dS, v[b, t])
            dv_[b, t] = np.einsum("hkv,hk->hv", dS, k[b, t])
            a = np.exp(g[b, t])
            dg[b, t] = np.where(a == 0.0, 0.0, a * np.einsum("hkv,hkv->h", S[t], dS))
            dS = a[:, None, None] * dS
        d0[b] = dS
    return dq, dk_, dv_, dg, d0


def _norm(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    m = x.shape[-1] if norm == "rms" else 1
    return np.sqrt((x * x).sum(-1, keepdims=True) / m + eps)


def _pairs(rotary, layout):
    i = np.arange(rotary // 2)
    return (i, i + rotary // 2) if layout == "half" else (2 * i, 2 * i + 1)


def qk_norm(x, w, pos, freqs, norm, layout, rotary, eps, rscale):
    """x [B, N, H, D], pos [B, N] -> y."""
    y = x / _norm(x, norm, eps) * (1.0 if w is None or norm == "none" else w)
    a, b = _pairs(rotary, layout)
    t = pos[:, :, None, None] * freqs
    out = y.copy()
    out[..., a] = rscale * (y[..., a] * np.cos(t) - y[..., b] * np.sin(t))
    out[..., b] = rscale * (y[..., a] * np.sin(t) + y[..., b] * np.cos(t))
    return out


def qk_norm_grad(dy, x, w, pos, freqs, norm, layout, rotary, eps, rscale):
    """(dx, dw or None) and the absolute sum behind dw."""
    a, b = _pairs(rotary, layout)
    t = pos[:, :, None, None] * freqs
    dn = dy.copy()
    dn[..., a] = rscale * (dy[..., a] * np.cos(t) + dy[..., b] * np.sin(t))
    dn[..., b] = rscale * (dy[..., b] * np.cos(t) - dy[..., a] * np.sin(t))
    if norm == "none":
        return dn, None, None
    n = _norm(x, norm, eps)
    m = x.shape[-1] if norm == "rms" else 1
    h = dn * (1.0 if w is None else w)
    dx = h / n - x * (h * x).sum(-1, keepdims=True) / (m * n ** 3)
    return dx, (dn * x / n).sum((0, 1, 2)), np.abs(dn * x / n).sum((0, 1, 2))

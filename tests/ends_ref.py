"""Float64 references of the embedding, the norm of whole tokens and the loss
over a vocabulary, written from their definitions, with the sums of absolute
values that bound their rounding errors."""
from __future__ import annotations

import numpy as np

from mixer_ref import HALF_STEP  # noqa: F401  (half a step, relative to the value)

# half a step of the smallest values (binary16 loses its bits below 2^-14)
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def embedding(tokens, table, scale):
    V = table.shape[0]
    live = (tokens >= 0) & (tokens < V)
    return np.where(live[..., None], table[np.where(live, tokens, 0)] * scale, 0.0)


def embedding_grad(d_out, tokens, V, scale, old=None):
    """(d_table, the same of absolute values, tokens of each value)."""
    d = d_out.shape[-1]
    g = np.zeros((V, d)) if old is None else old.copy()
    a, n = np.abs(g), np.zeros(V)
    for t, v in enumerate(tokens.reshape(-1)):
        if 0 <= v < V:
            row = d_out.reshape(-1, d)[t] * scale
            g[v] += row
            a[v] += np.abs(row)
            n[v] += 1
    return g, a, n


def residual_norm(x, residual, w, eps):
    s = x if residual is None else x + residual
    return s * w / np.sqrt((s * s).mean(-1, keepdims=True) + eps), s


def residual_norm_grad(dy, s, w, ds, eps):
    """(dx, dweight, the sums of absolute values behind both)."""
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    n, dn = s * r, dy * w
    more = 0.0 if ds is None else ds
    dx = more + r * (dn - n * (dn * n).mean(-1, keepdims=True))
    size = np.abs(more) + r * (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(-1, keepdims=True))
    axes = tuple(range(s.ndim - 1))
    return dx, (dy * n).sum(axes), size, np.abs(dy * n).sum(axes)


def logits(x, table, scale):
    """(logits, sums of absolute values) of rows x [T, d]."""
    return scale * (x @ table.T), abs(scale) * (np.abs(x) @ np.abs(table).T)


def token_loss(x, table, targets, scale):
    """(loss, lse, largest sum of absolute values of each token), 0 where no target is."""
    l, size = logits(x, table, scale)
    live = (targets >= 0) & (targets < table.shape[0])
    m = l.max(-1)
    lse = m + np.log(np.exp(l - m[:, None]).sum(-1))
    at = l[np.arange(len(targets)), np.where(live, targets, 0)]
    return np.where(live, lse - at, 0.0), np.where(live, lse, 0.0), size.max(-1)


def token_loss_grad(d_loss, x, table, targets, lse, scale):
    """(dx, d_table, G, logits' sizes)."""
    l, size = logits(x, table, scale)
    live = (targets >= 0) & (targets < table.shape[0])
    p = np.exp(l - lse[:, None])
    g = p.copy()
    g[np.arange(len(targets)), np.where(live, targets, 0)] -= 1.0
    g = np.where(live[:, None], g * np.where(live, d_loss, 0.0)[:, None], 0.0)
    p = np.where(live[:, None], p, 0.0)
    return scale * (g @ table), scale * (g.T @ np.where(live[:, None], x, 0.0)), g, p, size.max(-1)

"""Float64 oracle of the token rows (include/ds_token_rows.h): embedding rows and
their gradient, RMS-normed rotated q/k heads and their gradient, log
probabilities of logits rows and their gradient.

Every function takes the values the kernels take (bf16 as float arrays already
decoded) and computes the definition in float64, loop by loop where that is
the plainest way.  Each returns, beside its values, the magnitude of the terms
they were summed from, which the tests' error bounds are multiples of.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- embedding

def embed_rows(table: np.ndarray, ids: np.ndarray, scale: float) -> np.ndarray:
    """fp32(scale) * table[ids] as one fp32 product; zeros for unknown ids."""
    out = np.zeros((len(ids), table.shape[1]), np.float32)
    for i, t in enumerate(ids):
        if 0 <= t < table.shape[0]:
            out[i] = table[t].astype(np.float32) * np.float32(scale)
    return out


def embed_rows_backward(dy: np.ndarray, ids: np.ndarray, vocab: int, scale: float):
    """(dtable, sum of |terms|, rows of each token)."""
    s = float(np.float32(scale))
    out = np.zeros((vocab, dy.shape[1]))
    mag = np.zeros_like(out)
    count = np.zeros(vocab, np.int64)
    for i, t in enumerate(ids):
        if 0 <= t < vocab:
            out[t] += dy[i]
            mag[t] += np.abs(dy[i])
            count[t] += 1
    return out * s, mag * abs(s), count


# ---------------------------------------------------------------- q/k heads

def _angles(positions, inv_freq):
    t = np.asarray(positions, np.float64)[:, None] * inv_freq.astype(np.float64)
    return np.cos(t)[:, None, :], np.sin(t)[:, None, :]


def _turn(x, c, s):
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def _swap_abs(x):
    """|x1| + |x2| of the pair each element turns with."""
    h = x.shape[-1] // 2
    m = np.abs(x[..., :h]) + np.abs(x[..., h:])
    return np.concatenate([m, m], axis=-1)


def qk_rows_rms(x, positions, inv_freq, weight, head_dim: int, eps: float):
    """(out, magnitude) of [rows, heads * head_dim] values; weight None for 1."""
    rows = x.shape[0]
    v = x.astype(np.float64).reshape(rows, -1, head_dim)
    w = np.ones(head_dim) if weight is None else weight.astype(np.float64)
    D = np.sqrt((v * v).sum(-1, keepdims=True) / head_dim + float(np.float32(eps)))
    n = v / D * w
    c, s = _angles(positions, inv_freq)
    return _turn(n, c, s).reshape(rows, -1), _swap_abs(n).reshape(rows, -1)


def qk_rows_rms_backward(x, positions, inv_freq, weight, dy, head_dim: int, eps: float):
    """(dx, dweight, magnitude of dx's terms, sum of |dweight's terms|)."""
    rows = x.shape[0]
    v = x.astype(np.float64).reshape(rows, -1, head_dim)
    g = dy.astype(np.float64).reshape(rows, -1, head_dim)
    w = np.ones(head_dim) if weight is None else weight.astype(np.float64)
    D = np.sqrt((v * v).sum(-1, keepdims=True) / head_dim + float(np.float32(eps)))
    u = v / D
    c, s = _angles(positions, inv_freq)
    d = _turn(g, c, -s)
    dm = _swap_abs(g)
    dw = (d * u).sum((0, 1))
    mean = (w * d * u).sum(-1, keepdims=True) / head_dim
    dx = (w * d - u * mean) / D
    mag = (np.abs(w) * dm + np.abs(u) * (np.abs(w) * dm * np.abs(u)).sum(-1, keepdims=True)
           / head_dim) / D
    return dx.reshape(rows, -1), dw, mag.reshape(rows, -1), (dm * np.abs(u)).sum((0, 1))


# ------------------------------------------------------------------- logits

def scaled_logits(x, scale, inv_temp) -> np.ndarray:
    """z as the kernels form it: fp32 products, in this order."""
    z = x.astype(np.float32)
    if scale is not None:
        z = z * scale.astype(np.float32)
    return z * np.float32(inv_temp)


def logprob_row(z32: np.ndarray, label: int, top_k: int):
    """(logp, entropy, lse, top ids, top logp) of one row of fp32 z.  Log
    probabilities are formed as (z - max) - log sum exp(z - max): beside a
    maximum of 1e38, float64 has no room for the logarithm."""
    z = z32.astype(np.float64)
    masked = z == -np.inf
    m, log_s = 0.0, np.nan
    if masked.all():
        lse, ent, log_s = -np.inf, 0.0, -np.inf
    elif np.isnan(z).any() or (z == np.inf).any():
        lse = ent = np.nan
    else:
        m = z.max()
        log_s = np.log(np.exp(z - m).sum())
        lse = m + log_s
        lp = (z[~masked] - m) - log_s
        ent = float(-(np.exp(lp) * lp).sum())
    if not 0 <= label < len(z):
        logp = 0.0
    elif masked.all():
        logp = -np.inf
    else:
        logp = (z[label] - m) - log_s
    listed = [j for j in range(len(z)) if z[j] > -np.inf]           # drops NaN too
    listed.sort(key=lambda j: (-z[j], j))
    ids = (listed + [-1] * top_k)[:top_k]
    top = [(z[j] - m) - log_s if j >= 0 else -np.inf for j in ids]
    return logp, ent, lse, ids, top


def logprob_rows(z32, labels, top_k: int = 0):
    rows = [logprob_row(z32[i], int(labels[i]), top_k) for i in range(len(z32))]
    return tuple(np.array(c) for c in zip(*rows))


def logprob_rows_backward(x, z32, labels, lse, entropy, dlogp, dentropy, scale, inv_temp):
    """(dlogits, dscale, error scales of both) for finite lse; ``lse`` and
    ``entropy`` are the forward call's fp32 outputs.  The scales: what one
    fp32 rounding of p's exponent, of its factors and of the products moves an
    element by, at most."""
    rows, vocab = z32.shape
    tau = float(np.float32(inv_temp))
    s64 = np.ones(vocab) if scale is None else scale.astype(np.float64)
    dx = np.zeros((rows, vocab))
    unit = np.zeros((rows, vocab))
    ds = np.zeros(vocab)
    ds_unit = np.zeros(vocab)
    ds_mag = np.zeros(vocab)
    for i in range(rows):
        live = z32[i] > -np.inf
        if not live.any():
            continue
        z = z32[i].astype(np.float64)
        lp = np.where(live, z, 0.0) - float(lse[i])
        p = np.where(live, np.exp(lp), 0.0)
        y = int(labels[i])
        known = 0 <= y < vocab
        g = float(dlogp[i]) if dlogp is not None and known else 0.0
        gh = float(dentropy[i]) if dentropy is not None else 0.0
        h = float(entropy[i]) if dentropy is not None else 0.0
        inner = g + gh * (lp + h)
        d = -p * inner
        if known and live[y]:
            d[y] += g
        d *= tau
        size = p * (np.abs(g) + np.abs(gh) * (np.abs(lp) + np.abs(h)))
        u = size * (np.abs(lp) + 1.0) * tau
        if known:
            u[y] += abs(g) * tau
        dx[i] = d * s64
        unit[i] = u * np.abs(s64)
        xv = np.where(live, x[i].astype(np.float64), 0.0)
        ds += d * xv
        ds_unit += u * np.abs(xv)
        ds_mag += np.abs(d * xv)
    return dx, ds, unit, ds_unit, ds_mag

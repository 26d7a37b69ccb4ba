"""Float64 oracle of the rows of a decoding step (include/ds_decode_rows.h):
rotary positions and their gradient, the append to a paged cache, attention
over it, and the verification of drafted tokens.

Every function takes the values the kernels take (bf16 and e4m3 as float
arrays already decoded) and computes the definition in float64, loop by loop
where that is the plainest way.  Where a test's error bound is a multiple of
the terms that a value was summed from, their magnitude is returned beside it.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The 256 values of e4m3 by code: 4 exponent bits of bias 7, 3 of
    significand, no infinities, NaN at 0x7f and 0xff."""
    out = np.zeros(256)
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        v = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        out[code] = math.nan if (code & 127) == 127 else (-v if code & 128 else v)
    return out


def frequencies(rotary: int, base=10000.0, factor=1.0, original=1.0, low=0.0, high=0.0) -> np.ndarray:
    out = []
    for i in range(rotary // 2):
        f = base ** (-2.0 * i / rotary)
        turns = original * f / (2 * math.pi)
        keep = 0.0 if high == 0.0 else min(1.0, max(0.0, (turns - low) / (high - low)))
        out.append(keep * f + (1 - keep) * f / factor)
    return np.array(out)


def rope_heads(x, positions, inv_freq, head_dim: int, interleaved=False, amplitude=1.0, back=False):
    """(out, magnitude of the terms) of [rows, heads * head_dim] values; ``back``
    turns the other way, as the gradient does.  A value that does not turn has
    magnitude 0: it comes out bit for bit."""
    rows, pairs = x.shape[0], len(inv_freq)
    v = x.astype(np.float64).reshape(rows, -1, head_dim)
    out, mag = v.copy(), np.zeros_like(v)
    amp = float(np.float32(amplitude))
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)
        t = positions.astype(np.float64) * float(inv_freq[i])
        c, s = (amp * np.cos(t))[:, None], (amp * np.sin(t) * (-1 if back else 1))[:, None]
        with np.errstate(invalid="ignore"):
            out[:, :, a] = v[:, :, a] * c - v[:, :, b] * s
            out[:, :, b] = v[:, :, b] * c + v[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = abs(amp) * (np.abs(v[:, :, a]) + np.abs(v[:, :, b]))
    return out.reshape(rows, -1), mag.reshape(rows, -1)


def normed_heads(x, weight, head_dim: int, eps: float):
    """x / sqrt(mean x^2 + eps) * weight, a head at a time."""
    v = x.astype(np.float64).reshape(x.shape[0], -1, head_dim)
    D = np.sqrt((v * v).sum(-1, keepdims=True) / head_dim + float(np.float32(eps)))
    w = np.ones(head_dim) if weight is None else weight.astype(np.float64)
    return (v / D * w).reshape(x.shape)


def token_place(table, n_pages: int, page_size: int, seq: int, token: int):
    """(page, offset) of a sequence's token, or None."""
    if not (0 <= seq < table.shape[0] and token >= 0 and token // page_size < table.shape[1]):
        return None
    page = int(table[seq, token // page_size])
    return (page, token % page_size) if 0 <= page < n_pages else None


def visible(length: int, n_new: int, j: int, window: int, capacity: int):
    """The tokens that new token j of a sequence sees, were all pages there."""
    t = min(max(length, 0), capacity) - n_new + j
    lo = max(0, t - window + 1) if window else 0
    return range(lo, t + 1)


def attention(q, k, v, table, lens, n_new: int, n_q_heads: int, window: int, scale: float,
              k_scale=None, v_scale=None):
    """(out, lse, sum of p |v|, largest sum of |scale q k|, tokens seen) for q
    [seqs * n_new, n_q_heads * hd] over k, v [pages, page_size, heads, hd]."""
    pages, page_size, heads, hd = k.shape
    rows = q.shape[0]
    q = q.astype(np.float64).reshape(rows, n_q_heads, hd)
    out, mag = np.zeros((rows, n_q_heads, hd)), np.zeros((rows, n_q_heads, hd))
    lse, big = np.full((rows, n_q_heads), -np.inf), np.zeros((rows, n_q_heads))
    seen = np.zeros(rows, np.int64)
    ks = np.ones(heads) if k_scale is None else k_scale.astype(np.float64)
    vs = np.ones(heads) if v_scale is None else v_scale.astype(np.float64)
    for row in range(rows):
        seq, j = divmod(row, n_new)
        at = [token_place(table, pages, page_size, seq, t)
              for t in visible(int(lens[seq]), n_new, j, window, table.shape[1] * page_size)]
        at = [a for a in at if a is not None]
        seen[row] = len(at)
        if not at:
            continue
        page, off = np.array(at).T
        for g in range(n_q_heads):
            h = g // (n_q_heads // heads)
            kk, vv = k[page, off, h].astype(np.float64) * ks[h], v[page, off, h].astype(np.float64) * vs[h]
            with np.errstate(invalid="ignore", over="ignore"):
                z = (kk @ q[row, g]) * float(np.float32(scale))
                if (z == -np.inf).all():
                    continue
                top = z.max()
                w = np.exp(z - top)
                lse[row, g] = top + math.log(w.sum()) if np.isfinite(w.sum()) else np.nan
                p = w / w.sum()
                out[row, g] = p @ vv
                mag[row, g] = p @ np.abs(vv)
                big[row, g] = (np.abs(kk) @ np.abs(q[row, g]))[z > -np.inf].max(initial=0) * abs(scale)
    return out.reshape(rows, -1), lse, mag.reshape(rows, -1), big, seen


def scaled_logits(x, scale, inv_temp) -> np.ndarray:
    """z as the kernels form it: fp32 products, in this order."""
    z = x.astype(np.float32)
    if scale is not None:
        z = z * scale.astype(np.float32)
    return z * np.float32(inv_temp)


def probabilities(z32):
    """(p, log p) of a row of z; (None, None) where the row says nothing."""
    z = z32.astype(np.float64)
    if not (z < np.inf).all() or (z == -np.inf).all():     # a NaN or +infinity, or masked whole
        return None, None
    d = z - z.max()
    e = np.exp(d)
    return e / e.sum(), d - math.log(e.sum())


def verify_sequence(target, draft, drafted, u_accept, u_sample):
    """(tokens, log probabilities, smallest relative distance from a border)
    of one sequence: target z [n + 1, vocab], draft z [n, vocab] or None."""
    tokens, logp, margin = [], [], np.inf
    vocab = target.shape[1]
    weight = None
    for i, d in enumerate(drafted):
        if not 0 <= d < vocab:
            break
        p, lp = probabilities(target[i])
        if draft is None:
            q = np.zeros(vocab)
            q[d] = 1.0
        else:
            q, _ = probabilities(draft[i])
        pd = 0.0 if p is None else p[d]
        if q is None:
            weight = p if p is not None else np.zeros(vocab)
            break
        edge = float(u_accept[i]) * q[d]
        if edge > 0 or pd > 0:
            margin = min(margin, abs(edge - pd) / max(edge, pd))
        if p is None or not edge < pd:
            weight = np.zeros(vocab) if p is None else np.maximum(p - q, 0)
            if p is not None and not weight.any():
                weight = p
            break
        tokens.append(int(d))
        logp.append(lp[d])
    p, lp = probabilities(target[len(tokens)])
    if weight is None:
        weight = np.zeros(vocab) if p is None else p
    if not weight.any():
        return tokens + [-1], logp + [0.0], margin
    run = np.cumsum(weight)
    u = float(u_sample)
    edge = (0.0 if u < 0 else u) * run[-1]
    past = np.flatnonzero((run > edge) & (weight > 0))
    token = int(past[0]) if len(past) else int(np.flatnonzero(weight)[-1])
    if len(past) and edge > 0:
        margin = min(margin, np.abs(run - edge).min() / run[-1])
    return tokens + [token], logp + [lp[token]], margin

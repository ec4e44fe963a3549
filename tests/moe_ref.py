"""Plain 64-bit definitions of the router, the expert order, the rows' way there
and back, and the 4-bit products, for the tests: written from the formulas in
include/gbmm.h, row by row."""

from __future__ import annotations

import numpy as np


def route(logits32, bias32, top_k, selected):
    """ids, weights and the live mask.  `logits32`: the stored values as f32."""
    m, E = logits32.shape
    with np.errstate(invalid="ignore"):
        score = logits32 if bias32 is None else (logits32 + bias32[None, :]).astype(np.float32)
    live = score > -np.inf
    ids = np.full((m, top_k), E, np.int64)
    w = np.zeros((m, top_k))
    p = np.zeros((m, E))
    for t in range(m):
        cand = [e for e in range(E) if live[t, e]]
        cand.sort(key=lambda e: (-float(score[t, e]), e))
        pick = cand[:top_k]
        ids[t, :len(pick)] = pick
        over = pick if selected else [e for e in range(E) if live[t, e]]
        if over:
            l = logits32[t, over].astype(np.float64)
            with np.errstate(invalid="ignore"):
                v = np.exp(l - l.max())
                p[t, over] = v / v.sum()
        w[t, :len(pick)] = p[t, pick]
    return ids, w, p, live


def route_backward(ids, w, p, d_w, E):
    """The softmax's Jacobian over the experts that p runs over."""
    m, k = ids.shape
    out = np.zeros((m, E))
    for t in range(m):
        slots = [s for s in range(k) if ids[t, s] < E]
        c = sum(w[t, s] * d_w[t, s] for s in slots)
        out[t] = -p[t] * c
        for s in slots:
            out[t, ids[t, s]] += w[t, s] * d_w[t, s]
    return out


def sort(ids, E):
    """offsets, order, position."""
    key = np.minimum(np.asarray(ids, np.int64).reshape(-1), E)
    order = np.array(sorted(range(key.size), key=lambda r: (key[r], r)), np.int64)
    position = np.empty(key.size, np.int64)
    position[order] = np.arange(key.size)
    offsets = np.array([int((key < e).sum()) for e in range(E + 1)], np.int64)
    return offsets, order, position


def dispatch(x, position, valid, top_k):
    out = np.zeros((position.size, x.shape[1]))
    for r, at in enumerate(position):
        if at < valid:
            out[at] = x[r // top_k]
    return out


def combine(ys, w, position, valid, m, top_k):
    """y and the sum of the terms' magnitudes."""
    y, mag = np.zeros((m, ys.shape[1])), np.zeros((m, ys.shape[1]))
    for r, at in enumerate(position):
        if at < valid:
            term = (1.0 if w is None else w.reshape(-1)[r]) * ys[at]
            y[r // top_k] += term
            mag[r // top_k] += np.abs(term)
    return y, mag


def combine_backward(ys, w, d_y, position, valid, top_k):
    d_ys, d_w, mag = np.zeros_like(ys), np.zeros(position.size), np.zeros(position.size)
    for r, at in enumerate(position):
        if at < valid:
            g = d_y[r // top_k]
            d_ys[at] = w.reshape(-1)[r] * g
            d_w[r] = float(g @ ys[at])
            mag[r] = float(np.abs(g) @ np.abs(ys[at]))
    return d_ys, d_w.reshape(w.shape), mag.reshape(w.shape)


def q4_matrix(q, scales, zeros, k, group):
    """W [.., n, k] from bytes [.., n, (k + 1) // 2]."""
    w = np.empty(q.shape[:-1] + (2 * q.shape[-1],))
    w[..., 0::2] = q & 15
    w[..., 1::2] = q >> 4
    g = np.arange(k) // group
    z = 8.0 if zeros is None else zeros[..., g].astype(np.float64)
    return (w[..., :k] - z) * scales[..., g].astype(np.float64)


def pack_q4(codes):
    """Bytes of codes 0..15 [.., k]: even columns in the low half."""
    if codes.shape[-1] % 2:
        codes = np.concatenate([codes, np.full(codes.shape[:-1] + (1,), 15, codes.dtype)], axis=-1)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)

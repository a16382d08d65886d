"""Drafted trees over a placed KV cache and rows that move between requests -- oracle (fp64, plain
definitions).

Attention: token t of request b sees the first lens[b] rows and, of the n_new[b] drafted rows
behind them, those whose bit is set in its mask (None: the drafts 0..t); softmax over what it
sees; zeros for a token that sees nothing.

Rotation by axes: pair i of a token turns by its position on axis[i] times f_i.

Commit: row lens + path[i] becomes row lens + i; entries of the drafts that are not kept become
-1 and 0. Fork: request b's rows first[b] .. n - 1 become those of request src_of[b].
"""
import math

import numpy as np

from .cache import _f64


def bits(mask, T):
    """[.., T][words] of 64 bits -> bool [.., T][T]."""
    m = np.asarray(mask).view(np.uint64)
    s = np.arange(T)
    return (m[..., s // 64] >> (s % 64).astype(np.uint64)) & np.uint64(1) == 1


def attention(q, k, v, lens, mask=None, n_new=None, scale=None):
    """q [B][T][Hq][D], k, v [B][Hkv][L][D]. Returns (o, spread [B][T][Hq][D] = sum_j p_j |v_j|, reach
    [B][T][Hq] = max_j scale * sum_d |q_d k_jd|); rows of tokens t >= n_new[b] are zero."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, T, Hq, D = q.shape
    Hkv, L = k.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o, spread, reach = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    seen = np.tril(np.ones((T, T), bool)) if mask is None else bits(mask, T)
    seen = np.broadcast_to(seen, (B, T, T))
    for b in range(B):
        n = int(np.clip(lens[b], 0, L))
        m = T if n_new is None else int(np.clip(n_new[b], 0, T))
        d = min(m, L - n)
        for t in range(m):
            rows = np.concatenate([np.arange(n), n + np.flatnonzero(seen[b, t, :d])])
            if not len(rows):
                continue
            for g in range(Hkv):
                hs = slice(g * G, (g + 1) * G)
                kk, vv = k[b, g, rows], v[b, g, rows]
                s = scale * (q[b, t, hs] @ kk.T)
                e = np.exp(s - s.max(1, keepdims=True))
                p = e / e.sum(1, keepdims=True)
                o[b, t, hs], spread[b, t, hs] = p @ vv, p @ np.abs(vv)
                reach[b, t, hs] = abs(scale) * (np.abs(q[b, t, hs]) @ np.abs(kk).T).max(1)
    return o, spread, reach


def rotate_axes(x, positions, axis, freqs, interleaved=False, attn_scale=1.0):
    """x [N][H][D], positions [N][axes] -> rotated fp64 [N][H][D]."""
    x = _f64(x)
    R = 2 * len(freqs)
    a = (np.asarray(positions, np.float64)[:, np.asarray(axis)] * np.asarray(freqs))[:, None]
    c, s = np.cos(a) * attn_scale, np.sin(a) * attn_scale
    i = np.arange(R // 2)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y = x.copy()
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def commit(rows, lens, path, n_path, n_new, slot_pos=None, acc=None):
    """rows: arrays [B][H][L][..] (K, V). Returns (rows, lens, slot_pos, acc) after the commit."""
    rows = [np.array(r) for r in rows]
    pos = None if slot_pos is None else np.array(slot_pos)
    acc = None if acc is None else np.array(acc)
    B, _, L = rows[0].shape[:3]
    out = np.zeros(B, np.int64)
    for b in range(B):
        n = int(np.clip(lens[b], 0, L))
        m = min(int(n_new[b]), L - n)
        at = np.asarray(path[b])[:int(np.clip(n_path[b], 0, len(path[b])))]
        if len(at) and (at.min() < 0 or at.max() >= m or (np.diff(at) <= 0).any()):
            at = at[:0]
        out[b] = n + len(at)
        for r in rows + [x for x in (pos, acc) if x is not None]:
            r[b, :, n:n + len(at)] = r[b][:, n + at]
        for r, empty in ((pos, -1), (acc, 0)):
            if r is not None:
                r[b, :, n + len(at):n + m] = empty
    return rows, out, pos, acc


def fork(to, src, src_of, lens, first=None, same=True, lens_out=None):
    """to, src: lists of arrays [B][H][L][..] (rows and tables; src may be to). Returns (to, lens_out)."""
    old = [np.array(x) for x in src]
    new = [np.array(x) for x in to]
    B, L, S = new[0].shape[0], new[0].shape[2], old[0].shape[2]
    out = np.clip(lens, 0, L) if same else np.array(lens_out)
    for b in range(B):
        f = int(src_of[b])
        if f < 0 or f >= old[0].shape[0] or (same and f == b):
            continue
        n = min(int(np.clip(lens[f], 0, S)), L)
        lo = 0 if first is None else int(np.clip(first[b], 0, n))
        out[b] = n
        for x, y in zip(new, old):
            x[b, :, lo:n] = y[f, :, lo:n]
    return new, out

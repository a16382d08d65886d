"""What changes a placed KV cache between attention calls, and attention over a shared prefix or
with accumulated weights -- oracle (fp64, plain definitions).

Rotation: pair i of a token at position p, (x1, x2) -> (x1 c - x2 s, x2 c + x1 s) with
c, s = attn_scale * cos, sin(p f_i); pairs are halves (i, i + R/2) or neighbours (2i, 2i + 1).
Frequencies f_i = theta^(-2i/R), and for long contexts divided by a factor, taken from a larger
base, or mixed by the turns that the pair makes over the original context.

Attention: softmax over the rows of the request's prefix and then its own cache; the weights of
the own rows are summed over the query heads of a kv head.

Eviction: n_keep slots per (request, kv head): the newest n_recent positions, then the largest
weights, equal ones by the lower slot, NaN last; kept rows from slots >= n_keep fill the freed
slots below, both in ascending order.
"""
import math

import numpy as np

from .bf16 import to_f64


def _f64(x):
    x = np.asarray(x)
    return to_f64(x) if x.dtype == np.uint16 else x.astype(np.float64)


def inv_freq(rot_dim, theta=500000.0, scaling="none", factor=1.0, orig_len=0.0, low_turns=1.0, high_turns=32.0):
    i = np.arange(0, rot_dim, 2, dtype=np.float64)
    f = theta ** (-i / rot_dim)
    if scaling == "linear":
        return f / factor
    if scaling == "ntk":
        return (theta * factor ** (rot_dim / (rot_dim - 2))) ** (-i / rot_dim) if rot_dim > 2 else f
    if scaling == "by_parts":
        mix = np.clip((orig_len * f / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0, 1)
        return f / factor * (1 - mix) + f * mix
    return f


def rotate(x, positions, freqs, interleaved=False, attn_scale=1.0):
    """x [N][H][D] (bf16 bits or floats), positions [N] -> rotated fp64 [N][H][D]."""
    x = _f64(x)
    R = 2 * len(freqs)
    a = np.asarray(positions, np.float64)[:, None, None] * np.asarray(freqs)
    c, s = np.cos(a) * attn_scale, np.sin(a) * attn_scale
    i = np.arange(R // 2)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y = x.copy()
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def attention(q, k, v, seq_lens, prefix=None, prefix_of=None, prefix_lens=None, scale=None):
    """q [B][Hq][D], k, v [B][Hkv][L][D], prefix (k, v) [P][Hkv][Lp][D]. Returns (o [B][Hq][D],
    weights [B][Hkv][L] summed over query heads, spread [B][Hq][D] = sum_j p_j |v_j|,
    reach [B][Hq] = max_j scale * sum_d |q_d k_jd|), the last two for error bounds."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Hq, D = q.shape
    Hkv, L = k.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o, spread, reach = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq))
    w = np.zeros((B, Hkv, L))
    if prefix is not None:
        pk, pv = _f64(prefix[0]), _f64(prefix[1])
        prefix_of = [0] * B if prefix_of is None else prefix_of
        prefix_lens = [pk.shape[2]] * pk.shape[0] if prefix_lens is None else prefix_lens
    for b in range(B):
        n = L if seq_lens is None else int(seq_lens[b])
        f = int(prefix_of[b]) if prefix is not None else -1
        if prefix is not None and f >= pk.shape[0]:
            f = -1
        m = int(prefix_lens[f]) if f >= 0 else 0
        for g in range(Hkv):
            kk, vv = k[b, g, :n], v[b, g, :n]
            if m:
                kk, vv = np.concatenate([pk[f, g, :m], kk]), np.concatenate([pv[f, g, :m], vv])
            if not len(kk):
                continue
            qq = q[b, g * G:(g + 1) * G]
            s = scale * (qq @ kk.T)
            e = np.exp(s - s.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            rows = slice(g * G, (g + 1) * G)
            o[b, rows] = p @ vv
            spread[b, rows] = p @ np.abs(vv)
            reach[b, rows] = abs(scale) * (np.abs(qq) @ np.abs(kk).T).max(1)
            w[b, g, :n] = p[:, m:].sum(0)
    return o, w, spread, reach


def evict(seq_lens, n_keep, n_recent, acc, slot_pos):
    """(lens, src [B][H][n_keep], acc, slot_pos) after the eviction; a row i < lens[b] of the new
    cache is row src[b][g][i] of the old one."""
    acc, pos = np.array(acc, np.float32), np.array(slot_pos, np.int64)
    B, H, L = acc.shape
    src = np.full((B, H, n_keep), -1, np.int64)
    lens = np.minimum(np.clip(seq_lens, 0, L), n_keep)
    for b in range(B):
        n = int(np.clip(seq_lens[b], 0, L))
        for g in range(H):
            if n <= n_keep:
                src[b, g, :n] = np.arange(n)
                continue
            newest = pos[b, g, :n] > pos[b, g, :n].max() - n_recent
            a = acc[b, g, :n].astype(np.float64)
            a[np.isnan(a)] = -np.inf
            nan = np.isnan(acc[b, g, :n])
            order = sorted(range(n), key=lambda i: (not newest[i], nan[i] and not newest[i], 0.0 if newest[i] else -a[i], i))
            kept = np.zeros(n, bool)
            kept[order[:n_keep]] = True
            s = np.arange(n_keep)
            s[~kept[:n_keep]] = n_keep + np.flatnonzero(kept[n_keep:])
            src[b, g] = s
            new_a, new_p = acc[b, g].copy(), pos[b, g].copy()
            new_a[:n_keep], new_p[:n_keep] = acc[b, g, s], pos[b, g, s]
            new_a[n_keep:n], new_p[n_keep:n] = 0.0, -1
            acc[b, g], pos[b, g] = new_a, new_p
    return lens, src, acc, pos


def slab_rows(slabs, H_kv, L):
    """[slabs][chunks][2][64][D] as a placed cache lies -> K, V [B][H_kv][L][D]."""
    slabs = np.asarray(slabs)
    S, C, _, _, D = slabs.shape
    t = np.arange(L)[:, None]
    d = np.arange(D)[None, :]
    at = ((d // 8) ^ (t % 8)) * 8 + d % 8
    k, v = (slabs[:, t // 64, kv, t % 64, at] for kv in (0, 1))
    return k.reshape(-1, H_kv, L, D), v.reshape(-1, H_kv, L, D)

"""NumPy fp64 restatement of the operators on a paged history: rotary positions, the
append to a paged cache and attention over a shared prefix and per-sequence tails."""
from __future__ import annotations

import math

import numpy as np


def rotary_freqs(dim, base=10000.0, scaling="plain", factor=1.0, trained_len=0.0):
    """Frequencies of one axis, pair by pair, and the magnitude."""
    out = []
    for j in range(dim // 2):
        b = base
        if scaling == "base" and dim > 2:
            b = base * factor ** (dim / (dim - 2))
        f = b ** (-2.0 * j / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "parts":
            first = max(math.floor(dim * math.log(trained_len / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
            last = min(math.ceil(dim * math.log(trained_len / (2 * math.pi)) / (2 * math.log(base))), dim - 1)
            r = (j - first) / max(last - first, 1e-3)
            r = 0.0 if r < 0 else 1.0 if r > 1 else r
            f = (1 - r) * f + r * (f / factor)
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0)


def grid_positions(S, Hg, W, axes, first=0):
    """Positions [S, axes] of the tokens first .. first + S - 1."""
    n = np.arange(first, first + S, dtype=np.int64)
    return np.stack((n // (Hg * W), n // W % Hg, n % W), -1) if axes == 3 else n[:, None]


def pair_axes(axis_dims):
    """Axis of every pair."""
    return np.concatenate([np.full(d // 2, a, dtype=np.int64) for a, d in enumerate(axis_dims)])


def rotary(x, pos, inv_freq, interleaved, axis_dims=None, magnitude=1.0, adjoint=False):
    """x [B, H, S, D], pos [B or 1, S, axes]."""
    half = len(inv_freq)
    axis = np.zeros(half, dtype=np.int64) if axis_dims is None else pair_axes(axis_dims)
    a = pos[..., axis].astype(np.float64) * inv_freq
    a = -a if adjoint else a
    c, s = (magnitude * np.cos(a))[:, None], (magnitude * np.sin(a))[:, None]
    i = np.arange(half)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = np.array(x, dtype=np.float64)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def append(cache, new, table, start, counts):
    """Rows new[b, :, :counts[b]] ([B, H, S, D]) into the pages of [pages, H, page, D]."""
    out = cache.copy()
    page = cache.shape[2]
    for b in range(new.shape[0]):
        for s in range(counts[b]):
            at = start[b] + s
            out[table[b][at // page], :, at % page] = new[b, :, s]
    return out


def prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len, tail_pages, tail_len, q_len, causal,
                     scale, part_o=None, part_lse=None):
    """(o, lse) [B, Hq, Sq, D], [B, Hq, Sq] in fp64; rows behind q_len are NaN."""
    B, Hq, Sq, D = q.shape
    Hkv, page = k_cache.shape[1:3]
    o = np.full((B, Hq, Sq, D), np.nan)
    lse = np.full((B, Hq, Sq), np.nan)
    for b in range(B):
        at = [(prefix_pages[j // page], j % page) for j in range(prefix_len)]
        at += [(tail_pages[b][j // page], j % page) for j in range(tail_len[b])]
        pg = np.array([x[0] for x in at], dtype=np.int64)
        sl = np.array([x[1] for x in at], dtype=np.int64)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = k_cache[pg, g, sl], v_cache[pg, g, sl]
            for i in range(q_len[b]):
                n = len(at) - q_len[b] + i + 1 if causal else len(at)
                n = min(max(n, 0), len(at))
                s = scale * (k[:n] @ q[b, h, i])
                m = s.max() if n else -np.inf
                e = np.exp(s - m)
                acc, tot = (e @ v[:n], e.sum()) if n else (np.zeros(D), 0.0)
                r = acc / tot if n else acc
                z = m + math.log(tot) if n else -np.inf
                if part_lse is not None and part_lse[b, h, i] != -np.inf:
                    both = np.logaddexp(z, part_lse[b, h, i])
                    r = r * math.exp(z - both) + part_o[b, h, i] * math.exp(part_lse[b, h, i] - both)
                    z = both
                o[b, h, i], lse[b, h, i] = r, z
    return o, lse

"""Oracle of block-sparse decoding, in fp64: the rotary append, the per-block key
bounds, the block selection and attention over the selected blocks.

TEST INFRASTRUCTURE: only tests/, __graft_entry__.smoke() and bench.py may use it.

Values are float64 arrays (exact copies of what the GPU reads); pools are
``[NB, Hkv, bs, D]``, bounds ``[NB, Hkv, 2, D]`` (largest, smallest).
"""

from __future__ import annotations

import math

import numpy as np

from .attention import attend


def _pairs(rot: int, interleaved: bool):
    half = rot // 2
    if interleaved:
        return np.arange(0, rot, 2), np.arange(1, rot, 2)
    return np.arange(half), np.arange(half, rot)


def rotate(x, cos_sin_rows, interleaved: bool, dtype=np.float64) -> np.ndarray:
    """Rows ``x [T, H, D]`` rotated by their table rows ``[T, rot]`` (cosines, then
    sines). With ``dtype`` float32 every product and sum is rounded on its own."""
    x = np.asarray(x, dtype=dtype)
    cs = np.asarray(cos_sin_rows, dtype=dtype)
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = _pairs(rot, interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotation_error(x, cos_sin_rows, interleaved: bool) -> np.ndarray:
    """Bound on |fp32 result - exact| of :func:`rotate`: each product and the sum
    is off by at most 2^-24 of itself."""
    x, cs = np.abs(np.asarray(x, np.float64)), np.abs(np.asarray(cos_sin_rows, np.float64))
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = _pairs(rot, interleaved)
    size = np.zeros_like(x)
    size[..., a] = x[..., a] * c + x[..., b] * s
    size[..., b] = x[..., b] * c + x[..., a] * s
    return size * (2.0**-23 + 2.0**-46) + 2.0**-148


def key_bounds(bounds, k_cache, block_tables, context_lens, new_tokens=None) -> np.ndarray:
    """``bounds`` with the rows of every touched block recomputed."""
    out = np.array(bounds, dtype=np.float64)
    bs = k_cache.shape[2]
    for s, n in enumerate(np.asarray(context_lens).tolist()):
        fresh = n if new_tokens is None else min(n, int(new_tokens[s]))
        if fresh == 0:
            continue
        for lb in range((n - fresh) // bs, -(-n // bs)):
            b = block_tables[s][lb]
            keys = k_cache[b][:, :min(bs, n - lb * bs)]
            out[b, :, 0], out[b, :, 1] = keys.max(axis=1), keys.min(axis=1)
    return out


def block_scores(q, bounds, table, n_blocks: int) -> np.ndarray:
    """``[Hkv, n_blocks]`` upper bounds on the sum of a group's logits for queries
    ``q [Hq, D]``: Q+ . max + Q- . min with the group's sums Q+ of the positive and Q-
    of the negative parts; finite scores are correctly rounded."""
    Hq, D = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    out = np.empty((Hkv, n_blocks))
    for h in range(Hkv):
        rows = q[h * G:(h + 1) * G]
        weight = np.stack([np.maximum(rows, 0).sum(0), np.minimum(rows, 0).sum(0)])
        for b in range(n_blocks):
            terms = (weight * bounds[table[b], h]).ravel()
            out[h, b] = math.fsum(terms) if np.isfinite(terms).all() else terms.sum()
    return out


def select_blocks(q, bounds, block_tables, context_lens, block_size: int, num_selected: int,
                  num_sink: int, num_recent: int) -> np.ndarray:
    """int32 ``[S, Hkv, num_selected]``: ascending logical blocks, -1 behind them."""
    S, Hkv = q.shape[0], bounds.shape[1]
    out = np.full((S, Hkv, num_selected), -1, np.int32)
    for s in range(S):
        n = -(-int(context_lens[s]) // block_size)
        if n <= num_selected:
            out[s, :, :n] = np.arange(n)
            continue
        score = block_scores(q[s], bounds, block_tables[s], n)
        nan = np.isnan(score)  # a NaN score counts as the best, above infinity
        score = np.where(nan, 0.0, score)
        index = np.arange(n)
        forced = (index < num_sink) | (index >= n - num_recent)
        for h in range(Hkv):
            free = index[~forced]
            order = free[np.lexsort((free, -score[h][free], ~nan[h][free]))]
            best = np.concatenate([index[forced], order[:num_selected - forced.sum()]])
            out[s, h] = np.sort(best)
    return out


def decode_sparse(q, k_cache, v_cache, block_tables, context_lens, selected, scale: float):
    """Attention of ``q [S, Hq, D]`` over the listed blocks; float64 ``[S, Hq, D]``."""
    S, Hq, D = q.shape
    Hkv, bs = k_cache.shape[1:3]
    G = Hq // Hkv
    out = np.zeros((S, Hq, D))
    for s in range(S):
        for h in range(Hkv):
            K, V = listed(k_cache, v_cache, block_tables[s], int(context_lens[s]),
                          selected[s, h], h)
            out[s, h * G:(h + 1) * G] = attend(q[s, h * G:(h + 1) * G], K, V, scale)
    return out


def listed(k_cache, v_cache, table, ctx: int, blocks, h: int):
    """Keys and values of the listed blocks' tokens below ``ctx``, in list order."""
    bs, D = k_cache.shape[2:]
    K, V = [np.empty((0, D))], [np.empty((0, D))]
    for lb in blocks:
        if lb < 0:
            continue
        n = min(bs, ctx - int(lb) * bs)
        K.append(k_cache[table[lb], h, :n])
        V.append(v_cache[table[lb], h, :n])
    return np.concatenate(K), np.concatenate(V)


def decode_error(q, k_cache, v_cache, block_tables, context_lens, selected, scale: float,
                 p_half_step: float, p_floor: float = 2.0**-25) -> np.ndarray:
    """Bound on |fp32 kernel - exact| before the output's own rounding, ``[S, Hq, D]``.

    A logit is a sum of D fp32 products, off by at most dz = (D + 4) 2^-23 of the sum
    of its terms' sizes (2^-23: a tensor core may cut instead of round), plus 2^-22 of
    1 + |z| for the scaling, the subtraction and exp2. A weight e^z is then off by a
    relative 2 dz or less (its own logit and the maximum's), plus ``p_half_step`` when
    it is rounded for the second product; the same 2 dz stands in the denominator. The
    second product and the merge add 2^-22 per accumulated term's share, below
    2^-15 for 2^7 terms in a row. A weight below fp16's normal range is off by
    ``p_floor`` of the largest: 2^-25, or less where the largest is more than 1."""
    S, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    out = np.zeros((S, Hq, D))
    for s in range(S):
        for h in range(Hkv):
            K, V = listed(k_cache, v_cache, block_tables[s], int(context_lens[s]),
                          selected[s, h], h)
            if not len(K):
                continue
            rows = q[s, h * G:(h + 1) * G]
            z = scale * rows @ K.T
            dz = (abs(scale) * np.abs(rows) @ np.abs(K).T).max(1) * (D + 4) * 2.0**-23
            dz = dz + (1 + np.abs(z).max(1)) * 2.0**-22
            p = np.exp(z - z.max(1, keepdims=True))
            size = p @ np.abs(V) / p.sum(1, keepdims=True)
            rel = 4 * dz[:, None] + p_half_step + 2.0**-15
            out[s, h * G:(h + 1) * G] = size * rel + len(K) * p_floor * np.abs(V).max(0)
    return out

"""Plain fp64 definitions of the steps beyond plain causal attention (test infrastructure
only): rotary positions of several axes, attention under score rules, and the verdict on
drafted tokens.

* ``norm_rope_append_axes``  the append, frequency i turned by the position of its axis.
* ``scored_attention``       softmax attention with a tanh cap, a bias by distance, and a
                             visible interval of keys per row.
* ``verify_drafts``          accepted drafts and the token that follows, in whole numbers.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from .reference import _gather_rows, bf16_bits_to_f64, f64_to_bf16_bits, rms_norm, rope_neox

DRAFT_UNIT = 44                                # probabilities count as multiples of 2^-44


def norm_rope_append_axes(q, k, v, positions, freq_axes, slot_mapping, gamma_q, gamma_k,
                          theta, eps, k_cache, v_cache, block_size):
    """positions int [axes, T], freq_axes [D // 2]; returns (q_hat_bits, k_cache, v_cache)."""
    eps64, theta64 = np.float64(np.float32(eps)), np.float64(np.float32(theta))
    axes = np.asarray(list(freq_axes))
    dims = np.concatenate([axes, axes])

    def turned(x, gamma):
        y = rms_norm(bf16_bits_to_f64(x), bf16_bits_to_f64(gamma), eps64)
        out = np.empty_like(y)
        for a in range(len(positions)):
            r = rope_neox(y, np.asarray(positions[a], np.int64)[:, None], theta64)
            out[..., dims == a] = r[..., dims == a]
        return f64_to_bf16_bits(out)

    q_bits, k_bits = turned(q, gamma_q), turned(k, gamma_k)
    kc, vc = (np.array(x, dtype=np.uint16, copy=True) for x in (k_cache, v_cache))
    for t, s in enumerate(np.asarray(slot_mapping, np.int64).tolist()):
        if 0 <= s < kc.shape[0] * block_size:
            kc[s // block_size, s % block_size] = k_bits[t]
            vc[s // block_size, s % block_size] = v[t]
    return q_bits, kc, vc


def visible(p, seq_len, window=0, first_key=0, prefix_len=0):
    """Keys [lo, hi) that a row at position p of a sequence of seq_len keys sees.

    first_key bounds from below alone: of the documents after a row's own the causal bound
    p + 1 keeps it, which a prefix_len past its document's end lifts.
    """
    lo = max(0, first_key, p - window + 1 if window > 0 else 0)
    hi = max(p + 1, min(prefix_len, seq_len))
    return lo, max(lo, hi)


def scored_attention(q, k_cache, v_cache, block_tables, seq_lens, block_size, q_lens, *,
                     scale=None, softcap=0.0, window=0, slopes=None, first_keys=None,
                     prefix_lens=None, seqs=None):
    """q: uint16 [rows, Hq, D], the sequences' new tokens packed back to back.

    Returns (out float64 [rows, Hq, D], lse [rows, Hq]); rows of sequences outside `seqs`
    are NaN.
    """
    qf = bf16_bits_to_f64(q)
    R, Hq, D = qf.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.full((R, Hq, D), np.nan), np.full((R, Hq), np.nan)
    row = 0
    for b, n in enumerate(q_lens):
        rows = range(row, row + n)
        row += n
        if seqs is not None and b not in seqs:
            continue
        L = int(seq_lens[b])
        for t, r in enumerate(rows):
            p = L - n + t
            lo, hi = visible(p, L, window, 0 if first_keys is None else int(first_keys[r]),
                             0 if prefix_lens is None else int(prefix_lens[b]))
            keys = np.arange(lo, hi, dtype=np.int64)
            for g in range(Hkv):
                heads = slice(g * G, (g + 1) * G)
                if hi <= lo:
                    out[r, heads], lse[r, heads] = 0.0, -np.inf
                    continue
                K = _gather_rows(k_cache, block_tables[b], keys, block_size, g)
                V = _gather_rows(v_cache, block_tables[b], keys, block_size, g)
                s = scale * (qf[r, heads] @ K.T)
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - np.asarray(slopes, np.float64)[heads, None] * np.abs(p - keys)
                m = s.max(axis=1, keepdims=True)
                w = np.exp(s - m)
                l = w.sum(axis=1, keepdims=True)
                out[r, heads] = (w @ V) / l
                lse[r, heads] = (m + np.log(l))[:, 0]
    return out, lse


def verify_drafts(target, draft, tokens, uniforms, lens=None):
    """target [B, K + 1, V], draft [B, K, V] or None (float64, any values), tokens [B, K],
    uniforms [B, K + 1].  Returns (tokens [B, K + 1], accepted [B])."""
    B, K1, V = target.shape
    K = K1 - 1
    out, accepted = np.full((B, K1), -1, np.int64), np.zeros(B, np.int64)

    def counted(x):                            # above 1 as 1, NaN and negative ones as 0
        with np.errstate(invalid="ignore"):
            return np.where(x > 0, np.minimum(x, 1.0), 0.0)

    def units(row):
        return np.rint(np.ldexp(counted(row), DRAFT_UNIT)).astype(np.int64)

    for b in range(B):
        n = K if lens is None else min(max(int(lens[b]), 0), K)
        j = 0
        while j < n:
            x = int(tokens[b, j])
            if not 0 <= x < V:
                break
            qx = 1.0 if draft is None else float(counted(draft[b, j, x]))
            px, u = float(counted(target[b, j, x])), float(uniforms[b, j])
            if not np.isfinite(u):
                if not u * qx < px:
                    break
            elif not Fraction(u) * Fraction(qx) < Fraction(px):
                break
            j += 1
        p = units(target[b, j])
        w = p
        if j < n:
            if draft is None:
                w = p.copy()
                if 0 <= int(tokens[b, j]) < V:
                    w[int(tokens[b, j])] = 0
            else:
                w = np.maximum(p - units(draft[b, j]), 0)
            if not w.any():
                w = p
        out[b, :j] = tokens[b, :j]
        accepted[b] = j
        cum = np.cumsum(w.astype(np.uint64))
        total = int(cum[-1])
        if total == 0:
            continue
        u = float(uniforms[b, K])
        u = 0.0 if np.isnan(u) else u
        at = min(max(int(Fraction(u) * total), 0), total - 1) if np.isfinite(u) else \
            (total - 1 if u > 0 else 0)
        out[b, j] = int(np.searchsorted(cum, np.uint64(at), side="right"))
    return out, accepted

"""Oracle for latent attention over a paged cache of shared latent vectors.

TEST INFRASTRUCTURE.  Only the tests and the smoke check may import this
module; the library never does, and this module imports nothing from it.

A cached row is [c_t (512) ; r_t (64)], one a token, shared by the heads.
Packed tensors hold the sequences one after the other.  Query i of sequence b
sits at position L_b - q_lens[b] + i and sees positions 0 .. that one.

Every attention returns (out, tol_base, tol_scores), the last two for
tolerances: tol_base[row] = sum_t p_t |v_t| per output value, what a relative
error of the weights is multiplied by; tol_scores[row] = the largest sum of
absolute products of a score, what a relative error of the products is
multiplied by.
"""

from __future__ import annotations

import numpy as np

from .prefill import cu_lens

LATENT = 512


def latent_rows(pages, block_table, b, L):
    """The cached rows [L][576] of sequence b, float64."""
    S = pages.shape[1]
    t = np.arange(L)
    return np.asarray(pages[block_table[b, t // S], t % S], np.float64)


def latent_append(pages, c_new, r_new, block_table, seq_lens, q_lens):
    """A new pool with the step's rows written."""
    out = pages.copy()
    S = pages.shape[1]
    cu = cu_lens(q_lens)
    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), int(q_lens[b])
        for i in range(n):
            pos = L - n + i
            out[block_table[b, pos // S], pos % S] = np.concatenate([c_new[cu[b] + i],
                                                                     r_new[cu[b] + i]])
    return out


def latent_gather(pages, block_table, seq_lens):
    """Packed rows [Tk][576] of every sequence."""
    parts = [pages[block_table[b, np.arange(L) // pages.shape[1]], np.arange(L) % pages.shape[1]]
             for b, L in enumerate(int(x) for x in seq_lens)]
    return np.concatenate(parts) if parts else np.zeros((0, pages.shape[2]), pages.dtype)


def _attend(q, k, v, scale, seen):
    """q [n][dk] over k [L][dk], v [L][dv]; seen [n][L]."""
    s = np.where(seen, (q @ k.T) * scale, -np.inf)
    size = (np.abs(q) @ np.abs(k).T * scale * seen).max(axis=1, initial=0.0)
    m = s.max(axis=1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = p.sum(axis=1, keepdims=True)
    w = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    return w @ v, w @ np.abs(v), size


def latent_attention(q, pages, block_table, seq_lens, q_lens, scale, bad_pages=()):
    """Absorbed form.  q [T][H][576]; tokens of a page in bad_pages, given as
    (sequence, entry of its table), are left out."""
    T, H, _ = q.shape
    out, base, size = np.zeros((T, H, LATENT)), np.zeros((T, H, LATENT)), np.zeros((T, H))
    cu = cu_lens(q_lens)
    S = pages.shape[1]
    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), int(q_lens[b])
        if n == 0:
            continue
        table = block_table.copy()
        ok = np.ones(L, bool)
        for (bb, j) in bad_pages:
            if bb == b:
                table[b, j] = 0
                ok[j * S:(j + 1) * S] = False
        z = latent_rows(pages, table, b, L)
        z = np.where(ok[:, None], z, 0.0)
        for i in range(n):
            seen = np.broadcast_to(ok & (np.arange(L) <= L - n + i), (H, L))
            r = cu[b] + i
            out[r], base[r], size[r] = _attend(np.asarray(q[r], np.float64), z, z[:, :LATENT],
                                               scale, seen)
    return out, base, size


def latent_prefill(q, k, k_rope, v, seq_lens, q_lens, scale):
    """Expanded form.  q [T][H][D + 64], k and v [Tk][H][D], k_rope [Tk][64]."""
    T, H, _ = q.shape
    D = v.shape[2]
    out, base, size = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H))
    cq, ck = cu_lens(q_lens), cu_lens(seq_lens)
    for b in range(len(seq_lens)):
        L, n = int(seq_lens[b]), int(q_lens[b])
        rows, toks = slice(cq[b], cq[b] + n), slice(ck[b], ck[b] + L)
        seen = np.arange(L)[None] <= L - n + np.arange(n)[:, None]
        for h in range(H if n else 0):
            kk = np.concatenate([k[toks, h], k_rope[toks]], 1).astype(np.float64)
            out[rows, h], base[rows, h], size[rows, h] = _attend(
                np.asarray(q[rows, h], np.float64), kk, np.asarray(v[toks, h], np.float64), scale,
                seen)
    return out, base, size

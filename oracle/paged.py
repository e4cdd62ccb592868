"""fp64 oracle of rotary positions, the paged cache's append and the attention over it.

TEST INFRASTRUCTURE ONLY: the product never calls this.  Everything is written from the
definitions, one token or one sequence at a time: rotations as complex numbers, pages
looked up key by key, and the attention of a sequence by ``reference.forward`` on its
gathered keys and values.
"""
from __future__ import annotations

import numpy as np
import torch

from . import reference as ref


def rotate(x, positions, inv_freq, sections=None, interleaved=False, inverse=False):
    """x [tokens, H, D] (fp64), positions [axes, tokens] -> the rotated x."""
    x = np.array(ref.to_f64(x))
    inv_freq = ref.to_f64(inv_freq)
    n = len(inv_freq)
    sections = (n,) if sections is None else sections
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = np.asarray(positions, dtype=np.float64)[axis].T * inv_freq  # [tokens, n]
    turn = np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    re, im = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = (x[..., re] + 1j * x[..., im]) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return x


def slots(page_table, seq_len, q_start, page_size):
    """For each token row of a sequence: (row, sequence, key index, page, slot)."""
    out = []
    for b in range(len(seq_len)):
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            key = seq_len[b] - n + i
            out.append((q_start[b] + i, b, key, page_table[b][key // page_size], key % page_size))
    return out


def gather(cache, pages, length, scale=1.0):
    """[length, H_kv, D] fp64 of one sequence's pages (cache [n_pages, page_size, H_kv, D])."""
    page_size = cache.shape[1]
    index = np.arange(length)
    rows = np.asarray(pages)[index // page_size] if length else np.zeros(0, dtype=int)
    return ref.to_f64(cache[torch.as_tensor(rows), torch.as_tensor(index % page_size)]) * scale


def attend(q, k_cache, v_cache, page_table, seq_len, q_start, causal, scale, k_scale=1.0, v_scale=1.0):
    """(o [tokens, H_q, D], lse [H_q, tokens], a, f [tokens, H_q, D]) with a = P |V|, the scale in o of the
    weights' relative errors, and f = max_j P_j x sum of the visible |V|, that of errors of a fixed part of the
    largest weight; rows of no sequence are NaN."""
    T, H_q, D = q.shape
    o = np.full((T, H_q, D), np.nan)
    a = np.full((T, H_q, D), np.nan)
    f = np.full((T, H_q, D), np.nan)
    lse = np.full((H_q, T), np.nan)
    for b in range(len(seq_len)):
        r = slice(q_start[b], q_start[b + 1])
        n = q_start[b + 1] - q_start[b]
        if n == 0:
            continue
        if seq_len[b] == 0:
            o[r], a[r], f[r], lse[:, r] = 0.0, 0.0, 0.0, -np.inf
            continue
        k = gather(k_cache, page_table[b], seq_len[b], k_scale)[None]
        v = gather(v_cache, page_table[b], seq_len[b], v_scale)[None]
        ob, lb = ref.forward(q[r][None], k, v, causal, scale)
        ab, _ = ref.forward(q[r][None], k, np.abs(v), causal, scale)
        o[r], a[r], lse[:, r] = ob[0], ab[0], lb[0]
        seen = ref.visible(n, seq_len[b], causal)
        for h in range(H_q):
            g = h // (H_q // k.shape[2])
            s = np.where(seen, scale * (ref.to_f64(q[r, h]) @ k[0, :, g].T), -np.inf).max(axis=1)
            top = np.where(np.isneginf(s), 0.0, np.exp(np.where(np.isneginf(s), 0.0, s) - np.where(np.isneginf(s), 0.0, lb[0, h])))
            f[r, h] = top[:, None] * (seen.astype(float) @ np.abs(v[0, :, g]))
    return o, lse, a, f

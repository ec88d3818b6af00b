"""fp64 definitions of the beam-decoding step (numpy): norm and rotation of
heads, selection of continuations, reordering of page tables. Test
infrastructure, like the rest of this package; pinned by tests/test_beam_step.py.
"""
from __future__ import annotations

import numpy as np

PAGE = 256


def rope_rows(x, positions, inv_freq, rotary_dim, interleaved=False, weight=None, eps=1e-6) -> np.ndarray:
    """x [tokens, heads, 128] (values) -> normalised and rotated rows, fp64."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out = y.copy()
    half = rotary_dim // 2
    for j in range(half):
        t = np.asarray(positions, np.float64) * np.float64(inv_freq[j])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        p, q = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        out[..., p] = y[..., p] * c - y[..., q] * s
        out[..., q] = y[..., p] * s + y[..., q] * c
    return out


def pair_size(y, rotary_dim, interleaved=False) -> np.ndarray:
    """|a| + |b| of each value's pair (its own magnitude where it is not rotated):
    what the rounding errors of a rotated value are proportional to."""
    a = np.abs(np.array(y, np.float64))
    out = a.copy()
    half = rotary_dim // 2
    for j in range(half):
        p, q = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        out[..., p] = out[..., q] = a[..., p] + a[..., q]
    return out


def beam_select(logits, scores, num_select, finished=None, eos=-1):
    """One group: logits [W, V], scores [W] -> (tokens, parents, values), the
    num_select best in order. Values are fp64."""
    W, V = logits.shape
    every = []
    for w in range(W):
        score = -np.inf if np.isnan(scores[w]) else float(scores[w])
        if finished is not None and finished[w]:
            order = [eos] + [t for t in range(min(V, num_select + 1)) if t != eos]
            value = [score] + [-np.inf] * (len(order) - 1)
        else:
            x = np.array(logits[w], np.float64)
            x[np.isnan(x)] = -np.inf
            x = np.minimum(x, np.float64(np.finfo(np.float32).max))
            top = x.max()
            with np.errstate(invalid="ignore"):
                lse = top if top == -np.inf else top + np.log(np.exp(x - top).sum())
                order = np.lexsort((np.arange(V), -x))[:num_select]
                value = score + (x[order] - lse)
            value = np.where(np.isnan(value), -np.inf, value)
        every += [(-v, w, rank, int(t)) for rank, (t, v) in enumerate(zip(order, value))]
    every.sort()
    best = every[:num_select]
    return (np.array([e[3] for e in best], np.int32), np.array([e[1] for e in best], np.int32),
            np.array([-e[0] for e in best], np.float64))


def beam_reorder(block_table, seq_lens, parents, beam_width):
    """(new table, copies): rows of a new table and the copies [(from page, to
    page, rows)] that its tail pages need."""
    new = np.array(block_table)
    copies = []
    for r0 in range(0, len(seq_lens), beam_width):
        T = int(seq_lens[r0])
        full, rem = divmod(T, PAGE)
        p = [int(v) for v in parents[r0:r0 + beam_width]]
        childless = [b for b in range(beam_width) if b not in p]
        seen = set()
        for i, parent in enumerate(p):
            owner = parent if parent not in seen else childless.pop(0)
            new[r0 + i, :full] = block_table[r0 + parent, :full]
            new[r0 + i, full:] = block_table[r0 + owner, full:]
            if parent in seen and rem:
                copies.append((int(block_table[r0 + parent, full]), int(block_table[r0 + owner, full]), rem))
            seen.add(parent)
    return new, copies

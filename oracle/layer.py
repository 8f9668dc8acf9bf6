"""The layer around the indexer (oracle side; test infrastructure), in fp64.

Only tests/ use this module; the CUDA path shares no code with it.

* RMS norm with the residual's addition, and its E4M3 rows with one scale per row or per 128 values.
* The paged latent cache: which row holds a position, and what the append writes there ("Study MLA Indexer",
  section 数学流 and the 两条 cache 区分 table: the latent c^KV, d_c = 512 per token, beside the rotated key part).
* Attention in the latent's space (the same section: an MQA whose keys and values are the cached latents),
  over a selection or over every position below a length.
"""

from __future__ import annotations

import numpy as np

from .fp8_e4m3 import E4M3_MAX, e4m3_encode
from .rope import rope_rows


def rmsnorm(x, weight, eps, residual=None):
    """fp64 (s = x + residual, y = s / sqrt(mean s^2 + eps) * weight)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    return s, s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def group_scales(y, group):
    """absmax / 448 of every group of y's values (group 0: of every row), 1 for groups of zeros."""
    step = group or y.shape[1]
    amax = np.stack([np.abs(y[:, i:i + step]).max(1) for i in range(0, y.shape[1], step)], 1)
    return np.where(amax > 0, amax / E4M3_MAX, 1.0)


def pow2_scale(amax):
    """The smallest power of two s >= 2^-100 with amax <= 448 s (1 for 0)."""
    if amax == 0:
        return 1.0
    s = 2.0 ** -100
    while s * E4M3_MAX < amax:
        s *= 2.0
    return s


def page_row(table, page_size, num_pages, seq, pos):
    """Cache row of position pos of sequence seq, or -1 where the page table has none."""
    if not 0 <= seq < table.shape[0] or pos < 0 or pos // page_size >= table.shape[1]:
        return -1
    page = int(table[seq, pos // page_size])
    return page * page_size + pos % page_size if 0 <= page < num_pages else -1


def append_values(c, kr, positions, fp8, rope_dim, base, interleaved):
    """(latents: values, or codes where fp8; scales; rotated key parts in fp64) of n tokens."""
    c = np.asarray(c, np.float64)
    rot = rope_rows(kr, positions, rope_dim, base, interleaved)
    if not fp8:
        return c, None, rot
    scale = np.array([pow2_scale(a) for a in np.abs(c).max(1)])
    return e4m3_encode(c / scale[:, None]), scale, rot


def attend(q, keys, d_c, sm_scale):
    """q [H, d], keys [n, d]: out [H, d_c], lse [H], sum of |weight * value| [H, d_c], and the largest
    sum over a dot product's terms' magnitudes, times the scale."""
    H = q.shape[0]
    if len(keys) == 0:
        return np.zeros((H, d_c)), np.full(H, -np.inf), np.zeros((H, d_c)), 0.0
    s = q @ keys.T * sm_scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(1, keepdims=True)
    w = p / total
    mags = float((np.abs(q) @ np.abs(keys).T).max() * abs(sm_scale))
    return w @ keys[:, :d_c], (m + np.log(total))[:, 0], w @ np.abs(keys[:, :d_c]), mags

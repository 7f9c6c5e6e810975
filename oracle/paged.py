"""CPU oracle for the paged cache of keys and values and the attention of new
tokens over it -- TEST INFRASTRUCTURE ONLY.

Only the tests may use this module. The product path never imports or calls
it, and shares no code with it.

* position p of sequence b is row p % page_size of page table[b, p // page_size];
  an entry outside [0, pages) is a page that the sequence does not have;
* a 4-bit row of x: low = bf16(min x), step = bf16((max x - low) / 15), 0 below
  2^-60, code = clamp(rint((x - low) / step), 0, 15); it reads low + step code;
* the query at position p sees key j iff j <= p, and j >= p - left (left >= 0)
  or j < sinks, and the sequence has j's page;
  O = sum softmax(scale q.k) v, LSE = ln sum exp(scale q.k).

Plain definitions in float64, one sequence, query and head at a time.
"""

from __future__ import annotations

import numpy as np

from oracle.sel_attn import round_bf16

__all__ = ["place", "quantise", "attend"]

LEAST_STEP = 2.0 ** -60


def place(table_row, position, page_size, pages):
    """(page, row) of a position of a sequence, or None."""
    col = position // page_size
    if position < 0 or col >= len(table_row) or not 0 <= table_row[col] < pages:
        return None
    return int(table_row[col]), position % page_size


def quantise(x):
    """Codes, step and low of every row of x [..., D]."""
    x = np.asarray(x, np.float64)
    low = round_bf16(x.min(-1, keepdims=True)).astype(np.float64)
    step = round_bf16((x.max(-1, keepdims=True) - low) / 15).astype(np.float64)
    step = np.where(step >= LEAST_STEP, step, 0.0)
    code = np.clip(np.rint((x - low) / np.where(step > 0, step, 1.0)), 0, 15)
    return np.where(step > 0, code, 0.0), step, low


def attend(q, keys, values, present, positions, left, sinks, scale):
    """One sequence. q [M, H, D]; keys, values [N, G, D] of positions 0 .. N - 1;
    present [N]: whether the sequence has the page. Returns O [M, H, D], LSE
    [H, M], sum p |v| [M, H, D] and the number of keys seen [M]."""
    q = np.asarray(q, np.float64)
    M, H, D = q.shape
    N, G, _ = keys.shape
    o, mag, lse = np.zeros((M, H, D)), np.zeros((M, H, D)), np.full((H, M), -np.inf)
    seen = np.zeros(M, np.int64)
    j = np.arange(N)
    for m in range(M):
        p = int(positions[m])
        if p < 0:
            continue
        see = present & (j <= p)
        if left >= 0:
            see &= (j >= p - left) | (j < sinks)
        seen[m] = see.sum()
        if not seen[m]:
            continue
        for h in range(H):
            g = h // (H // G)
            s = keys[see, g].astype(np.float64) @ q[m, h] * scale
            top = s.max()
            e = np.exp(s - top)
            v = values[see, g].astype(np.float64)
            o[m, h] = e @ v / e.sum()
            mag[m, h] = e @ np.abs(v) / e.sum()
            lse[h, m] = top + np.log(e.sum())
    return o, lse, mag, seen

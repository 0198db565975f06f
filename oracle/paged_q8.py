"""The 8-bit paged cache (oracle; test infrastructure only).

Codes are e4m3 values (float64 arrays here, NaN for the NaN code) in the cache
shape [H][n_pages * page_size][D]; scales are float64 [H][rows / G]: row r of head
h stands for codes[h, r] * scales[h, r // G].

A call appends runs of consecutive tokens. For each head and each block of G rows
that a run touches:
    a    = the largest finite |x| of the run's tokens there,
    need = the smallest power of two >= 2^-126 with a / need <= 448,
    s    = need if the run covers the block's first row, else max(need, held),
           a held scale that is no power of two being rounded up to one and one
           that is not finite and positive counting as 0,
and the rows before the run become round(code * held / s), the run's round(x / s)
clamped to +-448. Slot 0 is skipped; invalid tokens are skipped and reported as in
paged_kv.kv_append.
"""
from __future__ import annotations

import numpy as np

from .paged_kv import _checked_row

E4M3_MAX = 448.0
ERR_ORDER = 32


def round_e4m3(x):
    """Nearest e4m3 value, ties to even, clamped to +-448; NaN stays NaN. The
    spacing is 2^(e-3) in [2^e, 2^(e+1)) down to e = -6 and 2^-9 below."""
    x = np.clip(np.asarray(x, np.float64), -E4M3_MAX, E4M3_MAX)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))    # |x| = m 2^e, m in [0.5, 1)
        step = np.ldexp(1.0, e - 1 - 3)
        return np.rint(x / step) * step


def pow2_at_least(v: float) -> float:
    """Smallest power of two in [2^-126, 2^126] that is >= v (2^126 if none)."""
    m, e = np.frexp(max(float(v), 0.0))
    k = -126 if m == 0 else (e - 1 if m == 0.5 else e)
    return float(np.ldexp(1.0, int(min(max(k, -126), 126))))


def need_scale(a: float) -> float:
    return pow2_at_least(a / E4M3_MAX)


def _append_run(codes, scales, x, h, row, first, G):
    """x: [n][D] tokens for the rows row .. row + n - 1 of one block."""
    blk = row // G
    finite = np.isfinite(x)
    a = float(np.abs(x[finite]).max()) if finite.any() else 0.0
    held = float(scales[h, blk]) if first else 0.0
    if not (0.0 < held < np.inf):
        held = 0.0
    s = need_scale(a)
    if held > 0:
        s = max(s, pow2_at_least(held))
    if first and s != scales[h, blk]:
        old = codes[h, row - first:row]
        codes[h, row - first:row] = round_e4m3(old * (held / s))
    scales[h, blk] = s
    codes[h, row:row + len(x)] = round_e4m3(x / s)


def kv_append_q8(codes, scales, x, table, batch_idx, input_pos, page_size, n_pages, G) -> int:
    """Appends x ([N][H][D] float64) in place; returns the OR of error bits. The
    call's tokens must be in order (runs of consecutive positions)."""
    N, H, _ = x.shape
    slots = np.arange(N) if batch_idx is None else np.asarray(batch_idx)
    pos = np.asarray(input_pos)
    err, i = 0, 0
    while i < N:
        n = 1
        while (i + n < N and slots[i + n] == slots[i] and pos[i + n] == pos[i] + n
               and pos[i] >= 0 and (pos[i] + n) % G):
            n += 1
        if slots[i] != 0:
            row, e = _checked_row(table, int(slots[i]), int(pos[i]), page_size, n_pages)
            err |= e
            if row is not None:
                for h in range(H):
                    _append_run(codes, scales, x[i:i + n, h], h, row, int(pos[i]) % G, G)
        i += n
    return err


def dequantise(codes, scales, G):
    return codes * np.repeat(scales, G, axis=1)[:, :, None]

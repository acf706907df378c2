"""The paged 8-bit KV cache operators (oracle; test infrastructure).

Plain float64 / integer restatements of the definitions in include/ssv.h:
tables of a pass from the requests' lengths (``page_plan``), the head norm
with the RoPE-copy rotation (``norm_rope_batch``; SimSD summary, section 3
"Position Encoding Alignment"), the quantising commit (``commit_pages``;
section 4 "Speculative decoding pipeline") and the gather of a sequence's
cached rows from its pages (``gather_cache``) for ``oracle.attention``.
"""
from __future__ import annotations

import math

import numpy as np

from .commit import committed_rows
from .rope import rope_copy_batch

SCALE_MIN = -100


# ---------------------------------------------------------------------------
# e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f / 0xff are NaN
# ---------------------------------------------------------------------------
def _code_values() -> np.ndarray:
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = -v if c & 0x80 else v
    out[0x7F] = out[0xFF] = np.nan
    return out


E4M3 = _code_values()


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    return E4M3[np.asarray(codes, np.uint8)]


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code (ties to the even mantissa); |x| <= 448, non-finite to NaN."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert a.size == 0 or a.max() <= 448
    pos = E4M3[:0x7F]                                   # 0 .. 448, increasing
    i = np.clip(np.searchsorted(pos, a), 1, 0x7E)       # pos[i - 1] <= a <= pos[i]
    lo, hi = pos[i - 1], pos[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    c = np.where(up, i, i - 1).astype(np.uint8)
    c = c | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isfinite(x), c, 0x7F).astype(np.uint8)


def scale_for(amax: float) -> float:
    """Smallest power of two 2^e, e >= SCALE_MIN, with amax <= 448 * 2^e."""
    if amax <= 0:
        return 2.0 ** SCALE_MIN
    e = math.floor(math.log2(amax / 448)) - 2
    while e < SCALE_MIN or amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------
def page_plan(cache_len, new_len, block, held, pages, free_list, n_free, page_size, total_rows):
    """One request at a time; returns a dict of the outputs and the set of
    errors met."""
    batch, max_pages = pages.shape
    pages, free_list = pages.copy(), free_list.copy()
    errors = set()
    if not 0 <= n_free <= len(free_list):
        n_free = 0
        errors.add("invalid")
    stack = list(free_list[:n_free])
    held_out = np.array(held).copy()
    live = []
    for b in range(batch):
        if cache_len[b] < 0:
            if 0 <= held[b] <= max_pages:
                stack += list(pages[b, : held[b]])
                held_out[b] = 0
            else:
                errors.add("invalid")
    if len(stack) > len(free_list):
        stack = stack[: len(free_list)]
        errors.add("invalid")
    seqs = np.zeros((batch, 6), np.int32)
    slot_off = np.zeros(batch, np.int32)
    slot_map = np.full(total_rows, -1, np.int32)
    q = t = 0
    dry = False
    for b in range(batch):
        C, N, B = int(cache_len[b]), int(new_len[b]), int(block[b])
        seqs[b] = (0, 0, 0, q, b * max_pages, t)
        slot_off[b] = t
        if C < 0:
            continue
        need = -(-(C + N + B) // page_size)
        if N < 0 or not 1 <= B <= 64 or not 0 <= held[b] <= max_pages or need > max_pages:
            errors.add("invalid")
            continue
        q0 = q
        q, t = q + N + 2 * B, t + B
        if q > total_rows:
            errors.add("invalid")
            continue
        want = max(need - int(held[b]), 0)
        if want and (dry or want > len(stack)):
            dry = True
            errors.add("no pages")
            continue
        for j in range(want):
            pages[b, held[b] + j] = stack.pop()
        held_out[b] = held[b] + want
        live.append(b)
        seqs[b, :3] = (C, N, B)
        for j in range(N + B):
            tok = C + j
            slot_map[q0 + j] = pages[b, tok // page_size] * page_size + tok % page_size
    free_list[n_free:len(stack)] = stack[n_free:]
    return dict(seqs=seqs, slot_off=slot_off, slot_map=slot_map, held=held_out, n_free=len(stack), pages=pages,
                free_list=free_list), errors


# ---------------------------------------------------------------------------
# head norm and rotation
# ---------------------------------------------------------------------------
def rms_norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def norm_rope_batch(seqs, q, k, q_weight, k_weight, base=10000.0, eps=1e-6, positions=None):
    return rope_copy_batch(seqs, rms_norm(q, q_weight, eps), rms_norm(k, k_weight, eps), base, positions)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def gather_cache(seq, pages, codes, scale):
    """float64 [C, Hkv, d]: the cached rows of one sequence."""
    ps, C = codes.shape[2], int(seq[0])
    out = np.empty((C, codes.shape[1], codes.shape[3]))
    for t in range(C):
        p = pages[int(seq[4]) + t // ps]
        out[t] = e4m3_values(codes[p, :, t % ps]) * scale[p].astype(np.float64)[:, None]
    return out


def commit_pages(seqs, pages, tau_all, n_acc, fresh, codes, scale, cache_len=None):
    """Appends rows of `fresh` (float64 [rows, Hkv, d]) to one of K / V;
    returns (codes, scale, new_len).  Idle records keep their length, that of
    `cache_len` where it is given."""
    codes, scale = codes.copy(), scale.copy()
    ps = codes.shape[2]
    new_len = np.zeros(len(seqs), np.int64)
    for b, s in enumerate(np.asarray(seqs)):
        C, N, B, q_off, kv, t_off = (int(v) for v in s)
        if N == 0 and B == 0:
            new_len[b] = C if cache_len is None else cache_len[b]
            continue
        rows = committed_rows(N, B, tau_all[t_off:t_off + B], int(n_acc[b]))
        new_len[b] = C + len(rows)
        by_page = {}
        for j, r in enumerate(rows):
            by_page.setdefault((C + j) // ps, []).append((C + j, r))
        for j, items in by_page.items():
            p, first = pages[kv + j], items[0][0] % ps
            for h in range(codes.shape[1]):
                x = np.stack([fresh[q_off + r, h] for _, r in items])
                fin = np.abs(x[np.isfinite(x)])
                new = scale_for(float(fin.max()) if fin.size else 0.0)
                if first > 0:
                    old = float(scale[p, h])
                    new = max(old, new)
                    if new > old:
                        codes[p, h, :first] = e4m3_codes(e4m3_values(codes[p, h, :first]) * (old / new))
                for (t, _), row in zip(items, x):
                    codes[p, h, t % ps] = e4m3_codes(row / new)
                scale[p, h] = new
    return codes, scale, new_len

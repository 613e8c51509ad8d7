"""Runs of new tokens over a page-scaled 8-bit cache: page maps, quantized append and causal attention, in float64.

Plain statements of ``kvq_map_runs``, ``kvq_append_runs`` and ``kvq_attn_runs`` as include/kvq.h defines them: one request, one
page, one row at a time.  (No counterpart on the source pages: they quantize per token.)
"""
from __future__ import annotations

import math

import numpy as np

from .encoders import e4m3_bits_rne_satfinite, e4m3_value

__all__ = ["PAGE", "MAX_PAGE", "E_MIN", "E_MAX", "QMAX", "map_runs", "page_exponent", "encode", "values", "append_runs", "attend"]

PAGE = 16
MAX_PAGE = (1 << 27) - 1  # the last page whose slots 16 page .. fit 31 bits
E_MIN, E_MAX = -24, 15
QMAX = {"e4m3p": 448.0, "int8p": 127.0}


def map_runs(new_lens, seq_lens, stack, count, table, max_rows, kept=None, held=None):
    """-> dict(ok, run_starts, seq_lens, count, stack, table, slots, positions, held); inputs are not changed.  kept: per request
    the first pages that do not go back when it is finished; held: the pages that it has (None: those of its length)."""
    B, width = table.shape
    stack, table = list(stack), table.copy()
    pages = [-(-n // PAGE) for n in seq_lens]
    held = pages if held is None else [int(h) for h in held]
    out = dict(held=np.array(held, dtype=int), run_starts=np.zeros(B + 1, int), seq_lens=np.array(seq_lens), count=count, stack=np.array(stack), table=table,
               slots=np.full(max_rows, -1), positions=np.zeros(max_rows, int))
    cap = len(stack)
    cur = stack[:count]
    kept = [0] * B if kept is None else kept
    for s in range(B):
        if new_lens[s] < 0:
            cur += [int(p) for p in table[s, kept[s]:held[s]]]
    lens = [0 if n < 0 else l + n for n, l in zip(new_lens, seq_lens)]
    want = [0 if n < 0 else max(0, -(-e // PAGE) - h) for n, h, e in zip(new_lens, held, lens)]
    rows = sum(max(n, 0) for n in new_lens)
    bad = any(e > width * PAGE or l < 0 or l > width * PAGE for l, e in zip(seq_lens, lens)) or rows > max_rows
    bad = bad or any(h < p or h > width for h, p in zip(held, pages))
    bad = bad or any(n < 0 and not 0 <= k <= h for n, h, k in zip(new_lens, held, kept))
    bad = bad or count < 0 or count > cap or len(cur) - sum(want) > cap
    if bad or sum(want) > len(cur):
        return dict(out, ok=False)
    moved = cur[min(count, len(cur) - sum(want)):]  # handed back or out
    going_on = [int(p) for s in range(B) if new_lens[s] > 0 for p in table[s, seq_lens[s] // PAGE:min(held[s], -(-lens[s] // PAGE))]]
    if not all(0 <= p <= MAX_PAGE for p in moved + going_on):
        return dict(out, ok=False)
    r = 0
    for s in range(B):
        n = new_lens[s]
        if n < 0:
            out["run_starts"][s + 1] = r
            continue
        for j in range(want[s]):
            table[s, held[s] + j] = cur.pop()
        for p in range(seq_lens[s], lens[s]):
            out["slots"][r] = table[s, p // PAGE] * PAGE + p % PAGE
            out["positions"][r] = p
            r += 1
        out["run_starts"][s + 1] = r
    left = np.array(stack)
    if len(cur) > count:
        left[count:len(cur)] = cur[count:]
    out["held"] = np.array([0 if n < 0 else h + w for n, h, w in zip(new_lens, held, want)], dtype=int)
    return dict(out, ok=True, seq_lens=np.array(lens), count=len(cur), stack=left)


def page_exponent(amax: float, fmt: str) -> int:
    """The smallest e in [E_MIN, E_MAX] with amax <= qmax 2^e (E_MAX where there is none)."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= QMAX[fmt] * 2.0 ** e:
            return e
    return E_MAX


def encode(x, fmt: str) -> np.ndarray:
    """Codes as stored (E4M3 bits, or code + 128) of values in units of the scale; half to even, saturating."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8p":
        return (np.clip(np.rint(x), -127, 127) + 128).astype(np.uint8)
    return e4m3_bits_rne_satfinite(np.clip(x, -448, 448).astype(np.float32)).astype(np.uint8)


def values(codes, fmt: str) -> np.ndarray:
    return np.asarray(codes, dtype=np.float64) - 128 if fmt == "int8p" else e4m3_value(np.asarray(codes, dtype=np.uint8))


def append_runs(codes, exps, x, run_starts, seq_lens, table, fmt):
    """codes [pages, H, 16, 128] (as stored) and exps [pages, H], updated in place from rows x [rows, H, 128]."""
    zero = 128 if fmt == "int8p" else 0
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x)
    clean = np.where(np.isnan(x), 0.0, x)
    for s in range(len(seq_lens)):
        a, b, end = int(run_starts[s]), int(run_starts[s + 1]), int(seq_lens[s])
        first = end - (b - a)
        for page in range(first // PAGE, -(-end // PAGE)) if b > a else ():
            phys = int(table[s, page])
            p0 = page * PAGE
            lo, hi = max(first, p0), min(end, p0 + PAGE)
            rows = slice(a + lo - first, a + hi - first)
            for h in range(codes.shape[1]):
                amax = np.max(np.abs(x[rows, h]), where=finite[rows, h], initial=0.0)
                e = page_exponent(float(amax), fmt)
                if lo > p0:
                    e0 = int(exps[phys, h])
                    e = max(e, e0)
                    if e > e0:
                        codes[phys, h, :lo - p0] = encode(values(codes[phys, h, :lo - p0], fmt) * 2.0 ** (e0 - e), fmt)
                with np.errstate(invalid="ignore"):
                    codes[phys, h, lo - p0:hi - p0] = encode(clean[rows, h] * 2.0 ** -e, fmt)
                codes[phys, h, hi - p0:] = zero
                exps[phys, h] = e


def attend(k_codes, k_exps, v_codes, v_exps, q, run_starts, seq_lens, table, sm_scale, fmt):
    """-> out [rows, Hq, 128], lse [rows, Hq], and per (row, head) the quantities that rounding errors are relative to:
    sum_t p_t |v_t| [128], max_t sum_c |x terms|, and max_t (p_t 2^ev_t) sum_t |value code_t| [128].  Rows of no run are NaN."""
    rows, Hq, D = q.shape
    H = k_codes.shape[1]
    G = Hq // H
    out, lse = np.full((rows, Hq, D), np.nan), np.full((rows, Hq), np.nan)
    pv, xa, low = np.zeros((rows, Hq, D)), np.zeros((rows, Hq)), np.zeros((rows, Hq, D))
    q = np.asarray(q, dtype=np.float64)
    for s in range(len(seq_lens)):
        a, b, end = int(run_starts[s]), int(run_starts[s + 1]), int(seq_lens[s])
        pages = [int(p) for p in table[s, :-(-end // PAGE)]]
        for h in range(H if b > a else 0):
            k = np.concatenate([values(k_codes[p, h], fmt) * 2.0 ** int(k_exps[p, h]) for p in pages] or [np.zeros((0, D))])[:end]
            v = np.concatenate([values(v_codes[p, h], fmt) * 2.0 ** int(v_exps[p, h]) for p in pages] or [np.zeros((0, D))])[:end]
            scale = np.repeat([2.0 ** int(v_exps[p, h]) for p in pages], PAGE)[:end]
            for r in range(a, b):
                n = max(0, end - (b - a) + (r - a) + 1)
                for g in range(h * G, h * G + G):
                    if n == 0:
                        out[r, g], lse[r, g] = 0.0, -math.inf
                        continue
                    x = sm_scale * (k[:n] @ q[r, g])
                    m = x.max()
                    w = np.exp(x - m)
                    lse[r, g] = m + math.log(w.sum())
                    p = w / w.sum()
                    out[r, g] = p @ v[:n]
                    pv[r, g] = p @ np.abs(v[:n])
                    low[r, g] = (p * scale[:n]).max() * (np.abs(v[:n]) / scale[:n, None]).sum(0)
                    xa[r, g] = abs(sm_scale) * (np.abs(k[:n]) @ np.abs(q[r, g])).max()
    return out, lse, pv, xa, low

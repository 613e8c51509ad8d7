"""Inputs and comparisons shared by the tests of kvq_map_runs, kvq_append_runs and kvq_attn_runs."""
import numpy as np

from oracle import runs as R
from quantized_kv_cache_kvq_gb300 import layout as L

FMTS = ("e4m3p", "int8p")
TILE_FMT = {"e4m3p": "e4m3", "int8p": "int8"}  # the 8-bit tile layouts are those of the per-token formats


def pages_of(n):
    return -(-n // R.PAGE)


def random_codes(rng, pages, heads, fmt):
    if fmt == "int8p":
        return np.clip(np.rint(rng.standard_normal((pages, heads, 16, 128)) * 36), -127, 127).astype(np.int64) + 128
    return R.encode(rng.standard_normal((pages, heads, 16, 128)) * 110, fmt).astype(np.int64)


def pack(codes, fmt, plane):
    """codes [pages, heads, 16, 128] -> tile bytes [pages * heads, 2048]."""
    offs = (L.k_offsets if plane == "k" else L.v_offsets)(TILE_FMT[fmt])
    out = np.zeros((codes.shape[0] * codes.shape[1], 2048), dtype=np.uint8)
    out[:, offs.reshape(-1)] = codes.reshape(out.shape[0], -1).astype(np.uint8)
    return out


def unpack(tiles, heads, fmt, plane):
    offs = (L.k_offsets if plane == "k" else L.v_offsets)(TILE_FMT[fmt])
    return tiles.reshape(-1, heads, 2048)[..., offs].astype(np.int64)


def tables(rng, lens, spare=3, width=None):
    """Block table over randomly ordered pages, -1 where a request has none -> (table, number of pages)."""
    counts = [pages_of(n) for n in lens]
    total = sum(counts) + spare
    width = width or max(counts + [1])
    perm = rng.permutation(total)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = perm[at:at + c]
        at += c
    return table, total


def starts_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def attn_tolerance(out, pv, xa, low, bf16):
    """Bound of |kernel - exact| for every output element.

    A logit sums 128 products in binary32: its error is at most 128 2^-24 times the sum of their magnitudes (xa), and the
    exponent's own rounding adds 2^-22 of the weight (ex2.approx), so each weight is off by d = 2^-17 xa + 2^-21 relative.
    The numerator and the denominator carry it once each, and the value product's binary32 sums add 2^-21 more.
    bf16: weights rounded to fp16 (half a step, 2^-11) and the result to bf16 (2^-8).  fp32: weights in two fp16 parts (2^-22).
    Weights that are subnormal in fp16 round to multiples of 2^-24.  bf16: the largest weight (page scale included) is held as
    2^7 or more, so that is off by 2^-25-7 of the largest, times the value code; fp32 holds it as 2^12 or more: 2^-25-12."""
    d = 2.0 ** -17 * xa[..., None] + 2.0 ** -21
    w = 2 * d + 2.0 ** -21 + (2.0 ** -11 if bf16 else 2.0 ** -22)
    return (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(out) + 1.01 * w * pv + (2.0 ** -32 if bf16 else 2.0 ** -37) * low + 1e-30


def lse_tolerance(lse, xa):
    return 2.0 ** -17 * xa + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))

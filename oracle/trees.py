"""A speculative step whose drafts are trees of tokens: masks, norms and rotation, attention, verification, the kept path.

Plain statements of ``kvq_tree_runs``, ``kvq_rope_runs``, ``kvq_attn_tree``, ``kvq_verify_runs`` and ``kvq_keep_runs`` as
include/kvq.h defines them, one request and one row at a time.  (No counterpart on the source pages: they decode one token.)
"""
from __future__ import annotations

import math

import numpy as np

from .runs import E_MIN, PAGE, encode, values

__all__ = ["ancestors", "tree_runs", "rope", "attend_tree", "residual", "verify_runs", "keep_runs"]

ONE = 1 << 44  # probabilities are summed as whole numbers of 2^-44


def ancestors(parents):
    """Per row of one run the set of what it sees: itself and its ancestors."""
    seen = []
    for i, p in enumerate(parents):
        seen.append({i} | (seen[p] if 0 <= p < i else set()))
    return seen


def tree_runs(parents, run_starts, seq_lens, words):
    """-> mask [rows, words] int32 and positions [rows] of the runs' rows."""
    mask = np.zeros((len(parents), words), dtype=np.int64)
    positions = np.zeros(len(parents), dtype=np.int64)
    for s, end in enumerate(seq_lens):
        a, b = int(run_starts[s]), int(run_starts[s + 1])
        for i, see in enumerate(ancestors([int(p) for p in parents[a:b]])):
            for j in see:
                mask[a + i, j // 32] |= 1 << (j % 32)
            positions[a + i] = int(end) - (b - a) + len(see) - 1
    return mask.astype(np.uint32).view(np.int32), positions


def rope(x, weight, eps, positions, cos_sin):
    """x [rows, heads, 128] normed (where weight is given) and rotated, in float64."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    cs = np.asarray(cos_sin, dtype=np.float64)[positions][:, None, :]
    a, b, c, s = x[..., :64], x[..., 64:], cs[..., :64], cs[..., 64:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def attend_tree(k_codes, k_exps, v_codes, v_exps, q, run_starts, seq_lens, table, mask, sm_scale, fmt):
    """As runs.attend, with the rows of a run seeing what their masks say of it."""
    rows, Hq, D = q.shape
    H = k_codes.shape[1]
    G = Hq // H
    out, lse = np.full((rows, Hq, D), np.nan), np.full((rows, Hq), np.nan)
    pv, xa, low = np.zeros((rows, Hq, D)), np.zeros((rows, Hq)), np.zeros((rows, Hq, D))
    q = np.asarray(q, dtype=np.float64)
    bits = np.asarray(mask).view(np.uint32)
    for s in range(len(seq_lens)):
        a, b, end = int(run_starts[s]), int(run_starts[s + 1]), int(seq_lens[s])
        pages = [int(p) for p in table[s, :-(-end // PAGE)]]
        before = end - (b - a)
        for h in range(H if b > a else 0):
            k = np.concatenate([values(k_codes[p, h], fmt) * 2.0 ** int(k_exps[p, h]) for p in pages] or [np.zeros((0, D))])[:end]
            v = np.concatenate([values(v_codes[p, h], fmt) * 2.0 ** int(v_exps[p, h]) for p in pages] or [np.zeros((0, D))])[:end]
            scale = np.repeat([2.0 ** int(v_exps[p, h]) for p in pages], PAGE)[:end]
            for r in range(a, b):
                t = np.array([t for t in range(end) if t < before or int(bits[r, (t - before) // 32]) >> ((t - before) % 32) & 1], dtype=int)
                for g in range(h * G, h * G + G):
                    if len(t) == 0:
                        out[r, g], lse[r, g] = 0.0, -math.inf
                        continue
                    x = sm_scale * (k[t] @ q[r, g])
                    m = x.max()
                    w = np.exp(x - m)
                    lse[r, g] = m + math.log(w.sum())
                    p = w / w.sum()
                    out[r, g] = p @ v[t]
                    pv[r, g] = p @ np.abs(v[t])
                    low[r, g] = (p * scale[t]).max() * (np.abs(v[t]) / scale[t, None]).sum(0)
                    xa[r, g] = abs(sm_scale) * (np.abs(k[t]) @ np.abs(q[r, g])).max()
    return out, lse, pv, xa, low


def _whole(w):
    return [int(float(x) * ONE) for x in w]


def residual(p, q, c):
    """max(p - c q, 0) in binary32, product and difference rounded."""
    p, q, c = np.asarray(p, np.float32), np.asarray(q, np.float32), np.float32(c)
    return np.maximum(p - c * q, np.float32(0))


def _draw(w, u):
    """The lowest index whose cumulative sum exceeds floor(u sum)."""
    total = sum(w)
    t = min(max(int(math.floor(float(u) * float(total))), 0), total - 1)
    cum = 0
    for i, x in enumerate(w):
        cum += x
        if cum > t:
            return i
    return -1


def verify_runs(target, draft, tokens, parents, uniform, run_starts):
    """-> keep [rows] (untouched rows of no run: -1), kept [B], next [B]."""
    keep = np.full(len(tokens), -1)
    kept, following = [], []
    for s in range(len(run_starts) - 1):
        a, b = int(run_starts[s]), int(run_starts[s + 1])
        if a == b:
            kept.append(0)
            following.append(-1)
            continue
        path, last = [0], -1
        while True:
            cur = path[-1]
            p = np.asarray(target[a + cur], dtype=np.float32)
            kids = [i for i in range(1, b - a) if parents[a + i] == cur]
            go = None
            if uniform is None:
                last = int(np.argmax(np.where(np.isnan(p), -np.inf, p)))
            else:
                w = _whole(p)
                if draft is not None:
                    q = np.asarray(draft[a + cur], dtype=np.float32)
                    c, z = np.float32(0), sum(w)
                    for i in kids:
                        x = int(tokens[a + i])
                        u = float(uniform[a + i][0])
                        if u * float(q[x]) * (float(z) / ONE) < float(p[x]) - float(c) * float(q[x]):
                            go = i
                            break
                        c = np.float32(float(c) + float(z) / ONE)
                        w = _whole(residual(p, q, c))
                        z = sum(w)
                    if z == 0:
                        w = _whole(p)
                last = _draw(w, uniform[a + cur][1])
            if draft is None:
                go = next((i for i in kids if int(tokens[a + i]) == last), None)
            if go is None:
                break
            path.append(go)
        keep[a:a + len(path)] = path
        kept.append(len(path))
        following.append(last)
    return keep, np.array(kept), np.array(following)


def keep_runs(codes, exps, keep, kept, run_starts, seq_lens, table, fmt):
    """codes [pages, H, 16, 128] (as stored) and exps [pages, H] of one plane of one layer, updated in place; seq_lens count the kept tokens."""
    zero = 128 if fmt == "int8p" else 0
    was, had = codes.copy(), exps.copy()
    for s in range(len(seq_lens)):
        a, m, end = int(run_starts[s]), int(kept[s]), int(seq_lens[s])
        first = end - m
        path = [int(i) for i in keep[a:a + m]]
        for page in range(first // PAGE, -(-end // PAGE)) if m else ():
            at = range(page * PAGE, min(end, page * PAGE + PAGE))
            home = [p if p < first else first + path[p - first] for p in at]
            if list(at) == home:
                continue
            phys = int(table[s, page])
            for h in range(codes.shape[1]):
                src = [(int(table[s, p // PAGE]), p % PAGE) for p in home]
                e = max([int(had[p, h]) for p, _ in src] + [E_MIN])
                codes[phys, h] = zero
                for t, (p, slot) in enumerate(src):
                    x = was[p, h, slot]
                    if had[p, h] < e:
                        x = encode(values(x, fmt) * 2.0 ** (int(had[p, h]) - e), fmt)
                    codes[phys, h, t] = x
                exps[phys, h] = e

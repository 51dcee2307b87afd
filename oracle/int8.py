"""Scored routing, int8 quantisation and the int8 expert SwiGLU in 64 bits.

Definitions (symmetric int8, one scale per activation row and per weight row):

* quantise: a = max |x|, r = 127 / a, code = rint(x r), scale = a / 127.  The
  codes are whole numbers defined by fp32 operations, so this file evaluates
  exactly those; everything else is float64.
* product: y[m, n] = sx[m] sw[n] sum_k q[m, k] w[n, k].
* SwiGLU: h = bf16(silu(g) u), quantised again, times down.

``moe_layer`` also returns how far a correct evaluation may be from it: h is a
float between two roundings, so an element whose last fp32 bits decide its bf16
value may fall either way; the bound adds up what those elements can move.
"""
from __future__ import annotations

import numpy as np


def bf16_round(v):
    """float64 -> nearest bf16 value (ties to even), as float64."""
    u = np.asarray(v, dtype=np.float32)
    # the double rounding float64 -> fp32 -> bf16 only matters within 2^-24 of a tie,
    # which the ambiguity bound covers
    b = np.ascontiguousarray(u).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return b.view(np.float32).astype(np.float64)


def quantize(x):
    """codes int64 [rows, cols], scales float32 [rows] of bf16 values x."""
    x = np.asarray(x, dtype=np.float32)
    a = np.abs(x).max(axis=1)
    bad = ~np.isfinite(x).all(axis=1)
    zero = ~bad & (a < np.float32(2.0 ** -100))
    ok = ~bad & ~zero
    safe = np.where(ok, a, np.float32(1)).astype(np.float32)
    r = (np.float32(127) / safe).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.rint(np.where(ok[:, None], x * r[:, None], np.float32(0)))
    s = np.where(ok, safe / np.float32(127), np.where(bad, np.float32(np.nan), np.float32(0)))
    return q.astype(np.int64), s.astype(np.float32)


def product(q, s, wq, ws):
    """float64 [M, N]; the integer sums are exact (|sum| < 2^53)."""
    acc = np.asarray(q, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T
    return acc * np.asarray(s, np.float64)[:, None] * np.asarray(ws, np.float64)


def regions(H, I):
    """(codes offset, scales offset, outputs, inputs) of gate, up, down in an expert blob."""
    out, at = [], 0
    for rows, cols in ((I, H), (I, H), (H, I)):
        out.append((at, at + rows * cols, rows, cols))
        at += rows * cols + 4 * rows
    return out


def expert_bytes(H, I):
    return 3 * H * I + 4 * (2 * I + H)


def make_expert(rng, H, I):
    """A random blob (uint8 [S]): codes over the whole int8 range, scales that keep outputs near 1."""
    b = np.empty(expert_bytes(H, I), dtype=np.uint8)
    for q, s, rows, cols in regions(H, I):
        b[q:s] = np.clip(np.rint(rng.normal(0, 40, rows * cols)), -128, 127).astype(np.int8).view(np.uint8)
        sc = (np.exp(rng.normal(0, 0.4, rows)) / (40 * np.sqrt(cols))).astype(np.float32)
        b[s:s + 4 * rows] = sc.view(np.uint8)
    return b


def matrices(blob, H, I):
    return [(blob[q:s].view(np.int8).reshape(rows, cols), blob[s:s + 4 * rows].view(np.float32))
            for q, s, rows, cols in regions(H, I)]


# relative error of an fp32 evaluation of silu(g) u: three roundings of each sum's
# scaling, the product, and an exponential whose argument carries 2^-23 |g|
# (|g| < 64 wherever e^-|g| still shows in bf16)
H_EPS = 80 * 2.0 ** -23


def swiglu(x, blob, H, I):
    """y float64 [n, H] of bf16 rows x [n, H], and the largest error of a correct evaluation."""
    (gq, gs), (uq, us), (dq, ds) = matrices(blob, H, I)
    q, s = quantize(x)
    g, u = product(q, s, gq, gs), product(q, s, uq, us)
    with np.errstate(over="ignore"):
        hx = g / (1.0 + np.exp(-g)) * u
    lo, hi = bf16_round(hx - np.abs(hx) * H_EPS), bf16_round(hx + np.abs(hx) * H_EPS)
    h = bf16_round(hx)
    hq, hs = quantize(h)
    y = product(hq, hs, dq, ds)
    # |codes| that may differ, row by row: with the row's largest value settled the factor
    # r is settled too and an unsettled element moves by whole codes; with it unsettled
    # every element's value may move by its spacing and two half steps
    a = np.abs(h).max(axis=1)
    top_open = (np.maximum(np.abs(lo), np.abs(hi)).max(axis=1) != a) | (np.minimum(np.abs(lo), np.abs(hi)).max(axis=1) != a)
    safe = np.where(a > 0, a, 1.0)
    r = (np.float32(127) / safe.astype(np.float32)).astype(np.float64)[:, None]
    move = np.where(lo != hi, np.ceil(np.abs(hi - lo) * r) + 1, 0.0) * hs.astype(np.float64)[:, None]
    move = np.where(top_open[:, None], np.abs(hi - lo) + 1.02 * safe[:, None] / 127, move)
    bound = move @ np.abs(dq.astype(np.float64)).T * ds.astype(np.float64)
    return y, bound


def moe_layer(x, ids, w, blob_of, H, I, y_bf16):
    """out float64 [T, H] and the tolerance of a bf16 output; y_bf16: each expert's
    output is rounded to bf16 before the sum (prefill)."""
    T, k = ids.shape
    out, tol, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    w = np.asarray(w, dtype=np.float64)
    for e in sorted({int(v) for v in ids.ravel() if v >= 0}):
        t, j = np.nonzero(ids == e)
        y, b = swiglu(x[t], blob_of(e), H, I)
        wt = w[t, j][:, None]
        np.add.at(out, t, wt * y)
        np.add.at(tol, t, np.abs(wt) * b)
        np.add.at(mag, t, np.abs(wt) * (np.abs(y) + b))
    # per term: int32 -> fp32, two scales, the weighted sum of k terms, y in bf16 where kept so
    tol += mag * ((4 + k) * 2.0 ** -24 + (2.0 ** -8 if y_bf16 else 0.0))
    tol += (np.abs(out) + tol) * 2.0 ** -8
    return out, tol


def route_scored(logits, bias, k, score, n_group, topk_group, renorm, scale):
    """ids int32 [T, k], weights float64 [T, k]; score: "softmax" or "sigmoid"."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    b = np.zeros(E) if bias is None else np.array(bias, dtype=np.float64)
    b[np.isnan(b)] = -np.inf
    ids, w = np.empty((T, k), dtype=np.int32), np.empty((T, k))
    for t in range(T):
        row = l[t]
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-row))
        else:
            m = row.max()
            s = np.zeros(E)
            for e in range(E):
                if row[e] > -np.inf:
                    s[e] = 1.0 if row[e] == m else np.exp(row[e] - m) if m < np.inf else 0.0
            s = s / s.sum() if s.sum() > 0 else s
        live = (row > -np.inf) & (b > -np.inf)
        c = np.where(live, s + np.where(live, b, 0.0), -np.inf)
        size = E // n_group
        rank = []
        for g in range(n_group):
            best = sorted((v for v in c[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:2]
            rank.append(sum(best) if best else -np.inf)
        keep = sorted(range(n_group), key=lambda g: (-rank[g], g))[:topk_group]
        inside = [e for e in range(E) if e // size in keep]
        sel = sorted(inside, key=lambda e: (-c[e], e))[:k]
        v = np.where(live[sel], s[sel], 0.0)
        ids[t] = sel
        w[t] = (v / (v.sum() + 1e-20) if renorm else v) * scale
    return ids, w

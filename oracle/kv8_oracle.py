"""Plain 64-bit definitions of the 8-bit latent cache's operators (numpy).

A cached row is decode(codes) * 2^e with one exponent e per block of 64 tokens;
codes are OCP e4m3. Written from the definitions in include/dsa.h; shares no
code with the CUDA path or with the workloads.
"""
from __future__ import annotations

import numpy as np

from .dsa_oracle import e4m3_decode

E_MIN, E_MAX = -64, 63


def round_e4m3(v):
    """The e4m3 value nearest to v, ties to even, saturating at +-448; NaN stays."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 448.0)
    _, x = np.frexp(np.where(a > 0, a, 1.0))            # a = f * 2^x, f in [0.5, 1)
    step = np.exp2(np.maximum(x - 1, -6) - 3.0)
    return np.where(np.isnan(v), np.nan, np.copysign(np.rint(a / step) * step, v))


def encode_e4m3(v):
    """Codes of values that e4m3 holds exactly."""
    table = e4m3_decode(np.arange(127, dtype=np.uint8))  # 0 .. 448, ascending
    v = np.asarray(v, dtype=np.float64)
    c = np.searchsorted(table, np.abs(np.where(np.isnan(v), 0.0, v)))
    return np.where(np.isnan(v), 0x7F, c | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def block_exponent(x):
    """Smallest e in [-64, 63] with max |finite x| <= 448 * 2^e."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    a = np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0)
    e = E_MIN
    while e < E_MAX and a > 448.0 * 2.0 ** e:
        e += 1
    return e


def store(codes, exps, rows, seqs, pos, table):
    """Writes rows[i] at position pos[i] of sequence seqs[i] (runs of consecutive
    positions); codes [pages, 64, 576], exps [pages]: copies are returned."""
    codes, exps = codes.copy(), exps.copy()
    rows = np.asarray(rows, dtype=np.float64)
    groups = {}
    for i, (b, p) in enumerate(zip(seqs, pos)):
        groups.setdefault((b, p // 64), []).append((p % 64, i))
    for (b, blk), items in groups.items():
        pg = table[b][blk]
        first = min(s for s, _ in items)
        e = block_exponent(rows[[i for _, i in items]])
        if first > 0:
            e = max(e, int(exps[pg]))
            if e != exps[pg]:
                old = e4m3_decode(codes[pg, :first]) * 2.0 ** (int(exps[pg]) - e)
                codes[pg, :first] = encode_e4m3(round_e4m3(old))
        for s, i in items:
            codes[pg, s] = encode_e4m3(round_e4m3(rows[i] * 2.0 ** -e))
        exps[pg] = e
    return codes, exps


def values(codes, exps):
    """The cache as float64 rows [pages * 64, 576]."""
    return (e4m3_decode(codes) * np.exp2(exps.astype(np.float64))[:, None, None]).reshape(-1, codes.shape[-1])


def attend(q, rows, scale, d_v=512):
    """q [H, d], rows [n, d] -> (out [H, d_v], lse [H], p [H, n])."""
    if len(rows) == 0:
        return np.zeros((len(q), d_v)), np.full(len(q), -np.inf), np.zeros((len(q), 0))
    z = scale * (np.asarray(q, dtype=np.float64) @ rows.T)
    m = z.max(axis=1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(axis=1, keepdims=True)
    p = p / l
    return p @ rows[:, :d_v], (m + np.log(l))[:, 0], p


def keep(acc, n, budget, sink, recent):
    """Positions that stay, ascending, of n tokens with weights acc[0..n-1]."""
    if n <= budget:
        return list(range(n))
    w = np.asarray(acc[sink:n - recent], dtype=np.float64) + 0.0
    w = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(np.asarray(acc[sink:n - recent], dtype=np.float64))
    order = sorted(range(len(w)), key=lambda i: (nan[i], -w[i], i))
    mid = sorted(order[:budget - sink - recent])
    return list(range(sink)) + [sink + i for i in mid] + list(range(n - recent, n))


def move(codes, exps, src, dst_pages):
    """Rows src (cache rows page * 64 + slot, in order) into dst_pages: copies."""
    out, eo = codes.copy(), exps.copy()
    flat = codes.reshape(-1, codes.shape[-1])
    for j in range(0, len(src), 64):
        rows = np.asarray(src[j:j + 64])
        e_src = exps[rows // 64].astype(np.int64)
        e = int(e_src.max())
        v = e4m3_decode(flat[rows]) * np.exp2((e_src - e).astype(np.float64))[:, None]
        out[dst_pages[j // 64], :len(rows)] = encode_e4m3(round_e4m3(v))
        eo[dst_pages[j // 64]] = e
    return out, eo

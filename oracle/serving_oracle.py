"""fp64 CPU oracle of the serving calls (include/sas_serving.h): rotary
positions, page tables and slots, the cache write and decode of drafted trees.

Written from the definitions, one token at a time; it shares no code with the
CUDA path. The tree rests on the decode oracle alone: a drafted token gets what
a decode step gives on the cache with its path appended.
"""
from __future__ import annotations

import numpy as np

from oracle import sas_oracle as O

BLOCK = 64


def rotate(x, pos, inv_freq, interleaved=False, amplitude=1.0, inverse=False):
    """x [B][H][N][d] (fp64) rotated at pos [B][N]; inv_freq [rot/2]."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    y = x.copy()
    theta = np.asarray(pos, dtype=np.float64)[:, None, :, None] * f
    c, s = amplitude * np.cos(theta), amplitude * np.sin(theta)
    if inverse:
        s = -s
    for p in range(f.size):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + f.size)
        y[..., a] = x[..., a] * c[..., p] - x[..., b] * s[..., p]
        y[..., b] = x[..., b] * c[..., p] + x[..., a] * s[..., p]
    return y


def depths(parents):
    """Number of ancestors of each token; parents [B][N], -1 at a root."""
    parents = np.asarray(parents)
    out = np.zeros_like(parents)
    for b in range(parents.shape[0]):
        for i in range(parents.shape[1]):
            out[b, i] = 0 if parents[b, i] < 0 else out[b, parents[b, i]] + 1
    return out


def page_map(lens, nnew, table, free, head, T, npages):
    """(slots, new_lens, taken, head, table): see sas_page_map."""
    table = np.array(table)
    B, width = table.shape
    slots = np.full((B, T), -1, dtype=np.int64)
    new_lens, taken = np.array(lens, dtype=np.int64), np.full(B, -1, dtype=np.int64)
    wanted, granted = 0, 0
    for b in range(B):
        n, m = int(lens[b]), int(nnew[b])
        if n < 0 or m < 0 or m > T or n + m > BLOCK * width:
            continue
        have, need = -(-n // BLOCK), -(-(n + m) // BLOCK) - (-(-n // BLOCK))
        first = head + wanted
        wanted += need
        if need and (head < 0 or first + need > len(free)):
            continue
        table[b, have:have + need] = free[first:first + need]
        granted += need
        for j in range(m):
            page = int(table[b, (n + j) // BLOCK])
            if 0 <= page < npages:
                slots[b, j] = page * BLOCK + (n + j) % BLOCK
        new_lens[b], taken[b] = n + m, need
    return slots, new_lens, taken, head + granted, table


def append(k, v, lens, kc, vc, ksum, ntok, rows=None, slots=None, rot=None, store=None,
           store_sum=None):
    """kc, vc, ksum (fp64 copies) after the write; see sas_cache_append.

    rot(x, pos) rotates k at its positions (None: not rotated); store and
    store_sum round to the cache's and the summaries' types.
    """
    kc, vc, ksum = (np.array(x, dtype=np.float64) for x in (kc, vc, ksum))
    B, Hkv, T, d = k.shape
    pos = np.asarray(lens)[:, None] + np.arange(T)
    src = np.arange(T)[None].repeat(B, 0) if rows is None else np.asarray(rows)
    kk = np.stack([k[b][:, src[b]] for b in range(B)])
    vv = np.stack([v[b][:, src[b]] for b in range(B)])
    if rot is not None:
        kk = rot(kk, pos)
    kk = store(kk)
    for b in range(B):
        for j in range(int(ntok[b])):
            p = int(pos[b, j])
            if slots is None:
                kc[b, :, p], vc[b, :, p] = kk[b, :, j], vv[b, :, j]
                if p % BLOCK == BLOCK - 1:
                    ksum[b, :, p // BLOCK] = store_sum(kc[b, :, p - BLOCK + 1:p + 1].mean(1))
            elif slots[b, j] >= 0:
                page, row = divmod(int(slots[b, j]), BLOCK)
                kc[page, :, row], vc[page, :, row] = kk[b, :, j], vv[b, :, j]
                if row == BLOCK - 1:
                    ksum[page] = store_sum(kc[page].mean(1))
    return kc, vc, ksum


def decode_tree(q, kd, vd, kc, vc, lens, ksum, parents, ntok, topk, gated=1,
                store_sum=lambda x: x):
    """o, idx and the mass sum_j p_j |v_j| (same shape as o) of drafted tokens.

    Contiguous caches [B][Hkv][N][d]; rows from ntok on are NaN and -2. The
    tokens' path is appended to the cached ones and one decode step taken.
    """
    q, kd, vd, kc, vc, ksum = (np.asarray(x, dtype=np.float64)
                               for x in (q, kd, vd, kc, vc, ksum))
    B, Hq, T, d = q.shape
    Hkv = kd.shape[1]
    o, mass = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    idx = np.full((B, Hkv, T, topk), -2, dtype=np.int64)
    for b in range(B):
        n = int(lens[b])
        for i in range(int(ntok[b])):
            path = [i]
            while parents[b][path[0]] >= 0:
                path.insert(0, int(parents[b][path[0]]))
            N = -(-(n + len(path)) // BLOCK) * BLOCK
            kk, vv = np.zeros((1, Hkv, N, d)), np.zeros((1, Hkv, N, d))
            kk[0, :, :n], vv[0, :, :n] = kc[b, :, :n], vc[b, :, :n]
            kk[0, :, n:n + len(path)], vv[0, :, n:n + len(path)] = kd[b][:, path], vd[b][:, path]
            ks = np.zeros((1, Hkv, N // BLOCK, d))
            whole = n // BLOCK
            ks[0, :, :whole] = ksum[b, :, :whole]
            for m in range(whole, (n + len(path)) // BLOCK):
                ks[0, :, m] = store_sum(kk[0, :, m * BLOCK:(m + 1) * BLOCK].mean(1))
            at = np.array([n + len(path)])
            qi = q[b:b + 1, :, i]
            sel, cnt, logg, _ = O.select_decode(qi, ks, at, Hkv, topk, None)
            oi, _ = O.decode_attend(qi, kk, vv, at, sel, cnt, logg, Hkv, gated, None)
            mi, _ = O.decode_attend(qi, kk, np.abs(vv), at, sel, cnt, logg, Hkv, gated, None)
            o[b, :, i], mass[b, :, i] = oi[0], mi[0]
            idx[b, :, i] = sel[0]
    return o, idx, mass

"""fp64 restatements of the packed-request operators -- TEST INFRASTRUCTURE ONLY.

Plain loops over sequences and tokens, from the definitions in include/kda.h;
they share no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def offsets(R, rows, cu):
    """[R + 1] row offsets of the sequences."""
    return np.arange(R + 1) * (rows // max(R, 1)) if cu is None else np.asarray(cu, dtype=np.int64)


def block_map(lens, ctx, free, table, page, rows):
    """(cu, table, slots, used): sequence offsets, block table with the new blocks, pool slots of the rows."""
    table = np.array(table, copy=True)
    cu, slots, taken = [0], [], 0
    for r, n in enumerate(int(v) for v in lens):
        n, c = max(n, 0), 0 if ctx is None else max(int(ctx[r]), 0)
        for j in range(-(-c // page), -(-(c + n) // page)):
            if j < table.shape[1]:
                table[r, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(c, c + n):
            b = table[r, p // page] if p // page < table.shape[1] else -1
            slots.append(b * page + p % page if b >= 0 else -1)
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * rows)[:rows]
    return np.array(cu), table, np.array(slots, dtype=np.int64), taken


def short_conv(x, w, bias, state=None, slots=None, ctx=None, cu=None, R=1, silu=True, head_dim=0, eps=None):
    """Packed rows x [rows, C] -> (y [rows, C], pool).  Rows of no sequence, and of padded ones, are NaN.
    eps: of the L2 norm of each head, None without it."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    rows, C = x.shape
    K = w.shape[1]
    pool = None if state is None else np.array(state, dtype=np.float64, copy=True)
    y = np.full((rows, C), np.nan)
    cu = offsets(R, rows, cu)
    for r in range(R):
        lo, hi = int(cu[r]), int(cu[r + 1])
        slot = r if slots is None else int(slots[r])
        if slot < 0 or hi == lo:
            continue
        old = np.zeros((K - 1, C))
        if pool is not None and ctx is not None and ctx[r] > 0:
            old = pool[slot].copy()
        u = np.concatenate([old, x[lo:hi]])
        for t in range(hi - lo):
            v = np.zeros(C) if bias is None else np.asarray(bias, np.float64).copy()
            for i in range(K):
                v += w[:, i] * u[t + i]
            if silu:
                v = v / (1 + np.exp(-v))
            if eps is not None:
                h = v.reshape(-1, head_dim)
                v = (h / np.sqrt((h * h).sum(1, keepdims=True) + eps)).reshape(-1)
            y[lo + t] = v
        if pool is not None:
            pool[slot] = u[len(u) - (K - 1):]
    return y, pool


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=True, state=None, slots=None, ctx=None, cu=None, R=1,
             table=None, pages=None, page=0):
    """Packed rows x [rows, H, P] -> (y, pool, pages).  Rows of no sequence, and of padded ones, are NaN."""
    x, dt, A, B, C = (np.asarray(t, np.float64) for t in (x, dt, A, B, C))
    rows, H, P = x.shape
    G, N = B.shape[1:]
    D = np.zeros(H) if D is None else np.asarray(D, np.float64)
    d = dt + (0 if dt_bias is None else np.asarray(dt_bias, np.float64))
    if softplus:
        d = np.maximum(d, 0) + np.log1p(np.exp(-np.abs(d)))
    pool = None if state is None else np.array(state, dtype=np.float64, copy=True)
    pages = None if pages is None else np.array(pages, dtype=np.float64, copy=True)
    y = np.full((rows, H, P), np.nan)
    cu = offsets(R, rows, cu)
    group = np.arange(H) // (H // G)
    for r in range(R):
        lo, hi = int(cu[r]), int(cu[r + 1])
        slot = r if slots is None else int(slots[r])
        if slot < 0 or hi == lo:
            continue
        c = 0 if ctx is None else max(int(ctx[r]), 0)
        S = pool[slot].copy() if pool is not None and c > 0 else np.zeros((H, N, P))
        for t in range(lo, hi):
            S = np.exp(d[t] * A)[:, None, None] * S + (d[t][:, None] * B[t][group])[:, :, None] * x[t][:, None, :]
            y[t] = np.einsum("hn,hnp->hp", C[t][group], S) + D[:, None] * x[t]
            pos = c + t - lo + 1
            if page and pos % page == 0 and pos // page - 1 < table.shape[1]:
                b = int(table[r, pos // page - 1])
                if 0 <= b < len(pages):
                    pages[b] = S
        if pool is not None:
            pool[slot] = S
    return y, pool, pages

"""Plain implementations of the 8-bit paged cache's operators on the host
(numpy; attention in float64), and cases shared by their tests."""
import math

import numpy as np

F32 = np.float32


def cdiv(a, b):
    return -(-a // b)


def block_tables(lens, add, table, free, block, cap):
    """-> (lens_out, cu, slots, pos, used, table): request by request."""
    table = table.copy()
    width = table.shape[1]
    cu, slots, pos, used = [0], [], [], 0
    for b, (n, m) in enumerate(zip(lens, add)):
        n, m = max(int(n), 0), max(int(m), 0)
        have, need = min(cdiv(n, block), width), min(cdiv(n + m, block), width)
        for j in range(have, need):
            table[b, j] = free[used] if used < len(free) else -1
            used += 1
        for p in range(n, n + m):
            j = p // block
            page = table[b, j] if j < width else -1
            slots.append(int(page) * block + p % block if page >= 0 else -1)
            pos.append(p)
        cu.append(cu[-1] + m)
    pad = max(0, cap - len(slots))
    return (np.array([max(int(n), 0) + max(int(m), 0) for n, m in zip(lens, add)], np.int32),
            np.array(cu, np.int32), np.array((slots + [-1] * pad)[:cap], np.int64),
            np.array((pos + [-1] * pad)[:cap], np.int32), used, table)


def new_cache(rng, P, Hk, bs, D):
    """A cache in use: every array holds something."""
    k = np.clip(np.rint(rng.standard_normal((P, Hk, bs, D)) * 35), -127, 127).astype(np.int8)
    v = np.clip(np.rint(rng.standard_normal((P, Hk, bs, D)) * 35), -127, 127).astype(np.int8)
    ks = (0.02 * np.exp(rng.standard_normal((P, Hk)))).astype(F32)
    vs = (0.02 * np.exp(rng.standard_normal((P, Hk)))).astype(F32)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs,
            "k_sum": k.sum(2, dtype=np.int32).astype(np.int16)}


def append(c, k_new, v_new, slots):
    """In place; k_new, v_new fp32 [n, Hk, D]."""
    P, Hk, bs, D = c["k"].shape
    i = 0
    while i < len(slots):
        s = int(slots[i])
        if s < 0 or s >= P * bs:
            i += 1
            continue
        page, r0, m = s // bs, s % bs, 1
        while i + m < len(slots) and r0 + m < bs and slots[i + m] == s + m:
            m += 1
        for x, name in ((k_new, "k"), (v_new, "v")):
            for h in range(Hk):
                rows = x[i:i + m, h]
                old = F32(c[name + "_scale"][page, h]) if r0 else F32(0)
                new = max(old, F32(np.abs(rows).max() / F32(127)))
                if new > old:
                    ratio = F32(old / new)
                    c[name][page, h, :r0] = np.rint(c[name][page, h, :r0].astype(F32) * ratio)
                q = np.rint(rows / new) if new > 0 else np.zeros_like(rows)
                c[name][page, h, r0:r0 + m] = np.clip(q, -127, 127)
                c[name + "_scale"][page, h] = new
        c["k_sum"][page] = c["k"][page, :, :r0 + m].sum(1, dtype=np.int32)
        i += m


def positions(cu, lens, n):
    """(sequence, position) of each token; (-1, 0) for padding."""
    for i in range(n):
        b = next((b for b in range(len(lens)) if cu[b] <= i < cu[b + 1]), -1)
        yield (i, b, int(lens[b]) - int(cu[b + 1]) + i if b >= 0 else 0)


def select(q, c, table, cu, lens, n_sel, n_first, n_last, out):
    """q fp32 [n, H, D]; writes into out [n, Hk, n_sel]."""
    P, Hk, bs, D = c["k"].shape
    n, H = q.shape[:2]
    G = H // Hk
    for i, b, pos in positions(cu, lens, n):
        if b < 0:
            continue
        nblk = min(pos // bs + 1, table.shape[1]) if pos >= 0 else 0
        for h in range(Hk):
            qs = q[i, h * G:(h + 1) * G].astype(np.float64).sum(0).astype(F32)
            big = np.abs(qs).max()
            q8 = np.zeros(D, np.int64)
            if big > 0 and np.isfinite(big):
                q8 = np.rint(qs * F32(F32(127) / big)).astype(np.int64)
            first = min(n_first, nblk)
            last = max(first, nblk - n_last)
            score = []
            for j in range(first, last):
                page = table[b, j]
                if page < 0 or page >= P:
                    score.append(-np.inf)
                    continue
                dot = F32(int(q8 @ c["k_sum"][page, h].astype(np.int64)))
                score.append(F32(dot * c["k_scale"][page, h]) + F32(0))
            want = min(n_sel - (first + nblk - last), last - first)
            best = np.argsort(-np.array(score, F32), kind="stable")[:want] + first
            kept = sorted(list(range(first)) + [int(j) for j in best] + list(range(last, nblk)))
            out[i, h] = -1
            out[i, h, :len(kept)] = kept


def attn(q, c, table, cu, lens, sel=None, sm_scale=None):
    """float64 -> (out [n, H, D], lse [n, H], bound on |out| error's weights).

    The third result is (A, S, N, M) per row: the mean of |value| under the
    softmax per dim, the largest sum of |q_d k_d| * scale over the keys, the
    number of keys and the largest value that their pages' scales can hold
    (127 max vs) -- what an error bound needs.  Padding rows are NaN."""
    P, Hk, bs, D = c["k"].shape
    n, H = q.shape[:2]
    G = H // Hk
    sm_scale = 1 / math.sqrt(D) if sm_scale is None else sm_scale
    out, lse = np.full((n, H, D), np.nan), np.full((n, H), np.nan)
    A, S, N = np.zeros((n, H, D)), np.zeros((n, H)), np.zeros((n, H))
    M = np.zeros((n, H))
    for i, b, pos in positions(cu, lens, n):
        if b < 0:
            continue
        nblk = pos // bs + 1 if pos >= 0 else 0
        for h in range(Hk):
            blocks = range(nblk) if sel is None else [j for j in sel[i, h] if 0 <= j < nblk]
            ks, vs, top = [np.zeros((0, D))], [np.zeros((0, D))], 0.0
            for j in blocks:
                page = table[b, j] if j < table.shape[1] else -1
                if page < 0 or page >= P:
                    continue
                r = min(bs, pos + 1 - j * bs)
                top = max(top, 127 * float(c["v_scale"][page, h]))
                ks.append(c["k"][page, h, :r].astype(np.float64) * float(c["k_scale"][page, h]))
                vs.append(c["v"][page, h, :r].astype(np.float64) * float(c["v_scale"][page, h]))
            k, v = np.concatenate(ks), np.concatenate(vs)
            for g in range(G):
                a = h * G + g
                if len(k) == 0:
                    out[i, a], lse[i, a] = 0.0, -np.inf
                    continue
                x = (k @ q[i, a].astype(np.float64)) * sm_scale
                m = x.max()
                p = np.exp(x - m)
                out[i, a] = p @ v / p.sum()
                lse[i, a] = m + np.log(p.sum())
                A[i, a] = p @ np.abs(v) / p.sum()
                S[i, a] = (np.abs(k) @ np.abs(q[i, a].astype(np.float64))).max() * abs(sm_scale)
                N[i, a] = len(k)
                M[i, a] = top
    return out, lse, (A, S, N, M)


def attn_bounds(out, lse, info):
    """How far bf16 out and fp32 lse may be off.

    A logit is D exact products summed in fp32, scaled by two fp32 factors and
    taken through exp2: |error| <= delta = (D + 8) 2^-24 S (any order of the
    sum, S the sum of magnitudes).  Weights are then off by a factor within
    1 +- (2 delta + 2^-20) and rounded once to fp16 (half a step, 2^-11); sums
    of N terms in fp32 add N 2^-24.  The weights -- or weight times page scale,
    in the kernel for many rows -- are held so that a row's largest is at least
    2^10: below 2^-24 of it one is an fp16 subnormal, whose half step is
    2^-25 / 2^10 = 2^-35 of the largest.  The sum of weights is at least the
    largest weight and a code at most 127, so the N weights of a row add at
    most N 2^-35 M.
    out is rounded once to bf16 (2^-8 of its value); lse once to fp32."""
    A, S, N, M = info
    D = out.shape[-1]
    delta = (D + 8) * 2.0 ** -24 * S
    rel = 2 * delta + 2.0 ** -20 + 2 * N * 2.0 ** -24
    tol_out = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + rel)[..., None] * A
    tol_out += (N * 2.0 ** -35 * M)[..., None] + 1e-30
    with np.errstate(invalid="ignore"):
        tol_lse = rel + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0) + 2.0 ** -24
    return tol_out, tol_lse


def bf16(x):
    """fp32 -> the nearest bf16 value (ties to even), as fp32."""
    u = np.ascontiguousarray(x, F32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)).view(F32)

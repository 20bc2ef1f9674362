"""Plain CPU form of the paged-cache operators: the page plan request by request, the append row by row, and
the shared-prefix decode in fp64, one query row at a time over the list of its visible tokens.

A page holds 64 tokens. Position i of a request lives in page table[i // 64] at row i % 64.
"""
import math

import numpy as np

PAGE = 64


def pages(n):
    return (n + PAGE - 1) // PAGE


def page_plan(cache_len, new_len, table, ring, pool, max_tokens):
    """Returns (cu_new, slots, total_len, table, ring, pool) after the step; the inputs are not changed."""
    table, ring = table.copy(), ring.copy()
    B, width = table.shape
    F = len(ring)
    taken, returned = int(pool[0]), int(pool[1])
    available = min(max(returned - taken, 0), F)
    cu, slots, total = [0], [-1] * max_tokens, []
    want = refused = used = back = 0
    for b in range(B):
        c, n = int(cache_len[b]), int(new_len[b])
        rows = cu[-1]
        cu.append(rows + max(n, 0))
        if not 0 <= c <= width * PAGE:
            refused += 1
            total.append(c)
            continue
        if n < 0:
            for j in range(pages(c)):
                ring[(returned + back + j) % F] = table[b, j]
            back += pages(c)
            total.append(0)
            continue
        if n == 0:
            total.append(c)
            continue
        fits = c + n <= width * PAGE and cu[-1] <= max_tokens
        need = pages(c + n) - pages(c) if fits else 0
        first = want
        want += need
        if not fits or (need > 0 and want > available):
            refused += 1
            total.append(c)
            continue
        for j in range(need):
            table[b, pages(c) + j] = ring[(taken + first + j) % F]
        used += need
        for i in range(n):
            slots[rows + i] = int(table[b, (c + i) // PAGE]) * PAGE + (c + i) % PAGE
        total.append(c + n)
    return (np.minimum(np.array(cu, np.int64), 2**31 - 1).astype(np.int32), np.array(slots, np.int64),
            np.array(total, np.int64), table, ring, np.array([taken + used, returned + back, refused], np.int64))


def page_append(K, V, slots, Kp, Vp):
    """Copies of the pools with rows K, V [n, Hkv, D] in their slots (rows outside the pool are skipped)."""
    Kp, Vp = Kp.copy(), Vp.copy()
    for t, slot in enumerate(slots):
        if 0 <= slot < Kp.shape[0] * PAGE:
            Kp[slot // PAGE, :, slot % PAGE] = K[t]
            Vp[slot // PAGE, :, slot % PAGE] = V[t]
    return Kp, Vp


def prefix_decode(q, Kp, Vp, prefix_table, prefix_len, table, own_len, scale):
    """q [B, H, Tq, D]; pools [num_pages, Hkv, 64, D] (any float type, read as fp64).

    Returns a dict of out [B, H, Tq, D], lse [B, H, Tq], and, for error bounds, per row: mean_abs (the
    attention of |V|), reach (the largest scale * sum |q_i k_i| over its keys) and keys (their number)."""
    q = np.asarray(q, np.float64)
    B, H, Tq, D = q.shape
    num_pages, Hkv = Kp.shape[:2]
    prefix_len = min(max(int(prefix_len), 0), len(prefix_table) * PAGE)
    out, mean_abs = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, H, Tq), -math.inf)
    reach, keys = np.zeros((B, H, Tq)), np.zeros((B, H, Tq), np.int64)
    for b in range(B):
        n = min(int(own_len[b]), table.shape[1] * PAGE)
        if n < 0:
            continue
        pos = np.concatenate([np.arange(prefix_len), prefix_len + np.arange(n)])
        page = np.concatenate([np.repeat(prefix_table, PAGE)[:prefix_len], np.repeat(table[b], PAGE)[:n]]).astype(np.int64)
        row = np.concatenate([np.arange(prefix_len) % PAGE, np.arange(n) % PAGE])
        ok = (page >= 0) & (page < num_pages)
        pos, page, row = pos[ok], page[ok], row[ok]
        for h in range(H):
            k = np.asarray(Kp[page, h // (H // Hkv), row], np.float64)
            v = np.asarray(Vp[page, h // (H // Hkv), row], np.float64)
            for i in range(Tq):
                see = pos <= prefix_len + n - Tq + i
                if not see.any():
                    continue
                s = scale * (k[see] @ q[b, h, i])
                e = np.exp(s - s.max())
                w = e / e.sum()
                out[b, h, i], mean_abs[b, h, i] = w @ v[see], w @ np.abs(v[see])
                lse[b, h, i] = s.max() + math.log(e.sum())
                reach[b, h, i] = scale * (np.abs(k[see]) @ np.abs(q[b, h, i])).max()
                keys[b, h, i] = see.sum()
    return dict(out=out, lse=lse, mean_abs=mean_abs, reach=reach, keys=keys)


def prefix_tolerance(ref, D):
    """Elementwise error bounds (out, lse) of a kernel that takes bf16 inputs, sums in fp32 and rounds the
    probabilities and the result to bf16.

    A logit is a sum of D exact products, off by at most D 2^-24 reach, also after the scale and its fused multiply-add. It is
    taken relative to a reference that need not be the row's maximum: some visible logit as the kernel has it, the same number in
    numerator and denominator, added to lse in the end. The difference y, in powers of two, is rounded once, which makes
    ln 2 2^-24 |y| of the exponential, and so is each factor by which sums are brought to another reference. A term is at most 2^70 over
    its reference; one that counts in the end is scaled down by at most that and the 24 bits below which it is lost, and references only
    rise, so the arguments of its factors are 70 + 70 + 24 at most in all: 57 2^-23. The exponentials themselves are off by 2^-22 each, two
    of them: e relative. Numerator and denominator both carry e and the rounding of a sum of ``keys`` terms; the
    numerator's terms are rounded to bf16 (2^-8), and so is the result."""
    e = 2 * D * 2.0**-24 * ref["reach"] + 2 * 2.0**-22 + 57 * 2.0**-23
    sums = (ref["keys"] + 64) * 2.0**-24
    rel = 2 * (e + sums)
    out = (2.0**-8 + rel)[..., None] * ref["mean_abs"] + 2.0**-8 * np.abs(ref["out"])
    lse = e + sums + 2.0**-22 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0)) + 2.0**-22
    return out, lse

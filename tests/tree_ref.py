"""Plain 64-bit forms of the draft-tree and eviction operators over host arrays
(a `workloads.Workload`), and random draft masks."""
import numpy as np
import torch

import workloads as W

BLOCK = W.BLOCK


def values(a):
    """bf16 bit patterns or e4m3 codes -> float64"""
    t = torch.from_numpy(np.ascontiguousarray(a))
    if a.dtype == np.uint16:
        return t.view(torch.int16).view(torch.bfloat16).double().numpy()
    return t.view(torch.float8_e4m3fn).double().numpy()


def _scaled(w, pool, scale, pages, n):
    x = values(pool[pages]).reshape(-1, 128)[:n]
    if w.scale_mode == W.SCALE_SCALAR:
        return x * float(scale[0])
    if w.scale_mode == W.SCALE_PER_TOKEN_HEAD:
        return x * scale[pages].astype(np.float64).reshape(-1, 1)[:n]
    return x


def visible(ctx, qlen, j, words=None, picks=None):
    """Which of the ctx + qlen tokens row j sees."""
    see = np.zeros(ctx + qlen, bool)
    if picks is None:
        see[:ctx] = True
    else:
        whole = ctx // BLOCK
        see[whole * BLOCK:ctx] = True
        for b in picks:
            if 0 <= b < whole:
                see[b * BLOCK:(b + 1) * BLOCK] = True
    for i in range(qlen):
        see[ctx + i] = i <= j if words is None else bool((int(words[i // 32]) >> (i % 32)) & 1)
    return see


def tree_attn(w, mask=None, topk_idx=None, bad=()):
    """out [N, H, 128], lse [N, H], and the absolute-error bounds that a kernel with 16-bit
    P, 32-bit sums and a bf16 result meets.

    Bounds: a logit is a 128-term fp32 sum, off by at most 130 * 2^-23 of the sum of its terms'
    absolute values (truncating accumulation: a whole step per term); 2^x by 2^-22 and P's
    rounding by 2^-8 (bf16; f16 is finer) of each term, so of a = sum p |v|; sums of n terms in
    fp32 by at most n / 32 * 2^-24 per lane chain plus the joins (taken as 2e-5); the bf16 result
    by 2^-8 of itself.  With e4m3 values P is f16, whose steps below 2^-14 are 2^-24: P holds
    2^(x - m) times the token's scale over a power of two r that is at most twice the largest
    scale (1, with one scale or none), and 2^m / den <= 1, so that a weight is off by at most
    2^-25 r, and the result by that times the sum of the visible tokens' |codes|."""
    n, h, _ = w.q.shape
    out, lse = np.zeros((n, h, 128)), np.full((n, h), -np.inf)
    out_tol, lse_tol = np.zeros((n, h, 128)), np.zeros((n, h))
    q = values(w.q)
    if w.sinks is not None:
        lse[:] = w.sinks.astype(np.float64)
    for r in range(w.num_reqs):
        if r in bad:
            continue
        ctx, q0, q1 = int(w.context_lens[r]), int(w.cu_seqlens_q[r]), int(w.cu_seqlens_q[r + 1])
        if q1 == q0:
            continue
        tot = ctx + q1 - q0
        pages = w.block_table[r, :(tot + BLOCK - 1) // BLOCK]
        k, v = _scaled(w, w.k_cache, w.k_scale, pages, tot), _scaled(w, w.v_cache, w.v_scale, pages, tot)
        for j in range(q1 - q0):
            see = visible(ctx, q1 - q0, j, None if mask is None else mask[q0 + j],
                          None if topk_idx is None else topk_idx[q0 + j])
            if not see.any():
                continue
            z = w.softmax_scale * (q[q0 + j] @ k[see].T)
            dz = 130 * 2.0 ** -23 * w.softmax_scale * (np.abs(q[q0 + j]) @ np.abs(k[see]).T)
            m = z.max(1, keepdims=True)
            if w.sinks is not None:
                m = np.maximum(m, w.sinks[:, None])
            p = np.exp(z - m)
            den = p.sum(1, keepdims=True)
            if w.sinks is not None:
                den = den + np.exp(w.sinks[:, None] - m)
            p /= den
            out[q0 + j] = p @ v[see]
            lse[q0 + j] = (m + np.log(den))[:, 0]
            d = dz.max(1, keepdims=True)
            out_tol[q0 + j] = (2.0 ** -8 + 2 * d + 3e-5) * (p @ np.abs(v[see])) + 2.0 ** -8 * np.abs(out[q0 + j]) + 1e-30
            if w.kv_dtype == W.KV_FP8:
                codes = np.abs(values(w.v_cache[pages]).reshape(-1, 128)[:tot][see]).sum(0)
                r16 = 1.0
                if w.scale_mode == W.SCALE_SCALAR:
                    r16 = abs(float(w.v_scale[0]))
                elif w.scale_mode == W.SCALE_PER_TOKEN_HEAD:
                    r16 = 2 * float(np.abs(w.v_scale[pages].reshape(-1)[:tot]).max())
                out_tol[q0 + j] += 2.0 ** -25 * r16 * codes
            lse_tol[q0 + j] = d[:, 0] + 2e-5 + 2.0 ** -22 * np.abs(lse[q0 + j])
    return out, lse, out_tol, lse_tol


def attn_mass(w, lse, mass, mask=None, topk_idx=None, bad=()):
    """The updated weights [P, 128] in 64 bits and their bounds (the same terms as above)."""
    mass = mass.astype(np.float64).copy()
    tol = np.zeros_like(mass)
    q = values(w.q)
    for r in range(w.num_reqs):
        if r in bad:
            continue
        ctx, q0, q1 = int(w.context_lens[r]), int(w.cu_seqlens_q[r]), int(w.cu_seqlens_q[r + 1])
        if q1 == q0:
            continue
        tot = ctx + q1 - q0
        pages = w.block_table[r, :(tot + BLOCK - 1) // BLOCK]
        k = _scaled(w, w.k_cache, w.k_scale, pages, tot)
        got, err = np.zeros(tot), np.zeros(tot)
        for j in range(q1 - q0):
            see = visible(ctx, q1 - q0, j, None if mask is None else mask[q0 + j],
                          None if topk_idx is None else topk_idx[q0 + j])
            live = np.isfinite(lse[q0 + j])
            z = w.softmax_scale * (q[q0 + j][live] @ k[see].T)
            dz = 130 * 2.0 ** -23 * w.softmax_scale * (np.abs(q[q0 + j][live]) @ np.abs(k[see]).T)
            p = np.exp(z - lse[q0 + j][live][:, None].astype(np.float64))
            got[see] += p.sum(0)
            # the exponent's own rounding: a few steps of |s| + |lse| in log2 units
            err[see] += (p * (2 * dz + 2.0 ** -21 * (np.abs(z) + np.abs(lse[q0 + j][live][:, None]) + 1))).sum(0)
        rows = (q1 - q0) * w.hq
        pos = np.arange(tot)
        at = (pages[pos // BLOCK], pos % BLOCK)
        old = np.where(pos < ctx, mass[at], 0.0)
        mass[at] = old + got
        tol[at] = err + rows * 2.0 ** -24 * got + 2.0 ** -23 * np.abs(old + got) + 1e-30
    return mass, tol


def key(x):
    """Orders as the selection does: NaN lowest, -0 equal to 0."""
    return (not np.isnan(x), 0.0 if np.isnan(x) else float(x))


def evict(lens, block_table, mass, budget, first, recent):
    out = np.full((len(lens), budget), -1, np.int32)
    kl = np.zeros(len(lens), np.int32)
    for r, n in enumerate(lens):
        if n <= budget:
            out[r, :n] = np.arange(n)
            kl[r] = n
            continue
        pos = np.arange(n)
        m = mass[block_table[r, pos // BLOCK], pos % BLOCK]
        mid = sorted(range(first, n - recent), key=lambda t: (tuple(-x for x in key(m[t])), t))
        kept = list(range(first)) + mid[:budget - first - recent] + list(range(n - recent, n))
        out[r] = sorted(kept)
        kl[r] = budget
    return out, kl


def compact(pools, lens, block_table, keep, keep_len, base=None, skip=()):
    """Copies of the pools [P, 128, ...] with the kept tokens moved."""
    pools = [p.copy() for p in pools]
    for r in range(len(lens)):
        n, b = int(keep_len[r]), 0 if base is None else int(base[r])
        if n <= 0 or r in skip:
            continue
        src, dst = b + keep[r, :n], b + np.arange(n)
        s = (block_table[r, src // BLOCK], src % BLOCK)
        d = (block_table[r, dst // BLOCK], dst % BLOCK)
        for p in pools:
            p[d] = p[s]
    return pools


def random_mask(rng, q_lens, words, kind="tree"):
    """Draft masks uint32 [N, words]: trees, or arbitrary bits (rows that miss themselves, empty
    rows, bits at and above the request's rows)."""
    out = np.zeros((int(sum(q_lens)), words), np.uint32)
    row = 0
    for n in q_lens:
        anc = []
        for j in range(n):
            if kind == "tree":
                parent = int(rng.integers(-1, j)) if j else -1
                bits = (anc[parent] if parent >= 0 else 0) | (1 << j)
            else:
                bits = 0 if rng.random() < 0.2 else int.from_bytes(rng.bytes(4 * words), "little")
            anc.append(bits)
            out[row] = [(bits >> (32 * x)) & 0xffffffff for x in range(words)]
            row += 1
    return out


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a.view(np.int32) if a.dtype == np.uint32 else a)).cuda()

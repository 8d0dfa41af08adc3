"""Plain 64-bit forms of the prompt operators over host arrays, and batches with several KV heads."""
import dataclasses

import numpy as np
import torch

import workloads as W
from tests.tree_ref import values

BLOCK = W.BLOCK


def batch(seed, q_lens, ctxs, heads=16, kv_heads=1, kv=W.KV_BF16, scale=W.SCALE_NONE, sink=False, **kw):
    """A workload whose pools have kv_heads heads; slots behind a request's end hold NaN."""
    w = W.custom(seed, q_lens, [c + q for c, q in zip(ctxs, q_lens)], hq=heads, kv_dtype=kv, scale_mode=scale,
                 with_sink=sink, fill_unused_nan=True, **kw)
    if kv_heads == 1:
        return w
    rng = np.random.default_rng(seed)
    pools = []
    for pool in (w.k_cache, w.v_cache):
        x = rng.standard_normal((w.num_pages, BLOCK, kv_heads, 128))
        x = W.fp8_codes(x) if kv == W.KV_FP8 else W.bf16_bits(x)
        x[np.broadcast_to(pool_nan(pool), x.shape)] = 0x7f if kv == W.KV_FP8 else 0x7fc0
        pools.append(x)
    w = dataclasses.replace(w, k_cache=pools[0], v_cache=pools[1])
    if scale == W.SCALE_PER_TOKEN_HEAD:
        shape = (w.num_pages, BLOCK, kv_heads)
        w = dataclasses.replace(w, k_scale=rng.lognormal(0, 0.5, shape).astype(np.float32),
                                v_scale=rng.lognormal(0, 0.5, shape).astype(np.float32))
    return w


def pool_nan(pool):
    return np.isnan(values(pool[..., :1]))


def cached(w, name, r, n, head):
    """K or V [n, 128] of one request and KV head in 64 bits."""
    pool, scale = (w.k_cache, w.k_scale) if name == "k" else (w.v_cache, w.v_scale)
    pages = w.block_table[r, :(n + BLOCK - 1) // BLOCK]
    x = values(pool[pages][:, :, head]).reshape(-1, 128)[:n]
    if w.scale_mode == W.SCALE_SCALAR:
        return x * float(scale[0])
    if w.scale_mode == W.SCALE_PER_TOKEN_HEAD:
        return x * scale[pages][:, :, head].astype(np.float64).reshape(-1, 1)[:n]
    return x


def attn(w, bad=()):
    """out [N, H, 128], lse [N, H] and their absolute-error bounds, derived as those of
    tree_ref.tree_attn: a logit is a 128-term fp32 sum (130 steps of 2^-23 of the sum of its terms'
    magnitudes), 2^x and P's rounding 2^-8 of each term, fp32 sums 3e-5, the bf16 result 2^-8 of
    itself; with e4m3 pools P is f16, whose steps below 2^-14 are 2^-24 of a weight kept within a
    factor of two of the largest scale."""
    n, h, _ = w.q.shape
    g = h // w.hkv
    out, lse = np.zeros((n, h, 128)), np.full((n, h), -np.inf)
    out_tol, lse_tol = np.zeros((n, h, 128)), np.zeros((n, h))
    q = torch.from_numpy(values(w.q))
    if w.sinks is not None:
        lse[:] = w.sinks.astype(np.float64)
    for r in range(w.num_reqs):
        ctx, q0, q1 = int(w.context_lens[r]), int(w.cu_seqlens_q[r]), int(w.cu_seqlens_q[r + 1])
        if r in bad or q1 == q0:
            continue
        tot = ctx + q1 - q0
        hide = torch.arange(tot)[None, :] > ctx + torch.arange(q1 - q0)[:, None]
        for head in range(w.hkv):
            k = torch.from_numpy(cached(w, "k", r, tot, head))
            v = torch.from_numpy(cached(w, "v", r, tot, head))
            for i in range(head * g, head * g + g):
                x = q[q0:q1, i]
                z = w.softmax_scale * (x @ k.T)
                z[hide] = -np.inf
                dz = 130 * 2.0 ** -23 * abs(w.softmax_scale) * (x.abs() @ k.abs().T)
                dz[hide] = 0
                m = z.amax(1, keepdim=True)
                if w.sinks is not None:
                    m = m.clamp(min=float(w.sinks[i]))
                p = torch.exp(z - m)
                den = p.sum(1, keepdim=True)
                if w.sinks is not None:
                    den = den + torch.exp(float(w.sinks[i]) - m)
                p = p / den
                o, a, d = p @ v, p @ v.abs(), dz.amax(1, keepdim=True)
                tol = (2.0 ** -8 + 2 * d + 3e-5) * a + 2.0 ** -8 * o.abs() + 1e-30
                if w.kv_dtype == W.KV_FP8:
                    pages = w.block_table[r, :(tot + BLOCK - 1) // BLOCK]
                    codes = np.abs(values(w.v_cache[pages][:, :, head]).reshape(-1, 128)[:tot]).sum(0)
                    r16 = 1.0
                    if w.scale_mode == W.SCALE_SCALAR:
                        r16 = abs(float(w.v_scale[0]))
                    elif w.scale_mode == W.SCALE_PER_TOKEN_HEAD:
                        r16 = 2 * float(np.abs(w.v_scale[pages][:, :, head].reshape(-1)[:tot]).max())
                    tol = tol + torch.from_numpy(2.0 ** -25 * r16 * codes)
                out[q0:q1, i], out_tol[q0:q1, i] = o.numpy(), tol.numpy()
                lse[q0:q1, i] = (m + torch.log(den))[:, 0].numpy()
                lse_tol[q0:q1, i] = d[:, 0].numpy() + 2e-5 + 2.0 ** -22 * np.abs(lse[q0:q1, i])
    return out, lse, out_tol, lse_tol


def check_attn(c, ref, rows=slice(None)):
    out, lse, ot, lt = ref
    got, gl = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    err = np.abs(got - out)[rows]
    assert not np.isnan(got[rows]).any()
    assert (err <= ot[rows]).all(), (np.argwhere(err > ot[rows])[:4].tolist(), (err / (ot[rows] + 1e-300)).max())
    inf = np.isneginf(lse)
    assert np.array_equal(inf[rows], np.isneginf(gl)[rows])
    with np.errstate(invalid="ignore"):
        e = np.where(inf, 0.0, np.abs(gl - lse))[rows]
    assert (e <= lt[rows] + 1e-6 * (np.abs(np.where(inf, 0, lse))[rows] + 1)).all(), e.max()


def through(x, weight, shift, eps, cos_sin, pos, near):
    """Norm and rotation of x [N, h, d] in 64 bits, and the error bound of fp32 arithmetic on it:
    the sum of squares to 16 steps (a chain of 8 and four joins, twice the term itself), the root,
    the two products and the rotation's three operations to a step each, 2^-24 of the magnitudes;
    40 steps cover them."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (weight + shift)
    tol = np.abs(y)
    half = 0 if cos_sin is None else cos_sin.shape[1] // 2
    if half:
        t = cos_sin[pos].astype(np.float64)
        c, s = t[:, None, :half], t[:, None, half:]
        a, b = (np.s_[..., 0:2 * half:2], np.s_[..., 1:2 * half:2]) if near else (np.s_[..., :half], np.s_[..., half:2 * half])
        ya, yb = y[a].copy(), y[b].copy()
        y[a], y[b] = ya * c - yb * s, yb * c + ya * s
        ta, tb = np.abs(ya), np.abs(yb)
        tol[a], tol[b] = ta * np.abs(c) + tb * np.abs(s), tb * np.abs(c) + ta * np.abs(s)
    return y, 40 * 2.0 ** -24 * tol + 1e-30


def fork(lens, table, refs, parent, grow, width, pages):
    """New lens, table (-1 behind a request's blocks), refs, copies by the rules, step by step; the
    status bit that stops the call instead."""
    n = len(parent)
    blocks = lambda x: (x + BLOCK - 1) // BLOCK
    for r, x in enumerate(lens):
        if x < 0 or x > BLOCK * table.shape[1]:
            return 4
    for i in range(n):
        if not -1 <= parent[i] < len(lens) or grow[i] < 0:
            return 4
        if (lens[parent[i]] if parent[i] >= 0 else 0) + grow[i] > BLOCK * width:
            return 4
    bits = 0
    for r, x in enumerate(lens):
        for b in range(blocks(x)):
            if not 0 <= table[r, b] < pages:
                bits |= 1
            elif refs[table[r, b]] < 1:
                bits |= 8
    if bits:
        return bits
    count = refs.astype(np.int64).copy()
    for r, x in enumerate(lens):
        for b in range(blocks(x)):
            count[table[r, b]] -= 1
    out = np.full((n, width), -1, np.int32)
    have = [lens[p] if p >= 0 else 0 for p in parent]
    part = [i for i in range(n) if grow[i] > 0 and have[i] % BLOCK]
    for i in range(n):
        for b in range(have[i] // BLOCK if i in part else blocks(have[i])):
            out[i, b] = table[parent[i], b]
            count[out[i, b]] += 1
    free_to_keep = {table[parent[i], have[i] // BLOCK] for i in part if count[table[parent[i], have[i] // BLOCK]] == 0}
    src, dst, tok = np.full(n, -1, np.int32), np.full(n, -1, np.int32), np.zeros(n, np.int32)
    for i in part:
        page = table[parent[i], have[i] // BLOCK]
        if page in free_to_keep and count[page] == 0:
            out[i, have[i] // BLOCK] = page
            count[page] = 1
        else:
            src[i], tok[i] = page, have[i] % BLOCK
    free = iter(np.flatnonzero(count == 0).tolist())
    try:
        for i in range(n):
            first = have[i] // BLOCK if tok[i] else blocks(have[i])
            for b in range(first, blocks(have[i] + grow[i])):
                page = next(free)
                out[i, b] = page
                count[page] = 1
                if tok[i] and b == first:
                    dst[i] = page
    except StopIteration:
        return 64
    return np.array(have, np.int32), out, count.astype(np.int32), src, dst, tok

"""Workloads of the draft-tree and cache-eviction operators, their plain forms and their exact values.

Four operators over the paged cache of block-sparse decode (one KV head, head dim 128, pages of 128 tokens):

  tree_attn     attention of a request's drafted tokens over its cached tokens and, by a bit mask, over each other;
                one row per request is ordinary single-token decode.  With selected blocks, a row reads of the cached
                whole blocks only those that its top-k names.
  attn_mass     the attention weight that each cached token received from the step's rows, added up per token.
  evict_select  the tokens that a request keeps under a budget: the first, the recent and the heaviest others.
  kv_compact    the kept tokens' K, V, scales, index keys and weights moved together in the pools, in place; the same
                call commits the accepted path of a draft tree.

`run` computes them in elementary torch operations in 32 bits, or, where `own` is set, calls the package.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
DIM = 128
SCALE = 1.0 / math.sqrt(DIM)
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    """Twelve cases; contexts are in tokens, `q_lo`..`q_hi` the drafted rows per request."""
    return [
        # one user's single-token decode over a short chat: launch and latency count
        dict(name="decode_one_short", op="tree_attn", reqs=1, q_lo=1, q_hi=1, ctx_lo=700, ctx_hi=700, heads=8,
             kv="bf16", scales="none", sinks=False, mask=False, topk=0),
        # a full batch of single-token decode on a dense-attention layer, ragged contexts
        dict(name="decode_batch", op="tree_attn", reqs=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=32768, heads=16,
             kv="bf16", scales="none", sinks=False, mask=False, topk=0),
        # small draft trees over an FP8 cache with sinks
        dict(name="verify_small_fp8", op="tree_attn", reqs=8, q_lo=5, q_hi=8, ctx_lo=4000, ctx_hi=16000, heads=8,
             kv="fp8", scales="scalar", sinks=True, mask=True, topk=0),
        # wide draft trees, the tensor cores' case
        dict(name="verify_wide", op="tree_attn", reqs=8, q_lo=48, q_hi=64, ctx_lo=8192, ctx_hi=32768, heads=16,
             kv="bf16", scales="none", sinks=False, mask=True, topk=0),
        # two long documents, FP8 cache with a scale per token, odd tree and head counts
        dict(name="verify_long_fp8", op="tree_attn", reqs=2, q_lo=33, q_hi=33, ctx_lo=100001, ctx_hi=131011, heads=12,
             kv="fp8", scales="token", sinks=True, mask=True, topk=0),
        # draft trees on a block-sparse layer: each row reads its own 16 selected blocks
        dict(name="verify_selected", op="tree_attn", reqs=16, q_lo=16, q_hi=32, ctx_lo=30720, ctx_hi=30720, heads=16,
             kv="bf16", scales="none", sinks=False, mask=True, topk=16),
        # the weights of one decode step of a full batch
        dict(name="mass_decode", op="attn_mass", reqs=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=32768, heads=16,
             kv="bf16", scales="none", sinks=False, mask=False, topk=0),
        # the weights that an observation window of 32 rows gives, FP8 cache with a scale per token
        dict(name="mass_window_fp8", op="attn_mass", reqs=8, q_lo=32, q_hi=32, ctx_lo=8191, ctx_hi=65000, heads=16,
             kv="fp8", scales="token", sinks=True, mask=False, topk=0),
        # a batch that outgrew its budget
        dict(name="evict_batch", op="evict_select", reqs=64, ctx_lo=4096, ctx_hi=32768, budget=2048, first=4,
             recent=256),
        # one long document
        dict(name="evict_long", op="evict_select", reqs=1, ctx_lo=500009, ctx_hi=500009, budget=16384, first=64,
             recent=1024),
        # the pools after an eviction, bf16 with index keys
        dict(name="compact_evicted", op="kv_compact", reqs=32, ctx_lo=8192, ctx_hi=32768, keep=4096, first=4,
             recent=256, tree=0, kv="bf16", scales="none"),
        # the accepted paths of 16 draft trees, FP8 pools with scales
        dict(name="commit_accepted", op="kv_compact", reqs=16, ctx_lo=900, ctx_hi=2900, keep=8, first=0, recent=0,
             tree=48, kv="fp8", scales="token"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_attn(rng, op):
    q_hi = 1 if rng.random() < 0.25 else _log_int(rng, 2, 96)
    reqs = _log_int(rng, 1, 64)
    c = dict(op=op, reqs=reqs, q_lo=max(1, q_hi - rng.randrange(0, 1 + q_hi // 3)), q_hi=q_hi, ctx_lo=0,
             ctx_hi=_log_int(rng, 60, 131072), heads=rng.randint(1, 16), kv=rng.choice(["bf16", "fp8"]),
             scales="none", sinks=rng.random() < 0.5, mask=rng.random() < 0.7,
             topk=rng.choice([0, 0, 0, 4, 16, 32]))
    c["ctx_lo"] = max(1, int(c["ctx_hi"] * rng.uniform(0.05, 1.0)))
    c["scales"] = rng.choice(["none", "scalar", "token"]) if c["kv"] == "fp8" else "none"
    return c


def _draw_any(rng):
    op = rng.choice(["tree_attn", "tree_attn", "attn_mass", "evict_select", "kv_compact"])
    if op in ("tree_attn", "attn_mass"):
        return _draw_attn(rng, op)
    hi = _log_int(rng, 300, 400000)
    reqs = _log_int(rng, 1, 64)
    lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
    if op == "evict_select":
        budget = _log_int(rng, 64, 16384)
        return dict(op=op, reqs=reqs, ctx_lo=lo, ctx_hi=hi, budget=budget, first=rng.randint(0, budget // 8),
                    recent=rng.randint(0, budget // 2))
    kv = rng.choice(["bf16", "fp8"])
    scales = rng.choice(["none", "scalar", "token"]) if kv == "fp8" else "none"
    if rng.random() < 0.5:
        tree = rng.randint(2, 128)
        return dict(op=op, reqs=reqs, ctx_lo=min(lo, 6000), ctx_hi=min(hi, 8000), keep=rng.randint(1, min(tree, 12)),
                    first=0, recent=0, tree=tree, kv=kv, scales=scales)
    keep = _log_int(rng, 64, 16384)
    return dict(op=op, reqs=reqs, ctx_lo=lo, ctx_hi=hi, keep=keep, first=rng.randint(0, keep // 8),
                recent=rng.randint(0, keep // 2), tree=0, kv=kv, scales=scales)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    """One more case: sizes log-uniform over the range, held to the largest listed case of its operator."""
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        c = _draw_any(rng)
        tokens = sum(x + y for x, y in zip(_ctx_lens(c), _q_lens(c)))
        longest = max(x + y for x, y in zip(_ctx_lens(c), _q_lens(c)))
        # the plain form pads to the longest request: bound what it holds
        if tokens > 600000 or c["reqs"] * longest > 2200000 or _cost(c) > top[c["op"]]:
            continue
        if c["op"] in ("tree_attn", "attn_mass") and c["reqs"] * longest * c["q_hi"] * c["heads"] > 280000000:
            continue
        return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, even over their logarithm, in a mixed order."""
    if n == 1:
        return [hi]
    v = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    return random.Random(n).sample(v, n)


def _ctx_lens(case):
    return _spread(case["ctx_lo"], case["ctx_hi"], case["reqs"])


def _q_lens(case):
    """Rows per request: drafted rows, or the tree's slots behind the context of a commit."""
    if case["op"] == "evict_select":
        return [0] * case["reqs"]
    if case["op"] == "kv_compact":
        return [case["tree"]] * case["reqs"]
    lo, hi = case["q_lo"], case["q_hi"]
    return [lo + (5 * i) % (hi - lo + 1) if case["reqs"] > 1 else hi for i in range(case["reqs"])]


def _keep_lens(case):
    """Kept tokens per request: an accepted path of 1 to `keep`, or the budget where the context outgrew it."""
    if case["tree"]:
        return [1 + (3 * i + 1) % case["keep"] for i in range(case["reqs"])]
    return [min(case["keep"], n) for n in _ctx_lens(case)]


def _union(case, ctx, rows):
    """Whole cached blocks, those that one row selects, and those that any row of the request selects."""
    whole = ctx // BLOCK
    if not case["topk"]:
        return whole, whole, whole
    each = min(case["topk"], whole)
    pool = min(whole, each + each // 2)
    return whole, each, (pool if rows > 1 else each)


# ------------------------------------------------------------------ inputs

def _tokens_bytes(case):
    """Bytes of one cached token of K or V, its scale included."""
    return 128 * (1 if case["kv"] == "fp8" else 2) + (4 if case["scales"] == "token" else 0)


def _rand_kv(gen, pages, kv):
    x = torch.randn((pages, BLOCK, 1, DIM), generator=gen, device=DEV, dtype=torch.float32 if pages < 20000 else torch.bfloat16)
    return x.to(torch.bfloat16) if kv == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def _paging(rs, lens):
    """A block table of shuffled pages (-1 behind each request's last block) and the pool's pages."""
    nb = [(n + BLOCK - 1) // BLOCK for n in lens]
    pages = max(1, int(sum(nb) * 1.1) + 1)
    perm = rs.permutation(pages).astype(np.int32)
    bt = np.full((len(lens), max(1, max(nb))), -1, np.int32)
    at = 0
    for r, n in enumerate(nb):
        bt[r, :n] = perm[at:at + n]
        at += n
    return bt, pages


def _tree_masks(rs, q_lens, words):
    """Random draft trees: each token's parent is an earlier one or the context; a row sees its ancestors and itself."""
    out = np.zeros((sum(q_lens), words), np.uint32)
    row = 0
    for n in q_lens:
        anc = []
        for j in range(n):
            parent = int(rs.randint(-1, j)) if j else -1
            anc.append((anc[parent] if parent >= 0 else 0) | (1 << j))
            out[row] = [(anc[j] >> (32 * w)) & 0xffffffff for w in range(words)]
            row += 1
    return out.view(np.int32)


def _selections(rs, case, ctx_lens, q_lens):
    """Per row the ascending selected blocks, -1 behind them: a request's rows share most of their blocks."""
    out = np.full((sum(q_lens), case["topk"]), -1, np.int32)
    row = 0
    for ctx, n in zip(ctx_lens, q_lens):
        whole, each, union = _union(case, ctx, n)
        pool = np.sort(rs.permutation(whole)[:union]) if union else np.zeros(0, np.int64)
        skip = union - each
        for j in range(n):
            if each:
                gone = (np.arange(skip) + j * max(1, skip)) % union
                out[row, :each] = np.delete(pool, gone)[:each]
            row += 1
    return out


def _dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV) if dtype is None else torch.tensor(x, dtype=dtype, device=DEV)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("tree_attn", "attn_mass"):
        return _prepare_attn(case, rs, gen)
    if case["op"] == "evict_select":
        return _prepare_evict(case, rs, gen)
    return _prepare_compact(case, rs, gen)


def _prepare_attn(case, rs, gen):
    ctx, ql = _ctx_lens(case), _q_lens(case)
    lens = [a + b for a, b in zip(ctx, ql)]
    bt, pages = _paging(rs, lens)
    n, h = sum(ql), case["heads"]
    words = (max(ql) + 31) // 32
    s = dict(case=case, pages=pages, rows=n, max_q=max(ql), max_len=max(lens))
    s["cu_q"] = _dev(np.cumsum([0] + ql), torch.int32)
    s["cu_k"] = _dev(np.cumsum([0] + lens), torch.int32)
    s["ctx"] = _dev(ctx, torch.int32)
    s["bt"] = _dev(bt)
    # logits of standard deviation 2: a softmax with some weight on few tokens
    s["q"] = (2.0 * torch.randn((n, h, DIM), generator=gen, device=DEV)).to(torch.bfloat16)
    s["k"], s["v"] = _rand_kv(gen, pages, case["kv"]), _rand_kv(gen, pages, case["kv"])
    shape = {"none": None, "scalar": (1,), "token": (pages, BLOCK, 1)}[case["scales"]]
    for name in ("k_scale", "v_scale"):
        s[name] = None if shape is None else torch.exp(0.3 * torch.randn(shape, generator=gen, device=DEV))
    s["sinks"] = torch.randn((h,), generator=gen, device=DEV) if case["sinks"] else None
    s["mask"] = _dev(_tree_masks(rs, ql, words)) if case["mask"] else None
    s["topk_idx"] = _dev(_selections(rs, case, ctx, ql)) if case["topk"] else None
    s["out"] = torch.empty((n, h, DIM), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((n, h), dtype=torch.float32, device=DEV)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    if case["op"] == "attn_mass":
        _, s["lse"] = _plain_attn(s)
        # weights of earlier steps: a few heavy tokens
        s["mass"] = torch.exp(torch.randn((pages, BLOCK), generator=gen, device=DEV) - 6.0)
    if own:  # the argument structs and the workspace that a serving program keeps beside its buffers
        import block_sparse_paged_02_gb300 as msa
        s["batch"] = msa.make_batch(s["cu_q"], s["cu_k"], s["ctx"], s["bt"], pages, n, max_q_len=max(ql))
        s["tree"] = msa.make_tree(mask=s["mask"], topk_idx=s["topk_idx"])
        s["attn"] = msa.make_attn_args(
            s["q"], s["k"], s["v"], msa.MSA_KV_FP8_E4M3 if case["kv"] == "fp8" else msa.MSA_KV_BF16, pages, s["out"],
            s["lse"], scale_mode={"none": msa.MSA_SCALE_NONE, "scalar": msa.MSA_SCALE_SCALAR,
                                  "token": msa.MSA_SCALE_PER_TOKEN_HEAD}[case["scales"]],
            k_scale=s["k_scale"], v_scale=s["v_scale"], sinks=s["sinks"], softmax_scale=SCALE)
        ws = msa.msa_tree_attn_workspace_size(case["reqs"], n, bt.shape[1], h, max(ql), case["topk"])
        s["ws"] = torch.empty((max(ws, 16),), dtype=torch.uint8, device=DEV)
    return s


def _prepare_evict(case, rs, gen):
    lens = _ctx_lens(case)
    bt, pages = _paging(rs, lens)
    s = dict(case=case, pages=pages, max_len=max(lens))
    s["lens"], s["bt"] = _dev(lens, torch.int32), _dev(bt)
    # accumulated weights: heavy-tailed, and a third of the tokens never attended to (ties at zero)
    m = torch.exp(2.0 * torch.randn((pages, BLOCK), generator=gen, device=DEV) - 4.0)
    s["mass"] = torch.where(torch.rand((pages, BLOCK), generator=gen, device=DEV) < 0.33, torch.zeros_like(m), m)
    s["keep"] = torch.empty((case["reqs"], case["budget"]), dtype=torch.int32, device=DEV)
    s["keep_len"] = torch.empty((case["reqs"],), dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    if own:
        import block_sparse_paged_02_gb300 as msa
        s["cache"] = msa.make_cache_view(s["lens"], s["bt"], pages)
    return s


def _prepare_compact(case, rs, gen):
    ctx, kl = _ctx_lens(case), _keep_lens(case)
    lens = [c + case["tree"] for c in ctx]
    bt, pages = _paging(rs, lens)
    keep = np.full((case["reqs"], case["keep"]), -1, np.int32)
    for r, n in enumerate(kl):
        if case["tree"]:
            keep[r, :n] = np.sort(rs.permutation(case["tree"])[:n])
            continue
        first, recent = min(case["first"], n), min(case["recent"], n)
        recent = min(recent, n - first)
        mid = n - first - recent
        keep[r, :first] = np.arange(first)
        keep[r, first:first + mid] = first + np.sort(rs.permutation(ctx[r] - first - recent)[:mid])
        keep[r, first + mid:n] = np.arange(ctx[r] - recent, ctx[r])
    s = dict(case=case, pages=pages)
    s["lens"], s["bt"] = _dev(lens, torch.int32), _dev(bt)
    s["base"] = _dev(ctx, torch.int32) if case["tree"] else None
    s["keep"], s["keep_len"] = _dev(keep), _dev(kl, torch.int32)
    s["k"], s["v"], s["idx"] = (_rand_kv(gen, pages, case["kv"]) for _ in range(3))
    for name in ("k_scale", "v_scale", "idx_scale"):
        s[name] = torch.exp(0.3 * torch.randn((pages, BLOCK, 1), generator=gen, device=DEV)) if case["scales"] == "token" else None
    s["mass"] = torch.rand((pages, BLOCK), generator=gen, device=DEV)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    if own:
        import block_sparse_paged_02_gb300 as msa
        kind = msa.MSA_KV_FP8_E4M3 if case["kv"] == "fp8" else msa.MSA_KV_BF16
        s["cache"] = msa.make_cache_view(s["lens"], s["bt"], pages)
        s["pools"] = msa.make_kv_pools(
            s["k"], s["v"], kind, scale_mode=msa.MSA_SCALE_PER_TOKEN_HEAD if case["scales"] == "token" else msa.MSA_SCALE_NONE,
            k_scale=s["k_scale"], v_scale=s["v_scale"], index=msa.make_index_cache(s["idx"], kind, s["idx_scale"]),
            mass=s["mass"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op == "tree_attn":
        if own:
            import block_sparse_paged_02_gb300 as msa
            msa.msa_tree_attn(s["batch"], s["tree"], s["attn"], s["ws"], s["status"])
            return {"out": s["out"], "lse": s["lse"]}
        out, lse = _plain_attn(s)
        return {"out": out, "lse": lse}
    if op == "attn_mass":
        if own:
            import block_sparse_paged_02_gb300 as msa
            msa.msa_attn_mass(s["batch"], s["tree"], s["attn"], s["mass"], s["ws"], s["status"])
        else:
            _plain_mass(s)
        return {"mass": s["mass"]}
    if op == "evict_select":
        if own:
            import block_sparse_paged_02_gb300 as msa
            msa.msa_evict_select(s["cache"], s["mass"], s["case"]["budget"], s["case"]["first"], s["case"]["recent"],
                                 s["keep"], s["keep_len"], s["status"])
            return {"keep": s["keep"], "keep_len": s["keep_len"]}
        return _plain_evict(s)
    if own:
        import block_sparse_paged_02_gb300 as msa
        msa.msa_kv_compact(s["cache"], s["base"], s["keep"], s["keep_len"], s["pools"], s["status"])
    else:
        _plain_compact(s)
    codes = torch.float8_e4m3fn if s["case"]["kv"] == "fp8" else torch.bfloat16
    out = {name: s[name].view(codes) for name in ("k", "v", "idx")}
    return out | {name: s[name] for name in ("k_scale", "v_scale", "idx_scale", "mass") if s[name] is not None}


def _slots(s, width):
    """Flat pool slots [R, width] of each request's positions (page 0 behind its end), and the positions."""
    pos = torch.arange(width, device=DEV)
    page = s["bt"].long()[:, pos // BLOCK].clamp(min=0)
    return page * BLOCK + pos % BLOCK, pos


def _gathered(pool, scale, slots):
    x = pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool
    x = x.view(-1, DIM)[slots].float()
    if scale is None:
        return x
    return x * (scale if scale.numel() == 1 else scale.view(-1)[slots].unsqueeze(-1))


def _plain_logits(s):
    """Logits [R, T, H, L] with -inf where a row does not see a token; the slots and each padded row's index."""
    t = s["max_q"]
    slots, pos = _slots(s, s["max_len"])
    j = torch.arange(t, device=DEV)
    cu = s["cu_q"].long()
    rows = (cu[:-1, None] + j).clamp(max=s["rows"] - 1)          # [R, T]
    there = j < (cu[1:] - cu[:-1])[:, None]                      # [R, T]
    q = s["q"].float()[rows]                                     # [R, T, H, D]
    k = _gathered(s["k"], s["k_scale"], slots)                   # [R, L, D]
    z = (q.flatten(1, 2) @ k.transpose(1, 2)).unflatten(1, (t, -1)) * SCALE
    ctx = s["ctx"].long()[:, None, None]
    i = pos - ctx                                                # [R, 1, L], the drafted token's index
    ic = i.clamp(0, t - 1)
    if s["mask"] is not None:
        words = s["mask"].long()[rows]                           # [R, T, W]
        word = torch.gather(words, 2, (ic // 32).expand(-1, t, -1))
        bit = (word >> (ic % 32)) & 1
        seen = bit.bool()
    else:
        seen = ic <= j[:, None]
    draft = seen & (i >= 0) & (i < (cu[1:] - cu[:-1])[:, None, None])
    cached = (i < 0).expand(-1, t, -1)
    if s["topk_idx"] is not None:
        blocks = s["bt"].shape[1]
        sel = s["topk_idx"].long()[rows]                         # [R, T, K]
        named = torch.zeros((*rows.shape, blocks + 1), dtype=torch.bool, device=DEV)
        named.scatter_(2, torch.where(sel < 0, blocks, sel), True)
        block = pos // BLOCK
        cached = cached & (named[:, :, :blocks][:, :, block] | (block >= ctx // BLOCK))
    visible = (cached | draft) & there[:, :, None]
    return z.masked_fill(~visible[:, :, None], -math.inf), slots, rows[there], there


def _plain_attn(s):
    z, slots, rows, there = _plain_logits(s)
    m = z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        m = torch.maximum(m, s["sinks"][None, None, :, None])
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(z - m)
    den = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + torch.exp(s["sinks"][None, None, :, None] - m)
    v = _gathered(s["v"], s["v_scale"], slots)
    o = (p.flatten(1, 2) @ v).unflatten(1, z.shape[1:3]) / den
    lse = (m + torch.log(den)).squeeze(-1)
    return o[there].to(torch.bfloat16), lse[there]


def _plain_mass(s):
    z, slots, rows, there = _plain_logits(s)
    lse = s["lse"][(s["cu_q"].long()[:-1, None] + torch.arange(s["max_q"], device=DEV)).clamp(max=s["rows"] - 1)]
    w = torch.exp(z - lse[..., None]).sum((1, 2))                # [R, L]
    _, pos = _slots(s, s["max_len"])
    ctx = s["ctx"].long()[:, None]
    new = (pos >= ctx) & (pos < ctx + (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None])
    mass = s["mass"].view(-1)
    old = torch.where(new, 0.0, mass[slots])                     # this step's tokens start at zero
    live = (pos < ctx) | new
    mass[slots[live]] = (old + w)[live]


def _plain_evict(s):
    c = s["case"]
    slots, pos = _slots(s, max(s["max_len"], c["budget"]) if s["bt"].shape[1] * BLOCK >= c["budget"] else s["max_len"])
    n = s["lens"].long()[:, None]
    v = s["mass"].view(-1)[slots]
    v = torch.where((pos < c["first"]) | (pos >= n - c["recent"]), math.inf, v)
    v = torch.where(pos < n, v, -math.inf)
    order = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :c["budget"]]
    kept = torch.minimum(n, torch.tensor(c["budget"], device=DEV))
    rank = torch.arange(order.shape[1], device=DEV)
    big = 1 << 40
    order = torch.where(rank < kept, order, big).sort(1).values
    out = torch.full((c["reqs"], c["budget"]), -1, dtype=torch.int32, device=DEV)
    out[:, :order.shape[1]] = torch.where(order == big, -1, order).int()
    return {"keep": out, "keep_len": kept.squeeze(1).int()}


def _plain_compact(s):
    keep, kl = s["keep"].long(), s["keep_len"].long()[:, None]
    i = torch.arange(keep.shape[1], device=DEV)
    base = s["base"].long()[:, None] if s["base"] is not None else torch.zeros_like(kl)
    live = i < kl
    bt = s["bt"].long()

    def flat(pos):
        pos = torch.where(live, pos, 0)
        return (torch.gather(bt, 1, pos // BLOCK) * BLOCK + pos % BLOCK)[live]

    src, dst = flat(base + keep), flat(base + i)
    rows = [s[n].view(-1, DIM) for n in ("k", "v", "idx")]
    rows += [s[n].view(-1) for n in ("k_scale", "v_scale", "idx_scale", "mass") if s[n] is not None]
    for x in rows:
        x[dst] = x[src]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    """Bytes of the visited tokens, queries, masks and results; multiply-adds of the visible (row, token) pairs."""
    ctx, ql = _ctx_lens(case), _q_lens(case)
    if case["op"] == "evict_select":
        return {"bytes": 4.0 * sum(ctx) + 4.0 * sum(min(n, case["budget"]) for n in ctx), "flops": 0.0}
    if case["op"] == "kv_compact":
        kl = _keep_lens(case)
        moved = sum(n - min(case["first"], n) if n < c or case["tree"] else 0 for n, c in zip(kl, ctx))
        return {"bytes": moved * 2.0 * (3 * _tokens_bytes(case) + 4) + 4.0 * sum(kl), "flops": 0.0}
    h, b = case["heads"], 0.0
    pairs = 0.0
    for c, t in zip(ctx, ql):
        whole, each, union = _union(case, c, t)
        tail = c - whole * BLOCK
        tokens = union * BLOCK + tail + t
        pairs += t * (each * BLOCK + tail + 1)
        b += tokens * _tokens_bytes(case) * (2 if case["op"] == "tree_attn" else 1)
        if case["op"] == "attn_mass":
            b += 8.0 * tokens
    n = sum(ql)
    b += n * h * (2.0 * DIM + 4) + (n * h * 2.0 * DIM if case["op"] == "tree_attn" else 0.0)
    b += n * (4.0 * case["topk"] + (4.0 * ((max(ql) + 31) // 32) if case["mask"] else 0.0))
    return {"bytes": b, "flops": pairs * h * DIM * (4.0 if case["op"] == "tree_attn" else 2.0)}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    """Request by request in 64 bits; None for the operators whose results are indexes or copies."""
    if case["op"] not in ("tree_attn", "attn_mass"):
        return None
    s = prepare(case, seed)
    ctx, cu, bt = s["ctx"].tolist(), s["cu_q"].tolist(), s["bt"]
    as_values = (lambda x: x.view(torch.float8_e4m3fn).double()) if case["kv"] == "fp8" else (lambda x: x.double())
    outs, lses = [], []
    mass = s["mass"].double() if case["op"] == "attn_mass" else None
    for r, c in enumerate(ctx):
        rows = range(cu[r], cu[r + 1])
        n = c + len(rows)
        pages = bt[r, :(n + BLOCK - 1) // BLOCK].long()
        keys, vals = (as_values(s[x][pages]).reshape(-1, DIM)[:n] for x in ("k", "v"))
        if case["scales"] == "scalar":
            keys, vals = keys * s["k_scale"].double(), vals * s["v_scale"].double()
        if case["scales"] == "token":
            keys, vals = (a * s[b][pages].double().reshape(-1, 1)[:n] for a, b in ((keys, "k_scale"), (vals, "v_scale")))
        got = torch.zeros(n, dtype=torch.float64, device=DEV)
        words = s["mask"][cu[r]:cu[r + 1]].cpu().numpy().view(np.uint32) if case["mask"] else None
        picks = s["topk_idx"][cu[r]:cu[r + 1]].cpu().numpy() if case["topk"] else None
        for j in range(len(rows)):
            see = np.zeros(n, bool)
            if picks is None:
                see[:c] = True
            else:
                see[c // BLOCK * BLOCK:c] = True
                for blk in picks[j]:
                    if 0 <= blk < c // BLOCK:
                        see[blk * BLOCK:(blk + 1) * BLOCK] = True
            for i in range(len(rows)):
                see[c + i] = bool(words[j, i // 32] >> (i % 32) & 1) if words is not None else i <= j
            at = torch.from_numpy(np.flatnonzero(see)).to(DEV)
            z = s["q"][rows[j]].double() @ keys[at].T * SCALE    # [H, seen]
            if mass is None:
                every = z if s["sinks"] is None else torch.cat([z, s["sinks"].double()[:, None]], 1)
                den = torch.logsumexp(every, 1)
                outs.append(torch.exp(z - den[:, None]) @ vals[at])
                lses.append(den)
            else:
                got[at] += torch.exp(z - s["lse"][rows[j]].double()[:, None]).sum(0)
        if mass is not None:
            flat = (pages[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).reshape(-1)[:n]
            got[:c] += mass.view(-1)[flat[:c]]
            mass.view(-1)[flat] = got
    if mass is not None:
        return {"mass": mass}
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}

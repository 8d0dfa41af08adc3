"""Workloads of the operators that bring a prompt into the paged cache and share its pages, their plain forms and their
exact values.

Four operators over the paged cache of block-sparse decode (head dim 128, pages of 128 tokens):

  qk_rope_insert  the new tokens' queries and keys normed per head and rotated by position, K, V and index keys written
                  into the pools (bf16, or e4m3 with or without scales), queries and index queries handed on.
  prompt_attn     causal attention of whole prompts, or of their chunks behind cached tokens, over the cache: packed
                  sequences of different lengths, grouped heads.
  page_fork       the tables and reference counts of the requests that go on after a step: forked, reordered, dropped
                  and grown ones; full pages are shared, a partial last page gets an owner or a copy.
  page_copy       the pages that a fork says to copy, in every pool of several layers.

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
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    """Twelve cases; `q_lo`..`q_hi` are the new tokens of a request, `ctx_lo`..`ctx_hi` those cached before."""
    return [
        # the new tokens of one user's decode step: launch and latency count
        dict(name="insert_one", op="qk_rope_insert", reqs=1, q_lo=1, q_hi=1, ctx_lo=700, ctx_hi=700, heads=8, kv_heads=1,
             idx_heads=1, idx_dim=128, rotary=64, near=False, norm=True, shift=0.0, kv="bf16", scales="none", given=False),
        # a full batch's decode step into an FP8 cache with a scale per token, index keys in e4m3 too
        dict(name="insert_batch_fp8", op="qk_rope_insert", reqs=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=8192, heads=16,
             kv_heads=1, idx_heads=1, idx_dim=128, rotary=64, near=False, norm=True, shift=1.0, kv="fp8", scales="token",
             given=False),
        # chunks of several prompts in one step, two index heads, rotation of neighbours over the whole head
        dict(name="insert_prompts", op="qk_rope_insert", reqs=7, q_lo=501, q_hi=4093, ctx_lo=1, ctx_hi=9000, heads=16,
             kv_heads=1, idx_heads=2, idx_dim=64, rotary=64, near=True, norm=True, shift=0.0, kv="bf16", scales="none",
             given=False),
        # a short question
        dict(name="prompt_short", op="prompt_attn", reqs=1, q_lo=200, q_hi=200, ctx_lo=0, ctx_hi=0, heads=8, kv_heads=1,
             kv="bf16", scales="none", sinks=False),
        # a batch of prompts of mixed lengths
        dict(name="prompt_batch", op="prompt_attn", reqs=16, q_lo=97, q_hi=4001, ctx_lo=0, ctx_hi=0, heads=16, kv_heads=1,
             kv="bf16", scales="none", sinks=False),
        # one long document
        dict(name="prompt_long", op="prompt_attn", reqs=1, q_lo=16384, q_hi=16384, ctx_lo=0, ctx_hi=0, heads=16, kv_heads=1,
             kv="bf16", scales="none", sinks=False),
        # chunks of long documents behind an FP8 cache with a scale per token
        dict(name="prompt_chunk_fp8", op="prompt_attn", reqs=2, q_lo=511, q_hi=512, ctx_lo=30001, ctx_hi=60000, heads=12,
             kv_heads=1, kv="fp8", scales="token", sinks=True),
        # several KV heads on one device, groups of six, sinks
        dict(name="prompt_grouped", op="prompt_attn", reqs=4, q_lo=1000, q_hi=2500, ctx_lo=0, ctx_hi=700, heads=24, kv_heads=4,
             kv="bf16", scales="none", sinks=True),
        # a step of beam search: 64 requests of 4 beams, each beam going on from any of its request's
        dict(name="fork_beams", op="page_fork", groups=64, width=4, spread=4, ctx_lo=512, ctx_hi=8192, grow=1, kind="beams"),
        # long prompts, each sampled 16 times
        dict(name="fork_samples", op="page_fork", groups=8, width=1, spread=16, ctx_lo=8000, ctx_hi=65000, grow=256,
             kind="samples"),
        # the partial pages that a step of beam search copies, in the pools of one layer
        dict(name="copy_beams", op="page_copy", copies=96, layers=1, kv="bf16", scales="none", kv_heads=1),
        # the last pages of sampled prompts in all the layers of a model with an FP8 cache
        dict(name="copy_layers_fp8", op="page_copy", copies=120, layers=40, kv="fp8", scales="token", kv_heads=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_insert(rng):
    q_hi = 1 if rng.random() < 0.4 else _log_int(rng, 2, 6000)
    idx_heads, idx_dim = rng.choice([(1, 128), (1, 64), (2, 64), (0, 0)])
    kv = rng.choice(["bf16", "fp8"])
    kv_heads = rng.choice([1, 1, 1, 2, 3])
    return dict(op="qk_rope_insert", reqs=_log_int(rng, 1, 64), q_lo=max(1, q_hi - rng.randrange(0, 1 + q_hi // 2)), q_hi=q_hi,
                ctx_lo=0, ctx_hi=_log_int(rng, 60, 60000), heads=kv_heads * rng.randint(1, 16 // kv_heads), kv_heads=kv_heads,
                idx_heads=idx_heads, idx_dim=idx_dim, rotary=rng.choice([0, 16, 32, 48, 64] + ([96, 128] if idx_dim != 64 else [])),
                near=rng.random() < 0.5, norm=rng.random() < 0.8, shift=rng.choice([0.0, 1.0]), kv=kv,
                scales=rng.choice(["none", "scalar", "token"]) if kv == "fp8" else "none", given=rng.random() < 0.3)


def _draw_prompt(rng):
    kv_heads = rng.choice([1, 1, 1, 2, 4, 8])
    q_hi = _log_int(rng, 1, 16384)
    kv = rng.choice(["bf16", "bf16", "fp8"])
    return dict(op="prompt_attn", reqs=_log_int(rng, 1, 32), q_lo=max(1, int(q_hi * rng.uniform(0.03, 1.0))), q_hi=q_hi,
                ctx_lo=0, ctx_hi=0 if rng.random() < 0.5 else _log_int(rng, 1, 100000),
                heads=kv_heads * rng.randint(1, 16 if kv_heads < 4 else 8), kv_heads=kv_heads, kv=kv,
                scales=rng.choice(["none", "scalar", "token"]) if kv == "fp8" else rng.choice(["none", "none", "none", "token"]),
                sinks=rng.random() < 0.5)


def _draw_any(rng):
    op = rng.choice(["qk_rope_insert", "prompt_attn", "prompt_attn", "page_fork", "page_copy"])
    if op == "qk_rope_insert":
        return _draw_insert(rng)
    if op == "prompt_attn":
        return _draw_prompt(rng)
    if op == "page_fork":
        kind = rng.choice(["beams", "samples"])
        width = rng.randint(2, 8) if kind == "beams" else 1
        hi = _log_int(rng, 100, 100000)
        return dict(op=op, groups=_log_int(rng, 1, 64), width=width, spread=width if kind == "beams" else rng.randint(1, 16),
                    ctx_lo=max(1, int(hi * rng.uniform(0.05, 1.0))), ctx_hi=hi, grow=rng.choice([0, 1, 1, 17, 300]), kind=kind)
    kv = rng.choice(["bf16", "fp8"])
    return dict(op=op, copies=_log_int(rng, 1, 300), layers=_log_int(rng, 1, 64), kv=kv,
                scales=rng.choice(["none", "scalar", "token"]) if kv == "fp8" else "none", kv_heads=rng.choice([1, 1, 2, 4]))


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
        if c["op"] in ("qk_rope_insert", "prompt_attn"):
            if c["ctx_hi"]:
                c["ctx_lo"] = max(0, int(c["ctx_hi"] * rng.uniform(0.02, 1.0)))
            tokens = sum(_ctx_lens(c)) + sum(_q_lens(c))
            if tokens * c["kv_heads"] > 700000 or sum(_q_lens(c)) > 30000:
                continue
        if _cost(c) > top[c["op"]]:
            continue
        return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, even over their logarithm, in a mixed order."""
    if n == 1 or lo == hi:
        return [hi] * n
    v = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    return random.Random(n).sample(v, n)


def _ctx_lens(case):
    return _spread(case["ctx_lo"], case["ctx_hi"], case["reqs"])


def _q_lens(case):
    return _spread(case["q_lo"], case["q_hi"], case["reqs"])[::-1]


def _copy_tokens(case):
    """Tokens of each copied page: partial pages of every fill."""
    return [1 + (37 * i + 60) % 127 for i in range(case["copies"])]


def _fork_sets(case, rs):
    """Old lengths, the number of shared prefix pages of each group, parents and growth."""
    base = _spread(case["ctx_lo"], case["ctx_hi"], case["groups"])
    lens, shared, parent, grow = [], [], [], []
    for g, n in enumerate(base):
        first = g * case["width"]
        for b in range(case["width"]):
            lens.append(n)
            shared.append(n // BLOCK if case["kind"] == "beams" and case["width"] > 1 else 0)
        for b in range(case["spread"]):
            parent.append(first + (int(rs.randint(0, case["width"])) if case["kind"] == "beams" else 0))
            grow.append(case["grow"] if case["grow"] < 2 else 1 + (case["grow"] * (b + 1)) // case["spread"])
    return lens, shared, parent, grow


# ------------------------------------------------------------------ inputs

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


def _dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV) if dtype is None else torch.tensor(x, dtype=dtype, device=DEV)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)


def _pool(gen, pages, heads, dim, kv):
    x = _normal(gen, (pages, BLOCK, heads, dim), "bf16")
    return x if kv == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def _scale(gen, pages, heads, scales):
    shape = {"none": None, "scalar": (1,), "token": (pages, BLOCK, heads)}[scales]
    return None if shape is None else torch.exp(0.3 * torch.randn(shape, generator=gen, device=DEV))


def _kinds(case):
    import block_sparse_paged_02_gb300 as msa
    return (msa.MSA_KV_FP8_E4M3 if case["kv"] == "fp8" else msa.MSA_KV_BF16,
            {"none": msa.MSA_SCALE_NONE, "scalar": msa.MSA_SCALE_SCALAR, "token": msa.MSA_SCALE_PER_TOKEN_HEAD}[case["scales"]])


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"qk_rope_insert": _prepare_insert, "prompt_attn": _prepare_prompt, "page_fork": _prepare_fork,
            "page_copy": _prepare_copy}[case["op"]](case, rs, gen)


def _geometry(case, rs):
    ctx, ql = _ctx_lens(case), _q_lens(case)
    lens = [a + b for a, b in zip(ctx, ql)]
    bt, pages = _paging(rs, lens)
    s = dict(case=case, pages=pages, rows=sum(ql), ql=ql, ctxs=ctx)
    s["cu_q"] = _dev(np.cumsum([0] + ql), torch.int32)
    s["cu_k"] = _dev(np.cumsum([0] + lens), torch.int32)
    s["ctx"] = _dev(ctx, torch.int32)
    s["bt"] = _dev(bt)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    if own:
        import block_sparse_paged_02_gb300 as msa
        s["batch"] = msa.make_batch(s["cu_q"], s["cu_k"], s["ctx"], s["bt"], pages, s["rows"], max_q_len=max(ql))
    return s


def _prepare_insert(case, rs, gen):
    s = _geometry(case, rs)
    n, h, hk, hi, di = s["rows"], case["heads"], case["kv_heads"], case["idx_heads"], case["idx_dim"]
    # the output of one projection: q, k, v, index q and index k side by side
    width = (h + 2 * hk) * DIM + 2 * hi * di
    x = 1.7 * _normal(gen, (n, width), "f32")
    s["proj"] = x.to(torch.bfloat16)
    parts = torch.split(s["proj"], [h * DIM, hk * DIM, hk * DIM, hi * di, hi * di], dim=1)
    for name, part, heads, dim in zip(("q", "k", "v", "idx_q", "idx_k"), parts, (h, hk, hk, hi, hi), (DIM, DIM, DIM, di, di)):
        s[name] = part.unflatten(1, (heads, dim)) if heads else None
    for name, dim in (("q_norm", DIM), ("k_norm", DIM), ("idx_q_norm", di), ("idx_k_norm", di)):
        w = 1.0 - case["shift"] + 0.2 * torch.randn((dim,), generator=gen, device=DEV)
        s[name] = w.to(torch.bfloat16) if case["norm"] and dim else None
    # the table of a model with a context of 128 K tokens, angles in 64 bits
    half = case["rotary"] // 2
    top = 131072
    s["cos_sin"] = None
    if half:
        freq = 5e6 ** -(torch.arange(half, device=DEV, dtype=torch.float64) / half)
        angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["positions"] = _dev(rs.randint(0, top, n), torch.int32) if case["given"] else None
    s["k_pool"], s["v_pool"] = (_pool(gen, s["pages"], hk, DIM, case["kv"]) for _ in range(2))
    s["k_scale"], s["v_scale"] = (_scale(gen, s["pages"], hk, case["scales"]) for _ in range(2))
    s["idx_pool"] = _pool(gen, s["pages"], hi, di, case["kv"]) if hi else None
    s["idx_scale"] = _scale(gen, s["pages"], hi, case["scales"]) if hi and case["scales"] == "token" else None
    s["q_out"] = torch.empty((n, h, DIM), dtype=torch.bfloat16, device=DEV)
    s["idx_q_out"] = torch.empty((n, hi, di), dtype=torch.bfloat16, device=DEV) if hi else None
    if own:
        import block_sparse_paged_02_gb300 as msa
        kind, mode = _kinds(case)
        s["qkv"] = msa.make_qkv(s["q"], s["k"], s["v"], s["q_out"], idx_q=s["idx_q"], idx_k=s["idx_k"], idx_q_out=s["idx_q_out"],
                                q_norm=s["q_norm"], k_norm=s["k_norm"], idx_q_norm=s["idx_q_norm"], idx_k_norm=s["idx_k_norm"],
                                eps=EPS, norm_shift=case["shift"])
        s["rope"] = msa.make_rope(s["cos_sin"], interleaved=case["near"], positions=s["positions"])
        index = msa.make_index_cache(s["idx_pool"], kind, s["idx_scale"]) if hi else None
        s["pools"] = msa.make_kv_pools(s["k_pool"], s["v_pool"], kind, scale_mode=mode, k_scale=s["k_scale"],
                                       v_scale=s["v_scale"], index=index)
    return s


def _prepare_prompt(case, rs, gen):
    s = _geometry(case, rs)
    n, h, hk = s["rows"], case["heads"], case["kv_heads"]
    # logits of standard deviation 2: a softmax with some weight on few tokens
    s["q"] = (2.0 * _normal(gen, (n, h, DIM), "f32")).to(torch.bfloat16)
    s["k"], s["v"] = (_pool(gen, s["pages"], hk, DIM, case["kv"]) for _ in range(2))
    s["k_scale"], s["v_scale"] = (_scale(gen, s["pages"], hk, case["scales"]) for _ in range(2))
    s["sinks"] = torch.randn((h,), generator=gen, device=DEV) if case["sinks"] else None
    s["out"] = torch.empty((n, h, DIM), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((n, h), dtype=torch.float32, device=DEV)
    if own:
        import block_sparse_paged_02_gb300 as msa
        kind, mode = _kinds(case)
        s["attn"] = msa.make_attn_args(s["q"], s["k"], s["v"], kind, s["pages"], s["out"], s["lse"], scale_mode=mode,
                                       k_scale=s["k_scale"], v_scale=s["v_scale"], sinks=s["sinks"], softmax_scale=SCALE)
        s["ws"] = torch.empty((max(16, msa.msa_prompt_attn_workspace_size(h, hk)),), dtype=torch.uint8, device=DEV)
    return s


def _prepare_fork(case, rs, gen):
    lens, shared, parent, grow = _fork_sets(case, rs)
    nb = [(n + BLOCK - 1) // BLOCK for n in lens]
    most = max((lens[p] + g + BLOCK - 1) // BLOCK for p, g in zip(parent, grow))
    old = np.full((len(lens), max(nb)), -1, np.int32)
    pages = int(1.25 * (sum(nb) + sum((lens[p] % BLOCK > 0) + g // BLOCK + 2 for p, g in zip(parent, grow)))) + 8
    perm = rs.permutation(pages).astype(np.int32)
    refs = np.zeros(pages, np.int32)
    at = 0
    for r, n in enumerate(nb):
        head = shared[r] if r % case["width"] else 0    # a beam holds its group's pages, and its own last one
        old[r, :head] = old[r - r % case["width"], :head]
        old[r, head:n] = perm[at:at + n - head]
        at += n - head
        np.add.at(refs, old[r, :n], 1)
    # a prefix cache holds some pages of its own
    refs[perm[:at:5]] += 1
    refs[perm[at:at + (pages - at) // 8]] = 1
    s = dict(case=case, pages=pages, n_old=len(lens), n_new=len(parent), width=max(nb), wide=most)
    s["lens"], s["bt"], s["refs"] = _dev(lens, torch.int32), _dev(old), _dev(refs)
    s["parent"], s["grow"] = _dev(parent, torch.int32), _dev(grow, torch.int32)
    n = len(parent)
    s["new_bt"] = torch.full((n, most), -1, dtype=torch.int32, device=DEV)
    s["new_refs"] = torch.empty_like(s["refs"])
    for name in ("new_lens", "copy_src", "copy_dst", "copy_tokens"):
        s[name] = torch.empty((n,), dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    if own:
        import block_sparse_paged_02_gb300 as msa
        s["from"] = msa.make_cache_view(s["lens"], s["bt"], pages)
        s["to"] = msa.make_page_set(s["new_lens"], s["new_bt"], s["new_refs"], s["copy_src"], s["copy_dst"], s["copy_tokens"])
    return s


def _prepare_copy(case, rs, gen):
    tokens = _copy_tokens(case)
    pages = 2 * case["copies"] + 5
    perm = rs.permutation(pages).astype(np.int32)
    s = dict(case=case, pages=pages)
    s["src"], s["dst"] = _dev(perm[:case["copies"]]), _dev(perm[case["copies"]:2 * case["copies"]])
    s["tokens"] = _dev(tokens, torch.int32)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=DEV)
    # one allocation of each kind for all the layers
    heads = {"k": case["kv_heads"], "v": case["kv_heads"], "idx": 1}
    s["all"] = {}
    for name, n in heads.items():
        x = _normal(gen, (case["layers"], pages, BLOCK, n, DIM), "bf16")
        s["all"][name] = x if case["kv"] == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)
    if case["scales"] == "token":
        for name, n in heads.items():
            s["all"][name + "_scale"] = torch.exp(0.3 * torch.randn((case["layers"], pages, BLOCK, n), generator=gen, device=DEV))
    s["layers"] = [{name: x[i] for name, x in s["all"].items()} for i in range(case["layers"])]
    if own:
        import block_sparse_paged_02_gb300 as msa
        kind, mode = _kinds(case)
        mode = mode if case["scales"] == "token" else msa.MSA_SCALE_NONE
        s["pools"] = [msa.make_kv_pools(x["k"], x["v"], kind, scale_mode=mode, k_scale=x.get("k_scale"), v_scale=x.get("v_scale"),
                                        index=msa.make_index_cache(x["idx"], kind, x.get("idx_scale"))) for x in s["layers"]]
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import block_sparse_paged_02_gb300 as msa
        if op == "qk_rope_insert":
            msa.msa_qk_rope_insert(s["batch"], s["qkv"], s["rope"], s["pools"], s["status"])
        elif op == "prompt_attn":
            msa.msa_prompt_attn(s["batch"], s["attn"], s["ws"], s["status"])
        elif op == "page_fork":
            msa.msa_page_fork(s["from"], s["refs"], s["parent"], s["grow"], s["to"], s["status"])
        else:
            msa.msa_page_copy(s["pools"], s["src"], s["dst"], s["tokens"], s["status"])
    else:
        {"qk_rope_insert": _plain_insert, "prompt_attn": _plain_prompt, "page_fork": _plain_fork,
         "page_copy": _plain_copy}[op](s)
    return _outputs(s)


def _values(pool, kv):
    return pool.view(torch.float8_e4m3fn) if kv == "fp8" else pool


def _outputs(s):
    """The state's own buffers; what is held in 8 bits as the values it stands for."""
    case = s["case"]
    if case["op"] == "qk_rope_insert":
        out = {name: s[name] for name in ("q_out", "idx_q_out") if s[name] is not None}
        out |= {name: _values(s[name], case["kv"]) for name in ("k_pool", "v_pool", "idx_pool") if s[name] is not None}
        if case["scales"] == "token":
            out |= {name: s[name] for name in ("k_scale", "v_scale", "idx_scale") if s[name] is not None}
        return out
    if case["op"] == "prompt_attn":
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "page_fork":
        return {name: s[name] for name in ("new_lens", "new_bt", "new_refs", "copy_src", "copy_dst", "copy_tokens")}
    return {name: x if name.endswith("_scale") else _values(x, case["kv"]) for name, x in s["all"].items()}


def _rows(s):
    """Each row's request and position."""
    row = torch.arange(s["rows"], device=DEV)
    req = torch.searchsorted(s["cu_q"].long(), row, right=True) - 1
    return req, s["ctx"].long()[req] + row - s["cu_q"].long()[req]


def _plain_insert(s):
    case = s["case"]
    req, pos = _rows(s)
    slot = s["bt"].long()[req, pos // BLOCK] * BLOCK + pos % BLOCK
    half = case["rotary"] // 2
    if half:
        cs = s["cos_sin"][pos if s["positions"] is None else s["positions"].long()]
        cos, sin = cs[:, None, :half], cs[:, None, half:]

    def normed(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + case["shift"])
        if not half:
            return x
        a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if case["near"] else (x[..., :half], x[..., half:2 * half])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], -1).flatten(-2) if case["near"] else torch.cat([a, b], -1)
        return torch.cat([turned, x[..., 2 * half:]], -1)

    def write(x, pool, scale):
        flat = pool.view(-1, *pool.shape[2:])
        if case["kv"] == "bf16":
            flat[slot] = x.to(torch.bfloat16)
            return
        if scale is not None and scale.numel() == 1 and case["scales"] == "scalar":
            x = x / scale
        elif scale is not None:
            top = x.abs().amax(-1)
            by = torch.where(top > 0, top / 448.0, 1.0)
            scale.view(-1, scale.shape[2])[slot] = by
            x = x / by[..., None]
        flat[slot] = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)

    s["q_out"].copy_(normed(s["q"], s["q_norm"]))
    write(normed(s["k"], s["k_norm"]), s["k_pool"], s["k_scale"])
    write(s["v"].float(), s["v_pool"], s["v_scale"])
    if case["idx_heads"]:
        s["idx_q_out"].copy_(normed(s["idx_q"], s["idx_q_norm"]))
        write(normed(s["idx_k"], s["idx_k_norm"]), s["idx_pool"], s["idx_scale"])


def _cached(s, name, r, n, head):
    """K or V of a request's n tokens for one KV head, in 32 bits."""
    pages = s["bt"][r, :(n + BLOCK - 1) // BLOCK].long()
    x = _values(s[name], s["case"]["kv"])[pages, :, head].float().view(-1, DIM)[:n]
    scale = s[name + "_scale"]
    if scale is None:
        return x
    return x * (scale if s["case"]["scales"] == "scalar" else scale[pages, :, head].view(-1, 1)[:n])


def _plain_prompt(s):
    case = s["case"]
    hk = case["kv_heads"]
    g = case["heads"] // hk
    q0 = 0
    for r, (ctx, ql) in enumerate(zip(s["ctxs"], s["ql"])):
        n = ctx + ql
        pos = torch.arange(n, device=DEV)
        for head in range(hk):
            heads = slice(head * g, head * g + g)
            k, v = _cached(s, "k", r, n, head), _cached(s, "v", r, n, head)
            step = max(1, (1 << 28) // (g * n))
            for j in range(0, ql, step):
                rows = slice(q0 + j, q0 + min(ql, j + step))
                q = s["q"][rows, heads].float()
                z = (q.reshape(-1, DIM) @ k.T).view(q.shape[0], g, n) * SCALE
                last = ctx + j + torch.arange(q.shape[0], device=DEV)
                z.masked_fill_((pos > last[:, None])[:, None], -math.inf)
                m = z.amax(-1, keepdim=True)
                sink = None if s["sinks"] is None else s["sinks"][heads][None, :, None]
                if sink is not None:
                    m = torch.maximum(m, sink)
                p = z.sub_(m).exp_()
                den = p.sum(-1, keepdim=True)
                if sink is not None:
                    den = den + torch.exp(sink - m)
                o = (p.view(-1, n) @ v).view(q.shape[0], g, DIM) / den
                s["out"][rows, heads] = o.to(torch.bfloat16)
                s["lse"][rows, heads] = (m + torch.log(den)).squeeze(-1)
        q0 += ql


def _plain_fork(s):
    old_len, parent, grow = s["lens"].long(), s["parent"].long(), s["grow"].long()
    blk = torch.arange(s["width"], device=DEV)
    refs = s["refs"].long().clone()
    old = s["bt"].long()
    held = blk < ((old_len + BLOCK - 1) // BLOCK)[:, None]
    refs.scatter_add_(0, old[held], torch.full((1,), -1, device=DEV).expand(old[held].numel()))
    n = torch.where(parent >= 0, old_len[parent.clamp(min=0)], 0)
    have, full = (n + BLOCK - 1) // BLOCK, n // BLOCK
    src = old[parent.clamp(min=0)]                                # the parents' tables
    grows = (grow > 0) & (have > full)                            # a partial page that will be written
    keep = blk < torch.where(grows, full, have)[:, None]
    refs.scatter_add_(0, src[keep], torch.ones(1, dtype=torch.long, device=DEV).expand(src[keep].numel()))
    # the lowest row that goes on writing a page that nobody else holds keeps it
    row = torch.arange(s["n_new"], device=DEV)
    last = torch.gather(src, 1, full.clamp(max=s["width"] - 1)[:, None]).squeeze(1)
    last = torch.where(grows, last, 0)
    free = grows & (refs[last] == 0)
    first = torch.full_like(refs, 1 << 40)
    first.scatter_reduce_(0, last[free], row[free], "amin")
    owner = free & (first[last] == row)
    refs[last[owner]] = 1
    copied = grows & ~owner
    # the lowest free pages, in the order of rows and blocks
    need = copied.long() + (n + grow + BLOCK - 1) // BLOCK - have
    at = torch.cumsum(need, 0) - need
    lowest = torch.nonzero(refs == 0).squeeze(1)
    total = int(need.sum())
    refs[lowest[:total]] = 1
    wide = torch.arange(s["wide"], device=DEV)
    shared = torch.full((s["n_new"], s["wide"]), -1, dtype=torch.long, device=DEV)
    w = min(s["wide"], s["width"])
    shared[:, :w] = src[:, :w]
    start = torch.where(copied, full, have)[:, None]              # the first block that is a new page
    fresh = wide >= start
    place = (at[:, None] + wide - start).clamp(0, max(0, lowest.numel() - 1))
    blocks = torch.where(fresh, lowest[place], shared)
    live = wide < ((n + grow + BLOCK - 1) // BLOCK)[:, None]
    s["new_bt"].copy_(torch.where(live, blocks, s["new_bt"].long()))
    s["new_refs"].copy_(refs)
    s["new_lens"].copy_(n)
    s["copy_src"].copy_(torch.where(copied, last, -1))
    s["copy_dst"].copy_(torch.where(copied, lowest[at.clamp(max=lowest.numel() - 1)], -1))
    s["copy_tokens"].copy_(torch.where(copied, n % BLOCK, 0))


def _plain_copy(s):
    tok = torch.arange(BLOCK, device=DEV)
    some = tok < s["tokens"][:, None]
    src = (s["src"].long()[:, None] * BLOCK + tok)[some]
    dst = (s["dst"].long()[:, None] * BLOCK + tok)[some]
    for layer in s["layers"]:
        for x in layer.values():
            flat = x.view(-1, *x.shape[2:])
            flat[dst] = flat[src]


# ------------------------------------------------------------------ what a pass cannot do without

def _token_bytes(case, heads, dim, scaled):
    return heads * (dim * (1 if case["kv"] == "fp8" else 2) + (4 if scaled else 0))


def work(case):
    """Bytes of what is read and written once; multiply-adds of the visible (row, token) pairs."""
    if case["op"] == "page_copy":
        token = (2 * _token_bytes(case, case["kv_heads"], DIM, case["scales"] == "token")
                 + _token_bytes(case, 1, DIM, case["scales"] == "token"))
        return {"bytes": 2.0 * case["layers"] * token * sum(_copy_tokens(case)) + 12.0 * case["copies"], "flops": 0.0}
    if case["op"] == "page_fork":
        lens, shared, parent, grow = _fork_sets(case, np.random.RandomState(0))
        nb = [(n + BLOCK - 1) // BLOCK for n in lens]
        made = [(lens[p] + g + BLOCK - 1) // BLOCK for p, g in zip(parent, grow)]
        held = sum(nb) - sum(shared[r] for r in range(len(lens)) if r % case["width"])
        return {"bytes": 4.0 * (sum(nb) + sum(made) + 2 * held + len(lens) + 6 * len(parent)), "flops": 0.0}
    n = sum(_q_lens(case))
    if case["op"] == "qk_rope_insert":
        h, hk, hi, di = case["heads"], case["kv_heads"], case["idx_heads"], case["idx_dim"]
        read = 2.0 * ((h + 2 * hk) * DIM + 2 * hi * di) + 4.0 * case["rotary"] + (4.0 if case["given"] else 0.0)
        token = case["scales"] == "token"
        write = 2.0 * (h * DIM + hi * di) + 2 * _token_bytes(case, hk, DIM, token) + _token_bytes(case, hi, di, token)
        return {"bytes": n * (read + write), "flops": 6.0 * n * ((h + hk) * DIM + 2 * hi * di)}
    h, hk = case["heads"], case["kv_heads"]
    pairs = sum(t * c + t * (t + 1) / 2 for c, t in zip(_ctx_lens(case), _q_lens(case)))
    tokens = sum(_ctx_lens(case)) + n
    return {"bytes": 2.0 * tokens * _token_bytes(case, hk, DIM, case["scales"] == "token") + n * h * (4.0 * DIM + 4),
            "flops": 4.0 * DIM * h * pairs}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    """None for the operators whose results are indexes or copies."""
    if case["op"] == "qk_rope_insert":
        return _exact_insert(prepare(case, seed))
    if case["op"] == "prompt_attn":
        return _exact_prompt(prepare(case, seed))
    return None


def _exact_insert(s):
    case = s["case"]
    half = case["rotary"] // 2
    slots, where = [], []
    bt = s["bt"].cpu().numpy().astype(np.int64)
    for r, (c, t) in enumerate(zip(s["ctxs"], s["ql"])):
        p = np.arange(c, c + t)
        where.append(p)
        slots.append(bt[r, p // BLOCK] * BLOCK + p % BLOCK)
    slot, pos = _dev(np.concatenate(slots)), _dev(np.concatenate(where))
    if s["positions"] is not None:
        pos = s["positions"].long()

    def through(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + EPS) * (w.double() + case["shift"])
        if half:
            z = torch.view_as_complex(torch.stack(
                (y[..., :2 * half:2], y[..., 1:2 * half:2]) if case["near"] else (y[..., :half], y[..., half:2 * half]), -1).contiguous())
            t = s["cos_sin"][pos].double()
            z = z * torch.complex(t[:, :half], t[:, half:])[:, None]
            if case["near"]:
                y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
            else:
                y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    def into(pool, scale, y):
        new = _values(pool, case["kv"]).double()
        by = None
        if case["kv"] == "fp8" and case["scales"] == "scalar" and scale is not None:
            y = y / scale.double()
        elif case["kv"] == "fp8" and scale is not None:
            by = scale.double()
            amax = y.abs().amax(-1)
            one = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
            by.view(-1, by.shape[2])[slot] = one
            y = y / one.unsqueeze(-1)
        if case["kv"] == "fp8":
            y = y.clamp(-448, 448)
        new.view(-1, *new.shape[2:])[slot] = y
        return new, by

    out = {"q_out": through(s["q"], s["q_norm"])}
    if case["idx_heads"]:
        out["idx_q_out"] = through(s["idx_q"], s["idx_q_norm"])
    out["k_pool"], ks = into(s["k_pool"], s["k_scale"], through(s["k"], s["k_norm"]))
    out["v_pool"], vs = into(s["v_pool"], s["v_scale"], s["v"].double())
    xs = None
    if case["idx_heads"]:
        out["idx_pool"], xs = into(s["idx_pool"], s["idx_scale"], through(s["idx_k"], s["idx_k_norm"]))
    if case["scales"] == "token":
        out["k_scale"], out["v_scale"] = ks, vs
        if case["idx_heads"]:
            out["idx_scale"] = xs
    return out


def _exact_prompt(s):
    case = s["case"]
    g = case["heads"] // case["kv_heads"]
    bt = s["bt"].cpu().numpy()
    outs, lses = [], []
    for r, (c, t) in enumerate(zip(s["ctxs"], s["ql"])):
        first = sum(s["ql"][:r])
        total = c + t
        pages = torch.from_numpy(bt[r, :-(-total // BLOCK)].astype(np.int64)).to(DEV)
        out = torch.empty((t, case["heads"], DIM), dtype=torch.float64, device=DEV)
        lse = torch.empty((t, case["heads"]), dtype=torch.float64, device=DEV)
        for h in range(case["heads"]):
            kv = []
            for name in ("k", "v"):
                x = _values(s[name], case["kv"])[pages][:, :, h // g].double()
                if case["scales"] == "scalar":
                    x = x * s[name + "_scale"].double()
                if case["scales"] == "token":
                    x = x * s[name + "_scale"][pages][:, :, h // g, None].double()
                kv.append(x.reshape(-1, DIM)[:total])
            for a in range(0, t, 2048):
                b = min(t, a + 2048)
                seen = c + b                                     # no row of the piece sees more
                z = s["q"][first + a:first + b, h].double() @ kv[0][:seen].T * SCALE
                z[:, c + a:] += torch.full((b - a, b - a), -math.inf, dtype=torch.float64, device=DEV).triu(1)
                m = z.amax(1)
                w = torch.exp(z - m[:, None])
                den = w.sum(1)
                if s["sinks"] is not None:
                    den = den + torch.exp(s["sinks"][h].double() - m)
                out[a:b, h] = (w @ kv[1][:seen]) / den[:, None]
                lse[a:b, h] = m + torch.log(den)
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}

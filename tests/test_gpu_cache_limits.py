"""The cache operators at sizes that reach their rarer forms: keys read again in every pass of
the selection, moves and selections of more blocks than fit their on-chip tables, rows joined
from very many partial results."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import tree_ref as T
from tests.test_gpu_evict import masses, move, pool_set, select, tables
from tests.test_gpu_tree import make, run_both

pytestmark = pytest.mark.gpu


def wide(bt, stride):
    out = np.full((bt.shape[0], stride), -1, np.int32)
    out[:, :bt.shape[1]] = bt
    return out


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd", "near"])
def test_select_behind_a_wide_table(kind):
    # (the form is taken from the table's width: shares of more tokens than are held on chip)
    lens = [5000, 300, 2049, 0, 70000]
    rng = np.random.default_rng(3)
    bt, pages = tables(rng, lens)
    m = masses(rng, pages, kind)
    for budget, first, recent in ((1000, 4, 500), (1, 0, 0), (5000, 0, 5000)):
        got = select(lens, wide(bt, 16384), m, budget, first, recent)
        want = T.evict(lens, bt, m, budget, first, recent)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


def test_select_of_many_requests_behind_a_wide_table():
    # (more requests than SMs: one CTA each)
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 1500, 200)]
    bt, pages = tables(rng, lens)
    m = masses(rng, pages, "ties")
    got = select(lens, wide(bt, 512), m, 300, 4, 64)
    want = T.evict(lens, bt, m, 300, 4, 64)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])
    bad = bt.copy()
    bad[7, 0] = pages
    lens[7] = max(lens[7], 1)
    got, kl = select(lens, wide(bad, 512), m, 300, 4, 64, status=1)
    assert kl[7] == -1 and (got[7] == -1).all()


def test_select_of_two_million_tokens():
    rng = np.random.default_rng(6)
    n = 128 * 16384 - 5
    bt, pages = tables(rng, [n])
    m = masses(rng, pages, "plain")
    m[rng.random((pages, 128)) < 0.5] = 0.0
    for budget in (3000, 1500000):
        got, kl = select([n], bt, m, budget, 100, 1000)
        pos = np.arange(n)
        v = m[bt[0, pos // 128], pos % 128].astype(np.float64)
        v[:100] = v[n - 1000:] = np.inf
        want = np.sort(np.argsort(-v, kind="stable")[:budget])
        assert kl[0] == budget and np.array_equal(got[0], want)


@pytest.mark.parametrize("stays", [0, 5, 290000])
def test_move_of_positions_past_the_page_table(stays):
    # more blocks than the page numbers held on chip; a prefix that stays ends inside a warp
    rng = np.random.default_rng(7)
    lens = [320003, 400]
    bt, pages = tables(rng, lens)
    n = stays + 9001
    keep = np.full((2, n), -1, np.int32)
    keep[0, :stays] = np.arange(stays)
    keep[0, stays:] = stays + 1 + np.sort(rng.permutation(lens[0] - stays - 1)[:9001])
    keep[1, :300] = np.sort(rng.permutation(400)[:300])
    move(pool_set(rng, pages, W.KV_FP8, 1, True, 1, 64, True, True), W.KV_FP8, lens, bt, keep, [n, 300])


@pytest.mark.parametrize("kv,scale", [(W.KV_BF16, W.SCALE_NONE), (W.KV_FP8, W.SCALE_PER_TOKEN_HEAD)])
def test_selected_blocks_of_a_very_long_context(kv, scale):
    # more blocks than one round of the plan's prefix sum takes
    ctx, topk = 128 * 9000 + 77, 6
    rng = np.random.default_rng(8)
    w = make(61, [2, 1], [300, 500], 16, kv, scale, True)
    # (entries of a table may name a page twice for the attention; for the weights the visited ones may not)
    w.block_table = wide(w.block_table, 9001)
    nb = (ctx + 2 + 127) // 128
    spare = np.setdiff1d(np.arange(w.num_pages), w.block_table[1, :4])
    w.block_table[0, :nb] = spare[0]
    sel = np.array([[0, 8191, 8192, 8999, 40, 8191], [8999, 17, 8640, -1, 9000, 8191], [0, 1, 2, 3, 4, 5]], np.int32)
    mine = sorted(set(sel[:2].ravel()) - {-1, 9000}) + [9000]
    pages = w.num_pages
    grow = lambda a, fill: np.concatenate([a, np.repeat(a[spare[:1]], len(mine), 0)])
    w.k_cache, w.v_cache, w.idx_k = (grow(a, 0).copy() for a in (w.k_cache, w.v_cache, w.idx_k))
    if scale:
        w.k_scale, w.v_scale = grow(w.k_scale, 0).copy(), grow(w.v_scale, 0).copy()
    vals = rng.standard_normal((2, len(mine), 128, 1, 128))
    code = W.fp8_codes if kv == W.KV_FP8 else W.bf16_bits
    w.k_cache[pages:], w.v_cache[pages:] = code(vals[0]), code(vals[1])
    for i, b in enumerate(mine):
        w.block_table[0, b] = pages + i
    w.num_pages = pages + len(mine)
    w.context_lens[0] = ctx
    w.cu_seqlens_k = np.concatenate([[0], np.cumsum(w.context_lens + np.diff(w.cu_seqlens_q))]).astype(np.int32)
    w.k_cache[spare[0]] = code(np.zeros(1))[0]
    w.v_cache[spare[0]] = code(np.zeros(1))[0]
    run_both(w, None, sel)


@pytest.mark.parametrize("kv,scale", [(W.KV_BF16, W.SCALE_NONE), (W.KV_FP8, W.SCALE_NONE), (W.KV_FP8, W.SCALE_PER_TOKEN_HEAD)])
@pytest.mark.parametrize("hq,ql", [(16, 1), (3, 1), (8, 4), (16, 20)])
def test_one_long_request(kv, scale, hq, ql):
    # a request's blocks on every SM: each row joins 100 partial results and more, all of them
    # with weight
    w = make(62, [ql], [45000], hq, kv, scale, True)
    assert (45000 + ql) // 128 > 300
    run_both(w)


@pytest.mark.parametrize("kv,hkv", [(W.KV_BF16, 1), (W.KV_FP8, 3)])
@pytest.mark.parametrize("stays", [1, 17, 63, 255, 2049])
def test_move_where_lanes_of_a_warp_differ(kv, hkv, stays):
    # the tokens that stay, and the list's end, divide warps; some requests move nothing, one token,
    # or their last token alone
    rng = np.random.default_rng(stays)
    lens = [6000, 4097, 2100, 2100, 5000]
    bt, pages = tables(rng, lens)
    n = stays + 1303
    keep = np.full((5, n), -1, np.int32)
    for r in (0, 1):
        keep[r, :stays] = np.arange(stays)
        keep[r, stays:] = stays + 1 + np.sort(rng.permutation(lens[r] - stays - 1)[:1303])
    keep[2, :stays] = keep[3, :stays] = np.arange(stays)
    keep[3, stays - 1] = 2099
    keep[4, :stays] = np.arange(1, stays + 1)
    move(pool_set(rng, pages, kv, hkv, kv == W.KV_FP8, 1, 128, True, True), kv, lens, bt, keep, [n, n, stays, stays, stays])


@pytest.mark.parametrize("lens,budget", [([1], 1), ([33], 32), ([4129, 1], 4128), ([20001, 31], 31)])
def test_select_where_lanes_of_a_warp_differ(lens, budget):
    # lengths that end inside a warp's run, on one CTA and on clusters
    rng = np.random.default_rng(budget)
    bt, pages = tables(rng, lens)
    m = masses(rng, pages, "near")
    for stride in (bt.shape[1], 200, 2000):
        if stride >= bt.shape[1]:
            got = select(lens, wide(bt, stride), m, budget, 0, min(budget, 3))
            want = T.evict(lens, bt, m, budget, 0, min(budget, 3))
            assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])

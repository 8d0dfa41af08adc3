"""Whole-prompt attention on the GPU against the 64-bit plain form of prompt_ref (its tolerances are
derived there)."""
import dataclasses

import numpy as np
import pytest
import torch

import workloads as W
from tests import prompt_ref as P

pytestmark = pytest.mark.gpu

BF, F8 = W.KV_BF16, W.KV_FP8
NONE, SCALAR, TOKEN = W.SCALE_NONE, W.SCALE_SCALAR, W.SCALE_PER_TOKEN_HEAD
TYPES = [(BF, NONE), (BF, SCALAR), (BF, TOKEN), (F8, NONE), (F8, SCALAR), (F8, TOKEN)]


def case(w, **kw):
    from block_sparse_paged_02_gb300 import DeviceCase
    c = DeviceCase(w, **kw)
    c.out.fill_(float("nan"))
    c.lse.fill_(float("nan"))
    return c


def run(w, bad=(), status=0):
    c = case(w)
    c.prompt_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == status
    P.check_attn(c, P.attn(w, bad))
    return c


@pytest.mark.parametrize("kv,scale", TYPES)
@pytest.mark.parametrize("heads,kv_heads,q_lens,ctxs", [
    (16, 1, [1], [0]), (8, 1, [200], [0]), (16, 1, [130, 7, 1], [0, 129, 700]), (12, 2, [45, 300], [63, 0]),
    (4, 4, [129, 260], [128, 1]), (24, 3, [1, 2, 90], [5, 127, 511])])
def test_types_and_heads(kv, scale, heads, kv_heads, q_lens, ctxs):
    run(P.batch(11, q_lens, ctxs, heads, kv_heads, kv, scale, sink=heads % 3 == 0))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, TOKEN)])
@pytest.mark.parametrize("group", [1, 3, 5, 7, 31, 64, 65, 128])
def test_groups(kv, scale, group):
    # a token's whole group in one tile, tiles that the group does not fill
    run(P.batch(12, [150 if group < 31 else 40, 3], [70, 0], group, 1, kv, scale, sink=True))


@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("ql", [1, 8, 9, 64, 127, 128, 129])
def test_lengths(ctx, ql):
    run(P.batch(13, [ql, 3], [ctx, 128 - 3], 16 if ql % 2 else 2))


@pytest.mark.parametrize("kv,scale", TYPES)
def test_long_context_is_shared_by_many(kv, scale):
    # one pair of tiles cut over most CTAs, and pairs that several share
    run(P.batch(14, [5], [20000], 16, 1, kv, scale, True))
    run(P.batch(15, [150, 33], [3000, 9000], 4, 2, kv, scale, True))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, SCALAR)])
def test_many_tiles(kv, scale):
    # more pairs than CTAs: rings that go round many times
    run(P.batch(16, [2500, 700], [0, 100], 16, 1, kv, scale))


def test_rows_of_one_request_or_none():
    run(P.batch(17, [0, 2, 0, 0, 65, 0], [10, 300, 0, 128, 40, 7], 16))
    rng = np.random.default_rng(2)
    n = 900  # more requests than a CTA has threads
    run(P.batch(18, rng.integers(0, 5, n).tolist(), rng.integers(0, 200, n).tolist(), 2, 1, F8, SCALAR))


@pytest.mark.parametrize("kv,scale", TYPES)
def test_growing_and_falling_logits(kv, scale):
    # maxima that move at every block: the running reference and O are rescaled all along
    for order in (1, -1):
        w = P.batch(19, [130], [900], 8, 1, kv, scale)
        k = P.values(w.k_cache)
        n = 1030
        pages = w.block_table[0, :9]
        grow = np.linspace(0, 4, n)[::order]
        flat = k[pages].reshape(-1, 128)
        flat[:n] = np.sign(P.values(w.q)[0, 0]) * grow[:, None]
        flat[np.isnan(flat)] = 0
        k[pages] = flat.reshape(9, 128, 1, 128)
        w.k_cache[pages] = (W.fp8_codes if kv == F8 else W.bf16_bits)(k[pages])
        run(w)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (BF, TOKEN), (F8, NONE), (F8, TOKEN)])
@pytest.mark.parametrize("ctx,ql,at", [(100, 90, 189), (0, 129, 128), (300, 40, 320), (1000, 200, 1100)])
def test_values_that_a_row_does_not_see(kv, scale, ctx, ql, at):
    """NaN and infinities in K and V of a token reach the rows from its position on, and no other."""
    clean = P.batch(20, [ql, 2], [ctx, 50], 16, 1, kv, scale, True)
    w = dataclasses.replace(clean, k_cache=clean.k_cache.copy(), v_cache=clean.v_cache.copy())
    page = w.block_table[0, at // 128]
    w.k_cache[page, at % 128, 0, 3] = 0x7f if kv == F8 else 0x7f80
    w.v_cache[page, at % 128, 0, 7] = 0x7f if kv == F8 else 0xff80
    w.v_cache[page, at % 128, 0, 99] = 0xff if kv == F8 else 0x7fc0
    if scale == TOKEN:
        w.k_scale[page, at % 128] = np.nan
        w.v_scale[page, at % 128] = np.inf
    c = case(w)
    c.prompt_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    keep = list(range(at - ctx)) + [ql, ql + 1]
    if scale == TOKEN:  # (the reference's own scales are clean)
        clean.k_scale[page, at % 128] = clean.v_scale[page, at % 128] = 1
    P.check_attn(c, P.attn(clean), keep)
    assert not torch.isfinite(c.out[at - ctx:ql].float()).all(dim=2).any()


def test_lowest_values_and_extreme_logits():
    w = P.batch(21, [140], [20], 4, 1)
    low = np.uint16(0xff7f)  # bf16's lowest
    w.q[:, 1] = 0
    w.k_cache[w.block_table[0, 0], 5] = 0
    w.v_cache[w.block_table[0, 0], 5, 0, :] = low
    c = case(w)
    c.prompt_attn()
    torch.cuda.synchronize()
    ref = P.attn(w)
    P.check_attn(c, ref)
    # logits far apart: a softmax of one token
    w = P.batch(22, [70], [300], 4, 1)
    w.q[:] = W.bf16_bits(P.values(w.q) * 60)
    run(w)
    w.softmax_scale = -w.softmax_scale
    run(w)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, SCALAR), (F8, TOKEN), (BF, TOKEN)])
@pytest.mark.parametrize("sink", [False, True])
def test_poisoned_requests(kv, scale, sink):
    w = P.batch(23, [3, 200, 4, 2, 60, 300], [300, 2000, 500, 64, 900, 0], 16, 1, kv, scale, sink)
    w.block_table[1, 15] = w.num_pages      # a page out of range, behind most rows' sight
    w.context_lens[2] += 1                  # lengths that do not add up
    w.block_table[5, 0] = -1
    run(w, bad=(1, 2, 5), status=1 | 2)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, TOKEN)])
def test_many_poisoned_requests(kv, scale):
    n = 400
    w = P.batch(24, [20] * n, [130] * n, 16, 1, kv, scale, True)
    w.context_lens[1::2] += 1
    w.block_table[4::8, 1] = -1
    run(w, bad=tuple(range(1, n, 2)) + tuple(range(4, n, 8)), status=3)
    # one long request, every page bad: its rows are shared by many CTAs
    w = P.batch(25, [600], [128 * 100], 16, 1, kv, scale, True)
    w.block_table[:] = -1
    run(w, bad=(0,), status=1)


def test_rows_that_no_request_owns_and_fewer_rows_than_the_bound():
    w = P.batch(26, [3, 2], [100, 100], 4, sink=True)
    w.cu_seqlens_q[2] = 4
    c = case(w)
    c.prompt_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4
    assert (c.out.float() == 0).all()
    assert np.array_equal(c.lse.cpu().numpy(), np.tile(w.sinks, (5, 1)))
    w = P.batch(27, [3, 200], [100, 100], 4)
    c = case(w, min_q_len_hint=100)
    c.prompt_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4
    P.check_attn(c, P.attn(w, bad=(0,)))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, TOKEN)])
def test_scales_of_every_size(kv, scale):
    # scales over many powers of two, zero among them
    w = P.batch(28, [100], [400], 8, 1, kv, TOKEN)
    rng = np.random.default_rng(1)
    w.v_scale[:] = np.ldexp(1.0, rng.integers(-30, 20, w.v_scale.shape)).astype(np.float32)
    w.v_scale[:, ::7] = 0
    w.k_scale[:, ::5] = 0
    run(w)


def test_agrees_with_the_tree_attention():
    w = P.batch(29, [200, 30], [500, 1000], 16, 1, BF, NONE, True)
    c = case(w)
    c.tree_attn()
    want, lse = c.out.double(), c.lse.double()
    c.prompt_attn()
    torch.cuda.synchronize()
    _, _, ot, lt = P.attn(w)
    assert ((c.out.double() - want).abs().cpu().numpy() <= 2 * ot).all()
    assert ((c.lse.double() - lse).abs().cpu().numpy() <= 2 * lt + 2e-6 * (lse.abs().cpu().numpy() + 1)).all()


def test_same_bits_twice_on_other_streams_and_in_graphs():
    w = P.batch(30, [400, 1, 77], [3000, 9000, 0], 16, 1, BF, NONE, True)
    c = case(w)
    c.prompt_attn()
    torch.cuda.synchronize()
    want = c.out.clone(), c.lse.clone()

    def again(run):
        c.out.fill_(float("nan")), c.lse.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])

    again(c.prompt_attn)
    side = torch.cuda.Stream()
    again(lambda: c.prompt_attn(stream=side))
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (graph, second):
        with torch.cuda.graph(g, stream=side):
            c.prompt_attn()
    again(graph.replay)
    again(graph.replay)
    again(lambda: (graph.replay(), second.replay()))
    # two cases' calls on two streams at once, each with its workspace
    w2 = P.batch(31, [300], [2000], 16, 1, BF, NONE)
    d = case(w2)
    d.prompt_attn()
    torch.cuda.synchronize()
    want2 = d.out.clone()
    for _ in range(10):
        c.prompt_attn(stream=side)
        d.prompt_attn()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want[0]) and torch.equal(d.out, want2)


def test_a_row_is_the_same_in_any_batch_of_whole_pairs():
    """Few long prompts are cut over the CTAs: a row's result is within tolerance of the one alone."""
    w = P.batch(32, [64, 64], [640, 640], 16, 1, BF, NONE)
    c = run(w)
    one = W.row_subset(w, [5, 70])
    d = case(one)
    d.prompt_attn()
    torch.cuda.synchronize()
    P.check_attn(d, P.attn(one))
    assert (c.out[[5, 70]].float() - d.out.float()).abs().max() < 0.05

"""Draft-tree attention and weight accumulation on the GPU against the 64-bit
plain forms of tree_ref (their tolerances are derived there)."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import tree_ref as T

pytestmark = pytest.mark.gpu

BF, F8 = W.KV_BF16, W.KV_FP8
NONE, SCALAR, TOKEN = W.SCALE_NONE, W.SCALE_SCALAR, W.SCALE_PER_TOKEN_HEAD


def case(w, **kw):
    from block_sparse_paged_02_gb300 import DeviceCase
    return DeviceCase(w, **kw)


def make(seed, q_lens, ctxs, hq=16, kv=BF, scale=NONE, sink=False, **kw):
    return W.custom(seed, q_lens, [c + q for c, q in zip(ctxs, q_lens)], hq=hq, kv_dtype=kv,
                    scale_mode=scale, with_sink=sink, fill_unused_nan=True, **kw)


def words_of(q_lens):
    return max(1, (max(q_lens) + 31) // 32)


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
    # a sink returned by itself is exact up to one rounding
    assert (e <= lt[rows] + 1e-6 * (np.abs(np.where(inf, 0, lse))[rows] + 1)).all(), e.max()


def run_both(w, mask=None, topk=None, bad=(), status=0):
    c = case(w)
    c.tree_attn(mask=None if mask is None else T.dev(mask), topk_idx=None if topk is None else T.dev(topk))
    torch.cuda.synchronize()
    assert int(c.status.item()) == status
    check_attn(c, T.tree_attn(w, mask, topk, bad))
    # the weights, from the lse that the call wrote
    rng = np.random.default_rng(5)
    mass = rng.random((w.num_pages, 128)).astype(np.float32)
    m = torch.from_numpy(mass).cuda()
    c.attn_mass(m, mask=None if mask is None else T.dev(mask), topk_idx=None if topk is None else T.dev(topk))
    torch.cuda.synchronize()
    want, tol = T.attn_mass(w, c.lse.cpu().numpy(), mass, mask, topk, bad)
    got = m.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / (tol + 1e-300))
    return c


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (BF, SCALAR), (BF, TOKEN), (F8, NONE), (F8, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("hq,q_lens", [(16, [1]), (1, [1, 3, 2]), (8, [4, 2, 1]), (16, [2, 1]), (12, [5, 3]),
                                       (16, [8, 4]), (5, [33, 7]), (16, [40, 64])])
def test_chain(kv, scale, hq, q_lens):
    ctxs = [700, 129, 1][:len(q_lens)]
    run_both(make(11, q_lens, ctxs, hq, kv, scale, sink=hq % 2 == 0))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, TOKEN)])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("hq,q_lens,ctxs", [
    (16, [7, 16, 1], [0, 250, 383]), (3, [31, 32, 33], [5, 127, 128]), (16, [64], [1000]),
    (4, [100, 130], [77, 513]), (16, [1, 1, 1, 1], [0, 1, 127, 640]), (7, [256], [300])])
def test_masks(kv, scale, kind, hq, q_lens, ctxs):
    rng = np.random.default_rng(3)
    run_both(make(12, q_lens, ctxs, hq, kv, scale, sink=True), T.random_mask(rng, q_lens, words_of(q_lens), kind))


@pytest.mark.parametrize("sink", [False, True])
def test_rows_that_see_nothing(sink):
    # no context and an empty mask: out 0, lse the sink's or -inf
    w = make(13, [4, 20, 3], [0, 0, 200], 8, BF, NONE, sink)
    mask = np.zeros((27, 1), np.uint32)
    mask[5] = 1 << 5
    c = run_both(w, mask)
    assert (c.out[0].float() == 0).all()


@pytest.mark.parametrize("ctx", [1, 63, 64, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("kv", [BF, F8])
def test_block_edges(ctx, kv):
    run_both(make(14, [3, 6], [ctx, ctx + 64], 16, kv, SCALAR))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (BF, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("hq,q_lens,ctxs", [(16, [1, 1], [5000, 900]), (16, [9, 40], [4100, 2600]),
                                            (2, [70, 3], [3333, 128 * 9]), (16, [64, 50], [20000, 3000])])
def test_split_tiles(kv, scale, hq, q_lens, ctxs):
    # long enough that tiles are shared by CTAs and joined
    run_both(make(15, q_lens, ctxs, hq, kv, scale, sink=True))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, TOKEN)])
@pytest.mark.parametrize("hq,q_lens,ctxs,topk", [
    (16, [1, 1], [3000, 100], 4), (16, [20, 7], [2500, 1280], 3), (4, [65, 40], [128 * 12 + 5, 128 * 7], 2),
    (16, [3, 30], [60, 9000], 16)])
def test_selected_blocks(kv, scale, hq, q_lens, ctxs, topk):
    # each row its own blocks, with repeats, -1 and numbers out of range
    w = make(16, q_lens, ctxs, hq, kv, scale, sink=True)
    rng = np.random.default_rng(7)
    sel = np.full((w.num_rows, topk), -1, np.int32)
    for r in range(w.num_reqs):
        for j in range(int(w.cu_seqlens_q[r]), int(w.cu_seqlens_q[r + 1])):
            sel[j] = rng.integers(-1, ctxs[r] // 128 + 2, topk)
    sel[0, -1] = 1 << 30
    run_both(w, T.random_mask(rng, q_lens, words_of(q_lens)), sel)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, TOKEN)])
@pytest.mark.parametrize("q_lens", [[5, 2], [64, 20]])
def test_hidden_values_do_not_leak(kv, scale, q_lens):
    # NaN (and infinities) in drafted tokens and selected blocks that some rows do not see
    ctxs = [700, 300]
    w = make(17, q_lens, ctxs, 16, kv, scale)
    rng = np.random.default_rng(9)
    mask = T.random_mask(rng, q_lens, words_of(q_lens), "tree")
    nan, inf = (0x7f, 0x7f) if kv == F8 else (0x7fc0, 0xff80)
    hidden = {}
    for r in range(2):
        q0, q1 = int(w.cu_seqlens_q[r]), int(w.cu_seqlens_q[r + 1])
        i = q1 - q0 - 1  # seen only by itself
        pos = ctxs[r] + i
        page = w.block_table[r, pos // 128]
        w.v_cache[page, pos % 128, 0, ::3] = nan
        w.v_cache[page, pos % 128, 0, 1::3] = inf
        w.k_cache[page, pos % 128, 0, 5] = nan
        hidden[r] = q1 - 1
    sel = np.full((w.num_rows, 2), -1, np.int32)
    sel[:, 0] = 1
    sel[0, 1] = 0  # row 0 alone reads block 0 of request 0
    for b, seq in ((0, 700),):
        w.v_cache[w.block_table[0, b], 3] = nan
    c = case(w)
    c.tree_attn(mask=T.dev(mask), topk_idx=T.dev(sel))
    torch.cuda.synchronize()
    keep = [r for r in range(w.num_rows) if r not in hidden.values() and r != 0]
    clean = W.custom(17, q_lens, [x + y for x, y in zip(ctxs, q_lens)], hq=16, kv_dtype=kv, scale_mode=scale)
    check_attn(c, T.tree_attn(clean, mask, sel), keep)
    got = c.out.float().cpu().numpy()
    assert np.isnan(got[0]).all()
    for r in hidden.values():
        assert np.isnan(got[r]).any()
    m = torch.zeros((w.num_pages, 128), device="cuda")
    lse = np.nan_to_num(c.lse.cpu().numpy(), nan=0.0)
    c.lse.copy_(torch.from_numpy(lse))
    c.attn_mass(m, mask=T.dev(mask), topk_idx=T.dev(sel))
    m = m.cpu().numpy()
    # only the drafted token that holds a NaN key, as seen by itself, has a NaN weight
    assert np.isnan(m).sum() == 2


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (BF, TOKEN), (F8, TOKEN)])
def test_hidden_values_in_many_requests(kv, scale):
    # more requests than CTAs: tiles of several blocks that one CTA holds whole, every
    # third with a token that only its own row sees and that holds NaN
    rng = np.random.default_rng(29)
    q_lens = [int(x) for x in rng.integers(3, 7, 200)]
    ctxs = [int(x) for x in rng.integers(0, 400, 200)]
    w = make(31, q_lens, ctxs, 16, kv, scale)
    clean = W.custom(31, q_lens, [x + y for x, y in zip(ctxs, q_lens)], hq=16, kv_dtype=kv, scale_mode=scale)
    mask = T.random_mask(rng, q_lens, 1, "tree")
    hidden = []
    for r in range(0, 200, 3):
        q1 = int(w.cu_seqlens_q[r + 1])
        pos = ctxs[r] + q_lens[r] - 1
        w.v_cache[w.block_table[r, pos // 128], pos % 128, 0, ::5] = 0x7f if kv == F8 else 0x7fc0
        mask[q1 - q_lens[r]:q1, 0] &= ~np.uint32(1 << (q_lens[r] - 1)).view(mask.dtype)
        mask[q1 - 1, 0] |= 1 << (q_lens[r] - 1)
        hidden.append(q1 - 1)
    c = case(w)
    c.tree_attn(mask=T.dev(mask))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check_attn(c, T.tree_attn(clean, mask), [r for r in range(w.num_rows) if r not in set(hidden)])
    got = c.out.float().cpu().numpy()
    assert all(np.isnan(got[r, :, ::5]).all() for r in hidden)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (BF, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("hq,ql,ctx", [(16, 40, 20), (16, 20, 100), (4, 60, 3), (16, 9, 0)])
def test_hidden_values_in_a_single_block(kv, scale, hq, ql, ctx):
    # one block holds the whole request: a CTA writes its tiles without a merge
    w = make(27, [ql, 2], [ctx, 50], hq, kv, scale, True)
    mask = np.zeros((ql + 2, 2), np.uint32)
    for j in range(ql + 2):
        i = j if j < ql else j - ql
        mask[j, i // 32] = 1 << (i % 32)  # each row sees the context and itself
    page = w.block_table[0, 0]
    w.v_cache[page, ctx + ql - 1, 0, 7] = 0x7f if kv == F8 else 0x7f80
    c = case(w)
    c.tree_attn(mask=T.dev(mask))
    torch.cuda.synchronize()
    keep = [r for r in range(ql + 2) if r != ql - 1]
    check_attn(c, T.tree_attn(make(27, [ql, 2], [ctx, 50], hq, kv, scale, True), mask), keep)
    assert not torch.isfinite(c.out[ql - 1].float()[:, 7]).any()


def test_poisoned_requests():
    q_lens, ctxs = [3, 20, 4, 2, 6], [300, 2000, 500, 64, 900]
    for sink in (False, True):
        w = make(18, q_lens, ctxs, 16, BF, NONE, sink)
        w.block_table[1, 7] = w.num_pages       # a page out of range
        w.context_lens[2] += 1                  # lengths that do not add up
        mask = T.random_mask(np.random.default_rng(1), q_lens, 1)
        run_both(w, mask, bad=(1, 2), status=1 | 2)
        topk = np.zeros((w.num_rows, 2), np.int32)
        run_both(w, mask, topk, bad=(1, 2), status=1 | 2)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("ql,hq", [(1, 4), (20, 16)])
def test_many_poisoned_requests_and_bad_pages(kv, scale, ql, hq):
    # far more empty blocks than any ring holds
    n = 400
    q_lens, ctxs = [ql] * n, [130] * n
    w = make(26, q_lens, ctxs, hq, kv, scale, True)
    w.context_lens[1::2] += 1
    w.block_table[4::8, 1] = -1
    bad = tuple(range(1, n, 2)) + tuple(range(4, n, 8))
    c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 3
    check_attn(c, T.tree_attn(w, None, None, bad))
    # one request, every page bad
    w = make(26, [ql], [128 * 300], hq, kv, scale, True)
    w.block_table[:] = -1
    run_both(w, bad=(0,), status=1)


def test_more_rows_than_the_mask_or_the_bound():
    q_lens, ctxs = [40, 3], [100, 100]
    w = make(19, q_lens, ctxs, 4)
    run_both(w, np.full((43, 1), 0xffffffff, np.uint32), bad=(0,), status=4)
    c = case(w)
    c.max_q_len = 8
    c._args()
    c.tree_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4
    check_attn(c, T.tree_attn(w, bad=(0,)))


def test_rows_that_no_request_owns():
    w = make(20, [3, 2], [100, 100], 4, sink=True)
    w.cu_seqlens_q[2] = 4
    c = case(w)
    c.tree_attn()
    m = torch.ones((w.num_pages, 128), device="cuda")
    c.attn_mass(m)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4
    assert (c.out.float() == 0).all() and (m == 1).all()
    assert np.array_equal(c.lse.cpu().numpy(), np.tile(w.sinks, (5, 1)))


def test_requests_without_rows_and_many_requests():
    run_both(make(21, [0, 2, 0, 0, 5, 0], [10, 300, 0, 128, 40, 7], 16))
    n = 700  # more requests than a CTA has threads
    rng = np.random.default_rng(2)
    q_lens = rng.integers(0, 4, n).tolist()
    run_both(make(22, q_lens, rng.integers(0, 300, n).tolist(), 2, F8, SCALAR))


def test_same_bits_twice_on_another_stream_and_in_a_graph():
    q_lens, ctxs = [20, 1, 64], [6000, 20000, 3000]
    w = make(23, q_lens, ctxs, 16, BF, NONE, True)
    mask = T.dev(T.random_mask(np.random.default_rng(4), q_lens, 2))
    c = case(w)
    m0 = torch.zeros((w.num_pages, 128), device="cuda")
    c.tree_attn(mask=mask)
    c.attn_mass(m0, mask=mask)
    torch.cuda.synchronize()
    want = c.out.clone(), c.lse.clone(), m0.clone()

    def again(run):
        c.out.zero_(), c.lse.zero_(), m0.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((c.out, c.lse, m0), want))

    def go(stream=None):
        c.tree_attn(mask=mask, stream=stream)
        c.attn_mass(m0, mask=mask, stream=stream)

    again(go)
    side = torch.cuda.Stream()
    again(lambda: go(side))
    # garbage left in the workspace does not matter
    for ws in c._tree_ws.values():
        ws.fill_(0xff)
    again(go)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    again(g.replay)
    again(g.replay)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("hq,q_lens", [(16, [1, 1, 1]), (8, [12, 5, 1]), (16, [40, 1, 24]), (16, [20, 70, 3])])
def test_long_slices(kv, hq, q_lens):
    # dozens of blocks per CTA, so that every ring goes round many times (reference in 64 bits
    # on the GPU; bounds as in tree_ref, with its terms bounded over all tokens)
    from block_sparse_paged_02_gb300 import binding as B
    ctxs = [250001, 300000, 170100]
    g = torch.Generator("cuda").manual_seed(5)
    seqs = [x + y for x, y in zip(ctxs, q_lens)]
    nb = [(n + 127) // 128 for n in seqs]
    pages, n = sum(nb), sum(q_lens)
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    bt = torch.full((3, max(nb)), -1, dtype=torch.int32, device="cuda")
    for r in range(3):
        bt[r, :nb[r]] = perm[sum(nb[:r]):sum(nb[:r + 1])]
    k, v = (torch.randn((pages, 128, 1, 128), generator=g, device="cuda") for _ in range(2))
    k, v = (x.to(torch.float8_e4m3fn if kv == F8 else torch.bfloat16) for x in (k, v))
    q = (2 * torch.randn((n, hq, 128), generator=g, device="cuda")).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    batch = B.make_batch(i32(cu.tolist()), i32(np.concatenate([[0], np.cumsum(seqs)]).tolist()), i32(ctxs), bt, pages, n,
                         max_q_len=max(q_lens))
    out, lse = torch.zeros((n, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, hq), device="cuda")
    raw = (lambda x: x.view(torch.uint8)) if kv == F8 else (lambda x: x)
    attn = B.make_attn_args(q, raw(k), raw(v), kv, pages, out, lse, softmax_scale=0.0883)
    ws = torch.empty((B.msa_tree_attn_workspace_size(3, n, bt.shape[1], hq, max(q_lens)),), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tree = B.make_tree()
    mass = torch.ones((pages, 128), device="cuda")
    B.msa_tree_attn(batch, tree, attn, ws, st)
    B.msa_attn_mass(batch, tree, attn, mass, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for r in range(3):
        at = bt[r, :nb[r]].long()
        kk, vv = (x[at].view(-1, 128)[:seqs[r]].double() for x in (k, v))
        got = torch.zeros(seqs[r], dtype=torch.float64, device="cuda")
        for j in range(q_lens[r]):
            row, end = int(cu[r]) + j, ctxs[r] + j + 1
            z = 0.0883 * q[row].double() @ kk[:end].T
            ref = torch.logsumexp(z, 1)
            p = torch.exp(z - ref[:, None])
            o, a = p @ vv[:end], p @ vv[:end].abs()
            d = 130 * 2.0 ** -23 * 0.0883 * float((q[row].double().abs() @ kk[:4096].abs().T).max()) * 1.5
            assert ((out[row].double() - o).abs() <= (2.0 ** -8 + 2 * d + 1e-4) * a + 2.0 ** -8 * o.abs()).all()
            assert ((lse[row].double() - ref).abs() <= d + 1e-4).all()
            got[:end] += torch.exp(z - lse[row].double()[:, None]).sum(0)
        m = mass[at].view(-1)[:seqs[r]].double()
        want = got + (torch.arange(seqs[r], device="cuda") < ctxs[r])
        # near 1 the stored sum rounds by 2^-24; the weights themselves by 2 d and 2^-21 |s|
        assert ((m - want).abs() <= (2 * d + 2.0 ** -21 * 60 + q_lens[r] * hq * 2.0 ** -24) * got + 2.0 ** -23 * want).all()


def test_offsets_past_32_bits():
    # pools of more than 2^32 bytes: pages near their end
    from block_sparse_paged_02_gb300 import binding as B
    pages, hq, ctx, ql = 140000, 16, 500, 5
    k = torch.empty((pages, 128, 1, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = make(24, [ql], [ctx], hq)
    at = np.array([pages - 1, 5, pages - 7, pages - 2], np.int32)
    for i in range(4):
        for dst, src in ((k, small.k_cache), (v, small.v_cache)):
            page = src[small.block_table[0, i]]
            dst[int(at[i])] = torch.from_numpy(page.view(np.int16)).view(torch.bfloat16).cuda()
    c = case(small)
    bt = torch.from_numpy(at[None]).cuda()
    batch = B.make_batch(c.cu_q, c.cu_k, c.ctx, bt, pages, ql, max_q_len=ql)
    attn = B.make_attn_args(c.q, k, v, B.MSA_KV_BF16, pages, c.out, c.lse, softmax_scale=small.softmax_scale)
    ws = torch.empty((B.msa_tree_attn_workspace_size(1, ql, 4, hq, ql),), dtype=torch.uint8, device="cuda")
    tree = B.make_tree()
    B.msa_tree_attn(batch, tree, attn, ws, c.status)
    mass = torch.zeros((pages, 128), device="cuda")
    B.msa_attn_mass(batch, tree, attn, mass, ws, c.status)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check_attn(c, T.tree_attn(small))
    want, tol = T.attn_mass(small, c.lse.cpu().numpy(), np.zeros((small.num_pages, 128), np.float32))
    got = mass[torch.from_numpy(at).long().cuda()].double().cpu().numpy()
    order = small.block_table[0, :4]
    assert (np.abs(got - want[order]) <= tol[order]).all()


def test_v_scales_over_a_wide_range():
    # per-token scales over 2^-30 .. 2^30: the heavy ones decide, none overflows
    w = make(25, [4], [600], 16, F8, TOKEN)
    rng = np.random.default_rng(3)
    w.v_scale[:] = np.exp2(rng.uniform(-30, 30, w.v_scale.shape)).astype(np.float32)
    c = case(w)
    c.tree_attn()
    torch.cuda.synchronize()
    out, lse, ot, lt = T.tree_attn(w)
    # P times its scale is rounded relative to the largest scale met so far: 2^-24 of it each
    vmax = float(w.v_scale.max()) * 448
    err = np.abs(c.out.double().cpu().numpy() - out)
    assert (err <= ot + 604 * 2.0 ** -24 * vmax).all()


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("scale", [2.0 ** 60, np.inf, np.nan])
@pytest.mark.parametrize("ql,ctx", [(2, 300), (7, 300), (7, 0), (20, 1000)])
def test_hidden_scales_do_not_leak(kv, scale, ql, ctx):
    # the last drafted token, which its own row alone sees, has a v scale beside which every
    # other one's P would round to nothing
    w = make(33, [ql], [ctx], 16, kv, TOKEN)
    clean = W.custom(33, [ql], [ctx + ql], hq=16, kv_dtype=kv, scale_mode=TOKEN)
    mask = T.random_mask(np.random.default_rng(2), [ql], 1, "tree")
    pos = ctx + ql - 1
    w.v_scale[w.block_table[0, pos // 128], pos % 128] = scale
    c = case(w)
    c.tree_attn(mask=T.dev(mask))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    check_attn(c, T.tree_attn(clean, mask), slice(0, ql - 1))


def test_two_calls_at_once():
    # two batches on two streams, each with its workspace: the bits of the calls one by one
    ws = [make(41, [20, 64], [3000, 700], 16, BF, NONE), make(42, [5, 1], [9000, 2000], 8, F8, TOKEN),
          make(43, [1] * 9, [500 + 900 * i for i in range(9)], 16, BF, TOKEN)]
    cases = [case(w) for w in ws]
    masses = [torch.zeros((w.num_pages, 128), device="cuda") for w in ws]
    alone = []
    for c, m in zip(cases, masses):
        c.tree_attn()
        c.attn_mass(m)
        torch.cuda.synchronize()
        alone.append((c.out.clone(), c.lse.clone(), m.clone()))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for m in masses:
            m.zero_()
        torch.cuda.synchronize()
        for c, m, s in zip(cases, masses, streams):
            c.tree_attn(stream=s)
            c.attn_mass(m, stream=s)
        torch.cuda.synchronize()
        for c, m, (o, l, want) in zip(cases, masses, alone):
            assert int(c.status.item()) == 0
            assert torch.equal(c.out.view(torch.int16), o.view(torch.int16))
            assert torch.equal(c.lse, l) and torch.equal(m, want)

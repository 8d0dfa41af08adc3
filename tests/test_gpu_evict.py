"""Eviction from the cache on the GPU: the kept positions and the in-place move
against plain forms (bit for bit), and a serving step of all operators."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import tree_ref as T
from tests.test_gpu_tree import case, make, run_both

pytestmark = pytest.mark.gpu


def tables(rng, lens, extra=3):
    nb = [(max(n, 0) + 127) // 128 for n in lens]
    pages = sum(nb) + extra
    perm = rng.permutation(pages).astype(np.int32)
    bt = np.full((len(lens), max(1, max(nb))), -1, np.int32)
    at = 0
    for r, n in enumerate(nb):
        bt[r, :n] = perm[at:at + n]
        at += n
    return bt, pages


def select(lens, bt, mass, budget, first, recent, status=0):
    import block_sparse_paged_02_gb300 as msa
    keep = torch.full((len(lens), budget), 77, dtype=torch.int32, device="cuda")
    kl = torch.full((len(lens),), 77, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    view = msa.make_cache_view(T.dev(np.asarray(lens, np.int32)), T.dev(bt), mass.shape[0])
    msa.msa_evict_select(view, torch.from_numpy(mass).cuda(), budget, first, recent, keep, kl, st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return keep.cpu().numpy(), kl.cpu().numpy()


def masses(rng, pages, kind):
    m = rng.lognormal(-4, 2, (pages, 128)).astype(np.float32)
    if kind == "ties":
        m = rng.integers(0, 3, (pages, 128)).astype(np.float32)
    elif kind == "equal":
        m[:] = 0.25
    elif kind == "odd":  # NaN, infinities, signed zeros, negatives, denormals
        m = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, -1.5, 1e-42, -1e-42, 2.0], np.float32),
                       (pages, 128))
    elif kind == "near":  # keys that differ in their last bits only
        m = (np.float32(1.0).view(np.int32) + rng.integers(0, 300, (pages, 128))).astype(np.int32).view(np.float32)
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd", "near"])
@pytest.mark.parametrize("lens,budget,first,recent", [
    ([1, 5, 0, 64], 16, 2, 3), ([1000, 129, 128, 127], 128, 0, 0), ([5000, 300, 2049], 1000, 4, 500),
    ([700], 700, 10, 10), ([701], 700, 350, 350), ([4097, 9000], 1, 0, 0), ([3000], 1, 1, 0),
    ([2600, 40000], 2048, 64, 256)])
def test_select(kind, lens, budget, first, recent):
    rng = np.random.default_rng(len(lens) * budget)
    bt, pages = tables(rng, lens)
    m = masses(rng, pages, kind)
    got = select(lens, bt, m, budget, first, recent)
    want = T.evict(lens, bt, m, budget, first, recent)
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])


def test_select_long():
    rng = np.random.default_rng(3)
    lens = [700001, 260000]
    bt, pages = tables(rng, lens)
    m = masses(rng, pages, "plain")
    m[rng.random((pages, 128)) < 0.5] = 0.0
    for budget, recent in ((20000, 1000), (600000, 0)):
        got, kl = select(lens, bt, m, budget, 100, recent)
        for r, n in enumerate(lens):
            pos = np.arange(n)
            v = m[bt[r, pos // 128], pos % 128].astype(np.float64)
            v[:100] = v[n - recent:] = np.inf
            want = np.sort(np.argsort(-v, kind="stable")[:budget])
            assert kl[r] == min(n, budget)
            assert np.array_equal(got[r, :kl[r]], want[:kl[r]])
            assert (got[r, kl[r]:] == -1).all()


def test_select_refuses_bad_requests():
    rng = np.random.default_rng(4)
    lens = [300, 500, 400]
    bt, pages = tables(rng, lens)
    m = masses(rng, pages, "plain")
    good = T.evict(lens, bt, m, 100, 1, 1)
    bad_bt = bt.copy()
    bad_bt[1, 2] = pages
    got, kl = select(lens, bad_bt, m, 100, 1, 1, status=1)
    assert kl[1] == -1 and (got[1] == -1).all()
    assert np.array_equal(got[[0, 2]], good[0][[0, 2]])
    got, kl = select([300, -1, 128 * bt.shape[1] + 1], bt, m, 100, 1, 1, status=4)
    assert kl.tolist() == [100, -1, -1] and np.array_equal(got[0], good[0][0])


def pool_set(rng, pages, kv, hkv, scales, hi, di, index, mass):
    el = np.uint8 if kv == W.KV_FP8 else np.uint16
    out = [rng.integers(0, 256 ** np.dtype(el).itemsize, (pages, 128, hkv, 128)).astype(el) for _ in range(2)]
    out += [rng.random((pages, 128, hkv)).astype(np.float32) for _ in range(2)] if scales else [None, None]
    out.append(rng.integers(0, 256 ** np.dtype(el).itemsize, (pages, 128, hi, di)).astype(el) if index else None)
    out.append(rng.random((pages, 128, hi)).astype(np.float32) if index and kv == W.KV_FP8 else None)
    out.append(rng.random((pages, 128)).astype(np.float32) if mass else None)
    return out


def on_device(a):
    if a is None:
        return None
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(a).cuda()


def on_host(t, like):
    t = t.cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if like.dtype == np.uint16 else t.numpy()


def move(pools, kv, lens, bt, keep, kl, base=None, status=0, check_skip=()):
    import block_sparse_paged_02_gb300 as msa
    d = [on_device(p) for p in pools]
    k, v, ks, vs, idx, idx_s, mass = d
    index = None if idx is None else msa.make_index_cache(idx, kv, idx_s)
    p = msa.make_kv_pools(k, v, kv, scale_mode=msa.MSA_SCALE_PER_TOKEN_HEAD if ks is not None else 0, k_scale=ks,
                          v_scale=vs, index=index, mass=mass)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    view = msa.make_cache_view(T.dev(np.asarray(lens, np.int32)), T.dev(bt), k.shape[0])
    msa.msa_kv_compact(view, None if base is None else T.dev(np.asarray(base, np.int32)), T.dev(keep),
                       T.dev(np.asarray(kl, np.int32)), p, st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    have = [x for x in pools if x is not None]
    want = T.compact(have, lens, bt, keep, kl, base, check_skip)
    for a, b, t in zip(have, want, [x for x in d if x is not None]):
        assert np.array_equal(on_host(t, a), b)


def lists(rng, lens, budget, base=None):
    keep = np.full((len(lens), budget), -1, np.int32)
    kl = []
    for r, n in enumerate(lens):
        free = n - (0 if base is None else base[r])
        m = int(min(budget, free, max(0, rng.integers(0, budget + 1))))
        keep[r, :m] = np.sort(rng.permutation(free)[:m])
        kl.append(m)
    return keep, kl


@pytest.mark.parametrize("kv,hkv,scales,hi,di", [(W.KV_BF16, 1, False, 1, 128), (W.KV_BF16, 1, True, 1, 64),
                                                 (W.KV_FP8, 1, True, 2, 64), (W.KV_FP8, 3, True, 1, 128),
                                                 (W.KV_BF16, 2, False, 1, 128)])
@pytest.mark.parametrize("lens,budget", [([1, 2, 130], 130), ([5000, 3, 700], 2600), ([129, 0, 4000], 512)])
def test_move(kv, hkv, scales, hi, di, lens, budget):
    rng = np.random.default_rng(budget + hkv)
    bt, pages = tables(rng, lens)
    keep, kl = lists(rng, lens, budget)
    kl[0] = min(lens[0], budget)  # one request keeps a full list
    keep[0, :kl[0]] = np.sort(rng.permutation(lens[0])[:kl[0]])
    for index in (True, False):
        move(pool_set(rng, pages, kv, hkv, scales, hi, di, index, index), kv, lens, bt, keep, kl)


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_FP8])
def test_commit_of_a_tree(kv):
    rng = np.random.default_rng(8)
    base = [0, 127, 128, 1000, 77]
    lens = [b + t for b, t in zip(base, [1, 8, 64, 200, 256])]
    bt, pages = tables(rng, lens)
    keep, kl = lists(rng, lens, 64, base)
    kl[1] = 0
    move(pool_set(rng, pages, kv, 1, kv == W.KV_FP8, 1, 128, True, True), kv, lens, bt, keep, kl, base)


def test_move_of_long_lists_and_everything_kept():
    rng = np.random.default_rng(9)
    lens = [60000, 30000]
    bt, pages = tables(rng, lens)
    keep = np.full((2, 30000), -1, np.int32)
    keep[0] = np.sort(rng.permutation(60000)[:30000])
    keep[1] = np.arange(30000)  # nothing moves
    move(pool_set(rng, pages, W.KV_FP8, 1, True, 1, 128, True, True), W.KV_FP8, lens, bt, keep, [30000, 30000])


def test_move_refuses_bad_lists():
    rng = np.random.default_rng(10)
    lens = [300, 300, 300, 300, 300, 300]
    bt, pages = tables(rng, lens)
    keep = np.tile(np.arange(0, 200, 2, dtype=np.int32), (6, 1))
    kl = [100] * 6
    keep[1, 50] = keep[1, 49]        # repeated
    keep[2, 0] = -1                  # negative
    keep[3, 99] = 300                # past the end
    kl[4] = 101                      # longer than the list
    pools = pool_set(rng, pages, W.KV_BF16, 1, False, 1, 128, True, True)
    move(pools, W.KV_BF16, lens, bt, keep, kl, status=8, check_skip=(1, 2, 3, 4))
    bt2 = bt.copy()
    bt2[5, 2] = -3
    move(pools, W.KV_BF16, lens, bt2, keep, [100, 0, 0, 0, 0, 100], status=1, check_skip=(5,))
    move(pools, W.KV_BF16, [300, 9000, 300, 300, 300, -4], bt, keep, [100, 100, 0, 0, -1, 100], status=4, check_skip=(1, 4, 5))
    move(pools, W.KV_BF16, lens, bt, keep, [100, 100, 0, 0, 0, 0], base=[-1, 400, 0, 0, 0, 0], status=8, check_skip=(0, 1))


def test_a_serving_step():
    """Drafts inserted, attended on their selected blocks, the accepted path committed, the cache
    evicted to a budget, and the next tokens attended over what is left: each step against the
    plain forms on the same state."""
    q_lens, ctxs = [9, 24, 17], [900, 2100, 1500]
    w = make(31, q_lens, ctxs, 16, W.KV_BF16, W.SCALE_NONE, True)
    rng = np.random.default_rng(6)
    mask = T.random_mask(rng, q_lens, 1)
    c = case(w, topk=4)
    n = w.num_rows
    new = [torch.randn((n, 1, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(s)).to(torch.bfloat16)
           for s in range(3)]
    c.kv_insert(*new)
    c.index_score()
    c.topk_build_table()
    c.tree_attn(mask=T.dev(mask), topk_idx=c.topk_idx)
    mass = torch.rand((w.num_pages, 128), device="cuda")
    m0 = mass.cpu().numpy().copy()
    c.attn_mass(mass, mask=T.dev(mask), topk_idx=c.topk_idx)
    torch.cuda.synchronize()
    w.k_cache, w.v_cache, w.idx_k = (on_host(t, np.zeros(0, np.uint16)).copy() for t in (c.k, c.v, c.idx_k))
    topk = c.topk_idx.cpu().numpy()
    from tests.test_gpu_tree import check_attn
    check_attn(c, T.tree_attn(w, mask, topk))
    want, tol = T.attn_mass(w, c.lse.cpu().numpy(), m0, mask, topk)
    assert (np.abs(mass.double().cpu().numpy() - want) <= tol).all()
    # commit an accepted path of each tree
    accepted = np.full((3, 4), -1, np.int32)
    for r, path in enumerate(([0, 3, 8], [1, 2, 20, 23], [16])):
        accepted[r, :len(path)] = path
    al = np.array([3, 4, 1], np.int32)
    seq = np.array(ctxs) + q_lens
    pools = [w.k_cache, w.v_cache, w.idx_k, mass.cpu().numpy()]
    c.kv_compact(T.dev(seq.astype(np.int32)), T.dev(accepted), T.dev(al), base=c.ctx, mass=mass)
    pools = T.compact(pools, seq, w.block_table, accepted, al, ctxs)
    lens = (np.array(ctxs) + al).astype(np.int32)
    # evict to a budget
    keep, kl = c.evict_select(T.dev(lens), mass, 600, 4, 64)
    c.kv_compact(T.dev(lens), keep, kl, mass=mass)
    torch.cuda.synchronize()
    wk, wl = T.evict(lens, w.block_table, pools[3], 600, 4, 64)
    assert np.array_equal(keep.cpu().numpy(), wk) and np.array_equal(kl.cpu().numpy(), wl)
    pools = T.compact(pools, lens, w.block_table, wk, wl)
    for t, p in zip((c.k, c.v, c.idx_k, mass), pools):
        assert np.array_equal(on_host(t, p), p)
    assert int(c.status.item()) == 0
    # the next step's single tokens over the evicted cache
    w2 = make(31, [1, 1, 1], (wl - 1).tolist(), 16, W.KV_BF16, W.SCALE_NONE, True)
    w2.k_cache, w2.v_cache, w2.num_pages = pools[0], pools[1], w.num_pages
    w2.idx_k = w.idx_k
    w2.block_table = w.block_table[:, :w2.bt_stride].copy()
    run_both(w2)

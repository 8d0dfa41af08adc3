"""Forked, reordered and grown page tables and page copies on the GPU against the rules taken step by
step (prompt_ref.fork); prompts, forks and decode together."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import prompt_ref as P
from tests import tree_ref as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class Fork:
    def __init__(self, msa, lens, table, refs, parent, grow, width, stream=None):
        self.n, self.width, self.pages = len(parent), width, len(refs)
        i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
        self.out = [i32(self.n), i32(self.n, width), i32(self.pages), i32(self.n), i32(self.n), i32(self.n)]
        self.to = msa.make_page_set(*self.out)
        self.args = (msa.make_cache_view(dev(lens), dev(table), self.pages), dev(refs), dev(parent),
                     None if grow is None else dev(grow), self.to)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        msa.msa_page_fork(*self.args, self.status, stream=stream)
        torch.cuda.synchronize()
        self.got = [t.cpu().numpy() for t in self.out]


def check(msa, lens, table, refs, parent, grow, width):
    f = Fork(msa, lens, table, refs, parent, grow, width)
    want = P.fork(np.asarray(lens), np.asarray(table), np.asarray(refs), parent,
                  [0] * len(parent) if grow is None else grow, width, len(refs))
    if isinstance(want, int):
        assert int(f.status.item()) == want
        assert (f.got[0] == -1).all() and (f.got[1] == 77).all() and np.array_equal(f.got[2], refs)
        assert (f.got[3] == -1).all() and (f.got[4] == -1).all() and (f.got[5] == 0).all()
        return None
    assert int(f.status.item()) == 0
    for i, name in ((0, "lens"), (2, "refs"), (3, "src"), (4, "dst"), (5, "tokens")):
        assert np.array_equal(f.got[i], want[i]), name
    live = want[1] >= 0
    assert np.array_equal(f.got[1][live], want[1][live]) and (f.got[1][~live] == 77).all()
    return want


def state(rng, n, most, extra, share=True):
    """Requests with tables over shuffled pages, some sharing a prefix, some pages held elsewhere too."""
    lens = rng.integers(0, most * 128 + 1, n)
    lens[rng.random(n) < 0.2] &= ~127      # whole pages
    nb = (lens + 127) // 128
    pages = int(nb.sum()) + extra
    perm = rng.permutation(pages)
    table = np.full((n, most + 1), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    at = 0
    for r in range(n):
        head = 0
        if share and r and rng.random() < 0.4:   # a prefix of whole pages, now and then the partial one too
            o = int(rng.integers(0, r))
            head = int(min(nb[r], lens[o] // 128))
            if lens[r] == lens[o]:
                head = nb[r]
            table[r, :head] = table[o, :head]
        table[r, head:nb[r]] = perm[at:at + nb[r] - head]
        at += nb[r] - head
        refs[table[r, :nb[r]]] += 1
    refs[perm[at:at + extra // 4]] = 1
    held = np.flatnonzero(refs)
    refs[held[rng.random(len(held)) < 0.1]] += 2
    return lens.astype(np.int32), table, refs


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("n,new,most", [(1, 1, 1), (1, 9, 5), (8, 8, 4), (40, 70, 6), (300, 200, 3), (5, 3, 400), (2000, 2500, 2)])
def test_random(msa, seed, n, new, most):
    rng = np.random.default_rng(1000 * seed + n)
    lens, table, refs = state(rng, n, most, 400 + 4 * new)
    parent = rng.integers(-1, n, new)
    grow = np.where(rng.random(new) < 0.3, 0, rng.integers(0, 200, new))
    check(msa, lens, table, refs, parent, grow, most + 4)


def test_beams_keep_and_copy(msa):
    # two beams: 0 goes on twice, 1 is dropped; a partial page of 5 tokens
    lens, table = [261, 261], [[4, 7, 9, -1], [4, 7, 2, -1]]
    refs = np.zeros(12, np.int32)
    refs[[4, 7]] = 2
    refs[[9, 2]] = 1
    want = check(msa, lens, table, refs, [0, 0], [1, 1], 4)
    assert want[1].tolist() == [[4, 7, 9, -1], [4, 7, 0, -1]]
    assert want[3].tolist() == [-1, 9] and want[4].tolist() == [-1, 0] and want[5].tolist() == [0, 5]
    assert want[2][2] == 0 and want[2][4] == 2
    # without growth nothing is copied, and the call that grows them later copies
    want = check(msa, lens, table, refs, [0, 0], None, 4)
    assert want[2][9] == 2 and (want[5] == 0).all()
    again = check(msa, want[0], want[1], want[2], [1, 0], [1, 130], 4)
    assert again[1][0, 2] == 9 and again[5].tolist() == [0, 5]
    # a prefix cache holds the partial page: both copy
    refs[9] += 1
    want = check(msa, lens, table, refs, [0, 0], [1, 1], 4)
    assert want[5].tolist() == [5, 5] and want[2][9] == 1


def test_new_requests_drops_and_whole_pages(msa):
    refs = np.array([1, 0, 1, 0, 0, 0], np.int32)
    want = check(msa, [256], [[0, 2]], refs, [-1, 0], [300, 1], 3)
    assert want[1].tolist() == [[1, 3, 4], [0, 2, 5]] and want[0].tolist() == [0, 256]
    # dropped pages are free for the requests that go on
    want = check(msa, [256], [[0, 2]], refs, [-1], [6 * 128], 6)
    assert want[1].tolist() == [[0, 1, 2, 3, 4, 5]]
    # nobody goes on; no old requests
    want = check(msa, [256], [[0, 2]], refs, [], [], 1)
    assert (want[2] == 0).all()
    want = check(msa, [], np.zeros((0, 1), np.int32), refs, [-1, -1], [0, 1], 1)
    assert want[1].tolist() == [[-1], [1]]


def test_refused_data(msa):
    lens, table, refs = [200, 100], [[0, 1], [2, -1]], np.array([1, 1, 1, 0, 0], np.int32)
    bad = lambda **k: check(msa, k.get("lens", lens), k.get("table", table), k.get("refs", refs), k.get("parent", [0, 1]),
                            k.get("grow", [1, 1]), k.get("width", 2))
    assert bad() is not None
    assert bad(lens=[-1, 100]) is None and bad(lens=[257, 100]) is None
    assert bad(parent=[0, 2]) is None and bad(parent=[-2, 0]) is None
    assert bad(grow=[1, -1]) is None and bad(grow=[57, 1]) is None and bad(grow=[2 ** 31 - 1, 1]) is None
    assert bad(table=[[0, 5], [2, -1]]) is None and bad(table=[[0, -1], [2, -1]]) is None
    assert bad(refs=np.array([1, 1, 0, 0, 0], np.int32)) is None
    # one page too few
    assert bad(parent=[0, 0, 1], grow=[1, 1, 29], width=2) is not None
    assert bad(parent=[0, 0, 0, 1], grow=[1, 1, 1, 29], width=2) is None


def test_most_requests_and_pages(msa):
    rng = np.random.default_rng(9)
    lens, table, refs = state(rng, 4096, 3, 5000, share=False)
    check(msa, lens, table, refs, rng.integers(-1, 4096, 4096), rng.integers(0, 130, 4096), 6)
    # a wide table, most of the pool behind the first free pages
    lens, table, refs = state(rng, 3, 9000, 300001)
    check(msa, lens, table, refs, [2, 0, 0, 1, -1], [5, 700, 1, 0, 30000], 16384)


def test_fork_streams_and_graphs(msa):
    rng = np.random.default_rng(5)
    lens, table, refs = state(rng, 30, 5, 300)
    parent, grow = rng.integers(-1, 30, 40), rng.integers(0, 99, 40)
    f = Fork(msa, lens, table, refs, parent, grow, 8)
    side = torch.cuda.Stream()
    g = Fork(msa, lens, table, refs, parent, grow, 8, stream=side)
    assert all(np.array_equal(a, b) for a, b in zip(f.got, g.got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_page_fork(*f.args, f.status)
    for t in f.out:
        t.fill_(77)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(t.cpu().numpy(), b) for t, b in zip(f.out, f.got))


@pytest.mark.parametrize("layers", [1, 3, 41])
@pytest.mark.parametrize("kv,scaled,hk,hi,di,xs", [("bf16", False, 1, 1, 128, False), ("fp8", True, 1, 1, 128, True),
                                                   ("fp8", False, 3, 2, 64, True), ("bf16", True, 2, 1, 64, False),
                                                   ("fp8", True, 5, 0, 0, False)])
def test_page_copy(msa, layers, kv, scaled, hk, hi, di, xs):
    rng = np.random.default_rng(layers)
    pages, n = 23, 9
    perm = rng.permutation(pages)
    src, dst = perm[:n], perm[n:2 * n]
    src[3] = src[1]                          # one page copied twice
    tokens = np.array([1, 128, 5, 127, 0, 64, -3, 33, 2])
    kind = msa.MSA_KV_FP8_E4M3 if kv == "fp8" else msa.MSA_KV_BF16
    mode = msa.MSA_SCALE_PER_TOKEN_HEAD if scaled else msa.MSA_SCALE_NONE
    raw = lambda *s: torch.from_numpy(rng.integers(0, 255, s).astype(np.uint8)).cuda()
    data, structs = [], []
    for i in range(layers):
        pool = lambda h, d: raw(pages, 128, h, d) if kv == "fp8" else raw(pages, 128, h, 2 * d).view(torch.bfloat16)
        f32 = lambda h: raw(pages, 128, 4 * h).view(torch.float32).view(pages, 128, h)
        t = dict(k=pool(hk, 128), v=pool(hk, 128))
        if scaled:
            t.update(ks=f32(hk), vs=f32(hk))
        if hi:
            t["x"] = pool(hi, di)
            if xs:
                t["xs"] = f32(hi)
        if i % 2:
            t["mass"] = f32(1).view(pages, 128)
        idx = msa.make_index_cache(t["x"], kind, t.get("xs")) if hi else None
        structs.append(msa.make_kv_pools(t["k"], t["v"], kind, scale_mode=mode, k_scale=t.get("ks"), v_scale=t.get("vs"),
                                         index=idx, mass=t.get("mass")))
        data.append(t)
    want = [{k: v.clone() for k, v in t.items()} for t in data]
    for t in want:
        for v in t.values():
            b = v.view(torch.uint8).view(pages, 128, -1)
            for a, c, m in zip(src, dst, tokens):
                if m > 0:
                    b[c, :m] = b[a, :m].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_page_copy(structs, dev(src), dev(dst), dev(tokens), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for t, u in zip(data, want):
        for k in t:
            assert torch.equal(t[k].view(torch.uint8), u[k].view(torch.uint8)), k


def test_page_copy_skips_what_is_out_of_range(msa):
    x = torch.arange(4 * 128 * 128, device="cuda").view(4, 128, 1, 128).to(torch.bfloat16)
    k, v = x.clone(), (x + 1).clone()
    p = msa.make_kv_pools(k, v, msa.MSA_KV_BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_page_copy([p], dev([0, 4, 0, 1]), dev([1, 2, -1, 3]), dev([10, 5, 5, 129]), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 1 | 4
    want = x.clone()
    want[1, :10] = x[0, :10]
    assert torch.equal(k, want)


@pytest.mark.parametrize("kv,scale", [(W.KV_BF16, W.SCALE_NONE), (W.KV_FP8, W.SCALE_PER_TOKEN_HEAD)])
def test_prompt_fork_and_decode_together(msa, kv, scale):
    """A prompt of two chunks through norm, rotation, insertion and attention; its cache forked for three
    continuations with one new token each; their decode reads the shared pages and their own copies."""
    n, heads, pages, width = 300, 8, 12, 4
    rng = np.random.default_rng(8)
    gen = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()
    fp8 = kv == W.KV_FP8
    pool = lambda: torch.full((pages, 128, 1, 128), 0x7f, dtype=torch.uint8, device="cuda") if fp8 else \
        torch.full((pages, 128, 1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v, ix = pool(), pool(), pool()
    sc = lambda: torch.ones((pages, 128, 1), device="cuda") if fp8 else None
    ks, vs, xs = sc(), sc(), sc()
    kind = msa.MSA_KV_FP8_E4M3 if fp8 else msa.MSA_KV_BF16
    idx = msa.make_index_cache(ix, kind, xs)
    pools = msa.make_kv_pools(k, v, kind, scale_mode=scale, k_scale=ks, v_scale=vs, index=idx)
    half = 32
    a = np.arange(1024)[:, None] * 1e4 ** -(np.arange(half) / half)
    rope = msa.make_rope(torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().cuda())
    weights = [gen(128).abs() for _ in range(4)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(rows, cu, ctx, table):
        """One layer's step for rows of a batch; returns q, out, lse"""
        m = rows.shape[0]
        part = lambda i, h: rows[:, i * 128:(i + h) * 128].unflatten(1, (h, 128))
        q, iq = (torch.empty((m, h, 128), dtype=torch.bfloat16, device="cuda") for h in (heads, 1))
        cu_q = dev(cu)
        cu_k = torch.zeros(len(cu), dtype=torch.int32, device="cuda")
        cu_k[1:] = torch.cumsum(cu_q[1:] - cu_q[:-1] + ctx, 0)
        batch = msa.make_batch(cu_q, cu_k, ctx, table, pages, m)
        qkv = msa.make_qkv(part(0, heads), part(heads, 1), part(heads + 1, 1), q, idx_q=part(heads + 2, 1), idx_k=part(heads + 3, 1),
                           idx_q_out=iq, q_norm=weights[0], k_norm=weights[1], idx_q_norm=weights[2], idx_k_norm=weights[3])
        msa.msa_qk_rope_insert(batch, qkv, rope, pools, status)
        out = torch.empty_like(q)
        lse = torch.empty((m, heads), device="cuda")
        attn = msa.make_attn_args(q, k, v, kind, pages, out, lse, scale_mode=scale, k_scale=ks, v_scale=vs, softmax_scale=128 ** -0.5)
        ws = torch.empty(msa.msa_prompt_attn_workspace_size(heads, 1), dtype=torch.uint8, device="cuda")
        msa.msa_prompt_attn(batch, attn, ws, status)
        return q, out, lse

    def fork(lens, table, refs, parent, grow):
        m = len(parent)
        i32 = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")
        to = msa.make_page_set(i32(m), i32(m, width), i32(pages), i32(m), i32(m), i32(m))
        msa.msa_page_fork(msa.make_cache_view(lens, table, pages), refs, dev(parent), dev(grow), to, status)
        msa.msa_page_copy([pools], *to._keep[3:], status)
        return to._keep[:3]

    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    rows = gen(n, (heads + 4) * 128)
    lens, table, refs = fork(none.view(-1), none, refs, [-1], [n])
    chunk = 190
    got = [step(rows[:chunk], [0, chunk], lens, table), step(rows[chunk:], [0, n - chunk], lens + chunk, table)]
    lens, table, refs = fork(lens + n, table, refs, [0, 0, 0], [1, 1, 1])
    more = gen(3, (heads + 4) * 128)
    got.append(step(more, [0, 1, 2, 3], lens, table))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    t = table.cpu().numpy()
    assert (t[:, :2] == t[0, :2]).all() and len(set(t[:, 2])) == 3 and lens.tolist() == [n] * 3
    assert sorted(refs.tolist(), reverse=True)[:6] == [3, 3, 1, 1, 1, 0]
    # each continuation's cache as it stands, in 64 bits
    host = lambda x: x.cpu().numpy() if fp8 else x.view(torch.int16).cpu().numpy().view(np.uint16)
    for r, (q, out, lse) in [(0, got[0]), (0, got[1])] + [(r, [x[r:r + 1] for x in got[2]]) for r in range(3)]:
        m = q.shape[0]
        ctx = {chunk: 0, n - chunk: chunk, 1: n}[m]
        w = P.batch(1, [m], [ctx], heads, 1, kv, scale)
        w.q[:] = q.view(torch.int16).cpu().numpy().view(np.uint16)
        w.num_pages = pages
        w.block_table = t[r:r + 1]
        w.k_cache, w.v_cache = host(k), host(v)
        if fp8:
            w.k_scale, w.v_scale = ks.cpu().numpy(), vs.cpu().numpy()

        class C:
            pass
        C.out, C.lse = out, lse
        P.check_attn(C, P.attn(w))
    # single tokens agree with the draft-tree attention over the same pages
    ctx = dev([n] * 3)
    batch = msa.make_batch(dev([0, 1, 2, 3]), dev([0, n + 1, 2 * n + 2, 3 * n + 3]), ctx, table, pages, 3, max_q_len=1)
    q, want, want_lse = got[2]
    out, lse = torch.empty_like(q), torch.empty((3, heads), device="cuda")
    attn = msa.make_attn_args(q, k, v, kind, pages, out, lse, scale_mode=scale, k_scale=ks, v_scale=vs, softmax_scale=128 ** -0.5)
    ws = torch.empty(msa.msa_tree_attn_workspace_size(3, 3, width, heads, 1), dtype=torch.uint8, device="cuda")
    msa.msa_tree_attn(batch, msa.make_tree(), attn, ws, status)
    torch.cuda.synchronize()
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
    assert (lse - want_lse).abs().max() < 1e-4


def test_case_methods(msa):
    w = P.batch(3, [5, 2], [300, 128], 8)
    c = msa.DeviceCase(w)
    lens = dev(w.context_lens)
    refs = torch.zeros(w.num_pages, dtype=torch.int32, device="cuda")
    for r in range(2):
        refs[torch.from_numpy(w.block_table[r, :(int(w.context_lens[r]) + 127) // 128].astype(np.int64)).cuda()] += 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    to = c.page_fork(lens, refs, dev([0, 0]), dev([1, 1]), bt_stride=4, stream=side)
    keep = c.k.clone()
    c.page_copy(*to._keep[3:], stream=side)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and to._keep[5].tolist() == [0, 300 % 128]
    src, dst = int(to._keep[3][1]), int(to._keep[4][1])
    assert torch.equal(c.k[dst, :44].view(torch.int16), keep[src, :44].view(torch.int16))

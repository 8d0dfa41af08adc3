"""Norm, rotation and insertion on the GPU against the 64-bit plain form, and against msa_kv_insert."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import prompt_ref as P

pytestmark = pytest.mark.gpu

BF, F8 = W.KV_BF16, W.KV_FP8
NONE, SCALAR, TOKEN = W.SCALE_NONE, W.SCALE_SCALAR, W.SCALE_PER_TOKEN_HEAD


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


def table(top, rotary, base=10000.0):
    a = np.arange(top)[:, None] * base ** -(np.arange(rotary // 2) / max(1, rotary // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Setup:
    """A batch with pools of hk heads and an index cache, its vectors side by side in one projection."""

    def __init__(self, msa, q_lens, ctxs, h=16, hk=1, hi=1, di=128, kv=BF, scale=NONE, idx_fp8=False, idx_scaled=True,
                 rotary=64, near=False, norm=True, shift=0.0, eps=1e-5, seed=3, given=False, pad=0, top=70000):
        self.msa, self.h, self.hk, self.hi, self.di = msa, h, hk, hi, di
        self.w = w = P.batch(seed, q_lens, ctxs, 16, hk, kv, scale)
        rng = np.random.default_rng(seed)
        n = w.num_rows
        width = (h + 2 * hk) * 128 + 2 * hi * di + pad
        x = rng.standard_normal((n, width)) * np.exp(rng.standard_normal((n, 1)))
        self.proj = torch.from_numpy(x).to(torch.bfloat16).cuda()
        cut = np.cumsum([0, h * 128, hk * 128, hk * 128, hi * di, hi * di])
        part = lambda i, heads, d: self.proj[:, cut[i]:cut[i + 1]].unflatten(1, (heads, d)) if heads else None
        self.q, self.k, self.v = part(0, h, 128), part(1, hk, 128), part(2, hk, 128)
        self.idx_q, self.idx_k = part(3, hi, di), part(4, hi, di)
        weight = lambda d: (torch.from_numpy(rng.standard_normal(d) * 0.3 + 1 - shift).to(torch.bfloat16).cuda()
                            if norm and d else None)
        self.norms = [weight(128), weight(128), weight(di) if hi else None, weight(di) if hi else None]
        self.shift, self.eps, self.near, self.top = shift, eps, near, top
        self.cs = table(top, rotary) if rotary else None
        ctx = np.asarray(w.context_lens)
        req = np.searchsorted(w.cu_seqlens_q, np.arange(n), side="right") - 1
        self.pos = ctx[req] + np.arange(n) - np.asarray(w.cu_seqlens_q)[req]
        self.slot = w.block_table[req, self.pos // 128].astype(np.int64) * 128 + self.pos % 128
        self.given = rng.integers(0, top, n).astype(np.int32) if given else None
        bits = lambda a: torch.from_numpy(a.copy()) if a.dtype == np.uint8 else torch.from_numpy(a.view(np.int16).copy()).view(torch.bfloat16)
        self.pools = [bits(w.k_cache).cuda(), bits(w.v_cache).cuda()]
        P_ = w.num_pages
        if hi:
            idx = torch.from_numpy(rng.standard_normal((P_, 128, hi, di))).to(torch.bfloat16)
            self.pools.append((idx.to(torch.float8_e4m3fn).view(torch.uint8) if idx_fp8 else idx).cuda())
        self.kv, self.scale, self.idx_fp8 = kv, scale, idx_fp8
        dev = lambda a: None if a is None else torch.from_numpy(a.copy()).cuda()
        self.ks, self.vs = dev(w.k_scale), dev(w.v_scale)
        self.xs = torch.ones((P_, 128, hi), device="cuda") if hi and idx_fp8 and idx_scaled else None
        self.before = [t.clone() for t in self.pools]
        self.q_out = torch.full((n, h, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.iq_out = torch.full((n, hi, di), float("nan"), dtype=torch.bfloat16, device="cuda") if hi else None
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self, index=True, mass=None, q=None, q_out=None):
        m, w = self.msa, self.w
        geo = [torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in (w.cu_seqlens_q, w.cu_seqlens_k, w.context_lens, w.block_table)]
        batch = m.make_batch(*geo, w.num_pages, w.num_rows)
        on = index and self.hi
        qkv = m.make_qkv(self.q if q is None else q, self.k, self.v, self.q_out if q_out is None else q_out,
                         idx_q=self.idx_q if on else None, idx_k=self.idx_k if on else None, idx_q_out=self.iq_out if on else None,
                         q_norm=self.norms[0], k_norm=self.norms[1], idx_q_norm=self.norms[2] if on else None,
                         idx_k_norm=self.norms[3] if on else None, eps=self.eps, norm_shift=self.shift)
        rope = m.make_rope(None if self.cs is None else torch.from_numpy(self.cs).cuda(), interleaved=self.near,
                           positions=None if self.given is None else torch.from_numpy(self.given).cuda())
        idx = m.make_index_cache(self.pools[2], m.MSA_KV_FP8_E4M3 if self.idx_fp8 else m.MSA_KV_BF16, self.xs) if on else None
        pools = m.make_kv_pools(self.pools[0], self.pools[1], m.MSA_KV_FP8_E4M3 if self.kv == F8 else m.MSA_KV_BF16,
                                scale_mode=self.scale, k_scale=self.ks, v_scale=self.vs, index=idx, mass=mass)
        return batch, qkv, rope, pools

    def run(self, **kw):
        self.msa.msa_qk_rope_insert(*self.args(**kw), self.status)
        torch.cuda.synchronize()
        return int(self.status.item())

    def wanted(self, x, i):
        """(positions outside the table: any, their rows are not looked at)"""
        w = self.norms[i]
        return P.through(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), self.shift, self.eps,
                         self.cs, self.pos if self.given is None else np.clip(self.given, 0, self.top - 1), self.near)

    def check_pool(self, pool, before, fp8, want, tol, scale, scaled, rows=None):
        """The rows' slots hold the wanted values, every other slot what it held."""
        rows = np.arange(len(self.slot)) if rows is None else np.asarray(rows)
        heads, dim = pool.shape[2:]
        flat = lambda t: t.view(-1, heads, dim)
        keep = torch.ones(pool.shape[0] * 128, dtype=torch.bool, device="cuda")
        keep[torch.from_numpy(self.slot[rows]).cuda()] = False
        raw = lambda t: flat(t).view(torch.uint8) if fp8 else flat(t).view(torch.int16)
        assert torch.equal(raw(pool)[keep], raw(before)[keep])
        got = flat(pool)[torch.from_numpy(self.slot[rows]).cuda()]
        got = (got.view(torch.float8_e4m3fn) if fp8 else got).double().cpu().numpy()
        want, tol = want[rows], tol[rows]
        if not fp8:
            assert (np.abs(got - want) <= tol + 2.0 ** -8 * np.abs(want)).all()
            return
        by = np.ones(want.shape[:2])
        if scaled == SCALAR:
            by[:] = float(scale.item())
        elif scaled == TOKEN:
            s = scale.view(-1, heads)[torch.from_numpy(self.slot[rows]).cuda()].double().cpu().numpy()
            top = np.abs(want).max(-1)
            by = np.where(top > 0, top / 448, 1)
            err = np.where(top > 0, tol.max(-1) / 448, 0) + 2.0 ** -24 * by
            assert (np.abs(s - by) <= err).all()
        x = np.clip(want / by[..., None], -448, 448)
        slack = tol / by[..., None] + 2.0 ** -22 * np.abs(x)
        # half a step of e4m3: 2^-4 of the value, 2^-10 below its normal range
        assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + slack).all()

    def check(self, rows=None, index=True):
        r = slice(None) if rows is None else rows
        out = [(self.q, self.q_out, 0)] + ([(self.idx_q, self.iq_out, 2)] if self.hi and index else [])
        for x, got, i in out:
            want, tol = self.wanted(x, i)
            err = np.abs(got.double().cpu().numpy() - want)
            assert (err <= tol + 2.0 ** -8 * np.abs(want))[r].all()
        k, kt = self.wanted(self.k, 1)
        v = self.v.double().cpu().numpy()
        self.check_pool(self.pools[0], self.before[0], self.kv == F8, k, kt, self.ks, self.scale, rows)
        self.check_pool(self.pools[1], self.before[1], self.kv == F8, v, 0 * v, self.vs, self.scale, rows)
        if self.hi and index:
            x, xt = self.wanted(self.idx_k, 3)
            self.check_pool(self.pools[2], self.before[2], self.idx_fp8, x, xt, self.xs, TOKEN if self.xs is not None else NONE, rows)


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, NONE), (F8, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("hi,di,idx_fp8", [(1, 128, False), (1, 64, True), (2, 64, False), (2, 64, True), (0, 0, False)])
@pytest.mark.parametrize("near", [False, True])
def test_types(msa, kv, scale, hi, di, idx_fp8, near):
    s = Setup(msa, [1, 40, 3], [700, 100, 0], kv=kv, scale=scale, hi=hi, di=di, idx_fp8=idx_fp8, near=near)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 48, 64, 112, 128])
@pytest.mark.parametrize("norm,shift", [(True, 0.0), (True, 1.0), (False, 0.0)])
def test_rotation_and_norm(msa, near, rotary, norm, shift):
    s = Setup(msa, [5, 130], [0, 60000], rotary=rotary, near=near, norm=norm, shift=shift, given=True)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("h,hk", [(1, 1), (5, 1), (12, 3), (32, 8), (40, 2)])
@pytest.mark.parametrize("rows", [1, 609, 2433, 5000])
def test_heads_and_row_counts(msa, h, hk, rows):
    # every way of sharing a row among warps
    s = Setup(msa, [rows // 2, rows - rows // 2], [33, 260], h=h, hk=hk, hi=0, di=0, pad=8, kv=F8, scale=TOKEN)
    assert s.run() == 0
    s.check()


def test_a_kind_without_its_norm_and_zero_vectors(msa):
    s = Setup(msa, [20], [7], kv=F8, scale=TOKEN, idx_fp8=True)
    s.norms[0] = s.norms[3] = None
    s.proj[3] = 0
    assert s.run() == 0
    s.check()
    assert (s.q_out[3] == 0).all()
    assert (s.ks.view(-1)[s.slot[3]] == 1) and (s.vs.view(-1)[s.slot[3]] == 1) and (s.xs.view(-1)[s.slot[3]] == 1)


def test_in_place(msa):
    s = Setup(msa, [200, 1], [0, 300])
    q = s.q.contiguous()
    assert s.run(q=q, q_out=q) == 0
    s.q_out = q
    s.check()


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (F8, NONE), (F8, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("idx_fp8", [False, True])
def test_without_norm_and_rotation_it_is_kv_insert(msa, kv, scale, idx_fp8):
    s = Setup(msa, [1, 300, 9], [700, 100, 0], kv=kv, scale=scale, idx_fp8=idx_fp8, rotary=0, norm=False)
    t = Setup(msa, [1, 300, 9], [700, 100, 0], kv=kv, scale=scale, idx_fp8=idx_fp8, rotary=0, norm=False)
    assert s.run() == 0
    batch, _, _, pools = t.args()
    msa.msa_kv_insert(batch, t.k.contiguous(), t.v.contiguous(), 1, 128, t.pools[0], t.pools[1], kv, scale, t.ks, t.vs,
                      t.idx_k.contiguous(), pools._keep[4], False, t.status)
    torch.cuda.synchronize()
    for a, b in zip(s.pools, t.pools):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in ((s.ks, t.ks), (s.vs, t.vs), (s.xs, t.xs)):
        assert a is None or torch.equal(a, b)
    assert torch.equal(s.q_out, s.q)


def test_index_reuse_layers_and_mass(msa):
    s = Setup(msa, [3, 70], [127, 300])
    mass = torch.ones((s.w.num_pages, 128), device="cuda")
    assert s.run(index=False, mass=mass) == 0
    s.check(index=False)
    assert torch.equal(s.pools[2], s.before[2]) and torch.isnan(s.iq_out.float()).all()
    hit = torch.zeros(s.w.num_pages * 128, dtype=torch.bool)
    hit[torch.from_numpy(s.slot)] = True
    assert torch.equal(mass.view(-1).cpu() == 0, hit) and torch.equal(mass.view(-1).cpu() == 1, ~hit)


@pytest.mark.parametrize("n", [1, 30])
def test_bad_requests_and_positions(msa, n):
    q_lens, ctxs = [3 * n, 2 * n, 4, 5], [300, 2000, 500, 64]
    s = Setup(msa, q_lens, ctxs, given=True, top=5000)
    w = s.w
    w.block_table[1, 3] = w.num_pages       # not a page that the rows go to
    w.context_lens[2] += 1
    last = w.num_rows - 2
    s.given[last] = 5000
    s.given[last - 1] = -1
    mass = torch.ones((w.num_pages, 128), device="cuda")
    assert s.run(mass=mass) == 1 | 2 | 32
    rows = list(range(3 * n)) + [w.num_rows - 5, w.num_rows - 4, w.num_rows - 1]
    out = np.setdiff1d(np.arange(w.num_rows), rows)
    s.check(rows=rows)
    assert (s.q_out[out] == 0).all() and (s.iq_out[out] == 0).all()
    assert (mass.view(-1)[torch.from_numpy(s.slot[out]).cuda()] == 1).all()


def test_rows_that_no_request_owns(msa):
    s = Setup(msa, [3, 2], [100, 100])
    s.w.cu_seqlens_q[2] = 4
    assert s.run() == 4
    assert (s.q_out == 0).all() and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(s.pools, s.before))


def test_many_requests(msa):
    rng = np.random.default_rng(4)
    n = 1500
    s = Setup(msa, rng.integers(0, 4, n).tolist(), rng.integers(0, 300, n).tolist(), h=2)
    assert s.run() == 0
    s.check()


def test_values_that_are_not_finite_stay_in_their_vector(msa):
    s = Setup(msa, [6], [0], kv=F8, scale=TOKEN)
    s.proj[2, 5] = float("nan")            # in q's first head
    s.proj[4, 16 * 128 + 3] = float("inf")  # in k
    assert s.run() == 0
    assert torch.isnan(s.q_out[2, 0].float()).all() and torch.isfinite(s.q_out[2, 1:].float()).all()
    rows = [0, 1, 3, 5]
    want, tol = s.wanted(s.q, 0)
    err = np.abs(s.q_out.double().cpu().numpy() - want)
    assert (err <= tol + 2.0 ** -8 * np.abs(want))[rows].all()
    k, kt = s.wanted(s.k, 1)
    before = s.before[0].clone()
    flat = before.view(-1, 1, 128)
    for r in (2, 4):
        flat[s.slot[r]] = s.pools[0].view(-1, 1, 128)[s.slot[r]]
    s.check_pool(s.pools[0], before, True, k, kt, s.ks, TOKEN, rows)


def test_streams_and_graphs(msa):
    s = Setup(msa, [2, 33], [500, 0], kv=F8, scale=TOKEN)
    args = s.args()
    side = torch.cuda.Stream()
    msa.msa_qk_rope_insert(*args, s.status, stream=side)
    torch.cuda.synchronize()
    want = [t.clone() for t in (*s.pools, s.q_out, s.iq_out, s.ks, s.vs)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.msa_qk_rope_insert(*args, s.status)
    for t, b in zip(s.pools, s.before):
        t.copy_(b)
    s.q_out.zero_(), s.ks.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = [*s.pools, s.q_out, s.iq_out]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))

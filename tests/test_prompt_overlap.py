"""Outputs of the prompt operators that share memory with inputs or with each other are refused, before anything
is launched; those beside them are not."""
import ctypes

import numpy as np
import pytest
import torch

from tests import prompt_ref as P
from tests.test_gpu_rope_insert import Setup
from tests.test_prompt_abi import B, attn, batch, index, pools, ref  # noqa: F401

BASE, FAR = 0x100000, 0x900000  # never dereferenced: every call on them is refused
H, ROW = 16, (16 + 2 + 2) * 128  # heads of q; elements of a projection's row: q, k, v, idx_q, idx_k


def insert(B, **kw):
    at = lambda i: ctypes.c_void_p(BASE + 256 * i)
    d = dict(q=at(0), k=at(H), v=at(H + 1), idx_q=at(H + 2), idx_k=at(H + 3), q_stride=ROW, k_stride=ROW, v_stride=ROW,
             idx_q_stride=ROW, idx_k_stride=ROW, num_heads=H, num_kv_heads=1, head_dim=128, eps=1e-6,
             q_out=ctypes.c_void_p(FAR), idx_q_out=ctypes.c_void_p(FAR + 2 * H * 256 + 256))
    fake = ctypes.c_void_p(0x80000000)
    b = batch(B, cu_seqlens_q=fake, cu_seqlens_k=fake, context_lens=fake, block_table=fake)
    p = pools(B, index(B, k_cache=fake), k_cache=fake, v_cache=fake)
    r = B.msa_rope(cos_sin=None, max_pos=0, rotary_dim=0, interleaved=0, positions=None)
    return B.lib().msa_qk_rope_insert(ref(b), ref(B.msa_qkv(**{**d, **kw})), ref(r), ref(p), fake, None)


@pytest.mark.parametrize("at", [BASE + 16, BASE + 256 * (H - 1), BASE + 256 * H, BASE + 256 * (H + 3), BASE + 2 * ROW,
                                BASE + 4 * ROW - 16, BASE - 16, BASE - 2 * H * 256 + 16])
def test_insertion_onto_its_vectors(B, at):  # noqa: F811
    # (two rows: q_out reaches 8 KB, a projection 10)
    assert insert(B, q_out=ctypes.c_void_p(at)) == B.MSA_ERR_SHAPE
    if at >= BASE:
        assert insert(B, idx_q_out=ctypes.c_void_p(at)) == B.MSA_ERR_SHAPE


def test_insertion_in_anothers_place(B):  # noqa: F811
    packed = dict(q=ctypes.c_void_p(BASE), q_stride=H * 128, k=ctypes.c_void_p(FAR + 0x10000))
    # the index queries' output in q's place, or q's over a k behind it
    assert insert(B, **packed, idx_q_out=ctypes.c_void_p(BASE)) == B.MSA_ERR_SHAPE
    assert insert(B, q=ctypes.c_void_p(BASE), q_stride=H * 128, k=ctypes.c_void_p(BASE + 256 * H),
                  q_out=ctypes.c_void_p(BASE)) == B.MSA_ERR_SHAPE
    # the outputs over each other
    assert insert(B, idx_q_out=ctypes.c_void_p(FAR + 2 * H * 256 - 256)) == B.MSA_ERR_SHAPE
    assert insert(B, idx_q_out=ctypes.c_void_p(FAR)) == B.MSA_ERR_SHAPE


@pytest.mark.parametrize("where", ["out", "lse"])
@pytest.mark.parametrize("by", [16, 2 * 16 * 256 - 16, -16])
def test_attention_onto_its_queries(B, where, by):  # noqa: F811
    fake = lambda a: ctypes.c_void_p(a)
    d = dict(q=fake(BASE), out=fake(FAR), lse=fake(FAR + 0x10000))
    d[where] = fake(BASE + by)
    go = lambda d: B.lib().msa_prompt_attn(ref(batch(B)), ref(attn(B, **d)), fake(0x80000000), 1 << 40, fake(0x10000), None)
    if where == "lse" and by < 0:
        by = d["lse"] = fake(BASE - 2 * 16 * 4 + 16)
    assert go(d) == B.MSA_ERR_SHAPE
    assert go(dict(q=fake(BASE), out=fake(FAR), lse=fake(FAR + 16))) == B.MSA_ERR_SHAPE


def test_a_set_of_pages_over_what_it_comes_from(B):  # noqa: F811
    # 3 old requests of 8 blocks, 5 new ones of 6, 40 pages
    size = dict(lens=12, block_table=96, refs=160, parent=20, grow=20)
    made = dict(lens=20, block_table=120, refs=160, copy_src=20, copy_dst=20, copy_tokens=20)
    src = {k: BASE + 0x1000 * i for i, k in enumerate(size)}
    dst = {k: FAR + 0x1000 * i for i, k in enumerate(made)}

    def go(**kw):
        s, t = dict(src), dict(dst)
        t.update(kw)
        view = B.msa_cache_view(lens=s["lens"], block_table=s["block_table"], bt_stride=8, num_reqs=3, num_pages=40)
        to = B.msa_page_set(**t, bt_stride=6, num_reqs=5)
        at = ctypes.c_void_p
        return B.lib().msa_page_fork(ref(view), at(s["refs"]), at(s["parent"]), at(s["grow"]), ref(to), at(0x80000000), None)

    for a in made:
        for b in size:
            assert go(**{a: src[b] + (size[b] - 1) // 16 * 16}) == B.MSA_ERR_SHAPE, (a, b)
            assert go(**{a: src[b] - (made[a] - 1) // 16 * 16}) == B.MSA_ERR_SHAPE, (a, b)
        for b in made:
            if a != b:
                assert go(**{a: dst[b] + (made[b] - 1) // 16 * 16}) == B.MSA_ERR_SHAPE, (a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_outputs_between_and_beside_the_vectors(rows):
    """An output in what a projection's rows leave free is no overlap; nor is one that ends where they begin."""
    import block_sparse_paged_02_gb300 as msa
    s = Setup(msa, [rows], [100], h=4, hi=1, pad=4 * 128)
    n = s.w.num_rows
    width = s.proj.shape[1]
    buf = torch.zeros(n * 4 * 128 + n * width + n * 128, dtype=torch.bfloat16, device="cuda")
    proj = buf[n * 4 * 128:n * 4 * 128 + n * width].view(n, width)
    proj.copy_(s.proj)
    cut = lambda t: proj[:, t.storage_offset():t.storage_offset() + t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])
    s.q, s.k, s.v, s.idx_q, s.idx_k = (cut(t) for t in (s.q, s.k, s.v, s.idx_q, s.idx_k))
    s.q_out, s.iq_out = buf[:n * 4 * 128].view(n, 4, 128), buf[n * 4 * 128 + n * width:].view(n, 1, 128)
    if rows == 1:  # one row's output in the projection's own tail
        s.q_out = proj[:, -4 * 128:].unflatten(1, (4, 128))
    assert s.run() == 0
    s.check()


@pytest.mark.gpu
@pytest.mark.parametrize("kv,scale", [(0, 0), (1, 2)])
@pytest.mark.parametrize("q_lens,ctxs", [([200], [0]), ([300, 5, 1, 77], [9000, 0, 40, 3000])])
def test_attention_in_its_queries_place(kv, scale, q_lens, ctxs):
    import block_sparse_paged_02_gb300 as msa
    w = P.batch(6, q_lens, ctxs, 24, 4, kv, scale, True)
    c = msa.DeviceCase(w)
    c.prompt_attn()
    torch.cuda.synchronize()
    want, lse = c.out.clone(), c.lse.clone()
    c.out = c.q
    c._args()
    c.prompt_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and torch.equal(c.q, want) and torch.equal(c.lse, lse)
    P.check_attn(c, P.attn(w))

"""include/msa_cache.h: the library exports what it declares, the ctypes mirrors
follow it, and bad arguments are refused before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call here is refused
ODD = ctypes.c_void_p(0x10008)


def header():
    src = open(os.path.join(ROOT, "include", "msa_cache.h")).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


@pytest.fixture(scope="module")
def B():
    from block_sparse_paged_02_gb300 import binding
    binding.lib()
    return binding


def test_declared_symbols_are_exported(B):
    names = set(re.findall(r"\b(msa_[a-z0-9_]+)\s*\(", header()))
    assert names == {"msa_tree_attn_workspace_size", "msa_tree_attn", "msa_attn_mass", "msa_evict_select",
                     "msa_kv_compact"}
    for n in names:
        assert hasattr(B.lib(), n) and n in B.EXPORTED


def test_struct_layouts(B):
    found = re.findall(r"typedef struct (\w+) \{(.*?)\} \1;", header(), flags=re.S)
    assert {n for n, _ in found} == {"msa_tree", "msa_cache_view", "msa_kv_pools"}
    for name, body in found:
        fields = [" ".join(d.split()) for d in body.split(";") if d.strip()]
        py = getattr(B, name)._fields_
        assert [re.search(r"(\w+)$", f).group(1) for f in fields] == [f for f, _ in py]
        for f, (_, t) in zip(fields, py):
            assert t is (ctypes.c_void_p if "*" in f else ctypes.c_int32)


def batch(B, **kw):
    d = dict(cu_seqlens_q=FAKE, cu_seqlens_k=FAKE, context_lens=FAKE, block_table=FAKE, bt_stride=4, num_reqs=1,
             num_rows=2, num_pages=10, max_q_len=2, min_q_len=0)
    return B.msa_batch(**{**d, **kw})


def attn(B, **kw):
    d = dict(q=FAKE, num_rows=2, num_heads=16, num_kv_heads=1, head_dim=128, k_cache=FAKE, v_cache=FAKE, kv_dtype=0,
             num_pages=10, scale_mode=0, k_scale=None, v_scale=None, sinks=None, softmax_scale=0.1, out=FAKE, lse=FAKE)
    return B.msa_attn_args(**{**d, **kw})


def tree(B, **kw):
    return B.msa_tree(**{**dict(mask=None, mask_words=0, topk_idx=None, topk=0), **kw})


def call(B, b=None, t=None, a=None, ws=FAKE, n=1 << 40, st=FAKE, mass=None):
    ref = lambda x: None if x is None else ctypes.byref(x)
    if mass is None:
        return B.lib().msa_tree_attn(ref(b), ref(t), ref(a), ws, n, st, None)
    return B.lib().msa_attn_mass(ref(b), ref(t), ref(a), mass, ws, n, st, None)


@pytest.mark.parametrize("mass", [None, FAKE])
def test_tree_refusals(B, mass):
    go = lambda b=batch(B), t=tree(B), a=attn(B), **kw: call(B, b, t, a, mass=mass, **kw)
    NULL, SHAPE, DTYPE, UNSUP, WS = (B.MSA_ERR_NULL, B.MSA_ERR_SHAPE, B.MSA_ERR_DTYPE, B.MSA_ERR_UNSUPPORTED,
                                     B.MSA_ERR_WORKSPACE)
    assert go(b=None) == NULL and go(t=None) == NULL and go(a=None) == NULL and go(st=None) == NULL
    assert go(b=batch(B, block_table=None)) == NULL
    assert go(b=batch(B, bt_stride=0)) == SHAPE and go(b=batch(B, max_q_len=-1)) == SHAPE
    assert go(b=batch(B, max_q_len=257)) == UNSUP and go(b=batch(B, bt_stride=16385)) == UNSUP
    assert go(b=batch(B, num_reqs=4097)) == UNSUP
    assert go(b=batch(B, num_rows=3)) == SHAPE and go(b=batch(B, num_pages=9)) == SHAPE
    assert go(b=batch(B, num_reqs=0)) == SHAPE
    assert go(a=attn(B, kv_dtype=3)) == DTYPE and go(a=attn(B, scale_mode=9)) == DTYPE
    assert go(a=attn(B, num_heads=17)) == UNSUP and go(a=attn(B, head_dim=64)) == UNSUP
    assert go(a=attn(B, num_kv_heads=2)) == UNSUP and go(a=attn(B, num_kv_heads=3)) == SHAPE
    assert go(a=attn(B, q=None)) == NULL and go(a=attn(B, lse=None)) == NULL
    assert go(a=attn(B, k_cache=ODD)) == SHAPE and go(a=attn(B, q=ODD)) == SHAPE
    assert go(a=attn(B, scale_mode=1)) == NULL
    assert go(a=attn(B, scale_mode=2, k_scale=ODD, v_scale=ODD)) == SHAPE
    assert go(t=tree(B, mask=FAKE)) == SHAPE and go(t=tree(B, mask=ODD, mask_words=1)) == SHAPE
    assert go(t=tree(B, topk_idx=FAKE)) == SHAPE and go(t=tree(B, topk_idx=FAKE, topk=2049)) == UNSUP
    assert go(ws=None) == WS and go(n=1000) == WS and go(ws=ODD) == WS
    # a size for a narrower tree does not do for a wider one
    small = B.msa_tree_attn_workspace_size(1, 2, 4, 1, 1, 0)
    assert go(n=small) == WS
    if mass is None:
        assert go(a=attn(B, v_cache=None)) == NULL and go(a=attn(B, out=None)) == NULL
        assert go(a=attn(B, out=ODD)) == SHAPE and go(a=attn(B, scale_mode=1, k_scale=FAKE)) == NULL
    else:
        assert call(B, batch(B), tree(B), attn(B), mass=ODD) == SHAPE
        assert B.lib().msa_attn_mass(ctypes.byref(batch(B)), ctypes.byref(tree(B)), ctypes.byref(attn(B)), None, FAKE,
                                     1 << 40, FAKE, None) == NULL
    # nothing to do
    assert go(b=batch(B, num_rows=0), a=attn(B, num_rows=0)) == B.MSA_OK


def test_workspace_sizes(B):
    size = B.msa_tree_attn_workspace_size
    assert 0 < size(1, 1, 8, 8) <= size(1, 64, 8, 16, 64) < size(4, 64, 256, 16, 64, 16)
    assert size(-1, 1, 8, 8) == 0 and size(1, 1, 0, 8) == 0 and size(1, 1, 8, 17) == 0
    assert size(1, 1, 8, 8, 257) == 0 and size(1, 1, 8, 8, 1, 2049) == 0


def test_evict_and_compact_refusals(B):
    L = B.lib()
    NULL, SHAPE, DTYPE, UNSUP = B.MSA_ERR_NULL, B.MSA_ERR_SHAPE, B.MSA_ERR_DTYPE, B.MSA_ERR_UNSUPPORTED
    view = lambda **kw: B.msa_cache_view(**{**dict(lens=FAKE, block_table=FAKE, bt_stride=4, num_reqs=2, num_pages=9), **kw})

    def ev(c=view(), mass=FAKE, budget=8, first=1, recent=1, keep=FAKE, kl=FAKE, st=FAKE):
        return L.msa_evict_select(None if c is None else ctypes.byref(c), mass, budget, first, recent, keep, kl, st, None)
    assert ev(c=None) == NULL and ev(st=None) == NULL and ev(mass=None) == NULL and ev(keep=None) == NULL
    assert ev(kl=None) == NULL and ev(c=view(lens=None)) == NULL and ev(keep=ODD) == SHAPE
    assert ev(budget=0) == SHAPE and ev(first=-1) == SHAPE and ev(recent=-1) == SHAPE and ev(first=5, recent=4) == SHAPE
    assert ev(first=2 ** 31 - 1, recent=2 ** 31 - 1) == SHAPE
    assert ev(c=view(bt_stride=0)) == SHAPE and ev(c=view(bt_stride=16385)) == UNSUP and ev(c=view(num_reqs=4097)) == UNSUP
    assert ev(c=view(num_reqs=0)) == B.MSA_OK
    idx = lambda **kw: B.msa_index_cache(**{**dict(k_cache=FAKE, k_scale=None, dtype=0, heads=1, dim=128), **kw})

    def cp(c=view(), base=None, keep=FAKE, stride=8, kl=FAKE, st=FAKE, index=None, null=False, **kw):
        d = dict(k_cache=FAKE, v_cache=FAKE, kv_dtype=0, num_kv_heads=1, head_dim=128, scale_mode=0, k_scale=None,
                 v_scale=None, index=None, mass=None)
        d.update(kw)
        p = B.msa_kv_pools(**d)
        if index is not None:
            p.index = ctypes.cast(ctypes.pointer(index), ctypes.c_void_p)
        return L.msa_kv_compact(None if c is None else ctypes.byref(c), base, keep, stride, kl,
                                None if null else ctypes.byref(p), st, None)
    assert cp(c=None) == NULL and cp(null=True) == NULL and cp(st=None) == NULL and cp(keep=None) == NULL and cp(kl=None) == NULL
    assert cp(k_cache=None) == NULL and cp(v_cache=None) == NULL and cp(scale_mode=2) == NULL
    assert cp(index=idx(k_cache=None)) == NULL
    assert cp(kv_dtype=2) == DTYPE and cp(scale_mode=3) == DTYPE and cp(index=idx(dtype=4)) == DTYPE
    assert cp(stride=0) == SHAPE and cp(num_kv_heads=0) == SHAPE and cp(k_cache=ODD) == SHAPE and cp(mass=ODD) == SHAPE
    assert cp(scale_mode=2, k_scale=ODD, v_scale=FAKE) == SHAPE and cp(index=idx(k_cache=ODD)) == SHAPE
    assert cp(head_dim=64) == UNSUP and cp(num_kv_heads=65) == UNSUP and cp(index=idx(heads=3)) == UNSUP
    assert cp(c=view(num_reqs=0)) == B.MSA_OK


def test_binding_refusals(B):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="int32"):
        B.make_tree(mask=torch.zeros((2, 1), dtype=torch.int64))
    with pytest.raises(ValueError, match="shape"):
        B.make_tree(topk_idx=i32(4))
    with pytest.raises(ValueError, match="device tensors"):
        B.make_tree(mask=i32(2, 1))
    with pytest.raises(ValueError, match="int32"):
        B.make_cache_view(torch.zeros(2), i32(2, 4), 9)
    with pytest.raises(ValueError, match="shape"):
        B.make_cache_view(i32(2), i32(3, 4), 9)
    k = torch.zeros((2, 128, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache"):
        B.make_kv_pools(k, k, B.MSA_KV_FP8_E4M3)
    with pytest.raises(ValueError, match="v_cache"):
        B.make_kv_pools(k, k[:1], B.MSA_KV_BF16)
    with pytest.raises(ValueError, match="mass"):
        B.make_kv_pools(k, k, B.MSA_KV_BF16, mass=torch.zeros((2, 64)))
    view = B.msa_cache_view(None, None, 4, 2, 9)
    with pytest.raises(ValueError, match="mass"):
        B.msa_evict_select(view, torch.zeros((8, 128)), 8, 0, 0, i32(2, 8), i32(2), i32(1))
    with pytest.raises(ValueError, match="keep"):
        B.msa_evict_select(view, torch.zeros((9, 128)), 8, 0, 0, i32(2, 7), i32(2), i32(1))
    t = B.msa_tree(None, 0, None, 0)
    t._keep = (i32(3, 1), None)
    with pytest.raises(ValueError, match="rows"):
        B.msa_tree_attn(B.msa_batch(None, None, None, None, 4, 1, 2, 9, 2, 0), t, B.msa_attn_args(), None, i32(1))

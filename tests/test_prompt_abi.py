"""include/msa_prompt.h: the library exports what it declares, the ctypes mirrors follow it, and
bad arguments are refused before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call here is refused
ODD = ctypes.c_void_p(0x10008)
ELSE = ctypes.c_void_p(0x20000)


def header():
    src = open(os.path.join(ROOT, "include", "msa_prompt.h")).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


@pytest.fixture(scope="module")
def B():
    from block_sparse_paged_02_gb300 import binding
    binding.lib()
    return binding


def test_declared_symbols_are_exported(B):
    names = set(re.findall(r"\b(msa_[a-z0-9_]+)\s*\(", header()))
    assert names == {"msa_qk_rope_insert", "msa_prompt_attn_workspace_size", "msa_prompt_attn", "msa_page_fork",
                     "msa_page_copy"}
    for n in names:
        assert hasattr(B.lib(), n) and n in B.EXPORTED


def test_struct_layouts(B):
    found = re.findall(r"typedef struct (\w+) \{(.*?)\} \1;", header(), flags=re.S)
    assert {n for n, _ in found} == {"msa_rope", "msa_qkv", "msa_page_set"}
    for name, body in found:
        fields = [" ".join(d.split()) for d in body.split(";") if d.strip()]
        py = getattr(B, name)._fields_
        assert [re.search(r"(\w+)$", f).group(1) for f in fields] == [f for f, _ in py]
        for f, (_, t) in zip(fields, py):
            want = ctypes.c_void_p if "*" in f else {"int64_t": ctypes.c_int64, "float": ctypes.c_float,
                                                     "int32_t": ctypes.c_int32}[f.split()[0]]
            assert t is want, (name, f)


def test_status_bits(B):
    src = open(os.path.join(ROOT, "include", "msa_prompt.h")).read()
    for name in ("MSA_DEV_BAD_POS", "MSA_DEV_NO_PAGES"):
        assert int(re.search(rf"#define {name} (\d+)u", src).group(1)) == getattr(B, name)


def batch(B, **kw):
    d = dict(cu_seqlens_q=FAKE, cu_seqlens_k=FAKE, context_lens=FAKE, block_table=FAKE, bt_stride=4, num_reqs=1,
             num_rows=2, num_pages=10, max_q_len=2, min_q_len=0)
    return B.msa_batch(**{**d, **kw})


def attn(B, **kw):
    d = dict(q=FAKE, num_rows=2, num_heads=16, num_kv_heads=1, head_dim=128, k_cache=FAKE, v_cache=FAKE, kv_dtype=0,
             num_pages=10, scale_mode=0, k_scale=None, v_scale=None, sinks=None, softmax_scale=0.1, out=FAKE, lse=FAKE)
    return B.msa_attn_args(**{**d, **kw})


def index(B, **kw):
    return B.msa_index_cache(**{**dict(k_cache=FAKE, k_scale=None, dtype=0, heads=1, dim=128), **kw})


def pools(B, idx=None, **kw):
    d = dict(k_cache=FAKE, v_cache=FAKE, kv_dtype=0, num_kv_heads=1, head_dim=128, scale_mode=0, k_scale=None,
             v_scale=None, index=None, mass=None)
    p = B.msa_kv_pools(**{**d, **kw})
    if idx is not None:
        p.index = ctypes.cast(ctypes.pointer(idx), ctypes.c_void_p)
        p._keep = idx
    return p


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_prompt_attn_refusals(B):
    def go(b=batch(B), a=attn(B), ws=FAKE, n=1 << 40, st=FAKE):
        return B.lib().msa_prompt_attn(ref(b), ref(a), ws, n, st, None)
    NULL, SHAPE, DTYPE, UNSUP, WS = (B.MSA_ERR_NULL, B.MSA_ERR_SHAPE, B.MSA_ERR_DTYPE, B.MSA_ERR_UNSUPPORTED,
                                     B.MSA_ERR_WORKSPACE)
    assert go(b=None) == NULL and go(a=None) == NULL and go(st=None) == NULL
    for f in ("cu_seqlens_q", "cu_seqlens_k", "context_lens", "block_table"):
        assert go(b=batch(B, **{f: None})) == NULL
    for f in ("q", "k_cache", "v_cache", "out", "lse"):
        assert go(a=attn(B, **{f: None})) == NULL and go(a=attn(B, **{f: ODD})) == SHAPE
    assert go(b=batch(B, bt_stride=0)) == SHAPE and go(b=batch(B, num_reqs=-1)) == SHAPE
    assert go(b=batch(B, bt_stride=16385)) == UNSUP and go(b=batch(B, num_reqs=4097)) == UNSUP
    assert go(b=batch(B, num_rows=3)) == SHAPE and go(b=batch(B, num_pages=9)) == SHAPE
    assert go(b=batch(B, num_reqs=0)) == SHAPE
    assert go(b=batch(B, num_pages=1 << 24), a=attn(B, num_pages=1 << 24)) == UNSUP
    assert go(a=attn(B, kv_dtype=3)) == DTYPE and go(a=attn(B, scale_mode=9)) == DTYPE
    assert go(a=attn(B, num_heads=129)) == UNSUP and go(a=attn(B, head_dim=64)) == UNSUP
    assert go(a=attn(B, num_heads=65, num_kv_heads=65)) == UNSUP
    assert go(a=attn(B, num_kv_heads=3)) == SHAPE and go(a=attn(B, num_heads=0)) == SHAPE
    assert go(a=attn(B, scale_mode=1)) == NULL and go(a=attn(B, scale_mode=1, k_scale=FAKE)) == NULL
    assert go(a=attn(B, scale_mode=2, k_scale=ODD, v_scale=FAKE)) == SHAPE
    assert go(ws=None) == WS and go(n=1000) == WS and go(ws=ODD) == WS
    assert go(n=B.msa_prompt_attn_workspace_size(16, 1) - 1) == WS
    assert go(b=batch(B, num_rows=0), a=attn(B, num_rows=0)) == B.MSA_OK


def test_prompt_workspace_sizes(B):
    size = B.msa_prompt_attn_workspace_size
    assert size(16, 1) > 0 and size(128, 1) > 0 and size(64, 64) > 0
    assert size(129, 1) == size(16, 3) == size(0, 1) == size(16, 0) == size(65, 65) == 0


def test_insert_refusals(B):
    def qkv(**kw):
        d = dict(q=FAKE, k=FAKE, v=FAKE, idx_q=FAKE, idx_k=FAKE, q_stride=2048, k_stride=128, v_stride=128,
                 idx_q_stride=128, idx_k_stride=128, num_heads=16, num_kv_heads=1, head_dim=128, q_norm=None, k_norm=None,
                 idx_q_norm=None, idx_k_norm=None, eps=1e-6, norm_shift=0.0, q_out=ELSE, idx_q_out=ELSE)
        return B.msa_qkv(**{**d, **kw})

    def rope(**kw):
        return B.msa_rope(**{**dict(cos_sin=FAKE, max_pos=64, rotary_dim=64, interleaved=0, positions=None), **kw})

    def go(b=batch(B), x=qkv(), r=rope(), p=pools(B, index(B)), st=FAKE):
        return B.lib().msa_qk_rope_insert(ref(b), ref(x), ref(r), ref(p), st, None)
    NULL, SHAPE, DTYPE, UNSUP = B.MSA_ERR_NULL, B.MSA_ERR_SHAPE, B.MSA_ERR_DTYPE, B.MSA_ERR_UNSUPPORTED
    assert go(b=None) == NULL and go(x=None) == NULL and go(r=None) == NULL and go(p=None) == NULL and go(st=None) == NULL
    for f in ("q", "k", "v", "idx_q", "idx_k", "q_out", "idx_q_out"):
        assert go(x=qkv(**{f: None})) == NULL and go(x=qkv(**{f: ODD})) == SHAPE
    for f in ("q_norm", "k_norm", "idx_q_norm", "idx_k_norm"):
        assert go(x=qkv(**{f: ODD})) == SHAPE
    for f, small in (("q_stride", 2040), ("k_stride", 120), ("v_stride", 0), ("idx_q_stride", -128), ("idx_k_stride", 64)):
        assert go(x=qkv(**{f: small})) == SHAPE and go(x=qkv(**{f: 4100})) == SHAPE
    assert go(x=qkv(num_heads=0)) == SHAPE and go(x=qkv(num_kv_heads=2)) == SHAPE and go(x=qkv(head_dim=64)) == SHAPE
    assert go(x=qkv(num_heads=1025, q_stride=1025 * 128)) == UNSUP
    assert go(r=rope(rotary_dim=-16)) == SHAPE and go(r=rope(max_pos=-1)) == SHAPE
    assert go(r=rope(rotary_dim=24)) == UNSUP and go(r=rope(rotary_dim=144)) == UNSUP
    assert go(r=rope(rotary_dim=128), p=pools(B, index(B, dim=64))) == UNSUP
    assert go(r=rope(cos_sin=None)) == NULL and go(r=rope(cos_sin=ODD)) == SHAPE and go(r=rope(positions=ODD)) == SHAPE
    assert go(p=pools(B, index(B), k_cache=None)) == NULL and go(p=pools(B, index(B), v_cache=ODD)) == SHAPE
    assert go(p=pools(B, index(B), kv_dtype=2)) == DTYPE and go(p=pools(B, index(B), scale_mode=3)) == DTYPE
    assert go(p=pools(B, index(B), kv_dtype=1, scale_mode=1)) == NULL
    assert go(p=pools(B, index(B), scale_mode=2)) == NULL and go(p=pools(B, index(B), mass=ODD)) == SHAPE
    assert go(p=pools(B, index(B, heads=3))) == UNSUP and go(p=pools(B, index(B, dtype=5))) == DTYPE
    assert go(p=pools(B, index(B, k_cache=None))) == NULL and go(p=pools(B, index(B, k_scale=ODD))) == SHAPE
    assert go(b=batch(B, num_reqs=0)) == SHAPE and go(b=batch(B, num_reqs=4097)) == UNSUP
    # in place: packed rows alone
    assert go(x=qkv(q_out=FAKE, q_stride=2056)) == SHAPE and go(x=qkv(idx_q_out=FAKE, idx_q_stride=136)) == SHAPE
    assert go(b=batch(B, num_rows=0)) == B.MSA_OK


def test_page_refusals(B):
    view = lambda **kw: B.msa_cache_view(**{**dict(lens=FAKE, block_table=FAKE, bt_stride=4, num_reqs=2, num_pages=9), **kw})

    def to(**kw):
        d = dict(lens=ELSE, block_table=ELSE, refs=ELSE, copy_src=ELSE, copy_dst=ELSE, copy_tokens=ELSE, bt_stride=4,
                 num_reqs=2)
        return B.msa_page_set(**{**d, **kw})

    def fork(c=view(), refs=FAKE, parent=FAKE, grow=FAKE, t=to(), st=FAKE):
        return B.lib().msa_page_fork(ref(c), refs, parent, grow, ref(t), st, None)
    NULL, SHAPE, UNSUP = B.MSA_ERR_NULL, B.MSA_ERR_SHAPE, B.MSA_ERR_UNSUPPORTED
    assert fork(c=None) == NULL and fork(t=None) == NULL and fork(st=None) == NULL and fork(refs=None) == NULL
    assert fork(parent=None) == NULL and fork(c=view(lens=None)) == NULL and fork(c=view(block_table=None)) == NULL
    for f in ("lens", "block_table", "refs", "copy_src", "copy_dst", "copy_tokens"):
        assert fork(t=to(**{f: None})) == NULL and fork(t=to(**{f: ODD})) == SHAPE
    assert fork(refs=ODD) == SHAPE and fork(parent=ODD) == SHAPE and fork(grow=ODD) == SHAPE
    assert fork(refs=ELSE) == SHAPE and fork(c=view(lens=ELSE)) == SHAPE and fork(c=view(block_table=ELSE)) == SHAPE
    assert fork(c=view(bt_stride=0)) == SHAPE and fork(c=view(num_pages=-1)) == SHAPE and fork(t=to(num_reqs=-1)) == SHAPE
    assert fork(t=to(bt_stride=0)) == SHAPE
    assert fork(c=view(num_reqs=4097)) == UNSUP and fork(t=to(num_reqs=4097)) == UNSUP
    assert fork(c=view(bt_stride=16385)) == UNSUP and fork(t=to(bt_stride=16385)) == UNSUP

    def copy(p=pools(B, index(B)), layers=1, pages=9, src=FAKE, dst=FAKE, tok=FAKE, n=3, st=FAKE):
        return B.lib().msa_page_copy(ref(p), layers, pages, src, dst, tok, n, st, None)
    assert copy(p=None) == NULL and copy(src=None) == NULL and copy(dst=None) == NULL and copy(tok=None) == NULL
    assert copy(st=None) == NULL and copy(src=ODD) == SHAPE and copy(layers=-1) == SHAPE and copy(n=-1) == SHAPE
    assert copy(pages=-1) == SHAPE and copy(n=(1 << 22) + 1) == UNSUP
    assert copy(p=pools(B, kv_dtype=4)) == B.MSA_ERR_DTYPE and copy(p=pools(B, num_kv_heads=65)) == UNSUP
    assert copy(p=pools(B, num_kv_heads=0)) == SHAPE and copy(p=pools(B, k_cache=None)) == NULL
    assert copy(p=pools(B, scale_mode=2)) == NULL and copy(p=pools(B, mass=ODD)) == SHAPE
    assert copy(p=pools(B, index(B, heads=2, dim=128))) == UNSUP
    assert copy(n=0) == B.MSA_OK and copy(p=None, layers=0) == B.MSA_OK


def test_binding_refusals(B, monkeypatch):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="float32"):
        B.make_rope(bf(8, 64))
    with pytest.raises(ValueError, match="int32"):
        B.make_rope(None, positions=torch.zeros(4))
    with pytest.raises(ValueError, match="device tensors"):
        B.make_rope(torch.zeros((8, 64)))
    with pytest.raises(ValueError, match="rows"):
        B.make_qkv(bf(3, 8, 128), bf(2, 1, 128), bf(2, 1, 128), bf(3, 8, 128))
    with pytest.raises(ValueError, match="device tensors"):
        B.make_qkv(bf(3, 8, 128), bf(3, 1, 128), bf(3, 1, 128), bf(3, 8, 128))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    good = dict(q=bf(3, 8, 128), k=bf(3, 1, 128), v=bf(3, 1, 128), q_out=bf(3, 8, 128))
    for name, t in (("k", bf(3, 1, 64)), ("v", bf(3, 2, 128)), ("q_out", bf(3, 8, 64)), ("q", torch.zeros((3, 8, 128))),
                    ("q_norm", bf(64)), ("k_norm", torch.ones(128))):
        with pytest.raises(ValueError, match=name):
            B.make_qkv(**{**good, name: t})
    with pytest.raises(ValueError, match="packed"):
        B.make_qkv(**{**good, "q": bf(3, 128, 8).transpose(1, 2)})
    wide = bf(3, 10, 128)
    with pytest.raises(ValueError, match="packed rows"):
        B.make_qkv(**{**good, "q": wide[:, :8], "q_out": wide.view(-1)[:3 * 8 * 128].view(3, 8, 128)})
    with pytest.raises(ValueError, match="together"):
        B.make_qkv(**good, idx_q=bf(3, 1, 128))
    with pytest.raises(ValueError, match="idx_k"):
        B.make_qkv(**good, idx_q=bf(3, 1, 128), idx_k=bf(3, 1, 64), idx_q_out=bf(3, 1, 128))
    x = B.make_qkv(**{**good, "q": wide[:, 1:9]})
    assert x.q_stride == 1280 and x.k_stride == 128 and x.q == wide.data_ptr() + 256
    b = batch(B, num_rows=4)
    kv = bf(10, 128, 1, 128)
    p = B.make_kv_pools(kv, kv, B.MSA_KV_BF16)
    r = B.make_rope(None)
    go = lambda b, x, r, p: B.msa_qk_rope_insert(b, x, r, p, i32(1))
    with pytest.raises(ValueError, match="rows"):
        go(b, x, r, p)
    b = batch(B, num_rows=3)
    with pytest.raises(ValueError, match="positions"):
        go(b, x, B.make_rope(None, positions=i32(4)), p)
    with pytest.raises(ValueError, match="pages"):
        go(b, x, r, B.make_kv_pools(kv[:9], kv[:9], B.MSA_KV_BF16))
    with pytest.raises(ValueError, match="index"):
        go(b, x, r, B.make_kv_pools(kv, kv, B.MSA_KV_BF16, index=B.make_index_cache(kv)))
    with pytest.raises(ValueError, match="k_scale"):
        go(b, x, r, B.make_kv_pools(kv, kv, B.MSA_KV_BF16, scale_mode=B.MSA_SCALE_SCALAR, k_scale=bf(1), v_scale=bf(1)))
    with pytest.raises(ValueError, match="copy_dst"):
        B.make_page_set(i32(2), i32(2, 4), i32(9), i32(2), i32(3), i32(2))
    to = B.make_page_set(i32(2), i32(2, 4), i32(9), i32(2), i32(2), i32(2))
    view = B.make_cache_view(i32(3), i32(3, 4), 9)
    for name, args in (("refs", (i32(8), i32(2), None)), ("parent", (i32(9), i32(3), None)), ("grow", (i32(9), i32(2), i32(1)))):
        with pytest.raises(ValueError, match=name):
            B.msa_page_fork(view, *args, to, i32(1))
    with pytest.raises(ValueError, match="pages"):
        B.msa_page_fork(B.make_cache_view(i32(3), i32(3, 4), 8), i32(8), i32(2), None, to, i32(1))
    with pytest.raises(ValueError, match="pages"):
        B.msa_page_copy([p, B.make_kv_pools(kv[:9], kv[:9], B.MSA_KV_BF16)], i32(1), i32(1), i32(1), i32(1))
    with pytest.raises(ValueError, match="tokens"):
        B.msa_page_copy([p], i32(1), i32(1), i32(2), i32(1))

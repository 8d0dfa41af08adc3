"""The prompt operators with pages whose offsets pass 32 bits, and with block tables of other widths.
Results go by the pages' contents alone, so they are compared bit by bit with those of a small pool."""
import dataclasses

import numpy as np
import pytest
import torch

import workloads as W
from tests import prompt_ref as P
from tests.test_gpu_rope_insert import Setup

pytestmark = pytest.mark.gpu

BF, F8 = W.KV_BF16, W.KV_FP8
NONE, SCALAR, TOKEN = W.SCALE_NONE, W.SCALE_SCALAR, W.SCALE_PER_TOKEN_HEAD
KINDS = [(BF, NONE, 131_080), (F8, TOKEN, 262_150)]  # pages before the small pool's: 2^32 bytes of it


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


def far(t, base):
    """t's pages at the end of a pool with `base` pages before them (of unknown contents)."""
    if t is None:
        return None
    x = torch.empty((base + t.shape[0], *t.shape[1:]), dtype=t.dtype, device="cuda")
    x[base:] = t
    return x


@pytest.mark.parametrize("kv,scale,base", KINDS)
def test_attention_over_far_pages(msa, kv, scale, base):
    w = P.batch(50, [130, 5, 300], [300, 2500, 0], 16, 1, kv, scale, True)
    c = msa.DeviceCase(w)
    c.prompt_attn()
    geo = [torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in (w.cu_seqlens_q, w.cu_seqlens_k, w.context_lens)]
    table = torch.from_numpy(w.block_table.astype(np.int32) + base).cuda()
    batch = msa.make_batch(*geo, table, base + w.num_pages, w.num_rows)
    bits = lambda a: (torch.from_numpy(a.copy()) if a.dtype == np.uint8
                      else torch.from_numpy(a.view(np.int16).copy()).view(torch.bfloat16)).cuda()
    dev = lambda a: None if a is None else torch.from_numpy(a.copy()).cuda()
    k, v, ks, vs = far(bits(w.k_cache), base), far(bits(w.v_cache), base), far(dev(w.k_scale), base), far(dev(w.v_scale), base)
    out, lse = torch.full_like(c.out, float("nan")), torch.full_like(c.lse, float("nan"))
    kind = msa.MSA_KV_BF16 if kv == BF else msa.MSA_KV_FP8_E4M3
    attn = msa.make_attn_args(bits(w.q), k, v, kind, base + w.num_pages, out, lse, scale_mode=scale, k_scale=ks, v_scale=vs,
                              sinks=dev(w.sinks), softmax_scale=w.softmax_scale)
    ws = torch.empty(msa.msa_prompt_attn_workspace_size(16, 1), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_prompt_attn(batch, attn, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and int(c.status.item()) == 0
    assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("kv,scale,base", KINDS)
def test_insertion_into_far_pages(msa, kv, scale, base):
    near, there = (Setup(msa, [5, 1, 70], [130, 0, 60], kv=kv, scale=scale, idx_fp8=kv == F8) for _ in range(2))
    assert near.run() == 0
    there.w = dataclasses.replace(there.w, block_table=there.w.block_table + base, num_pages=base + there.w.num_pages)
    there.pools = [far(t, base) for t in there.pools]
    there.ks, there.vs, there.xs = far(there.ks, base), far(there.vs, base), far(there.xs, base)
    assert there.run() == 0
    raw = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32 if t.dtype == torch.float32 else t.dtype)
    for a, b in zip(near.pools + [near.ks, near.vs, near.xs], there.pools + [there.ks, there.vs, there.xs]):
        assert a is b is None or torch.equal(raw(a), raw(b)[base:])
    assert torch.equal(near.q_out, there.q_out) and torch.equal(near.iq_out, there.iq_out)


def test_copies_between_far_pages(msa):
    base, n = 131_080, 6
    data = [torch.randn((n, 128, 1, 128), device="cuda").to(torch.bfloat16) for _ in range(2)]
    mass = torch.rand((n, 128), device="cuda")
    k, v, m = far(data[0], base), far(data[1], base), far(mass, base)
    low = [x[:2].clone() for x in (k, v, m)]
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_page_copy([msa.make_kv_pools(k, v, msa.MSA_KV_BF16, mass=m)], ints([base + 1, base + 4, base + 2]),
                      ints([base, base + 5, 1]), ints([128, 77, 3]), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    raw = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
    for x, small, before in zip((k, v, m), (*data, mass), low):
        want = small.clone()
        want[0], want[5, :77], before[1, :3] = small[1], small[4, :77], small[2, :3]
        assert torch.equal(raw(x)[base:], raw(want)) and torch.equal(raw(x[:2].clone()), raw(before))


@pytest.mark.parametrize("kv,scale", [(BF, NONE), (BF, TOKEN), (F8, SCALAR), (F8, TOKEN)])
@pytest.mark.parametrize("q_lens,ctxs", [([200], [0]), ([64], [1900]), ([300, 40, 513], [0, 700, 120])])
@pytest.mark.parametrize("stride", [0, 24, 700])
def test_tables_wider_than_the_requests(msa, kv, scale, q_lens, ctxs, stride):
    # (the width decides whether pairs of tiles are shared by CTAs; what lies behind a request's
    # blocks is no page)
    w = P.batch(51, q_lens, ctxs, 16, 1, kv, scale, True)
    if stride:
        wide = np.full((w.block_table.shape[0], stride), 2 ** 30, w.block_table.dtype)
        wide[:, :w.block_table.shape[1]] = w.block_table
        w = dataclasses.replace(w, block_table=wide)
    c = msa.DeviceCase(w)
    c.out.fill_(float("nan")), c.lse.fill_(float("nan"))
    c.prompt_attn()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    P.check_attn(c, P.attn(w))

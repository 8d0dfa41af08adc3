"""cu_seqlens_q whose entries fall, far enough apart that the differences in 32 bits pass as lengths: no entry
point takes it for a batch."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import prompt_ref as P

pytestmark = pytest.mark.gpu

# entries behind the first, of four rows
FAR = [[2 ** 31 - 1, -2, 4], [2 ** 31 - 10, 5 - 2 ** 31, 4], [-1, 3, 4], [9, 2, 4]]


def lengths(cu):
    return [int(d) for d in np.diff(np.array([0] + cu, np.int64)).astype(np.int32)]


def test_the_differences_pass_as_lengths():
    assert all(d >= 0 for cu in FAR[:2] for d in lengths(cu))


@pytest.fixture(params=FAR, ids=str)
def case(request):
    from block_sparse_paged_02_gb300 import DeviceCase
    cu = request.param
    w = P.batch(3, [1, 1, 2], [300, 200, 100], 16, 1)
    w.cu_seqlens_q[1:] = cu
    # lengths of K that go with those of Q where these are small
    lens = [100 + min(max(d, 0), 20) for d in lengths(cu)]
    w.context_lens[:] = [100] * 3
    w.cu_seqlens_k[:] = np.concatenate([[0], np.cumsum(lens)])
    c = DeviceCase(w, min_q_len_hint=False)
    c.out.fill_(3.0), c.lse.fill_(3.0)
    c.max_q_len = 2
    c._args()
    return c


def end(c):
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4


def empty(c):
    end(c)
    assert (c.out.float() == 0).all() and torch.isneginf(c.lse).all()


def test_prompt_attention(case):
    case.prompt_attn()
    empty(case)


def test_tree_attention_and_weights(case):
    case.tree_attn()
    empty(case)
    mass = torch.full((case.w.num_pages, 128), 5.0, device="cuda")
    case.attn_mass(mass)
    end(case)
    assert (mass == 5).all()


@pytest.mark.parametrize("rows", [2, 64])
def test_decode_and_scores(case, rows):
    case.max_q_len = rows   # (64: the scores' kernel on the tensor cores takes part)
    case._args()
    case.decode()
    empty(case)


def test_insertions(case):
    import block_sparse_paged_02_gb300 as msa
    c, pools = case, (case.k.clone(), case.v.clone(), case.idx_k.clone())
    rows = lambda h: torch.ones((4, h, 128), dtype=torch.bfloat16, device="cuda")
    q, iq = rows(16) * 7, rows(1) * 7
    qkv = msa.make_qkv(rows(16), rows(1), rows(1), q, idx_q=rows(1), idx_k=rows(1), idx_q_out=iq)
    c.qk_rope_insert(qkv, msa.make_rope(None))
    end(c)
    assert (q == 0).all() and (iq == 0).all()
    msa.msa_kv_insert(c.batch, rows(1), rows(1), 1, 128, c.k, c.v, W.KV_BF16, W.SCALE_NONE, None, None, rows(1), c.index,
                      False, c.status)
    end(c)
    raw = lambda t: t.view(torch.int16)
    assert all(torch.equal(raw(a), raw(b)) for a, b in zip(pools, (c.k, c.v, c.idx_k)))

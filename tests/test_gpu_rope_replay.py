"""A replayed insertion writes everything again: pools, scales, the queries and index queries handed on, the mass."""
import pytest
import torch

import workloads as W
from tests.test_gpu_rope_insert import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("kv,scale,idx_fp8", [(W.KV_FP8, W.SCALE_PER_TOKEN_HEAD, True), (W.KV_BF16, W.SCALE_NONE, False)])
@pytest.mark.parametrize("q_lens,ctxs", [([2, 33], [500, 0]), ([700, 1], [0, 90]), ([3000], [200])])
def test_replay_writes_every_output(msa, kv, scale, idx_fp8, q_lens, ctxs):
    s = Setup(msa, q_lens, ctxs, kv=kv, scale=scale, idx_fp8=idx_fp8)
    mass = torch.full((s.w.num_pages, 128), 3.0, device="cuda")
    written = [t for t in (*s.pools, s.q_out, s.iq_out, s.ks, s.vs, s.xs, mass) if t is not None]
    assert len(written) == (9 if idx_fp8 else 6)
    start = [t.clone() for t in written]
    args = s.args(mass=mass)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    msa.msa_qk_rope_insert(*args, s.status, stream=side)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    s.check()
    raw = lambda t: t.contiguous().view(torch.uint8)
    want = [t.clone() for t in written]
    assert all(not torch.equal(raw(a), raw(b)) for a, b in zip(start, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_qk_rope_insert(*args, s.status)
    for _ in range(2):
        for t, b in zip(written, start):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, b) in enumerate(zip(written, want)):
            assert torch.equal(raw(t), raw(b)), i
        assert int(s.status.item()) == 0

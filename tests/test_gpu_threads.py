"""The library called from several host threads."""
import ctypes
import dataclasses
import threading

import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("op", ["score", "tree", "prompt"])
@pytest.mark.parametrize("kv,scale", [(W.KV_BF16, W.SCALE_NONE), (W.KV_FP8, W.SCALE_PER_TOKEN_HEAD)])
def test_first_cuda_call_of_a_thread(msa, op, kv, scale):
    """A thread that has called nothing else of CUDA yet: the tensor maps of its first call are encoded."""
    w = W.custom(5, [70, 3, 100], [300, 900, 100], hq=8, kv_dtype=kv, scale_mode=scale)
    c = msa.DeviceCase(W.fp8_index(w, 2))
    ref, st, stream = ctypes.byref, c.status.data_ptr(), torch.cuda.current_stream().cuda_stream
    ws = torch.empty(max(msa.msa_prompt_attn_workspace_size(8, 1), msa.msa_tree_attn_workspace_size(
        w.num_rows, 3, w.bt_stride, 8, c.max_q_len)), dtype=torch.uint8, device="cuda")
    tree = msa.make_tree()
    L = msa.lib()
    fn, args, out = {
        "score": (L.msa_index_score, (ref(c.batch), c.idx_q.data_ptr(), ref(c.index), c.scores.data_ptr(), w.bt_stride, st,
                                      stream), c.scores),
        "tree": (L.msa_tree_attn, (ref(c.batch), ref(tree), ref(c.attn), ws.data_ptr(), ws.numel(), st, stream), c.out),
        "prompt": (L.msa_prompt_attn, (ref(c.batch), ref(c.attn), ws.data_ptr(), ws.numel(), st, stream), c.out)}[op]
    out.zero_()
    codes = [fn(*args)]
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        t = threading.Thread(target=lambda: codes.append(fn(*args)))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert codes == [0] * 4
    assert torch.equal(out, want) and int(c.status.item()) == 0


def together(works, times=4000):
    """works: functions of a stream that return a call's status; each runs in a thread of its own."""
    start, codes = threading.Barrier(len(works)), []

    def many(work):
        stream = torch.cuda.Stream()
        start.wait()
        codes.append({work(stream.cuda_stream) for _ in range(times)})
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=many, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(works)


@pytest.mark.parametrize("fp8,q", [(False, 1), (True, 1), (False, 64)])
def test_scores_of_few_and_many_requests(msa, fp8, q):
    def case(n):
        w = W.custom(n, [q] * n, [79 + q] * n, hq=4, topk=4)
        c = msa.DeviceCase(W.fp8_index(w, n) if fp8 else w)
        c.scores.zero_()
        return c

    cases = [case(n) for n in (3, 1500) * 3]

    def work(c):
        args = (ctypes.byref(c.batch), c.idx_q.data_ptr(), ctypes.byref(c.index), c.scores.data_ptr(), c.w.bt_stride,
                c.status.data_ptr())
        return lambda stream: msa.lib().msa_index_score(*args, stream)

    alone = []
    for c in cases:
        assert work(c)(None) == 0
        torch.cuda.synchronize()
        alone.append(c.scores.clone())
        c.scores.zero_()
    together([work(c) for c in cases])
    for c, want in zip(cases, alone):
        assert torch.equal(c.scores, want) and int(c.status.item()) == 0


def test_topk_of_wide_and_wider_tables(msa):
    def case(n, width):
        w = W.custom(n, [1] * n, [700] * n, hq=4, topk=4)
        table = np.zeros((n, width), w.block_table.dtype)
        table[:, :w.block_table.shape[1]] = w.block_table
        c = msa.DeviceCase(dataclasses.replace(w, block_table=table))
        c.scores.copy_(torch.arange(c.scores.numel(), device="cuda").view_as(c.scores) % 7919)
        return c

    cases = [case(2, width) for width in (12500, 16384) * 3]

    def work(c):
        args = (ctypes.byref(c.batch), c.scores.data_ptr(), c.w.bt_stride, c.topk, c.topk_idx.data_ptr(), c.tbl.data_ptr(),
                c.tbl_stride, c.sparse_len.data_ptr(), c.status.data_ptr())
        return lambda stream: msa.lib().msa_topk_build_table(*args, stream)

    alone = []
    for c in cases:
        assert work(c)(None) == 0
        torch.cuda.synchronize()
        alone.append(c.topk_idx.clone())
        c.topk_idx.fill_(-7)
    together([work(c) for c in cases])
    for c, want in zip(cases, alone):
        assert torch.equal(c.topk_idx, want) and int(c.status.item()) == 0


@pytest.mark.parametrize("kv,scale", [(W.KV_BF16, W.SCALE_NONE), (W.KV_FP8, W.SCALE_PER_TOKEN_HEAD)])
def test_decode_beside_other_work(msa, kv, scale):
    """The CTAs of a row write into each other's shared memory: the same results however late some of them start."""
    cases = [msa.DeviceCase(W.custom(n, [1] * n, [3000 + 100 * n] * n, hq=16, topk=16, kv_dtype=kv, scale_mode=scale))
             for n in (1, 2, 5, 9, 13)]
    for c in cases:
        c.decode()
    torch.cuda.synchronize()
    want = [c.out.clone() for c in cases]
    a = torch.randn((1024, 1024), device="cuda")
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        for c in cases:
            c.out.zero_()
        torch.cuda.synchronize()
        for c, s in zip(cases, streams):
            a = (a @ a).clamp(-1, 1)
            c.decode(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, t) and int(c.status.item()) == 0 for c, t in zip(cases, want))

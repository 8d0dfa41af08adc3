"""The library called from several host threads."""
import ctypes
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

"""DeviceCase on streams other than the current one: what a call's kernels write is
allocated on the call's stream, and no two streams or graphs share a workspace."""
import contextlib
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import workloads as W


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def fake(monkeypatch):
    """A DeviceCase without a GPU, whose streams, allocations and calls are recorded."""
    from block_sparse_paged_02_gb300 import case as C
    log = SimpleNamespace(current=[FakeStream(7)], made={}, capturing=False, calls=[])

    @contextlib.contextmanager
    def on(s):
        log.current.append(s)
        yield
        log.current.pop()

    empty = torch.empty

    def recording(*a, **k):
        t = empty(*a, **k)
        log.made[t.data_ptr()] = log.current[-1].cuda_stream
        return t

    cuda = torch.cuda
    monkeypatch.setattr(cuda, "stream", on)
    monkeypatch.setattr(cuda, "current_stream", lambda *a: log.current[-1])
    monkeypatch.setattr(cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(cuda, "is_current_stream_capturing", lambda: log.capturing)
    monkeypatch.setattr(torch, "empty", recording)
    monkeypatch.setattr(C.B, "make_tree", lambda mask=None, topk_idx=None: SimpleNamespace(topk=topk_idx or 0))
    monkeypatch.setattr(C.B, "make_cache_view", lambda *a: None)
    monkeypatch.setattr(C.B, "msa_tree_attn_workspace_size", lambda *a: 4096)
    for name in ("msa_tree_attn", "msa_attn_mass", "msa_evict_select"):
        monkeypatch.setattr(C.B, name, lambda *a, name=name: log.calls.append((name, a)))
    c = C.DeviceCase.__new__(C.DeviceCase)
    c.w = SimpleNamespace(num_reqs=2, num_pages=9, bt_stride=4, hq=8)
    c.device, c.num_rows, c.max_q_len, c._tree_ws = "cpu", 2, 1, {}
    c.batch = c.attn = c.bt = c.status = None
    return c, log


@pytest.mark.parametrize("stream,handle", [(None, 7), (FakeStream(5), 5), (9, 9), (0, 0)])
def test_allocated_on_the_stream_of_the_call(fake, stream, handle):
    c, log = fake
    for t in c.evict_select(None, None, 64, stream=stream):
        assert log.made[t.data_ptr()] == handle
    c.tree_attn(stream=stream)
    c.attn_mass(None, stream=stream)
    ws = [a[3 if name == "msa_tree_attn" else 4] for name, a in log.calls[1:]]
    assert log.made[ws[0].data_ptr()] == handle and ws[0] is ws[1]
    assert all(a[-1] is stream for _, a in log.calls)


def test_no_workspace_shared_by_streams_or_graphs(fake):
    c, log = fake

    def workspace(**kw):
        c.tree_attn(**kw)
        return log.calls[-1][1][3]

    here, there = workspace(), workspace(stream=FakeStream(5))
    assert here is not there and workspace() is here and workspace(stream=FakeStream(5)) is there
    assert workspace(topk_idx=4) is not here
    log.capturing = True
    graphs = [workspace(), workspace()]
    assert graphs[0] is not graphs[1] and here is not graphs[0] is not there
    log.capturing = False
    assert workspace() is here


@pytest.mark.gpu
def test_first_calls_on_a_side_stream():
    # work is pending on the current stream on blocks that it has just freed
    from block_sparse_paged_02_gb300 import DeviceCase
    w = W.custom(3, [20, 3], [3020, 703], hq=16)
    budget = 256
    lens = torch.tensor([3020, 703], dtype=torch.int32, device="cuda")
    mass = torch.rand((w.num_pages, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    base = DeviceCase(w)
    base.tree_attn()
    want = [t.clone() for t in base.evict_select(lens, mass, budget, 4, 32)]
    torch.cuda.synchronize()
    c = DeviceCase(w)
    need = base._tree_ws[next(iter(base._tree_ws))].numel()
    side = torch.cuda.Stream()
    for _ in range(3):
        c._tree_ws.clear()
        c.out.zero_()
        torch.cuda.synchronize()
        # about 20 ms of work in front of writes to blocks of the sizes that the calls ask for
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, 2 * budget * 4, 2 * 4)]
        torch.cuda._sleep(40_000_000)
        for t in junk:
            t.fill_(0x5a)
        del junk
        c.tree_attn(stream=side)
        keep = c.evict_select(lens, mass, budget, 4, 32, stream=side)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        assert torch.equal(c.out, base.out) and torch.equal(c.lse, base.lse)
        assert all(torch.equal(a, b) for a, b in zip(keep, want))


@pytest.mark.gpu
def test_one_case_on_two_streams_and_in_two_graphs():
    # the same batch with two masks at once: every result is that of a call by itself.  The
    # calls write one out and lse, so each stream has its own (two sets of one case)
    from block_sparse_paged_02_gb300 import DeviceCase
    w = W.custom(4, [30, 64], [6030, 2064], hq=16)
    c = DeviceCase(w)
    c.pack_step_inputs(sets=2)
    rng = np.random.default_rng(1)
    masks = [torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (94, 2)).astype(np.int32)).cuda() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def go(i, stream=None):
        c.use_step_set(i)
        c.tree_attn(mask=masks[i], stream=stream)
        return c.out, c.lse

    want = []
    for i in range(2):
        o, l = go(i)
        torch.cuda.synchronize()
        want.append((o.clone(), l.clone()))
    assert not torch.equal(want[0][0], want[1][0])

    def check(run):
        for i in range(2):
            c.use_step_set(i)
            c.out.zero_(), c.lse.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(2):
                run(i)
        torch.cuda.synchronize()
        for i in range(2):
            c.use_step_set(i)
            assert torch.equal(c.out, want[i][0]) and torch.equal(c.lse, want[i][1])

    check(lambda i: go(i, streams[i]))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(i)
        graphs.append(g)

    def replay(i):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()

    check(replay)
    assert int(c.status.item()) == 0

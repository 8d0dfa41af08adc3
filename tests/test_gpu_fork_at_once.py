"""msa_page_fork called many times at once: CTAs of a cluster that start late, host threads."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from tests import prompt_ref as P
from tests.test_gpu_pages import dev, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


class Call:
    """One fork's arguments and outputs, launched by run()."""

    def __init__(self, msa, lens, table, refs, parent, grow, width):
        n = len(parent)
        i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
        self.msa, self.refs = msa, refs
        self.out = [i32(n), i32(n, width), i32(len(refs)), i32(n), i32(n), i32(n)]
        self.args = (msa.make_cache_view(dev(lens), dev(table), len(refs)), dev(refs), dev(parent), dev(grow),
                     msa.make_page_set(*self.out))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.want = P.fork(np.asarray(lens), np.asarray(table), np.asarray(refs), parent, grow, width, len(refs))

    def run(self, stream=None):
        self.msa.msa_page_fork(*self.args, self.status, stream=stream)

    def check(self):
        got = [t.cpu().numpy() for t in self.out]
        if isinstance(self.want, int):
            assert int(self.status.item()) == self.want
            assert (got[0] == -1).all() and (got[1] == 77).all() and np.array_equal(got[2], self.refs)
            assert (got[3] == -1).all() and (got[4] == -1).all() and (got[5] == 0).all()
            return
        assert int(self.status.item()) == 0
        live = self.want[1] >= 0
        assert np.array_equal(got[1][live], self.want[1][live]) and (got[1][~live] == 77).all()
        for i in (0, 2, 3, 4, 5):
            assert np.array_equal(got[i], self.want[i]), i


def test_refused_and_good_ones_beside_other_work(msa):
    """A bad page that one CTA of the eight sees stops all of them, however late the others start."""
    rng = np.random.default_rng(3)
    calls = []
    for i in range(64):
        lens, table, refs = state(rng, 200, 6, 2000, share=False)
        if i % 2:
            r = int(np.flatnonzero(lens)[-1 - i % 7])
            table[r, (lens[r] - 1) // 128] = len(refs)
        calls.append(Call(msa, lens, table, refs, rng.integers(-1, 200, 240), rng.integers(0, 90, 240), 8))
    a = torch.randn((2048, 2048), device="cuda")
    streams = [torch.cuda.Stream() for _ in range(8)]
    torch.cuda.synchronize()
    for i, c in enumerate(calls):
        a = (a @ a).clamp(-1, 1)
        c.run(streams[i % 8])
    torch.cuda.synchronize()
    assert sum(isinstance(c.want, int) for c in calls) == 32
    for c in calls:
        c.check()


def two_sizes(msa, each=1):
    rng = np.random.default_rng(4)
    calls = []
    for n in (2100, 4096) * each:
        lens, table, refs = state(rng, n, 2, 6000, share=False)
        calls.append(Call(msa, lens, table, refs, rng.integers(-1, n, n), rng.integers(0, 90, n), 4))
    torch.cuda.synchronize()
    return calls


def test_host_threads_with_other_numbers_of_requests(msa):
    """Calls of two sizes from several threads, each on a stream of its own: none is refused by what the others
    need of shared memory."""
    calls = two_sizes(msa, 4)
    start, codes = threading.Barrier(len(calls)), []

    def many(c):
        stream = torch.cuda.Stream()
        cache, refs, parent, grow, to = c.args
        args = (ctypes.byref(cache), refs.data_ptr(), parent.data_ptr(), grow.data_ptr(), ctypes.byref(to),
                c.status.data_ptr(), stream.cuda_stream)
        fork = msa.lib().msa_page_fork
        start.wait()
        codes.append({fork(*args) for _ in range(4000)})
        stream.synchronize()

    threads = [threading.Thread(target=many, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(calls)
    for c in calls:
        c.check()


def test_two_sizes_in_one_graph(msa):
    small, large = two_sizes(msa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        large.run()
        small.run()
    graph.replay()
    torch.cuda.synchronize()
    small.check()
    large.check()

"""Compaction of requests that a fork left with common pages: refused where it would write them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import block_sparse_paged_02_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class Cache:
    """Two siblings of 300 tokens (two common pages, a last one each) and one request alone, of 200."""
    lens, table = [300, 300, 200], [[3, 5, 0], [3, 5, 1], [7, 6, -1]]

    def __init__(self, msa, width=600):
        rng = np.random.default_rng(1)
        self.msa, self.width = msa, width
        raw = lambda *s: torch.from_numpy(rng.integers(0, 255, s).astype(np.uint8)).cuda()
        self.pools = [raw(9, 128, 1, 256).view(torch.bfloat16) for _ in range(2)] + [raw(9, 128, 4).view(torch.float32).view(9, 128)]
        refs = np.zeros(9, np.int32)
        for row, n in zip(self.table, self.lens):
            refs[row[:(n + 127) // 128]] += 1
        self.refs = dev(refs)

    def compact(self, keeps, base=None, refs=True):
        """Returns the status and, per request, whether its pages hold what moving its tokens gives (True), what they
        held (False) or something else."""
        before = [t.clone() for t in self.pools]
        keep = np.full((3, self.width), -1, np.int32)
        for r, k in enumerate(keeps):
            keep[r, :len(k)] = k
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        view = self.msa.make_cache_view(dev(self.lens), dev(self.table), 9, refs=self.refs if refs else None)
        self.msa.msa_kv_compact(view, None if base is None else dev(base), dev(keep), dev([len(k) for k in keeps]),
                                self.msa.make_kv_pools(*self.pools[:2], self.msa.MSA_KV_BF16, mass=self.pools[2]), status)
        torch.cuda.synchronize()
        raw = lambda t: t.contiguous().view(torch.uint8).view(9 * 128, -1).cpu().numpy()
        ends = []
        for r, (row, n, k) in enumerate(zip(self.table, self.lens, keeps)):
            slots = np.array([row[t // 128] * 128 + t % 128 for t in range(n)])
            b = 0 if base is None else base[r]
            ok = {True: True, False: True}
            for t, old in zip(self.pools, before):
                got, was = raw(t)[slots], raw(old)[slots]
                want = was.copy()
                want[b:b + len(k)] = was[b + np.asarray(k, int)]
                ok[False] &= np.array_equal(got, was)
                ok[True] &= np.array_equal(got, want)
            ends.append(True if ok[True] else False if ok[False] else None)
        return int(status.item()), ends


@pytest.mark.parametrize("width", [200, 600])
def test_a_sibling_is_refused_alone_and_the_others_move(msa, width):
    c = Cache(msa, width)
    some = list(range(1, 150))
    assert c.compact([some, [], []]) == (8, [False, True, True])
    assert c.compact([[], some, some]) == (8, [True, False, True])
    # the request without shared pages
    assert c.compact([[], [], some]) == (0, [True, True, True])
    # a holder outside the tables counts
    c.refs[7] += 1
    assert c.compact([[], [], some])[0] == 8


def test_what_stays_where_it_is_may_be_shared(msa):
    c = Cache(msa)
    head = list(range(256))
    assert c.compact([head + [260, 299], head + list(range(270, 299)), head[:100]]) == (0, [True, True, True])
    assert c.compact([head, head[:7], []]) == (0, [True, True, True])
    # one token too early: it moves into the second common page
    assert c.compact([head[:255] + [260], head, []]) == (8, [False, True, True])


def test_drafts_behind_a_fork_are_committed(msa):
    c = Cache(msa)
    assert c.compact([[1, 3, 8], [0, 4], [5]], base=[260, 270, 190]) == (0, [True, True, True])
    assert c.compact([[1, 3, 8], [1, 4], [5]], base=[254, 270, 190]) == (8, [False, True, True])


def test_refs_of_another_pool(msa):
    c = Cache(msa)
    with pytest.raises(ValueError, match="refs"):
        msa.make_cache_view(dev(c.lens), dev(c.table), 9, refs=c.refs[:8].clone())

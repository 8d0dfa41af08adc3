"""Forks of requests that hold more pages than their tokens fill: what was reserved and not written is given back."""
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


def wanted(lens, table, refs, blocks, parent, grow, width):
    """prompt_ref.fork of what is left when every request has given back the pages behind its tokens, and the pages held
    then; the status bit that stops the call."""
    have = (np.asarray(lens) + 127) // 128
    if (blocks < have).any() or (blocks > table.shape[1]).any():
        return 4
    left = refs.astype(np.int64).copy()
    for r in range(len(lens)):
        for page in table[r, have[r]:blocks[r]]:
            if not 0 <= page < len(refs):
                return 1
            if refs[page] < 1:
                return 8
            left[page] -= 1
    got = P.fork(np.asarray(lens), table, left, parent, grow, width, len(refs))
    return got if isinstance(got, int) else (*got, (got[0] + np.asarray(grow) + 127) // 128)


def check(msa, lens, table, refs, blocks, parent, grow, width):
    lens, table, refs, blocks = (np.asarray(x, np.int32) for x in (lens, table, refs, blocks))
    n = len(parent)
    i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")
    out = [i32(n), i32(n, width), i32(len(refs)), i32(n), i32(n), i32(n), i32(n)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_page_fork(msa.make_cache_view(dev(lens), dev(table), len(refs), dev(blocks)), dev(refs), dev(parent), dev(grow),
                      msa.make_page_set(*out), status)
    got = [t.cpu().numpy() for t in out]
    want = wanted(lens, table, refs, blocks, parent, grow, width)
    if isinstance(want, int):
        assert int(status.item()) == want
        assert (got[0] == -1).all() and (got[6] == -1).all() and (got[1] == 77).all() and np.array_equal(got[2], refs)
        assert (got[3] == -1).all() and (got[4] == -1).all() and (got[5] == 0).all()
        return None
    assert int(status.item()) == 0
    live = want[1] >= 0
    assert np.array_equal(got[1][live], want[1][live]) and (got[1][~live] == 77).all()
    for i in (0, 2, 3, 4, 5, 6):
        assert np.array_equal(got[i], want[i]), i
    return want


@pytest.mark.parametrize("steps,written", [(60, 1), (60, 3), (40, 0), (40, 8)])
def test_drafts_that_are_mostly_rejected(msa, steps, written):
    """One request in a pool of five pages reserves eight tokens a step and keeps fewer: no page is lost."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    status = i32(1)
    sets = [msa.make_page_set(i32(1), i32(1, 5), i32(5), i32(1), i32(1), i32(1), i32(1)) for _ in range(2)]
    msa.msa_page_fork(msa.make_cache_view(i32(0), i32(0, 1), 5, i32(0)), i32(5), dev([-1]), dev([125]), sets[0], status)
    lens = sets[0]._keep[0] + 125
    for step in range(steps):
        old, new = sets[step % 2], sets[1 - step % 2]
        msa.msa_page_fork(msa.make_cache_view(lens, old._keep[1], 5, old._blocks), old._keep[2], dev([0]), dev([8]), new, status)
        assert int(status.item()) == 0
        lens = new._keep[0] + written
        held = (125 + written * step + 8 + 127) // 128
        assert int(new._blocks.item()) == held and int(new._keep[2].sum().item()) == held
    assert int(lens.item()) == 125 + steps * written


def test_pages_behind_the_tokens_are_given_back(msa):
    # 130 of 600 reserved tokens were written
    table, refs = [[4, 2, 1, 0, 3, -1]], [1, 1, 1, 1, 1, 0, 0]
    want = check(msa, [130], table, refs, [5], [0], [200], 6)
    assert want[1].tolist() == [[4, 2, 0, -1, -1, -1]] and want[2].tolist() == [1, 0, 1, 0, 1, 0, 0] and want[6].tolist() == [3]
    # dropped: all of its pages are free
    want = check(msa, [130], table, refs, [5], [-1], [7 * 128], 7)
    assert want[1].tolist() == [[0, 1, 2, 3, 4, 5, 6]]
    # nobody writes: the reserved pages go all the same
    want = check(msa, [130], table, refs, [5], [0, 0], [0, 0], 2)
    assert want[2].tolist() == [0, 0, 2, 0, 2, 0, 0] and want[6].tolist() == [2, 2]
    # an empty request's pages, and one held elsewhere too
    want = check(msa, [0], table, [1, 1, 1, 2, 1, 0, 0], [5], [0], [1], 1)
    assert want[1].tolist() == [[0]] and want[2].tolist() == [1, 0, 0, 1, 0, 0, 0]


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("n,new,most", [(1, 3, 2), (9, 12, 5), (60, 40, 4), (4, 6, 300), (2500, 2000, 2)])
def test_random(msa, seed, n, new, most):
    rng = np.random.default_rng(100 * seed + n)
    lens, table, refs = state(rng, n, most, 600 + 4 * new)
    have = (lens + 127) // 128
    more = np.where(rng.random(n) < 0.5, 0, rng.integers(0, 4, n))
    free = np.flatnonzero(refs == 0)
    rng.shuffle(free)
    wide = np.full((n, most + 5), -1, np.int32)
    wide[:, :table.shape[1]] = table
    refs, at = refs.copy(), 0
    for r in range(n):
        take = free[at:at + more[r]]
        more[r] = len(take)
        wide[r, have[r]:have[r] + more[r]] = take
        refs[take] += 1
        at += len(take)
    parent = rng.integers(-1, n, new)
    grow = np.where(rng.random(new) < 0.3, 0, rng.integers(0, 300, new))
    check(msa, lens, wide, refs, have + more, parent, grow, most + 4)


def test_refused_data(msa):
    lens, table, refs = [200, 100], [[0, 1, 3], [2, -1, -1]], np.array([1, 1, 1, 1, 0, 0], np.int32)
    bad = lambda blocks, table=table, refs=refs, grow=(1, 1), parent=(0, 1): check(
        msa, lens, table, refs, blocks, list(parent), list(grow), 3)
    assert bad([3, 1]) is not None
    assert bad([1, 1]) is None and bad([4, 1]) is None and bad([2, 0]) is None and bad([-1, 1]) is None
    assert bad([2 ** 31 - 1, 1]) is None and bad([-2 ** 31, 1]) is None
    assert bad([3, 2]) is None                                        # its second page is -1
    assert bad([3, 1], table=[[0, 1, 6], [2, -1, -1]]) is None
    assert bad([3, 1], refs=np.array([1, 1, 1, 0, 0, 0], np.int32)) is None
    # the page given back is among the free ones, and they are too few all the same
    assert bad([3, 1], grow=(100, 1, 1), parent=(0, 0, 1)) is not None
    assert bad([3, 1], grow=(184, 184, 284), parent=(0, 0, 1)) is None


def test_case_method(msa):
    w = P.batch(3, [5, 2], [300, 128], 8)
    c = msa.DeviceCase(w)
    lens = dev(w.context_lens)
    refs = torch.zeros(w.num_pages, dtype=torch.int32, device="cuda")
    held = [3, 2]  # (the pages of the step's own tokens are in the tables too)
    for r in range(2):
        refs[torch.from_numpy(w.block_table[r, :held[r]].astype(np.int64)).cuda()] += 1
    to = c.page_fork(lens, refs, dev([0, 1]), dev([1, 0]), bt_stride=4, blocks=dev(held))
    assert int(c.status.item()) == 0 and to._blocks.tolist() == [3, 1] and int(to._keep[2].sum()) == 4
    assert to._keep[3].tolist() == [-1, -1]
    again = msa.make_cache_view(*to._keep[:2], w.num_pages, to._blocks)
    assert again.blocks == to._blocks.data_ptr()

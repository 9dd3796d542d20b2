"""Fork and compact on a pool of more 1,024-page chunks than their grids have
CTAs (4 per SM), so that a CTA counts, ranks and writes several chunks."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu

CHUNK = 1024
PAGE_INTS = 64 * 576 // 4


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _host(t):
    return t.cpu().numpy()


@pytest.fixture(scope="module")
def pool():
    """(blocks, fp8 cache, its pages' first four bytes): 26 GB on 152 SMs."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = 4 * sms * CHUNK + 75 * CHUNK + 611        # the last chunk is not whole
    cache = torch.empty((blocks, 64, 576), dtype=torch.uint8, device="cuda")
    yield blocks, cache, cache.view(-1).view(torch.int32).view(blocks, PAGE_INTS)[:, 0]
    del cache


@pytest.mark.parametrize("in_place", [True, False])
def test_fork_takes_pages_of_every_chunk(pool, in_place):
    import torch
    blocks, cache, marks = pool
    rng = np.random.default_rng(31)
    ref = rng.integers(1, 4, blocks).astype(np.int32)
    free = np.sort(rng.permutation(blocks)[:9000])
    ref[free] = 0
    free = np.flatnonzero(ref == 0)
    assert free[-1] >= blocks - 3 * CHUNK and len(np.unique(free // CHUNK)) > 600
    held = rng.permutation(np.flatnonzero(ref))[:40 * 30].reshape(40, 30)
    table = np.full((40, 240), -1, dtype=np.int32)
    table[:, :30] = held
    children = 50
    parents = rng.integers(0, 40, children)
    shared = rng.integers(0, 30 * 64 + 1, children)
    # all free pages but one are taken: 50 children of 179 or 180 fresh pages
    fresh = np.full(children, (len(free) - 1) // children)
    fresh[:(len(free) - 1) % children] += 1
    lens = (shared // 64 + fresh) * 64 - 63 * (shared % 64 == 0)
    first = np.concatenate([[0], np.cumsum(fresh)])
    marks.copy_(torch.arange(blocks, device="cuda", dtype=torch.int32))
    refs, out = _dev(ref), _dev(np.full(blocks, -7))
    ws = binding.new_cache_workspace(blocks, children)
    child, counts = binding.mla_cache_fork(cache, refs, _dev(table), _dev(parents), _dev(shared),
                                           _dev(lens), workspace=ws,
                                           ref_counts_out=None if in_place else out)
    assert binding.read_error(ws) == 0
    want_ref, want = ref.copy(), np.full((children, 240), -1, dtype=np.int32)
    moved = np.arange(blocks)
    for c in range(children):
        whole = shared[c] // 64
        mine = free[first[c]:first[c + 1]]
        want[c, :whole] = table[parents[c], :whole]
        want[c, whole:whole + len(mine)] = mine
        np.add.at(want_ref, want[c, :whole + len(mine)], 1)
        if shared[c] % 64:
            moved[mine[0]] = table[parents[c], whole]
    assert np.array_equal(_host(child), want) and np.array_equal(_host(counts), want_ref)
    assert np.array_equal(_host(marks), moved)
    if not in_place:
        assert np.array_equal(_host(refs), ref)
    # One page more than there is: nothing changes.
    # More pages than there are: nothing changes.
    lens[-1] += 2 * 64
    before = counts.clone()
    again, _ = binding.mla_cache_fork(cache, before if in_place else refs, _dev(table),
                                      _dev(parents), _dev(shared), _dev(lens), workspace=ws,
                                      ref_counts_out=None if in_place else out)
    assert binding.read_error(ws) == binding.MLA_ERR_NO_PAGES
    assert bool((again == -1).all())
    assert np.array_equal(_host(before if in_place else out), want_ref if in_place else ref)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("density", [0.004, 0.5, 0.97])
def test_compact_moves_pages_between_distant_chunks(pool, density, in_place):
    import torch
    blocks, cache, marks = pool
    rng = np.random.default_rng(32)
    ref = (rng.random(blocks) < density).astype(np.int32)
    ref[-5:] = 1
    live = np.flatnonzero(ref)
    count = len(live)
    rows = 64
    width = -(-count // rows)
    table = np.full((rows, width), -1, dtype=np.int32)
    lens = np.zeros(rows, dtype=np.int32)
    order = rng.permutation(live)
    for r in range(rows):
        mine = order[r * width:(r + 1) * width]
        table[r, :len(mine)] = mine
        lens[r] = 64 * len(mine)
    ref[live] = 1 + live % 3                      # (counts that tables kept elsewhere add to)
    src, dst = live[live >= count], np.setdiff1d(np.arange(count), live)
    page_map = np.where(ref > 0, np.arange(blocks), -1)
    page_map[src] = dst
    want_ref = ref.copy()
    want_ref[dst], want_ref[src] = ref[src], 0
    moved = np.arange(blocks)
    moved[dst] = src
    marks.copy_(torch.arange(blocks, device="cuda", dtype=torch.int32))
    refs, tab = _dev(ref), _dev(table)
    ws = binding.new_cache_workspace(blocks)
    kw = {} if in_place else dict(ref_counts_out=_dev(np.full(blocks, -7)),
                                  block_table_out=_dev(np.full((rows, width), -9)))
    got, counts, mapped, alive = binding.mla_cache_compact(cache, refs, tab, _dev(lens),
                                                           workspace=ws, **kw)
    assert binding.read_error(ws) == 0 and int(alive) == count
    held = np.arange(width) < (lens // 64)[:, None]
    want = np.where(held, page_map[np.maximum(table, 0)], -1 if in_place else -9)
    assert np.array_equal(_host(got), want) and np.array_equal(_host(counts), want_ref)
    assert np.array_equal(_host(mapped), page_map) and np.array_equal(_host(marks), moved)

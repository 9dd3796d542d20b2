"""Fork, free and compact of the paged cache, against plain Python page lists.

Everything here is whole numbers and copied bytes, so every comparison is
exact; the pages that a call may not write are compared too.
"""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from oracle import cache_compact, cache_fork, cache_free

pytestmark = pytest.mark.gpu


def _dev(a, dtype=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).cuda()


def _cache(rng, shape, fp8):
    import torch
    bits = rng.integers(0, 256, shape, dtype=np.uint8) if fp8 else \
        rng.integers(-32768, 32768, shape, dtype=np.int16)
    t = torch.from_numpy(bits).cuda()
    return bits, (t if fp8 else t.view(torch.bfloat16))


def _host(t):
    import torch
    return (t if t.dtype != torch.bfloat16 else t.view(torch.int16)).cpu().numpy()


def _state(rng, blocks, lens, share=0.0, max_blocks=None):
    """Tables of rows over random pages (some entries shared) and their counts."""
    pages = [-(-n // 64) for n in lens]
    total = sum(pages)
    ids = rng.permutation(blocks)[:total]
    if total:
        ids = np.where(rng.random(total) < share, ids[rng.integers(0, total, total)], ids)
    width = max_blocks or max(1, max(pages, default=1))
    table = np.full((len(lens), width), -7, dtype=np.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, np.bincount(ids, minlength=blocks).astype(np.int32)


FORKS = [
    # blocks, layers, parents' lengths, (parent, shared, room) per child
    (8, 1, [64], [(0, 64, 64)]),                                   # whole pages only
    (8, 1, [64], [(0, 0, 0)]),                                     # nothing at all
    (9, 2, [65], [(0, 65, 65), (0, 1, 1), (0, 64, 65), (0, 63, 200)]),
    (40, 3, [130, 1], [(-1, 0, 100), (1, 1, 1), (0, 130, 192), (0, 130, 193), (1, 0, 64)]),
    (2100, 1, [700, 64 * 20], [(0, 700, 1000)] * 5 + [(1, 1280, 1281)] * 300 + [(1, 77, 640)] * 40),
    (1024, 2, [64 * 5 + 63], [(0, 64 * 5 + 63, 64 * 6)] * 257),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(FORKS)))
def test_fork(case, in_place, fp8):
    import torch
    blocks, layers, lens, kids = FORKS[case]
    rng = np.random.default_rng(100 + case)
    width = max(-(-max(k[2] for k in kids) // 64), max(-(-n // 64) for n in lens), 1) + 2
    table, ref = _state(rng, blocks, lens, max_blocks=width)
    bits, cache = _cache(rng, (layers, blocks, 64, 576), fp8)
    want = cache_fork(ref, table, *zip(*kids))
    assert want is not None
    ws = binding.new_cache_workspace(blocks, len(kids))
    refs, out = _dev(ref), (None if in_place else _dev(np.full(blocks, 99)))
    child = _dev(np.full((len(kids), width), -5))
    got_child, got_ref = binding.mla_cache_fork(
        cache, refs, _dev(table), *(_dev(x) for x in zip(*kids)), workspace=ws,
        child_table=child, ref_counts_out=out)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert got_ref is (refs if in_place else out)
    if not in_place:
        assert np.array_equal(_host(refs), ref)
    assert np.array_equal(_host(got_ref), want[0])
    expect = np.full((len(kids), width), -5)
    for c, row in enumerate(want[1]):
        expect[c, :len(row)] = row
    assert np.array_equal(_host(got_child), expect)
    for src, dst, rows in want[2]:
        bits[:, dst, :rows] = bits[:, src, :rows]
    assert np.array_equal(_host(cache), bits)


def test_fork_uses_every_last_page_and_then_refuses():
    rng = np.random.default_rng(7)
    table, ref = _state(rng, 3000, [64 * 10], max_blocks=3000)
    bits, cache = _cache(rng, (3000, 64, 576), True)
    ws = binding.new_cache_workspace(3000, 2)
    refs = _dev(ref)
    child, _ = binding.mla_cache_fork(cache, refs, _dev(table), _dev([-1, 0]), _dev([0, 640]),
                                      _dev([64 * 2000, 640 + 64 * 990]), workspace=ws)
    assert binding.read_error(ws) == 0
    now = _host(refs)
    assert (now > 0).all() and now.sum() == 10 + 2000 + 1000
    before = _host(child).copy()
    binding.mla_cache_fork(cache, refs, _dev(table), _dev([-1, 0]), _dev([0, 0]), _dev([1, 0]),
                           workspace=ws, child_table=child)
    assert binding.read_error(ws) == binding.MLA_ERR_NO_PAGES
    assert np.array_equal(_host(refs), now) and np.array_equal(_host(child), before)
    assert np.array_equal(_host(cache), bits)


@pytest.mark.parametrize("kids,table_edit,code", [
    ([(0, 10, 100), (3, 1, 1)], None, binding.MLA_ERR_BAD_ROW),
    ([(0, 10, 100), (-1, 1, 1)], None, binding.MLA_ERR_BAD_ROW),
    ([(0, 10, 9)], None, binding.MLA_ERR_BAD_SEQ_LEN),
    ([(0, -1, 9)], None, binding.MLA_ERR_BAD_SEQ_LEN),
    ([(0, 10, 64 * 4 + 1)], None, binding.MLA_ERR_BAD_SEQ_LEN),
    ([(0, 10, 2 ** 31 - 1)], None, binding.MLA_ERR_BAD_SEQ_LEN),
    ([(0, 65, 65)], (0, 1, 20), binding.MLA_ERR_BAD_BLOCK_ID),
    ([(0, 65, 65)], (0, 1, -1), binding.MLA_ERR_BAD_BLOCK_ID),
    ([(0, 65, 65)], (0, 1, "free"), binding.MLA_ERR_PAGE_STATE),
    ([(-1, 0, 256)] * 8192, None, binding.MLA_ERR_NO_PAGES),
])
def test_fork_refusals_change_nothing(kids, table_edit, code):
    rng = np.random.default_rng(3)
    table, ref = _state(rng, 20, [200, 64], max_blocks=4)
    if table_edit:
        r, j, v = table_edit
        table[r, j] = int(np.flatnonzero(ref == 0)[0]) if v == "free" else v
    bits, cache = _cache(rng, (20, 64, 576), False)
    ws = binding.new_cache_workspace(20, len(kids))
    child, out = _dev(np.full((len(kids), 4), -5)), _dev(np.full(20, 99))
    binding.mla_cache_fork(cache, _dev(ref), _dev(table), *(_dev(x) for x in zip(*kids)),
                           workspace=ws, child_table=child, ref_counts_out=out)
    assert binding.read_error(ws) == code
    assert np.array_equal(_host(out), ref)
    assert (_host(child) == -5).all() and np.array_equal(_host(cache), bits)


def test_fork_of_nobody_and_of_strided_layers():
    import torch
    rng = np.random.default_rng(5)
    table, ref = _state(rng, 12, [100])
    bits, cache = _cache(rng, (3, 14, 64, 576), False)
    ws = binding.new_cache_workspace(12, 1)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    child, out = binding.mla_cache_fork(cache[:, :12], _dev(ref), _dev(table), none, none, none,
                                        workspace=ws, ref_counts_out=_dev(np.zeros(12)))
    assert binding.read_error(ws) == 0 and np.array_equal(_host(out), ref)
    # layers further apart than their pages
    want = cache_fork(ref, table, [0], [100], [100])
    binding.mla_cache_fork(cache[:, :12], _dev(ref), _dev(table), _dev([0]), _dev([100]),
                           _dev([100]), workspace=ws)
    assert binding.read_error(ws) == 0
    for src, dst, rows in want[2]:
        bits[:, dst, :rows] = bits[:, src, :rows]
    assert np.array_equal(_host(cache), bits)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("blocks,lens,share,rows", [
    (4, [1], 0.0, [0]),
    (4, [0, 64], 0.0, [0]),
    (50, [64, 65, 700, 0, 63], 0.0, [2, 0, 4]),
    (1025, [64 * 300, 64 * 257, 5], 0.3, [1, 2]),
    (5000, [64 * 9 + 3] * 400, 0.9, list(range(0, 400, 3))),
    (9, [64], 0.0, []),
])
def test_free(blocks, lens, share, rows, in_place):
    import torch
    rng = np.random.default_rng(blocks)
    table, ref = _state(rng, blocks, lens, share)
    want, freed = cache_free(ref, table, lens, rows)
    ws = binding.new_status_workspace()
    refs, out = _dev(ref), (None if in_place else _dev(np.full(blocks, 99)))
    got, n = binding.mla_cache_free(refs, _dev(table), _dev(lens), _dev(rows), workspace=ws,
                                    ref_counts_out=out)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert np.array_equal(_host(got), want) and int(n) == freed
    if not in_place:
        assert np.array_equal(_host(refs), ref)


@pytest.mark.parametrize("lens,rows,edit,code", [
    ([64, 200], [0, 2], None, binding.MLA_ERR_BAD_ROW),
    ([64, 200], [0, -1], None, binding.MLA_ERR_BAD_ROW),
    ([64, 64 * 4 + 1], [0, 1], None, binding.MLA_ERR_BAD_SEQ_LEN),
    ([64, -5], [0, 1], None, binding.MLA_ERR_BAD_SEQ_LEN),
    ([64, 64], [0, 1], (1, 0, 30), binding.MLA_ERR_BAD_BLOCK_ID),
    ([64, 64], [0, 1], (1, 0, -3), binding.MLA_ERR_BAD_BLOCK_ID),
])
def test_free_skips_what_is_bad(lens, rows, edit, code):
    rng = np.random.default_rng(1)
    table, ref = _state(rng, 30, [64, 200], max_blocks=4)
    if edit:
        table[edit[0], edit[1]] = edit[2]
    ws = binding.new_status_workspace()
    got, n = binding.mla_cache_free(_dev(ref), _dev(table), _dev(lens), _dev(rows), workspace=ws)
    assert binding.read_error(ws) == code
    want, freed = cache_free(ref, table, lens, [0])
    assert np.array_equal(_host(got), want) and int(n) == freed


def test_free_of_a_row_named_too_often_ends_at_zero():
    rng = np.random.default_rng(2)
    table, ref = _state(rng, 700, [64 * 500, 64 * 100], max_blocks=500)
    table[1, :100] = table[0, :100]
    ref = np.bincount(np.concatenate([table[0], table[1, :100]]), minlength=700)
    ws = binding.new_status_workspace()
    got, n = binding.mla_cache_free(_dev(ref), _dev(table), _dev([64 * 500, 64 * 100]),
                                    _dev([0] * 50 + [1] * 3), workspace=ws)
    assert binding.read_error(ws) == binding.MLA_ERR_PAGE_STATE
    assert (_host(got) == 0).all() and int(n) == int((ref > 0).sum())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("blocks,layers,lens,share,pattern", [
    (1, 1, [5], 0.0, "random"),
    (6, 2, [0], 0.0, "random"),            # nothing live
    (10, 1, [640], 0.0, "random"),         # everything live
    (100, 2, [1, 64, 65, 700], 0.2, "random"),
    (300, 1, [64 * 20] * 5, 0.0, "high"),  # every live page moves
    (300, 1, [64 * 20] * 5, 0.0, "low"),   # none does
    (2048, 1, [64 * 64] * 16, 0.0, "high"),        # M on a chunk border
    (3000, 1, [64 * 100 + 1] * 20, 0.5, "random"),
    (1024, 1, [64 * 8] * 128, 0.0, "random"),      # a full pool of one chunk
])
def test_compact(blocks, layers, lens, share, pattern, in_place, fp8):
    import torch
    rng = np.random.default_rng(blocks + len(lens))
    table, ref = _state(rng, blocks, lens, share)
    if pattern != "random":
        total = sum(-(-n // 64) for n in lens)
        ids = rng.permutation(total) + (blocks - total if pattern == "high" else 0)
        table = ids.reshape(len(lens), -1).astype(np.int32)
        ref = np.bincount(ids, minlength=blocks).astype(np.int32)
    bits, cache = _cache(rng, (layers, blocks, 64, 576), fp8)
    want_ref, want_map, moves, live = cache_compact(ref)
    ws = binding.new_cache_workspace(blocks)
    tab, refs = _dev(table), _dev(ref)
    outs = {} if in_place else {"block_table_out": _dev(np.full(table.shape, -9)),
                                "ref_counts_out": _dev(np.full(blocks, 99))}
    got_t, got_r, got_map, got_live = binding.mla_cache_compact(cache, refs, tab, _dev(lens),
                                                                workspace=ws, **outs)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert int(got_live) == live
    assert np.array_equal(_host(got_r), want_ref) and np.array_equal(_host(got_map), want_map)
    want_t = (table if in_place else np.full(table.shape, -9)).copy()
    for r, n in enumerate(lens):
        k = -(-n // 64)
        want_t[r, :k] = want_map[table[r, :k]]
    assert np.array_equal(_host(got_t), want_t)
    for a, b in moves:
        bits[:, b] = bits[:, a]
    assert np.array_equal(_host(cache), bits)


def test_compact_passes_bad_entries_on():
    rng = np.random.default_rng(11)
    table, ref = _state(rng, 40, [64 * 3, 64 * 3, 64 * 3], max_blocks=4)
    free = np.flatnonzero(ref == 0)
    for edit, lens, code in [((0, 1, 40), [192] * 3, binding.MLA_ERR_BAD_BLOCK_ID),
                             ((0, 1, -1), [192] * 3, binding.MLA_ERR_BAD_BLOCK_ID),
                             ((0, 1, int(free[-1])), [192] * 3, binding.MLA_ERR_PAGE_STATE),
                             ((0, 1, int(free[0])), [192] * 3, binding.MLA_ERR_PAGE_STATE),
                             ((0, 3, 17), [192, 257, 192], binding.MLA_ERR_BAD_SEQ_LEN)]:
        bad = table.copy()
        bad[edit[0], edit[1]] = edit[2]
        _, cache = _cache(rng, (40, 64, 576), True)
        ws = binding.new_cache_workspace(40)
        got, _, page_map, _ = binding.mla_cache_compact(cache, _dev(ref), _dev(bad), _dev(lens),
                                                        workspace=ws,
                                                        ref_counts_out=_dev(np.zeros(40)))
        assert binding.read_error(ws) == code
        m = _host(page_map)
        want = bad.copy()
        for r in range(3):
            for j in range(3):
                if lens[r] == 192 and (r, j) != edit[:2]:
                    want[r, j] = m[bad[r, j]]
        assert np.array_equal(_host(got), want)


def test_a_life_of_forks_frees_and_compactions():
    """Random operations on one pool, the counts always those of the tables."""
    rng = np.random.default_rng(42)
    blocks, width = 400, 12
    bits, cache = _cache(rng, (2, blocks, 64, 576), True)
    refs = _dev(np.zeros(blocks))
    ws = binding.new_cache_workspace(blocks, 64)
    rows = {}                              # a request: its pages, its length, its tokens' bytes
    next_id = 0
    for step in range(40):
        kids, parents = int(rng.integers(1, 12)), sorted(rows)
        table = np.full((max(1, len(parents)), width), -1, dtype=np.int32)
        for r, k in enumerate(parents):
            table[r, :len(rows[k][0])] = rows[k][0]
        spec = []
        for _ in range(kids):
            p = int(rng.integers(-1, len(parents))) if parents else -1
            s = int(rng.integers(0, rows[parents[p]][1] + 1)) if p >= 0 else 0
            spec.append((p, s, int(min(64 * width, s + rng.integers(0, 150)))))
        before = _host(refs).copy()
        child, _ = binding.mla_cache_fork(cache, refs, _dev(table), *(_dev(x) for x in zip(*spec)),
                                          workspace=ws)
        err = binding.read_error(ws)
        want = cache_fork(before, table, *zip(*spec))
        if want is None:
            assert err == binding.MLA_ERR_NO_PAGES and np.array_equal(_host(refs), before)
        else:
            assert err == 0 and np.array_equal(_host(refs), want[0])
            got, now = _host(child), _host(cache)
            for c, (p, s, n) in enumerate(spec):
                pages = got[c, :-(-n // 64)].copy()
                tokens = now[:, pages].reshape(2, -1, 576)[:, :s].copy()
                if p >= 0:
                    assert np.array_equal(tokens, rows[parents[p]][2][:, :s])
                rows[next_id] = (pages, s, tokens)
                next_id += 1
        gone = [k for k in rows if rng.random() < (0.6 if want is None else 0.2)]
        if gone:
            keys = sorted(rows)
            table = np.full((len(keys), width), -1, dtype=np.int32)
            lens = [64 * len(rows[k][0]) for k in keys]
            for r, k in enumerate(keys):
                table[r, :len(rows[k][0])] = rows[k][0]
            binding.mla_cache_free(refs, _dev(table), _dev(lens),
                                   _dev([keys.index(k) for k in gone]), workspace=ws)
            assert binding.read_error(ws) == 0
            for k in gone:
                del rows[k]
        if step % 5 == 4 and rows:
            keys = sorted(rows)
            table = np.full((len(keys), width), -1, dtype=np.int32)
            for r, k in enumerate(keys):
                table[r, :len(rows[k][0])] = rows[k][0]
            t, _, _, live = binding.mla_cache_compact(
                cache, refs, _dev(table), _dev([64 * len(rows[k][0]) for k in keys]), workspace=ws)
            assert binding.read_error(ws) == 0
            t, now = _host(t), _host(cache)
            assert (_host(refs)[:int(live)] > 0).all() and (_host(refs)[int(live):] == 0).all()
            for r, k in enumerate(keys):
                pages = t[r, :len(rows[k][0])].copy()
                assert np.array_equal(now[:, pages].reshape(2, -1, 576)[:, :rows[k][1]], rows[k][2])
                rows[k] = (pages, rows[k][1], rows[k][2])
        count = np.bincount(np.concatenate([np.asarray(r[0], dtype=np.int64) for r in rows.values()]
                                           + [np.zeros(0, np.int64)]), minlength=blocks)
        assert np.array_equal(_host(refs), count)


def test_pages_calls_replay_in_a_graph():
    import torch
    rng = np.random.default_rng(8)
    table, ref = _state(rng, 500, [64 * 6 + 5] * 4, max_blocks=10)
    bits, cache = _cache(rng, (2, 500, 64, 576), True)
    ws = binding.new_cache_workspace(500, 6)
    refs, out, out2 = _dev(ref), _dev(np.zeros(500)), _dev(np.zeros(500))
    tab, parents = _dev(table), _dev([0, 1, 2, 3, 0, 0])
    shared, room = _dev([389, 64, 100, 0, 1, 389]), _dev([400, 64, 300, 10, 1, 640])
    child, lens = _dev(np.full((6, 10), -1)), _dev([400, 64, 300, 10, 1, 640])
    rows, freed = _dev([0, 1, 2, 3, 4, 5]), _dev([0])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        binding.mla_cache_fork(cache, refs, tab, parents, shared, room, workspace=ws,
                               child_table=child, ref_counts_out=out, stream=stream)
        binding.mla_cache_free(out, child, lens, rows, workspace=ws, ref_counts_out=out2,
                               num_freed=freed, stream=stream)
    want = cache_fork(ref, table, [0, 1, 2, 3, 0, 0], [389, 64, 100, 0, 1, 389],
                      [400, 64, 300, 10, 1, 640])
    for _ in range(3):
        child.fill_(-1)
        out.zero_()
        out2.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        assert np.array_equal(_host(out), want[0]) and np.array_equal(_host(out2), ref)
        assert int(freed) == sum(-(-n // 64) for n in [400, 64, 300, 10, 1, 640]) - \
            sum(s // 64 for s in [389, 64, 100, 0, 1, 389])


def test_page_operations_on_two_streams_at_once():
    """Two pools, two streams, nothing between the calls: every result is the
    one that a stream of its own gives."""
    import torch
    rng = np.random.default_rng(21)
    pools = []
    for blocks in (900, 1500):
        table, ref = _state(rng, blocks, [64 * 7 + 9] * 30, max_blocks=12)
        bits, cache = _cache(rng, (3, blocks, 64, 576), False)
        kids = [(int(rng.integers(0, 30)), int(rng.integers(0, 458)), 500) for _ in range(40)]
        want = cache_fork(ref, table, *zip(*kids))
        pools.append(dict(cache=cache, refs=_dev(ref), table=_dev(table), want=want, bits=bits,
                          kids=[_dev(x) for x in zip(*kids)], out=_dev(np.zeros(blocks)),
                          back=_dev(np.zeros(blocks)), child=_dev(np.full((40, 12), -1)),
                          rows=_dev(np.arange(40)), lens=_dev([500] * 40), freed=_dev([0]),
                          ref=ref, ws=binding.new_cache_workspace(blocks, 40),
                          stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for p in pools:
            binding.mla_cache_fork(p["cache"], p["refs"], p["table"], *p["kids"], workspace=p["ws"],
                                   child_table=p["child"], ref_counts_out=p["out"],
                                   stream=p["stream"])
            binding.mla_cache_free(p["out"], p["child"], p["lens"], p["rows"], workspace=p["ws"],
                                   ref_counts_out=p["back"], num_freed=p["freed"],
                                   stream=p["stream"])
    torch.cuda.synchronize()
    for p in pools:
        assert binding.read_error(p["ws"]) == 0
        assert np.array_equal(_host(p["out"]), p["want"][0])
        assert np.array_equal(_host(p["back"]), p["ref"])
        for src, dst, rows in p["want"][2]:
            p["bits"][:, dst, :rows] = p["bits"][:, src, :rows]
        assert np.array_equal(_host(p["cache"]), p["bits"])


def test_a_pool_of_many_chunks_and_a_cache_past_2_31_bytes():
    """700,000 pages' counts (more chunks than a grid has CTAs), and pages
    behind the first 2^31 bytes of a layer."""
    import torch
    rng = np.random.default_rng(22)
    blocks = 700_000
    ref = (rng.random(blocks) < 0.5).astype(np.int32)
    live = np.flatnonzero(ref)
    table = live[-64:].reshape(1, -1).astype(np.int32)
    ws = binding.new_status_workspace()
    got, freed = binding.mla_cache_free(_dev(ref), _dev(table), _dev([64 * 64]), _dev([0]),
                                        workspace=ws, ref_counts_out=_dev(np.zeros(blocks)))
    assert binding.read_error(ws) == 0 and int(freed) == 64
    assert np.array_equal(_host(got), np.where(np.isin(np.arange(blocks), table), 0, ref))
    blocks = 70_000
    ref = np.zeros(blocks, dtype=np.int32)
    ref[-3000:] = 1
    cache = torch.zeros((blocks, 64, 576), dtype=torch.uint8, device="cuda")
    cache[-3000:] = torch.arange(3000, device="cuda").remainder(251).to(torch.uint8)[:, None, None]
    ws = binding.new_cache_workspace(blocks)
    refs = _dev(ref)
    table = _dev(np.arange(blocks - 3000, blocks).reshape(3, 1000))
    table, _, page_map, live = binding.mla_cache_compact(cache, refs, table, _dev([64000] * 3),
                                                         workspace=ws)
    assert binding.read_error(ws) == 0 and int(live) == 3000
    assert np.array_equal(_host(table).reshape(-1), np.arange(3000))
    assert torch.equal(cache[:3000, 0, 0].long(),
                       torch.arange(3000, device="cuda").remainder(251))
    assert bool((cache[:3000] == cache[:3000, :1, :1]).all())


def test_lengths_near_the_largest_int_are_counted_right():
    """A row of 2^25 entries may be 2^31 - 1 tokens long: its pages are 2^25,
    not a negative number that is passed over."""
    import torch
    width, blocks, longest = 1 << 25, 4, 2 ** 31 - 1
    ws = binding.new_cache_workspace(blocks, 1)
    table = torch.full((1, width), -3, dtype=torch.int32, device="cuda")
    table[0, 0] = 2
    ref = _dev([0, 0, 1, 0])
    cache = torch.zeros((blocks, 64, 576), dtype=torch.uint8, device="cuda")
    child = torch.full((1, width), -5, dtype=torch.int32, device="cuda")
    binding.mla_cache_fork(cache, ref, table, _dev([0]), _dev([64]), _dev([longest]), workspace=ws,
                           child_table=child)
    assert binding.read_error(ws) == binding.MLA_ERR_NO_PAGES
    assert ref.tolist() == [0, 0, 1, 0] and bool((child == -5).all())
    # The one good entry is counted down, the others are reported.
    _, freed = binding.mla_cache_free(ref, table, _dev([longest]), _dev([0]), workspace=ws)
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    assert ref.tolist() == [0, 0, 0, 0] and int(freed) == 1
    ref = _dev([0, 0, 1, 0])
    table, _, _, live = binding.mla_cache_compact(cache, ref, table, _dev([longest]), workspace=ws)
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    assert int(live) == 1 and int(table[0, 0]) == 0 and bool((table[0, 1:] == -3).all())

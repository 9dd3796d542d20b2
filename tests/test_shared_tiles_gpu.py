"""mla_decode_shared where prefixes are read together (span_sharing.py restates
when that is; every test here asserts that it happened), against the 64-bit
definition (tolerances: span_util.py)."""

import functools

import numpy as np
import pytest

import test_shared_gpu
import test_span_serving_gpu
from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64, bf16_tensor_bits
from span_sharing import assert_shared, pool_problem, saved_steps, tile_rows, tile_rows_left_in
from span_util import K_SCALE, NAN, SCALE, check, dev, ints, random_q, reference, run_shared, shared_problem

pytestmark = pytest.mark.gpu


def _all(lens):
    return [np.arange(n) for n in lens]


# (lens, group starts, shared lengths, heads, SMs)
CASES = [
    ([1700 + 9 * i for i in range(32)], [0, 8, 16, 24, 32], [1664, 1600, 1690, 1664], 16, 152),    # a full tile a group
    ([1700 + 9 * i for i in range(32)], [0, 8, 16, 24, 32], [1664, 1600, 1690, 1664], 16, 9),
    ([4600 + i for i in range(12)], [0, 12], [4544], 65, 152),               # tiles that begin inside a request
    ([1000 + i for i in range(3)], [0, 3], [960], 65, 2),
    ([7400 + 3 * i for i in range(14)], [0, 14], [7360], 100, 152),
    ([2600] * 14, [0, 14], [2560], 100, 10),
    ([5200 + 5 * i for i in range(16)], [0, 16], [5120], 120, 6),
    ([6500, 6400, 6401] * 3, [0, 9], [6400], 33, 152),                       # lengths at the prefix's end
    ([384 + i * (i % 3 > 0) for i in range(64)], [0, 64], [384], 3, 152),    # rows whose last tokens are the prefix
    ([0 if i % 7 == 0 else 400 + i for i in range(70)], [1, 66], [390], 3, 152),    # padding, the first among them
    ([500, 0, 2000, 2100, 2200, 0, 2300, 2400] + [800 + i for i in range(12)], [2, 8, 8, 20], [1920, 64, 780], 16, 20),
    ([64 * 9 + 1] * 24, [0, 24], [64 * 9], 1, 16),                           # a prefix of an odd number of pages
    ([1100] * 5 + [90] + [1100] * 5, [0, 5, 11], [1050, 1050], 24, 4),       # one group's prefix cut to 64 tokens
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tiles_against_the_definition(case, fp8):
    import torch
    lens, starts, shared, heads, num_sms = CASES[case]
    rng = np.random.default_rng(500 + case)
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, len(lens), heads)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=num_sms)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert_shared(ws, lens, starts, shared, heads, num_sms)
    check(out, lse, reference(q, cache, table, _all(lens), SCALE), (case, fp8))


@pytest.mark.parametrize("seed", range(24))
def test_random_batches_that_share(seed):
    """Groups between requests of no group, padding, prefixes that end inside a page, some members short of it."""
    import torch
    rng = np.random.default_rng(31000 + seed)
    heads = int(rng.choice([1, 3, 8, 16, 33, 48, 65, 80]))
    num_sms = int(rng.choice([2, 6, 20, 40]))
    fp8 = bool(seed % 2)
    while True:
        sizes = [int(rng.integers(2, 13)) for _ in range(int(rng.integers(1, 5)))]
        starts = np.concatenate([[0], np.cumsum(sizes)]) + int(rng.integers(0, 3))
        B = int(starts[-1] + rng.integers(0, 3))
        shared = [int(rng.integers(200, 3000)) for _ in sizes]
        lens = [int(rng.integers(0, 300)) for _ in range(B)]
        for g, s in enumerate(shared):
            for b in range(starts[g], starts[g + 1]):
                lens[b] = 0 if rng.integers(9) == 0 else lens[b] + s - int(rng.integers(0, 70))
        if max(tile_rows(lens, starts, shared, heads, num_sms)) >= 0:
            break
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    shared = [min(s, 64 * table.shape[1]) for s in shared]
    q = random_q(rng, B, heads, float(rng.choice([0.2, 1.0, 3.0])))
    scale = float(rng.choice([SCALE, -SCALE, 0.3]))
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, scale, num_sms)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert_shared(ws, lens, starts, shared, heads, num_sms)
    check(out, lse, reference(q, cache, table, _all(lens), scale), (seed, lens, starts, shared))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("members,pages,saved", [(8, 44, 152), (4, 102, 151), (4, 104, 154), (8, 42, 145)])
def test_both_sides_of_the_rule(members, pages, saved, fp8):
    """16 heads: one tile, on 76 pairs. 152 steps saved are enough, 151 are not."""
    import torch
    rng = np.random.default_rng(pages)
    lens, starts, shared = [64 * pages + 17 * i for i in range(members)], [0, members], [64 * pages]
    assert saved_steps(lens, starts, shared, 16) == [saved]
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, members, 16)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=152)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert (max(tile_rows_left_in(ws, members)) >= 0) == (saved >= 152)
    check(out, lse, reference(q, cache, table, _all(lens), SCALE))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_thousand_groups(fp8):
    """4,096 requests, 1,100 groups of one to six; more tiles than a CTA keeps records of."""
    import torch
    rng = np.random.default_rng(78)
    B = 4096
    starts = [0]
    while len(starts) <= 1100:
        starts.append(min(B - 40, starts[-1] + int(rng.integers(1, 7))))
    shared = [64 * int(x) for x in rng.integers(0, 7, len(starts) - 1)]
    lens = rng.integers(0, 50, B)
    for g, s in enumerate(shared):
        for b in range(starts[g], starts[g + 1]):
            lens[b] = 0 if rng.integers(30) == 0 else lens[b] + s
    cache, table = pool_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, B, 1)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert_shared(ws, lens, starts, shared, 1)
    check(out, lse, reference(q, cache, table, _all(lens), SCALE))


@pytest.mark.parametrize("fp8", [False, True])
def test_repeated_calls_and_the_workspace_bounds(fp8):
    """Bit for bit the same, with NaN in the workspace in between, nothing
    written behind the workspace; and what the plain decode gives."""
    import torch
    rng = np.random.default_rng(4)
    lens, starts, shared, heads = [3000 + 31 * i for i in range(20)], [0, 9, 20], [2944, 2900], 24
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, 20, heads)
    ref = reference(q, cache, table, _all(lens), SCALE)
    plan = binding.make_span_plan(20, heads, table.shape[1], max_groups=2)
    nbytes = int(plan.workspace_bytes)
    store = torch.full((nbytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = store[:nbytes]
    binding.load_library().mla_workspace_init(binding._ptr(ws), nbytes, binding._stream_ptr(None))
    first = run_shared(q, cache, table, lens, starts, shared, plan=plan, ws=ws)[:2]
    assert_shared(ws, lens, starts, shared, heads)
    check(*first, ref)
    for _ in range(3):
        store[8192:nbytes] = 0xFF
        out, lse, _ = run_shared(q, cache, table, lens, starts, shared, plan=plan, ws=ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    torch.cuda.synchronize()
    assert (store[nbytes:] == 0x5A).all()
    assert not ws[:binding.STATUS_BYTES].any()
    args = (dev(q), dev(cache), ints(table), ints(lens), SCALE)
    check(*(binding.mla_decode_fp8(*args, K_SCALE) if fp8 else binding.mla_decode(*args)), ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_replays_that_share_and_do_not(fp8):
    """One captured call behind copies of its inputs, replayed with groups that
    are read together, groups that are not, and none, one after another."""
    import torch
    rng = np.random.default_rng(32)
    B, N, M, num_sms = 12, 16, 40, 152
    plan = binding.make_span_plan(B, N, M, max_groups=3, num_sms=num_sms)
    ws = binding.new_workspace(plan)
    cache = torch.zeros((B * M, 64, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    q = torch.zeros((B, N, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((B, M), dtype=torch.int32, device="cuda")
    given = [ints([0] * B), ints([0] * 4), ints([0] * 3)]
    held = [t.clone() for t in given]
    out = torch.empty((B, N, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, N), dtype=torch.float32, device="cuda")

    def call():
        for h, t in zip(held, given):
            h.copy_(t)
        lens, starts, shared = held
        args = (q, cache, table, lens, starts, shared, SCALE)
        kw = dict(plan=plan, workspace=ws, out=out, lse=lse)
        binding.mla_decode_shared_fp8(*args, K_SCALE, **kw) if fp8 else binding.mla_decode_shared(*args, **kw)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    seen = set()
    for starts, shared, top in (([0, 12, 12, 12], [1920, 0, 0], 600), ([0, 4, 8, 12], [640, 700, 64], 500),
                                ([0, 8, 8, 12], [2000, 64, 2100], 300), ([0, 0, 0, 0], [0, 0, 0], 900),
                                ([1, 11, 12, 12], [2240, 0, 0], 60)):
        lens = [int(x) for x in rng.integers(0, top, B)]
        for g, s in enumerate(shared):
            for b in range(starts[g], starts[g + 1]):
                lens[b] += s
        host, rows = shared_problem(rng, lens, starts, shared, fp8)
        full = np.full((B, M), -1, dtype=np.int32)
        full[:, :rows.shape[1]] = rows
        query = random_q(rng, B, N)
        cache[:host.shape[0]] = dev(host)
        q.copy_(dev(query)), table.copy_(ints(full))
        for t, v in zip(given, (lens, starts, shared)):
            t.copy_(ints(v))
        graph.replay()
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        want = tile_rows(lens, starts, shared, N, num_sms)
        assert tile_rows_left_in(ws, B) == want
        seen.add(max(want) >= 0)
        check(out, lse, reference(query, host, full, _all(lens), SCALE), (starts, shared))
    assert seen == {False, True}


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_and_bad_pages_in_a_prefix_that_is_read_together(fp8):
    """A NaN reaches the group's rows and no others; a page that is not there is
    zeros for them; rows of requests without tokens stay empty."""
    import torch
    rng = np.random.default_rng(81)
    lens, starts, shared, heads = [2300 + i for i in range(10)] + [2200] * 10, [0, 10, 20], [2240, 2176], 16
    lens[3] = 0
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, 20, heads)
    ref = reference(q, cache, table, _all(lens), SCALE)
    clean = cache.copy()
    cache[table[0, 20], 63, 5] = NAN[fp8]
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert_shared(ws, lens, starts, shared, heads)
    hit = np.array([b < 10 and b != 3 for b in range(20)])
    assert np.isnan(bf16_bits_to_f64(bf16_tensor_bits(out))[hit]).all()
    assert lse.isnan().cpu().numpy()[hit].all()
    keep = np.nonzero(~hit)[0]
    at = torch.from_numpy(keep).cuda()
    check(out[at], lse[at], [x[keep] for x in ref])
    broken = table.copy()
    broken[10:, 7] = -1
    out, lse, ws = run_shared(q, clean, broken, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    zeros = np.concatenate([clean, np.zeros((1, 64, 576), clean.dtype)])
    check(out, lse, reference(q, zeros, np.where(broken < 0, clean.shape[0], broken), _all(lens), SCALE))


# Tests of batches that a whole GPU's pairs do not share, on as few as share them.
FEWER_SMS = [
    (test_shared_gpu.test_many_requests_and_groups, {}, 8),
    (test_shared_gpu.test_it_equals_the_plain_decode, {}, 100),
    (test_shared_gpu.test_results_repeat_bit_for_bit_and_the_workspace_keeps_its_bounds, {}, 80),
    (test_shared_gpu.test_replays_with_other_lengths_and_groups_on_two_streams, {}, 2),
    (test_span_serving_gpu.test_forked_requests_step_by_step, {"fp8": False}, 2),
    (test_span_serving_gpu.test_forked_requests_step_by_step, {"fp8": True}, 2),
    (test_span_serving_gpu.test_calls_behind_one_another_without_a_wait, {"fp8": False}, 2),
    (test_span_serving_gpu.test_calls_behind_one_another_without_a_wait, {"fp8": True}, 2),
]


@pytest.mark.parametrize("which", range(len(FEWER_SMS)))
def test_again_on_fewer_sms(which, monkeypatch):
    import torch
    test, kw, num_sms = FEWER_SMS[which]
    make, rows, spaces = binding.make_span_plan, [], []

    def plan_for(batch, heads, blocks, **a):
        return make(batch, heads, blocks, **{**a, "num_sms": num_sms})

    def recorded(fn, q, *args, **a):
        results = fn(q, *args, **a)
        tiles = a["workspace"][binding.STATUS_BYTES:binding.STATUS_BYTES + 4 * q.shape[0]]
        spaces.append(tiles)
        if not torch.cuda.is_current_stream_capturing():
            rows.append(tiles.clone())               # (before the next call has the workspace)
        return results

    monkeypatch.setattr(binding, "make_span_plan", plan_for)
    for name in ("mla_decode_shared", "mla_decode_shared_fp8"):
        monkeypatch.setattr(binding, name, functools.partial(recorded, getattr(binding, name)))
    test(**kw)
    torch.cuda.synchronize()
    assert any((t.view(torch.int32) >= 0).any() for t in rows + spaces)

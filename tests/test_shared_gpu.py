"""mla_decode_shared against the 64-bit definition (tolerances: span_util.py)."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64, bf16_tensor_bits
from span_util import (K_SCALE, NAN, SCALE, check, dev, ints, random_q, reference, run_shared,
                       shared_problem)

pytestmark = pytest.mark.gpu


def _all(lens):
    return [np.arange(n) for n in lens]


# (lens, group starts, shared lengths, heads)
CASES = [
    ([1], [0, 1], [0], 1),
    ([64, 64], [0, 2], [64], 128),
    ([200, 130], [0, 2], [128], 16),
    ([500] * 8, [0, 8], [448], 16),                          # a full tile
    ([500, 449, 700, 460, 448, 1000, 449, 512, 470], [0, 9], [448], 16),   # a tile and a bit; L = prefix
    ([300, 400, 500], [0, 3], [299], 5),                     # the prefix ends inside a page
    ([700] * 5, [0, 5], [640], 100),                         # tiles that begin inside a request
    ([700] * 6, [0, 6], [640], 127),
    ([2100] * 3, [0, 3], [2048], 64),
    ([900, 20, 800, 850], [0, 4], [768], 16),                # one shorter than the prefix
    ([0, 900, 0, 800, 850, 0], [0, 6], [768], 16),           # padding, the first among them
    ([0] * 5, [0, 5], [64], 16),                             # nothing but padding
    ([600, 610, 5, 0, 1200, 1300, 1250, 77], [1, 2, 2, 4, 7], [500, 64, 3, 1152], 16),  # some in no group
    ([1000] * 40, [0, 13, 26, 40], [900, 640, 963], 8),
    ([1500] * 4, [0, 4], [100000 // 64 * 64], 16),           # shared further than any reaches
    ([320 + i for i in range(33)], [0, 33], [320], 3),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_sms", [2, 9, 152])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_shared_against_the_definition(case, num_sms, fp8):
    import torch
    lens, starts, shared, heads = CASES[case]
    rng = np.random.default_rng(100 + case)
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    if max(shared) > 64 * table.shape[1]:                    # (as long as the block table allows)
        shared = [min(s, 64 * table.shape[1]) for s in shared]
    q = random_q(rng, len(lens), heads)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=num_sms)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _all(lens), SCALE), (case, num_sms, fp8))


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(seed):
    import torch
    rng = np.random.default_rng(9000 + seed)
    B, fp8 = int(rng.integers(1, 24)), bool(rng.integers(2))
    heads = int(rng.choice([1, 2, 3, 7, 8, 16, 24, 33, 64, 65, 96, 128]))
    G = int(rng.integers(0, 4))
    starts = sorted(int(x) for x in rng.integers(0, B + 1, G + 1)) if G else [0]
    if G == 1 and rng.integers(2):
        starts = [0, B]
    shared = [int(rng.choice([0, 64, 130, int(rng.integers(0, 1500))])) for _ in range(G)]
    lens = [int(rng.choice([0, 1, 64, int(rng.integers(0, 400))])) for _ in range(B)]
    for g in range(G):
        for b in range(starts[g], starts[g + 1]):
            if lens[b] and rng.integers(8):
                lens[b] += shared[g]
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    shared = [min(s, 64 * table.shape[1]) for s in shared]
    q = random_q(rng, B, heads, float(rng.choice([0.2, 1.0, 3.0])))
    scale = float(rng.choice([SCALE, -SCALE, 0.0, 0.3]))
    num_sms = int(rng.choice([2, 4, 20, 152]))
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, scale, num_sms)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _all(lens), scale), (seed, lens, starts, shared))


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_that_rise_and_fall(fp8):
    """Row maxima that move by far more than the rescaling threshold, up and
    down, and between the two pages of a step."""
    import torch
    rng = np.random.default_rng(5)
    lens, starts, shared, heads = [1300] * 8, [0, 8], [1024], 16
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, 8, heads, 4.0)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, 1.0, 6)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _all(lens), 1.0))


def test_many_requests_and_groups():
    import torch
    rng = np.random.default_rng(77)
    B, heads = 4096, 1
    sizes, starts = rng.integers(0, 9, 1500), [0]
    for n in sizes:
        starts.append(min(B - 100, starts[-1] + int(n)))
    lens = rng.integers(0, 130, B)
    shared = [64 * int(x) for x in rng.integers(0, 2, len(starts) - 1)]
    cache, table = shared_problem(rng, lens, starts, shared, False)
    table = np.concatenate([table, np.full_like(table, -1)], 1)
    q = random_q(rng, B, heads)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _all(lens), SCALE))


def test_one_request_over_all_pairs():
    """One request of 16 heads: an item in as many pieces as there are pairs."""
    import torch
    rng = np.random.default_rng(6)
    lens, starts, shared = [20000], [0, 1], [19968]
    cache, table = shared_problem(rng, lens, starts, shared, False)
    q = random_q(rng, 1, 16)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _all(lens), SCALE))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_nan_reaches_those_that_see_it_and_no_others(fp8):
    import torch
    rng = np.random.default_rng(8)
    lens, starts, shared, heads = [700] * 6 + [650] * 6, [0, 6, 12], [640, 576], 16
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, 12, heads)
    clean = cache.copy()
    cache[table[2, 10], 3, 100] = NAN[fp8]                   # request 2's own tokens
    cache[table[6, 4], 63, 5] = NAN[fp8]                     # the second group's prefix
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=20)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    hit = np.array([False] * 2 + [True] + [False] * 3 + [True] * 6)
    assert np.isnan(bf16_bits_to_f64(bf16_tensor_bits(out))[hit]).all()
    assert lse.isnan().cpu().numpy()[hit].all()
    keep = np.nonzero(~hit)[0]
    ref = [x[keep] for x in reference(q, clean, table, _all(lens), SCALE)]
    check(out[torch.from_numpy(keep).cuda()], lse[torch.from_numpy(keep).cuda()], ref)


def test_it_equals_the_plain_decode():
    import torch
    rng = np.random.default_rng(3)
    lens, starts, shared = [1500 + 7 * i for i in range(16)], [0, 10, 16], [1472, 1400]
    cache, table = shared_problem(rng, lens, starts, shared, False)
    q = random_q(rng, 16, 32)
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared)
    plain, plain_lse = binding.mla_decode(dev(q), dev(cache), ints(table), ints(lens), SCALE)
    torch.cuda.synchronize()
    ref = reference(q, cache, table, _all(lens), SCALE)
    check(out, lse, ref)
    check(plain, plain_lse, ref)


def test_results_repeat_bit_for_bit_and_the_workspace_keeps_its_bounds():
    import torch
    rng = np.random.default_rng(4)
    lens, starts, shared = [900 + 31 * i for i in range(20)], [0, 9, 20], [832, 896]
    cache, table = shared_problem(rng, lens, starts, shared, False)
    q = random_q(rng, 20, 24)
    plan = binding.make_span_plan(20, 24, table.shape[1], max_groups=2)
    nbytes = int(plan.workspace_bytes)
    store = torch.full((nbytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = store[:nbytes]
    binding.load_library().mla_workspace_init(binding._ptr(ws), nbytes, binding._stream_ptr(None))
    first = run_shared(q, cache, table, lens, starts, shared, plan=plan, ws=ws)[:2]
    store[8192:nbytes] = 0xFF                                # (NaN partials, if any were read)
    for _ in range(3):
        out, lse, _ = run_shared(q, cache, table, lens, starts, shared, plan=plan, ws=ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    torch.cuda.synchronize()
    assert (store[nbytes:] == 0x5A).all()
    assert not ws[:binding.STATUS_BYTES].any()


def test_bad_starts_lengths_and_pages():
    import torch
    rng = np.random.default_rng(12)
    lens, starts, shared = [700] * 8, [0, 8], [640]
    cache, table = shared_problem(rng, lens, starts, shared, False)
    q = random_q(rng, 8, 16)
    ref = reference(q, cache, table, _all(lens), SCALE)

    def run(code, lens=lens, starts=starts, shared=shared, table=table):
        out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=12)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == code
        return out, lse

    for bad in ([0, 9], [-1, 8], [5, 3], [0, 6, 2], [2 ** 31 - 1, 2 ** 31 - 1]):
        check(*run(binding.MLA_ERR_BAD_ROW, starts=bad, shared=[640] * (len(bad) - 1)), ref)
    for bad in (-1, 64 * table.shape[1] + 1, 2 ** 31 - 1):
        check(*run(binding.MLA_ERR_BAD_SEQ_LEN, shared=[bad]), ref)
    for bad in (-5, 64 * table.shape[1] + 1):
        out, lse = run(binding.MLA_ERR_BAD_SEQ_LEN, lens=[700] * 3 + [bad] + [700] * 4)
        want = [x.copy() for x in ref]
        for x, fill in zip(want, (0, -np.inf, 0, 0)):
            x[3] = fill
        check(out, lse, want)
    # a page that is not there: its rows are zeros
    for row, bad in ((0, cache.shape[0]), (0, -1), (5, 2 ** 31 - 1)):
        broken = table.copy()
        col = 3 if row == 0 else 10
        broken[:, col] = bad if row == 0 else broken[:, col]
        broken[row, col] = bad
        zeros = np.concatenate([cache, np.zeros((1, 64, 576), np.uint16)])
        where = np.where(broken == bad, cache.shape[0], broken)
        check(*run(binding.MLA_ERR_BAD_BLOCK_ID, table=broken),
              reference(q, zeros, where, _all(lens), SCALE))


def test_replays_with_other_lengths_and_groups_on_two_streams():
    """Two graphs with a workspace each, captured once and replayed at the same
    time on two streams with other queries, lengths and groups."""
    import torch
    rng = np.random.default_rng(31)
    B, N, M = 12, 16, 30
    calls = []
    for k in range(2):
        plan = binding.make_span_plan(B, N, M, max_groups=3)
        c = dict(plan=plan, ws=binding.new_workspace(plan), stream=torch.cuda.Stream(),
                 q=torch.zeros((B, N, 576), dtype=torch.bfloat16, device="cuda"),
                 cache=torch.zeros((B * M, 64, 576), dtype=torch.bfloat16, device="cuda"),
                 table=torch.zeros((B, M), dtype=torch.int32, device="cuda"), lens=ints([0] * B),
                 starts=ints([0] * 4), shared=ints([0] * 3),
                 out=torch.empty((B, N, 512), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty((B, N), dtype=torch.float32, device="cuda"))
        calls.append(c)

    def call(c):
        binding.mla_decode_shared(c["q"], c["cache"], c["table"], c["lens"], c["starts"], c["shared"],
                                  SCALE, plan=c["plan"], workspace=c["ws"], out=c["out"], lse=c["lse"])

    for c in calls:
        call(c)
        torch.cuda.synchronize()
        c["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c["graph"]):
            call(c)
    for turn in range(3):
        refs = []
        for c in calls:
            starts = sorted(int(x) for x in rng.integers(0, B + 1, 4))
            shared = [64 * int(x) for x in rng.integers(0, 18, 3)]
            lens = [int(x) for x in rng.integers(0, 600, B)]
            for g in range(3):
                for b in range(starts[g], starts[g + 1]):
                    lens[b] += shared[g]
            cache, table = shared_problem(rng, lens, starts, shared, False)
            full = np.full((B, M), -1, dtype=np.int32)
            full[:, :table.shape[1]] = table
            q = random_q(rng, B, N)
            c["cache"][:cache.shape[0]] = dev(cache)
            for name, v in (("q", dev(q)), ("table", ints(full)), ("lens", ints(lens)),
                            ("starts", ints(starts)), ("shared", ints(shared))):
                c[name].copy_(v)
            refs.append(reference(q, cache, table, _all(lens), SCALE))
        torch.cuda.synchronize()
        for c in calls:
            with torch.cuda.stream(c["stream"]):
                c["graph"].replay()
        torch.cuda.synchronize()
        for c, ref in zip(calls, refs):
            assert binding.read_error(c["ws"]) == 0
            check(c["out"], c["lse"], ref, turn)


def test_a_wait_that_runs_out_is_reported():
    """The first CTA withholds a load: the wait for it runs out, the kernel
    drains and returns, and the workspace serves the next call."""
    import torch
    rng = np.random.default_rng(2)
    lens, starts, shared = [700] * 8, [0, 8], [640]
    for fp8 in (False, True):
        cache, table = shared_problem(rng, lens, starts, shared, fp8)
        q = random_q(rng, 8, 16)
        plan = binding.make_span_plan(8, 16, table.shape[1], max_groups=1, num_sms=12)
        bad = binding.make_span_plan(8, 16, table.shape[1], max_groups=1, num_sms=12,
                                     extra_flags=binding.MLA_PLAN_DEBUG_WITHHOLD_LOAD)
        ws = binding.new_workspace(plan)
        run_shared(q, cache, table, lens, starts, shared, plan=bad, ws=ws)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == binding.MLA_ERR_TIMEOUT
        out, lse, _ = run_shared(q, cache, table, lens, starts, shared, plan=plan, ws=ws)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        check(out, lse, reference(q, cache, table, _all(lens), SCALE))


def test_fp8_queries_beyond_f16_are_reported():
    import torch
    rng = np.random.default_rng(13)
    lens, starts, shared = [200] * 3, [0, 3], [128]
    cache, table = shared_problem(rng, lens, starts, shared, True)
    q = random_q(rng, 3, 70)
    q[2, 69, 575] = 0x4780                                   # 65536
    _, _, ws = run_shared(q, cache, table, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == binding.MLA_ERR_RANGE
    q[2, 69, 575] = 0x477F                                   # 65280
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0


def test_no_allocation_is_needed_and_results_may_be_given():
    import torch
    rng = np.random.default_rng(14)
    lens, starts, shared = [300] * 4, [0, 4], [256]
    cache, table = shared_problem(rng, lens, starts, shared, False)
    q = random_q(rng, 4, 16)
    a = (dev(q), dev(cache), ints(table), ints(lens), ints(starts), ints(shared), SCALE)
    side = torch.cuda.Stream()
    out, lse = binding.mla_decode_shared(*a)                 # its own plan and workspace
    torch.cuda.synchronize()
    out2, none = binding.mla_decode_shared(*a, return_lse=False, stream=side)
    torch.cuda.synchronize()
    assert none is None and torch.equal(out, out2)
    check(out, lse, reference(q, cache, table, _all(lens), SCALE))

"""mla_decode_window against the 64-bit definition (tolerances: span_util.py)."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64, bf16_tensor_bits
from oracle import mla_decode_window_reference
from span_util import (K_SCALE, NAN, SCALE, check, dev, ints, random_cache, random_q, reference, run_window, values)

pytestmark = pytest.mark.gpu


def _seen(lens, window, sinks):
    return [np.array([t for t in range(n) if t < sinks or t >= n - window], dtype=np.int64) for n in lens]


def _problem(rng, lens, window, sinks, fp8):
    """A cache in which every row that no request sees is NaN and no page of
    which nothing is seen has a table entry."""
    pages = [sorted({int(t) // 64 for t in s}) for s in _seen(lens, window, sinks)]
    blocks = sum(map(len, pages)) + 2
    ids, at = rng.permutation(blocks), 0
    table = np.full((len(lens), max(1, max(-(-n // 64) for n in lens))), -3, dtype=np.int32)
    cache = random_cache(rng, blocks, fp8)
    keep = np.zeros((blocks, 64), dtype=bool)
    for b, (p, s) in enumerate(zip(pages, _seen(lens, window, sinks))):
        table[b, p] = ids[at:at + len(p)]
        at += len(p)
        keep[table[b, s // 64], s % 64] = True
    cache[~keep] = NAN[fp8]
    return cache, table


LENS = [0, 1, 3, 63, 64, 65, 127, 128, 129, 200, 511, 700, 1030]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_sms", [2, 152])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 64), (63, 4), (64, 0), (64, 64), (65, 1), (100, 65),
                                          (128, 130), (200, 7), (511, 0), (512, 3), (5000, 0), (5, 5000)])
def test_window_against_the_definition(window, sinks, num_sms, fp8):
    import torch
    rng = np.random.default_rng(window * 7 + sinks)
    cache, table = _problem(rng, LENS, window, sinks, fp8)
    q = random_q(rng, len(LENS), 6)
    out, lse, ws = run_window(q, cache, table, LENS, window, sinks, num_sms=num_sms)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _seen(LENS, window, sinks), SCALE))


@pytest.mark.parametrize("seed", range(40))
def test_random_windows(seed):
    import torch
    rng = np.random.default_rng(4000 + seed)
    B, heads = int(rng.integers(1, 20)), int(rng.choice([1, 5, 16, 32, 63, 64, 65, 128]))
    window, sinks = int(np.exp(rng.uniform(0, 7))), int(rng.choice([0, 1, 4, 64, 100, 300]))
    lens = [int(x) for x in np.exp(rng.uniform(0, 8, B))]
    fp8 = bool(rng.integers(2))
    cache, table = _problem(rng, lens, window, sinks, fp8)
    q = random_q(rng, B, heads, float(rng.choice([0.3, 1.0, 3.0])))
    scale = float(rng.choice([SCALE, -SCALE, 0.25]))
    out, lse, ws = run_window(q, cache, table, lens, window, sinks, scale,
                              num_sms=int(rng.choice([2, 6, 30, 152])))
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    check(out, lse, reference(q, cache, table, _seen(lens, window, sinks), scale), (seed, window, sinks, lens))


def test_the_oracle_agrees_with_the_reference_of_these_tests():
    import torch
    rng = np.random.default_rng(1)
    lens = [300, 40]
    cache, table = _problem(rng, lens, 50, 5, False)
    q = random_q(rng, 2, 3)
    out, lse, ws = run_window(q, cache, table, lens, 50, 5)
    torch.cuda.synchronize()
    ref = mla_decode_window_reference(bf16_bits_to_f64(q), values(cache), table, lens, SCALE, 50, 5)
    mine = reference(q, cache, table, _seen(lens, 50, 5), SCALE)
    assert np.allclose(ref[0], mine[0], rtol=0, atol=1e-12) and np.allclose(ref[1], mine[1])
    check(out, lse, mine)


def test_a_window_past_every_length_is_the_plain_decode():
    import torch
    rng = np.random.default_rng(2)
    lens = [100, 1000, 5, 0]
    cache, table = _problem(rng, lens, 1000, 0, False)
    q = random_q(rng, 4, 16)
    ref = reference(q, cache, table, [np.arange(n) for n in lens], SCALE)
    for window, sinks in ((1000, 0), (2 ** 31 - 1, 0), (2 ** 40, 2 ** 40), (1, 2 ** 31 - 1)):
        out, lse, ws = run_window(q, cache, table, lens, window, sinks)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        check(out, lse, ref)


def test_infinities_that_are_not_seen_do_not_matter_and_seen_ones_do():
    import torch
    rng = np.random.default_rng(3)
    lens, window, sinks = [500, 500], 100, 70
    cache, table = _problem(rng, lens, window, sinks, False)
    cache[cache == NAN[False]] = 0x7F80                      # +inf
    q = random_q(rng, 2, 16)
    ref = reference(q, cache, table, _seen(lens, window, sinks), SCALE)
    out, lse, ws = run_window(q, cache, table, lens, window, sinks)
    torch.cuda.synchronize()
    check(out, lse, ref)
    cache[table[1, 0], 69 % 64, 3] = 0x7F80                  # token 5 of request 1, a value column
    out, lse, ws = run_window(q, cache, table, lens, window, sinks)
    torch.cuda.synchronize()
    assert not np.isfinite(bf16_bits_to_f64(bf16_tensor_bits(out))[1, :, 3]).any()
    check(out[:1], lse[:1], [x[:1] for x in ref])


def test_bad_pages_and_lengths_are_recorded():
    import torch
    rng = np.random.default_rng(4)
    lens, window, sinks = [500, 300], 100, 4
    cache, table = _problem(rng, lens, window, sinks, False)
    q = random_q(rng, 2, 16)
    broken = table.copy()
    broken[0, 7] = cache.shape[0]
    out, lse, ws = run_window(q, cache, broken, lens, window, sinks)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    zeros = np.concatenate([cache, np.zeros((1, 64, 576), np.uint16)])
    check(out, lse, reference(q, zeros, broken, _seen(lens, window, sinks), SCALE))
    for bad in (-1, 64 * table.shape[1] + 1):
        out, lse, ws = run_window(q, cache, table, [500, bad], window, sinks)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == binding.MLA_ERR_BAD_SEQ_LEN
        check(out, lse, reference(q, cache, table, _seen([500, 0], window, sinks), SCALE))


def test_pages_past_two_to_the_31():
    """Pages whose entries lie past 2^31 elements of the pool, bf16 and fp8."""
    import torch
    rng = np.random.default_rng(9)
    lens, heads, blocks = [150], 16, 60000
    for fp8 in (False, True):
        small = random_cache(rng, 3, fp8)
        pool = torch.zeros((blocks, 64, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        ids = [blocks - 1, 58300, 2]
        from span_util import K_SCALE, dev, ints
        pool[torch.tensor(ids, device="cuda")] = dev(small)
        q = random_q(rng, 1, heads)
        args = (dev(q), pool, ints([ids]), ints(lens), SCALE)
        out, lse = (binding.mla_decode_window_fp8(*args, K_SCALE, window=140, sinks=2) if fp8
                    else binding.mla_decode_window(*args, window=140, sinks=2))
        torch.cuda.synchronize()
        check(out, lse, reference(q, small, np.array([[0, 1, 2]]), _seen(lens, 140, 2), SCALE))
        del pool


def test_replays_with_other_lengths_at_the_same_time():
    """Two captured calls, a workspace each, replayed together on two streams."""
    import torch
    rng = np.random.default_rng(8)
    B, N, M, window, sinks = 5, 16, 12, 200, 66
    calls = []
    for k in range(2):
        plan = binding.make_span_plan(B, N, M)
        c = dict(plan=plan, ws=binding.new_workspace(plan), stream=torch.cuda.Stream(),
                 q=torch.zeros((B, N, 576), dtype=torch.bfloat16, device="cuda"),
                 table=torch.zeros((B, M), dtype=torch.int32, device="cuda"), lens=ints([0] * B),
                 out=torch.empty((B, N, 512), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty((B, N), dtype=torch.float32, device="cuda"))
        calls.append(c)
    host = random_cache(rng, B * M, False)
    cache = dev(host)

    def call(c):
        binding.mla_decode_window(c["q"], cache, c["table"], c["lens"], SCALE, window=window, sinks=sinks,
                                  plan=c["plan"], workspace=c["ws"], out=c["out"], lse=c["lse"])

    for c in calls:
        call(c)
        torch.cuda.synchronize()
        c["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c["graph"]):
            call(c)
    for turn in range(3):
        refs = []
        for c in calls:
            lens, q = rng.integers(0, 64 * M + 1, B), random_q(rng, B, N)
            table = rng.permutation(B * M).reshape(B, M)
            c["q"].copy_(dev(q)), c["lens"].copy_(ints(lens)), c["table"].copy_(ints(table))
            refs.append(reference(q, host, table, _seen(lens, window, sinks), SCALE))
        torch.cuda.synchronize()
        for c in calls:
            with torch.cuda.stream(c["stream"]):
                c["graph"].replay()
        torch.cuda.synchronize()
        for c, ref in zip(calls, refs):
            assert binding.read_error(c["ws"]) == 0
            check(c["out"], c["lse"], ref, turn)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_wait_that_runs_out_is_reported(fp8):
    """The first CTA withholds a load: the wait for it runs out, the kernel
    drains and returns, and the workspace serves the next call."""
    import torch
    rng = np.random.default_rng(3)
    lens, window, sinks = [900, 40, 300], 400, 10
    host, table = random_cache(rng, 30, fp8), rng.permutation(30).reshape(2, 15)
    table = np.concatenate([table, table[:1, ::-1]])
    q = random_q(rng, 3, 16)
    bad = binding.make_span_plan(3, 16, 15, num_sms=4, extra_flags=binding.MLA_PLAN_DEBUG_WITHHOLD_LOAD)
    plan = binding.make_span_plan(3, 16, 15, num_sms=4)
    ws = binding.new_workspace(plan)
    for p, status in ((bad, binding.MLA_ERR_TIMEOUT), (plan, 0)):
        args = (dev(q), dev(host), ints(table), ints(lens), SCALE)
        if fp8:
            out, lse = binding.mla_decode_window_fp8(*args, K_SCALE, window=window, sinks=sinks, plan=p,
                                                     workspace=ws)
        else:
            out, lse = binding.mla_decode_window(*args, window=window, sinks=sinks, plan=p, workspace=ws)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == status
    check(out, lse, reference(q, host, table, _seen(lens, window, sinks), SCALE))

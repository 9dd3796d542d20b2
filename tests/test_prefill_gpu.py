"""Expanded-form attention (mla_prefill) against the 64-bit definition.

Tolerances, per output element with w_j the exact softmax weights and
A = sum_j w_j |v_j|:
  * a score is a sum of 192 exact products in fp32: off by at most
    d = scale * 192 * 2^-23 * max_j sum |q k_j| (a whole step counted per
    addition), plus 2^-22 of itself for scaling; every weight by 2 d + 2^-20
    (the exponential's own error and the sum's included);
  * a weight is rounded to bf16 once (2^-8 of it), the result once (2^-8).
So |out - exact| <= 2^-8 |exact| + (2^-8 + 2 d + 2^-20) A (1 + 2^-7), and the
LSE is off by at most d + 2^-20 (1 + |lse|). Split partials are fp32.
"""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import (bf16_bits_to_f64, bf16_tensor_bits,
                                                    f32_to_bf16_bits)
from oracle import prefill_attention

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
FILL = 0x1234


def _bf16(rng, shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _dev(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _int(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _problem(seed, q_lens, k_lens, heads, q_scale=1.0):
    rng = np.random.default_rng(seed)
    return (_bf16(rng, (sum(q_lens), heads, 192), q_scale), _bf16(rng, (sum(k_lens), heads, 256)),
            _bf16(rng, (sum(k_lens), 64)))


def _run(q, kv, pe, q_lens, k_lens, causal, splits=0, spare=0, scale=SCALE, max_q=None, **kw):
    """(out bits, lse) of one call; `spare` rows follow the last sequence.
    `max_q` (the plan's longest query length) picks the kernel: 1 the CUDA-core
    kernel for single rows, more the tensor cores'."""
    import torch
    heads = kv.shape[1]
    if spare:
        q = np.concatenate([q, np.full((spare, heads, 192), 0x7FC0, np.uint16)])
        kv = np.concatenate([kv, np.full((spare, heads, 256), 0x7FC0, np.uint16)])
        pe = np.concatenate([pe, np.full((spare, 64), 0x7FC0, np.uint16)])
    out = _dev(np.full((q.shape[0], heads, 128), FILL, np.uint16))
    lse = torch.full((q.shape[0], heads), 77.0, device="cuda")
    plan = binding.make_prefill_plan(len(q_lens), heads, q.shape[0],
                                     max(q_lens, default=0) if max_q is None else max_q,
                                     max(k_lens, default=0), num_kv_splits=splits)
    assert plan.single_rows == ((max(q_lens, default=0) if max_q is None else max_q) <= 1)
    ws = binding.new_workspace(plan)
    binding.mla_prefill(_dev(q), _dev(kv), _dev(pe), _int(_starts(q_lens)), _int(_starts(k_lens)),
                        scale, causal=causal, plan=plan, workspace=ws, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    bits, z = bf16_tensor_bits(out), lse.cpu().numpy().astype(np.float64)
    n = sum(q_lens)
    assert (bits[n:] == FILL).all() and (z[n:] == 77.0).all()
    return bits[:n], z[:n]


def _check(bits, lse, q, kv, pe, q_lens, k_lens, causal, scale=SCALE):
    q, kv, pe = (bf16_bits_to_f64(x) for x in (q, kv, pe))
    ref, z = prefill_attention(q, kv, pe, q_lens, k_lens, scale, causal)
    kv_abs = np.concatenate([kv[..., :128], np.abs(kv[..., 128:])], -1)
    size, _ = prefill_attention(q, kv_abs, pe, q_lens, k_lens, scale, causal)
    norm_k = np.sqrt((kv[..., :128] ** 2).sum(-1) + (pe ** 2).sum(-1)[:, None])
    top_k = norm_k.max(0) if norm_k.shape[0] else np.zeros(kv.shape[1])
    d = scale * 192 * 2.0 ** -23 * np.sqrt((q ** 2).sum(-1)) * top_k      # >= sum |q k|
    got = bf16_bits_to_f64(bits)
    tol = 2.0 ** -8 * np.abs(ref) + \
        (2.0 ** -8 + 2 * d + 2.0 ** -20)[..., None] * size * (1 + 2.0 ** -7)
    err = np.abs(got - ref)
    assert not np.isnan(got).any()
    assert (err <= tol + 1e-30).all(), f"worst {np.max(err / np.maximum(tol, 1e-30))} of the tolerance"
    none = np.isneginf(z)
    assert np.array_equal(np.isneginf(lse), none) and (bits[none] == 0).all()
    assert (np.abs(lse[~none] - z[~none]) <= (d + 2.0 ** -20 * (1 + np.abs(z)))[~none]).all()


CASES = [
    # q lengths, k lengths, heads
    ([1], [1], 1),
    ([1], [129], 3),
    ([2], [1], 2),                       # causal: the first query sees nothing
    ([64], [64], 2),
    ([128], [128], 1),
    ([129], [129], 2),
    ([256], [256], 1),
    ([257], [300], 2),
    ([300], [40], 1),                    # 260 rows see nothing
    ([5, 0, 7, 1], [5, 3, 20, 0], 4),
    ([0, 0], [0, 10], 1),
    ([1] * 40, list(range(1, 400, 10)), 2),
    ([130, 1, 255, 70], [700, 513, 256, 71], 3),
    ([513], [513], 2),
    ([17], [2000], 5),
    ([33, 90], [128, 384], 16),
    ([3], [260], 128),
    ([3, 2], [0, 0], 2),                 # no keys at all
]


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_prefill_against_the_oracle(case, causal, max_q):
    q_lens, k_lens, heads = CASES[case]
    q, kv, pe = _problem(700 + case, q_lens, k_lens, heads)
    bits, lse = _run(q, kv, pe, q_lens, k_lens, causal, spare=5, max_q=max_q)
    _check(bits, lse, q, kv, pe, q_lens, k_lens, causal)


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [2, 5, 8, 9, 12, 14])
def test_prefill_with_split_keys(case, causal, splits, max_q):
    q_lens, k_lens, heads = CASES[case]
    q, kv, pe = _problem(800 + case, q_lens, k_lens, heads, q_scale=2.0)
    bits, lse = _run(q, kv, pe, q_lens, k_lens, causal, splits=splits, spare=3, max_q=max_q)
    _check(bits, lse, q, kv, pe, q_lens, k_lens, causal)


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("order", ["rising", "falling", "far below"])
def test_prefill_as_the_reference_maximum_moves(order, splits, max_q):
    """Scores that climb by far more than the rescale threshold step after
    step, that only fall, and that are all far below zero."""
    rng = np.random.default_rng(31)
    n, heads = 700, 2
    direction = rng.standard_normal((heads, 192))
    direction /= np.linalg.norm(direction, axis=-1, keepdims=True)
    height = np.linspace(-20, 90, n) if order == "rising" else \
        np.linspace(90, -20, n) if order == "falling" else np.full(n, -400.0)
    pe = rng.standard_normal((n, 64)) * 0.1
    kv = rng.standard_normal((n, heads, 256))
    kv[..., :128] = 0.1 * kv[..., :128] + height[:, None, None] * direction[None, :, :128]
    q = np.repeat(direction[None], 200, 0) * rng.uniform(10, 20, (200, 1, 1))
    q, kv, pe = (f32_to_bf16_bits(x.astype(np.float32)) for x in (q, kv, pe))
    bits, lse = _run(q, kv, pe, [200], [n], True, splits=splits, max_q=max_q)
    _check(bits, lse, q, kv, pe, [200], [n], True)


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_what_a_query_does_not_see_does_not_reach_it(value, splits, max_q):
    """Non-finite keys and values at positions from `at` on: queries before
    `at` keep their results bit for bit, later ones see them."""
    q_lens, k_lens, heads = [300, 200], [420, 200], 2
    q, kv, pe = _problem(41, q_lens, k_lens, heads)
    clean, clean_lse = _run(q, kv, pe, q_lens, k_lens, True, splits=splits, max_q=max_q)
    bad = f32_to_bf16_bits(np.array([value], dtype=np.float32))[0]
    starts_q, starts_k = _starts(q_lens), _starts(k_lens)
    for seq, at, col in [(0, 419, 130), (0, 300, 255), (1, 0, 128), (1, 77, 200), (0, 130, 180)]:
        x = kv.copy()
        x[starts_k[seq] + at, 1, col] = bad
        got, lse = _run(q, x, pe, q_lens, k_lens, True, splits=splits, max_q=max_q)
        want = bf16_bits_to_f64(clean).copy()
        rows = starts_q[seq] + max(0, at - (k_lens[seq] - q_lens[seq]))
        want[rows:starts_q[seq + 1], 1, col - 128] = value
        assert np.array_equal(bf16_bits_to_f64(got), want, equal_nan=True), (seq, at, col)
        assert np.array_equal(lse, clean_lse)
    # keys: the whole row of scores; every later query is NaN or ignores it
    x, y = kv.copy(), pe.copy()
    x[starts_k[0] + 400, 0, 5] = 0x7FC0
    y[starts_k[1] + 190, 3] = 0x7FC0
    got, lse = _run(q, x, y, q_lens, k_lens, True, splits=splits, max_q=max_q)
    keep = np.ones((500, 2), dtype=bool)
    keep[280:300, 0] = False
    keep[490:500, :] = False
    assert np.array_equal(got[keep], clean[keep]) and np.array_equal(lse[keep], clean_lse[keep])
    assert np.isnan(bf16_bits_to_f64(got)[~keep]).all() and np.isnan(lse[~keep]).all()
    # queries: their own rows only
    x = q.copy()
    x[100, 1, 7] = 0x7FC0
    got, lse = _run(x, kv, pe, q_lens, k_lens, True, splits=splits, max_q=max_q)
    keep = np.ones((500, 2), dtype=bool)
    keep[100, 1] = False
    assert np.array_equal(got[keep], clean[keep])
    assert np.isnan(bf16_bits_to_f64(got)[100, 1]).all()


@pytest.mark.parametrize("max_q", [1, 1000])
def test_both_infinities_seen_give_nan(max_q):
    q, kv, pe = _problem(42, [10], [140], 1)
    kv[135, 0, 128 + 9], kv[138, 0, 128 + 9] = 0x7F80, 0xFF80
    bits, _ = _run(q, kv, pe, [10], [140], True, max_q=max_q)
    col = bf16_bits_to_f64(bits)[:, 0, 9]
    assert np.isfinite(col[:5]).all() and (col[5:8] == np.inf).all() and np.isnan(col[8:]).all()


@pytest.mark.parametrize("max_q", [1, 1000])
def test_scores_of_the_lowest_value(max_q):
    """A key of the type's lowest value gives scores of -inf or near it: its
    weight is 0; a row that sees nothing else has no sum."""
    q, kv, pe = _problem(43, [4], [4], 1)
    q[:, 0, 0] = 0x7F7F                    # the largest finite bf16
    kv[:2, 0, 0] = 0xFF7F
    bits, lse = _run(q, kv, pe, [4], [4], True, max_q=max_q)
    assert np.isneginf(lse[:2, 0]).all() and (bits[:2] == 0).all()
    assert not np.isneginf(lse[2:, 0]).any()


def test_prefill_is_deterministic_and_replays_in_a_graph():
    import torch
    q_lens, k_lens, heads = [300, 77, 1], [300, 500, 900], 4
    q, kv, pe = _problem(51, q_lens, k_lens, heads)
    args = (_dev(q), _dev(kv), _dev(pe), _int(_starts(q_lens)), _int(_starts(k_lens)))
    for splits, max_q in ((1, 300), (4, 300), (1, 1), (4, 1)):
        plan = binding.make_prefill_plan(3, heads, sum(q_lens), max_q, 900, num_kv_splits=splits)
        ws = binding.new_workspace(plan)
        out, lse = binding.mla_prefill(*args, SCALE, plan=plan, workspace=ws)
        torch.cuda.synchronize()
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            binding.mla_prefill(*args, SCALE, plan=plan, workspace=ws, out=out2, lse=lse2,
                                stream=stream)
        for _ in range(3):
            out2.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert binding.read_error(ws) == 0
            assert torch.equal(out2.view(torch.int16), out.view(torch.int16))
            assert torch.equal(lse2, lse)


def test_prefill_on_two_streams_at_once():
    import torch
    problems = []
    for seed in (61, 62):
        q, kv, pe = _problem(seed, [400], [600], 4)
        plan = binding.make_prefill_plan(1, 4, 400, 400, 600, num_kv_splits=2)
        stream = torch.cuda.Stream()
        problems.append(((q, kv, pe), (_dev(q), _dev(kv), _dev(pe), _int([0, 400]), _int([0, 600])),
                         plan, binding.new_workspace(plan), stream))
    torch.cuda.synchronize()
    results = [binding.mla_prefill(*args, SCALE, plan=plan, workspace=ws, stream=stream)
               for _ in range(4) for _, args, plan, ws, stream in problems]
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(results):
        q, kv, pe = problems[i % 2][0]
        if i >= 6:
            _check(bf16_tensor_bits(out), lse.cpu().numpy().astype(np.float64), q, kv, pe, [400],
                   [600], True)
        assert torch.equal(out, results[i % 2][0])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("splits", [1, 2, 3, 8])
def test_many_items_of_few_steps(splits, causal):
    """Several items per SM, many without steps of their own: the loads wait
    for an item between two steps, and every split gives the same result."""
    import torch
    rng = np.random.default_rng(5)
    q_lens = [int(x) for x in rng.integers(2, 700, 24)]
    k_lens = [n + (0 if b % 3 else int(rng.integers(0, 900))) for b, n in enumerate(q_lens)]
    heads = 16
    q, kv, pe = _problem(55, q_lens, k_lens, heads)
    args = (_dev(q), _dev(kv), _dev(pe), _int(_starts(q_lens)), _int(_starts(k_lens)))
    ref, ref_lse = None, None
    plan = binding.make_prefill_plan(24, heads, sum(q_lens), max(q_lens), max(k_lens),
                                     num_kv_splits=splits)
    ws = binding.new_workspace(plan)
    for _ in range(30):
        out, lse = binding.mla_prefill(*args, SCALE, causal=causal, plan=plan, workspace=ws)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        if ref is None:
            ref, ref_lse = out, lse
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    # three of the sequences and two heads against the definition
    bits, z = bf16_tensor_bits(ref), ref_lse.cpu().numpy().astype(np.float64)
    starts_q, starts_k = _starts(q_lens), _starts(k_lens)
    for b in (0, 9, 23):
        rq, rk = slice(starts_q[b], starts_q[b + 1]), slice(starts_k[b], starts_k[b + 1])
        _check(bits[rq, 3:5], z[rq, 3:5], q[rq, 3:5], kv[rk, 3:5], pe[rk], [q_lens[b]],
               [k_lens[b]], causal)


@pytest.mark.parametrize("max_q", [1, 1000])
def test_prefill_of_many_short_sequences(max_q):
    rng = np.random.default_rng(6)
    q_lens = [int(x) for x in rng.integers(0, 4, 700)]
    k_lens = [int(x) for x in rng.integers(0, 40, 700)]
    q, kv, pe = _problem(56, q_lens, k_lens, 2)
    bits, lse = _run(q, kv, pe, q_lens, k_lens, True, max_q=max_q, spare=2)
    _check(bits, lse, q, kv, pe, q_lens, k_lens, True)


@pytest.mark.parametrize("max_q", [1, 1000])
def test_prefill_behind_the_first_2_31_elements(max_q):
    """kv of 70,000 tokens x 128 heads x 256: the last sequence lies past 2^31
    elements; the first takes the rest as keys that are not looked at here."""
    import torch
    heads, lk, lq = 128, 70000, 3
    kv = torch.zeros((lk, heads, 256), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((lk, 64), dtype=torch.bfloat16, device="cuda")
    q, kv_end, pe_end = _problem(57, [lq], [200], heads)
    kv[-200:], pe[-200:] = _dev(kv_end), _dev(pe_end)
    plan = binding.make_prefill_plan(2, heads, lq, max_q, 200)
    ws = binding.new_workspace(plan)
    out, lse = binding.mla_prefill(_dev(q), kv, pe, _int([0, 0, lq]), _int([0, lk - 200, lk]),
                                   SCALE, plan=plan, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    _check(bf16_tensor_bits(out), lse.cpu().numpy().astype(np.float64), q, kv_end, pe_end, [lq],
           [200], True)


def test_prefill_without_lse_plan_and_workspace():
    q, kv, pe = _problem(71, [50], [60], 2)
    out, lse = binding.mla_prefill(_dev(q), _dev(kv), _dev(pe), _int([0, 50]), _int([0, 60]), SCALE,
                                   return_lse=False)
    assert lse is None
    bits, z = _run(q, kv, pe, [50], [60], True)
    assert np.array_equal(bf16_tensor_bits(out), bits)


def test_prefill_with_starts_that_make_no_sense():
    """Such a sequence has no rows, or no keys; the others keep theirs."""
    import torch
    q, kv, pe = _problem(81, [20, 20], [30, 30], 2)
    good, good_lse = _run(q, kv, pe, [20, 20], [30, 30], True)
    for cu_q, cu_k, what in [([0, 20, 41], [0, 30, 60], "rows"), ([0, 20, 10], [0, 30, 60], "rows"),
                             ([0, 20, 40], [0, 30, 61], "keys"), ([0, 20, 40], [0, 30, 29], "keys")]:
        plan = binding.make_prefill_plan(2, 2, 40, 40, 60)
        ws = binding.new_workspace(plan)
        out = _dev(np.full((40, 2, 128), FILL, np.uint16))
        _, lse = binding.mla_prefill(_dev(q), _dev(kv), _dev(pe), _int(cu_q), _int(cu_k), SCALE,
                                     plan=plan, workspace=ws, out=out)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == binding.MLA_ERR_BAD_SEQ_LEN
        bits = bf16_tensor_bits(out)
        assert np.array_equal(bits[:20], good[:20])
        assert (bits[20:] == (FILL if what == "rows" else 0)).all()


def test_prefill_refuses_tensors_that_do_not_fit():
    import torch
    q, kv, pe = (_dev(x) for x in _problem(91, [10], [10], 2))
    cu = _int([0, 10])
    ok = dict(q=q, kv=kv, k_pe=pe, cu_seqlens_q=cu, cu_seqlens_k=cu, softmax_scale=SCALE)
    for kw, exc in [(dict(q=q.half()), TypeError), (dict(q=q[:, :, :128]), ValueError),
                    (dict(kv=kv[:, :1]), ValueError), (dict(kv=kv.float()), TypeError),
                    (dict(k_pe=pe[:5]), ValueError), (dict(cu_seqlens_k=cu[:1]), ValueError),
                    (dict(cu_seqlens_q=cu.long()), TypeError), (dict(q=q.cpu()), TypeError),
                    (dict(softmax_scale=0.0), binding.MlaError),
                    (dict(softmax_scale=float("nan")), binding.MlaError),
                    (dict(plan=binding.make_prefill_plan(1, 2, 11, 11, 10)), ValueError),
                    (dict(out=torch.empty(10 * 2 * 128 + 8, dtype=torch.bfloat16,
                                          device="cuda")[8:].view(10, 2, 128)), binding.MlaError)]:
        with pytest.raises(exc):
            binding.mla_prefill(**{**ok, **kw})


REST = [
    # q lengths, k lengths, heads, SMs of the plan (so the waves); items, those left over
    ([300], [2300], 3, 5),                             # 6, 1
    ([256], [2048], 5, 3),                             # 5, 2
    ([129, 200, 70], [2500, 2200, 2049], 2, 4),        # 6, 2 of three sequences
    ([600, 3], [2600, 90], 2, 7),                      # 8, 1 of the short ones
    ([70, 0, 300, 5], [2100, 10, 0, 700], 3, 8),       # 12, 4, some without keys
    ([255], [2050], 31, 16),                           # 31, 15: nearly a wave
    ([256], [2048], 8, 4),                             # 8, none
    ([2], [700], 4, 9),                                # 4: less than a wave
]


@pytest.mark.parametrize("splits", [2, 7])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(REST)))
def test_only_the_last_wave_is_split(case, causal, splits):
    import torch
    q_lens, k_lens, heads, sms = REST[case]
    q, kv, pe = _problem(900 + case, q_lens, k_lens, heads, q_scale=2.0)
    n, spare = sum(q_lens), 4
    plan = binding.make_prefill_plan(len(q_lens), heads, n + spare, max(q_lens), max(k_lens),
                                     num_sms=sms, num_kv_splits=splits)
    plan.split_rest = 1
    out = _dev(np.full((n + spare, heads, 128), FILL, np.uint16))
    lse = torch.full((n + spare, heads), 77.0, device="cuda")
    ws = binding.new_workspace(plan)
    ws[binding.STATUS_BYTES:].fill_(0xA5)              # what an earlier call left behind
    q_all = _dev(np.concatenate([q, np.full((spare, heads, 192), 0x7FC0, np.uint16)]))
    args = (q_all, _dev(kv), _dev(pe), _int(_starts(q_lens)), _int(_starts(k_lens)), SCALE)
    for _ in range(2):                                 # and this call itself
        binding.mla_prefill(*args, causal=causal, plan=plan, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    bits, z = bf16_tensor_bits(out), lse.cpu().numpy().astype(np.float64)
    assert (bits[n:] == FILL).all() and (z[n:] == 77.0).all()
    _check(bits[:n], z[:n], q, kv, pe, q_lens, k_lens, causal)
    again = binding.mla_prefill(*args, causal=causal, plan=plan, workspace=ws, return_lse=False)
    assert again[1] is None
    assert torch.equal(again[0][:n].view(torch.int16), out[:n].view(torch.int16))


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_split_and_whole_rows_with_values_that_are_not_finite(value):
    """A result that is NaN is not taken for the mark of a row that was not split."""
    import torch
    q, kv, pe = _problem(920, [300], [2300], 3)
    kv[5, 1, 128:] = 0x7FC0 if np.isnan(value) else 0x7F80
    kv[7, 2, 0] = kv[9, 0, 3] = 0x7FC0
    want = None
    for sms, split in ((5, 1), (152, 0)):
        plan = binding.make_prefill_plan(1, 3, 300, 300, 2300, num_sms=sms,
                                         num_kv_splits=4 if split else 1)
        plan.split_rest = split
        ws = binding.new_workspace(plan)
        out, lse = binding.mla_prefill(_dev(q), _dev(kv), _dev(pe), _int([0, 300]), _int([0, 2300]),
                                       SCALE, plan=plan, workspace=ws)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        got = (torch.isnan(out), torch.isinf(out), torch.isnan(lse))
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
    # (each query sees key 7 and key 9: heads 0 and 2 are NaN; head 1 is what its value is)
    nan, inf, nan_z = want
    assert nan[:, [0, 2]].all() and nan_z[:, [0, 2]].all() and not nan_z[:, 1].any()
    assert (nan if np.isnan(value) else inf)[:, 1].all()


def test_new_results_are_ordinary_tensors(monkeypatch):
    """Allocated either way, with and without rows: contiguous, of the stated
    type and shape, and the same bits."""
    import torch
    q, kv, pe = _problem(930, [5], [9], 2)
    args = (_dev(q), _dev(kv), _dev(pe), _int([0, 5]), _int([0, 9]), SCALE)
    got = [binding.mla_prefill(*args)]
    assert binding._empty_strided is not None
    monkeypatch.setitem(__import__("sys").modules, "torch._C._dynamo.guards", None)
    monkeypatch.setattr(binding, "_empty_strided", None)
    got.append(binding.mla_prefill(*args))
    got.append(binding.mla_prefill(*args, stream=torch.cuda.current_stream()))
    none = binding.mla_prefill(_dev(q[:0]), _dev(kv), _dev(pe), _int([0, 0]), _int([0, 9]), SCALE)
    for out, lse in got:
        assert out.shape == (5, 2, 128) and out.dtype == torch.bfloat16 and out.is_contiguous()
        assert lse.shape == (5, 2) and lse.dtype == torch.float32 and lse.is_contiguous()
        assert out.device == args[0].device and torch.equal(out, got[0][0])
        assert torch.equal(lse, got[0][1])
    assert none[0].shape == (0, 2, 128) and none[1].shape == (0, 2)

"""Expansion of paged latent rows into keys and values, against the 64-bit definition.

Tolerance. An output is a sum of 512 products of bf16 (or E4M3) numbers, exact
in fp32, accumulated in fp32 and rounded once to bf16: at most half a bf16 step
(2^-8 of the value) from the rounded exact value, plus the fp32 accumulation's
error, at most 512 * 2^-23 of the sum of the products' magnitudes (the tensor
cores may truncate, so a whole step is counted for each addition). k_pe of a
bf16 cache is copied, that of an fp8 cache rounded once.
"""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import (bf16_bits_to_f64, bf16_tensor_bits,
                                                    f32_to_bf16_bits)
from oracle import e4m3_to_float, expand_kv

pytestmark = pytest.mark.gpu


def _bf16(rng, shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _dev(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _int(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _problem(rng, lens, first, heads, fp8, extra=2):
    held = [a + b for a, b in zip(lens, first)]
    pages = [-(-n // 64) for n in held]
    blocks = sum(pages) + extra
    ids = rng.permutation(blocks)
    table = np.full((len(lens), max(1, max(pages))), 2 ** 30, dtype=np.int32)
    at = 0
    if fp8:
        cache = rng.integers(0, 256, (blocks, 64, 576), dtype=np.uint8)
        cache[(cache & 0x7F) == 0x7F] = 0x7E
    else:
        cache = _bf16(rng, (blocks, 64, 576))
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
        if held[b] % 64:           # rows past the request's end hold NaN
            cache[table[b, n - 1], held[b] % 64:] = 0x7F if fp8 else 0x7FC0
    w_uk = _bf16(rng, (heads, 128, 512), 512 ** -0.5)
    w_uv = _bf16(rng, (heads, 512, 128), 512 ** -0.5)
    return cache, table, w_uk, w_uv


def _check(got_kv, got_pe, cache, k_scale, table, first, lens, w_uk, w_uv, fp8):
    values = e4m3_to_float(cache) * k_scale if fp8 else bf16_bits_to_f64(cache)
    uk, uv = bf16_bits_to_f64(w_uk), bf16_bits_to_f64(w_uv)
    ref, pe = expand_kv(values, table, first, lens, uk, uv)
    size, _ = expand_kv(np.abs(values), table, first, lens, np.abs(uk), np.abs(uv))
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + 512 * 2.0 ** -23 * size
    err = np.abs(got_kv - ref)
    assert not (err > tol).any(), f"worst {np.nanmax(err / tol)} of the tolerance"
    assert not np.isnan(got_kv).any()
    if fp8:
        assert (np.abs(got_pe - pe) <= 2.0 ** -8 * np.abs(pe)).all()
    else:
        assert np.array_equal(got_pe, pe)


CASES = [([1], [0], 1), ([64], [0], 2), ([128], [1], 1), ([129], [0], 3), ([5, 0, 7], [60, 3, 0], 16),
         ([256], [0], 2), ([257], [63], 1), ([300, 1, 500], [0, 640, 65], 5), ([1000], [17], 8),
         ([0, 0, 3], [0, 0, 0], 1), ([40] * 33, list(range(33)), 4), ([70], [10], 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_expand_against_the_oracle(case, fp8):
    import torch
    lens, first, heads = CASES[case]
    rng = np.random.default_rng(500 + case)
    cache, table, w_uk, w_uv = _problem(rng, lens, first, heads, fp8)
    total, spare = sum(lens), 3
    kv = _dev(np.full((total + spare, heads, 256), 0x1234, np.uint16))
    pe = _dev(np.full((total + spare, 64), 0x1234, np.uint16))
    ws = binding.new_status_workspace()
    cu = np.concatenate([[0], np.cumsum(lens)])
    kw = dict(total_k=total + spare, workspace=ws, kv=kv, k_pe=pe, first_token=_int(first))
    k_scale = 0.037109375
    if fp8:
        binding.mla_expand_kv_fp8(torch.from_numpy(cache).cuda(), _int(table), _int(cu), _dev(w_uk),
                                  _dev(w_uv), k_scale, **kw)
    else:
        binding.mla_expand_kv(_dev(cache), _int(table), _int(cu), _dev(w_uk), _dev(w_uv), **kw)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    kv_bits, pe_bits = bf16_tensor_bits(kv), bf16_tensor_bits(pe)
    assert (kv_bits[total:] == 0x1234).all() and (pe_bits[total:] == 0x1234).all()
    _check(bf16_bits_to_f64(kv_bits[:total]), bf16_bits_to_f64(pe_bits[:total]), cache, k_scale,
           table, first, lens, w_uk, w_uv, fp8)


def test_expand_without_first_tokens_and_on_a_side_stream():
    import torch
    rng = np.random.default_rng(9)
    lens = [200, 31]
    cache, table, w_uk, w_uv = _problem(rng, lens, [0, 0], 4, False)
    ws = binding.new_status_workspace()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    args = (_dev(cache), _int(table), _int([0, 200, 231]), _dev(w_uk), _dev(w_uv))
    torch.cuda.synchronize()
    kv, pe = binding.mla_expand_kv(*args, total_k=231, workspace=ws, stream=stream)
    stream.synchronize()
    assert binding.read_error(ws) == 0
    _check(bf16_bits_to_f64(bf16_tensor_bits(kv)), bf16_bits_to_f64(bf16_tensor_bits(pe)), cache,
           1.0, table, [0, 0], lens, w_uk, w_uv, False)


@pytest.mark.parametrize("what", ["page", "negative", "past", "first"])
def test_expand_of_bad_pages_gives_zeros_and_an_error(what):
    import torch
    rng = np.random.default_rng(10)
    lens, first = [150, 90], [0, 0]
    cache, table, w_uk, w_uv = _problem(rng, lens, first, 2, False)
    code = binding.MLA_ERR_BAD_BLOCK_ID
    bad = np.zeros(240, dtype=bool)
    good_table = table.copy()
    if what in ("page", "negative"):
        table[0, 1] = len(cache) if what == "page" else -1
        bad[64:128] = True
    elif what == "past":
        first, code = [0, 64 * 3 - 40], binding.MLA_ERR_BAD_SEQ_LEN   # 50 tokens past the table
        table[1], good_table[1] = table[0], table[0]
        bad[150 + 40:] = True
    else:
        first, code = [0, -10], binding.MLA_ERR_BAD_SEQ_LEN
        bad[150:160] = True
    ws = binding.new_status_workspace()
    kv, pe = binding.mla_expand_kv(_dev(cache), _int(table), _int([0, 150, 240]), _dev(w_uk),
                                   _dev(w_uv), total_k=240, workspace=ws, first_token=_int(first))
    torch.cuda.synchronize()
    assert binding.read_error(ws) == code
    kv, pe = bf16_tensor_bits(kv), bf16_tensor_bits(pe)
    assert (kv[bad] == 0).all() and (pe[bad] == 0).all()
    if what in ("page", "negative"):
        ref, _ = expand_kv(bf16_bits_to_f64(cache), good_table, first, lens, bf16_bits_to_f64(w_uk),
                           bf16_bits_to_f64(w_uv))
        err = np.abs(bf16_bits_to_f64(kv) - ref)[~bad]
        # |sum| <= 512 terms; sqrt-sized products of unit normals with 512^-1/2 weights
        assert (err <= 2.0 ** -8 * np.abs(ref[~bad]) + 512 * 2.0 ** -23 * 512).all()


def test_expand_from_and_to_offsets_past_2_31_elements():
    """Pages at the end of a cache of 60,000 (2.2 G elements), into the rows at
    the end of 70,000 x 128 x 256 (2.3 G elements)."""
    import torch
    rng = np.random.default_rng(13)
    lens, heads, blocks, rows = [150], 128, 60000, 70000
    cache, table, w_uk, w_uv = _problem(rng, lens, [0], heads, False)
    big = torch.zeros((blocks, 64, 576), dtype=torch.bfloat16, device="cuda")
    big[blocks - len(cache):] = _dev(cache)
    kv = torch.zeros((rows, heads, 256), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    ws = binding.new_status_workspace()
    binding.mla_expand_kv(big, _int(table[:, :3] + blocks - len(cache)),
                          _int([rows - 150, rows]), _dev(w_uk), _dev(w_uv), total_k=rows,
                          workspace=ws, kv=kv, k_pe=pe)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    _check(bf16_bits_to_f64(bf16_tensor_bits(kv[-150:])),
           bf16_bits_to_f64(bf16_tensor_bits(pe[-150:])), cache, 1.0, table, [0], lens, w_uk, w_uv,
           False)
    assert not kv[:-150].any() and not pe[:-150].any()


def test_expand_replays_in_a_graph():
    import torch
    rng = np.random.default_rng(14)
    lens, first = [300, 70], [5, 64]
    cache, table, w_uk, w_uv = _problem(rng, lens, first, 3, False)
    args = (_dev(cache), _int(table), _int([0, 300, 370]), _dev(w_uk), _dev(w_uv))
    ws, start = binding.new_status_workspace(), _int(first)
    want = binding.mla_expand_kv(*args, total_k=370, workspace=ws, first_token=start)
    kv, pe = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        binding.mla_expand_kv(*args, total_k=370, workspace=ws, first_token=start, kv=kv, k_pe=pe,
                              stream=stream)
    for _ in range(2):
        kv.zero_(), pe.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kv, want[0]) and torch.equal(pe, want[1])


def test_expand_with_starts_that_make_no_sense_stays_in_bounds():
    """Decreasing or oversized starts: what is written lies in the outputs."""
    import torch
    rng = np.random.default_rng(12)
    cache, table, w_uk, w_uv = _problem(rng, [100, 100], [0, 0], 2, False)
    ws = binding.new_status_workspace()
    for cu in ([0, 90, 50], [0, 500, 700], [-3, 10, 20], [5, 5, 5]):
        kv, _ = binding.mla_expand_kv(_dev(cache), _int(table), _int(cu), _dev(w_uk), _dev(w_uv),
                                      total_k=120, workspace=ws)
        torch.cuda.synchronize()
        binding.read_error(ws)
        assert kv.shape == (120, 2, 256)


@pytest.mark.parametrize("cu,total", [([0, 100, 200], 150), ([0, 100, 200], 100), ([0, 0, 200], 1)])
def test_expand_into_too_few_rows_is_reported(cu, total):
    """Rows that there is room for are those of the whole call; the error says
    that there were more, whether a sequence is cut or left out."""
    import torch
    rng = np.random.default_rng(13)
    cache, table, w_uk, w_uv = _problem(rng, [200, 200], [0, 0], 2, False)
    args = (_dev(cache), _int(table), _int(cu), _dev(w_uk), _dev(w_uv))
    ws = binding.new_status_workspace()
    want = binding.mla_expand_kv(*args, total_k=cu[-1], workspace=ws)
    assert binding.read_error(ws) == 0
    got = binding.mla_expand_kv(*args, total_k=total, workspace=ws)
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_SEQ_LEN
    assert all(torch.equal(g.view(torch.int16), w[:total].view(torch.int16))
               for g, w in zip(got, want))


def test_expansions_on_two_streams_at_once():
    """Pairs of CTAs of two calls share the GPU: each call's result is the one
    it has alone (ragged ends, so both ways out of the kernel are taken)."""
    import torch
    rng = np.random.default_rng(14)
    calls = []
    for lens, heads, fp8 in (([700, 31, 300], 32, False), ([257, 600], 17, True)):
        first = [0] * len(lens)
        cache, table, w_uk, w_uv = _problem(rng, lens, first, heads, fp8)
        args = (torch.from_numpy(cache).cuda() if fp8 else _dev(cache), _int(table),
                _int(np.concatenate([[0], np.cumsum(lens)])), _dev(w_uk), _dev(w_uv))
        calls.append((binding.mla_expand_kv_fp8 if fp8 else binding.mla_expand_kv,
                      args + ((0.25,) if fp8 else ()), sum(lens), binding.new_status_workspace(),
                      torch.cuda.Stream()))
    want = [fn(*args, total_k=total, workspace=ws) for fn, args, total, ws, _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(20):
        for i, (fn, args, total, ws, stream) in enumerate(calls):
            got[i].append(fn(*args, total_k=total, workspace=ws, stream=stream))
    torch.cuda.synchronize()
    for i, (_, _, _, ws, _) in enumerate(calls):
        assert binding.read_error(ws) == 0
        for kv, pe in got[i]:
            assert torch.equal(kv.view(torch.int16), want[i][0].view(torch.int16))
            assert torch.equal(pe.view(torch.int16), want[i][1].view(torch.int16))

"""Writing the cache's rows and reading them back, against the definitions.

Written rows and the rows gathered from a bf16 cache are copies, and codes are
compared with the nearest code of the exact quotient: all equal bit for bit.
Rows gathered from an fp8 cache are fp32 products of a code and the scale
(half a step, 2^-24 of the value) rounded to bf16 (2^-8): 2^-8 + 2^-23 of the
exact product.
"""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import (bf16_bits_to_f64, bf16_tensor_bits,
                                                    f32_to_bf16_bits)
from oracle import cache_write, e4m3_codes, e4m3_to_float, gather_rows, mla_decode_reference_fp8

pytestmark = pytest.mark.gpu


def _bf16(rng, shape):
    return f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def _dev(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _u8(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _int(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _slots(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda()


def _write(kv_c, k_pe, slots, cache, fp8, k_scale, ws, **kw):
    if fp8:
        return binding.mla_cache_write_fp8(kv_c, k_pe, slots, cache, k_scale, workspace=ws, **kw)
    return binding.mla_cache_write(kv_c, k_pe, slots, cache, workspace=ws, **kw)


def _gather(cache, table, cu, fp8, k_scale, **kw):
    if fp8:
        return binding.mla_cache_gather_fp8(cache, table, cu, k_scale, **kw)
    return binding.mla_cache_gather(cache, table, cu, **kw)


def _bits(cache, fp8):
    return cache.cpu().numpy() if fp8 else bf16_tensor_bits(cache)


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 63, 257, 4096, 4097, 5003])
def test_write_against_the_oracle(tokens, fp8):
    """Padding among the slots, rows in any order, the others left as they were."""
    import torch
    rng = np.random.default_rng(tokens)
    blocks = -(-tokens // 64) + 2
    before = (rng.integers(0, 256, (blocks, 64, 576), dtype=np.uint8) if fp8
              else _bf16(rng, (blocks, 64, 576)))
    kv, pe = _bf16(rng, (tokens, 512)), _bf16(rng, (tokens, 64))
    slots = rng.permutation(blocks * 64)[:tokens].astype(np.int64)
    slots[rng.random(tokens) < 0.2] = -1
    cache = _u8(before) if fp8 else _dev(before)
    ws = binding.new_status_workspace()
    got = _write(_dev(kv), _dev(pe), _slots(slots), cache, fp8, 0.0117, ws)
    torch.cuda.synchronize()
    assert got is cache and binding.read_error(ws) == 0
    new = [e4m3_codes(bf16_bits_to_f64(x), 0.0117) if fp8 else x for x in (kv, pe)]
    assert np.array_equal(_bits(cache, fp8), cache_write(before, *new, slots))


def _steps(x, n):
    """The fp32 number ``n`` steps above ``x``."""
    return float((np.asarray(x, np.float32).view(np.int32) + n).view(np.float32))


@pytest.mark.parametrize("k_scale", [
    1.0, 0.25, 3.0, 1 / 3, 5.5 / 448, 7.03125 / 448, 448.0, 1.9999999, 1e-30, 2.0 ** -126, 2.0 ** -149,
    7 * 2.0 ** -149, 1e30, 3.0e38, _steps(1, 1), _steps(1, -1), _steps(255 / 31, 0), _steps(255 / 31, 1),
    _steps(255 / 31, -1), _steps(0.2, 500), _steps(0.2, -500), _steps(129 / 13, 600), _steps(129 / 13, -600),
    _steps(11.0, 400), _steps(11.0, -700), 1.2345e-5, 77.7])
def test_every_bf16_value_gets_the_nearest_code(k_scale):
    import torch
    bits = np.arange(65536, dtype=np.uint16)
    rows = np.resize(bits, (114, 576))
    cache = torch.zeros((2, 64, 576), dtype=torch.uint8, device="cuda")
    ws = binding.new_status_workspace()
    t = _dev(rows)
    binding.mla_cache_write_fp8(t[:, :512], t[:, 512:], torch.arange(114, device="cuda"), cache, k_scale,
                                workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    got = cache.cpu().numpy().reshape(-1, 576)[:114]
    want = e4m3_codes(bf16_bits_to_f64(rows), k_scale)
    nan = (got & 0x7F) == 0x7F                      # the NaN code of either sign
    assert np.array_equal(nan, want == 0x7F)
    assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kv_stride,pe_stride,offset", [(576, 576, 0), (2112, 2112, 8), (512, 72, 16),
                                                        (0, 64, 0)])
def test_rows_of_wider_tensors(kv_stride, pe_stride, offset, fp8):
    import torch
    rng = np.random.default_rng(kv_stride + offset)
    T = 37
    store = [_dev(_bf16(rng, (T * max(s, 512) + 64,))) for s in (kv_stride, pe_stride)]
    kv = torch.as_strided(store[0], (T, 512), (kv_stride, 1), offset)
    pe = torch.as_strided(store[1], (T, 64), (pe_stride, 1), offset)
    cache = torch.zeros((1, 64, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    before = _bits(cache, fp8)
    slots = np.arange(T)[::-1]
    ws = binding.new_status_workspace()
    _write(kv, pe, _slots(slots.copy()), cache, fp8, 0.02, ws)
    torch.cuda.synchronize()
    rows = [bf16_tensor_bits(x.contiguous()) for x in (kv, pe)]
    new = [e4m3_codes(bf16_bits_to_f64(x), 0.02) if fp8 else x for x in rows]
    assert binding.read_error(ws) == 0
    assert np.array_equal(_bits(cache, fp8), cache_write(before, *new, slots))


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_past_the_cache_are_recorded_and_not_written(fp8):
    import torch
    rng = np.random.default_rng(8)
    kv, pe = _bf16(rng, (4, 512)), _bf16(rng, (4, 64))
    store = torch.zeros((3, 64, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    ws = binding.new_status_workspace()
    slots = [2 ** 62, 5, 2 * 64, -2 ** 62]
    _write(_dev(kv), _dev(pe), _slots(slots), store[:2], fp8, 0.5, ws)
    torch.cuda.synchronize()
    assert ws[4:8].view(torch.int32).item() in (2 ** 31 - 1, 2)
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    new = [e4m3_codes(bf16_bits_to_f64(x), 0.5) if fp8 else x for x in (kv, pe)]
    want = cache_write(np.zeros((3, 64, 576), np.uint8 if fp8 else np.uint16), *new, [-1, 5, -1, -1])
    assert np.array_equal(_bits(store, fp8), want)


def test_write_refuses_what_does_not_fit():
    import torch
    bf16, z = torch.bfloat16, torch.zeros
    ws = binding.new_status_workspace()
    cache, slots = z((1, 64, 576), dtype=bf16, device="cuda"), _slots([0, 1])
    kv, pe = z((2, 512), dtype=bf16, device="cuda"), z((2, 64), dtype=bf16, device="cuda")
    for bad in (dict(kv=kv[:1]), dict(kv=kv[:, :511]), dict(pe=pe.t().contiguous().t()),
                dict(pe=z((2, 68), dtype=bf16, device="cuda")[:, :64]), dict(slots=slots[:1]),
                dict(cache=z((1, 64, 512), dtype=bf16, device="cuda"))):
        a = dict(kv=kv, pe=pe, slots=slots, cache=cache)
        a.update(bad)
        with pytest.raises(ValueError):
            binding.mla_cache_write(a["kv"], a["pe"], a["slots"], a["cache"], workspace=ws)
    for bad in (dict(kv=kv.float()), dict(slots=slots.int()), dict(cache=cache.view(torch.int16))):
        a = dict(kv=kv, pe=pe, slots=slots, cache=cache)
        a.update(bad)
        with pytest.raises(TypeError):
            binding.mla_cache_write(a["kv"], a["pe"], a["slots"], a["cache"], workspace=ws)


# ------------------------------------------------------------------ gather

def _problem(rng, lens, first, fp8, extra=2):
    held = [a + b for a, b in zip(lens, first)]
    pages = [-(-n // 64) for n in held]
    blocks = sum(pages) + extra
    ids = rng.permutation(blocks)
    table = np.full((len(lens), max(1, max(pages, default=1))), 2 ** 30, dtype=np.int32)
    at = 0
    cache = (rng.integers(0, 256, (blocks, 64, 576), dtype=np.uint8) if fp8
             else _bf16(rng, (blocks, 64, 576)))
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    return cache, table


CASES = [([1], [0]), ([64], [0]), ([65], [63]), ([5, 0, 7], [60, 3, 0]), ([0, 0, 3], [0, 0, 0]),
         ([300, 1, 500], [0, 640, 65]), ([40] * 33, list(range(33))), ([4096], [1]), ([4097], [0]),
         ([3000, 0, 2000, 1], [17, 5, 0, 64])]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_gather_against_the_oracle(case, fp8):
    import torch
    lens, first = CASES[case]
    rng = np.random.default_rng(700 + case)
    cache, table = _problem(rng, lens, first, fp8)
    total, spare, k_scale = sum(lens), 3, 0.037109375
    rows = _dev(np.full((total + spare, 576), 0x1234, np.uint16))
    ws = binding.new_status_workspace()
    cu = np.concatenate([[0], np.cumsum(lens)])
    got = _gather(_u8(cache) if fp8 else _dev(cache), _int(table), _int(cu), fp8, k_scale,
                  total_k=total + spare, first_token=_int(first), rows=rows, workspace=ws)
    torch.cuda.synchronize()
    assert got is rows and binding.read_error(ws) == 0
    bits = bf16_tensor_bits(rows)
    assert (bits[total:] == 0x1234).all()
    want = gather_rows(cache, table, first, lens)
    if not fp8:
        assert np.array_equal(bits[:total], want)
        return
    want = e4m3_to_float(want) * k_scale
    value = bf16_bits_to_f64(bits[:total])
    assert np.array_equal(np.isnan(value), np.isnan(want))
    assert not (np.abs(value - want) > (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_gather_of_bad_pages_lengths_and_starts(fp8):
    """Zeros for tokens whose page is not there, errors recorded; starts that
    pass total_k; without first tokens."""
    import torch
    rng = np.random.default_rng(3)
    cache, table = _problem(rng, [130], [0], fp8)
    table[0, 1] = cache.shape[0]
    dev = _u8(cache) if fp8 else _dev(cache)
    ws = binding.new_status_workspace()
    rows = _gather(dev, _int(table), _int([0, 130]), fp8, 1.0, total_k=130, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    bits = bf16_tensor_bits(rows)
    assert not bits[64:128].any()
    table[0, 1] = -1
    rows = _gather(dev, _int(table), _int([0, 130]), fp8, 1.0, total_k=130, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_BLOCK_ID
    assert np.array_equal(bf16_tensor_bits(rows)[:64], bits[:64])
    # past the table (3 pages), before its start, more rows than there is room for
    for first, n in ((190, 5), (-3, 5)):
        rows = _gather(dev, _int(table), _int([0, n]), fp8, 1.0, total_k=n, workspace=ws,
                       first_token=_int([first]))
        torch.cuda.synchronize()
        assert binding.read_error(ws) == binding.MLA_ERR_BAD_SEQ_LEN
        there = [t for t in range(n) if 0 <= first + t < 192]
        assert not np.delete(bf16_tensor_bits(rows), there, axis=0).any()
    rows = _gather(dev, _int(table), _int([0, 20]), fp8, 1.0, total_k=11, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == binding.MLA_ERR_BAD_SEQ_LEN
    assert np.array_equal(bf16_tensor_bits(rows), bits[:11])


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_past_two_to_the_31(fp8):
    """Blocks whose entries lie past 2^31 elements (and 2^32 bytes) of the pool."""
    import torch
    blocks = 60000
    pool = torch.zeros((blocks, 64, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    rng = np.random.default_rng(5)
    kv, pe = _bf16(rng, (3, 512)), _bf16(rng, (3, 64))
    slots = [blocks * 64 - 1, 58255 * 64 + 7, 0]
    ws = binding.new_status_workspace()
    _write(_dev(kv), _dev(pe), _slots(slots), pool, fp8, 0.5, ws)
    rows = _gather(pool, _int([[s // 64] for s in slots]), _int([0, 1, 2, 3]), fp8, 0.5, total_k=3,
                   first_token=_int([s % 64 for s in slots]), workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    new = np.concatenate([kv, pe], 1)
    if fp8:
        new = f32_to_bf16_bits((e4m3_to_float(e4m3_codes(bf16_bits_to_f64(new), 0.5)) * 0.5)
                               .astype(np.float32))
    assert np.array_equal(bf16_tensor_bits(rows), new)


# ------------------------------------------------------------------ together

def test_a_written_fp8_cache_is_what_the_decode_reads():
    """Three steps of a small batch: each step's new token is quantised into the
    cache, which the fp8 decode then reads; on a side stream, and again as a
    replayed graph, bit for bit."""
    import torch
    rng = np.random.default_rng(21)
    B, N, k_scale, lens = 3, 16, 0.013, np.array([60, 5, 127])
    table = np.arange(9).reshape(3, 3)[:, ::-1].astype(np.int32)
    cache = torch.zeros((9, 64, 576), dtype=torch.uint8, device="cuda")
    host = np.zeros((9, 64, 576), dtype=np.uint8)
    # the prompts, in one call
    prompt = _bf16(rng, (int(lens.sum()), 576))
    slots = [int(table[b, t // 64]) * 64 + t % 64 for b in range(B) for t in range(lens[b])]
    ws = binding.new_status_workspace()
    d = _dev(prompt)
    binding.mla_cache_write_fp8(d[:, :512], d[:, 512:], _slots(slots), cache, k_scale, workspace=ws)
    codes = e4m3_codes(bf16_bits_to_f64(prompt), k_scale)
    host = cache_write(host, codes[:, :512], codes[:, 512:], slots)
    plan = binding.make_plan(B, N, 3)
    dws = binding.new_workspace(plan)
    new, slot = _dev(np.zeros((B, 576), np.uint16)), _slots([0] * B)
    q, seq, dt = _dev(np.zeros((B, N, 576), np.uint16)), _int(lens), _int(table)
    out = torch.empty((B, N, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, N), dtype=torch.float32, device="cuda")

    def step():
        binding.mla_cache_write_fp8(new[:, :512], new[:, 512:], slot, cache, k_scale, workspace=ws)
        binding.mla_decode_fp8(q, cache, dt, seq, 192 ** -0.5, k_scale, plan=plan, workspace=dws,
                               out=out, lse=lse)

    graph = None
    side = torch.cuda.Stream()
    for i in range(3):
        row, query = _bf16(rng, (B, 576)), _bf16(rng, (B, N, 576))
        at = [int(table[b, lens[b] // 64]) * 64 + lens[b] % 64 for b in range(B)]
        lens = lens + 1
        new.copy_(_dev(row)), q.copy_(_dev(query)), slot.copy_(_slots(at)), seq.copy_(_int(lens))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        eager = (out.clone(), lse.clone())
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        codes = e4m3_codes(bf16_bits_to_f64(row), k_scale)
        host = cache_write(host, codes[:, :512], codes[:, 512:], at)
        assert np.array_equal(cache.cpu().numpy(), host)
        ref, ref_lse = mla_decode_reference_fp8(bf16_bits_to_f64(query), host, table, lens, 192 ** -0.5, k_scale)
        assert np.abs(bf16_bits_to_f64(bf16_tensor_bits(out)) - ref).max() <= 2e-2
        assert np.abs(lse.double().cpu().numpy() - ref_lse).max() <= 1e-3
    assert binding.read_error(ws) == 0 and binding.read_error(dws) == 0


@pytest.mark.parametrize("on_a_stream", [False, True])
def test_a_dispatch_mode_sees_the_gathered_rows(on_a_stream):
    import torch
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        made = set()

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if isinstance(out, torch.Tensor):
                self.made.add(out.data_ptr())
            return out

    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    ws = binding.new_status_workspace()
    table, cu = _int([[0, 1]]), _int([0, 70])
    torch.cuda.synchronize()
    with Seen() as seen:
        rows = binding.mla_cache_gather(cache, table, cu, total_k=70, workspace=ws,
                                        stream=torch.cuda.Stream() if on_a_stream else None)
    torch.cuda.synchronize()
    assert rows.data_ptr() in seen.made and not rows.any()

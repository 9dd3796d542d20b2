"""What mla_expand_kv leaves alone, and what it still gives where a call's
starts, tokens or pages are bad. Tolerance: half a bf16 step of the result
(2^-8 of it) and 512 fp32 additions, a whole step (2^-23) of the products'
magnitudes each."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import (bf16_bits_to_f64, bf16_tensor_bits,
                                                    f32_to_bf16_bits)
from oracle import e4m3_to_float, expand_kv

pytestmark = pytest.mark.gpu

FILL = 0x1234
GUARD = 64              # rows before and behind the results
K_SCALE = 0.037109375


def _bf16(rng, shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _dev(bits):
    import torch
    bits = np.ascontiguousarray(bits)
    if bits.dtype == np.uint8:
        return torch.from_numpy(bits).cuda()
    return torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()


def _int(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


class _Problem:
    """Three pages of 64 tokens for each of two requests, and one spare page."""

    def __init__(self, fp8, heads=3):
        rng = np.random.default_rng(77)
        self.fp8, self.heads = fp8, heads
        self.table = rng.permutation(7)[:6].reshape(2, 3).astype(np.int32)
        if fp8:
            self.cache = rng.integers(0, 256, (7, 64, 576), dtype=np.uint8)
            self.cache[(self.cache & 0x7F) == 0x7F] = 0x7E
        else:
            self.cache = _bf16(rng, (7, 64, 576))
        self.w_uk = _bf16(rng, (heads, 128, 512), 512 ** -0.5)
        self.w_uv = _bf16(rng, (heads, 512, 128), 512 ** -0.5)

    def run(self, cu, total, table=None, first=None):
        """(kv bits, k_pe bits, status) of a call into rows with guards around them."""
        import torch
        kv = _dev(np.full((total + 2 * GUARD, self.heads, 256), FILL, np.uint16))
        pe = _dev(np.full((total + 2 * GUARD, 64), FILL, np.uint16))
        inner = slice(GUARD, GUARD + total)
        ws = binding.new_status_workspace()
        args = (_dev(self.cache), _int(self.table if table is None else table), _int(cu),
                _dev(self.w_uk), _dev(self.w_uv)) + ((K_SCALE,) if self.fp8 else ())
        fn = binding.mla_expand_kv_fp8 if self.fp8 else binding.mla_expand_kv
        fn(*args, total_k=total, workspace=ws, kv=kv[inner], k_pe=pe[inner],
           first_token=None if first is None else _int(first))
        torch.cuda.synchronize()
        status = binding.read_error(ws)
        kv, pe = bf16_tensor_bits(kv), bf16_tensor_bits(pe)
        for x in (kv, pe):
            assert (x[:GUARD] == FILL).all() and (x[GUARD + total:] == FILL).all()
        return kv[inner], pe[inner], status

    def check(self, kv, pe, tokens):
        """Row t holds request r's token j, tokens[t] = (r, j); None: never written;
        "zero": zeros."""
        values = e4m3_to_float(self.cache) * K_SCALE if self.fp8 else bf16_bits_to_f64(self.cache)
        uk, uv = bf16_bits_to_f64(self.w_uk), bf16_bits_to_f64(self.w_uv)
        ref, ref_pe = expand_kv(values, self.table, [0, 0], [192, 192], uk, uv)
        size, _ = expand_kv(np.abs(values), self.table, [0, 0], [192, 192], np.abs(uk), np.abs(uv))
        left = np.array([x is None for x in tokens])
        zero = np.array([isinstance(x, str) for x in tokens])
        assert (kv[left] == FILL).all() and (pe[left] == FILL).all()
        assert (kv[zero] == 0).all() and (pe[zero] == 0).all()
        rows = np.flatnonzero(~left & ~zero)
        at = np.array([192 * tokens[t][0] + tokens[t][1] for t in rows], dtype=np.int64)
        err = np.abs(bf16_bits_to_f64(kv[rows]) - ref[at])
        assert (err <= 2.0 ** -8 * np.abs(ref[at]) * (1 + 2.0 ** -8)
                + 512 * 2.0 ** -23 * size[at]).all()
        err = np.abs(bf16_bits_to_f64(pe[rows]) - ref_pe[at])
        assert (err <= (2.0 ** -8 * np.abs(ref_pe[at]) if self.fp8 else 0)).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu,status,rows", [
    ([0, 90, 50], None, [(0, 0, 90)]),                     # request 1 would end before it starts
    ([0, 500, 700], binding.MLA_ERR_BAD_SEQ_LEN, [(0, 0, 150)]),
    ([-3, 10, 20], None, [(1, 10, 20)]),                   # request 0 starts before the rows do
    ([5, 5, 5], 0, []),
    ([30, 100, 140], 0, [(0, 30, 100), (1, 100, 140)]),
    ([0, 100, 150], 0, [(0, 0, 100), (1, 100, 150)]),
])
def test_rows_of_no_request_and_the_bytes_around_are_left(cu, status, rows, fp8):
    p = _Problem(fp8)
    kv, pe, got = p.run(cu, 150)
    assert status is None or got == status              # (None: starts that make no sense)
    tokens = [None] * 150
    for r, begin, end in rows:
        for t in range(begin, end):
            tokens[t] = (r, t - begin)
    p.check(kv, pe, tokens)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["page", "negative", "past", "first"])
def test_good_rows_beside_bad_ones(what, fp8):
    """Rows of a bad page or token are zeros, all others what they always are."""
    p = _Problem(fp8)
    table, first, code = p.table.copy(), [0, 0], binding.MLA_ERR_BAD_BLOCK_ID
    tokens = [(0, t) for t in range(150)] + [(1, t) for t in range(90)]
    if what in ("page", "negative"):
        table[0, 1] = len(p.cache) if what == "page" else -1
        tokens[64:128] = ["zero"] * 64
    else:
        code = binding.MLA_ERR_BAD_SEQ_LEN
        first[1] = 192 - 40 if what == "past" else -10
        tokens[150:] = [(1, t + first[1]) if 0 <= t + first[1] < 192 else "zero"
                        for t in range(90)]
    kv, pe, got = p.run([0, 150, 240], 240, table, first)
    assert got == code
    p.check(kv, pe, tokens)

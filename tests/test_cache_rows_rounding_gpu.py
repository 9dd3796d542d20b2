"""The roundings that the cache's row calls promise, bit for bit: a gathered
fp8 row is k_scale times its codes' values rounded once to bf16, a written NaN
is the code 0x7F."""

import math

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_tensor_bits
from oracle import e4m3_to_float

pytestmark = pytest.mark.gpu


def _fp32(bits):
    return float(np.asarray(bits, np.uint32).view(np.float32))


def _near(numerator, denominator, exponent, steps):
    """The fp32 number ``steps`` steps above a ratio times a power of two."""
    x = np.float32(math.ldexp(numerator / denominator, exponent))
    return float((x.view(np.int32) + np.int32(steps)).view(np.float32))


def _bf16_once(x):
    """float64 to bf16, nearest even, in one rounding."""
    exponent = np.frexp(x)[1] - 1
    step = np.exp2(np.maximum(np.where(x == 0, -126, exponent), -126) - 7.0)
    y = np.rint(x / step) * step                   # (exact but for the rounding)
    with np.errstate(over="ignore"):
        return (y.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


# An fp32 product of a code's value (4 bits) and the scale (24) is itself a
# rounding: it makes a tie between two bf16 numbers of a product next to one.
TIES = [_fp32(b) for b in (0x3EB6E8BA, 0x3C6B8E39, 0x1B622E8B, 0x7DF2AAAB, 0x518ECCCD, 0x42564924, 0x2A33332,
                           0x13FFFF, 0x02F00003, 0x1680005)]
NEAR = [_near(t, f, k, n) for t, f, k, n in [
    (511, 15, -12, 1), (511, 15, -12, -1), (257, 13, -9, 200), (257, 13, -9, -300), (301, 11, -20, 700),
    (485, 7, -130, 2), (485, 7, -130, -2), (333, 9, 100, 1), (333, 9, 117, -1), (259, 3, -140, 1), (511, 1, 119, -1)]]


@pytest.mark.parametrize("k_scale", TIES + NEAR + [
    1.0, 0.75, 1 / 3, 5.5 / 448, 0.0117, 2.0 ** -126, 2.0 ** -149, 7 * 2.0 ** -149, 3.0 ** -83, 1e-37, 3.4e38, 7.5e35])
def test_gathered_rows_are_rounded_once(k_scale):
    import torch
    codes = np.resize(np.arange(256, dtype=np.uint8), (64, 576))
    cache = torch.from_numpy(codes.reshape(1, 64, 576)).cuda()
    ws = binding.new_status_workspace()
    rows = binding.mla_cache_gather_fp8(cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                        torch.tensor([0, 64], dtype=torch.int32, device="cuda"), k_scale,
                                        total_k=64, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    got = bf16_tensor_bits(rows)
    nan = (codes & 0x7F) == 0x7F
    assert ((got[nan] & 0x7FFF) > 0x7F80).all()
    want = _bf16_once(e4m3_to_float(np.where(nan, 0, codes)) * float(np.float32(k_scale)))
    assert np.array_equal(got[~nan], want[~nan]), np.unique(codes[~nan][got[~nan] != want[~nan]])


@pytest.mark.parametrize("k_scale", [1.0, 0.0123, 1e-30, 1e30])
def test_a_nan_of_either_sign_is_written_as_0x7f(k_scale):
    import torch
    bits = np.array([0x7F81, 0x7FC0, 0x7FFF, 0xFF81, 0xFFC0, 0xFFFF], np.uint16)
    rows = torch.from_numpy(np.resize(bits, (5, 576)).view(np.int16)).view(torch.bfloat16).cuda()
    cache = torch.zeros((1, 64, 576), dtype=torch.uint8, device="cuda")
    ws = binding.new_status_workspace()
    binding.mla_cache_write_fp8(rows[:, :512], rows[:, 512:], torch.arange(5, device="cuda"), cache, k_scale,
                                workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert (cache[0, :5] == 0x7F).all() and not cache[0, 5:].any()

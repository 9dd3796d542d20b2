"""Queries of small numbers in the decodes over an fp8 cache, whose tensor cores
multiply in f16. A row whose greatest is below 2^-4 is multiplied by the power
of two that brings it to 2^14 or more (at most by 2^126, which brings a normal
number to 1 or more), so that what f16 loses of an entry (2^-25) is at most
2^-21 of the row's greatest, or 2^-25 of it in a row that was multiplied: less
than the 2^-23 of the sum of magnitudes, for each of 576 additions, that
span_util.py counts. Its tolerance holds as it is."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import f32_to_bf16_bits
from span_sharing import assert_shared
from span_util import SCALE, check, random_q, reference, run_shared, run_window, shared_problem

pytestmark = pytest.mark.gpu


def _all(lens):
    return [np.arange(n) for n in lens]


@pytest.mark.parametrize("exponent", [-14, -18, -20, -26, -60, -110, -125])
def test_small_queries(exponent):
    """Queries of 2^exponent and a scale that makes up for them, in tiles, in
    requests' own items and through a window."""
    import torch
    rng = np.random.default_rng(-exponent)
    lens, starts, shared, heads = [700 + 13 * i for i in range(8)] + [130], [0, 8], [640], 24
    cache, table = shared_problem(rng, lens, starts, shared, True)
    q = random_q(rng, 9, heads, 2.0 ** exponent)
    scale = SCALE * 2.0 ** -exponent
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, scale, num_sms=12)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert_shared(ws, lens, starts, shared, heads, 12)
    check(out, lse, reference(q, cache, table, _all(lens), scale), exponent)
    out, lse, ws = run_window(q, cache, table, lens, 300, 66, scale)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    seen = [np.array([t for t in range(n) if t < 66 or t >= n - 300]) for n in lens]
    check(out, lse, reference(q, cache, table, seen, scale), exponent)


def test_rows_of_very_different_sizes():
    """Each row has its own power of two, piece after piece of a pair's work."""
    import torch
    rng = np.random.default_rng(41)
    B, heads = 40, 12
    lens = [int(x) for x in rng.integers(1, 700, B)]
    cache, table = shared_problem(rng, lens, [0, B], [0], True)
    gain = np.exp2(rng.integers(-40, 3, (B, heads, 1)).astype(np.float64))
    q = f32_to_bf16_bits((rng.standard_normal((B, heads, 576)) * gain).astype(np.float32))
    q[3], q[5, 2], q[7, :, 100:] = 0, 0x8000, 0
    q[9, 4, :] = 0
    q[9, 4, 17] = 0x477F                                    # 65280, alone in its row
    q[11, 0, :] = 0x0003                                    # bf16's smallest numbers
    for scale in (SCALE, -2.0 ** 20, 0.0):
        for num_sms in (2, 14, 152):
            out, lse, ws = run_window(q, cache, table, lens, 500, 3, scale, num_sms=num_sms)
            torch.cuda.synchronize()
            assert binding.read_error(ws) == 0
            seen = [np.array([t for t in range(n) if t < 3 or t >= n - 500]) for n in lens]
            check(out, lse, reference(q, cache, table, seen, scale), (scale, num_sms))

"""Pins of the oracle's definitions of the cache's written, gathered and windowed rows (CPU only)."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64
from oracle import (cache_write, e4m3_codes, e4m3_to_float, gather_rows, mla_decode_reference,
                    mla_decode_window_reference)


def test_a_codes_value_gives_the_code():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    for scale in (1.0, 0.25, 0.012276786, 3.0):
        assert np.array_equal(e4m3_codes(e4m3_to_float(codes) * float(np.float32(scale)), scale), codes)


def test_hand_worked_codes():
    # 1.0625 lies halfway between 1 (0x38) and 1.125 (0x39): even; 1.1875 between
    # 0x39 and 1.25 (0x3A); 2^-10 between 0 and the smallest; 464 beyond 448.
    x = [1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 464.0, -1e30, np.inf, np.nan, 0.0]
    assert e4m3_codes(x, 1.0).tolist() == [0x38, 0x3A, 0xB8, 0, 2, 0x7E, 0xFE, 0x7E, 0x7F, 0]
    # 1 / 3 of them: 3 * 1.0625 is halfway, a bf16 step more is not.
    assert e4m3_codes([3.1875, 3.203125], 3.0).tolist() == [0x38, 0x39]


def test_codes_against_torch_where_the_quotient_is_exact():
    import torch
    x = bf16_bits_to_f64(np.arange(65536, dtype=np.uint16))
    want = torch.from_numpy(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    nan = np.isnan(x)
    assert np.array_equal(e4m3_codes(x, 1.0)[~nan], want[~nan])
    assert (e4m3_codes(x, 1.0)[nan] == 0x7F).all()


def test_written_rows_are_gathered_again():
    rng = np.random.default_rng(1)
    cache = rng.standard_normal((4, 64, 576))
    rows = rng.standard_normal((3, 576))
    out = cache_write(cache, rows[:, :512], rows[:, 512:], [2 * 64 + 63, -1, 0 * 64 + 0])
    assert np.array_equal(out[2, 63], rows[0]) and np.array_equal(out[0, 0], rows[2])
    out[2, 63], out[0, 0] = cache[2, 63], cache[0, 0]
    assert np.array_equal(out, cache)
    out = cache_write(cache, rows[:, :512], rows[:, 512:], [2 * 64 + 63, 4 * 64, 0])
    assert np.array_equal(gather_rows(out, [[2, 0]], [63], [2]), rows[[0, 2]])


@pytest.mark.parametrize("window,sinks", [(1, 0), (10, 0), (10, 3), (64, 64), (500, 0), (10, 500)])
def test_the_windowed_decode_is_the_decode_of_what_is_seen(window, sinks):
    rng = np.random.default_rng(window + sinks)
    cache = rng.standard_normal((4, 64, 576))
    table, L = [[3, 0, 2]], 140
    q = rng.standard_normal((1, 2, 576))
    got = mla_decode_window_reference(q, cache, table, [L], 0.07, window, sinks)
    rows = gather_rows(cache, table, [0], [L])
    seen = rows[sorted(set(range(min(sinks, L))) | set(range(max(0, L - window), L)))]
    pool = np.zeros((4, 64, 576))
    pool.reshape(-1, 576)[:len(seen)] = seen
    want = mla_decode_reference(q, pool, np.array([[0, 1, 2]]), np.array([len(seen)]), 0.07)
    assert np.allclose(got[0], want[0], rtol=0, atol=1e-12) and np.allclose(got[1], want[1])

"""Tokens of small weight in the decodes over an fp8 cache, whose tensor cores
take weights in f16: the row's reference has weight 2^7 and moves when a weight
passes 2^15, so the greatest lies between 2^7 and 2^15, and what f16 loses of one
(2^-25) is at most 2^-32 of the greatest."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64, bf16_tensor_bits, f32_to_bf16_bits
from oracle import e4m3_codes, e4m3_to_float
from span_util import K_SCALE, run_window

pytestmark = pytest.mark.gpu


def test_many_tokens_of_small_weight():
    """One token far above all others: columns in which it is zero come from the
    many, each of 2^-20 to 2^-30 of its weight."""
    import torch
    rng = np.random.default_rng(6)
    L, down = 6000, np.array([20.0, 23.0, 24.0, 25.5, 26.5, 28.0, 30.0])
    cache = np.zeros((-(-L // 64), 64, 576), np.uint8)
    codes = e4m3_codes(rng.uniform(0.5, 400.0, (L, 512)).astype(np.float32), 1.0)
    codes[:, ::2] = 0
    cache.reshape(-1, 576)[:L, :512] = codes
    for top in (0, 4099, L - 1):
        rows = cache.copy()
        rows.reshape(-1, 576)[top] = 0
        rows.reshape(-1, 576)[top, :512:2] = 0x38           # 1, where the others are 0
        rows.reshape(-1, 576)[top, 570] = 0x38
        q = np.zeros((1, len(down), 576), np.uint16)
        q[0, :, 570] = f32_to_bf16_bits(down.astype(np.float32))
        scale = float(np.float32(np.log(2.0) / K_SCALE))    # scores: log2 of the weights, but for the rounding
        table = np.arange(rows.shape[0]).reshape(1, -1)
        out, lse, ws = run_window(q, rows, table, [L], L, 0, scale)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        k = e4m3_to_float(rows.reshape(-1, 576)[:L]) * K_SCALE
        s = scale * (bf16_bits_to_f64(q[0]) @ k.T)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(-1, keepdims=True)
        want = (p / z) @ k[:, :512]
        # Weights: half a step of f16 (2^-11), and 2^-32 of the greatest; scores: 2^-22 of the largest and 2^-21;
        # sums of L; one rounding to bf16; and the sum of the rounded weights as far as these move it.
        rel = 2.0 ** -11 * (1 + 2.0 ** -10) + 2 * (2.0 ** -22 * np.abs(s).max(-1) + 2.0 ** -21) + (L + 64) * 2.0 ** -22
        lost = 2.0 ** -32 * (np.abs(k[:, :512]).sum(0) + L * want) / z
        tol = 2.0 ** -8 * want * (1 + 2.0 ** -8) + 2 * rel[:, None] * want + lost
        got = bf16_bits_to_f64(bf16_tensor_bits(out))[0]
        assert (np.abs(got - want) <= tol).all(), (top, (np.abs(got - want) / np.maximum(tol, 1e-30)).max(-1))
        assert np.abs(lse.double().cpu().numpy()[0] - (m + np.log(z))[:, 0]).max() <= 1e-4

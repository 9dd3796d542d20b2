"""Scores so large that fp32 has them 2^4 to 2^20 apart: the softmax is the token
of the greatest score, the result its values (rounded once to bf16) and the
LSE its score.

A row counts where the greatest of the exact scores leads by more than what
two scores can be off together: 576 additions that truncate, 2^-23 of the sum of
magnitudes each, and 2^-22 of the score, each twice."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64, bf16_tensor_bits
from span_util import random_q, run_shared, run_window, shared_problem, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** 22, -2.0 ** 25, 2.0 ** 31, 1e11])
def test_the_greatest_score_wins(scale, fp8):
    import torch
    rng = np.random.default_rng(64)
    lens, starts, shared, heads = [700 + 9 * i for i in range(8)] + [130], [0, 8], [640], 24
    cache, table = shared_problem(rng, lens, starts, shared, fp8)
    q = random_q(rng, 9, heads)
    for call in (lambda: run_shared(q, cache, table, lens, starts, shared, scale, 12),
                 lambda: run_window(q, cache, table, lens, 2000, 0, scale, 12)):
        out, lse, ws = call()
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        got, z = bf16_bits_to_f64(bf16_tensor_bits(out)), lse.double().cpu().numpy()
        clear = 0
        for b, n in enumerate(lens):
            t = np.arange(n)
            k = values(cache[table[b, t // 64], t % 64])
            x = bf16_bits_to_f64(q[b])
            s = scale * (x @ k.T)
            off = 2 * (abs(scale) * 576 * 2.0 ** -23 * (np.abs(x) @ np.abs(k).T).max(-1)
                       + 2.0 ** -22 * np.abs(s).max(-1))
            order = np.argsort(s, -1)
            top = order[:, -1]
            h = np.nonzero(s[np.arange(heads), top] - s[np.arange(heads), order[:, -2]] > off)[0]
            clear += len(h)
            want = k[top[h], :512]
            assert (np.abs(got[b, h] - want) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want)).all(), (b, n)
            assert (np.abs(z[b, h] - s[h, top[h]]) <= off[h]).all()
        assert clear > 9 * heads // 2

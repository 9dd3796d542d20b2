"""The queries of the decodes over an fp8 cache that f16, which their tensor
cores multiply in, cannot hold: named by request, and nothing to rows of no
tokens."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from span_sharing import assert_shared
from span_util import SCALE, check, random_q, reference, run_shared, shared_problem

pytestmark = pytest.mark.gpu


def _all(lens):
    return [np.arange(n) for n in lens]


@pytest.mark.parametrize("bits", [0x4780, 0x7F80, 0xFFC0])
def test_rows_without_tokens_may_hold_anything(bits):
    """A padded row of a tile: its queries count for nothing, whatever they are."""
    import torch
    rng = np.random.default_rng(19)
    lens, starts, shared, heads = [700, 0, 710, 720, 0, 700, 690], [0, 7], [640], 24
    cache, table = shared_problem(rng, lens, starts, shared, True)
    q = random_q(rng, 7, heads)
    q[1], q[4, 20:] = bits, bits
    out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=6)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert_shared(ws, lens, starts, shared, heads, 6)
    q[1], q[4] = 0, 0
    check(out, lse, reference(q, cache, table, _all(lens), SCALE))


@pytest.mark.parametrize("request_,head", [(0, 0), (2, 23), (5, 8), (6, 0)])
def test_the_request_of_a_query_beyond_f16_is_named(request_, head):
    import torch
    rng = np.random.default_rng(20)
    lens, starts, shared, heads = [700] * 7, [0, 7], [640], 24
    cache, table = shared_problem(rng, lens, starts, shared, True)
    q = random_q(rng, 7, heads)
    q[request_, head, 575] = 0xC780                          # -65536
    for num_sms in (6, 152):                                 # in tiles, and request by request
        out, lse, ws = run_shared(q, cache, table, lens, starts, shared, num_sms=num_sms)
        torch.cuda.synchronize()
        assert ws[4:8].view(torch.int32).item() == request_
        assert binding.read_error(ws) == binding.MLA_ERR_RANGE

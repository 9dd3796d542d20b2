"""A query's result does not depend, to the last bit, on the other queries that
lie in its tile of rows: those behind it in its sequence, and the next
sequence's."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


@pytest.mark.parametrize("gain", [0.0, 60.0, 4000.0, float("inf"), float("nan")])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("rows,changed", [(3, 3), (100, 100), (130, 130), (200, 200), (100, 41),
                                          (200, 7), (200, 177)])
def test_queries_behind_one_change_nothing(rows, changed, splits, gain):
    """`rows` queries of one sequence and 90 of the next; those from `changed` on change."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(29)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)

    def starts(*at):
        return torch.from_numpy(np.array(at, dtype=np.int32)).cuda()

    keys, heads = 900, 2
    q, kv, pe = normal(rows + 90, heads, 192), normal(2 * keys, heads, 256), normal(2 * keys, 64)
    plan = binding.make_prefill_plan(2, heads, rows + 90, max(rows, 90), keys,
                                     num_kv_splits=splits)
    ws = binding.new_workspace(plan)
    args = (kv, pe, starts(0, rows, rows + 90), starts(0, keys, 2 * keys), SCALE)
    want = binding.mla_prefill(q, *args, plan=plan, workspace=ws)
    q[changed:] *= gain
    got = binding.mla_prefill(q, *args, plan=plan, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    assert torch.equal(got[0][:changed].view(torch.int16), want[0][:changed].view(torch.int16))
    assert torch.equal(got[1][:changed], want[1][:changed])

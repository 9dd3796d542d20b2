"""Infinite values that a query sees, by the weight they get: infinity where it
is more than 0 in fp32, NaN (0 times infinity) where it underflows, at every
position of the sequence and in both kernels.

Every query is 16 in column 0 and small elsewhere. A key's column 0 is 0, but
for the one with the infinite value, whose score is 16 * SCALE * x below the
others': 58 (weight e^-58 = 2^-83, far above the smallest fp32 number) for x =
-50, 173 (2^-250, far below it) for x = -150; the rest of a score is under 4."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _int(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _problem(q_rows, keys, heads):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(23)

    def normal(scale, *shape):
        return (torch.empty(shape, device="cuda").normal_(generator=gen) * scale).to(torch.bfloat16)

    q, kv, pe = normal(0.5, q_rows, heads, 192), normal(1, keys, heads, 256), normal(0.5, keys, 64)
    q[..., 0] = 16
    kv[..., 0] = 0
    kv[..., 1:128] *= 0.5
    return q, kv, pe


def _run(q, kv, pe, max_q, splits, causal=True):
    import torch
    plan = binding.make_prefill_plan(1, q.shape[1], q.shape[0], max_q, kv.shape[0],
                                     num_kv_splits=splits)
    assert plan.single_rows == (max_q == 1)
    ws = binding.new_workspace(plan)
    out, lse = binding.mla_prefill(q, kv, pe, _int([0, q.shape[0]]), _int([0, kv.shape[0]]), SCALE,
                                   causal=causal, plan=plan, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    return out, lse


@pytest.mark.parametrize("value", [np.inf, -np.inf])
@pytest.mark.parametrize("x,zero", [(-50, False), (-150, True)])
@pytest.mark.parametrize("at", [3, 200, 520, 640, 645, 699])
@pytest.mark.parametrize("max_q,splits", [(1, 1), (1, 2), (1000, 1), (1000, 3)])
def test_an_infinite_value_counts_by_its_weight(max_q, splits, at, x, zero, value):
    """190 queries over 700 keys: position 3 is seen by all in a whole step, 520
    to 699 lie where rows' limits fall."""
    import torch
    rows, keys, heads = 190, 700, 2
    q, kv, pe = _problem(rows, keys, heads)
    kv[at, 1, 0] = x
    clean, clean_lse = _run(q, kv, pe, max_q, splits)
    assert not torch.isnan(clean).any() and not torch.isinf(clean).any()
    kv[at, 1, 128 + 77] = value
    got, lse = _run(q, kv, pe, max_q, splits)
    sees = torch.arange(rows, device="cuda") + (keys - rows) >= at
    # A query whose last key is the infinite one has other keys to compare with.
    column = got[:, 1, 77].float()
    assert torch.equal(lse, clean_lse)
    if zero:
        assert torch.isnan(column[sees]).all()
    else:
        assert (column[sees] == value).all()
    got[sees, 1, 77] = clean[sees, 1, 77]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))


@pytest.mark.parametrize("max_q,splits", [(1, 1), (1000, 1), (1000, 4)])
def test_the_only_keys_of_a_split_may_have_no_weight(max_q, splits):
    """The last 130 keys are all far below the others: their own split's
    maximum is theirs, and the join takes the weight away."""
    import torch
    q, kv, pe = _problem(20, 700, 1)
    kv[570:, 0, 0] = -150
    kv[690, 0, 128 + 5] = np.inf
    out, lse = _run(q, kv, pe, max_q, splits, causal=False)
    assert torch.isnan(out[:, 0, 5]).all() and not torch.isnan(lse).any()
    assert int(torch.isnan(out).sum()) == 20 and not torch.isinf(out).any()

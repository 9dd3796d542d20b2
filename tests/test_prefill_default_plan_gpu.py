"""The plan that mla_prefill makes when it is given none: which kernel and
which splits it picks, and that its results are those of a plan by hand."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _args(q_lens, k_lens, heads, spare=0):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(17)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)

    def starts(lens):
        return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()

    tk = sum(k_lens)
    return (normal(sum(q_lens) + spare, heads, 192), normal(tk, heads, 256), normal(tk, 64),
            starts(q_lens), starts(k_lens), SCALE)


@pytest.fixture
def plans(monkeypatch):
    """The plans made, with the number of SMs asked for."""
    made = []
    make = binding.make_prefill_plan

    def spy(*args, **kw):
        made.append((make(*args, **kw), kw.get("num_sms")))
        return made[-1][0]

    monkeypatch.setattr(binding, "make_prefill_plan", spy)
    return made


def _same(a, b):
    import torch
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("batch", [1, 8, 64])
def test_single_rows_take_the_single_row_kernel(plans, batch):
    """One query a sequence, as a decode step has it."""
    import torch
    args = _args([1] * batch, [100 + 7 * b for b in range(batch)], 4)
    got = binding.mla_prefill(*args)
    assert plans[0][0].single_rows == 1
    by_hand = binding.make_prefill_plan(batch, 4, batch, 1, args[1].shape[0] // batch)
    want = binding.mla_prefill(*args, plan=by_hand, workspace=binding.new_workspace(by_hand))
    torch.cuda.synchronize()
    assert _same(got, want)


def test_a_ragged_batch_is_not_split_by_its_total_length(plans):
    """24 short prompts, 10,000 tokens in all: work enough, and no long keys."""
    lens = [417] * 16 + [416] * 8
    binding.mla_prefill(*_args(lens, lens, 8))
    assert plans[0][0].num_kv_splits == 1
    assert plans[0][0].workspace_bytes == binding.STATUS_BYTES


def test_the_lengths_given_are_the_plans(plans):
    import torch
    q_lens, k_lens = [1, 200, 1, 1], [3000, 300, 20, 10]
    args = _args(q_lens, k_lens, 3)
    got = binding.mla_prefill(*args, max_q_len=200, max_k_len=3000)
    plan = plans[0][0]
    by_hand = binding.make_prefill_plan(4, 3, 203, 200, 3000)
    assert bytes(plan) == bytes(by_hand) and plan.num_kv_splits > 1
    want = binding.mla_prefill(*args, plan=by_hand, workspace=binding.new_workspace(by_hand))
    torch.cuda.synchronize()
    assert _same(got, want)
    rows = binding.mla_prefill(*args, max_q_len=1)      # the hint picks the kernel alone
    torch.cuda.synchronize()
    assert plans[-1][0].single_rows == 1
    # Apart by the two results' roundings and the weights' (2^-8 each) of values
    # of at most 6: 3 * 6 / 256. A score is 192 products' sum in fp32, off by at
    # most 192 * 2^-23 |q| |k| SCALE (5e-4 at norms of 17.5) on either side.
    assert float((rows[0].float() - got[0].float()).abs().max()) <= 3 * 6 / 256
    assert float((rows[1] - got[1]).abs().max()) <= 2 * 5.1e-4


def test_the_plan_is_for_the_tensors_device(plans):
    """The SMs are those of the queries' device, not of device 0."""
    import torch
    args = _args([5, 9], [30, 40], 2)
    binding.mla_prefill(*args)
    sms = torch.cuda.get_device_properties(args[0].device).multi_processor_count
    assert plans[0][1] == sms


@pytest.mark.parametrize("q_lens,k_lens", [([], []), ([0, 0], [0, 5]), ([0], [0])])
def test_a_default_plan_without_rows(q_lens, k_lens):
    out, lse = binding.mla_prefill(*_args(q_lens, k_lens, 2))
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)

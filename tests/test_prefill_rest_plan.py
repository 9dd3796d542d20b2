"""Workspaces of prefill plans that split only the last wave's items, on the
host: sized by the SMs, not by the queries."""

import ctypes

import pytest

from mla_latent_cache_paged_gb300 import binding, build

X = 0x10000000          # an address that a refused call never reads
ROW = 128 * 4 + 4 + 8   # a partial row, its LSE, the result row it belongs to


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _plan(lib, batch, heads, total_q, max_q, max_k, splits=0, sms=152):
    plan = binding.MlaPrefillPlan()
    assert lib.mla_prefill_plan(batch, heads, total_q, max_q, max_k, splits, sms,
                                ctypes.byref(plan)) == 0
    return plan


def _call(lib, plan, nbytes):
    return lib.mla_prefill(ctypes.byref(plan), X, X, X, 2000, X, X, 1, 0.1, X, None, X, nbytes,
                           None)


@pytest.mark.parametrize("args", [(3, 128, 1536, 512, 8000), (1, 128, 1536, 1536, 8000),
                                  (1, 80, 512, 512, 8000), (1, 3, 40000, 40000, 40000)])
def test_a_split_last_wave_needs_room_for_one_part_an_sm(lib, args):
    plan = _plan(lib, *args)
    assert plan.split_rest == 1 and plan.num_kv_splits == 4
    assert plan.lse_partial_offset == plan.partial_offset + 152 * 256 * 512
    assert plan.workspace_bytes <= binding.STATUS_BYTES + 152 * 256 * ROW + 512
    assert plan.workspace_bytes % 256 == 0


def test_a_plan_that_splits_all_has_room_for_the_last_wave_alone(lib):
    for args, parts in [((2, 16, 600, 300, 1000, 5), 152), ((1, 4, 6, 2, 700, 2), 8),
                        ((1, 1, 300, 300, 2300, 64), 128)]:
        plan = _plan(lib, *args)
        rows = args[2] * args[1] * args[5]
        assert plan.split_rest == 0 and plan.num_kv_splits == args[5]
        assert plan.lse_partial_offset >= plan.partial_offset + rows * 512
        full = plan.lse_partial_offset - binding.STATUS_BYTES + rows * 4
        least = binding.STATUS_BYTES + parts * 256 * ROW
        assert plan.workspace_bytes >= max(full + binding.STATUS_BYTES, least)
        # no more than the larger of the two, up to rounding
        assert plan.workspace_bytes <= max(full + binding.STATUS_BYTES, least) + 1024
        plan.split_rest = 1
        assert _call(lib, plan, int(plan.workspace_bytes) - 1) == binding.MLA_ERR_WORKSPACE


def test_a_short_workspace_of_a_changed_plan_is_refused(lib):
    plan = _plan(lib, 1, 80, 512, 512, 8000)
    assert plan.split_rest == 1
    for rest in (1, 0):
        plan.split_rest = rest
        assert _call(lib, plan, int(plan.workspace_bytes) - 1) == binding.MLA_ERR_WORKSPACE


@pytest.mark.parametrize("field,value", [("workspace_bytes", 8192), ("partial_offset", 0),
                                         ("lse_partial_offset", 8192), ("num_sms", 200),
                                         ("num_sms", 100), ("num_kv_splits", 0),
                                         ("num_kv_splits", 65), ("single_rows", 1)])
@pytest.mark.parametrize("rest", [0, 1])
def test_an_edited_plan_is_refused(lib, field, value, rest):
    plan = _plan(lib, 1, 80, 512, 512, 8000)
    plan.split_rest = rest
    setattr(plan, field, value)
    assert _call(lib, plan, 1 << 30) == binding.MLA_ERR_INVALID_ARG

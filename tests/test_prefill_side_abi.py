"""Refusals of the prefill-side entry points, on the host (no GPU needed)."""

import ctypes

import pytest

from mla_latent_cache_paged_gb300 import binding, build

X = 0x10000000          # an address that a refused call never reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _expand(lib, fp8=False, **kw):
    a = dict(cache=X, scale=0.5, blocks=10, table=X, mb=4, first=None, cu=X, batch=2, total=100,
             heads=16, uk=X, uv=X, kv=X, pe=X, ws=X, nbytes=8192)
    a.update(kw)
    tail = (a["blocks"], a["table"], a["mb"], a["first"], a["cu"], a["batch"], a["total"],
            a["heads"], a["uk"], a["uv"], a["kv"], a["pe"], a["ws"], a["nbytes"], None)
    if fp8:
        return lib.mla_expand_kv_fp8(a["cache"], a["scale"], *tail)
    return lib.mla_expand_kv(a["cache"], *tail)


@pytest.mark.parametrize("kw,code", [
    (dict(heads=129), binding.MLA_ERR_UNSUPPORTED),
    (dict(heads=0), binding.MLA_ERR_INVALID_ARG),
    (dict(batch=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(total=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=0), binding.MLA_ERR_INVALID_ARG),
    (dict(mb=0), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=X + 16), binding.MLA_ERR_INVALID_ARG),
    (dict(kv=X + 16), binding.MLA_ERR_INVALID_ARG),
    (dict(pe=X + 4), binding.MLA_ERR_INVALID_ARG),
    (dict(uk=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(uv=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cu=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(first=X + 1), binding.MLA_ERR_INVALID_ARG),
    (dict(ws=None), binding.MLA_ERR_WORKSPACE),
    (dict(ws=X + 128), binding.MLA_ERR_WORKSPACE),
    (dict(nbytes=8191), binding.MLA_ERR_WORKSPACE),
    (dict(total=0, kv=None), binding.MLA_OK),
    (dict(batch=0, cu=None), binding.MLA_OK),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_expand_refusals(lib, kw, code, fp8):
    assert _expand(lib, fp8, **kw) == code


@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan")])
def test_expand_fp8_scale(lib, scale):
    assert _expand(lib, True, scale=scale) == binding.MLA_ERR_INVALID_ARG


def _fork(lib, **kw):
    a = dict(cache=X, layers=1, stride=0, blocks=100, size=2, ref=X, out=X, table=X, rows=4, mb=8,
             parents=X, shared=X, room=X, children=3, child=X + 4096, ws=X, nbytes=1 << 20)
    a.update(kw)
    return lib.mla_cache_fork(*(a[k] for k in ("cache", "layers", "stride", "blocks", "size", "ref",
                                               "out", "table", "rows", "mb", "parents", "shared",
                                               "room", "children", "child", "ws", "nbytes")), None)


PAGE = 64 * 576 * 2
COMMON = [
    (dict(cache=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(layers=0), binding.MLA_ERR_INVALID_ARG),
    (dict(layers=2, stride=100 * PAGE - 16), binding.MLA_ERR_INVALID_ARG),
    (dict(layers=2, stride=100 * PAGE + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=0), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=(1 << 23) - 1), binding.MLA_ERR_UNSUPPORTED),
    (dict(size=4), binding.MLA_ERR_UNSUPPORTED),
    (dict(ref=None), binding.MLA_ERR_INVALID_ARG),
    (dict(out=X + 100), binding.MLA_ERR_INVALID_ARG),      # overlaps the counts read
    (dict(rows=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(mb=0), binding.MLA_ERR_INVALID_ARG),
    (dict(ws=None), binding.MLA_ERR_WORKSPACE),
    (dict(ws=X + 64), binding.MLA_ERR_WORKSPACE),
    (dict(nbytes=8192), binding.MLA_ERR_WORKSPACE),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(children=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(children=8193), binding.MLA_ERR_UNSUPPORTED),
    (dict(parents=None), binding.MLA_ERR_INVALID_ARG),
    (dict(shared=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(child=X), binding.MLA_ERR_INVALID_ARG),          # overlaps the parents' table
    (dict(child=X + 4 * 8 * 4 - 4), binding.MLA_ERR_INVALID_ARG),
    (dict(child=X - 4 * 8 * 3 + 4), binding.MLA_ERR_INVALID_ARG),
    (dict(table=None), binding.MLA_ERR_INVALID_ARG),
])
def test_fork_refusals(lib, kw, code):
    assert _fork(lib, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(table_out=X + 4), binding.MLA_ERR_INVALID_ARG),
    (dict(lens=None), binding.MLA_ERR_INVALID_ARG),
    (dict(page_map=X + 1), binding.MLA_ERR_INVALID_ARG),
    (dict(live=X + 2), binding.MLA_ERR_INVALID_ARG),
])
def test_compact_refusals(lib, kw, code):
    a = dict(cache=X, layers=1, stride=0, blocks=100, size=2, ref=X, out=X, table=X, table_out=X,
             rows=4, mb=8, lens=X, page_map=None, live=None, ws=X, nbytes=1 << 20)
    a.update(kw)
    rc = lib.mla_cache_compact(*(a[k] for k in ("cache", "layers", "stride", "blocks", "size", "ref",
                                                "out", "table", "table_out", "rows", "mb", "lens",
                                                "page_map", "live", "ws", "nbytes")), None)
    assert rc == code


@pytest.mark.parametrize("kw,code", [
    (dict(blocks=0), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=(1 << 23) - 1), binding.MLA_ERR_UNSUPPORTED),
    (dict(out=X + 100), binding.MLA_ERR_INVALID_ARG),
    (dict(count=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(free_rows=None), binding.MLA_ERR_INVALID_ARG),
    (dict(freed=None), binding.MLA_ERR_INVALID_ARG),
    (dict(lens=None), binding.MLA_ERR_INVALID_ARG),
    (dict(ws=X + 4), binding.MLA_ERR_WORKSPACE),
])
def test_free_refusals(lib, kw, code):
    a = dict(ref=X, out=X, blocks=100, table=X, rows=4, mb=8, lens=X, free_rows=X, count=2, freed=X,
             ws=X, nbytes=8192)
    a.update(kw)
    rc = lib.mla_cache_free(*(a[k] for k in ("ref", "out", "blocks", "table", "rows", "mb", "lens",
                                             "free_rows", "count", "freed", "ws", "nbytes")), None)
    assert rc == code


def test_cache_workspace_sizes(lib):
    size = lib.mla_cache_workspace_bytes
    assert size(1, 0) > 8192 and size(1, 0) % 256 == 0
    assert size(1 << 20, 0) >= 8192 + 3 * 4 * (1 << 19)
    assert size(100, 8192) > size(100, 0)
    for blocks, children in [(0, 0), (-1, 0), ((1 << 23) - 1, 0), (10, -1), (10, 8193)]:
        assert size(blocks, children) == 0
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def _plan(lib, batch=2, heads=16, total_q=600, max_q=300, max_k=1000, splits=0, sms=152):
    plan = binding.MlaPrefillPlan()
    rc = lib.mla_prefill_plan(batch, heads, total_q, max_q, max_k, splits, sms, ctypes.byref(plan))
    return rc, plan


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), binding.MLA_ERR_INVALID_ARG),
    (dict(heads=129), binding.MLA_ERR_UNSUPPORTED),
    (dict(batch=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(total_q=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(max_q=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(max_k=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(splits=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(splits=65), binding.MLA_ERR_UNSUPPORTED),
    (dict(sms=0), binding.MLA_ERR_INVALID_ARG),
    (dict(batch=0, total_q=0, max_q=0, max_k=0), binding.MLA_OK),
])
def test_prefill_plan_refusals(lib, kw, code):
    assert _plan(lib, **kw)[0] == code
    assert lib.mla_prefill_plan(1, 1, 1, 1, 1, 0, 152, None) == binding.MLA_ERR_INVALID_ARG


def test_prefill_plan_layout_and_splits(lib):
    rc, p = _plan(lib, splits=1)
    assert rc == 0 and p.workspace_bytes == binding.STATUS_BYTES
    rc, p = _plan(lib, splits=5)
    rows = 600 * 16 * 5
    assert p.partial_offset == binding.STATUS_BYTES
    assert p.lse_partial_offset == p.partial_offset + rows * 512
    assert p.workspace_bytes >= p.lse_partial_offset + rows * 4 and p.workspace_bytes % 256 == 0
    # split only while SMs would idle, and only keys that are long enough
    assert _plan(lib, batch=1, heads=16, total_q=1, max_q=1, max_k=8192)[1].num_kv_splits > 1
    assert _plan(lib, batch=1, heads=16, total_q=200, max_q=200, max_k=300)[1].num_kv_splits == 1
    assert _plan(lib, batch=8, heads=128, total_q=8, max_q=1, max_k=8192)[1].num_kv_splits == 1
    assert _plan(lib, batch=1, heads=16, total_q=200, max_q=200, max_k=8192)[1].num_kv_splits > 1
    # the kernel follows from the longest query length
    for splits, got in [(1, 1), (3, 2), (7, 4), (64, 8)]:
        rc, p = _plan(lib, max_q=1, splits=splits)
        assert rc == 0 and p.num_kv_splits == got and p.workspace_bytes == binding.STATUS_BYTES
    for max_q, rows in [(0, 1), (1, 1), (2, 0), (4096, 0)]:
        assert _plan(lib, total_q=5000, max_q=max_q)[1].single_rows == rows


def test_prefill_plan_struct_matches_the_header(tmp_path):
    import os
    import subprocess
    src = tmp_path / "layout.c"
    src.write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "mla_decode.h"\n'
        "int main(void){printf(\"%zu %zu %zu %zu\\n\", sizeof(mla_prefill_plan_t),"
        " offsetof(mla_prefill_plan_t, num_sms), offsetof(mla_prefill_plan_t, workspace_bytes),"
        " offsetof(mla_prefill_plan_t, reserved));return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    P = binding.MlaPrefillPlan
    assert got == [ctypes.sizeof(P), P.num_sms.offset, P.workspace_bytes.offset, P.reserved.offset]
    assert os.path.exists(build.INCLUDE)


@pytest.mark.parametrize("kw,code", [
    (dict(plan=None), binding.MLA_ERR_INVALID_ARG),
    (dict(q=None), binding.MLA_ERR_INVALID_ARG),
    (dict(q=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(kv=None), binding.MLA_ERR_INVALID_ARG),
    (dict(kv=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(pe=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(total_k=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(cu_q=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cu_k=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(scale=0.0), binding.MLA_ERR_INVALID_ARG),
    (dict(scale=-1.0), binding.MLA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), binding.MLA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), binding.MLA_ERR_INVALID_ARG),
    (dict(scale=3e38), binding.MLA_ERR_INVALID_ARG),
    (dict(out=X + 16), binding.MLA_ERR_INVALID_ARG),
    (dict(out=None), binding.MLA_ERR_INVALID_ARG),
    (dict(lse=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(ws=None), binding.MLA_ERR_WORKSPACE),
    (dict(ws=X + 128), binding.MLA_ERR_WORKSPACE),
    (dict(nbytes=8192), binding.MLA_ERR_WORKSPACE),
])
def test_prefill_refusals(lib, kw, code):
    plan = _plan(lib, splits=3)[1]
    a = dict(plan=ctypes.byref(plan), q=X, kv=X, pe=X, total_k=2000, cu_q=X, cu_k=X, causal=1,
             scale=0.1, out=X, lse=None, ws=X, nbytes=int(plan.workspace_bytes))
    a.update(kw)
    assert lib.mla_prefill(*(a[k] for k in ("plan", "q", "kv", "pe", "total_k", "cu_q", "cu_k",
                                            "causal", "scale", "out", "lse", "ws", "nbytes")),
                           None) == code


@pytest.mark.parametrize("field,value", [("workspace_bytes", 8192), ("partial_offset", 0),
                                         ("lse_partial_offset", 8192), ("num_kv_splits", 0),
                                         ("num_kv_splits", 2), ("num_heads", 200), ("batch", -1),
                                         ("total_q", -5), ("num_sms", 0),
                                         ("single_rows", 2), ("single_rows", -1)])
def test_prefill_refuses_an_edited_plan(lib, field, value):
    plan = _plan(lib, splits=3)[1]
    setattr(plan, field, value)
    assert lib.mla_prefill(ctypes.byref(plan), X, X, X, 2000, X, X, 1, 0.1, X, None, X, 1 << 30,
                           None) == binding.MLA_ERR_INVALID_ARG


def test_prefill_plan_splits_the_rest_of_few_waves(lib):
    """More work than SMs, but few waves of it, the last one less than half
    full, and keys that are long enough."""
    def rest(**kw):
        p = _plan(lib, splits=0, **kw)[1]
        return p.split_rest, p.num_kv_splits > 1
    few = dict(batch=1, heads=80, total_q=512, max_q=512, max_k=8000)
    assert rest(**few) == (1, True)                                # 160 items
    assert rest(**{**few, "heads": 64}) == (0, False)             # 128: one wave, not split
    assert rest(**{**few, "heads": 120}) == (0, False)            # 240: the last is half full
    assert rest(**{**few, "heads": 76}) == (0, False)             # 152: no rest
    assert rest(**{**few, "max_k": 2000}) == (0, False)           # short
    assert rest(**{**few, "batch": 6, "total_q": 3070}) == (0, False)   # 6.3 waves
    assert rest(**{**few, "total_q": 1, "max_q": 1}) == (0, True)  # single rows: a cluster
    assert _plan(lib, splits=4, **few)[1].split_rest == 0         # asked for


@pytest.mark.parametrize("field,value", [("split_rest", 2), ("split_rest", -1)])
def test_prefill_refuses_an_edited_rest(lib, field, value):
    plan = _plan(lib, splits=3)[1]
    setattr(plan, field, value)
    assert lib.mla_prefill(ctypes.byref(plan), X, X, X, 2000, X, X, 1, 0.1, X, None, X, 1 << 30,
                           None) == binding.MLA_ERR_INVALID_ARG
    single = _plan(lib, max_q=1, splits=2)[1]
    single.split_rest = 1
    assert lib.mla_prefill(ctypes.byref(single), X, X, X, 2000, X, X, 1, 0.1, X, None, X, 1 << 30,
                           None) == binding.MLA_ERR_INVALID_ARG

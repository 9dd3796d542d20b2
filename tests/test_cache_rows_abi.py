"""Refusals of the cache's row operations, on the host (no GPU needed)."""

import pytest

from mla_latent_cache_paged_gb300 import binding, build

X = 0x10000000          # an address that a refused call never reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _write(lib, fp8, **kw):
    a = dict(kv=X, kv_stride=576, pe=X, pe_stride=576, slots=X, T=3, scale=0.5, cache=X, blocks=10,
             ws=X, nbytes=8192)
    a.update(kw)
    head = (a["kv"], a["kv_stride"], a["pe"], a["pe_stride"], a["slots"], a["T"])
    tail = (a["cache"], a["blocks"], a["ws"], a["nbytes"], None)
    return (lib.mla_cache_write_fp8(*head, a["scale"], *tail) if fp8
            else lib.mla_cache_write(*head, *tail))


def _gather(lib, fp8, **kw):
    a = dict(cache=X, scale=0.5, blocks=10, table=X, mb=4, first=None, cu=X, batch=2, total=100,
             rows=X, ws=X, nbytes=8192)
    a.update(kw)
    tail = (a["blocks"], a["table"], a["mb"], a["first"], a["cu"], a["batch"], a["total"],
            a["rows"], a["ws"], a["nbytes"], None)
    return (lib.mla_cache_gather_fp8(a["cache"], a["scale"], *tail) if fp8
            else lib.mla_cache_gather(a["cache"], *tail))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=0), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=2 ** 60), binding.MLA_ERR_UNSUPPORTED),
    (dict(kv_stride=-576), binding.MLA_ERR_INVALID_ARG),
    (dict(kv_stride=577), binding.MLA_ERR_INVALID_ARG),
    (dict(pe_stride=68), binding.MLA_ERR_INVALID_ARG),
    (dict(kv=None), binding.MLA_ERR_INVALID_ARG),
    (dict(kv=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(pe=None), binding.MLA_ERR_INVALID_ARG),
    (dict(pe=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(slots=None), binding.MLA_ERR_INVALID_ARG),
    (dict(slots=X + 4), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(ws=None), binding.MLA_ERR_WORKSPACE),
    (dict(ws=X + 64), binding.MLA_ERR_WORKSPACE),
    (dict(nbytes=8191), binding.MLA_ERR_WORKSPACE),
    (dict(T=0, kv=None, cache=None), binding.MLA_OK),
])
def test_write_refusals(lib, kw, code, fp8):
    assert _write(lib, fp8, **kw) == code


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(total=-1), binding.MLA_ERR_INVALID_ARG),
    (dict(blocks=0), binding.MLA_ERR_INVALID_ARG),
    (dict(mb=0), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cache=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(rows=None), binding.MLA_ERR_INVALID_ARG),
    (dict(rows=X + 8), binding.MLA_ERR_INVALID_ARG),
    (dict(table=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(cu=None), binding.MLA_ERR_INVALID_ARG),
    (dict(cu=X + 2), binding.MLA_ERR_INVALID_ARG),
    (dict(first=X + 1), binding.MLA_ERR_INVALID_ARG),
    (dict(ws=None), binding.MLA_ERR_WORKSPACE),
    (dict(ws=X + 128), binding.MLA_ERR_WORKSPACE),
    (dict(nbytes=100), binding.MLA_ERR_WORKSPACE),
    (dict(total=0, rows=None), binding.MLA_OK),
    (dict(batch=0, cu=None), binding.MLA_OK),
])
def test_gather_refusals(lib, kw, code, fp8):
    assert _gather(lib, fp8, **kw) == code


@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan")])
def test_fp8_scales(lib, scale):
    assert _write(lib, True, scale=scale) == binding.MLA_ERR_INVALID_ARG
    assert _gather(lib, True, scale=scale) == binding.MLA_ERR_INVALID_ARG


def test_binding_refuses_tensors_on_the_host():
    import torch
    bf16 = torch.bfloat16
    kv, pe, slots = torch.zeros(2, 512, dtype=bf16), torch.zeros(2, 64, dtype=bf16), torch.zeros(2).long()
    with pytest.raises(TypeError):
        binding.mla_cache_write(kv, pe, slots, torch.zeros(1, 64, 576, dtype=bf16), workspace=None)
    with pytest.raises(TypeError):
        binding.mla_cache_gather(torch.zeros(1, 64, 576, dtype=bf16), torch.zeros(1, 1).int(),
                                 torch.zeros(2).int(), total_k=1, workspace=None)

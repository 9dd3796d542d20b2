"""Refusals of the decodes over parts of the tokens, and their plan, on the host (no GPU needed)."""

import ctypes

import pytest

from mla_latent_cache_paged_gb300 import binding, build

X = 0x10000000          # an address that a refused call never reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _plan(batch=4, heads=16, mb=10, groups=2, sms=152, **kw):
    return binding.make_span_plan(batch, heads, mb, max_groups=groups, num_sms=sms, **kw)


def _call(lib, op, fp8, plan=None, **kw):
    plan = plan or _plan(groups=2 if op == "shared" else 0)
    a = dict(q=X, cache=X, blocks=10, table=X, lens=X, starts=X, shared=X, groups=2, window=100, sinks=4,
             scale=0.07, k_scale=0.5, out=X, lse=X, ws=X, nbytes=plan.workspace_bytes)
    a.update(kw)
    head = (ctypes.byref(plan), a["q"], a["cache"], a["blocks"], a["table"], a["lens"])
    mid = (a["starts"], a["shared"], a["groups"]) if op == "shared" else (a["window"], a["sinks"])
    scales = (a["scale"], a["k_scale"]) if fp8 else (a["scale"],)
    fn = getattr(lib, f"mla_decode_{op}" + ("_fp8" if fp8 else ""))
    return fn(*head, *mid, *scales, a["out"], a["lse"], a["ws"], a["nbytes"], None)


BAD = binding.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("op", ["shared", "window"])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(q=X + 8), BAD), (dict(cache=None), BAD), (dict(cache=X + 4), BAD),
    (dict(blocks=0), BAD), (dict(blocks=2 ** 31), binding.MLA_ERR_UNSUPPORTED),
    (dict(table=None), BAD), (dict(table=X + 1), BAD), (dict(lens=None), BAD), (dict(lens=X + 2), BAD),
    (dict(out=None), BAD), (dict(out=X + 8), BAD), (dict(lse=X + 2), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(scale=3e38, k_scale=2.0), BAD),
    (dict(ws=None), binding.MLA_ERR_WORKSPACE), (dict(ws=X + 128), binding.MLA_ERR_WORKSPACE),
    (dict(nbytes=8192), binding.MLA_ERR_WORKSPACE),
])
def test_refusals(lib, op, kw, code, fp8):
    assert _call(lib, op, fp8, **kw) == code


@pytest.mark.parametrize("kw", [dict(starts=None), dict(starts=X + 2), dict(shared=None), dict(shared=X + 1),
                                dict(groups=-1), dict(groups=3)])
def test_shared_refusals(lib, kw):
    assert _call(lib, "shared", False, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(window=0), dict(window=-5), dict(sinks=-1)])
def test_window_refusals(lib, kw):
    assert _call(lib, "window", False, **kw) == BAD


@pytest.mark.parametrize("op", ["shared", "window"])
@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan")])
def test_fp8_scales(lib, op, scale):
    assert _call(lib, op, True, k_scale=scale) == BAD


@pytest.mark.parametrize("op", ["shared", "window"])
def test_plans_that_do_not_follow_from_their_sizes(lib, op):
    for field, value in (("pairs", 77), ("pairs", 0), ("workspace_bytes", 8192), ("batch", 5), ("batch", -1),
                         ("num_heads", 129), ("max_groups", 5000), ("flags", 1), ("reserved0", 1)):
        plan = _plan()
        nbytes = plan.workspace_bytes
        setattr(plan, field, value)
        assert _call(lib, op, False, plan=plan, nbytes=nbytes) != binding.MLA_OK
    fn = lib.mla_decode_shared
    assert fn(None, X, X, 1, X, X, X, X, 0, 0.1, X, X, X, 1 << 30, None) == BAD


def test_an_empty_batch_needs_no_tensors(lib):
    plan = _plan(batch=0)
    assert _call(lib, "shared", False, plan=plan, q=None, out=None) == binding.MLA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(heads=0), BAD), (dict(mb=0), BAD), (dict(groups=-1), BAD), (dict(sms=0), BAD),
    (dict(extra_flags=1), BAD), (dict(heads=129), binding.MLA_ERR_UNSUPPORTED),
    (dict(batch=4097), binding.MLA_ERR_UNSUPPORTED), (dict(groups=4097), binding.MLA_ERR_UNSUPPORTED),
    (dict(mb=2 ** 31 - 1), binding.MLA_ERR_UNSUPPORTED),
    (dict(batch=4096, mb=2 ** 19 - 6), binding.MLA_ERR_UNSUPPORTED),
])
def test_plan_refusals(lib, kw, code):
    with pytest.raises(binding.MlaError) as e:
        _plan(**kw)
    assert e.value.status == code


def test_the_workspace_holds_the_pieces():
    """A row of fp32 results and its LSE for every row of every tile and
    request, and 128 more for every cut."""
    for batch, heads, groups, sms in ((1, 1, 0, 2), (64, 128, 1, 152), (48, 16, 5, 152), (4096, 128, 4096, 512)):
        plan = _plan(batch, heads, 10, groups, sms)
        assert plan.pairs == min(256, max(1, sms // 2))
        tiles = (batch * heads // 128 + min(groups, batch // 2)) if groups else 0
        rows = 128 * tiles + batch * heads + 128 * plan.pairs
        assert plan.workspace_bytes >= 8192 + rows * (512 * 4 + 4)


def test_binding_checks(lib):
    with pytest.raises(ValueError):
        binding._window(0, 0)
    with pytest.raises(ValueError):
        binding._window(1, -1)
    assert binding._window(2 ** 40, 2 ** 33) == (2 ** 31 - 1, 2 ** 31 - 1)

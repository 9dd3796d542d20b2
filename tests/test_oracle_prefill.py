"""Pins of the oracle's prefill-side definitions (CPU only)."""

import numpy as np
import pytest

from oracle import (absorb_query, cache_compact, cache_fork, cache_free, expand_kv,
                    mla_decode_reference, prefill_attention)

SCALE = 192 ** -0.5


@pytest.mark.parametrize("lq,lk", [(1, 1), (4, 4), (3, 7), (6, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_attention_against_torch_in_64_bits(lq, lk, causal):
    import torch
    rng = np.random.default_rng(10 * lq + lk)
    q, kv, pe = rng.standard_normal((lq, 2, 192)), rng.standard_normal((lk, 2, 256)), \
        rng.standard_normal((lk, 64))
    out, lse = prefill_attention(q, kv, pe, [lq], [lk], SCALE, causal)
    k = np.concatenate([kv[..., :128], np.repeat(pe[:, None], 2, 1)], -1)
    mask = np.ones((lq, lk), dtype=bool)
    if causal:
        mask = np.arange(lk)[None] <= np.arange(lq)[:, None] + (lk - lq)
    t = [torch.from_numpy(x.transpose(1, 0, 2).copy()) for x in (q, k, kv[..., 128:])]
    ref = torch.nn.functional.scaled_dot_product_attention(
        *t, attn_mask=torch.from_numpy(mask), scale=SCALE).numpy().transpose(1, 0, 2)
    seen = mask.any(1)
    assert np.allclose(out[seen], ref[seen], rtol=0, atol=1e-12)
    s = np.where(mask[:, None], np.einsum("ind,jnd->inj", q, k) * SCALE, -np.inf)
    want = np.log(np.exp(s[seen]).sum(-1))
    assert np.allclose(lse[seen], want, rtol=0, atol=1e-12)
    assert (out[~seen] == 0).all() and np.isneginf(lse[~seen]).all()


def test_expanded_equals_absorbed():
    """One new token over a paged cache: the expansion and the expanded
    attention give the absorbed decode's result, up-projected."""
    rng = np.random.default_rng(3)
    heads, lens = 3, [5, 130]
    table = np.array([[4, 0, 0], [2, 5, 1]])
    cache = rng.standard_normal((6, 64, 576))
    w_uk_t, w_uv = rng.standard_normal((heads, 128, 512)) / 20, rng.standard_normal((heads, 512, 128))
    q = rng.standard_normal((2, heads, 192))
    kv, pe = expand_kv(cache, table, [0, 0], lens, w_uk_t, w_uv)
    out, lse = prefill_attention(q, kv, pe, [1, 1], lens, SCALE, True)
    ql = np.einsum("bnp,npl->bnl", q[..., :128], w_uk_t)
    assert np.allclose(ql, absorb_query(q[..., :128], w_uk_t.transpose(2, 0, 1)))
    mqa = np.concatenate([ql, q[..., 128:]], -1)
    latent, z = mla_decode_reference(mqa, cache, table, np.array(lens), SCALE)
    assert np.allclose(out, np.einsum("bnl,nlv->bnv", latent, w_uv), rtol=0, atol=1e-9)
    assert np.allclose(lse, z, rtol=0, atol=1e-9)


def test_expand_kv_from_a_first_token_on():
    rng = np.random.default_rng(4)
    cache = rng.standard_normal((3, 64, 576))
    w_uk_t, w_uv = rng.standard_normal((1, 128, 512)), rng.standard_normal((1, 512, 128))
    kv, pe = expand_kv(cache, [[2, 0]], [63], [2], w_uk_t, w_uv)
    rows = np.stack([cache[2, 63], cache[0, 0]])
    assert np.array_equal(pe, rows[:, 512:])
    assert np.allclose(kv[:, 0, 5], rows[:, :512] @ w_uk_t[0, 5])
    assert np.allclose(kv[:, 0, 128 + 9], rows[:, :512] @ w_uv[0, :, 9])


def test_cache_bookkeeping_by_hand():
    # pages 0..7; row 0 holds pages 3, 5, 1 (150 tokens), row 1 page 6
    table = [[3, 5, 1], [6, -1, -1]]
    ref = [0, 1, 0, 1, 0, 1, 1, 0]
    # child 0: 130 of row 0's tokens, room for 200: shares 3 and 5, copies two
    # rows of page 1 into page 0, gets page 2; child 1: nothing, room for 10
    got, children, copies = cache_fork(ref, table, [0, -1], [130, 0], [200, 10])
    assert children == [[3, 5, 0, 2], [4]] and copies == [(1, 0, 2)]
    assert got.tolist() == [1, 1, 1, 2, 1, 2, 1, 0]
    assert cache_fork(ref, table, [-1], [0], [64 * 5]) is None       # four are free
    now, freed = cache_free(got, table, [150, 64], [0])
    assert now.tolist() == [1, 0, 1, 1, 1, 1, 1, 0] and freed == 1
    # six live; 6 is past them and goes to the free id 1
    moved, page_map, moves, live = cache_compact(now)
    assert live == 6 and moves == [(6, 1)]
    assert moved.tolist() == [1, 1, 1, 1, 1, 1, 0, 0]
    assert page_map.tolist() == [0, -1, 2, 3, 4, 5, 1, -1]

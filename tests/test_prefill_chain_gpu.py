"""The prefill side as a server runs it: fork requests from a cached prompt,
insert their new tokens, expand their pages, attend, decode, free, compact.

Tolerance against the 64-bit result from the cache's own bits: keys and values
are rounded to bf16 by the expansion, weights and results by the attention, so
with A = sum_j w_j |v_j| and e = scale * 2^-8 * max_j |q_nope| |k_j| (Cauchy's
bound on a score's error from the rounded keys),
|out - exact| <= 2^-8 |exact| + (2 * 2^-8 + 2 (e + d)) A (1 + 2^-6), d as in the
attention's own test; the absorbed path adds q's and the latent result's rounding.
"""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import (bf16_bits_to_f64, bf16_tensor_bits,
                                                    f32_to_bf16_bits)
from oracle import expand_kv, prefill_attention

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _bf16(rng, shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _dev(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _int(a, dtype=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).cuda()


def test_fork_insert_expand_prefill_decode_free_compact():
    import torch
    rng = np.random.default_rng(77)
    heads, blocks, width, new = 16, 40, 8, 70
    prompt, shared = 200, [200, 130]
    w_uk, w_uv = _bf16(rng, (heads, 128, 512), 128 ** -0.5), _bf16(rng, (heads, 512, 128), 512 ** -0.5)
    uk, uv = _dev(w_uk), _dev(w_uv)
    cache = _dev(_bf16(rng, (blocks, 64, 576)))
    refs = _int(np.zeros(blocks))
    ws = binding.new_cache_workspace(blocks, 4)
    none = _int(np.full((1, width), -1))

    # A prompt from nothing, then two requests that start from it.
    parent, _ = binding.mla_cache_fork(cache, refs, none, _int([-1]), _int([0]), _int([prompt]),
                                       workspace=ws)
    lens = [s + new for s in shared]
    table, _ = binding.mla_cache_fork(cache, refs, parent, _int([0, 0]), _int(shared), _int(lens),
                                      workspace=ws)
    assert binding.read_error(ws) == 0
    host = table.cpu().numpy()
    own = parent.cpu().numpy()[0]
    assert np.array_equal(host[0, :3], own[:3]) and np.array_equal(host[1, :2], own[:2])
    assert host[0, 3] != own[3] and host[1, 2] != own[2]

    # Their new tokens go into the cache; the same call gives the absorbed queries.
    q = _bf16(rng, (2, new, heads, 192))
    kv_c, k_pe = _bf16(rng, (2 * new, 512)), _bf16(rng, (2 * new, 64))
    slots = [host[b, (shared[b] + i) // 64] * 64 + (shared[b] + i) % 64
             for b in range(2) for i in range(new)]
    mqa_q = binding.mla_q_absorb_concat_cache(_dev(q.reshape(-1, heads, 192)), uk, _dev(kv_c),
                                              _dev(k_pe), _int(slots, np.int64), cache, workspace=ws)

    # Expanded form over everything cached, in one call.
    cu_q, cu_k = _int([0, new, 2 * new]), _int([0, lens[0], sum(lens)])
    kv, pe = binding.mla_expand_kv(cache, table, cu_k, uk, uv, total_k=sum(lens), workspace=ws)
    packed = _dev(q.reshape(-1, heads, 192))
    out, lse = binding.mla_prefill(packed, kv, pe, cu_q, cu_k, SCALE)

    # The same in two pieces: the shared context (all of it seen) and the new
    # tokens (causal), combined.
    cu_c = _int([0, shared[0], sum(shared)])
    kv_1, pe_1 = binding.mla_expand_kv(cache, table, cu_c, uk, uv, total_k=sum(shared), workspace=ws)
    kv_2, pe_2 = binding.mla_expand_kv(cache, table, cu_q, uk, uv, total_k=2 * new, workspace=ws,
                                       first_token=_int(shared))
    parts = [binding.mla_prefill(packed, kv_1, pe_1, cu_q, cu_c, SCALE, causal=False),
             binding.mla_prefill(packed, kv_2, pe_2, cu_q, cu_q, SCALE)]
    both, both_lse = binding.mla_dcp_combine(torch.stack([o for o, _ in parts]),
                                             torch.stack([z for _, z in parts]))

    # The absorbed form of the same attention, up-projected.
    latent, lse_a = binding.mla_decode_multi_token(mqa_q.view(2, new, heads, 576), cache, table,
                                                   _int(lens), SCALE)
    absorbed = binding.mla_v_up_proj(latent.view(2 * new, heads, 512), uv, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0

    values = bf16_bits_to_f64(bf16_tensor_bits(cache))
    ref_kv, ref_pe = expand_kv(values, host, [0, 0], lens, bf16_bits_to_f64(w_uk),
                               bf16_bits_to_f64(w_uv))
    q64 = bf16_bits_to_f64(q).reshape(-1, heads, 192)
    ref, z = prefill_attention(q64, ref_kv, ref_pe, [new] * 2, lens, SCALE, True)
    size_kv = np.concatenate([ref_kv[..., :128], np.abs(ref_kv[..., 128:])], -1)
    size, _ = prefill_attention(q64, size_kv, ref_pe, [new] * 2, lens, SCALE, True)
    norm_q = np.sqrt((q64 ** 2).sum(-1))
    top_k = np.sqrt((ref_kv[..., :128] ** 2).sum(-1) + (ref_pe ** 2).sum(-1)[:, None]).max(0)
    e = SCALE * norm_q * top_k * (2.0 ** -8 + 192 * 2.0 ** -23)
    tol = 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -8 + 2 * e)[..., None] * size * (1 + 2.0 ** -6)
    assert (np.abs(bf16_bits_to_f64(bf16_tensor_bits(out)) - ref) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - z) <= e + 1e-5).all()
    # (one more rounding each: the parts' results, and their combination)
    assert (np.abs(bf16_bits_to_f64(bf16_tensor_bits(both)) - ref) <= tol + 2.0 ** -8 * size).all()
    assert (np.abs(both_lse.cpu().numpy() - z) <= e + 2e-5).all()
    # (absorbed: q, the weights and the 512-wide latent result are rounded;
    # the last by 2^-8 of sum_j w_j |c_j| through W_UV)
    lat = np.concatenate([np.abs(values[host[b, t // 64], t % 64, :512])[None]
                          for b in range(2) for t in range(lens[b])])
    through = (lat.max(0) @ np.abs(bf16_bits_to_f64(w_uv))).max()
    assert (np.abs(bf16_bits_to_f64(bf16_tensor_bits(absorbed)) - ref)
            <= tol + 2 * 2.0 ** -8 * through).all()
    assert np.abs(lse_a.reshape(-1, heads).cpu().numpy() - z).max() <= e.max() + 1e-3

    # The prompt and the first request end; what is left is squeezed together
    # and still gives the second request's results, bit for bit.
    _, freed = binding.mla_cache_free(refs, parent, _int([prompt]), _int([0]), workspace=ws)
    assert int(freed) == 1            # three of its four pages are the first request's too
    _, freed = binding.mla_cache_free(refs, table, _int(lens), _int([0]), workspace=ws)
    assert int(freed) == -(-lens[0] // 64) - 2
    left = -(-lens[1] // 64)
    table, _, page_map, live = binding.mla_cache_compact(cache, refs, table, _int([0, lens[1]]),
                                                         workspace=ws)
    assert binding.read_error(ws) == 0
    assert int(live) == left and int((refs > 0).sum()) == left
    row = table[1:2].contiguous()
    assert sorted(row[0, :left].tolist()) == list(range(left))
    again, again_pe = binding.mla_expand_kv(cache, row, _int([0, lens[1]]), uk, uv, total_k=lens[1],
                                            workspace=ws)
    out2, _ = binding.mla_prefill(packed[new:], again, again_pe, _int([0, new]),
                                  _int([0, lens[1]]), SCALE)
    torch.cuda.synchronize()
    assert torch.equal(again, kv[lens[0]:]) and torch.equal(again_pe, pe[lens[0]:])
    assert torch.equal(out2, out[new:])


def test_prefill_expand_decode_and_page_calls_on_streams_of_their_own():
    """A server overlaps them: each call's result is the one it has alone. (The
    first fork asks for 720 tokens in rows of 11 pages and is refused each time;
    the second one fits.)"""
    import torch
    rng = np.random.default_rng(78)
    heads, lens = 32, [700, 130, 1, 513]
    pages = [-(-n // 64) for n in lens]
    blocks = sum(pages)
    table = np.full((len(lens), max(pages)), -1, np.int32)
    ids, at = rng.permutation(blocks), 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    cache, tab, cu = _dev(_bf16(rng, (blocks, 64, 576))), _int(table), _int(np.r_[0, np.cumsum(lens)])
    uk, uv = _dev(_bf16(rng, (heads, 128, 512), 0.05)), _dev(_bf16(rng, (heads, 512, 128), 0.05))
    q = _dev(_bf16(rng, (sum(lens), heads, 192)))
    kv, pe = _dev(_bf16(rng, (sum(lens), heads, 256))), _dev(_bf16(rng, (sum(lens), 64)))
    one, latent = _dev(_bf16(rng, (4, heads, 576))), _dev(_bf16(rng, (4, heads, 512)))
    refs, kids = _int(np.bincount(ids, minlength=blocks + 40)), _int([0, 1, 3])
    pplan = binding.make_prefill_plan(len(lens), heads, sum(lens), max(lens), max(lens))
    dplan = binding.make_plan(len(lens), heads, table.shape[1], seq_lens_host=lens)
    ews, pws, dws, uws, cws, fws = (
        binding.new_status_workspace(), binding.new_workspace(pplan), binding.new_workspace(dplan),
        binding.new_status_workspace(), binding.new_cache_workspace(blocks + 40, 3),
        binding.new_cache_workspace(blocks + 40, 3))
    big = torch.zeros((blocks + 40, 64, 576), dtype=torch.uint8, device="cuda")
    shared, room, ref_out = _int([700, 100, 64]), _int([720, 300, 64]), torch.empty_like(refs)
    fits, ref_fits = _int([704, 300, 64]), torch.empty_like(refs)
    calls = [
        lambda s: binding.mla_expand_kv(cache, tab, cu, uk, uv, total_k=sum(lens), workspace=ews,
                                        stream=s),
        lambda s: binding.mla_prefill(q, kv, pe, cu, cu, SCALE, plan=pplan, workspace=pws, stream=s),
        lambda s: binding.mla_decode(one, cache, tab, _int_lens, SCALE, plan=dplan, workspace=dws,
                                     stream=s),
        lambda s: (binding.mla_v_up_proj(latent, uv, workspace=uws, stream=s),),
        lambda s: binding.mla_cache_fork(big, refs, tab, kids, shared, room, workspace=cws,
                                         ref_counts_out=ref_out, stream=s),
        lambda s: binding.mla_cache_fork(big, refs, tab, kids, shared, fits, workspace=fws,
                                         ref_counts_out=ref_fits, stream=s),
    ]
    _int_lens = _int(lens)
    bits = lambda r: [x.view(torch.int16).clone() for x in r]   # noqa: E731
    want = []
    for call in calls:
        want.append(bits(call(None)))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(12):
        for i, (call, stream) in enumerate(zip(calls, streams)):
            got.append((i, call(stream)))
    torch.cuda.synchronize()
    for i, result in got:
        assert all(torch.equal(a, b) for a, b in zip(bits(result), want[i])), i
    assert torch.equal(ref_out, refs) and int((ref_fits != refs).sum()) > 0
    assert binding.read_error(cws) == binding.MLA_ERR_BAD_SEQ_LEN
    for ws in (ews, pws, dws, uws, fws):
        assert binding.read_error(ws) == 0

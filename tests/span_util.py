"""Problems, references and tolerances for the tests of the decodes over parts of the cached tokens.

Tolerance, from the arithmetic the calls state. With p_t the exact weights, of
a row, V_t its values and o = sum p_t V_t:
  * A score is a sum of 576 products, exact in fp32, accumulated in fp32 (the
    tensor cores may truncate: a whole step, 2^-23 of the sum of magnitudes,
    for each addition), times the scale and less the maximum in one fma (half
    a step of the larger, 2^-23 of |s| log2 e counted), then exp2 (2 steps):
    eps = scale 576 2^-23 sum|q||k| + 2^-22 max|s| + 2^-21 relative error of a
    weight.
  * A weight is rounded (u = 2^-8 for bf16, 2^-11 for f16) and the result
    normalised by the sum of the rounded ones. A relative error d_t of the
    weights moves o by at most max|d| sum p_t |V_t - o| <= max|d| (sum p_t|V_t|
    + |o|).
  * Weights below the tensor cores' smallest: bf16 has fp32's range; f16 loses
    2^-25 absolute of a weight whose row's greatest is between 2^-8 and 2^8:
    2^-17 of sum |V_t| over the tokens, counted with the weights' sum.
  * Sums over L tokens in fp32, and the merge: (L + 64) 2^-22 of the same sum.
  * One rounding of o to bf16: 2^-8 |o|.
The LSE is off by eps, the error of summing the weights and of the logarithm:
eps + (L + 64) 2^-22 + 2^-20 + 2^-22 |lse|.
"""

import numpy as np

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import (bf16_bits_to_f64, bf16_tensor_bits,
                                                    f32_to_bf16_bits)
from oracle import e4m3_to_float

SCALE = 192 ** -0.5
K_SCALE = float(np.float32(5.5 / 448))


def dev(bits):
    import torch
    if bits.dtype == np.uint8:
        return torch.from_numpy(np.ascontiguousarray(bits)).cuda()
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def ints(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def values(cache):
    return e4m3_to_float(cache) * K_SCALE if cache.dtype == np.uint8 else bf16_bits_to_f64(cache)


def random_cache(rng, blocks, fp8):
    x = rng.standard_normal((blocks, 64, 576)).astype(np.float32)
    if fp8:
        from mla_latent_cache_paged_gb300.workloads import f32_to_e4m3_bits
        return f32_to_e4m3_bits(x / np.float32(K_SCALE))
    return f32_to_bf16_bits(x)


def random_q(rng, batch, heads, gain=1.0):
    return f32_to_bf16_bits((rng.standard_normal((batch, heads, 576)) * gain).astype(np.float32))


NAN = {True: 0x7F, False: 0x7FC0}


def shared_problem(rng, lens, starts, shared, fp8, extra=2):
    """Pages of a batch whose groups share whole pages; rows past each
    request's end hold NaN, unused entries name no page."""
    lens = np.asarray(lens)
    width = max(1, int(-(-lens.max() // 64)))
    table = np.full((len(lens), width), -7, dtype=np.int64)
    tail = []
    used = 0
    for g in range(len(shared)):
        members = [b for b in range(starts[g], starts[g + 1])]
        reach = max([int(lens[b]) for b in members], default=0)
        n = min(shared[g], reach) // 64            # pages that the group has together
        for b in members:
            have = min(n, -(-int(lens[b]) // 64))
            table[b, :have] = used + np.arange(have)
        used += n
    for b, L in enumerate(lens):
        for j in range(-(-int(L) // 64)):
            if table[b, j] == -7:
                table[b, j] = used
                used += 1
                if j == (int(L) - 1) // 64 and L % 64:
                    tail.append((table[b, j], int(L) % 64))
    ids = rng.permutation(used + extra)
    cache = random_cache(rng, used + extra, fp8)
    for page, at in tail:
        cache[ids[page], at:] = NAN[fp8]
    for page in ids[used:]:
        cache[page] = NAN[fp8]
    table = np.where(table >= 0, ids[np.maximum(table, 0)], 2 ** 30)
    return cache, table.astype(np.int32)


def reference(q, cache, table, seen, scale):
    """out, lse and their tolerances' parts, request b over the tokens seen[b]."""
    q = bf16_bits_to_f64(q)
    fp8 = cache.dtype == np.uint8
    B, N, _ = q.shape
    out, lse = np.zeros((B, N, 512)), np.full((B, N), -np.inf)
    tol, lse_tol = np.zeros((B, N, 512)), np.zeros((B, N))
    u = 2.0 ** -11 if fp8 else 2.0 ** -8
    for b, t in enumerate(seen):
        t = np.asarray(t, dtype=np.int64)
        if t.size == 0:
            continue
        k = values(cache[table[b, t // 64], t % 64])
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (q[b] @ k.T)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(-1, keepdims=True)
            out[b], lse[b] = (p / z) @ k[:, :512], (m + np.log(z))[:, 0]
            size = (p / z) @ np.abs(k[:, :512])
            eps = (abs(scale) * 576 * 2.0 ** -23 * (np.abs(q[b]) @ np.abs(k).T).max(-1)
                   + 2.0 ** -22 * np.abs(s).max(-1) + 2.0 ** -21)
            add = (t.size + 64) * 2.0 ** -22
            rel = u * (1 + 2 * u) + 2 * eps + add
            tol[b] = 2.0 ** -8 * np.abs(out[b]) * (1 + 2.0 ** -8) + rel[:, None] * (size + np.abs(out[b]))
            if fp8:
                tol[b] += 2.0 ** -17 * np.abs(k[:, :512]).sum(0) / z
            lse_tol[b] = eps + add + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[b])
    return out, lse, tol, lse_tol


def check(got_out, got_lse, ref, what=""):
    out, lse, tol, lse_tol = ref
    g = bf16_bits_to_f64(bf16_tensor_bits(got_out))
    z = got_lse.double().cpu().numpy()
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (what, "out", int(bad.sum()), np.argwhere(bad)[0],
                           np.nanmax(np.abs(g - out) / np.maximum(tol, 1e-30)))
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(z), empty), (what, "empty rows")
    assert not (np.abs(z[~empty] - lse[~empty]) > lse_tol[~empty]).any(), (
        what, "lse", np.abs(z[~empty] - lse[~empty]).max())


def run_shared(q, cache, table, lens, starts, shared, scale=SCALE, num_sms=None, plan=None, ws=None, **kw):
    B, N, _ = q.shape
    if plan is None:
        plan = binding.make_span_plan(B, N, table.shape[1], max_groups=len(shared), num_sms=num_sms)
    if ws is None:
        ws = binding.new_workspace(plan)
    args = (dev(q), dev(cache), ints(table), ints(lens), ints(starts), ints(shared), scale)
    if cache.dtype == np.uint8:
        out, lse = binding.mla_decode_shared_fp8(*args, K_SCALE, plan=plan, workspace=ws, **kw)
    else:
        out, lse = binding.mla_decode_shared(*args, plan=plan, workspace=ws, **kw)
    return out, lse, ws


def run_window(q, cache, table, lens, window, sinks, scale=SCALE, num_sms=None, **kw):
    B, N, _ = q.shape
    plan = binding.make_span_plan(B, N, table.shape[1], num_sms=num_sms)
    ws = binding.new_workspace(plan)
    args = (dev(q), dev(cache), ints(table), ints(lens), scale)
    kw.update(window=window, sinks=sinks, plan=plan, workspace=ws)
    if cache.dtype == np.uint8:
        out, lse = binding.mla_decode_window_fp8(*args, K_SCALE, **kw)
    else:
        out, lse = binding.mla_decode_window(*args, **kw)
    return out, lse, ws

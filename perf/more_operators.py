"""Cases that measure the operators around a shared, windowed or quantised latent cache: the decode of batches whose
requests share a cached prefix, the decode through a sliding window with sink tokens, the write of new tokens' entries
(bf16, or quantised to E4M3) and the read-back of cached rows.

``own = False`` computes each operator with elementary torch operations in fp32 (the quantisation in fp64: its
quotients lie next to rounding borders); ``own = True`` makes the calls of this package's binding. The writes change
the cache in place, with the same entries each time, so a pass can be repeated on one state.
"""

import math
import random

import numpy as np
import torch

own = False

LKV, R, PAGE = 512, 64, 64
D = LKV + R
SCALE = 1.0 / math.sqrt(192)
K_SCALE = float(np.float32(5.5 / 448))     # an fp8 cache's calibrated scale: N(0, 1) entries rarely saturate


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # Decode of requests that share a prefix. A few chats over one system prompt, 16 heads per rank: latency.
        {"name": "shared_chats_b8_n16", "op": "shared", "groups": 1, "batch": 8, "heads": 16, "pre_lo": 500,
         "pre_hi": 500, "own_lo": 20, "own_hi": 300, "fp8": False, "shape_seed": 11},
        # Several documents, each asked about by a handful of requests; prefixes that end inside a page.
        {"name": "shared_documents_b48_n16", "op": "shared", "groups": 5, "batch": 48, "heads": 16, "pre_lo": 1000,
         "pre_hi": 6000, "own_lo": 1, "own_hi": 900, "fp8": False, "shape_seed": 12},
        # Two long prefixes in an fp8 cache.
        {"name": "shared_fp8_b64_n32", "op": "shared", "groups": 2, "batch": 64, "heads": 32, "pre_lo": 8000,
         "pre_hi": 12000, "own_lo": 50, "own_hi": 1000, "fp8": True, "shape_seed": 13},
        # All heads on the GPU, 64 samples from one long prompt.
        {"name": "shared_long_b64_n128", "op": "shared", "groups": 1, "batch": 64, "heads": 128, "pre_lo": 16384,
         "pre_hi": 16384, "own_lo": 100, "own_hi": 1500, "fp8": False, "shape_seed": 14},
        # Decode through a window. A few requests, a short window: latency.
        {"name": "window_b4_n16_w256", "op": "window", "batch": 4, "heads": 16, "window": 256, "sinks": 4,
         "len_lo": 100, "len_hi": 2000, "fp8": False, "shape_seed": 21},
        # A full batch of 128 with all heads, a window of 1024 tokens.
        {"name": "window_b128_n128_w1024", "op": "window", "batch": 128, "heads": 128, "window": 1024, "sinks": 4,
         "len_lo": 500, "len_hi": 8192, "fp8": False, "shape_seed": 22},
        # Lengths from 16 to 32K, an odd window, an fp8 cache.
        {"name": "window_fp8_b96_n32_w4000", "op": "window", "batch": 96, "heads": 32, "window": 4000, "sinks": 70,
         "len_lo": 16, "len_hi": 32768, "fp8": True, "shape_seed": 23},
        # New tokens' entries into the cache. One decode step of 32 requests.
        {"name": "write_step_t32", "op": "write", "tokens": 32, "fp8": False, "shape_seed": 31},
        # One decode step of 256 requests with an fp8 cache.
        {"name": "write_fp8_step_t256", "op": "write", "tokens": 256, "fp8": True, "shape_seed": 32},
        # A scheduler's chunk of prompt tokens with an fp8 cache.
        {"name": "write_fp8_chunk_t16384", "op": "write", "tokens": 16384, "fp8": True, "shape_seed": 33},
        # Cached rows read back. One piece of context of a few requests.
        {"name": "gather_b6", "op": "gather", "batch": 6, "len_lo": 900, "len_hi": 1800, "first_hi": 4000,
         "fp8": False, "shape_seed": 41},
        # A large batch's whole context out of an fp8 cache.
        {"name": "gather_fp8_b24", "op": "gather", "batch": 24, "len_lo": 500, "len_hi": 8000, "first_hi": 100,
         "fp8": True, "shape_seed": 42},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "window", "window", "write", "gather"])
    seed, fp8 = rng.randrange(1 << 30), rng.random() < 0.4
    if op == "shared":
        batch, heads = _log_int(rng, 1, 256), _log_int(rng, 1, 128)
        tokens = 1.2e8 / (batch * heads)                    # (the largest listed case has 1.4e8 rows x tokens)
        pre = _log_int(rng, 1, int(max(2, min(32768, tokens))))
        mine = _log_int(rng, 1, int(max(2, min(2000, tokens / 4))))
        return {"op": op, "groups": rng.randint(1, min(batch, 8)), "batch": batch, "heads": heads,
                "pre_lo": rng.randint(0, pre), "pre_hi": pre, "own_lo": rng.randint(0, mine), "own_hi": mine,
                "fp8": fp8, "shape_seed": seed}
    if op == "window":
        batch, heads = _log_int(rng, 1, 256), _log_int(rng, 1, 128)
        window = _log_int(rng, 1, int(min(8192, 4e5 / batch)))
        hi = _log_int(rng, 1, 32768 if batch <= 128 else 16384)
        return {"op": op, "batch": batch, "heads": heads, "window": window, "sinks": rng.choice([0, 1, 4, 64, 130]),
                "len_lo": rng.randint(1, hi), "len_hi": hi, "fp8": fp8, "shape_seed": seed}
    if op == "write":
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "fp8": fp8, "shape_seed": seed}
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, int(min(16000, 1.2e5 / batch)))
    return {"op": op, "batch": batch, "len_lo": rng.randint(batch == 1, hi), "len_hi": hi,
            "first_hi": rng.choice([0, _log_int(rng, 1, 5000)]), "fp8": fp8, "shape_seed": seed}


def _uniform(r, lo, hi, count):
    return [r.randint(lo, hi) for _ in range(count)]


def _shapes(case):
    """The whole numbers of a case that its work follows from."""
    r = random.Random(case["shape_seed"])
    op = case["op"]
    if op == "shared":
        # group starts, the groups' prefixes (of which whole pages are shared), the requests' lengths
        cuts = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1))
        starts = [0] + cuts + [case["batch"]]
        pre = _uniform(r, case["pre_lo"], case["pre_hi"], case["groups"])
        mine = _uniform(r, case["own_lo"], case["own_hi"], case["batch"])
        of = [g for g in range(case["groups"]) for _ in range(starts[g], starts[g + 1])]
        return starts, pre, [pre[g] + n for g, n in zip(of, mine)], of
    if op == "window":
        lo, hi = math.log(case["len_lo"]), math.log(case["len_hi"])
        return [int(round(math.exp(r.uniform(lo, hi)))) for _ in range(case["batch"])]
    if op == "write":
        return [t for t in range(case["tokens"]) if r.random() < 0.97]       # the others are padding
    return (_uniform(r, case["len_lo"], case["len_hi"], case["batch"]),
            _uniform(r, 0, case["first_hi"], case["batch"]))


def _whole(n):
    """The tokens of the whole pages of a prefix."""
    return n // PAGE * PAGE


def work(case):
    op, entry = case["op"], D * (1 if case["fp8"] else 2)
    if op == "shared":
        starts, pre, lens, of = _shapes(case)
        b, n = case["batch"], case["heads"]
        cached = sum(_whole(p) for p in pre) + sum(l - _whole(pre[g]) for l, g in zip(lens, of))
        return {"bytes": cached * entry + b * n * (2 * D + 2 * LKV + 4), "flops": 2 * n * (D + LKV) * sum(lens)}
    if op == "window":
        b, n = case["batch"], case["heads"]
        seen = sum(min(l, case["window"] + case["sinks"]) for l in _shapes(case))
        return {"bytes": seen * entry + b * n * (2 * D + 2 * LKV + 4), "flops": 2 * n * (D + LKV) * seen}
    if op == "write":
        there = len(_shapes(case))
        return {"bytes": there * (2 * D + entry) + 8 * case["tokens"], "flops": 0}
    total = sum(_shapes(case)[0])
    return {"bytes": total * (entry + 2 * D), "flops": 0}


# ----------------------------------------------------------------------------------------------- inputs

def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _int32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def _cache(case, blocks, gen):
    shape = (blocks, PAGE, D)
    if case["fp8"]:
        return (torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=gen) / K_SCALE).clamp(
            -448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _normal(shape, gen)


def _query(case, gen):
    gain = torch.rand((1, case["heads"], 1), device="cuda", generator=gen) * 3 + 0.5       # flat and peaked heads
    return (_normal((case["batch"], case["heads"], D), gen, torch.float32) * gain * 0.6).to(torch.bfloat16)


def _table(lens, ids):
    """The rows' page ids, one row after another from `ids`; entries past a row's pages are -1."""
    pages = [-(-n // PAGE) for n in lens]
    table = np.full((len(lens), max(1, max(pages))), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = ids[at:at + n]
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    op = case["op"]
    s = {"case": case}
    if op == "shared":
        starts, pre, lens, of = _shapes(case)
        shared = [p // PAGE for p in pre]
        mine = [l - PAGE * shared[g] for l, g in zip(lens, of)]
        pages = sum(shared) + sum(-(-n // PAGE) for n in mine)
        ids = rs.permutation(pages + 3)
        prefix = np.split(ids[:sum(shared)], np.cumsum(shared)[:-1])
        tail = _table(mine, ids[sum(shared):])
        table = np.full((len(lens), max(1, max(-(-l // PAGE) for l in lens))), -1, dtype=np.int32)
        for b, g in enumerate(of):
            n = -(-mine[b] // PAGE)
            table[b, :shared[g]] = prefix[g]
            table[b, shared[g]:shared[g] + n] = tail[b, :n]
        s["q"], s["cache"], s["table"], s["lens"] = _query(case, gen), _cache(case, pages + 3, gen), _int32(table), _int32(lens)
        s["starts"], s["pre"] = _int32(starts), _int32(pre)
        s["host"] = (starts, pre, lens)
    elif op == "window":
        lens = _shapes(case)
        pages = sum(-(-n // PAGE) for n in lens)
        s["q"], s["cache"] = _query(case, gen), _cache(case, pages + 3, gen)
        s["table"], s["lens"] = _int32(_table(lens, rs.permutation(pages + 3))), _int32(lens)
        s["host"] = lens
    elif op == "write":
        there, tokens = _shapes(case), case["tokens"]
        blocks = -(-tokens // PAGE) + 7
        # the latent projection's output: both parts lie in one row
        latent = _normal((tokens, D), gen)
        s["kv_c"], s["k_pe"] = latent[:, :LKV], latent[:, LKV:]
        slots = np.full(tokens, -1, dtype=np.int64)
        if tokens > 1024:               # a chunk: its pages in any order, their rows in order
            slots[there] = (rs.permutation(blocks)[:, None] * PAGE + np.arange(PAGE)).reshape(-1)[:len(there)]
        else:                           # a step: a row of some page each
            slots[there] = rs.permutation(blocks * PAGE)[:len(there)]
        s["slots"] = torch.tensor(slots, device="cuda")
        s["cache"] = _cache(case, blocks, gen)
    else:
        lens, first = _shapes(case)
        held = [a + b for a, b in zip(lens, first)]
        pages = sum(-(-n // PAGE) for n in held)
        s["cache"], s["table"] = _cache(case, pages + 3, gen), _int32(_table(held, rs.permutation(pages + 3)))
        s["cu_k"], s["first"], s["total_k"] = _int32(np.concatenate([[0], np.cumsum(lens)])), _int32(first), sum(lens)
    if own:
        from mla_latent_cache_paged_gb300 import binding as mla
        if op in ("shared", "window"):
            s["plan"] = mla.make_span_plan(case["batch"], case["heads"], s["table"].shape[1],
                                           max_groups=case.get("groups", 0))
            s["ws"] = mla.new_workspace(s["plan"])
        else:
            s["ws"] = mla.new_status_workspace()
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _entries(s, table, pos):
    """The fp32 cache entries at token positions `pos` [..., T] of the table rows `table` [..., M]."""
    rows = s["cache"][table.gather(-1, pos // PAGE).long(), pos % PAGE]
    return rows.view(torch.float8_e4m3fn).float() * K_SCALE if s["case"]["fp8"] else rows.float()


def _softmax(scores):
    """Weights that are not normalised yet, their sums, and the LSE; a row of -inf gives zeros."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    return weights, torch.where(total == 0, torch.ones_like(total), total), (torch.log(total) + top)[..., 0]


def _plain_shared(s):
    starts, pre, lens = s["host"]
    n = s["q"].shape[1]
    out, lse = [], []
    for g, p in enumerate(map(_whole, pre)):
        a, e = starts[g], starts[g + 1]
        q, width = s["q"][a:e].float(), max(lens[a:e]) - p
        at = torch.arange(p, device="cuda")
        k = _entries(s, s["table"][a], at)                                           # the prefix, once
        scores = torch.empty((e - a, n, p + width), device="cuda")
        scores[..., :p] = torch.matmul(q, k.t())
        pos = p + torch.arange(width, device="cuda").expand(e - a, -1)
        there = pos < s["lens"][a:e, None]
        mine = _entries(s, s["table"][a:e], torch.where(there, pos, 0))
        scores[..., p:] = torch.matmul(q, mine.transpose(1, 2))
        scores *= SCALE
        scores[..., p:].masked_fill_(~there[:, None], -math.inf)
        weights, total, z = _softmax(scores)
        o = torch.matmul(weights[..., p:], mine[..., :LKV])
        if p:
            o += torch.matmul(weights[..., :p], k[:, :LKV])
        out.append((o / total).to(torch.bfloat16))
        lse.append(z)
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _plain_window(s):
    case, lens = s["case"], s["lens"].long()[:, None]
    window, sinks = case["window"], case["sinks"]
    first = (lens - window).clamp(min=sinks)            # the window's first token behind the sinks
    i = torch.arange(min(sinks + window, max(s["host"])), device="cuda")
    pos = torch.where(i < sinks, i, first + i - sinks)
    there = pos < lens
    k = _entries(s, s["table"], torch.where(there, pos, 0))
    scores = torch.matmul(s["q"].float(), k.transpose(1, 2)) * SCALE
    scores.masked_fill_(~there[:, None], -math.inf)
    weights, total, z = _softmax(scores)
    return {"out": (torch.matmul(weights, k[..., :LKV]) / total).to(torch.bfloat16), "lse": z}


def _plain_write(s):
    rows = torch.cat([s["kv_c"], s["k_pe"]], 1)
    there = s["slots"] >= 0
    if s["case"]["fp8"]:
        x = (rows.double() / K_SCALE).clamp(-448, 448)
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        rows = (torch.round(x / step) * step).float().to(torch.float8_e4m3fn).view(torch.uint8)
    s["cache"].view(-1, D)[s["slots"][there]] = rows[there]
    return {"cache": s["cache"].view(torch.float8_e4m3fn) if s["case"]["fp8"] else s["cache"]}


def _plain_gather(s):
    t = torch.arange(s["total_k"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu_k"][1:], t, right=True)
    pos = (t - s["cu_k"][b] + s["first"][b]).long()
    return {"rows": _entries(s, s["table"][b], pos[:, None])[:, 0].to(torch.bfloat16)}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"shared": _plain_shared, "window": _plain_window, "write": _plain_write, "gather": _plain_gather}[op](s)
    from mla_latent_cache_paged_gb300 import binding as mla
    if op == "shared":
        if case["fp8"]:
            out, lse = mla.mla_decode_shared_fp8(s["q"], s["cache"], s["table"], s["lens"], s["starts"], s["pre"],
                                                 SCALE, K_SCALE, plan=s["plan"], workspace=s["ws"])
        else:
            out, lse = mla.mla_decode_shared(s["q"], s["cache"], s["table"], s["lens"], s["starts"], s["pre"],
                                             SCALE, plan=s["plan"], workspace=s["ws"])
        return {"out": out, "lse": lse}
    if op == "window":
        if case["fp8"]:
            out, lse = mla.mla_decode_window_fp8(s["q"], s["cache"], s["table"], s["lens"], SCALE, K_SCALE,
                                                 window=case["window"], sinks=case["sinks"], plan=s["plan"],
                                                 workspace=s["ws"])
        else:
            out, lse = mla.mla_decode_window(s["q"], s["cache"], s["table"], s["lens"], SCALE, window=case["window"],
                                             sinks=case["sinks"], plan=s["plan"], workspace=s["ws"])
        return {"out": out, "lse": lse}
    if op == "write":
        if case["fp8"]:
            mla.mla_cache_write_fp8(s["kv_c"], s["k_pe"], s["slots"], s["cache"], K_SCALE, workspace=s["ws"])
            return {"cache": s["cache"].view(torch.float8_e4m3fn)}
        mla.mla_cache_write(s["kv_c"], s["k_pe"], s["slots"], s["cache"], workspace=s["ws"])
        return {"cache": s["cache"]}
    if case["fp8"]:
        return {"rows": mla.mla_cache_gather_fp8(s["cache"], s["table"], s["cu_k"], K_SCALE, total_k=s["total_k"],
                                                 first_token=s["first"], workspace=s["ws"])}
    return {"rows": mla.mla_cache_gather(s["cache"], s["table"], s["cu_k"], total_k=s["total_k"],
                                         first_token=s["first"], workspace=s["ws"])}


# ---------------------------------------------------------------------------------------- from definitions

def _values(s, at):
    """The entries in the slots `at`, in 64 bits."""
    rows = s["cache"].view(-1, D)[at]
    return rows.view(torch.float8_e4m3fn).double() * K_SCALE if s["case"]["fp8"] else rows.double()


def _slots(s, b, tokens):
    """Where the tokens (a list of ranges) of request b lie."""
    t = torch.cat([torch.arange(lo, hi, device="cuda") for lo, hi in tokens])
    return s["table"][b].long()[t // PAGE] * PAGE + t % PAGE


def exact(case, seed):
    """What ``run`` returns, in 64 bits, one request at a time."""
    s = prepare(case, seed)
    op, fp8 = case["op"], case["fp8"]
    if op in ("shared", "window"):
        lens = s["host"] if op == "window" else s["host"][2]
        out = torch.zeros((case["batch"], case["heads"], LKV), dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, l in enumerate(lens):
            seen = [(0, l)]
            if op == "window" and case["sinks"] + case["window"] < l:
                seen = [(0, case["sinks"]), (l - case["window"], l)]
            if l == 0:
                continue
            k = _values(s, _slots(s, b, seen))
            x = (s["q"][b].double() @ k.t()) * SCALE
            z = torch.logsumexp(x, -1)
            out[b], lse[b] = torch.exp(x - z[:, None]) @ k[:, :LKV], z
        return {"out": out, "lse": lse}
    if op == "gather":
        lens, first = _shapes(case)
        at = [_slots(s, b, [(f, f + l)]) for b, (l, f) in enumerate(zip(lens, first))]
        return {"rows": _values(s, torch.cat(at))}
    held = s["cache"].view(torch.float8_e4m3fn).double() if fp8 else s["cache"].double()
    x = torch.cat([s["kv_c"], s["k_pe"]], 1).double()
    if fp8:
        # the nearest of the format's 127 magnitudes; halfway the one with an even code
        grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        q = (x.abs() / K_SCALE).contiguous()
        hi = torch.searchsorted(grid, q).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - q, q - grid[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        x = torch.where(q >= 448, 448.0, grid[code]) * torch.sign(x)
    there = s["slots"] >= 0
    held.view(-1, D)[s["slots"][there]] = x[there]
    return {"cache": held}

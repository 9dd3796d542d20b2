"""Cases that measure the prefill-side operators: the expansion of paged latent rows, the expanded-form
attention over them, and the page bookkeeping (fork, free, compact) of the latent cache.

``own = False`` computes each operator with elementary torch operations in fp32; ``own = True`` makes the calls
of this package's binding. The page operators write the cache in place but only pages that are free before the
call, and take their counts and tables out of place, so a pass can be repeated on one state.
"""

import math
import random

import numpy as np
import torch

own = False

P, R, LKV, V = 128, 64, 512, 128      # qk_nope, rope, latent and v widths
QD, D, PAGE = P + R, LKV + R, 64
SCALE = 1.0 / math.sqrt(QD)


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # Expanded-form attention. One new token per request over its own context (a short decode step
        # taken through the prefill path): latency counts.
        {"name": "prefill_step_b8_n16", "op": "prefill", "batch": 8, "heads": 16, "q_lo": 1, "q_hi": 1,
         "ctx_lo": 100, "ctx_hi": 1500, "causal": True, "shape_seed": 11},
        # A batch of fresh prompts of very different lengths on one of 8 tensor-parallel ranks (16 heads).
        {"name": "prefill_prompts_b24_n16", "op": "prefill", "batch": 24, "heads": 16, "q_lo": 1, "q_hi": 1000,
         "ctx_lo": 0, "ctx_hi": 0, "causal": True, "shape_seed": 12},
        # A scheduler's chunk of about 500 new tokens per request over thousands of cached ones.
        {"name": "prefill_chunk_b4_n32", "op": "prefill", "batch": 4, "heads": 32, "q_lo": 450, "q_hi": 520,
         "ctx_lo": 2500, "ctx_hi": 6000, "causal": True, "shape_seed": 13},
        # One long prompt with all 128 heads on the GPU.
        {"name": "prefill_long_b1_n128_l4096", "op": "prefill", "batch": 1, "heads": 128, "q_lo": 4096,
         "q_hi": 4096, "ctx_lo": 0, "ctx_hi": 0, "causal": True, "shape_seed": 14},
        # Expansion of a few short contexts of an fp8 cache.
        {"name": "expand_fp8_b4_n16", "op": "expand", "batch": 4, "heads": 16, "len_lo": 20, "len_hi": 200,
         "first_hi": 100, "fp8": True, "shape_seed": 21},
        # Expansion of one workspace-sized piece of context for all heads, bf16 cache.
        {"name": "expand_bf16_b6_n128", "op": "expand", "batch": 6, "heads": 128, "len_lo": 1000, "len_hi": 1700,
         "first_hi": 4000, "fp8": False, "shape_seed": 22},
        # A beam of 8 from 2 requests, one layer.
        {"name": "fork_beam_c8", "op": "fork", "layers": 1, "blocks": 512, "parents": 2, "children": 8,
         "len_lo": 100, "len_hi": 700, "room": 64, "fp8": False, "shape_seed": 31},
        # 400 requests that start from 16 cached prompts, 8 layers at once.
        {"name": "fork_prefix_c400", "op": "fork", "layers": 8, "blocks": 8192, "parents": 16, "children": 400,
         "len_lo": 2000, "len_hi": 8000, "room": 512, "fp8": False, "shape_seed": 32},
        # A handful of requests end.
        {"name": "free_r6", "op": "free", "blocks": 512, "rows": 12, "freed": 6, "len_lo": 1, "len_hi": 900,
         "shape_seed": 41},
        # A large batch of long requests ends at once.
        {"name": "free_r500", "op": "free", "blocks": 262144, "rows": 512, "freed": 500, "len_lo": 1000,
         "len_hi": 32768, "shape_seed": 42},
        # A small pool squeezed together.
        {"name": "compact_small", "op": "compact", "layers": 1, "blocks": 300, "rows": 9, "len_lo": 1,
         "len_hi": 1200, "moved": 25, "fp8": False, "shape_seed": 51},
        # A fragmented pool of 8 layers: half of its live pages move.
        {"name": "compact_large", "op": "compact", "layers": 8, "blocks": 8192, "rows": 60, "len_lo": 1000,
         "len_hi": 8192, "moved": 1900, "fp8": False, "shape_seed": 52},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "expand", "expand", "fork", "free", "compact"])
    seed = rng.randrange(1 << 30)
    if op == "prefill":
        batch, heads = _log_int(rng, 1, 32), _log_int(rng, 1, 128)
        causal = rng.random() < 0.7
        most = (2e9 if causal else 1e9) / (batch * heads)        # score elements of the padded batch
        q_hi = _log_int(rng, 1, int(min(4096, math.sqrt(most))))
        ctx_hi = rng.choice([0, _log_int(rng, 1, int(max(1, min(16000, most / q_hi - q_hi))))])
        return {"op": op, "batch": batch, "heads": heads, "q_lo": rng.randint(1, q_hi), "q_hi": q_hi,
                "ctx_lo": rng.randint(0, ctx_hi), "ctx_hi": ctx_hi, "causal": causal, "shape_seed": seed}
    if op == "expand":
        batch, heads = _log_int(rng, 1, 32), _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, int(min(8000, 6.5e8 / 642 / heads / batch)))
        return {"op": op, "batch": batch, "heads": heads, "len_lo": rng.randint(batch == 1, hi), "len_hi": hi,
                "first_hi": rng.choice([0, _log_int(rng, 1, 5000)]), "fp8": rng.random() < 0.5,
                "shape_seed": seed}
    if op == "fork":
        children, hi = _log_int(rng, 1, 400), _log_int(rng, 1, 8000)
        parents, room = rng.randint(1, 16), _log_int(rng, 1, 512)
        need = parents * -(-hi // PAGE) + children * (2 + room // PAGE)
        return {"op": op, "layers": rng.randint(1, 4 if need > 4000 else 8), "blocks": need + _log_int(rng, 1, 2000),
                "parents": parents, "children": children, "len_lo": rng.randint(1, hi), "len_hi": hi, "room": room,
                "fp8": rng.random() < 0.3, "shape_seed": seed}
    rows, hi = _log_int(rng, 1, 512), _log_int(rng, 1, 32768)
    if op == "free":
        return {"op": op, "blocks": rows * -(-hi // PAGE) + _log_int(rng, 1, 1000), "rows": rows,
                "freed": rng.randint(1, rows), "len_lo": rng.randint(0, hi), "len_hi": hi, "shape_seed": seed}
    rows = min(rows, max(1, int(5000 * PAGE / (hi + PAGE))))
    pages = rows * -(-hi // PAGE)
    moved = rng.randint(0, max(1, pages // 4))
    layers = max(1, min(8, int(1900 * 8 / max(1, moved)), int(60000 / (pages + moved + 64))))
    return {"op": op, "layers": layers, "blocks": pages + moved + _log_int(rng, 1, 500), "rows": rows,
            "len_lo": rng.randint(0, hi), "len_hi": hi, "moved": moved, "fp8": rng.random() < 0.3,
            "shape_seed": seed}


def _uniform(r, lo, hi, count):
    return [r.randint(lo, hi) for _ in range(count)]


def _shapes(case):
    """The whole numbers of a case that its work follows from."""
    r = random.Random(case["shape_seed"])
    op = case["op"]
    if op == "prefill":
        lq = _uniform(r, case["q_lo"], case["q_hi"], case["batch"])
        lk = [a + c for a, c in zip(lq, _uniform(r, case["ctx_lo"], case["ctx_hi"], case["batch"]))]
        return lq, lk
    if op == "expand":
        return (_uniform(r, case["len_lo"], case["len_hi"], case["batch"]),
                _uniform(r, 0, case["first_hi"], case["batch"]))
    if op == "fork":
        lens = _uniform(r, case["len_lo"], case["len_hi"], case["parents"])
        parents = _uniform(r, 0, case["parents"] - 1, case["children"])
        shared = [r.randint(0, lens[p]) if r.random() < 0.5 else lens[p] for p in parents]
        return lens, parents, shared, [s + r.randint(0, case["room"]) for s in shared]
    lens = _uniform(r, case["len_lo"], case["len_hi"], case["rows"])
    if op == "free":
        return lens, r.sample(range(case["rows"]), case["freed"])
    pages = sum(-(-n // PAGE) for n in lens)
    live = pages - pages // 10                         # a tenth of the table entries share a page
    return lens, pages, live, min(case["moved"], live, case["blocks"] - live)


def _visible(lq, lk, causal):
    if not causal:
        return lq * lk
    first = lk - lq + 1                                # keys that query 0 sees (>= 1 here)
    return lq * first + lq * (lq - 1) // 2


def work(case):
    op = case["op"]
    if op == "prefill":
        lq, lk = _shapes(case)
        n, tq, tk = case["heads"], sum(lq), sum(lk)
        pairs = sum(_visible(a, b, case["causal"]) for a, b in zip(lq, lk))
        return {"bytes": tq * n * (2 * QD + 2 * V + 4) + tk * (n * 2 * (P + V) + 2 * R) + 8 * (case["batch"] + 1),
                "flops": 2 * n * (QD + V) * pairs}
    if op == "expand":
        lens, _ = _shapes(case)
        t, n = sum(lens), case["heads"]
        return {"bytes": t * D * (1 if case["fp8"] else 2) + n * 2 * LKV * (P + V) + t * (n * 2 * (P + V) + 2 * R),
                "flops": 2 * t * n * LKV * (P + V)}
    if op == "fork":
        lens, parents, shared, room = _shapes(case)
        rows = sum(s % PAGE for s in shared)
        entries = sum(s // PAGE for s in shared) + sum(-(-n // PAGE) for n in room)
        return {"bytes": 2 * case["layers"] * rows * D * (1 if case["fp8"] else 2) + 4 * entries +
                8 * case["blocks"] + 12 * len(parents), "flops": 0}
    if op == "free":
        lens, rows = _shapes(case)
        return {"bytes": 4 * sum(-(-lens[i] // PAGE) for i in rows) + 8 * case["blocks"] + 8 * len(rows) + 4,
                "flops": 0}
    lens, pages, live, moved = _shapes(case)
    return {"bytes": 2 * case["layers"] * moved * PAGE * D * (1 if case["fp8"] else 2) + 8 * pages +
            12 * case["blocks"] + 4 * len(lens) + 4, "flops": 0}


# ----------------------------------------------------------------------------------------------- inputs

def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _int32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def _starts(lens):
    return _int32(np.concatenate([[0], np.cumsum(lens)]))


def _e4m3(shape, gen):
    return (torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=gen) * 64).clamp(
        -448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(case, gen):
    shape = (case["layers"], case["blocks"], PAGE, D)
    if case["fp8"]:
        return torch.randint(0, 127, shape, dtype=torch.uint8, device="cuda", generator=gen)
    return _normal(shape, gen)


def _table(lens, ids, width=None):
    """The rows' page ids in a [rows, width] table; entries past a row's pages are -1."""
    pages = [-(-n // PAGE) for n in lens]
    table = np.full((len(lens), width or max(1, max(pages))), -1, dtype=np.int32)
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
    if op == "prefill":
        lq, lk = _shapes(case)
        n = case["heads"]
        gain = torch.rand((1, n, 1), device="cuda", generator=gen) * 3 + 0.5     # flat and peaked heads
        s["q"] = (_normal((sum(lq), n, QD), gen, torch.float32) * gain).to(torch.bfloat16)
        s["kv"] = _normal((sum(lk), n, P + V), gen)
        s["k_pe"] = _normal((sum(lk), R), gen)
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _starts(lq), _starts(lk), max(lq), max(lk)
    elif op == "expand":
        lens, first = _shapes(case)
        held = [a + b for a, b in zip(lens, first)]
        pages = sum(-(-n // PAGE) for n in held)
        blocks = pages + 3
        s["table"] = _int32(_table(held, rs.permutation(blocks)[:pages]))
        s["cache"] = (_e4m3 if case["fp8"] else _normal)((blocks, PAGE, D), gen)
        s["k_scale"] = 1.0 / 64
        n = case["heads"]
        s["w_uk_t"] = (_normal((n, P, LKV), gen, torch.float32) * LKV ** -0.5).to(torch.bfloat16)
        s["w_uv"] = (_normal((n, LKV, V), gen, torch.float32) * LKV ** -0.5).to(torch.bfloat16)
        s["first"], s["cu_k"], s["total_k"] = _int32(first), _starts(lens), sum(lens)
    elif op == "fork":
        lens, parents, shared, room = _shapes(case)
        pages = [-(-n // PAGE) for n in lens]
        ids = rs.permutation(case["blocks"])[:sum(pages)]
        width = max(max(pages), max(-(-n // PAGE) for n in room), 1)
        refs = np.zeros(case["blocks"], dtype=np.int32)
        refs[ids] = 1
        s["cache"], s["refs"], s["table"] = _cache(case, gen), _int32(refs), _int32(_table(lens, ids, width))
        s["parents"], s["shared"], s["room"] = _int32(parents), _int32(shared), _int32(room)
        s["child_table"] = torch.full((len(parents), width), -1, dtype=torch.int32, device="cuda")
    elif op == "free":
        lens, rows = _shapes(case)
        entries = sum(-(-n // PAGE) for n in lens)
        ids = rs.permutation(case["blocks"])[:entries]
        ids[rs.rand(entries) < 0.1] = rs.randint(0, case["blocks"])          # one page that many rows share
        refs = np.bincount(ids, minlength=case["blocks"]).astype(np.int32)
        s["refs"], s["table"], s["lens"], s["rows"] = _int32(refs), _int32(_table(lens, ids)), _int32(lens), _int32(rows)
    else:
        lens, pages, live, moved = _shapes(case)
        ids = np.concatenate([rs.permutation(live)[:live - moved],
                              live + rs.permutation(case["blocks"] - live)[:moved]])
        rs.shuffle(ids)
        entries = np.concatenate([ids, ids[rs.randint(0, max(1, live), pages - live)]])
        rs.shuffle(entries)
        s["cache"] = _cache(case, gen)
        s["refs"] = _int32(np.bincount(entries, minlength=case["blocks"]))
        s["table"], s["lens"] = _int32(_table(lens, entries)), _int32(lens)
        s["table_out"] = s["table"].clone()
    if "refs" in s:
        s["refs_out"] = torch.empty_like(s["refs"])
    if own:
        from mla_latent_cache_paged_gb300 import binding as mla
        if op == "prefill":
            s["plan"] = mla.make_prefill_plan(case["batch"], case["heads"], s["q"].shape[0], s["max_q"], s["max_k"])
            s["ws"] = mla.new_workspace(s["plan"])
        elif op == "expand":
            s["ws"] = mla.new_status_workspace()
        else:
            s["ws"] = mla.new_cache_workspace(case["blocks"], case.get("children", 0))
    return s


# ------------------------------------------------------------------------------------------- plain forms

def _padded(lens_cu, width):
    """[B, width] row numbers of a packed tensor and which of them exist."""
    i = torch.arange(width, device="cuda")
    lens = (lens_cu[1:] - lens_cu[:-1]).long()
    there = i < lens[:, None]
    return torch.where(there, lens_cu[:-1, None].long() + i, 0), there, lens


def _plain_prefill(s):
    at_q, q_there, lq = _padded(s["cu_q"], s["max_q"])
    at_k, k_there, lk = _padded(s["cu_k"], s["max_k"])
    q = s["q"][at_q].float().transpose(1, 2)                                  # [B, N, Lq, 192]
    kv, pe = s["kv"][at_k].float(), s["k_pe"][at_k].float()
    n = kv.shape[2]
    k = torch.cat([kv[..., :P], pe[:, :, None, :].expand(-1, -1, n, -1)], -1).permute(0, 2, 3, 1)
    scores = torch.matmul(q, k)
    scores *= SCALE
    j = torch.arange(s["max_k"], device="cuda")
    i = torch.arange(s["max_q"], device="cuda")
    seen = k_there[:, None, :]
    if s["case"]["causal"]:
        seen = seen & (j <= (lk - lq)[:, None, None] + i[:, None])
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores -= top
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores, kv[..., P:].transpose(1, 2)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top)[..., 0]
    return {"out": out.transpose(1, 2)[q_there].to(torch.bfloat16), "lse": lse.transpose(1, 2)[q_there]}


def _plain_rows(s):
    """The latent rows of the packed tokens, fp32 [T, 576]."""
    t = torch.arange(s["total_k"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu_k"][1:], t, right=True)
    pos = (t - s["cu_k"][b] + s["first"][b]).long()
    rows = s["cache"][s["table"][b, pos // PAGE].long(), pos % PAGE]
    if s["case"]["fp8"]:
        return rows.view(torch.float8_e4m3fn).float() * s["k_scale"]
    return rows.float()


def _plain_expand(s):
    rows = _plain_rows(s)
    t, n = rows.shape[0], s["w_uv"].shape[0]
    c = rows[:, :LKV]
    k = c @ s["w_uk_t"].float().reshape(n * P, LKV).t()
    v = c @ s["w_uv"].float().permute(1, 0, 2).reshape(LKV, n * V)
    kv = torch.cat([k.view(t, n, P), v.view(t, n, V)], -1).to(torch.bfloat16)
    return {"kv": kv, "k_pe": rows[:, LKV:].to(torch.bfloat16)}


def _plain_fork(s):
    refs, table, out = s["refs"], s["table"], s["child_table"]
    shared, room = s["shared"].long(), s["room"].long()
    full, pages = shared // PAGE, (room + PAGE - 1) // PAGE
    need = pages - full
    before = torch.cumsum(need, 0) - need
    free = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)     # free pages, ascending, first
    j = torch.arange(table.shape[1], device="cuda")
    is_shared, is_fresh = j < full[:, None], (j >= full[:, None]) & (j < pages[:, None])
    parent = table[s["parents"].long()]
    fresh = free[torch.where(is_fresh, before[:, None] + j - full[:, None], 0)]
    out.copy_(torch.where(is_shared, parent, torch.where(is_fresh, fresh, out)))
    held = out[is_shared | is_fresh].long()
    refs_out = refs.clone().index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    row = torch.arange(PAGE, device="cuda")
    copied = row < (shared % PAGE)[:, None]
    last = full.clamp(max=table.shape[1] - 1)[:, None]
    src = (parent.gather(1, last).long() * PAGE + row)[copied]
    dst = (out.gather(1, last).long() * PAGE + row)[copied]
    flat = s["cache"].view(s["cache"].shape[0], -1, D)
    flat[:, dst] = flat[:, src]
    return {"child_table": out, "refs": refs_out, "cache": s["cache"]}


def _plain_free(s):
    rows, refs = s["rows"].long(), s["refs"]
    table, pages = s["table"][rows].long(), (s["lens"][rows] + PAGE - 1) // PAGE
    held = table[torch.arange(table.shape[1], device="cuda") < pages[:, None]]
    refs_out = refs.clone().index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    return {"refs": refs_out, "freed": ((refs > 0) & (refs_out == 0)).sum(dtype=torch.int32).view(1)}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    ids = torch.arange(refs.shape[0], device="cuda", dtype=torch.int32)
    live = refs > 0
    count = live.sum(dtype=torch.int32)
    src, dst = ids[live & (ids >= count)], ids[~live & (ids < count)]
    page_map = torch.where(live, ids, -1)
    page_map[src.long()] = dst
    refs_out = refs.clone()
    refs_out[dst.long()] = refs[src.long()]
    refs_out[src.long()] = 0
    held = torch.arange(table.shape[1], device="cuda") < ((s["lens"] + PAGE - 1) // PAGE)[:, None]
    s["table_out"].copy_(torch.where(held, page_map[table.clamp(min=0).long()], s["table_out"]))
    s["cache"][:, dst.long()] = s["cache"][:, src.long()]
    return {"table": s["table_out"], "refs": refs_out, "page_map": page_map, "live": count.view(1), "cache": s["cache"]}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"prefill": _plain_prefill, "expand": _plain_expand, "fork": _plain_fork, "free": _plain_free,
                "compact": _plain_compact}[op](s)
    from mla_latent_cache_paged_gb300 import binding as mla
    if op == "prefill":
        out, lse = mla.mla_prefill(s["q"], s["kv"], s["k_pe"], s["cu_q"], s["cu_k"], SCALE, causal=case["causal"],
                                   plan=s["plan"], workspace=s["ws"])
        return {"out": out, "lse": lse}
    if op == "expand":
        if case["fp8"]:
            kv, k_pe = mla.mla_expand_kv_fp8(s["cache"], s["table"], s["cu_k"], s["w_uk_t"], s["w_uv"], s["k_scale"],
                                             total_k=s["total_k"], first_token=s["first"], workspace=s["ws"])
        else:
            kv, k_pe = mla.mla_expand_kv(s["cache"], s["table"], s["cu_k"], s["w_uk_t"], s["w_uv"],
                                         total_k=s["total_k"], first_token=s["first"], workspace=s["ws"])
        return {"kv": kv, "k_pe": k_pe}
    if op == "fork":
        table, refs = mla.mla_cache_fork(s["cache"], s["refs"], s["table"], s["parents"], s["shared"], s["room"],
                                         child_table=s["child_table"], ref_counts_out=s["refs_out"], workspace=s["ws"])
        return {"child_table": table, "refs": refs, "cache": s["cache"]}
    if op == "free":
        refs, freed = mla.mla_cache_free(s["refs"], s["table"], s["lens"], s["rows"], ref_counts_out=s["refs_out"],
                                         workspace=s["ws"])
        return {"refs": refs, "freed": freed}
    table, refs, page_map, live = mla.mla_cache_compact(s["cache"], s["refs"], s["table"], s["lens"],
                                                        block_table_out=s["table_out"], ref_counts_out=s["refs_out"],
                                                        workspace=s["ws"])
    return {"table": table, "refs": refs, "page_map": page_map, "live": live, "cache": s["cache"]}


# ---------------------------------------------------------------------------------------- from definitions

def exact(case, seed):
    """What ``run`` returns, in 64 bits, one sequence and a few heads at a time."""
    if case["op"] == "prefill":
        s = prepare(case, seed)
        lq, lk = _shapes(case)
        n = case["heads"]
        out = torch.zeros((sum(lq), n, V), dtype=torch.float64, device="cuda")
        lse = torch.full((sum(lq), n), -math.inf, dtype=torch.float64, device="cuda")
        a = c = 0
        for m, l in zip(lq, lk):
            step = max(1, int(2e8 / (m * l)))
            pe = s["k_pe"][c:c + l].double()
            hidden = torch.arange(l, device="cuda") > torch.arange(m, device="cuda")[:, None] + (l - m)
            for h in range(0, n, step):
                q = s["q"][a:a + m, h:h + step].double().transpose(0, 1)
                kv = s["kv"][c:c + l, h:h + step].double().transpose(0, 1)
                x = (q[..., :P] @ kv[..., :P].transpose(1, 2) + q[..., P:] @ pe.t()) * SCALE
                if case["causal"]:
                    x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                out[a:a + m, h:h + step] = (torch.exp(x - z[..., None]) @ kv[..., P:]).transpose(0, 1)
                lse[a:a + m, h:h + step] = z.t()
                del x
            a, c = a + m, c + l
        return {"out": out, "lse": lse}
    if case["op"] == "expand":
        s = prepare(case, seed)
        lens, first = _shapes(case)
        n = case["heads"]
        cache = s["cache"].view(torch.float8_e4m3fn).double() / 64 if case["fp8"] else s["cache"].double()
        flat = cache.view(-1, D)
        rows = torch.cat([flat[(s["table"][b].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).view(-1)
                               [f:f + l]] for b, (l, f) in enumerate(zip(lens, first))])
        kv = torch.empty((rows.shape[0], n, P + V), dtype=torch.float64, device="cuda")
        for h in range(n):
            kv[:, h, :P] = rows[:, :LKV] @ s["w_uk_t"][h].double().t()
            kv[:, h, P:] = rows[:, :LKV] @ s["w_uv"][h].double()
        return {"kv": kv, "k_pe": rows[:, LKV:]}
    return None

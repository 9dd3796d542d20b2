"""The cache's row calls and the decodes over shared prefixes and windows as a
server runs them: a prompt is written, requests fork from it, and each step
writes the new tokens' entries and attends to them, eagerly and as a graph."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64, bf16_tensor_bits, f32_to_bf16_bits
from oracle import cache_write, e4m3_codes, e4m3_to_float, gather_rows
from span_util import K_SCALE, NAN, SCALE, check, dev, ints, random_q, reference

pytestmark = pytest.mark.gpu

BLOCKS, PAGES, CHILDREN, HEADS = 40, 6, 5, 16     # a batch row more than requests: padding


def _entries(rng, n):
    return f32_to_bf16_bits(rng.standard_normal((n, 576)).astype(np.float32))


class _Server:
    def __init__(self, fp8):
        import torch
        self.fp8 = fp8
        self.host = np.full((BLOCKS, 64, 576), NAN[fp8], np.uint8 if fp8 else np.uint16)
        self.cache = dev(self.host)
        self.ws = binding.new_status_workspace()
        B = CHILDREN + 1
        self.plan = binding.make_span_plan(B, HEADS, PAGES, max_groups=2)
        self.span_ws = binding.new_workspace(self.plan)
        self.new = torch.zeros((B, 640), dtype=torch.bfloat16, device="cuda")[:, :576]
        self.slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
        self.q = torch.zeros((B, HEADS, 576), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((B, PAGES), -1, dtype=torch.int32, device="cuda")
        self.lens, self.starts, self.shared = ints([0] * B), ints([0, 0, 0]), ints([0, 0])
        self.out = [torch.zeros((B, HEADS, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.lse = [torch.zeros((B, HEADS), dtype=torch.float32, device="cuda") for _ in range(2)]
        self.cu = ints([0] * (B + 1))
        self.rows = torch.zeros((B * PAGES * 64, 576), dtype=torch.bfloat16, device="cuda")

    def write(self, rows, slots):
        if self.fp8:
            binding.mla_cache_write_fp8(rows[:, :512], rows[:, 512:], slots, self.cache, K_SCALE,
                                        workspace=self.ws)
        else:
            binding.mla_cache_write(rows[:, :512], rows[:, 512:], slots, self.cache, workspace=self.ws)

    def host_write(self, rows, slots):
        codes = e4m3_codes(bf16_bits_to_f64(rows), K_SCALE) if self.fp8 else rows
        self.host = cache_write(self.host, codes[:, :512], codes[:, 512:], slots)

    def step(self, window, sinks):
        """Everything a decode step and a later chunk's read of the cache launch."""
        self.write(self.new, self.slots)
        scale = (SCALE, K_SCALE) if self.fp8 else (SCALE,)
        tail = "_fp8" if self.fp8 else ""
        args = (self.q, self.cache, self.table, self.lens)
        getattr(binding, "mla_decode_shared" + tail)(
            *args, self.starts, self.shared, *scale, plan=self.plan, workspace=self.span_ws,
            out=self.out[0], lse=self.lse[0])
        getattr(binding, "mla_decode_window" + tail)(
            *args, *scale, window=window, sinks=sinks, plan=self.plan, workspace=self.span_ws,
            out=self.out[1], lse=self.lse[1])
        getattr(binding, "mla_cache_gather" + tail)(
            self.cache, self.table, self.cu, *scale[1:], total_k=self.rows.shape[0], rows=self.rows,
            workspace=self.ws)


@pytest.mark.parametrize("fp8", [False, True])
def test_forked_requests_step_by_step(fp8):
    import torch
    rng = np.random.default_rng(77)
    s = _Server(fp8)
    window, sinks, prompt_len, shared = 70, 5, 200, 192
    # the prompt of one request, on pages in no order
    pages = rng.permutation(BLOCKS)[:4]
    prompt = _entries(rng, prompt_len)
    where = [int(pages[t // 64]) * 64 + t % 64 for t in range(prompt_len)]
    s.write(dev(prompt), torch.tensor(where, device="cuda"))
    s.host_write(prompt, where)
    # requests that go on from it: they share its whole pages
    counts = np.zeros(BLOCKS, np.int32)
    counts[pages] = 1
    parent = np.full((1, PAGES), -1, np.int32)
    parent[0, :4] = pages
    table, _ = binding.mla_cache_fork(
        s.cache, ints(counts), ints(parent), ints([0] * CHILDREN), ints([prompt_len] * CHILDREN),
        ints([prompt_len + 130] * CHILDREN), workspace=binding.new_cache_workspace(BLOCKS, CHILDREN))
    torch.cuda.synchronize()
    host_table = table.cpu().numpy()
    assert (host_table[:, :3] == pages[:3]).all()
    for c in range(CHILDREN):
        s.host[host_table[c, 3]] = s.host[pages[3]]
    s.table[:CHILDREN] = table
    s.starts.copy_(ints([0, 3, 5])), s.shared.copy_(ints([shared, shared]))
    lens = np.array([prompt_len] * CHILDREN + [0])
    full = np.concatenate([host_table, np.full((1, PAGES), -1, np.int32)])
    graph, side = None, torch.cuda.Stream()
    # (the fourth child stops after the first step: a padded row from then on)
    for turn in range(3):
        for _ in range(61 if turn == 1 else 1):       # a page's end is passed in between
            live = np.array([b for b in range(CHILDREN) if turn == 0 or b != 3])
            row = _entries(rng, CHILDREN + 1)
            at = np.full(CHILDREN + 1, -1, np.int64)
            at[live] = [int(full[b, lens[b] // 64]) * 64 + lens[b] % 64 for b in live]
            lens[live] += 1
            if turn > 0:
                lens[3] = 0
            query = random_q(rng, CHILDREN + 1, HEADS)
            cu = np.concatenate([[0], np.cumsum(lens)])
            s.new.copy_(dev(row)), s.slots.copy_(torch.from_numpy(at)), s.q.copy_(dev(query))
            s.lens.copy_(ints(lens)), s.cu.copy_(ints(cu))
            s.host_write(row, at)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                s.step(window, sinks)
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        eager = [t.clone() for t in (*s.out, *s.lse, s.cache, s.rows)]
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.step(window, sinks)
        for t in (*s.out, *s.lse, s.rows):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert binding.read_error(s.ws) == 0 and binding.read_error(s.span_ws) == 0
        for a, b in zip(eager, (*s.out, *s.lse, s.cache, s.rows)):
            # (rows that no request has are zeros or an older step's)
            n = int(cu[-1]) if a is eager[-1] else a.shape[0]
            assert torch.equal(a[:n].view(torch.uint8), b[:n].view(torch.uint8))
        host = s.cache.cpu().numpy() if fp8 else bf16_tensor_bits(s.cache)
        for b, n in enumerate(lens):
            at = np.arange(n)
            assert np.array_equal(host[full[b, at // 64], at % 64], s.host[full[b, at // 64], at % 64])
        seen = [np.arange(n) for n in lens]
        check(s.out[0], s.lse[0], reference(query, s.host, full, seen, SCALE), ("shared", turn))
        part = [t[(t < sinks) | (t >= n - window)] for t, n in zip(seen, lens)]
        check(s.out[1], s.lse[1], reference(query, s.host, full, part, SCALE), ("window", turn))
        want = gather_rows(s.host, full, [0] * len(lens), lens)
        if fp8:
            want = f32_to_bf16_bits((e4m3_to_float(want).astype(np.float32) * np.float32(K_SCALE)))
        got = bf16_tensor_bits(s.rows)
        assert np.array_equal(got[:cu[-1]], want[:cu[-1]])
        assert not got[cu[-1]:].any()      # rows behind the last request are left as they were


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_behind_one_another_without_a_wait(fp8):
    """Each call's queries and lengths are written by kernels right in front of
    it, its results read by one right behind it, all over the same tensors."""
    import torch
    rng = np.random.default_rng(5)
    B, N, M, turns = 6, 16, 9, 24
    host = f32_to_bf16_bits(rng.standard_normal((B * M, 64, 576)).astype(np.float32))
    if fp8:
        host = e4m3_codes(bf16_bits_to_f64(host), K_SCALE)
    cache, table = dev(host), rng.permutation(B * M).reshape(B, M).astype(np.int32)
    table[1:3, :4] = table[0, :4]                       # 256 tokens together
    queries = [random_q(rng, B, N) for _ in range(turns)]
    lens = [np.concatenate([rng.integers(256, 576, 3), rng.integers(0, 576, 3)]) for _ in range(turns)]
    d_q, d_l = torch.stack([dev(q) for q in queries]), torch.stack([ints(n) for n in lens])
    plan = binding.make_span_plan(B, N, M, max_groups=1, num_sms=4)
    ws = binding.new_workspace(plan)
    q, length = d_q[0].clone(), d_l[0].clone()
    out = torch.empty((B, N, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, N), dtype=torch.float32, device="cuda")
    got = torch.empty((2, turns, B, N, 512), dtype=torch.bfloat16, device="cuda")
    got_lse = torch.empty((2, turns, B, N), dtype=torch.float32, device="cuda")
    starts, shared, d_table = ints([0, 3]), ints([256]), ints(table)
    scale, tail = ((SCALE, K_SCALE), "_fp8") if fp8 else ((SCALE,), "")
    load = torch.ones((2048, 2048), device="cuda")
    kw = dict(plan=plan, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    for i in range(turns):
        (load @ load)                                   # the kernels behind it queue up
        q.copy_(d_q[i]), length.copy_(d_l[i])
        getattr(binding, "mla_decode_shared" + tail)(q, cache, d_table, length, starts, shared, *scale, **kw)
        got[0, i].copy_(out), got_lse[0, i].copy_(lse)
        getattr(binding, "mla_decode_window" + tail)(q, cache, d_table, length, *scale, window=130, sinks=3, **kw)
        got[1, i].copy_(out), got_lse[1, i].copy_(lse)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0
    for i in range(turns):
        seen = [np.arange(n) for n in lens[i]]
        part = [t[(t < 3) | (t >= n - 130)] for t, n in zip(seen, lens[i])]
        for k, s in enumerate((seen, part)):
            check(got[k, i], got_lse[k, i], reference(queries[i], host, table, s, SCALE), (k, i))

"""The span decodes in the order of a real step: right behind the front end
(which lets the kernel behind it start before it has written the queries and
the cache), right behind the plain decode, and the up-projection right behind
them; as single calls, as a chain, and as a replayed graph, bit for bit."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding
from mla_latent_cache_paged_gb300.workloads import bf16_tensor_bits, f32_to_bf16_bits
from oracle import cache_write, e4m3_codes
from mla_latent_cache_paged_gb300.workloads import bf16_bits_to_f64
from span_sharing import assert_shared
from span_util import K_SCALE, SCALE, check, dev, ints, reference

pytestmark = pytest.mark.gpu

B, N, M, TURNS, SMS, WINDOW, SINKS = 6, 16, 10, 8, 4, 130, 3
STARTS, SHARED = [0, 4], [320]


def _bits(rng, shape, gain=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * gain).astype(np.float32))


class _Step:
    """Tensors that each turn's step reads and writes, and the step."""

    def __init__(self, rng, fp8):
        import torch
        self.fp8, bf16 = fp8, torch.bfloat16
        self.host = _bits(rng, (B * M, 64, 576))
        if fp8:
            self.host = e4m3_codes(bf16_bits_to_f64(self.host), K_SCALE)
        self.rows = rng.permutation(B * M).reshape(B, M)
        self.rows[1:4, :5] = self.rows[0, :5]
        self.table = ints(self.rows)
        self.w_uk, self.w_uv = dev(_bits(rng, (N, 128, 512), 0.09)), dev(_bits(rng, (N, 512, 128), 0.05))
        self.ws = binding.new_status_workspace()
        self.plan = binding.make_span_plan(B, N, M, max_groups=1, num_sms=SMS)
        self.span_ws = binding.new_workspace(self.plan)
        self.plain_plan = binding.make_plan(B, N, M)
        self.plain_ws = binding.new_workspace(self.plain_plan)
        self.starts, self.shared = ints(STARTS), ints(SHARED)
        # what a turn brings
        self.q = torch.zeros((B, N, 192), dtype=bf16, device="cuda")
        self.new = [torch.zeros((B, n), dtype=bf16, device="cuda") for n in (512, 64)]
        self.slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
        self.lens = ints([0] * B)
        # what it leaves
        self.mqa_q = torch.zeros((B, N, 576), dtype=bf16, device="cuda")
        self.out = [torch.zeros((B, N, 512), dtype=bf16, device="cuda") for _ in range(3)]
        self.lse = [torch.zeros((B, N), dtype=torch.float32, device="cuda") for _ in range(3)]
        self.up = [torch.zeros((B, N, 128), dtype=bf16, device="cuda") for _ in range(2)]
        self.cache = dev(self.host)

    def results(self):
        return [self.mqa_q, *self.out, *self.lse, *self.up]

    def calls(self, order):
        ks, tail = ((K_SCALE,), "_fp8") if self.fp8 else ((), "")
        args = (self.cache, self.table, self.lens)

        def front():
            if self.fp8:
                binding.mla_cache_write_fp8(*self.new, self.slots, self.cache, K_SCALE, workspace=self.ws)
                binding.mla_q_absorb_concat_cache(self.q, self.w_uk, workspace=self.ws, out=self.mqa_q)
            else:
                binding.mla_q_absorb_concat_cache(self.q, self.w_uk, *self.new, self.slots, self.cache,
                                                  workspace=self.ws, out=self.mqa_q)

        def decode(k):
            kw = dict(out=self.out[k], lse=self.lse[k])
            if k == 2:
                getattr(binding, "mla_decode" + tail)(self.mqa_q, *args, SCALE, *ks, plan=self.plain_plan,
                                                      workspace=self.plain_ws, **kw)
            elif k == 1:
                getattr(binding, "mla_decode_window" + tail)(
                    self.mqa_q, *args, SCALE, *ks, window=WINDOW, sinks=SINKS, plan=self.plan,
                    workspace=self.span_ws, **kw)
            else:
                getattr(binding, "mla_decode_shared" + tail)(
                    self.mqa_q, *args, self.starts, self.shared, SCALE, *ks, plan=self.plan,
                    workspace=self.span_ws, **kw)

        def up(k):
            binding.mla_v_up_proj(self.out[k], self.w_uv, workspace=self.ws, out=self.up[k])

        first, last = order
        return [front, lambda: decode(first), lambda: up(first), lambda: decode(2), lambda: decode(last),
                lambda: up(last)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_a_step_as_it_runs(order, fp8):
    import torch
    rng = np.random.default_rng(90 + order[0])
    s = _Step(rng, fp8)
    turns, lens = [], np.array([330, 325, 460, 384, 1, 200])
    for _ in range(TURNS):
        slots = np.array([s.rows[b, lens[b] // 64] * 64 + lens[b] % 64 for b in range(B)], np.int64)
        lens = lens + 1
        turns.append((_bits(rng, (B, N, 192)), _bits(rng, (B, 512)), _bits(rng, (B, 64)), slots, lens))
    given = [(dev(q), dev(kv), dev(pe), torch.from_numpy(at).cuda(), ints(n)) for q, kv, pe, at, n in turns]
    held = (s.q, *s.new, s.slots, s.lens)
    calls = s.calls(order)
    load = torch.ones((3000, 3000), device="cuda")
    start = dev(s.host)

    def run(step):
        s.cache.copy_(start)
        kept = [torch.zeros((TURNS, *t.shape), dtype=t.dtype, device="cuda") for t in s.results()]
        torch.cuda.synchronize()
        for i in range(TURNS):
            (load @ load)                              # what is behind it queues up
            for t, v in zip(held, given[i]):
                t.copy_(v)
            step()
            for t, v in zip(kept, s.results()):
                t[i].copy_(v)
        torch.cuda.synchronize()
        assert binding.read_error(s.ws) == 0 and binding.read_error(s.span_ws) == 0
        return kept + [s.cache.clone()]

    def one_by_one():
        for call in calls:
            torch.cuda.synchronize()
            call()

    def chain():
        for call in calls:
            call()

    alone = run(one_by_one)
    eager = run(chain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    replayed = run(graph.replay)
    for a, b, c in zip(alone, eager, replayed):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    if order == (1, 0):                                # (the shared decode was the last on the workspace)
        assert_shared(s.span_ws, turns[-1][4], STARTS, SHARED, N, SMS)
    host = s.host
    for i, (_, kv, pe, at, n) in enumerate(turns):
        new = [e4m3_codes(bf16_bits_to_f64(x), K_SCALE) if fp8 else x for x in (kv, pe)]
        host = cache_write(host, *new, at)
        query = bf16_tensor_bits(alone[0][i])
        seen = [np.arange(k) for k in n]
        part = [t[(t < SINKS) | (t >= k - WINDOW)] for t, k in zip(seen, n)]
        for k, tokens in enumerate((seen, part)):
            check(alone[1 + k][i], alone[4 + k][i], reference(query, host, s.rows, tokens, SCALE), (i, k))
    bits = alone[-1].cpu().numpy() if fp8 else bf16_tensor_bits(alone[-1])
    assert np.array_equal(bits, host)

"""Plans that split only the last wave's items: the workspace they ask for is
all that they write, and the flag may be set or cleared on a plan."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _args(q_lens, k_lens, heads, seed=5):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)

    def starts(lens):
        return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()

    return (normal(sum(q_lens), heads, 192), normal(sum(k_lens), heads, 256),
            normal(sum(k_lens), 64), starts(q_lens), starts(k_lens), SCALE)


def _exact(args, q_lens, k_lens, causal):
    """(out, lse, sum of weights times |v|) in 64 bits."""
    import torch
    q, kv, pe = (x.double() for x in args[:3])
    outs, lses, sizes = [], [], []
    a = c = 0
    for m, n in zip(q_lens, k_lens):
        x, k = q[a:a + m].transpose(0, 1), kv[c:c + n].transpose(0, 1)
        s = (x[..., :128] @ k[..., :128].transpose(1, 2) + x[..., 128:] @ pe[c:c + n].t()) * SCALE
        if causal:
            j, i = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")
            s = s.masked_fill(j > i[:, None] + (n - m), -torch.inf)
        z = torch.logsumexp(s, -1)
        w = torch.where(torch.isneginf(z)[..., None], 0.0, torch.exp(s - z[..., None]))
        outs.append((w @ k[..., 128:]).transpose(0, 1))
        sizes.append((w @ k[..., 128:].abs()).transpose(0, 1))
        lses.append(z.t())
        a, c = a + m, c + n
    return torch.cat(outs), torch.cat(lses), torch.cat(sizes)


def _check(got, args, q_lens, k_lens, causal):
    """Scores: 192 products summed in fp32, off by d = 192 * 2^-23 * SCALE * |q| |k|
    <= 2e-3 at norms of up to 34 (unit normals: 14); a weight by 2 d + 2^-20 and
    its rounding to bf16 (2^-8), the result by 2^-8 of itself."""
    import torch
    out, lse = got
    ref, z, size = _exact(args, q_lens, k_lens, causal)
    assert float(args[0].double().norm(dim=-1).max()) * float(
        (args[1][..., :128].double().pow(2).sum(-1) + args[2].double().pow(2).sum(-1)[:, None])
        .sqrt().max()) <= 34 ** 2
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 4e-3 + 2.0 ** -20) * size * (1 + 2.0 ** -7)
    assert bool(((out.double() - ref).abs() <= tol + 1e-30).all())
    none = torch.isneginf(z)
    assert torch.equal(torch.isneginf(lse), none) and not out[none].any()
    assert bool(((lse.double() - z).abs()[~none] <= 2e-3 + 2.0 ** -20 * (1 + z[~none].abs())).all())


def _guarded(plan):
    """A workspace of exactly the plan's size, and the bytes before and behind it."""
    import torch
    n = int(plan.workspace_bytes)
    memory = torch.full((n + 2 * 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = memory[65536:65536 + n]
    assert ws.data_ptr() % 256 == 0
    rc = binding.load_library().mla_workspace_init(
        ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    ws[binding.STATUS_BYTES:] = 0xA5           # what an earlier call left behind
    return ws, (memory[:65536], memory[65536 + n:])


def _unchanged(guards):
    return all(bool((g == 0x5A).all()) for g in guards)


CASES = [
    # q lengths, k lengths, heads, SMs of the plan
    ([512], [2300], 3, 5),                              # 6 items, 1 left over
    ([300, 0, 129, 70, 5], [2500, 9, 2200, 2049, 2], 2, 5),   # 12, 2
    ([255], [2050], 31, 25),                            # 31, 6
    ([700], [500], 4, 9),                               # rows that see nothing; 12, 3
    ([1300, 40], [2100, 2100], 5, 14),                  # 35, 7
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_the_planned_workspace_is_all_that_is_written(case, causal):
    import torch
    q_lens, k_lens, heads, sms = CASES[case]
    args = _args(q_lens, k_lens, heads)
    plan = binding.make_prefill_plan(len(q_lens), heads, sum(q_lens), max(q_lens), 2300,
                                     num_sms=sms)
    assert plan.split_rest == 1 and plan.num_kv_splits > 1
    ws, guards = _guarded(plan)
    for _ in range(2):
        got = binding.mla_prefill(*args, causal=causal, plan=plan, workspace=ws)
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0 and _unchanged(guards)
    _check(got, args, q_lens, k_lens, causal)


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("splits", [2, 5, 64])
def test_the_flag_set_on_a_plan_that_splits_all(case, splits):
    import torch
    q_lens, k_lens, heads, sms = CASES[case]
    args = _args(q_lens, k_lens, heads)
    plan = binding.make_prefill_plan(len(q_lens), heads, sum(q_lens), max(q_lens), 2300,
                                     num_sms=sms, num_kv_splits=splits)
    ws, guards = _guarded(plan)
    for rest in (0, 1, 0):                     # the calls of one workspace, in turn
        plan.split_rest = rest
        got = binding.mla_prefill(*args, plan=plan, workspace=ws)
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0 and _unchanged(guards)
        _check(got, args, q_lens, k_lens, True)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_the_flag_cleared_on_a_plan_made_with_it(case):
    """No keys are cut then: bit for bit the results of a plan without splits."""
    import torch
    q_lens, k_lens, heads, sms = CASES[case]
    args = _args(q_lens, k_lens, heads)
    sizes = (len(q_lens), heads, sum(q_lens), max(q_lens), 2300)
    plan = binding.make_prefill_plan(*sizes, num_sms=sms)
    plan.split_rest = 0
    ws, guards = _guarded(plan)
    got = binding.mla_prefill(*args, plan=plan, workspace=ws)
    whole = binding.make_prefill_plan(*sizes, num_sms=sms, num_kv_splits=1)
    want = binding.mla_prefill(*args, plan=whole, workspace=binding.new_workspace(whole))
    torch.cuda.synchronize()
    assert binding.read_error(ws) == 0 and _unchanged(guards)
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(got[1], want[1])


def test_calls_of_different_batches_share_a_workspace():
    """Captured one after the other on one workspace and replayed: each merge
    reads what its own call left."""
    import torch
    plans, graphs, outs, wants = [], [], [], []
    problems = [_args(*CASES[i][:3], seed=i) for i in (0, 1, 4)]
    for args, i in zip(problems, (0, 1, 4)):
        q_lens, _, heads, sms = CASES[i]
        plans.append(binding.make_prefill_plan(len(q_lens), heads, sum(q_lens), max(q_lens), 2300,
                                               num_sms=sms))
        assert plans[-1].split_rest == 1
        wants.append(binding.mla_prefill(*args, plan=plans[-1],
                                         workspace=binding.new_workspace(plans[-1])))
        outs.append((torch.zeros_like(wants[-1][0]), torch.zeros_like(wants[-1][1])))
    ws = binding.new_workspace(max(plans, key=lambda p: p.workspace_bytes))
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for args, plan, (out, lse) in zip(problems, plans, outs):
            binding.mla_prefill(*args, plan=plan, workspace=ws, out=out, lse=lse, stream=stream)
    for _ in range(3):
        for out, lse in outs:
            out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert binding.read_error(ws) == 0
        for (out, lse), want in zip(outs, wants):
            assert torch.equal(out.view(torch.int16), want[0].view(torch.int16))
            assert torch.equal(lse, want[1])

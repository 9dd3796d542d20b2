"""When mla_decode_shared reads a prefix for a group together, restated from the
rule that the header and the kernel's schedule state: as whole pages, as far as
the shortest member with tokens reaches, for groups where tiles of 128 rows
save steps of two pages (an item costs two steps), and only if all groups
together save two steps for every CTA pair."""

import numpy as np

from mla_latent_cache_paged_gb300 import binding


def pairs_of(num_sms):
    return min(256, max(1, num_sms // 2))


def saved_steps(lens, starts, shared, heads):
    """The steps that each group's tiles save (none if not more than 0)."""
    out = []
    for g, want in enumerate(shared):
        there = [int(n) for n in lens[starts[g]:starts[g + 1]] if n > 0]
        pages = min(int(want), min(there, default=0)) // 64
        members = starts[g + 1] - starts[g]
        tiles = -(-members * heads // 128)
        out.append(max(0, (members - tiles) * -(-pages // 2) - 2 * tiles))
    return out


def tile_rows(lens, starts, shared, heads, num_sms=152):
    """Each request's first row in the tiles of its group, or -1."""
    saved = saved_steps(lens, starts, shared, heads)
    rows, tiles = [-1] * len(lens), 0
    if sum(saved) < 2 * pairs_of(num_sms):
        return rows
    for g, s in enumerate(saved):
        if s > 0:
            for k, b in enumerate(range(starts[g], starts[g + 1])):
                if lens[b] > 0:
                    rows[b] = 128 * tiles + k * heads
            tiles += -(-(starts[g + 1] - starts[g]) * heads // 128)
    return rows


def tile_rows_left_in(workspace, batch):
    """The same, as the last call on a workspace left them."""
    import torch
    at = binding.STATUS_BYTES
    return workspace[at:at + 4 * batch].view(torch.int32).cpu().numpy().tolist()


def assert_shared(workspace, lens, starts, shared, heads, num_sms=152):
    want = tile_rows(lens, starts, shared, heads, num_sms)
    assert max(want) >= 0, "the batch is not shared at all"
    assert tile_rows_left_in(workspace, len(lens)) == want


def pool_problem(rng, lens, starts, shared, fp8, blocks=300):
    """Like shared_problem, from a pool of few pages that rows share at random
    (every row holds numbers), for batches of many requests."""
    from span_util import random_cache
    width = max(1, int(-(-np.max(lens) // 64)))
    table = rng.integers(0, blocks, (len(lens), width)).astype(np.int32)
    for g, n in enumerate(shared):
        a, e = starts[g], starts[g + 1]
        if e > a:
            table[a:e, :n // 64] = table[a, :n // 64]
    return random_cache(rng, blocks, fp8), table

"""A workspace whose call was abandoned at a grid barrier: the mark that such a
call leaves in the status header is set here by hand. Later calls stop at their
first barrier until the workspace is initialised again."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu

BARRIER_WORD = 5        # of the status header


def _int(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


class _Pool:
    def __init__(self):
        import torch
        self.cache = torch.arange(9 * 64 * 576, device="cuda").remainder(251).to(
            torch.uint8).view(9, 64, 576)
        self.refs = _int([0, 1, 0, 1, 1, 0, 1, 0, 0])
        self.table = _int([[3, 1], [6, 4]])
        self.child = _int(np.full((2, 2), -1))
        self.freed = _int([0])
        self.tensors = (self.cache, self.refs, self.table, self.child)

    def fork(self, ws):
        binding.mla_cache_fork(self.cache, self.refs, self.table, _int([0, 1]), _int([70, 64]),
                               _int([71, 128]), workspace=ws, child_table=self.child)

    def free(self, ws):
        binding.mla_cache_free(self.refs, self.table, _int([128, 128]), _int([1]), workspace=ws,
                               num_freed=self.freed)

    def compact(self, ws):
        binding.mla_cache_compact(self.cache, self.refs, self.table, _int([128, 128]),
                                  workspace=ws)


@pytest.mark.parametrize("call", ["fork", "free", "compact"])
def test_an_abandoned_workspace_is_refused_until_it_is_initialised(call):
    import torch
    pool = _Pool()
    before = [t.clone() for t in pool.tensors]
    ws = binding.new_cache_workspace(9, 2)
    ws.view(torch.int32)[BARRIER_WORD] = -2 ** 31 + 7
    for _ in range(2):
        getattr(pool, call)(ws)
        assert binding.read_error(ws) == binding.MLA_ERR_TIMEOUT
        assert all(torch.equal(a, b) for a, b in zip(pool.tensors, before))
    rc = binding.load_library().mla_workspace_init(
        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    getattr(pool, call)(ws)
    assert binding.read_error(ws) == 0
    assert int(ws.view(torch.int32)[BARRIER_WORD]) == 0
    refs = pool.refs.tolist()
    if call == "fork":
        assert pool.child.tolist() == [[3, 0], [6, 2]]
        assert refs == [1, 1, 1, 2, 1, 0, 2, 0, 0]
        assert torch.equal(pool.cache[0, :6], before[0][1, :6])
        assert torch.equal(pool.cache[0, 6:], before[0][0, 6:])
    elif call == "free":
        assert refs == [0, 1, 0, 1, 0, 0, 0, 0, 0] and int(pool.freed) == 2
    else:
        assert pool.table.tolist() == [[3, 1], [2, 0]] and refs == [1, 1, 1, 1, 0, 0, 0, 0, 0]
        assert torch.equal(pool.cache[0], before[0][4]) and torch.equal(pool.cache[2], before[0][6])

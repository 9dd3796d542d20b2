"""Results that the prefill-side calls allocate: PyTorch's modes see them, as
they see every other tensor of a program."""

import numpy as np
import pytest

from mla_latent_cache_paged_gb300 import binding

pytestmark = pytest.mark.gpu


def _int(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _zeros(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def _prefill(**kw):
    return binding.mla_prefill(_zeros(7, 2, 192), _zeros(9, 2, 256), _zeros(9, 64), _int([0, 5]),
                               _int([0, 9]), 0.1, **kw)


def _expand(**kw):
    return binding.mla_expand_kv(_zeros(3, 64, 576), _int([[2, 1]]), _int([0, 70]),
                                 _zeros(2, 128, 512), _zeros(2, 512, 128), total_k=80,
                                 workspace=binding.new_status_workspace(), **kw)


def _free(**kw):
    return binding.mla_cache_free(_int([1, 1, 0]), _int([[1, 0]]), _int([65]), _int([0]),
                                  workspace=binding.new_status_workspace(), **kw)[1:]


def _compact(**kw):
    return binding.mla_cache_compact(_zeros(3, 64, 576), _int([0, 1, 1]), _int([[1, 2]]),
                                     _int([65]), workspace=binding.new_cache_workspace(3), **kw)[2:]


CALLS = [_prefill, _expand, _free, _compact]


@pytest.mark.parametrize("on_a_stream", [False, True])
@pytest.mark.parametrize("call", CALLS)
def test_a_dispatch_mode_sees_the_results(call, on_a_stream):
    import torch
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.made = set()

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if isinstance(out, torch.Tensor):
                self.made.add(out.data_ptr())
            return out

    torch.cuda.synchronize()
    with Seen() as seen:
        results = call(stream=torch.cuda.Stream()) if on_a_stream else call()
        assert all(r.data_ptr() in seen.made for r in results)
    torch.cuda.synchronize()


@pytest.mark.parametrize("call,first", [(_prefill, 5), (_expand, 70)])
def test_rows_of_no_sequence_get_the_deterministic_fill(call, first):
    """With deterministic algorithms PyTorch fills new memory with NaN; the rows
    that a call does not write keep it."""
    import torch
    torch.use_deterministic_algorithms(True, warn_only=True)
    try:
        results = call()
    finally:
        torch.use_deterministic_algorithms(False)
    for r in results:
        assert not torch.isnan(r[:first]).any() and torch.isnan(r[first:]).all()

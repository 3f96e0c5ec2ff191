"""The paged cache's Python binding on the host (no GPU): what a cache struct keeps alive."""
import gc
import weakref

import torch

import speculative_decoding_verification_packed_gb300 as svp


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on a GPU: make_cache only checks and reads attributes."""

    @property
    def device(self):
        return torch.device("cuda", 0)


def tensor(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def test_a_dropped_cache_frees_its_pools_at_once():
    """No reference cycle holds the pools until (or past) the next garbage collection, which device
    memory that runs out does not start."""
    k, v = (tensor(4, 2, 16, 64, dtype=torch.float8_e4m3fn) for _ in range(2))
    ke, ve = (tensor(4, 2, 16, dtype=torch.uint8) for _ in range(2))
    table = tensor(1, 4, dtype=torch.int32)
    gc.disable()
    try:
        cache = svp.make_cache(k, v, table, k_exp=ke, v_exp=ve)
        held = [weakref.ref(x) for x in (cache, k, v, ke, ve, table)]
        del k, v, ke, ve, table
        assert all(x() is not None for x in held)     # the struct keeps its tensors
        del cache
        assert all(x() is None for x in held)
    finally:
        gc.enable()

"""8-bit caches without a GPU: tensors of a cache that change between calls, captures on a device that is not the current
one, and the frequencies of positions scaled for long contexts."""

import pytest
import torch

import block_sparse_attention_06_gb300 as m


# ------------------------------------------------------------------------------------------------ caches

SWAPS = [("k", lambda x: torch.zeros(4)), ("k", lambda x: x[:2].clone()), ("v", lambda x: x[:2].clone()),
         ("kidx", lambda x: x[:, :, :, ::2].clone()), ("kidx", lambda x: x.transpose(0, 1)),
         ("v_scale", lambda x: x[:2].clone()), ("k_scale", lambda x: torch.zeros(x.shape)),
         ("kidx_scale", lambda x: x.view(torch.uint8))]


@pytest.mark.parametrize("name,swap", SWAPS)
def test_tensors_of_a_cache_are_looked_at_in_every_call(name, swap):
    """A tensor keeps its place in the cache while its storage changes (a pool made smaller, another type): refused in
    the next call, as by a cache made anew."""
    dims = m.Dims(16, 4, 128, 64, 4, 3)
    c = m.CacheQ8.zeros(dims, 8, "cpu")
    dev = c.k.get_device()               # of a tensor on the host: stands for any device here
    for _ in range(2):
        assert c._struct(dims, dev, True, True)[1] == 8
    x = getattr(c, name)
    x.data = swap(x)
    for cache in (c, m.CacheQ8(c.k, c.k_scale, c.v, c.v_scale, c.kidx, c.kidx_scale)):
        with pytest.raises((TypeError, ValueError)):
            cache._struct(dims, dev, True, True)


def test_a_cache_that_grows_is_taken_as_it_is():
    dims = m.Dims(16, 4, 128, 64, 4, 3)
    c, big = m.CacheQ8.zeros(dims, 2, "cpu"), m.CacheQ8.zeros(dims, 5, "cpu")
    dev = c.k.get_device()
    assert c._struct(dims, dev, True, False)[1] == 2
    for name in ("k", "k_scale", "v", "v_scale"):
        getattr(c, name).data = getattr(big, name)
    assert c._struct(dims, dev, True, False)[1] == 5

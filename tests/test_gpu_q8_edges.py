"""8-bit caches on the GPU, where it can go wrong: rows of V without a nonzero code, rows that cannot be answered among
rows that can, q and unseen tokens of any bits, lengths and windows at the ends of their ranges, the last bit of cosines
and sines, and long streams (more items than CTAs, many refills of a ring).  References and bounds: tests/_q8.py."""
import math

import pytest
import torch

from tests import _q8 as Q
from tests.test_gpu_q8 import E4M3, E8M0, cuda, i32, make_cache, msa, u8  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ caches

def test_a_cache_whose_tensors_changed_is_refused(msa):  # noqa: F811
    dims = msa.Dims(8, 1, 64, 32, 1, 2)
    cache, _ = make_cache(msa, dims, 4, 3)
    q, z = Q.normal((1, 8, 64), 5).cuda(), i32([0]).cuda()
    table = i32([[3, 3]]).cuda()
    calls = [lambda: msa.msa_window_attn_q8(q, cache, table, z, z, 5, 0, dims, 0),
             lambda: msa.msa_index_score_q8(q[:, :1, :32].contiguous(), cache, table, z, z, dims)]
    for call, name in zip(calls, ("v", "kidx")):
        call()
        x = getattr(cache, name)
        x.data = x[:2].clone()
        with pytest.raises(ValueError, match="shape"):
            call()

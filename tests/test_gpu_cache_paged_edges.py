"""The paged cache calls at their edges, against the plain 64-bit
implementation, as test_gpu_cache_paged.py.
"""
import numpy as np
import pytest
import torch

import nvfp4_quantization_amax_b200 as mxq
import paged_reference as ref
from test_gpu_cache_paged import as_f64, dev

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("S", [1, 5, 24, 64])
@pytest.mark.parametrize("fmt,block", [("fp8", 8), ("mxfp4", 8), ("mxfp4", 16), ("nvfp4", 16),
                                       ("fp8", None)])
def test_bounds_of_every_head_size(fmt, block, S):
    # rows of 1 to 64 lanes: those that divide a warp and those that do not
    for D in range(8, 513, 8):
        B = block or D
        if D % B:
            continue
        lens = [S + max(1, S // 2), S]
        cache = ref.Cache(lens, 1, D, S, fmt, B, seed=D + S, spare=1, same=True, spread=6.0)
        want = ref.bounds(cache)
        got = as_f64(mxq.bound_cache_pages(dev(cache.k), dev(cache.table), dev(cache.lengths), fmt,
                                           B))
        held = ~np.isnan(want)
        assert np.array_equal(got[held], want[held]), D
        assert not got[~held].any(), D

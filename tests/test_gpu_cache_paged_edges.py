"""The paged cache calls at their edges, against the plain 64-bit
implementation, as test_gpu_cache_paged.py.
"""
import numpy as np
import pytest
import torch

import nvfp4_quantization_amax_b200 as mxq
import paged_reference as ref
from test_gpu_cache_paged import as_f64, dev, queries

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


# ----------------------------------------------------- queries not finite

# the tensor-core kernels with one and several scales a row, and the general one
KERNELS = [("fp8", 128, 128, 16), ("fp8", 32, 128, 16), ("mxfp4", 32, 64, 16), ("nvfp4", 16, 64, 16),
           ("fp8", 8, 40, 10), ("nvfp4", 8, 64, 16), ("mxfp4", 20, 80, 24)]


@pytest.mark.parametrize("fmt,block,D,S", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_a_query_that_is_not_finite_gives_nan(fmt, block, D, S, dtype):
    # in its own head's row; a sequence without tokens has zeros all the same
    lens = [0, 1, 37, 2500]
    cache = ref.Cache(lens, 2, D, S, fmt, block, seed=D)
    q = queries(4, 6, D, dtype)
    want, wl, spread, reach = ref.attend(cache, q)
    args = (dev(cache.k), dev(cache.v), dev(cache.table), dev(cache.lengths), fmt, block)
    tol = ref.out_tolerance(dtype, D, 2500, want, spread, reach)
    ltol = ref.lse_tolerance(D, 2500, wl, reach)
    for x in (float("nan"), float("inf"), float("-inf")):
        bad = q.clone()
        bad[:, 1, 5] = x
        out, lse = mxq.attend_cache_paged(dev(bad), *args, return_lse=True)
        out, lse = as_f64(out), as_f64(lse)
        assert not out[0].any() and np.isneginf(lse[0]).all()
        assert np.isnan(out[1:, 1]).all() and np.isnan(lse[1:, 1]).all()
        others = [0, 2, 3, 4, 5]
        assert (np.abs(out[1:, others] - want[1:, others]) <= tol[1:, others]).all()
        assert (np.abs(lse[1:, others] - wl[1:, others]) <= ltol[1:, others]).all()

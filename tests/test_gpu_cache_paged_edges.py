"""The paged cache calls at their edges, against the plain 64-bit
implementation, as test_gpu_cache_paged.py.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import nvfp4_quantization_amax_b200 as mxq
import paged_reference as ref
from test_gpu_cache_paged import as_f64, check_attend, dev, queries

pytestmark = pytest.mark.gpu

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# ------------------------------------------- keys and logits far from others

def query_error(cache, q):
    """[n, Hq]: what the rounding of queries to f16 terms adds to a logit's
    error.  A head's elements are scaled by a power of two, the largest to
    [2^13, 2^14).  Of an element the terms keep 22 bits (one term of a bf16 or
    f16 element all of it), but nothing under f16's smallest step: half of 2^-24
    beside 2^13 is 2^-38 of the largest, times the sum of the key's magnitudes."""
    n, Hq, D = q.shape
    top = q.double().abs().amax(-1).numpy()
    keys = np.zeros((n, Hq))
    for b in range(n):
        for j in range(Hq):
            k = np.abs(cache.values(cache.k, b, j * cache.H // Hq)).sum(1)
            keys[b, j] = k.max() if k.size else 0.0
    return 2.0 ** -38 * top * keys / D ** 0.5


def check_within(cache, q, spare):
    """check_attend's bounds with `spare` more of error for each head's logits."""
    out, lse = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(cache.table),
                                      dev(cache.lengths), cache.fmt, cache.block, return_lse=True)
    want, wl, spread, reach = ref.attend(cache, q)
    N, D = max(cache.lens), cache.D
    tol = ref.out_tolerance(q.dtype, D, N, want, spread, reach) + 2 * spare[..., None] * spread
    assert (np.abs(as_f64(out) - want) <= tol).all(), np.max(np.abs(as_f64(out) - want) / tol)
    tol = ref.lse_tolerance(D, N, wl, reach) + spare
    assert (np.abs(as_f64(lse) - wl) <= tol).all(), np.max(np.abs(as_f64(lse) - wl) / tol)


@pytest.mark.parametrize("fmt,block,D,S", [("fp8", 8, 40, 10), ("fp8", 16, 128, 16),
                                           ("fp8", 1, 7, 3), ("mxfp4", 8, 64, 16),
                                           ("mxfp4", 20, 80, 24), ("mxfp4", 64, 512, 16),
                                           ("fp8", 32, 128, 16), ("mxfp4", 32, 128, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_keys_with_a_block_far_above_the_others(fmt, block, D, S, dtype):
    # the second block's keys are 2^by times the others'; the query is zero or
    # as much smaller there, so that the logits are those of the other blocks,
    # or of all
    for by in (21, 22, 27, 28, 60, 120):
        cache = ref.Cache([70, 1, 33], 2, D, S, fmt, block, seed=D)
        live = cache.k[1][..., 1] != 0xFF
        live[::2] = live[::2] & (torch.arange(S) % 3 != 0)  # not every token's
        cache.k[1][..., 1] = torch.where(live, cache.k[1][..., 1] + by, cache.k[1][..., 1])
        q = queries(3, 4, D, dtype)
        q[..., block:2 * block] = 0
        check_attend(cache, q)
        if by < 30:
            q[..., block:2 * block] = queries(3, 4, D, dtype, seed=5)[..., :block] * 2.0 ** -by
            check_within(cache, q, query_error(cache, q))


@pytest.mark.parametrize("fmt,block", [("fp8", 8), ("mxfp4", 8)])
def test_keys_with_empty_blocks(fmt, block):
    # a block of zeros has the least scale
    cache = ref.Cache([70, 1, 33], 2, 64, 10, fmt, block, seed=2)
    codes, scales = cache.k
    width = block if fmt == "fp8" else block // 2
    live = scales[..., 3] != 0xFF
    codes[..., 3 * width:4 * width][live] = 0
    scales[..., 3] = torch.where(live, torch.tensor(1, dtype=torch.uint8), scales[..., 3])
    check_attend(cache, queries(3, 4, 64, torch.float32))


@pytest.mark.parametrize("fmt,block,D,S", [("fp8", 32, 128, 16), ("mxfp4", 32, 64, 16),
                                           ("fp8", 8, 40, 10), ("mxfp4", 20, 80, 24)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_with_a_block_as_far_below_as_still_counts(fmt, block, D, S, dtype):
    # 18 binades (mxfp4: 23) beneath the token's largest scale: every bit, in
    # channels of its own
    down = 18 if fmt == "fp8" else 23
    cache = ref.Cache([70, 1, 333], 2, D, S, fmt, block, seed=D)
    scales = cache.v[1]
    live = scales[..., 1] != 0xFF
    top = scales.int().amax(-1)
    scales[..., 1] = torch.where(live, (top - down).to(torch.uint8), scales[..., 1])
    check_attend(cache, queries(3, 4, D, dtype))


@pytest.mark.parametrize("fmt,block,D,S", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_first_logits_far_below_the_others(fmt, block, D, S, dtype):
    """The first tokens' logits are lower than the others' by so much that a
    difference from one of them has none of the others' bits.  Errors are
    those of the tokens with weight: a logit's is relative to its own terms."""
    far, n = 200, 700
    cache = ref.Cache([n], 1, D, S, fmt, block, seed=3)
    q = queries(1, 2, D, dtype)
    q[0, 1] = q[0, 0] * 0.5
    row = (q[0, 0].double() * (-400.0 if fmt == "nvfp4" else -2.0 ** 20)).to(torch.bfloat16)
    codes, scales = ref.pack(row.view(1, D), fmt, block)
    for t in range(far):
        page = int(cache.table[0, t // S])
        cache.k[0][page, 0, t % S], cache.k[1][page, 0, t % S] = codes[0], scales[0]
    z = (cache.values(cache.k, 0, 0) @ q[0].double().numpy().T) / D ** 0.5
    assert (z[:far].max(0) < z[far:].max(0) - (1000 if fmt == "nvfp4" else 10 ** 6)).all()
    out, lse = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(cache.table),
                                      dev(cache.lengths), fmt, block, return_lse=True)
    want, wl, spread, _ = ref.attend(cache, q)
    k = np.abs(cache.values(cache.k, 0, 0)[far:])
    reach = (k @ np.abs(q[0].double().numpy()).T).max(0)[None] / D ** 0.5
    tol = ref.out_tolerance(dtype, D, n, want, spread, reach)
    assert (np.abs(as_f64(out) - want) <= tol).all(), np.max(np.abs(as_f64(out) - want) / tol)
    tol = ref.lse_tolerance(D, n, wl, reach)
    assert (np.abs(as_f64(lse) - wl) <= tol).all(), np.max(np.abs(as_f64(lse) - wl) / tol)


@pytest.mark.parametrize("fmt,block,D,S", [x for x in KERNELS if x[0] != "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_logits_so_large_that_a_scale_is_lost_beside_them(fmt, block, D, S, dtype):
    """Logits of up to 2^100, exact ones (a query that is one channel): the
    weights are those of the tokens with the largest, each 1, whatever the
    values' scales; no error of a logit counts."""
    for by, by_v in ((20, 8), (30, 8), (30, -20), (100, 8),
                     (100, 10 if dtype == torch.float16 else 40)):
        lens = [0, 300, 21]
        cache = ref.Cache(lens, 1, D, S, fmt, block, seed=by + D)
        for which, add in ((cache.k, by), (cache.v, by_v)):
            which[1][:] = torch.where(which[1] == 0xFF, which[1], (which[1] + add).to(torch.uint8))
        q = torch.zeros(3, 2, D, dtype=dtype)
        q[:, 0, 3], q[:, 1, 2] = 1.0, -2.0
        out, lse = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(cache.table),
                                          dev(cache.lengths), fmt, block, scale=1.0,
                                          return_lse=True)
        want, wl, spread, reach = ref.attend(cache, q, scale=1.0)
        tol = ref.out_tolerance(dtype, D, 300, want, spread, 0 * reach)
        assert (np.abs(as_f64(out) - want) <= tol).all(), (by, by_v)
        tol = ref.lse_tolerance(D, 300, wl, 0 * reach)
        assert (np.abs(as_f64(lse)[1:] - wl[1:]) <= tol[1:]).all(), (by, by_v)
        assert not out[0].any() and torch.isneginf(lse[0]).all()


def weight_error(cache, q, scale):
    """[n, Hq]: what weights held to f16's smallest step add to a result.  The
    largest product of a weight and a value scale is at 2^11 or above, a
    weight off by at most half of 2^-24 there: 2^-36 of that product for each
    token, times the largest code.  Tokens with several scales of values are
    taken together where these lie within 2^20 (2^8 for f16 and f32 results),
    with the largest of them all, so the product may be that much above a
    token's own; and a token's largest value is at least half of the largest
    code times its scale."""
    n, Hq, D = q.shape
    step = np.zeros((n, Hq))
    together = 2.0 ** (20 if q.dtype == torch.bfloat16 else 8)
    if cache.fmt == "nvfp4" or cache.block == D:
        together = 1.0
    for b in range(n):
        for j in range(Hq):
            h = j * cache.H // Hq
            k, v = cache.values(cache.k, b, h), cache.values(cache.v, b, h)
            if len(k):
                z = scale * (k @ q[b, j].double().numpy())
                w = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
                step[b, j] = 2.0 ** -35 * together * len(z) * (w * np.abs(v).max(1)).max()
    return step


@pytest.mark.parametrize("fmt,block,D,S", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_values_far_apart_beside_large_logits(fmt, block, D, S, dtype):
    # tokens' values over forty binades, so that turns are taken in bands, and
    # logits of up to 2^28 of either sign: a band may hold none of the largest
    for seed in range(6):
        cache = ref.Cache([0, 700, 35], 1, D, S, fmt, block, seed=seed)
        if fmt != "nvfp4":
            g = torch.Generator().manual_seed(seed)
            live = cache.k[1] != 0xFF
            most = 8 if dtype == torch.float16 else 20
            k = torch.randint(0, 26, live.shape[:3] + (1,), generator=g)
            v = torch.randint(-20, most + 1, live.shape[:3] + (1,), generator=g)
            for which, add in ((cache.k, k), (cache.v, v)):
                which[1][:] = torch.where(live, (which[1].int() + add).to(torch.uint8), which[1])
        q = queries(3, 3, D, dtype, seed=seed)
        out, lse = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(cache.table),
                                          dev(cache.lengths), fmt, block, return_lse=True)
        want, wl, spread, reach = ref.attend(cache, q)
        tol = ref.out_tolerance(dtype, D, 700, want, spread, reach)
        tol = tol + weight_error(cache, q, D ** -0.5)[..., None]
        got = as_f64(out)
        over = np.isinf(got)  # of f16 results alone
        assert (np.abs(want)[over] + tol[over] >= torch.finfo(dtype).max).all()
        assert (np.abs(got - want)[~over] <= tol[~over]).all(), seed
        tol = ref.lse_tolerance(D, 700, wl, reach)
        assert (np.abs(as_f64(lse)[1:] - wl[1:]) <= tol[1:]).all(), seed


@pytest.mark.parametrize("fmt,block,D,S", [("fp8", 128, 128, 16), ("fp8", 32, 128, 16),
                                           ("mxfp4", 32, 64, 16), ("fp8", 32, 256, 32),
                                           ("fp8", 8, 40, 10), ("mxfp4", 20, 80, 24)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_small_weights_of_large_values(fmt, block, D, S, dtype):
    """16 tokens of weight about 1/16 and 48 of about 2^-40 whose values are
    2^17 times as large: 2^-14 of the result, which f32's weights have to hold.
    A token's error is relative to what it adds."""
    cache = ref.Cache([64], 1, D, S, fmt, block, seed=D, spread=0.0)
    q = queries(1, 1, D, dtype)
    u = q[0, 0].double()
    row = (u * (-25.3 * D ** 0.5 / (u @ u))).to(torch.bfloat16)
    first = [int(x) for x in torch.arange(64) % 4 == 0]  # in one turn with the others
    for t in range(64):
        page, slot = int(cache.table[0, t // S]), t % S
        codes, scales = ref.pack((0 * row if first[t] else row).view(1, D), fmt, block)
        cache.k[0][page, 0, slot], cache.k[1][page, 0, slot] = codes[0], scales[0]
        if not first[t]:  # the values of the first token, larger
            at = int(cache.table[0, 0])
            cache.v[0][page, 0, slot] = cache.v[0][at, 0, 0]
            cache.v[1][page, 0, slot] = cache.v[1][at, 0, 0] + 17
    out = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(cache.table),
                                 dev(cache.lengths), fmt, block)
    want, _, _, _ = ref.attend(cache, q)
    k, v = cache.values(cache.k, 0, 0), np.abs(cache.values(cache.v, 0, 0))
    z = (k @ u.numpy()) / D ** 0.5
    w = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
    assert 2.0 ** -44 < w[1] < 2.0 ** -39
    reach = (np.abs(k) @ np.abs(u.numpy())) / D ** 0.5
    delta = reach * ((D + 8) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -20 + 64 * 2.0 ** -24
    delta += 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21
    # as weight_error, with tokens of f16 and f32 results taken together where
    # their scales lie within 2^8
    together = 2.0 ** (20 if dtype == torch.bfloat16 else 8) if block < D else 1.0
    least = 64 * 2.0 ** -35 * together * (w[:, None] * v).max()
    tol = torch.finfo(dtype).eps / 2 * np.abs(want[0, 0]) + 2 * ((w * delta) @ v) + least
    assert (np.abs(as_f64(out)[0, 0] - want[0, 0]) <= tol).all()


# ---------------------------------------------------------- host arguments

def busy():
    """Work on the current stream that lasts about a tenth of a second."""
    torch.cuda._sleep(200_000_000)


def pinned(t):
    return t.cpu().clone().pin_memory()


def test_pinned_arguments_may_change_when_a_call_has_returned():
    """What a call reads of pinned host tensors it has read when it returns,
    or its results are on the host: the caller may write the next step's
    values into them."""
    cache = ref.Cache([40, 33], 2, 64, 16, "fp8", 64)
    table, lengths = cache.table, cache.lengths
    offs = torch.tensor([2, 3], dtype=torch.int32)
    x = torch.randn(3, 2, 64).to(torch.bfloat16)
    q, pages = queries(2, 4, 64, torch.bfloat16), torch.tensor([[[0, 2]] * 2, [[1, 2]] * 2]).int()
    bd = torch.randn(cache.P, 2, 2, 64).to(torch.bfloat16)

    def calls(k, v, host, x):
        """One call of each kind with new copies of its arguments by `host`;
        these are overwritten (with valid values) as soon as it returns."""
        def args():
            return host(table), host(lengths)

        def gone(*ts):
            for t in ts:
                if not t.is_cuda:
                    t.copy_(torch.where(t > 1, t - 1, t) if t.dtype == torch.int32 else t * 0 + 1)

        out = []
        t, n, o, new = *args(), host(offs), x(x0)
        busy()
        mxq.append_cache_paged(new, new, o, t, n, k, v, "fp8", 64)
        gone(t, n, o, new)
        out += [*k, *v]
        t, n = args()
        busy()
        out.append(mxq.bound_cache_pages(k, t, n, "fp8", 64))
        gone(t, n)
        t, n = args()
        busy()
        out.append(mxq.select_cache_pages(dev(q), dev(bd), t, n, 16, 2))
        gone(t, n)
        t, n, p = *args(), host(pages)
        busy()
        out.append(mxq.attend_cache_paged(dev(q), k, v, t, n, "fp8", 64, pages=p))
        gone(t, n, p)
        torch.cuda.synchronize()
        return [y.cpu() for y in out]

    x0 = x
    want = calls(dev(cache.k), dev(cache.v), dev, dev)
    for move in (dev, pinned):  # the rows on the device, or pinned too
        got = calls(dev(cache.k), dev(cache.v), pinned, move)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_pinned_offs_of_a_grouped_product_may_change_when_the_call_has_returned():
    x = torch.randn(40, 512, device=DEV).to(torch.bfloat16)
    packed, scales = mxq.mx_quantize(torch.randn(2, 256, 512, device=DEV).to(torch.bfloat16))
    offs = torch.tensor([16, 40], dtype=torch.int32)
    for product in (mxq.mxfp4_grouped_mm, mxq.w4a4_grouped_mm):
        want = product(x, packed, scales, dev(offs))
        host = pinned(offs)
        busy()
        got = product(x, packed, scales, host)
        host.copy_(torch.tensor([1, 40]))
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_a_captured_call_reads_pinned_lengths_at_every_replay():
    cache = ref.Cache([40, 33], 2, 64, 16, "fp8", 64)
    k, v, q = dev(cache.k), dev(cache.v), dev(queries(2, 4, 64, torch.bfloat16))
    host, table = pinned(cache.lengths), dev(cache.table)

    def attend(lengths):
        return mxq.attend_cache_paged(q, k, v, table, lengths, "fp8", 64)

    attend(host)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attend(host)
    for lens in ([40, 33], [20, 10]):
        host.copy_(torch.tensor(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, attend(dev(host)))


# ------------------------------------------------------------ failed launches

FAILED_LAUNCH = """
import ctypes
import torch
import nvfp4_quantization_amax_b200 as mxq

dev, n, H, D, S, P = "cuda", 1, 1, {dim}, {page}, 4
cache = [torch.zeros(P, H, S, w, dtype=torch.uint8, device=dev) for w in (D, 1)]
table = torch.arange(P, dtype=torch.int32, device=dev).view(n, P)
lengths = torch.tensor([P * S], dtype=torch.int32, device=dev)
q = torch.zeros(n, 2, D, dtype=torch.bfloat16, device=dev)
out, ws = torch.empty_like(q), torch.empty(16 << 20, dtype=torch.uint8, device=dev)
x = torch.randn(4, 64, device=dev).to(torch.bfloat16)

def attend():
    return mxq.attend_cache_paged(q, cache, cache, table, lengths, "fp8", D, out=out, workspace=ws)

attend()
want = mxq.quantize_cache(x, "fp8", 32)
torch.cuda.synchronize()
# while a stream that the legacy stream waits for is being captured, the
# runtime refuses launches on the legacy stream: nothing of the call runs
rt = ctypes.CDLL("libcudart.so.12")
stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
assert rt.cudaStreamBeginCapture(stream, 0) == 0
try:
    attend()
    failed = False
except mxq.MxqError as e:
    failed = e.status == -5
rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
rt.cudaGetLastError()
assert failed
got = mxq.quantize_cache(x, "fp8", 32)  # the next call is not told of it
attend()
torch.cuda.synchronize()
assert torch.equal(got, want) and not out.any()
print("next call ok")
"""


@pytest.mark.parametrize("dim,page", [(128, 64), (40, 100)])
def test_a_refused_launch_is_reported_once(dim, page):
    r = subprocess.run([sys.executable, "-c", FAILED_LAUNCH.format(dim=dim, page=page)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "next call ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("fmt,block", [("fp8", 16), ("fp8", 2), ("mxfp4", 32), ("nvfp4", 4)])
def test_head_sizes_in_any_order(fmt, block):
    # one kernel with more, less and again more shared memory
    for D in (384, 512, 320, 512, 384):
        cache = ref.Cache([33, 2], 1, D, 16, fmt, block, seed=D)
        check_attend(cache, queries(2, 2, D, torch.bfloat16))


# ------------------------------------------------------------ bad offs

def test_bad_offs_touch_no_slot_outside_the_sequences():
    rng = np.random.default_rng(4)
    few = [[2, 1, 6], [5, 3, 6], [6, 0, 2], [-1, 2, 6], [2, 4, 100], [3, 3, -2],
           [2 ** 31 - 1, 2, 4], [-2 ** 31, -2 ** 31, 6]]
    for lens, all_offs in (([20, 30, 8], few),
                           ([1 + i % 40 for i in range(90)],
                            [rng.integers(-3, 10, 90).tolist() for _ in range(4)])):
        for block in (32, 4):  # the fast and the general kernel
            for offs in all_offs:
                cache = ref.Cache(lens, 2, 64, 16, "fp8", block, empty=True)
                kc = dev(cache.k)
                status = torch.zeros(1, dtype=torch.int32, device=DEV)
                x = torch.randn(6, 2, 64).to(torch.bfloat16)
                mxq.append_cache_paged(dev(x), None, dev(torch.tensor(offs, dtype=torch.int32)),
                                       dev(cache.table), dev(cache.lengths), kc, None, "fp8", block,
                                       status=status)
                assert int(status) in (-6, -8)
                for got, was in zip(kc, cache.k):
                    free = ~cache.held[:, None].expand(-1, 2, -1)
                    assert torch.equal(got.cpu()[free], was[free])


# ------------------------------------------------------ very many sequences

@pytest.mark.parametrize("block", [64, 4])  # the fast and the general kernel
def test_append_to_as_many_sequences_as_are_counted(block):
    # 2^31 - 2 sequences, three of which own a row: places of the searches pass
    # 31 bits
    n, D, S = 2 ** 31 - 2, 64, 16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    owners = [0, 2 ** 30 + 5, n - 1]
    offs, lengths = [torch.zeros(n, dtype=torch.int32, device=DEV) for _ in range(2)]
    table = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    for i, b in enumerate(owners):
        offs[b:] = i + 1
        lengths[b], table[b, 0] = i + 1, i + 1
    cache = tuple(torch.full((5, 1, S, w), 0xAA, dtype=torch.uint8, device=DEV)
                  for w in (D, D // block))
    x = torch.randn(4, 1, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    mxq.append_cache_paged(dev(x), None, offs, table, lengths, cache, None, "fp8", block)
    want = [torch.full_like(t, 0xAA, device="cpu") for t in cache]
    for w, rows in zip(want, ref.pack(x, "fp8", block)):
        for i in range(3):  # the fourth row is padding
            w[i + 1, :, i] = rows[i]
    for got, w in zip(cache, want):
        assert torch.equal(got.cpu(), w)


# ------------------------------------------------------------ index checks

def test_debug_variant_without_a_failed_check():
    """The cases above on the library's debug variant, whose kernels check
    their indexes (tests/conftest.py asks for its record after each)."""
    from nvfp4_quantization_amax_b200 import build

    env = dict(os.environ, MXQ_LIBRARY=build.build(debug=True), MXQ_EXPECT_CLEAN_CHECKS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        "-k", "not debug_variant", os.path.abspath(__file__)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-1000:]

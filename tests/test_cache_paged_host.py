"""Refusals of the paged cache calls: every argument error comes back before
anything is launched (the pointers here are stand-ins that are never
dereferenced), and the binding refuses what it cannot hand on."""
import ctypes
import os

import numpy as np
import pytest
import torch

import nvfp4_quantization_amax_b200 as mxq
import paged_reference as ref
from nvfp4_quantization_amax_b200 import build as mxq_build
from test_binding_names import unbound_names

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EARG, ESHAPE, EALIGN, EUNSUP = 0, -1, -2, -3, -4
FP8, MXFP4, NVFP4 = 0, 1, 2


def P(i):
    return (i + 1) << 28  # distinct, far apart, 16-byte aligned


# Valid calls by argument name, in the order of the C prototypes.
CALLS = {
    "append_cache_paged": dict(
        k=P(0), v=P(1), dtype=0, rows=6, kv_heads=2, head_dim=64, k_stride=128, v_stride=128,
        offs=P(2), page_table=P(3), lengths=P(4), n_seqs=3, max_pages=4, format=MXFP4,
        block_size=32, num_pages=9, page_size=16, k_codes=P(5), k_scales=P(6), v_codes=P(7),
        v_scales=P(8), k_out=P(9), v_out=P(10), dev_status=P(11), stream=None),
    "bound_cache_pages": dict(
        k_codes=P(0), k_scales=P(1), kv_heads=2, head_dim=64, format=MXFP4, block_size=32,
        num_pages=9, page_size=16, page_table=P(2), lengths=P(3), n_seqs=3, max_pages=4,
        new_tokens=5, bounds=P(4), dev_status=P(5), stream=None),
    "select_cache_pages": dict(
        q=P(0), dtype=0, n_seqs=3, q_heads=4, kv_heads=2, head_dim=64, q_stride=256, bounds=P(1),
        num_pages=9, page_size=16, page_table=P(2), lengths=P(3), max_pages=4, top=3, keep_first=1,
        keep_last=1, selected=P(4), workspace=P(5), dev_status=P(6), stream=None),
    "attend_cache_paged": dict(
        q=P(0), dtype=0, n_seqs=3, q_heads=4, kv_heads=2, head_dim=64, q_stride=256, k_codes=P(1),
        k_scales=P(2), v_codes=P(3), v_scales=P(4), format=MXFP4, block_size=32, num_pages=9,
        page_size=16, page_table=P(5), lengths=P(6), max_pages=4, selected=P(7), top=3, window=0,
        softmax_scale=0.125, out=P(8), lse=P(9), workspace=P(10), dev_status=P(11), stream=None),
}
REQUIRED = {
    "append_cache_paged": ["k", "offs", "page_table", "lengths", "k_codes", "k_scales", "v_codes",
                           "v_scales"],
    "bound_cache_pages": ["k_codes", "k_scales", "page_table", "lengths", "bounds"],
    "select_cache_pages": ["q", "bounds", "page_table", "lengths", "selected", "workspace"],
    "attend_cache_paged": ["q", "k_codes", "k_scales", "v_codes", "v_scales", "page_table",
                           "lengths", "out", "workspace"],
}
ALIGNED = {
    "append_cache_paged": dict(k=2, v=2, offs=4, page_table=4, lengths=4, k_out=2, v_out=2,
                               dev_status=4),
    "bound_cache_pages": dict(page_table=4, lengths=4, bounds=2, dev_status=4),
    "select_cache_pages": dict(q=2, bounds=2, page_table=4, lengths=4, selected=4, workspace=16,
                               dev_status=4),
    "attend_cache_paged": dict(q=2, page_table=4, lengths=4, selected=4, out=16, lse=4,
                               workspace=16, dev_status=4),
}
OUTPUTS = {
    "append_cache_paged": ["k_codes", "k_scales", "v_codes", "v_scales", "k_out", "v_out",
                           "dev_status"],
    "bound_cache_pages": ["bounds", "dev_status"],
    "select_cache_pages": ["selected", "workspace", "dev_status"],
    "attend_cache_paged": ["out", "lse", "workspace", "dev_status"],
}
BIG = 1 << 40
BAD = {
    "append_cache_paged": [
        (dict(dtype=3), EARG), (dict(format=3), EARG), (dict(rows=-1), ESHAPE),
        (dict(n_seqs=-1), ESHAPE), (dict(kv_heads=0), ESHAPE), (dict(head_dim=48), ESHAPE),
        (dict(block_size=0), ESHAPE), (dict(head_dim=63, block_size=21), ESHAPE),
        (dict(max_pages=0), ESHAPE), (dict(num_pages=0), ESHAPE), (dict(page_size=0), ESHAPE),
        (dict(k_stride=127), ESHAPE), (dict(v_stride=127), ESHAPE),
        (dict(head_dim=1024, k_stride=2048, v_stride=2048), EUNSUP), (dict(rows=1 << 31), EUNSUP),
        (dict(num_pages=1 << 31), EUNSUP), (dict(max_pages=1 << 30), EUNSUP),
        (dict(kv_heads=65536, k_stride=BIG, v_stride=BIG), EUNSUP),
        (dict(k_stride=1 << 59), ESHAPE), (dict(v=None), EARG),
        (dict(v=None, v_codes=None, v_scales=None), EARG)],
    "bound_cache_pages": [
        (dict(format=-1), EARG), (dict(head_dim=40), ESHAPE), (dict(n_seqs=-1), ESHAPE),
        (dict(new_tokens=-1), ESHAPE), (dict(page_size=0), ESHAPE), (dict(head_dim=544), EUNSUP),
        (dict(page_size=1 << 29), EUNSUP)],
    "select_cache_pages": [
        (dict(dtype=-1), EARG), (dict(q_heads=3), ESHAPE), (dict(q_heads=0), ESHAPE),
        (dict(q_stride=255), ESHAPE), (dict(top=-1), ESHAPE), (dict(keep_first=3), ESHAPE),
        (dict(keep_last=-1), ESHAPE), (dict(keep_first=-1), ESHAPE), (dict(top=1), ESHAPE),
        (dict(keep_last=BIG), ESHAPE), (dict(top=BIG), EUNSUP), (dict(head_dim=513, q_stride=BIG),
                                                                  EUNSUP),
        (dict(n_seqs=1 << 29, q_stride=1 << 31), EUNSUP)],
    "attend_cache_paged": [
        (dict(dtype=9), EARG), (dict(format=7), EARG), (dict(q_heads=3), ESHAPE),
        (dict(q_stride=255), ESHAPE), (dict(window=-1), ESHAPE), (dict(top=-1), ESHAPE),
        (dict(head_dim=32, block_size=64), ESHAPE), (dict(block_size=64, head_dim=96), ESHAPE),
        (dict(top=0), EARG), (dict(selected=None), EARG),
        (dict(softmax_scale=float("nan")), EARG), (dict(softmax_scale=float("inf")), EARG),
        (dict(top=1 << 27), EUNSUP), (dict(num_pages=1 << 32), EUNSUP)],
}
NOOP = {
    "append_cache_paged": [dict(rows=0, k=None, v=None), dict(n_seqs=0, offs=None)],
    "bound_cache_pages": [dict(n_seqs=0, page_table=None), dict(new_tokens=0, bounds=None)],
    "select_cache_pages": [dict(n_seqs=0, q=None), dict(top=0, keep_first=0, keep_last=0,
                                                        selected=None)],
    "attend_cache_paged": [dict(n_seqs=0, q=None, out=None)],
}


@pytest.fixture(scope="module")
def call():
    mxq_build.build()
    L = mxq.lib()

    def go(name, **change):
        assert not set(change) - set(CALLS[name])
        return getattr(L, name)(*{**CALLS[name], **change}.values())

    return go


NAMES = sorted(CALLS)


@pytest.mark.parametrize("name", NAMES)
def test_bad_sizes_and_enums_are_refused(call, name):
    for change, want in BAD[name]:
        assert call(name, **change) == want, change


@pytest.mark.parametrize("name", NAMES)
def test_null_pointers_are_refused(call, name):
    for arg in REQUIRED[name]:
        assert call(name, **{arg: None}) == EARG, arg


@pytest.mark.parametrize("name", NAMES)
def test_pointers_off_their_boundary_are_refused(call, name):
    for arg, boundary in ALIGNED[name].items():
        for off in {1, boundary // 2} - {0}:
            assert call(name, **{arg: CALLS[name][arg] + off}) == EALIGN, (arg, off)
    for dtype_arg in ("k", "q"):
        if dtype_arg in CALLS[name]:  # f32 elements sit on 4 bytes
            assert call(name, dtype=2, **{dtype_arg: CALLS[name][dtype_arg] + 2}) == EALIGN


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_overlap_anything_are_refused(call, name):
    pointers = [a for a, x in CALLS[name].items() if isinstance(x, int) and x >= P(0)]
    for out in OUTPUTS[name]:
        for other in pointers:
            if other != out:
                assert call(name, **{out: CALLS[name][other]}) == EARG, (out, other)
    # the inputs may overlap one another (K and V in one buffer): nothing but
    # the outputs is compared, so the next error shows
    if name == "attend_cache_paged":
        assert call(name, v_codes=P(1), v_scales=P(2), out=P(1)) == EARG


@pytest.mark.parametrize("name", NAMES)
def test_nothing_to_do_is_no_error(call, name):
    for change in NOOP[name]:
        assert call(name, **change) == OK, change


def test_workspace_sizes(call):
    L = mxq.lib()
    assert L.select_cache_pages_workspace_bytes(3, 2, 5) == 3 * 2 * 5 * 8
    assert L.select_cache_pages_workspace_bytes(0, 2, 5) == 0
    assert L.attend_cache_paged_workspace_bytes(8, 2, 128) > 0
    assert L.attend_cache_paged_workspace_bytes(8, 3, 128) == 0
    assert L.attend_cache_paged_workspace_bytes(8, 2, 513) == 0
    assert mxq.status_string(-8) == "MXQ_ERR_BAD_PAGE"


def test_every_name_of_the_binding_is_bound():
    assert unbound_names(os.path.join(ROOT, "nvfp4_quantization_amax_b200", "_paged.py")) == []


def test_binding_refuses_caches_off_the_gpu():
    c = ref.Cache([5], 1, 64, 16, "fp8", 64)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mxq.attend_cache_paged(q, c.k, c.v, c.table, c.lengths, "fp8", 64)
    with pytest.raises(ValueError, match="CUDA"):
        mxq.append_cache_paged(q[:, :1], None, c.lengths, c.table, c.lengths, c.k, None, "fp8", 64)
    with pytest.raises(ValueError, match="CUDA"):
        mxq.bound_cache_pages(c.k, c.table, c.lengths, "fp8", 64)
    with pytest.raises(ValueError, match="CUDA"):
        mxq.select_cache_pages(q, torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16), c.table,
                               c.lengths, 16, 2)
    with pytest.raises(ValueError, match="format"):
        mxq.attend_cache_paged(q, c.k, c.v, c.table, c.lengths, "fp4", 64)
    with pytest.raises(ValueError, match="block_size"):
        mxq.append_cache_paged(q, None, c.lengths, c.table, c.lengths, c.k, None, "fp8", 0)


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors():
    c = ref.Cache([5, 20], 2, 64, 16, "fp8", 64)
    dev = "cuda"
    k, v = [tuple(t.to(dev) for t in x) for x in (c.k, c.v)]
    t, n = c.table.to(dev), c.lengths.to(dev)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    bd = torch.zeros(c.P, 2, 2, 64, dtype=torch.bfloat16, device=dev)
    pages = torch.zeros(2, 2, 1, dtype=torch.int32, device=dev)
    attend, append = mxq.attend_cache_paged, mxq.append_cache_paged
    ok = (q, k, v, t, n, "fp8", 64)

    def args(**change):
        names = ("q", "k_cache", "v_cache", "page_table", "lengths", "format", "block_size")
        return {**dict(zip(names, ok)), **change}

    for error, change in [
            (TypeError, dict(q=q.double())), (ValueError, dict(q=q[:, :3])),
            (ValueError, dict(q=q[..., :32])), (ValueError, dict(q=q[0])),
            (ValueError, dict(q=q[:1])), (TypeError, dict(lengths=n.long())),
            (TypeError, dict(page_table=t.long())), (ValueError, dict(lengths=n[:1])),
            (ValueError, dict(page_table=t[0])), (ValueError, dict(block_size=32)),
            (ValueError, dict(k_cache=(k[0][..., ::2], k[1]))),
            (ValueError, dict(v_cache=(v[0][:2].contiguous(), v[1][:2].contiguous()))),
            (ValueError, dict(k_cache=(k[0], k[1].cpu()))), (ValueError, dict(window=0)),
            (ValueError, dict(window=-3)), (TypeError, dict(pages=pages.long())),
            (ValueError, dict(pages=pages[:, :1])), (ValueError, dict(pages=pages[..., :0])),
            (ValueError, dict(out=torch.empty(2, 4, 63, dtype=torch.bfloat16, device=dev))),
            (TypeError, dict(out=torch.empty(2, 4, 64, dtype=torch.float16, device=dev))),
            (ValueError, dict(workspace=torch.empty(64, dtype=torch.uint8, device=dev))),
            (ValueError, dict(status=torch.zeros(1, dtype=torch.int32)))]:
        with pytest.raises(error):
            attend(**args(**change))
    for error, bad in [
            (TypeError, (x.double(), x.double())), (ValueError, (x, x[:2])),
            (ValueError, (x, x.half())), (ValueError, (x[:, :1], x[:, :1])),
            (ValueError, (x, None))]:
        with pytest.raises(error):
            append(*bad, n, t, n, k, v, "fp8", 64)
    with pytest.raises(ValueError):
        append(x, x, n[:1], t, n, k, v, "fp8", 64)
    for error, change in [(ValueError, dict(top=-1)), (mxq.MxqError, dict(keep_first=2, top=2)),
                          (ValueError, dict(bounds=bd.float())), (ValueError, dict(bounds=bd[0])),
                          (ValueError, dict(out=torch.empty(3, dtype=torch.int32, device=dev)))]:
        with pytest.raises(error):
            mxq.select_cache_pages(**{**dict(q=q, bounds=bd, page_table=t, lengths=n, page_size=16,
                                             top=2), **change})
    with pytest.raises(ValueError):
        mxq.bound_cache_pages(k, t, n, "fp8", 64, bd.cpu())
    with pytest.raises(mxq.MxqError):
        mxq.bound_cache_pages(k, t, n, "fp8", 64, bd, new_tokens=-1)


def test_the_plain_implementation_against_direct_sums():
    # the 64-bit reference itself, against a direct double loop
    c = ref.Cache([7, 0], 1, 8, 4, "mxfp4", 4, seed=3)
    q = torch.randn(2, 2, 8, generator=torch.Generator().manual_seed(1))
    out, lse, _, _ = ref.attend(c, q, window=5)
    k, v = c.values(c.k, 0, 0), c.values(c.v, 0, 0)
    for j in range(2):
        z = [sum(float(q[0, j, i]) * k[t, i] for i in range(8)) / 8 ** 0.5 for t in range(2, 7)]
        w = [np.exp(x) for x in z]
        assert abs(lse[0, j] - np.log(sum(w))) < 1e-12
        for i in range(8):
            assert abs(out[0, j, i] - sum(a * v[t + 2, i] for t, a in enumerate(w)) / sum(w)) < 1e-12
    assert not out[1].any() and np.isneginf(lse[1]).all()

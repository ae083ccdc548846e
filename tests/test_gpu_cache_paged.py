"""GPU parity of the paged cache calls against the plain 64-bit
implementation (tests/paged_reference.py), through the Python binding.

Codes, scale bytes, stored values, bounds and page choices must be equal;
attention must lie within the bound that its arithmetic gives.
"""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantization_amax_b200 as mxq
import oracle
import paged_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAD_OFFS, BAD_PAGE = -6, -8


def dev(x):
    return tuple(t.to(DEV) for t in x) if isinstance(x, tuple) else x.to(DEV)


def queries(n, Hq, D, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, Hq, D, generator=g) * 1.5).to(dtype)


# ------------------------------------------------------------------ append

def check_append(lens, new, H, D, S, fmt, block, dtype, pad=0, strided=False, with_v=True, seed=5):
    cache = ref.Cache(lens, H, D, S, fmt, block, seed=seed, empty=True)
    g = torch.Generator().manual_seed(seed)
    T = sum(new) + pad
    wide = torch.randn(T, (2 * H + 3) * D, generator=g) * torch.exp2(
        6 * torch.rand(T, 1, generator=g) - 3)
    wide[torch.rand(wide.shape, generator=g) < 0.02] = 0.0
    wide = wide.to(dtype)
    k, v = wide[:, D:(H + 1) * D], wide[:, (H + 2) * D:(2 * H + 2) * D]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    offs = torch.tensor(np.cumsum(new), dtype=torch.int32)
    kc, vc = dev(cache.k), dev(cache.v)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dk, dv = wide.to(DEV)[:, D:(H + 1) * D], wide.to(DEV)[:, (H + 2) * D:(2 * H + 2) * D]
    if not strided:
        dk, dv = dk.contiguous(), dv.contiguous()
    got = mxq.append_cache_paged(dk.unflatten(1, (H, D)), dv.unflatten(1, (H, D)) if with_v else None,
                                 dev(offs), dev(cache.table), dev(cache.lengths), kc,
                                 vc if with_v else None, fmt, block, values=True, status=status)
    assert int(status) == 0
    for x, held, back, vals in ((k, cache.k, kc, got[0]), (v, cache.v, vc, got[1])):
        want_c, want_s = held[0].clone(), held[1].clone()
        if x is k or with_v:
            codes, scales = ref.pack(x.contiguous().view(T, H, D), fmt, block)
            t = 0
            for b, m in enumerate(new):
                for i in range(m):
                    pos = lens[b] - m + i
                    page, slot = int(cache.table[b, pos // S]), pos % S
                    want_c[page, :, slot], want_s[page, :, slot] = codes[t], scales[t]
                    t += 1
            name = ref.BITS[dtype][2]
            q = oracle.quantize_cache(ref.bits(x.contiguous().view(T * H, D)), fmt, block, name)
            n = sum(new)
            assert np.array_equal(ref.bits(vals[:n]).reshape(n * H, D),
                                  np.asarray(q).reshape(T * H, D)[:n * H])
        else:
            assert vals is None
        # every byte of the cache: the new slots' and, untouched, all others
        assert torch.equal(back[0].cpu(), want_c) and torch.equal(back[1].cpu(), want_s)


@pytest.mark.parametrize("fmt,block", [("fp8", 128), ("fp8", 32), ("mxfp4", 32), ("nvfp4", 16),
                                       ("mxfp4", 8), ("fp8", 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_append_prompts(fmt, block, dtype):
    check_append([37, 1, 0, 130, 16], [37, 1, 0, 61, 3], 3, 128, 16, fmt, block, dtype)


@pytest.mark.parametrize("fmt,block,D", [("fp8", 20, 80), ("mxfp4", 6, 96), ("nvfp4", 10, 40),
                                         ("fp8", 1, 7), ("fp8", 256, 256), ("mxfp4", 512, 512)])
def test_append_odd_sizes(fmt, block, D):
    check_append([5, 19, 2], [2, 19, 1], 2, D, 7, fmt, block, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,block", [("fp8", 64), ("nvfp4", 16)])
def test_append_slices_of_a_projection_and_padding(fmt, block, dtype):
    check_append([9, 33], [1, 1], 2, 64, 16, fmt, block, dtype, pad=3, strided=True)
    check_append([9, 33], [4, 1], 1, 64, 16, fmt, block, dtype, pad=0, strided=True, with_v=False)


def test_append_one_row_and_many_sequences():
    check_append([1], [1], 1, 64, 16, "fp8", 64, torch.bfloat16)
    lens = [1 + (7 * i) % 50 for i in range(300)]
    check_append(lens, [i % 2 for i in range(300)], 1, 32, 16, "mxfp4", 32, torch.bfloat16)


def test_append_wide_rows_take_several_rounds_of_a_block():
    check_append([3, 2], [2, 1], 40, 128, 16, "nvfp4", 16, torch.bfloat16)


def test_append_leaves_out_what_is_out_of_range():
    H, D, S = 2, 64, 16
    for fault in ("page", "negative page", "length", "short", "offs", "offs end"):
        for block in (32, 4):  # the fast and the general kernel
            cache = ref.Cache([20, 30, 8], H, D, S, "fp8", block, empty=True)
            table, lengths = cache.table.clone(), cache.lengths.clone()
            offs = torch.tensor([2, 4, 6], dtype=torch.int32)
            hit = {1}
            if fault == "page":
                table[1, 1] = cache.P
            elif fault == "negative page":
                table[1, 1] = -1
            elif fault == "length":
                lengths[1] = cache.M * S + 1
            elif fault == "short":
                lengths[1] = 0  # shorter than its new rows
            elif fault == "offs":
                offs = torch.tensor([2, 1, 6], dtype=torch.int32)
                hit = {0, 1, 2}
            else:
                offs = torch.tensor([2, 4, 7], dtype=torch.int32)
                hit = {2}
            x = torch.randn(6, H, D).to(torch.bfloat16)
            codes, scales = ref.pack(x, "fp8", block)
            kc = dev(cache.k)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            mxq.append_cache_paged(dev(x), None, dev(offs), dev(table), dev(lengths), kc, None,
                                   "fp8", block, status=status)
            assert int(status) == (BAD_OFFS if "offs" in fault else BAD_PAGE), fault
            want = cache.k[0].clone()
            for b, (t0, t1) in enumerate(((0, 2), (2, 4), (4, 6))):
                if b in hit:
                    continue
                for t in range(t0, t1):
                    pos = int(cache.lens[b]) - (t1 - t)
                    want[table[b, pos // S], :, pos % S] = codes[t]
            got = kc[0].cpu()
            if fault != "offs":
                assert torch.equal(got, want), fault
            del scales


# ------------------------------------------------------------------ bounds

def as_f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("fmt,block,D,S", [("fp8", 128, 128, 64), ("mxfp4", 32, 64, 16),
                                           ("nvfp4", 16, 256, 32), ("fp8", 20, 80, 24),
                                           ("nvfp4", 6, 30, 5), ("mxfp4", 512, 512, 16),
                                           ("fp8", 8, 8, 1)])
def test_bounds_of_every_page_and_of_the_new_ones(fmt, block, D, S):
    lens = [3 * S + 1, 0, 1, 2 * S, S + max(0, S - 1)]
    cache = ref.Cache(lens, 3, D, S, fmt, block, seed=11)
    want = ref.bounds(cache)
    args = (dev(cache.k), dev(cache.table), dev(cache.lengths), fmt, block)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = as_f64(mxq.bound_cache_pages(*args, status=status))
    held = ~np.isnan(want)
    assert np.array_equal(got[held], want[held]) and not got[~held].any()
    for new in (1, S, S + 1, 10 ** 9):
        mark = torch.full((cache.P, 3, 2, D), 7.0, dtype=torch.bfloat16, device=DEV)
        assert mxq.bound_cache_pages(*args, mark, new_tokens=new, status=status) is mark
        expect = np.full(want.shape, 7.0)
        for b, x in enumerate(lens):
            for p in range(max(0, x - new) // S, -(-x // S)):
                expect[cache.table[b, p]] = want[cache.table[b, p]]
        assert np.array_equal(as_f64(mark), expect)
    assert int(status) == 0


def test_bounds_leave_out_bad_pages_and_lengths():
    cache = ref.Cache([40, 33], 2, 64, 16, "fp8", 64)
    table, lengths = cache.table.clone(), cache.lengths.clone()
    table[0, 1] = cache.P + 5
    lengths[1] = -3
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = as_f64(mxq.bound_cache_pages(dev(cache.k), dev(table), dev(lengths), "fp8", 64,
                                       status=status))
    want, full = np.zeros(got.shape), ref.bounds(cache)
    for p in (0, 2):
        want[cache.table[0, p]] = full[cache.table[0, p]]
    assert int(status) == BAD_PAGE and np.array_equal(got, want)


# ------------------------------------------------------------------ select

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,G,top,first,last", [(128, 4, 5, 1, 1), (64, 1, 1, 0, 1),
                                                (256, 3, 9, 2, 3), (30, 2, 4, 0, 0),
                                                (512, 1, 3, 0, 1), (6, 5, 40, 1, 1)])
def test_selected_pages_equal_the_plain_choice(dtype, D, G, top, first, last):
    S, H = 5, 2
    lens = [S * 37 + 2, 0, 3, S * top, S * top + 1, 90 * S]
    block = 6 if D % 8 else 8
    cache = ref.Cache(lens, H, D, S, "mxfp4", block if D % block == 0 else D, seed=D + top)
    q = queries(len(lens), G * H, D, dtype)
    bd = mxq.bound_cache_pages(dev(cache.k), dev(cache.table), dev(cache.lengths), "mxfp4",
                               cache.block)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = mxq.select_cache_pages(dev(q), bd, dev(cache.table), dev(cache.lengths), S, top,
                                 keep_first=first, keep_last=last, status=status)
    want = ref.select(cache, q, as_f64(bd), top, first, last)
    assert int(status) == 0 and np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n_pages,top", [(1000, 17), (1000, 999), (3000, 1), (257, 256), (5000, 700)])
def test_selection_among_many_pages_and_equal_scores(n_pages, top):
    # small whole numbers: exact sums, and many pages of one score
    g = torch.Generator().manual_seed(n_pages + top)
    H, D = 2, 8
    bd = torch.randint(-2, 3, (n_pages, H, 2, D), generator=g)
    bd = torch.sort(bd, dim=2).values.to(torch.bfloat16)
    table = torch.randperm(n_pages, generator=g).int()[None]
    q = torch.randint(-1, 2, (1, 2 * H, D), generator=g).to(torch.bfloat16)
    got = mxq.select_cache_pages(dev(q), dev(bd), dev(table), dev(torch.tensor([n_pages * 4]).int()),
                                 4, top, keep_first=0, keep_last=1)
    for h in range(H):
        qh = q[0, 2 * h:2 * h + 2].double()
        r = bd[table[0].long(), h].double()
        score = torch.maximum(qh[:, None] * r[None, :, 0], qh[:, None] * r[None, :, 1]).sum((0, 2))
        score[-1] = math.inf
        order = sorted(range(n_pages), key=lambda p: (-float(score[p]), p))[:top]
        assert got[0, h].tolist() == sorted(order)


def test_selection_at_zeros_and_a_full_table():
    # zero queries: every score is a zero, of either sign; the first pages win
    cache = ref.Cache([16 * 12], 1, 64, 16, "fp8", 64)
    bd = mxq.bound_cache_pages(dev(cache.k), dev(cache.table), dev(cache.lengths), "fp8", 64)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    q[0, 1] = -0.0
    got = mxq.select_cache_pages(dev(q), bd, dev(cache.table), dev(cache.lengths), 16, 4,
                                 keep_first=0, keep_last=1)
    assert got.tolist() == [[[0, 1, 2, 11]]]


def test_selection_passes_over_bad_pages_and_lengths():
    cache = ref.Cache([16 * 9, 16 * 9, 20], 1, 64, 16, "fp8", 64)
    table, lengths = cache.table.clone(), cache.lengths.clone()
    bd = mxq.bound_cache_pages(dev(cache.k), dev(table), dev(lengths), "fp8", 64)
    table[0, 3] = cache.P
    lengths[1] = cache.M * 16 + 1
    q = queries(3, 2, 64, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = mxq.select_cache_pages(dev(q), bd, dev(table), dev(lengths), 16, 8, status=status)
    assert int(status) == BAD_PAGE
    assert got[0, 0].tolist() == [0, 1, 2, 4, 5, 6, 7, 8]  # the bad page scores least
    assert got[1, 0].tolist() == [-1] * 8 and got[2, 0].tolist() == [0, 1] + [-1] * 6


# --------------------------------------------------------------- attention

def check_attend(cache, q, **kw):
    args = dict(kw)
    pages = args.pop("pages", None)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(cache.table),
                                      dev(cache.lengths), cache.fmt, cache.block,
                                      pages=None if pages is None else dev(pages), return_lse=True,
                                      status=status, **args)
    assert int(status) == 0
    want, wl, spread, reach = ref.attend(cache, q, pages=pages, **args)
    N, D = max(cache.lens + [1]), cache.D
    assert out.dtype == q.dtype and lse.dtype == torch.float32
    got, gl = as_f64(out), as_f64(lse)
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl)) and not np.isnan(got).any()
    fin = np.isfinite(wl)
    tol = ref.lse_tolerance(D, N, wl, reach)
    far = np.abs(np.where(fin, gl, 0.0) - np.where(fin, wl, 0.0))
    assert (far <= tol).all(), np.max(far / tol)
    tol = ref.out_tolerance(q.dtype, D, N, want, spread, reach)
    # a result beyond the dtype's largest value is an infinity of its sign
    most = torch.finfo(q.dtype).max
    over = np.isinf(got)
    assert (np.abs(want)[over] + tol[over] >= most).all()
    assert (np.sign(got[over]) == np.sign(want[over])).all()
    assert (np.abs(want)[~over] - tol[~over] <= most).all()
    assert (np.abs(got - want)[~over] <= tol[~over]).all(), np.max((np.abs(got - want) / tol)[~over])
    return out, lse


FORMATS = [("fp8", None), ("fp8", 32), ("mxfp4", 32), ("nvfp4", 16)]


@pytest.mark.parametrize("fmt,block", FORMATS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_ragged(fmt, block, D, dtype):
    lens = [97, 0, 1, 16, 15, 17, 640, 129, 128]
    cache = ref.Cache(lens, 2, D, 32, fmt, block or D, seed=D)
    check_attend(cache, queries(len(lens), 8, D, dtype))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("fmt,block", [("fp8", 128), ("mxfp4", 32)])
def test_attend_head_groups(G, fmt, block):
    cache = ref.Cache([50, 300, 7], 3, 128, 16, fmt, block, seed=G)
    check_attend(cache, queries(3, 3 * G, 128, torch.bfloat16))


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("G", [12, 16])
def test_attend_wide_groups_of_other_head_sizes(D, G):
    cache = ref.Cache([200, 33], 1, D, 16, "nvfp4", 16, seed=G)
    check_attend(cache, queries(2, G, D, torch.float16))


@pytest.mark.parametrize("fmt,block,D,S", [("mxfp4", 20, 80, 24), ("fp8", 1, 7, 3),
                                           ("nvfp4", 2, 34, 1), ("fp8", 16, 128, 16),
                                           ("nvfp4", 8, 64, 16), ("fp8", 64, 512, 16),
                                           ("mxfp4", 32, 96, 16), ("nvfp4", 16, 128, 40),
                                           ("mxfp4", 64, 128, 16), ("fp8", 128, 256, 48),
                                           ("nvfp4", 128, 128, 16), ("mxfp4", 256, 256, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attend_other_sizes(fmt, block, D, S, dtype):
    cache = ref.Cache([70, 1, 0, 133], 2, D, S, fmt, block, seed=D)
    check_attend(cache, queries(4, 6, D, dtype))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,block", FORMATS)
def test_attend_f32(fmt, block, D):
    cache = ref.Cache([500, 33, 0, 1], 2, D, 16, fmt, block or D, seed=D + 1)
    check_attend(cache, queries(4, 10, D, torch.float32))


@pytest.mark.parametrize("window", [1, 7, 16, 100, 128, 5000])
@pytest.mark.parametrize("S", [16, 64, 10])
def test_attend_window(window, S):
    cache = ref.Cache([300, 5, 0, 128, 1], 2, 64, S, "fp8", 64, seed=window)
    check_attend(cache, queries(5, 4, 64, torch.bfloat16), window=window)


def test_attend_window_over_freed_pages():
    # what lies before the window is gone: its pages are freed (entries out of
    # range) and the slots before it hold NaN bytes
    cache = ref.Cache([301], 1, 128, 32, "fp8", 128)
    q = queries(1, 4, 128, torch.bfloat16)
    start = 301 - 50
    k, v = [tuple(t.clone() for t in x) for x in (cache.k, cache.v)]
    page = int(cache.table[0, start // 32])
    for codes, scales in (k, v):
        codes[page, :, :start % 32] = 0x7F
        scales[page, :, :start % 32] = 0xFF
    table = cache.table.clone()
    table[0, :start // 32] = -1
    want = check_attend(cache, q, window=50)[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = mxq.attend_cache_paged(dev(q), dev(k), dev(v), dev(table), dev(cache.lengths), "fp8", 128,
                                 window=50, status=status)
    assert int(status) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("S", [16, 10])
def test_attend_window_reads_no_table_entry_before_it(S):
    # the entries of pages that lie before the window are out of range: they
    # are neither read nor reported, with and without a list that names them
    cache = ref.Cache([207], 1, 64, S, "fp8", 64)
    q = queries(1, 2, 64, torch.bfloat16)
    pages = torch.arange(21, dtype=torch.int32).expand(1, 1, 21).contiguous()
    for window in (1, S, 33, 34, 64, 90):
        table = cache.table.clone()
        table[0, :(207 - window) // S] = -1
        for listed in (None, pages):
            want = check_attend(cache, q, window=window, pages=listed)[0]
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            got = mxq.attend_cache_paged(dev(q), dev(cache.k), dev(cache.v), dev(table),
                                         dev(cache.lengths), "fp8", 64, window=window,
                                         pages=None if listed is None else dev(listed),
                                         status=status)
            assert int(status) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("S,fmt,block", [(16, "fp8", 128), (64, "mxfp4", 32), (24, "nvfp4", 16)])
def test_attend_listed_pages(S, fmt, block):
    H, D = 2, 128
    lens = [S * 9 + 3, 0, 5, S * 4]
    cache = ref.Cache(lens, H, D, S, fmt, block, seed=S)
    q = queries(4, 6, D, torch.bfloat16)
    pages = torch.full((4, H, 6), -1, dtype=torch.int32)
    pages[0, 0] = torch.tensor([0, 3, 4, 7, 9, -1])
    pages[0, 1] = torch.tensor([9, 9, 2, -5, 2, 10])  # in any order, twice, behind the end
    pages[1, 0, 0] = 0
    pages[2, 1, 3] = 0
    pages[3] = torch.tensor([3, 2, 1, 0, 4, 2 ** 31 - 1])
    check_attend(cache, q, pages=pages)
    check_attend(cache, q, pages=pages, window=S + 1)
    check_attend(cache, q, pages=pages[:, :, :1].contiguous())


def test_attend_scales_and_shared_pages():
    # K and V one buffer (a latent cache), a prefix page shared by sequences
    cache = ref.Cache([100, 90], 1, 64, 16, "fp8", 64, same=True)
    cache.table[1, 0] = cache.table[0, 0]
    for scale in (1.0, 0.0, -0.3, 4.0):
        check_attend(cache, queries(2, 4, 64, torch.bfloat16), scale=scale)


def test_attend_large_and_tiny_magnitudes():
    # logits of hundreds, values over forty binary orders between tokens
    for fmt, block in FORMATS[:3]:
        cache = ref.Cache([400, 60], 2, 64, 16, fmt, block or 64, seed=9)
        k, v = cache.k, cache.v
        k[1][:] = torch.where(k[1] == 0xFF, k[1], k[1] + 3)
        r = torch.randint(-20, 21, v[1].shape[:3] + (1,), generator=torch.Generator().manual_seed(2))
        v[1][:] = torch.where(v[1] == 0xFF, v[1], (v[1].int() + r).to(torch.uint8))
        check_attend(cache, queries(2, 4, 64, torch.bfloat16))
        check_attend(cache, queries(2, 4, 64, torch.float16) * 8, scale=1.0)


def test_attend_an_outlier_that_is_not_attended_to():
    # one token's values are 2^60 times the others', its weight 2^-200
    for fmt, block in FORMATS[:3]:
        cache = ref.Cache([80], 1, 64, 16, fmt, block or 64, seed=4)
        page = int(cache.table[0, 2])
        cache.v[1][page, 0, 5] += 60
        q = queries(1, 2, 64, torch.bfloat16)
        kv = torch.from_numpy(cache.values(cache.k, 0, 0))
        d = q[0].double().mean(0)
        row = (-d * 4000 / d.norm() ** 2).to(torch.bfloat16).view(1, 1, 1, 64)
        codes, scales = ref.pack(row, fmt, cache.block)
        cache.k[0][page, 0, 5], cache.k[1][page, 0, 5] = codes[0, 0, 0], scales[0, 0, 0]
        z = torch.from_numpy(cache.values(cache.k, 0, 0)) @ q[0].double().T
        assert (z[2 * 16 + 5] < z.max(0).values - 200).all() and kv.shape == (80, 64)
        check_attend(cache, q, scale=1.0)


def test_attend_one_long_sequence_is_split_and_joined():
    lens = [20011]
    cache = ref.Cache(lens, 1, 128, 128, "fp8", 128, seed=6)
    out, _ = check_attend(cache, queries(1, 4, 128, torch.bfloat16))
    again, _ = check_attend(cache, queries(1, 4, 128, torch.bfloat16))
    assert torch.equal(out, again)  # the split's order is fixed


def test_attend_many_short_sequences():
    lens = [(37 * i) % 90 for i in range(700)]
    cache = ref.Cache(lens, 1, 64, 16, "mxfp4", 32, seed=8)
    check_attend(cache, queries(700, 2, 64, torch.bfloat16))


def test_attend_strided_queries_and_given_buffers():
    cache = ref.Cache([70, 3], 2, 64, 16, "nvfp4", 16)
    wide = queries(2, 12, 64, torch.bfloat16)
    q = wide[:, 3:7]
    want, _ = check_attend(cache, q.contiguous())
    out = torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(16 << 20, dtype=torch.uint8, device=DEV)
    args = (dev(cache.k), dev(cache.v), dev(cache.table), dev(cache.lengths), "nvfp4", 16)
    got = mxq.attend_cache_paged(dev(wide)[:, 3:7], *args, out=out, workspace=ws)
    assert got is out and torch.equal(got, want)
    host = mxq.attend_cache_paged(q, *args)  # queries on the host
    assert not host.is_cuda and torch.equal(host, want.cpu())


def test_attend_leaves_out_bad_pages_and_lengths():
    for D, S in ((64, 16), (40, 10)):  # the tensor-core and the general kernel
        cache = ref.Cache([3 * S, 2 * S + 1, 9], 1, D, S, "fp8", D)
        q = queries(3, 2, D, torch.bfloat16)
        args = (dev(q), dev(cache.k), dev(cache.v))
        table, lengths = cache.table.clone(), cache.lengths.clone()
        for bad in (cache.P, -1):
            table[0, 1] = bad
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            got = mxq.attend_cache_paged(*args, dev(table), dev(lengths), "fp8", D, status=status)
            assert int(status) == BAD_PAGE
            pages = torch.tensor([[[0, 2, -1]], [[0, 1, 2]], [[0, -1, -1]]], dtype=torch.int32)
            want, wl, spread, reach = ref.attend(cache, q, pages=pages)
            tol = ref.out_tolerance(q.dtype, D, 3 * S, want, spread, reach)
            assert (np.abs(as_f64(got) - want) <= tol).all()
        for bad in (-1, cache.M * S + 1):
            lengths[2] = bad
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            got, lse = mxq.attend_cache_paged(*args, dev(cache.table), dev(lengths), "fp8", D,
                                              return_lse=True, status=status)
            assert int(status) == BAD_PAGE
            assert not got[2].any() and torch.isneginf(lse[2]).all()
            assert torch.isfinite(lse[:2]).all()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt,block,D,S", [("fp8", 128, 128, 16), ("mxfp4", 32, 64, 32),
                                           ("nvfp4", 16, 256, 16), ("fp8", 12, 36, 7)])
def test_a_serving_loop(fmt, block, D, S):
    """Prompts, then steps: append, bounds, selection, attention (over all, the
    selected and a window's tokens), each step against the plain form."""
    H, G, n, steps, top = 2, 3, 3, 4, 4
    start = [5 * S + 2, 1, 9 * S]
    lens = [x + steps for x in start]
    cache = ref.Cache(lens, H, D, S, fmt, block, empty=True, seed=21)
    kc, vc, table = dev(cache.k), dev(cache.v), dev(cache.table)
    bd = torch.zeros(cache.P, H, 2, D, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(77)
    for step in range(steps + 1):
        now = [x + step for x in start]
        new = start if step == 0 else [1] * n
        lengths = torch.tensor(now, dtype=torch.int32, device=DEV)
        offs = torch.tensor(np.cumsum(new), dtype=torch.int32, device=DEV)
        kv = torch.randn(2, sum(new), H, D, generator=g).to(torch.bfloat16).to(DEV)
        q = queries(n, G * H, D, torch.bfloat16, seed=step)
        mxq.append_cache_paged(kv[0], kv[1], offs, table, lengths, kc, vc, fmt, block,
                               status=status)
        mxq.bound_cache_pages(kc, table, lengths, fmt, block, bd, new_tokens=max(new),
                              status=status)
        pages = mxq.select_cache_pages(dev(q), bd, table, lengths, S, top, keep_first=1,
                                       status=status)
        cache.lens, cache.lengths = now, lengths.cpu()
        cache.k, cache.v = tuple(t.cpu() for t in kc), tuple(t.cpu() for t in vc)
        want = ref.bounds(cache)
        held = ~np.isnan(want)
        assert np.array_equal(as_f64(bd)[held], want[held])
        assert np.array_equal(pages.cpu().numpy(), ref.select(cache, q, as_f64(bd), top, 1, 1))
        check_attend(cache, q)
        check_attend(cache, q, pages=pages.cpu())
        check_attend(cache, q, window=S + 1)
    assert int(status) == 0


def test_a_captured_step_replays():
    """One step captured into a graph and replayed with new inputs in its
    buffers gives what the eager calls give; the second graph shares nothing."""
    fmt, block, H, G, D, S, n = "fp8", 128, 2, 4, 128, 16, 3
    cache = ref.Cache([60, 33, 100], H, D, S, fmt, block, empty=True)
    start = [50, 20, 90]
    torch.cuda.synchronize()

    class Step:
        def __init__(self):
            self.kc, self.vc, self.table = dev(cache.k), dev(cache.v), dev(cache.table)
            self.lengths = torch.tensor(start, dtype=torch.int32, device=DEV)
            self.offs = torch.arange(1, n + 1, dtype=torch.int32, device=DEV)
            self.k = torch.zeros(n, H, D, dtype=torch.bfloat16, device=DEV)
            self.v, self.q = torch.zeros_like(self.k), queries(n, H * G, D, torch.bfloat16).to(DEV)
            self.bd = torch.zeros(cache.P, H, 2, D, dtype=torch.bfloat16, device=DEV)
            prompt = torch.randn(2, sum(start), H, D, generator=torch.Generator().manual_seed(1))
            prompt = prompt.to(torch.bfloat16).to(DEV)
            mxq.append_cache_paged(prompt[0], prompt[1], torch.tensor(
                np.cumsum(start), dtype=torch.int32, device=DEV), self.table, self.lengths, self.kc,
                self.vc, fmt, block)
            mxq.bound_cache_pages(self.kc, self.table, self.lengths, fmt, block, self.bd)

        def run(self):
            self.lengths += 1
            mxq.append_cache_paged(self.k, self.v, self.offs, self.table, self.lengths, self.kc,
                                   self.vc, fmt, block)
            mxq.bound_cache_pages(self.kc, self.table, self.lengths, fmt, block, self.bd,
                                  new_tokens=1)
            pages = mxq.select_cache_pages(self.q, self.bd, self.table, self.lengths, S, 3)
            full = mxq.attend_cache_paged(self.q, self.kc, self.vc, self.table, self.lengths, fmt,
                                          block)
            part = mxq.attend_cache_paged(self.q, self.kc, self.vc, self.table, self.lengths, fmt,
                                          block, pages=pages)
            return pages, full, part

    eager, graphed = Step(), Step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.run()  # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    eager.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = graphed.run()
    graphed.lengths.copy_(eager.lengths)
    for i in range(3):
        x = torch.randn(2, n, H, D, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        for s in (eager, graphed):
            s.k.copy_(x[0])
            s.v.copy_(x[1])
            s.q.copy_(queries(n, H * G, D, torch.bfloat16, seed=i))
        want = eager.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    # each call has its own workspace: calls on two streams do not meet
    cache = ref.Cache([4000, 100], 2, 64, 16, "mxfp4", 32)
    qs = [queries(2, 8, 64, torch.bfloat16, seed=i) for i in range(6)]
    args = (dev(cache.k), dev(cache.v), dev(cache.table), dev(cache.lengths), "mxfp4", 32)
    dq = [dev(q) for q in qs]
    want = [mxq.attend_cache_paged(q, *args) for q in dq]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i, q in enumerate(dq):
        with torch.cuda.stream(streams[i % 3]):
            got.append(mxq.attend_cache_paged(q, *args))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_debug_variant_without_a_failed_check():
    """The cases above on the library's debug variant, whose kernels check
    every index (tests/conftest.py asks for its record after each)."""
    import os
    import subprocess
    import sys

    from nvfp4_quantization_amax_b200 import build

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, MXQ_LIBRARY=build.build(debug=True), MXQ_EXPECT_CLEAN_CHECKS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        "-k", "not debug_variant", os.path.abspath(__file__)],
                       cwd=root, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-1000:]


def test_odd_row_starts_of_scales_and_codes():
    # slices of larger buffers: pages that begin off every 16-byte boundary take
    # the general kernels, with the same results
    cache = ref.Cache([70, 9], 2, 64, 16, "mxfp4", 32)
    q = queries(2, 4, 64, torch.bfloat16)
    want, _ = check_attend(cache, q)

    def shifted(pair, by):
        out = []
        for t in pair:
            flat = torch.full((t.numel() + by,), 0xFF, dtype=torch.uint8, device=DEV)
            flat[by:] = t.reshape(-1).to(DEV)
            out.append(flat[by:].view(t.shape))
        return tuple(out)

    table, lengths = dev(cache.table), dev(cache.lengths)
    for by in (1, 2, 4, 8):
        k, v = shifted(cache.k, by), shifted(cache.v, by)
        got = mxq.attend_cache_paged(dev(q), k, v, table, lengths, "mxfp4", 32)
        o, _, spread, reach = ref.attend(cache, q)
        tol = ref.out_tolerance(q.dtype, 64, 70, o, spread, reach)
        assert (np.abs(as_f64(got) - o) <= tol).all()
        assert torch.equal(mxq.bound_cache_pages(k, table, lengths, "mxfp4", 32),
                           mxq.bound_cache_pages(dev(cache.k), table, lengths, "mxfp4", 32))
        x = torch.randn(3, 2, 64, dtype=torch.bfloat16, device=DEV)
        offs = torch.tensor([2, 3], dtype=torch.int32, device=DEV)
        mxq.append_cache_paged(x, None, offs, table, lengths, k, None, "mxfp4", 32)
        whole = dev(cache.k)
        mxq.append_cache_paged(x, None, offs, table, lengths, whole, None, "mxfp4", 32)
        assert torch.equal(k[0], whole[0]) and torch.equal(k[1], whole[1])
    assert want.shape == q.shape


def test_calls_without_rows_or_sequences():
    cache = ref.Cache([20], 2, 64, 16, "fp8", 64)
    k, v = dev(cache.k), dev(cache.v)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    out, lse = mxq.attend_cache_paged(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV), k, v,
                                      table, none, "fp8", 64, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    got = mxq.append_cache_paged(x, x, torch.zeros(1, dtype=torch.int32, device=DEV),
                                 dev(cache.table), dev(cache.lengths), k, v, "fp8", 64, values=True)
    assert got[0].shape == (0, 2, 64)
    assert torch.equal(k[0].cpu(), cache.k[0])
    bd = mxq.bound_cache_pages(k, table, none, "fp8", 64)
    assert not bd.any()
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert mxq.select_cache_pages(q, bd, table, none, 16, 3).shape == (0, 2, 3)

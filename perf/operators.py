"""Cases that measure the paged packed cache: append, page bounds, page
selection and the attention of one new token.

Each case is one call (or, for the sparse ones, the two calls that belong
together) as a serving loop makes it.  `run` computes it in elementary torch
operations, or, where `own` is true, with this package's kernels.

The cache of K (and of V) is a pair (codes, scales): codes uint8
[pages, kv_heads, page_size, D] (fp8) or [..., D/2] (mxfp4, nvfp4: the even
channel in the low nibble), scales uint8 [pages, kv_heads, page_size, D/block]
(E8M0 bytes for fp8 and mxfp4, E4M3 bytes for nvfp4).  page_table [sequences,
max_pages] lists each sequence's pages, lengths its tokens.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
QMAX = {"fp8": (0.875, 9), "mxfp4": (0.75, 3), "nvfp4": (0.75, 3)}  # fraction, exponent
CLAMP = {"fp8": (-126, 127), "mxfp4": (-126, 127), "nvfp4": (-9, 8)}


def case(name, kind, n, tokens, heads, group, dim, page, fmt, block, dtype="bf16", ragged=True,
         window=0, top=0, first=0, last=1, new=1):
    """n sequences of up to `tokens` tokens; heads kv heads, each read by
    `group` query heads of `dim` channels; pages of `page` tokens in `fmt`
    with one scale per `block` channels; window 0: no window."""
    return {"name": name, "kind": kind, "n": n, "tokens": tokens, "heads": heads, "group": group,
            "dim": dim, "page": page, "fmt": fmt, "block": block, "dtype": dtype, "ragged": ragged,
            "window": window, "top": top, "first": first, "last": last, "new": new}


def listed():
    return [
        # one decode step's write of 64 sequences: latency
        case("append_step_64", "append", 64, 200, 8, 1, 128, 64, "fp8", 128, new=1),
        # prompts of 512 channels (4 heads of 128) entering the cache, ragged
        case("append_prompts_mxfp4", "append", 8, 6000, 4, 1, 128, 64, "mxfp4", 32, new=6000),
        # the bounds of the page that a step has written to
        case("bounds_step_48", "bounds", 48, 3000, 8, 1, 128, 64, "nvfp4", 16, dtype="bf16", new=1),
        # the bounds of every page of long prompts
        case("bounds_prompts_fp8", "bounds", 4, 65536, 8, 1, 128, 64, "fp8", 128, new=0),
        # the smallest call: one short sequence, latency counts
        case("attend_1_short", "attend", 1, 97, 8, 4, 128, 16, "fp8", 128, ragged=False),
        # an ordinary batch of ragged sequences, one of them empty
        case("attend_32_ragged", "attend", 32, 8192, 8, 4, 128, 64, "fp8", 32),
        # the cache workload of 8192 tokens of 512 channels, many sequences
        case("attend_96_mxfp4", "attend", 96, 8192, 4, 8, 128, 64, "mxfp4", 32, ragged=False),
        # one very long sequence: the split over the length carries it
        case("attend_1_long", "attend", 1, 131071, 8, 8, 128, 128, "nvfp4", 16, ragged=False),
        # a sliding window, wide heads, f16
        case("attend_16_window", "attend", 16, 20000, 2, 8, 256, 32, "fp8", 64, dtype="f16",
             window=5001),
        # odd sizes and f32: heads of 80 channels, pages of 24 tokens, blocks of 20
        case("attend_5_odd_f32", "attend", 5, 3001, 3, 5, 80, 24, "mxfp4", 20, dtype="f32"),
        # 64 of 2048 pages of one long sequence
        case("sparse_1_long", "sparse", 1, 131072, 8, 4, 128, 64, "fp8", 128, ragged=False, top=64,
             first=1),
        # long ragged sequences in a batch, 32 pages each
        case("sparse_24_ragged", "sparse", 24, 32768, 8, 4, 128, 64, "mxfp4", 32, top=32, first=1,
             last=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "bounds", "attend", "attend", "attend", "sparse", "sparse"])
    dim = rng.choice([64, 128, 128, 128, 256, 96])
    fmt = rng.choice(["fp8", "mxfp4", "nvfp4"])
    block = {"fp8": rng.choice([dim, 32]), "mxfp4": 32, "nvfp4": 16}[fmt]
    heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16]) if kind in ("attend", "sparse") else 1
    page = rng.choice([16, 32, 64, 64, 128, 40])
    n = _log(rng, 1, 96)
    most = (96 * 8192 * 512) // (n * heads * dim)
    tokens = _log(rng, 1, min(100000, most))
    new = 1
    if kind == "append":
        new = rng.choice([1, 1, 3, tokens])
        most = (8 * 6000 * 512) // (n * heads * dim)  # as much as the largest listed append
        new = max(1, min(new, most))
    if kind == "bounds":
        tokens = max(1, min(tokens, (4 * 65536 * 1024) // (n * heads * dim)))
        new = rng.choice([0, 1])
    if kind == "sparse":
        tokens = max(tokens, min(most, 20 * page))
    window = _log(rng, 1, tokens) if kind == "attend" and rng.random() < 0.25 else 0
    top = _log(rng, 2, 64) if kind == "sparse" else 0
    return {k: v for k, v in case("", kind, n, tokens, heads, group, dim, page, fmt, block,
                                  dtype=rng.choice(["bf16", "bf16", "f16"]),
                                  ragged=rng.random() < 0.7, window=window, top=top,
                                  first=1 if kind == "sparse" and rng.random() < 0.5 else 0,
                                  new=new).items() if k != "name"}


# ------------------------------------------------------------------ sizes

def sizes(c):
    """(lengths, new rows) of the case's sequences: plain integers that follow
    from the case alone."""
    rng = random.Random(c["n"] * 1000003 + c["tokens"])
    lens = [c["tokens"]] * c["n"]
    if c["ragged"]:
        lens = [rng.randint(1, c["tokens"]) for _ in range(c["n"])]
        lens[0] = c["tokens"]
        if c["n"] > 3 and c["kind"] == "attend":
            lens[2] = 0
            lens[3] = 1
    new = [min(x, c["new"]) for x in lens] if c["new"] else lens
    return lens, new


def code_bytes(c):
    return c["dim"] if c["fmt"] == "fp8" else c["dim"] // 2


# ----------------------------------------------------------- the plain form

def pow2(k):
    """2^k in f32 for whole k in [-127, 127], from its bits."""
    return torch.where(k < -126, 1 << 22, (k + 127) << 23).int().view(torch.float32)


def plain_pack(x, fmt, block):
    """(codes, scale bytes, values) of x [..., D]; the values in f32."""
    g = x.float().unflatten(-1, (-1, block))
    frac, e = torch.frexp(g.abs().amax(-1, keepdim=True))
    f, q = QMAX[fmt]
    lo, hi = CLAMP[fmt]
    k = (e - q + (frac > f).to(e.dtype)).clamp(lo, hi)
    k = torch.where(frac == 0, torch.full_like(k, lo), k)
    y = g * pow2(-k)
    if fmt == "fp8":
        y8 = y.flatten(-2).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes, back = y8.view(torch.uint8), y8.float().unflatten(-1, (-1, block))
    else:
        a = y.abs()
        mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
               + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
        back = torch.tensor(E2M1, device=x.device)[mag.int()] * torch.where(g < 0, -1.0, 1.0)
        back = back + 0.0
        nib = (mag | ((g < 0).to(torch.uint8) << 3)).flatten(-2)
        codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    k = k.squeeze(-1)
    if fmt == "nvfp4":
        scales = pow2(k).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        scales = (k + 127).to(torch.uint8)
    return codes, scales, (back * pow2(k).unsqueeze(-1)).flatten(-2)


def plain_values(codes, scales, fmt, block):
    """f32 values [..., D] of codes and scale bytes."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
        table[8] = 0.0
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else pow2(scales.int() - 127)
    return (v.unflatten(-1, (-1, block)) * s.unsqueeze(-1)).flatten(-2)


def plain_append(s):
    c = s["case"]
    k, v, offs, lens = s["k"], s["v"], s["offs"].long(), s["lengths"].long()
    rows = torch.arange(k.shape[0], device=k.device)
    b = torch.searchsorted(offs, rows, right=True)
    pos = lens[b] - (offs[b] - rows)
    page, slot = s["page_table"].long()[b, pos // c["page"]], pos % c["page"]
    both = torch.stack((k, v), 1)  # [T, 2, H, D]
    codes, scales, val = plain_pack(both, c["fmt"], c["block"])
    s["k_cache"][0][page, :, slot] = codes[:, 0]
    s["k_cache"][1][page, :, slot] = scales[:, 0]
    s["v_cache"][0][page, :, slot] = codes[:, 1]
    s["v_cache"][1][page, :, slot] = scales[:, 1]
    return val.to(k.dtype).unbind(1)


def plain_bounds(s):
    c, P = s["case"], s["page_table"].long()
    S, lens = c["page"], s["lengths"].long()
    n_pages = (lens + S - 1) // S
    first = ((lens - c["new"]).clamp(min=0) // S) if c["new"] else torch.zeros_like(lens)
    m = s["most_new_pages"]
    idx = first[:, None] + torch.arange(m, device=lens.device)
    valid = idx < n_pages[:, None]
    b, j = valid.nonzero(as_tuple=True)
    logical = idx[b, j]
    phys = P[b, logical]
    codes, scales = s["k_cache"]
    val = plain_values(codes[phys], scales[phys], c["fmt"], c["block"])  # [n, H, S, D]
    pos = logical[:, None] * S + torch.arange(S, device=lens.device)
    dead = (pos >= lens[b][:, None])[:, None, :, None]
    lo = val.masked_fill(dead, math.inf).amin(2)
    hi = val.masked_fill(dead, -math.inf).amax(2)
    s["bounds"][phys] = torch.stack((lo, hi), 2).to(torch.bfloat16)
    return s["bounds"]


def plain_select(s):
    """Logical pages [n, H, top] with the largest upper bounds of the query
    group's summed logits, ascending, -1 behind."""
    c, P = s["case"], s["page_table"].long()
    H, S, M = c["heads"], c["page"], s["page_table"].shape[1]
    n_pages = ((s["lengths"].long() + S - 1) // S)[:, None, None]
    q = s["q"].double().unflatten(1, (H, -1))
    bd = s["bounds"][P.clamp(0, s["bounds"].shape[0] - 1)].double()  # [n, M, H, 2, D]
    score = (torch.einsum("bhd,bmhd->bhm", q.clamp(max=0).sum(2), bd[:, :, :, 0])
             + torch.einsum("bhd,bmhd->bhm", q.clamp(min=0).sum(2), bd[:, :, :, 1]))
    at = torch.arange(M, device=q.device)
    score = score.masked_fill((at < c["first"]) | (at >= n_pages - c["last"]), math.inf)
    score = score.masked_fill(at >= n_pages, -math.inf)
    top = min(c["top"], M)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    best = torch.where(torch.arange(top, device=q.device) < n_pages, best, M)
    best = torch.sort(best, -1).values
    best = torch.where(best == M, -1, best)
    return torch.nn.functional.pad(best, (0, c["top"] - top), value=-1).int()


def plain_attend(s, pages=None):
    c, H, S = s["case"], s["case"]["heads"], s["case"]["page"]
    P, lens = s["page_table"].long(), s["lengths"].long()
    n, M = P.shape
    if pages is None:
        pages = torch.arange(M, device=P.device).expand(n, H, M)
    pages = pages.long()
    phys = torch.gather(P[:, None].expand(n, H, M), 2, pages.clamp(min=0))
    phys = phys.clamp(0, s["k_cache"][0].shape[0] - 1)
    h = torch.arange(H, device=P.device)[:, None]
    q = s["q"].float().unflatten(1, (H, -1)) / math.sqrt(c["dim"])
    pos = pages[..., None] * S + torch.arange(S, device=P.device)  # [n, H, m, S]
    end = lens[:, None, None, None]
    live = (pages >= 0)[..., None] & (pos < end)
    if c["window"]:
        live &= pos >= end - c["window"]
    live = live.flatten(2)[:, :, None]
    codes, scales = s["k_cache"]
    k = plain_values(codes[phys, h], scales[phys, h], c["fmt"], c["block"]).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)).masked_fill(~live, -math.inf)
    del k
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m)).masked_fill(~live, 0.0)
    total = e.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1).flatten(1)
    codes, scales = s["v_cache"]
    v = plain_values(codes[phys, h], scales[phys, h], c["fmt"], c["block"]).flatten(2, 3)
    v = v.masked_fill(~live.transpose(2, 3), 0.0)
    out = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    return out.flatten(1, 2).to(s["q"].dtype), lse


# ------------------------------------------------------------- the interface

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    lens, new = sizes(c)
    n, H, D, S, dt = c["n"], c["heads"], c["dim"], c["page"], DTYPES[c["dtype"]]
    need = [-(-x // S) for x in lens]
    M = max(need + [1])
    total = sum(need) + 3  # a few free pages: the pool is never exactly full
    order = torch.randperm(total, generator=g, device=dev).int()
    starts = torch.tensor([sum(need[:i]) for i in range(n)], device=dev)
    at = torch.arange(M, device=dev)
    used = at < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, order[(starts[:, None] + at).clamp(max=total - 1)], -1).int()
    s = {"case": c, "page_table": table.contiguous(),
         "lengths": torch.tensor(lens, dtype=torch.int32, device=dev),
         "most_new_pages": max([1] + [-(-x // S) - max(0, x - (c["new"] or x)) // S for x in lens])}

    def values(shape):
        # channels of unequal size, a few large entries
        x = torch.randn(shape, generator=g, device=dev)
        x *= torch.exp2(4 * torch.rand(shape[-1], generator=g, device=dev) - 2.5)
        x *= torch.where(torch.rand(shape[:-1] + (1,), generator=g, device=dev) < 1e-3, 8.0, 1.0)
        return x

    def cache(empty):
        codes = torch.zeros(total, H, S, code_bytes(c), dtype=torch.uint8, device=dev)
        scales = torch.zeros(total, H, S, D // c["block"], dtype=torch.uint8, device=dev)
        if not empty:
            step = max(1, (1 << 26) // (H * S * D))
            for p in range(0, total, step):
                m = min(step, total - p)
                codes[p:p + m], scales[p:p + m], _ = plain_pack(values((m, H, S, D)), c["fmt"],
                                                                c["block"])
        return codes, scales

    s["k_cache"] = cache(c["kind"] == "append")
    s["v_cache"] = cache(c["kind"] == "append") if c["kind"] != "bounds" else None
    if c["kind"] == "append":
        T = sum(new)
        s["offs"] = torch.tensor([sum(new[:i + 1]) for i in range(n)], dtype=torch.int32,
                                 device=dev)
        s["k"] = values((T, H, D)).to(dt)
        s["v"] = values((T, H, D)).to(dt)
    if c["kind"] in ("attend", "sparse"):
        q = torch.randn((n, H * c["group"], D), generator=g, device=dev)
        s["q"] = (q * torch.exp2(2 * torch.rand((n, H * c["group"], 1), generator=g, device=dev)
                                 - 1)).to(dt)
    if c["kind"] in ("bounds", "sparse"):
        s["bounds"] = torch.zeros(total, H, 2, D, dtype=torch.bfloat16, device=dev)
    if c["kind"] == "sparse":  # a serving loop has them from the steps before
        step = max(1, (1 << 26) // (H * S * D))
        pos = torch.full((total,), S, device=dev)  # valid tokens of each page
        last = torch.tensor([max(0, x - 1) // S for x in lens], device=dev)
        full = torch.tensor(lens, device=dev) - last * S
        pos[table[torch.arange(n, device=dev), last].long()] = full
        for p in range(0, total, step):
            val = plain_values(s["k_cache"][0][p:p + step], s["k_cache"][1][p:p + step], c["fmt"],
                               c["block"])
            dead = (torch.arange(S, device=dev) >= pos[p:p + step, None])[:, None, :, None]
            s["bounds"][p:p + step, :, 0] = val.masked_fill(dead, math.inf).amin(2).bfloat16()
            s["bounds"][p:p + step, :, 1] = val.masked_fill(dead, -math.inf).amax(2).bfloat16()
    return s


def run(s):
    c = s["case"]
    if own:
        import nvfp4_quantization_amax_b200 as mxq

        fmt, block = c["fmt"], c["block"]
        if c["kind"] == "append":
            k, v = mxq.append_cache_paged(s["k"], s["v"], s["offs"], s["page_table"], s["lengths"],
                                          s["k_cache"], s["v_cache"], fmt, block, values=True)
            return [k, v, *s["k_cache"], *s["v_cache"]]
        if c["kind"] == "bounds":
            return mxq.bound_cache_pages(s["k_cache"], s["page_table"], s["lengths"], fmt, block,
                                         s["bounds"], new_tokens=c["new"] or None)
        if c["kind"] == "sparse":
            pages = mxq.select_cache_pages(s["q"], s["bounds"], s["page_table"], s["lengths"],
                                           c["page"], c["top"], keep_first=c["first"],
                                           keep_last=c["last"])
            out, lse = mxq.attend_cache_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                              s["lengths"], fmt, block, pages=pages,
                                              return_lse=True)
            return [pages, out, lse]
        return list(mxq.attend_cache_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                           s["lengths"], fmt, block, window=c["window"] or None,
                                           return_lse=True))
    if c["kind"] == "append":
        k, v = plain_append(s)
        # the cache's bytes are whole numbers, beside the values they stand for
        return [k, v, *s["k_cache"], *s["v_cache"]]
    if c["kind"] == "bounds":
        return plain_bounds(s)
    if c["kind"] == "sparse":
        pages = plain_select(s)
        return [pages, *plain_attend(s, pages)]
    return list(plain_attend(s))


def work(c):
    lens, new = sizes(c)
    H, D, S, G, e = c["heads"], c["dim"], c["page"], c["group"], DTYPES[c["dtype"]].itemsize
    row = H * (code_bytes(c) + D // c["block"])  # a token's codes and scales of K
    ints = 4 * c["n"]
    if c["kind"] == "append":
        T = sum(new)
        pages = sum(-(-x // S) - (x - y) // S for x, y in zip(lens, new))
        return {"bytes": 2 * T * (2 * H * D * e + row) + 2 * ints + 4 * pages,
                "flops": 4 * T * H * D}
    if c["kind"] == "bounds":
        part = [(x - y) // S for x, y in zip(lens, new)]  # whole pages are read again
        tokens = sum(x - p * S for x, p in zip(lens, part))
        pages = sum(-(-x // S) - p for x, p in zip(lens, part))
        return {"bytes": tokens * row + pages * (4 * H * D + 4) + ints, "flops": 3 * tokens * H * D}
    qo = c["n"] * H * G * (2 * D * e + 4)
    if c["kind"] == "sparse":
        pages = [-(-x // S) for x in lens]
        got = [min(c["top"], p) for p in pages]
        # whole pages but the last one, which holds what is left of the sequence
        tokens = sum(y * S - (p * S - x) for x, p, y in zip(lens, pages, got))
        return {"bytes": sum(pages) * (4 * H * D + 4) + 2 * tokens * row + qo + ints
                + c["n"] * H * c["top"] * 8,
                "flops": 4 * sum(pages) * H * D + 4 * tokens * H * G * D}
    tokens = [min(x, c["window"]) if c["window"] else x for x in lens]
    return {"bytes": 2 * sum(tokens) * row + 4 * sum(-(-x // S) for x in tokens) + qo + ints,
            "flops": 4 * sum(tokens) * H * G * D}


# ------------------------------------------------------- exact, in 64 bits

def grid_round(y, digits, low):
    """y to `digits` binary digits after the leading one, halves to even; the
    spacing does not shrink below the binade of 2^low."""
    _, e = torch.frexp(y)
    step = torch.exp2((torch.clamp(e - 1, min=low) - digits).double())
    return torch.round(y / step) * step


def byte_e4m3(b):
    b = b.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -mag, mag)


def exact_rows(codes, scales, c):
    """f64 values of cache rows from the formats' definitions."""
    if c["fmt"] == "fp8":
        v = byte_e4m3(codes)
    else:
        nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
        e, m = (nib >> 1) & 3, (nib & 1).double()
        mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
        v = torch.where(nib >= 8, -mag, mag)
    s = byte_e4m3(scales) if c["fmt"] == "nvfp4" else torch.exp2(scales.double() - 127)
    return v * s.repeat_interleave(c["block"], -1)


def exact_pages(s, lens):
    """Each (sequence, kv head)'s selected pages, in lists."""
    c, found = s["case"], []
    for b, x in enumerate(lens):
        m = -(-x // c["page"])
        bd = s["bounds"][s["page_table"][b, :m].long()].double()  # [m, H, 2, D]
        q = s["q"][b].double().unflatten(0, (c["heads"], -1))
        reach = torch.maximum(q * bd[:, :, None, 0], q * bd[:, :, None, 1]).sum((2, 3)).T.tolist()
        keep = set(range(m)[:c["first"]]) | set(range(max(0, m - c["last"]), m))
        found.append([sorted(sorted(range(m), key=lambda p: (p not in keep, -r[p], p))[:c["top"]])
                      for r in reach])
    return found


def exact(c, seed):
    s = prepare(c, seed)
    S, H, G = c["page"], c["heads"], c["group"]
    lens, new = sizes(c)
    if c["kind"] == "append":
        outs = []
        top = 448.0 if c["fmt"] == "fp8" else 6.0
        lo, hi = CLAMP[c["fmt"]]
        for x in (s["k"], s["v"]):
            g = x.double().unflatten(-1, (-1, c["block"]))
            ratio = g.abs().amax(-1, keepdim=True) / top
            k = torch.ceil(torch.log2(ratio.clamp(min=2.0 ** -200)))
            k = torch.where(torch.exp2(k - 1) >= ratio, k - 1, k)  # log2 is rounded: settle it
            k = torch.where(torch.exp2(k) < ratio, k + 1, k).clamp(lo, hi)
            y = grid_round(g * torch.exp2(-k), *((3, -6) if c["fmt"] == "fp8" else (1, 0)))
            outs.append((y.clamp(-top, top) * torch.exp2(k)).flatten(-2))
        return outs + [None] * 4
    if c["kind"] == "bounds":
        want = s["bounds"].double()
        for b, x in enumerate(lens):
            for p in range((x - new[b]) // S, -(-x // S)):
                at = int(s["page_table"][b, p])
                rows = min(S, x - p * S)
                v = exact_rows(s["k_cache"][0][at, :, :rows], s["k_cache"][1][at, :, :rows], c)
                want[at] = torch.stack((v.amin(1), v.amax(1)), 1)
        return want
    pages = exact_pages(s, lens) if c["kind"] == "sparse" else None
    out = torch.zeros(c["n"], H * G, c["dim"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["n"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    for b, x in enumerate(lens):
        if x == 0:
            continue
        every = list(range(-(-x // S)))
        for h in range(H):
            mine = every if pages is None else pages[b][h]
            at = s["page_table"][b, mine].long()
            pos = (torch.tensor(mine, device="cuda")[:, None] * S
                   + torch.arange(S, device="cuda")).flatten()
            keep = pos < x
            if c["window"]:
                keep &= pos >= x - c["window"]
            k = exact_rows(s["k_cache"][0][at, h].flatten(0, 1)[keep],
                           s["k_cache"][1][at, h].flatten(0, 1)[keep], c)
            v = exact_rows(s["v_cache"][0][at, h].flatten(0, 1)[keep],
                           s["v_cache"][1][at, h].flatten(0, 1)[keep], c)
            heads = slice(h * G, (h + 1) * G)
            z = s["q"][b, heads].double() @ k.T / math.sqrt(c["dim"])
            lse[b, heads] = torch.logsumexp(z, -1)
            out[b, heads] = torch.exp(z - lse[b, heads, None]) @ v
    return ([None] if pages is not None else []) + [out, lse]

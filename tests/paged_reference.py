"""Plain 64-bit implementation of the paged cache calls, for the tests: numpy
on top of the scalar oracle's pack and unpack."""
import math

import numpy as np
import torch

import oracle

BITS = {torch.bfloat16: (torch.int16, np.uint16, "bf16"),
        torch.float16: (torch.int16, np.uint16, "f16"),
        torch.float32: (torch.int32, np.uint32, "f32")}


def bits(t):
    as_int, as_np, _ = BITS[t.dtype]
    return t.detach().cpu().contiguous().view(as_int).numpy().view(as_np)


def pack(x, fmt, block):
    """(codes, scales) uint8 tensors of a CPU tensor [..., D] by the oracle."""
    lead, D = tuple(x.shape[:-1]), x.shape[-1]
    c, s = oracle.quantize_cache_packed(bits(x).reshape(-1, D), fmt, block, BITS[x.dtype][2])
    return (torch.from_numpy(np.ascontiguousarray(c, dtype=np.uint8)).view(*lead, -1),
            torch.from_numpy(np.ascontiguousarray(s, dtype=np.uint8)).view(*lead, -1))


def unpack(codes, scales, fmt, block):
    """float64 values [..., D]."""
    D = codes.shape[-1] * (1 if fmt == "fp8" else 2)
    w = oracle.dequantize_cache_packed(codes.reshape(-1, codes.shape[-1]).numpy(),
                                       scales.reshape(-1, scales.shape[-1]).numpy(), fmt, block, D,
                                       "f32")
    return np.asarray(w, dtype=np.uint32).view(np.float32).astype(np.float64).reshape(
        tuple(codes.shape[:-1]) + (D,))


class Cache:
    """K and V pages in `fmt` with the tables of sequences of the given
    lengths, on the CPU.  Everything that no sequence holds (free pages, slots
    behind the last token, unused table entries) is filled with bytes that
    decode to NaN or to the largest values."""

    def __init__(self, lens, H, D, S, fmt, block, seed=1, spare=2, same=False, spread=2.0,
                 empty=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.D, self.S, self.fmt, self.block = lens, H, D, S, fmt, block
        need = [-(-x // S) for x in lens]
        self.P, self.M = sum(need) + spare, max(need + [1]) + 1
        order = torch.randperm(self.P, generator=g).int()
        self.table = torch.full((len(lens), self.M), 2 ** 31 - 1, dtype=torch.int32)
        self.table[:, -1] = -7
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.lengths = torch.tensor(lens, dtype=torch.int32)
        rb = D if fmt == "fp8" else D // 2
        held = torch.zeros(self.P, S, dtype=torch.bool)
        for b, x in enumerate(lens):
            for p in range(need[b]):
                held[self.table[b, p], :min(S, x - p * S)] = True
        self.held = held
        out = []
        for _ in range(1 if same else 2):
            x = torch.randn(self.P, H, S, D, generator=g)
            x *= torch.exp2(spread * torch.rand(D, generator=g) - spread / 2)
            x = x.to(torch.bfloat16)
            codes, scales = pack(x, fmt, block)
            assert codes.shape[-1] == rb
            dead = ~held[:, None, :, None].expand(self.P, H, S, 1)
            if empty:
                dead = torch.ones_like(dead)
            codes = torch.where(dead, torch.tensor(0x7F, dtype=torch.uint8), codes)
            scales = torch.where(dead, torch.tensor(0xFF, dtype=torch.uint8), scales)
            out.append((codes.contiguous(), scales.contiguous()))
        self.k, self.v = out[0], out[-1]

    def values(self, which, b, h):
        """float64 [length, D] of one sequence and head."""
        codes, scales = which
        n = -(-self.lens[b] // self.S)
        if n == 0:
            return np.zeros((0, self.D))
        pages = self.table[b, :n].long()
        c = codes[pages, h].reshape(n * self.S, -1)[:self.lens[b]]
        s = scales[pages, h].reshape(n * self.S, -1)[:self.lens[b]]
        return unpack(c, s, self.fmt, self.block)


def attend(cache, q, scale=None, window=None, pages=None):
    """(out, lse, spread, reach) in float64: spread [n, Hq, D] = sum p |v|, the
    size of the terms of each output; reach [n, Hq] = the largest sum of a
    logit's terms' magnitudes (what its rounding error is relative to)."""
    n, Hq, D = q.shape
    G, S = Hq // cache.H, cache.S
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    qv = q.double().numpy()
    for b in range(n):
        x = cache.lens[b]
        for h in range(cache.H):
            at = np.arange(x)
            if pages is not None:
                n_pages = -(-x // S)
                at = np.concatenate([np.arange(p * S, min(x, (p + 1) * S))
                                     for p in pages[b, h].tolist() if 0 <= p < n_pages]
                                    + [np.arange(0)]).astype(np.int64)
            if window:
                at = at[at >= x - window]
            if at.size == 0:
                continue
            k, v = cache.values(cache.k, b, h)[at], cache.values(cache.v, b, h)[at]
            for j in range(h * G, (h + 1) * G):
                z = scale * (k @ qv[b, j])
                top = z.max()
                e = np.exp(z - top)
                lse[b, j] = top + np.log(e.sum())
                p = e / e.sum()
                out[b, j] = p @ v
                spread[b, j] = p @ np.abs(v)
                reach[b, j] = abs(scale) * (np.abs(k) @ np.abs(qv[b, j])).max()
    return out, lse, spread, reach


def bounds(cache):
    """float64 [P, H, 2, D] of every page that a sequence holds, NaN elsewhere."""
    want = np.full((cache.P, cache.H, 2, cache.D), np.nan)
    for b, x in enumerate(cache.lens):
        for h in range(cache.H):
            v = cache.values(cache.k, b, h)
            for p in range(-(-x // cache.S)):
                part = v[p * cache.S:(p + 1) * cache.S]
                want[cache.table[b, p], h] = part.min(0), part.max(0)
    return want


def select(cache, q, bd, top, first=0, last=1):
    """int32 [n, H, top]; bd float64 [P, H, 2, D]."""
    n, Hq, D = q.shape
    G = Hq // cache.H
    found = np.full((n, cache.H, top), -1, dtype=np.int32)
    for b, x in enumerate(cache.lens):
        m = -(-x // cache.S)
        for h in range(cache.H):
            qh = q[b, h * G:(h + 1) * G].double().numpy()
            score = []
            for p in range(m):
                lo, hi = bd[cache.table[b, p], h]
                score.append(math.fsum(np.maximum(qh * lo, qh * hi).ravel().tolist()))
            keep = [p < first or p >= m - last for p in range(m)]
            best = sorted(range(m), key=lambda p: (not keep[p], -score[p] if not keep[p] else 0, p))
            best = sorted(best[:top])
            found[b, h, :len(best)] = best
    return found


def out_tolerance(dtype, D, N, out, spread, reach):
    """Elementwise bound of |computed - out|.

    A logit of D products of a q and a k (q held in at least 22 bits) is off
    by (D + 8) 2^-24 + 2^-22 of the sum of its terms' magnitudes, its
    exponential by that much (relative) and 2^-21 for the function; sums over
    N tokens in f32 add N 2^-24.  The weights that multiply the values are
    rounded to f16 for a bf16 result (2^-11), else held in 22 bits.  Both the
    numerator and the denominator carry the error.  The result is rounded
    once: half a step of its dtype.
    """
    delta = reach * ((D + 8) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -20 + N * 2.0 ** -24
    delta = delta + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21)
    return (torch.finfo(dtype).eps / 2 * np.abs(out) + 2 * delta[..., None] * spread
            + torch.finfo(dtype).tiny * torch.finfo(dtype).eps)


def lse_tolerance(D, N, lse, reach):
    """As above, without the rounding of the weights: the logits' absolute
    error, the sum's relative one, and f32's half step of the result."""
    return (reach * ((D + 8) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -20 + N * 2.0 ** -24
            + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)))

// Attention of one new token over a paged packed cache: how the work is laid
// over the grid, shared by the general and the tensor-core kernel.
//
// The positions of every (sequence, kv head, tile of query heads), a pair, are
// cut into units of 128, the pairs' units are laid in one line, each behind a
// few units' length for what a pair costs by itself, and block i of n takes
// the i-th n-th of the line: sequences of any lengths keep all SMs busy for
// the same time, without a plan made on the host.  A block that holds all
// units of a pair writes its output; where a pair's units fall to several
// blocks, each writes a partial (the normalised sum in f32 and its weight) to
// one of its two workspace slots: slot 2i for a pair that began in an earlier
// block, slot 2i + 1 for one that begins here.  A second, small kernel joins them: the block after which a pair's first part lies
// looks through the slots of the blocks behind it.
#pragma once

#include <cuda_runtime.h>

#include "cache_format.cuh"
#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {
namespace attend {

constexpr int kUnit = 128;  // positions
// What a pair costs beside its units (queries, the first loads' latency, the
// join of the warps), in units: the line is laid in units plus this.  Measured
// with 0, 2, 4 and 6, us: 32 ragged sequences of up to 8192 tokens x 8 heads in
// fp8 88.6, 60.0, 58.7, 59.2; 96 even ones x 4 in mxfp4 119.7, 118.8, 119.4,
// 122.9; one of 131071 in nvfp4 47.0, 45.3, 45.1, 45.1; 16 in f16 with a window
// of 5001 33.2, 28.2, 28.1, 30.2; 24 with 32 listed pages 55.3, 53.3, 53.4, 55.3.
constexpr int kPairCost = 4;
// Before any token: finite, so that no difference of two of them is NaN.
constexpr float kLowest = -3.0e38f;
// The least exponent that weighted sums are held at, counted from the largest
// logit: what lies below is no f32 beside it.  (A band of values may hold only
// tokens far below that logit; taken from them, the exponent would have lost
// the scales' bits, and weights would overflow f16.)
constexpr float kFloor = -512.0f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kTcThreads = 128;
constexpr int kTcWarps = kTcThreads / 32;
constexpr int kTile = 16;           // tokens
constexpr float kLag = 4.0f;        // how far a logit may exceed the reference
constexpr float kWeightExp = 11.0f; // weights are held times 2^11: at most 2^15

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with a zero addend.
__device__ __forceinline__ void mma16816_first(float* c, const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes, or zeros where `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// BYTES (a power of two) bytes of shared memory, little-endian in words.
template <int BYTES>
__device__ __forceinline__ void lds_bytes(uint32_t* r, uint32_t a) {
  if constexpr (BYTES <= 2) {
    uint16_t h;
    if constexpr (BYTES == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
    else asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
    r[0] = h;
  } else if constexpr (BYTES == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(a) : "memory");
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
  } else {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
  }
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// y = (a - b) q of two columns, b negated; each operation rounded.
__device__ __forceinline__ void minus_times2(float* y, const float* a, const float* minus_b,
                                             const float* q) {
  asm("{\n\t.reg .b64 a, b, q;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "mov.b64 q, {%6, %7};\n\t"
      "add.rn.f32x2 a, a, b;\n\t"
      "mul.rn.f32x2 a, a, q;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(y[0]), "=f"(y[1])
      : "f"(a[0]), "f"(a[1]), "f"(minus_b[0]), "f"(minus_b[1]), "f"(q[0]), "f"(q[1]));
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) { return pack2<kF16>(lo, hi); }

struct Args {
  const void* q;
  int64_t q_stride;
  PagedCache c;
  const int32_t* selected;
  int top, window;  // window 0: none
  int q_heads, group, head_tiles, tile_heads;
  int least;  // units of a block's part, at least
  float scale_log2;  // softmax scale times log2(e)
  void* out;
  float* lse;
  int32_t* hdr;   // [2 n_ctas] pair + 1, or 0
  float2* part_w;  // [2 n_ctas][tile_heads] weight: y times 2^x
  float* part_o;  // [2 n_ctas][tile_heads][dim]
};

// One sequence's positions: [lo, lo + n) of its tokens, or of the listed
// pages' tokens one page after another (then lo is 0).
struct Span {
  int64_t len;  // tokens
  int lo, n, units;
};

__device__ __forceinline__ Span span_of(const Args& a, int64_t b) {
  Span s;
  s.len = MXQ_IN_RANGE(kChkAttendTable, b, a.c.n_seqs) ? __ldg(a.c.lengths + b) : 0;
  if (s.len < 0 || s.len > a.c.max_pages * a.c.page) {
    if (a.c.status) *a.c.status = MXQ_ERR_BAD_PAGE;
    s.len = 0;
  }
  if (a.selected) {
    s.lo = 0;
    s.n = s.len == 0 ? 0 : a.top * a.c.page;
  } else {
    const int64_t start = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.lo = (int)(start & ~(int64_t)15);  // tiles of 16 stay inside pages
    s.n = (int)(s.len - s.lo);
  }
  s.units = s.n > 0 ? (s.n - 1) / kUnit + 1 : 1;  // an empty pair has its output written too
  return s;
}

// The token of position v of a span: its place in the sequence, and its row in
// the cache ((page * heads + head) * page_size + slot) or -1 where there is
// none (a page list's -1, a page out of range, the end of the sequence).  The
// table is read only where one of the `count` positions from v on, which share
// a page, is attended to: entries before the window may be gone.
struct Token {
  int64_t pos, row;
};

__device__ __forceinline__ Token token_at(const Args& a, const Span& s, int64_t b, int head, int v,
                                          int count) {
  const PagedCache& c = a.c;
  Token t;
  int page_at, off;
  if (a.selected) {
    const int e = v / c.page;
    off = v - e * c.page;
    page_at = -1;
    if (MXQ_IN_RANGE(kChkAttendTable, e, a.top))
      page_at = __ldg(a.selected + (b * c.heads + head) * a.top + e);
    if (page_at < 0 || page_at >= (s.len + c.page - 1) / c.page) return Token{-1, -1};
  } else {
    page_at = (s.lo + v) / c.page;
    off = s.lo + v - page_at * c.page;
  }
  t.pos = (int64_t)page_at * c.page + off;
  t.row = -1;
  if (t.pos >= s.len || (a.window > 0 && t.pos + count <= s.len - a.window)) return t;
  if (!MXQ_IN_RANGE(kChkAttendTable, page_at, c.max_pages)) return t;
  const int64_t page = __ldg(c.page_table + b * c.max_pages + page_at);
  if (page < 0 || page >= c.num_pages) {
    if (c.status) *c.status = MXQ_ERR_BAD_PAGE;
    return t;
  }
  t.row = (page * c.heads + head) * c.page + off;
  return t;
}

// Whether the new token attends to a position.
__device__ __forceinline__ bool live(const Args& a, const Span& s, int64_t pos) {
  return pos >= 0 && pos < s.len && (a.window == 0 || pos >= s.len - a.window);
}

// Whether elements [i, i + n) are a query's.
__device__ __forceinline__ bool is_q(const Args& a, int64_t i, int n) {
  [[maybe_unused]] const int64_t all =
      (a.c.n_seqs - 1) * a.q_stride + (int64_t)a.q_heads * a.c.dim;
  return MXQ_IN_RANGE(kChkAttendQuery, i, all) && MXQ_IN_RANGE(kChkAttendQuery, i + n - 1, all);
}

__device__ __forceinline__ float load_q(const Args& a, int dt, int64_t i) {
  if (!is_q(a, i, 1)) return 0.0f;
  if (dt == kBF16) return elem_to_f32<kBF16>(((const uint16_t*)a.q)[i]);
  if (dt == kF16) return elem_to_f32<kF16>(((const uint16_t*)a.q)[i]);
  return ((const float*)a.q)[i];
}

// Where a block's part of the line begins: units before it and its first
// sequence.  All threads of the block call it.
struct Part {
  int64_t begin, end;  // of the line
  int64_t b, b_begin;  // the sequence at begin and where it starts
};

template <int kWarps>
__device__ __forceinline__ Part part_of(const Args& a) {
  constexpr int kThreads = 32 * kWarps;
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_b[2];
  const int64_t pairs = (int64_t)a.c.heads * a.head_tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto length = [&](int64_t b) {
    return b < a.c.n_seqs ? pairs * (span_of(a, b).units + kPairCost) : 0;
  };
  auto cut = [&](int64_t total) {
    // no part is shorter than least units: the parts of a pair lie in blocks
    // that follow one another, and are worth their join
    const int64_t most = total / a.least;
    const uint32_t n = most < gridDim.x ? (uint32_t)most : gridDim.x;
    const int64_t each = total < ((int64_t)1 << 32) ? (uint32_t)total / n : total / n;
    const uint32_t rest = (uint32_t)(total - each * n);  // below n, n below 2^16
    auto start = [&](uint32_t i) { return min(total, each * i + rest * i / n); };
    Part p;
    p.begin = start(blockIdx.x);
    p.end = start(blockIdx.x + 1);
    return p;
  };
  if (a.c.n_seqs <= 32) {  // each warp by itself
    const int64_t mine = length(lane);
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    Part p = cut(__shfl_sync(0xffffffffu, sum, 31));
    const unsigned in = __ballot_sync(0xffffffffu, sum - mine <= p.begin && p.begin < sum);
    const int who = in ? __ffs((int)in) - 1 : 0;  // none: an empty part at the end
    p.b = who;
    p.b_begin = __shfl_sync(0xffffffffu, sum - mine, who);
    return p;
  }
  const int64_t one = length(threadIdx.x);  // all there is for up to kThreads sequences
  int64_t total = one;
  for (int64_t b = threadIdx.x + kThreads; b < a.c.n_seqs; b += kThreads) total += length(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) total += s_sum[i];
  __syncthreads();
  Part p = cut(total);
  int64_t before = 0;
  for (int64_t b0 = 0; b0 < a.c.n_seqs; b0 += kThreads) {
    const int64_t b = b0 + threadIdx.x;
    const int64_t mine = b0 == 0 ? one : length(b);
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    int64_t first = before + sum - mine, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) first += s_sum[i];
      all += s_sum[i];
    }
    if (mine > 0 && first <= p.begin && p.begin < first + mine) s_b[0] = b, s_b[1] = first;
    before += all;
    __syncthreads();
    if (before > p.begin) break;
  }
  p.b = s_b[0];
  p.b_begin = s_b[1];
  return p;
}

// Where a finished (or partial) pair is written.
struct Target {
  int64_t b;
  int head, tile;
  bool whole;
  int slot;
};

__device__ __forceinline__ void store_out(const Args& a, int dt, int64_t i, float v) {
  if (dt == kBF16) store_one<kBF16>(a.out, i, v);
  else if (dt == kF16) store_one<kF16>(a.out, i, v);
  else store_one<kF32>(a.out, i, v);
}

// The joined value of channel ch of head r of a pair, and of its weight.
__device__ __forceinline__ void put(const Args& a, int dt, const Target& t, int r, int ch,
                                    float v) {
  if (t.whole) {
    const int64_t qh = (int64_t)t.head * a.group + t.tile * a.tile_heads + r;
    const int64_t i = (t.b * a.q_heads + qh) * a.c.dim + ch;
    if (MXQ_IN_RANGE(kChkAttendOut, i, a.c.n_seqs * a.q_heads * a.c.dim)) store_out(a, dt, i, v);
  } else {
    const int64_t i = ((int64_t)t.slot * a.tile_heads + r) * a.c.dim + ch;
    if (MXQ_IN_RANGE(kChkAttendWs, i, 2ll * gridDim.x * a.tile_heads * a.c.dim)) a.part_o[i] = v;
  }
}
// sum times 2^top; a partial keeps the two apart, as their sum would lose the
// first beside large logits.
__device__ __forceinline__ void put_weight(const Args& a, const Target& t, int r, float top,
                                           float sum) {
  if (t.whole) {
    const int64_t qh = (int64_t)t.head * a.group + t.tile * a.tile_heads + r;
    if (a.lse && MXQ_IN_RANGE(kChkAttendOut, t.b * a.q_heads + qh, a.c.n_seqs * a.q_heads))
      a.lse[t.b * a.q_heads + qh] =
          sum == 0.0f ? __int_as_float(0xFF800000) : (top + log2f(sum)) * kLn2;
  } else {
    const int64_t i = (int64_t)t.slot * a.tile_heads + r;
    if (MXQ_IN_RANGE(kChkAttendWs, i, 2ll * gridDim.x * a.tile_heads))
      a.part_w[i] = make_float2(top, sum);
  }
}

// Walk a block's part of the line: work(span, b, head, tile, first position,
// last position + 1, target) once per pair.
template <int kWarps, class Work>
__device__ __forceinline__ void walk(const Args& a, Work work) {
  const Part p = part_of<kWarps>(a);
  const int64_t pairs = (int64_t)a.c.heads * a.head_tiles;
  int32_t hdr[2] = {0, 0};
  int64_t u = p.begin, b = p.b, b_begin = p.b_begin;
  while (u < p.end) {
    const Span s = span_of(a, b);
    const int64_t length = s.units + kPairCost;
    const int64_t pl = (u - b_begin) / length;  // pair of the sequence
    const int64_t x0 = u - b_begin - pl * length, x1 = min(length, x0 + (p.end - u));
    const int j0 = (int)max((int64_t)0, x0 - kPairCost), j1 = (int)max((int64_t)0, x1 - kPairCost);
    Target t;
    t.b = b;
    t.head = (int)(pl / a.head_tiles);
    t.tile = (int)(pl - (int64_t)t.head * a.head_tiles);
    t.whole = j0 == 0 && j1 == s.units;
    t.slot = 2 * blockIdx.x + (j0 == 0 ? 1 : 0);
    if (j1 > j0) {
      if (!t.whole) hdr[j0 == 0 ? 1 : 0] = (int32_t)(b * pairs + pl + 1);
      work(s, t, j0 * kUnit, min(s.n, j1 * kUnit));
    }
    u += x1 - x0;
    if (u == b_begin + pairs * length) {
      b_begin = u;
      ++b;
    }
  }
  if (threadIdx.x == 0) {
    a.hdr[2 * blockIdx.x] = hdr[0];
    a.hdr[2 * blockIdx.x + 1] = hdr[1];
  }
}

// The tensor-core kernels of each format and head size: `nb` scales a row, a
// grid of at most `units` blocks (returned in *grid).
int tc_fp8_64(const Args& a, int dt, int nb, int64_t units, int* grid, cudaStream_t st);
int tc_fp8_128(const Args& a, int dt, int nb, int64_t units, int* grid, cudaStream_t st);
int tc_fp8_256(const Args& a, int dt, int nb, int64_t units, int* grid, cudaStream_t st);
int tc_mxfp4(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st);
int tc_nvfp4(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st);

}  // namespace attend
}  // namespace mxq

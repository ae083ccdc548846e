// Writing a paged packed cache: new rows quantized into their pages, and the
// channelwise bounds of the pages' keys (sm_100a).
//
// append: row t of sequence b (offs[b-1] <= t < offs[b]) is the token at
// position p = lengths[b] - (offs[b] - t); its codes go to slot p mod S of
// page page_table[b][p / S].  Quantization is that of the packed cache: per
// group of B channels k = the least exponent with 2^k qmax >= amax, code =
// cast(x 2^-k).  One pass: K and V are read once, codes and scale bytes (and,
// where asked for, the values they stand for) written once; bound by HBM for
// prompts and by the launch for a single step.
//
// bounds: lo / hi [page][head][channel] = the least / largest value over the
// page's valid tokens.  Every page is computed from its codes alone, so the
// result does not depend on what was there before (a page that was freed and
// taken again, a slot that was written twice).
#include "cache_format.cuh"
#include "mxq.h"
#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  const void *k, *v;
  void *k_out, *v_out;
  const int32_t* offs;
  int64_t rows, k_stride, v_stride;
  int tokens_per_cta;
  PagedCache c;
};

// Row of head 0 of the cache for row t, a token of sequence b (the first whose
// offs lies above t), or -1: padding, or a row whose position or page is out of
// range (reported).  The rows of the other heads lie S apart.
__device__ __forceinline__ int64_t row_of(const AppendArgs& a, int64_t t, int b) {
  if (b == a.c.n_seqs || !MXQ_IN_RANGE(kChkAppendTable, b, a.c.n_seqs)) return -1;
  const int64_t end = __ldg(a.offs + b), begin = b > 0 ? __ldg(a.offs + b - 1) : 0;
  const int64_t len = __ldg(a.c.lengths + b), pos = len - (end - t);
  if (begin < 0 || begin > t || end > a.rows) {
    if (a.c.status) *a.c.status = MXQ_ERR_BAD_OFFS;
    return -1;
  }
  int64_t page = -1;
  uint32_t at = 0;
  if (pos >= 0 && len <= a.c.max_pages * a.c.page) {  // positions end at 2^30
    const uint32_t j = (uint32_t)pos / (uint32_t)a.c.page;
    at = (uint32_t)pos - j * (uint32_t)a.c.page;
    if (MXQ_IN_RANGE(kChkAppendTable, j, a.c.max_pages))
      page = __ldg(a.c.page_table + b * a.c.max_pages + j);
  }
  if (page < 0 || page >= a.c.num_pages) {
    if (a.c.status) *a.c.status = MXQ_ERR_BAD_PAGE;
    return -1;
  }
  return page * a.c.heads * a.c.page + at;
}

// The first b >= from with offs[b] > t, n_seqs where there is none; the places
// near `from` first.
__device__ __forceinline__ int sequence_of(const AppendArgs& a, int64_t t, int from) {
  const int n = (int)a.c.n_seqs;
  int lo = from, step = 1;
  while (step <= n - lo && __ldg(a.offs + lo + step - 1) <= t) lo += step, step *= 2;
  int hi = lo + min(step - 1, n - lo);
  while (lo < hi) {
    const int mid = lo + ((hi - lo) >> 1);  // there may be 2^31 - 2 sequences
    if (__ldg(a.offs + mid) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
// The same from 0 by a warp, which looks at 32 places at a time: a block has
// few tokens, and the loads that wait for one another are what a search costs.
__device__ __forceinline__ int sequence_of_by_warp(const AppendArgs& a, int64_t t, int lane) {
  uint32_t lo = 0, hi = (uint32_t)a.c.n_seqs;  // lo <= b <= hi; places up to hi + 30 are formed
  while (lo < hi) {
    const uint32_t step = (hi - lo + 31) / 32;  // a lane: the last of its `step` sequences
    const uint32_t mid = min(lo + lane * step + step - 1, hi - 1);
    const uint32_t over = __ballot_sync(0xffffffffu, __ldg(a.offs + mid) > t);
    if (over == 0) return (int)hi;
    lo += (__ffs(over) - 1) * step;
    hi = min(lo + step - 1, hi - 1);
  }
  return (int)lo;
}

// Block 0 looks over the whole of offs: a sequence whose end lies before its
// start owns no row, and so would go unnoticed by the rows.
__device__ __forceinline__ void check_offs(const AppendArgs& a) {
  if (blockIdx.x != 0 || !a.c.status) return;
  for (int64_t b = threadIdx.x; b < a.c.n_seqs; b += blockDim.x)
    if (a.offs[b] < (b > 0 ? a.offs[b - 1] : 0) || a.offs[b] > a.rows)
      *a.c.status = MXQ_ERR_BAD_OFFS;
}

constexpr int kMaxCtaTokens = 32;

// Quotients of x < 2^15 by a divisor d <= 2^15 known at launch: floor(2x m /
// 2^32) with m = ceil(2^31 / d) is exact, as x (m d - 2^31) < x d < 2^31
// (Granlund and Montgomery, "Division by invariant integers", 1994).
constexpr int64_t kMaxItems = 1 << 15;
struct Divisor {
  uint32_t d, m;
  explicit Divisor(uint32_t x = 1) : d(x), m((uint32_t)((((uint64_t)1 << 31) + x - 1) / x)) {}
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return __umulhi(2 * x, m); }
};

struct AppendPlan {
  Divisor per_tok, per_head;  // items of a token, of a head
};

// Magnitude of the largest of eight elements, as f32 bits.
template <int DT>
__device__ __forceinline__ uint32_t amax8(const uint32_t* w) {
  if constexpr (ElemTraits<DT>::kBytes == 2) {  // 16-bit magnitudes order as integers
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, w[j] & 0x7FFFFFFFu);
    return m;
  }
}

// Fast path.  An item is 8 channels of one row of K and of V, which share the
// arithmetic of their place; a block takes tokens_per_cta tokens (all heads),
// about 2 items a thread, so that each thread has several loads in flight; B/8 lanes share a group's maximum,
// taken on the raw 16-bit magnitudes.  The place of each token is looked up
// once per block, while the first loads (which need no place) are under way.
// Bound by issue: 25 thousand tokens of 4 x 128 in mxfp4 with their values take
// 23 us (28 with K and V as items of their own, 33 with the loads after the
// lookup too), 18 at the speed of HBM.
template <int DT, int FMT, int LPB>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a, AppendPlan plan) {
  __shared__ int64_t s_row[kMaxCtaTokens];  // head 0's in the cache, in items; S rows to the next
  constexpr int kUnroll = ElemTraits<DT>::kBytes == 2 ? 2 : 1;
  constexpr uint32_t kItemBytes = 8 * ElemTraits<DT>::kBytes;
  constexpr int kWords = ElemTraits<DT>::kBytes == 2 ? 4 : 8;
  const PagedCache& c = a.c;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_cta;
  const int n_tok = (int)min((int64_t)a.tokens_per_cta, a.rows - t0);
  const uint32_t n_items = n_tok * plan.per_tok.d, per_head = plan.per_head.d;
  const uint32_t lane = threadIdx.x & 31;
  const int64_t in_bytes[2] = {a.k_stride * ElemTraits<DT>::kBytes,
                               a.v_stride * ElemTraits<DT>::kBytes};
  const char* const in[2] = {(const char*)a.k + t0 * in_bytes[0],
                             (const char*)a.v + t0 * in_bytes[1]};
  uint32_t w[kUnroll][2][kWords];
  auto load = [&](uint32_t base) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t item = base + u * kThreads + lane;
      if (item >= n_items) continue;
      const uint32_t tok = plan.per_tok.div(item), rem = item - tok * plan.per_tok.d;
      if (!MXQ_IN_RANGE(kChkAppendIn, t0 + tok, a.rows) ||
          !MXQ_IN_RANGE(kChkAppendIn, rem, plan.per_tok.d))
        continue;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s == 1 && !a.v) break;
        const char* from = in[s] + tok * in_bytes[s] + rem * kItemBytes;
#pragma unroll
        for (int j = 0; j < kWords; j += 4) {
          const uint4 v = ld_stream_v4(from + 4 * j);
          w[u][s][j] = v.x, w[u][s][j + 1] = v.y, w[u][s][j + 2] = v.z, w[u][s][j + 3] = v.w;
        }
      }
    }
  };
  uint32_t base = threadIdx.x & ~31;
  load(base);  // under way while the places are looked up
  check_offs(a);
  if (threadIdx.x < 32) {
    const int first = sequence_of_by_warp(a, t0, lane);
    if ((int)lane < n_tok) {
      const int64_t row = row_of(a, t0 + lane, sequence_of(a, t0 + lane, first));
      s_row[lane] = row < 0 ? -1 : row * per_head;
    }
  }
  __syncthreads();
  const int64_t head_items = (int64_t)(c.page - 1) * per_head;  // beyond a dense row's
  for (;;) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t item = base + u * kThreads + lane;
      const bool within = item < n_items;
      const uint32_t tok = within ? plan.per_tok.div(item) : 0;
      const uint32_t rem = item - tok * plan.per_tok.d;
      const int64_t row = s_row[tok];
      const bool valid = within && row >= 0;
      const int64_t dst = row + rem + plan.per_head.div(rem) * head_items;
      const int64_t src = t0 * plan.per_tok.d + item;  // dense
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s == 1 && !a.v) break;
        const uint32_t* raw = w[u][s];
        uint32_t m = valid ? amax8<DT>(raw) : 0;
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!valid) continue;
        const int k = group_scale_exp<FMT>(mag_as_f32_bits<DT>(m));
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (kWords == 4)
            x[j] = elem_to_f32<DT>((j & 1) ? raw[j / 2] >> 16 : raw[j / 2] & 0xFFFFu);
          else
            x[j] = elem_to_f32<DT>(raw[j]);
        }
        uint32_t h[4];  // the codes' values, as f16
        const uint2 code = encode8<FMT>(x, group_inverse(k), h);
        if (MXQ_IN_RANGE(kChkAppendOut, dst, c.num_pages * c.heads * c.page * per_head))
          store_codes<FMT>(s ? c.v_codes : c.k_codes, dst, code);
        if ((lane & (LPB - 1)) == 0 &&
            MXQ_IN_RANGE(kChkAppendScale, dst / LPB,
                         c.num_pages * c.heads * c.page * (int64_t)c.row_scales()))
          (s ? c.v_scales : c.k_scales)[(uint64_t)dst / LPB] = (uint8_t)scale_byte<FMT>(k);
        void* out = s ? a.v_out : a.k_out;
        if (out && MXQ_IN_RANGE(kChkAppendOut, src, a.rows * plan.per_tok.d)) {
          float y[8];
          scaled8<FMT>(h, group_scale(k), y);
          store8<DT>(out, src, y);
        }
      }
    }
    base += kThreads * kUnroll;
    if (base >= n_items) break;
    load(base);
  }
}

// General path: any block size, stride and alignment.  One thread per (row, K
// or V, head, group).
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) append_general_kernel(AppendArgs a) {
  const PagedCache& c = a.c;
  const int B = c.block, nb = c.row_scales(), rb = c.row_bytes();
  const int two = a.v ? 2 : 1;
  const int64_t per_tok = (int64_t)two * c.heads * nb, n = a.rows * per_tok;
  [[maybe_unused]] const int64_t n_rows = c.num_pages * c.heads * c.page;
  check_offs(a);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / per_tok;
    const int rem = (int)(i - t * per_tok);
    const bool is_v = rem >= c.heads * nb;
    const int hg = is_v ? rem - c.heads * nb : rem, head = hg / nb, g = hg - head * nb;
    int64_t row = row_of(a, t, sequence_of(a, t, 0));
    if (row < 0) continue;
    row += (int64_t)head * c.page;
    const void* in = is_v ? a.v : a.k;
    const int64_t src = t * (is_v ? a.v_stride : a.k_stride) + head * c.dim + g * B;
    const int64_t dense = (t * c.heads + head) * c.dim + g * B;
    uint8_t* codes = (is_v ? c.v_codes : c.k_codes) + row * rb;
    void* out = is_v ? a.v_out : a.k_out;
    if (!MXQ_IN_RANGE(kChkAppendIn, t, a.rows) || !MXQ_IN_RANGE(kChkAppendOut, row, n_rows) ||
        !MXQ_IN_RANGE(kChkAppendScale, row * nb + g, n_rows * nb) ||
        !MXQ_IN_RANGE(kChkAppendIn, head * c.dim + g * B + B - 1, c.heads * c.dim) ||
        !MXQ_IN_RANGE(kChkAppendOut, row * rb + (FMT == MXQ_FMT_FP8 ? g * B + B : (g + 1) * B / 2) - 1,
                      n_rows * rb) ||
        !MXQ_IN_RANGE(kChkAppendOut, dense + B - 1, a.rows * c.heads * c.dim))
      continue;
    uint32_t m = 0;
    for (int j = 0; j < B; ++j) m = max(m, mag_as_f32_bits<DT>(elem_bits_at<DT>(in, src + j)));
    const int k = group_scale_exp<FMT>(m);
    const float inv = exp2i(-k), s = exp2i(k);
    (is_v ? c.v_scales : c.k_scales)[row * nb + g] = (uint8_t)scale_byte<FMT>(k);
    for (int j = 0; j < B; j += 2) {
      const bool pair = j + 1 < B;
      const float x0 = elem_to_f32<DT>(elem_bits_at<DT>(in, src + j));
      const float x1 = pair ? elem_to_f32<DT>(elem_bits_at<DT>(in, src + j + 1)) : 0.0f;
      uint32_t h2;
      if constexpr (FMT == MXQ_FMT_FP8) {
        const uint32_t b = e4m3x2(x0 * inv, x1 * inv);
        codes[g * B + j] = (uint8_t)b;
        if (pair) codes[g * B + j + 1] = (uint8_t)(b >> 8);
        h2 = e4m3x2_to_f16x2(b);
      } else {
        const uint32_t b = e2m1x2(fmaf(x0, inv, 0.0f), fmaf(x1, inv, 0.0f));
        codes[(g * B + j) / 2] = (uint8_t)b;
        h2 = e2m1x2_to_f16x2(b);
      }
      if (out) {
        const float y0 = f16lo(h2) * s, y1 = f16hi(h2) * s;
        // fp4 zero magnitudes give +0, an fp8 zero keeps its sign
        store_one<DT>(out, dense + j, FMT == MXQ_FMT_FP8 ? y0 : y0 + 0.0f);
        if (pair) store_one<DT>(out, dense + j + 1, FMT == MXQ_FMT_FP8 ? y1 : y1 + 0.0f);
      }
    }
  }
}

template <int DT, int FMT>
void launch_append_fmt(AppendArgs a, bool fast, cudaStream_t st) {
  const int64_t per_tok = (int64_t)a.c.heads * (a.c.dim / 8);
  // a block's items are at most 512 or one token's
  if (!fast || per_tok > kMaxItems) {
    const int64_t n = a.rows * a.c.heads * a.c.row_scales() * (a.v ? 2 : 1);
    append_general_kernel<DT, FMT>
        <<<wave_grid((const void*)append_general_kernel<DT, FMT>, kThreads, n, kThreads), kThreads,
           0, st>>>(a);
    return;
  }
  a.tokens_per_cta = (int)(per_tok >= 512 ? 1 : 512 / per_tok);
  if (a.tokens_per_cta > kMaxCtaTokens) a.tokens_per_cta = kMaxCtaTokens;
  const unsigned grid = (unsigned)((a.rows + a.tokens_per_cta - 1) / a.tokens_per_cta);
  AppendPlan plan;
  plan.per_tok = Divisor((uint32_t)per_tok);
  plan.per_head = Divisor((uint32_t)(a.c.dim / 8));
  switch (a.c.block / 8) {
    case 1: append_kernel<DT, FMT, 1><<<grid, kThreads, 0, st>>>(a, plan); break;
    case 2: append_kernel<DT, FMT, 2><<<grid, kThreads, 0, st>>>(a, plan); break;
    case 4: append_kernel<DT, FMT, 4><<<grid, kThreads, 0, st>>>(a, plan); break;
    case 8: append_kernel<DT, FMT, 8><<<grid, kThreads, 0, st>>>(a, plan); break;
    case 16: append_kernel<DT, FMT, 16><<<grid, kThreads, 0, st>>>(a, plan); break;
    default: append_kernel<DT, FMT, 32><<<grid, kThreads, 0, st>>>(a, plan); break;
  }
}

template <int DT>
void launch_append_dt(const AppendArgs& a, bool fast, cudaStream_t st) {
  switch (a.c.fmt) {
    case MXQ_FMT_FP8: launch_append_fmt<DT, MXQ_FMT_FP8>(a, fast, st); break;
    case MXQ_FMT_MXFP4: launch_append_fmt<DT, MXQ_FMT_MXFP4>(a, fast, st); break;
    default: launch_append_fmt<DT, MXQ_FMT_NVFP4>(a, fast, st); break;
  }
}

// ---------------------------------------------------------------- bounds

struct BoundArgs {
  PagedCache c;
  int64_t new_tokens;
  uint16_t* bounds;
};

// Value of channel ch of a row of codes; the product is exact.
template <int FMT>
__device__ __forceinline__ float value_at(const uint8_t* codes, const uint8_t* scales, int ch,
                                          int B) {
  const float s = scale_value<FMT>(scales[ch / B]);
  if constexpr (FMT == MXQ_FMT_FP8) {
    return f16lo(e4m3x2_to_f16x2(codes[ch])) * s;
  } else {
    const uint32_t byte = codes[ch / 2];
    return fmaf(f16lo(e2m1x2_to_f16x2((ch & 1) ? byte >> 4 : byte & 15u)), s, 0.0f);
  }
}

constexpr int kBoundThreads = 128;

__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// One warp per (page of a sequence, head), pages counted from the sequence's
// last; a block takes four pages that follow one another.  VEC = 8 or 16
// channels a lane: D / VEC lanes hold a row, the other lanes further rows,
// eight rows a lane in flight; two rows at a time go into the running bounds
// (one three-way minimum and maximum for two values: these and the
// conversions, not the bytes, are what the kernel issues most), and the lanes
// of a channel are joined by shuffles.  (A block per page, its warps joined in
// shared memory, spent more on starting 33 thousand blocks than on the rows:
// 84 us against 45 for 136 thousand tokens x 8 heads in fp8.)  VEC = 1: a lane
// holds one channel over all rows, for any block size and alignment.
template <int FMT, int VEC>
__global__ void __launch_bounds__(kBoundThreads) bound_kernel(BoundArgs a) {
  const PagedCache& c = a.c;
  const int64_t b = blockIdx.y;
  const int head = blockIdx.z, lane = threadIdx.x & 31;
  const int64_t len = c.lengths[b];
  if (len < 0 || len > c.max_pages * c.page) {
    if (c.status) *c.status = MXQ_ERR_BAD_PAGE;
    return;
  }
  // lengths end at 2^30
  const int n_pages = ((uint32_t)len + c.page - 1) / (uint32_t)c.page;
  const int j = n_pages - 1 - (int)(blockIdx.x * (kBoundThreads / 32) + (threadIdx.x >> 5));
  if (j < 0 || (int64_t)(j + 1) * c.page <= len - a.new_tokens) return;
  if (!MXQ_IN_RANGE(kChkBoundTable, j, c.max_pages)) return;
  const int64_t page = c.page_table[b * c.max_pages + j];
  if (page < 0 || page >= c.num_pages) {
    if (c.status) *c.status = MXQ_ERR_BAD_PAGE;
    return;
  }
  const int rows = min(c.page, (int)len - j * c.page);
  const int rb = c.row_bytes(), nb = c.row_scales();
  const int64_t row0 = (page * c.heads + head) * c.page;
  const uint8_t* codes = c.k_codes + row0 * rb;
  const uint8_t* scales = c.k_scales + row0 * nb;
  uint16_t* out = a.bounds + (page * c.heads + head) * 2 * c.dim;
  [[maybe_unused]] const int64_t n_rows = c.num_pages * c.heads * c.page;
  const float inf = __int_as_float(0x7F800000);
  if constexpr (VEC > 1) {
    constexpr int UNROLL = 8;
    constexpr int WORDS = FMT == MXQ_FMT_FP8 ? VEC / 4 : VEC / 8;  // of a lane's codes of a row
    const int per_row = c.dim / VEC;
    for (int lane0 = 0; lane0 < per_row; lane0 += 32) {  // heads wider than a warp
      const int width = min(32, per_row - lane0), at_once = 32 / width;
      const int r = lane / width, cv = lane0 + lane - r * width, sb = cv * VEC / c.block;
      float lo[VEC], hi[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) lo[i] = inf, hi[i] = -inf;
      if (r < at_once) {
        for (int s = r; s < rows; s += at_once * UNROLL) {
          uint32_t w[UNROLL][WORDS], sc[UNROLL];
          const uint8_t* p = codes + (uint32_t)(s * rb) + cv * (WORDS * 4);
          const uint8_t* ps = scales + (uint32_t)(s * nb) + sb;
          // past the end: the batch's first row again, which changes no bound
          const int left = (rows - s + at_once - 1) / at_once;
          [[maybe_unused]] const int64_t last = row0 + s + (min(left, UNROLL) - 1) * at_once;
          if (!MXQ_IN_RANGE(kChkBoundIn, last * rb + (cv + 1) * (WORDS * 4) - 1, n_rows * rb) ||
              !MXQ_IN_RANGE(kChkBoundScale, last * nb + sb, n_rows * nb))
            break;
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            const int step = u < left ? u * at_once : 0;
            const uint32_t* q = (const uint32_t*)(p + step * rb);
            if constexpr (WORDS == 2) {
              const uint2 v = __ldg((const uint2*)q);
              w[u][0] = v.x, w[u][1] = v.y;
            } else {
              w[u][0] = __ldg(q);
            }
            sc[u] = __ldg(ps + step * nb);
          }
#pragma unroll
          for (int u = 0; u < UNROLL; u += 2) {
            float v[2][VEC];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float f = finite_scale<FMT>(sc[u + q]);
#pragma unroll
              for (int x = 0; x < VEC / 8; ++x)
                values8<FMT>(w[u + q] + x * (WORDS * 8 / VEC), f, v[q] + 8 * x);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              lo[i] = min3(lo[i], v[0][i], v[1][i]);
              hi[i] = max3(hi[i], v[0][i], v[1][i]);
            }
          }
        }
      }
      // the first row's lanes take the others' bounds; no other lane changes, so
      // that what is taken is of that lane's channels alone, whatever the width
      for (int q = 1; q < at_once; ++q) {
        const int from = (lane + q * width) & 31;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float l = __shfl_sync(0xffffffffu, lo[i], from);
          const float h = __shfl_sync(0xffffffffu, hi[i], from);
          if (r == 0) lo[i] = fminf(lo[i], l), hi[i] = fmaxf(hi[i], h);
        }
      }
      if (r == 0 && MXQ_IN_RANGE(kChkBoundOut, page, c.num_pages) &&
          MXQ_IN_RANGE(kChkBoundOut, cv * VEC + VEC - 1, c.dim)) {
#pragma unroll
        for (int x = 0; x < VEC / 8; ++x) {
          store8<kBF16>(out + cv * VEC + 8 * x, 0, lo + 8 * x);
          store8<kBF16>(out + c.dim + cv * VEC + 8 * x, 0, hi + 8 * x);
        }
      }
    }
  } else {
    for (int ch = lane; ch < c.dim; ch += 32) {
      float lo = inf, hi = -inf;
      for (int s = 0; s < rows; ++s) {
        if (!MXQ_IN_RANGE(kChkBoundIn, row0 + s, n_rows) ||
            !MXQ_IN_RANGE(kChkBoundScale, ch / c.block, nb))
          continue;
        const float v = value_at<FMT>(codes + (int64_t)s * rb, scales + (int64_t)s * nb, ch, c.block);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
      }
      if (!MXQ_IN_RANGE(kChkBoundOut, page, c.num_pages)) continue;
      out[ch] = (uint16_t)(pack2<kBF16>(lo, 0.0f) & 0xFFFFu);
      out[c.dim + ch] = (uint16_t)(pack2<kBF16>(hi, 0.0f) & 0xFFFFu);
    }
  }
}

template <int FMT>
void launch_bound_fmt(const BoundArgs& a, bool fast, dim3 grid, cudaStream_t st) {
  // a lane takes 8 bytes of codes where the scale blocks allow it
  if (!fast) bound_kernel<FMT, 1><<<grid, kBoundThreads, 0, st>>>(a);
  else if (FMT != MXQ_FMT_FP8 && a.c.block % 16 == 0)
    bound_kernel<FMT, FMT != MXQ_FMT_FP8 ? 16 : 8><<<grid, kBoundThreads, 0, st>>>(a);
  else bound_kernel<FMT, 8><<<grid, kBoundThreads, 0, st>>>(a);
}

}  // namespace

int launch_append_cache_paged(const void* k, const void* v, int dt, int64_t rows, int64_t k_stride,
                              int64_t v_stride, const int32_t* offs, const PagedCache& c,
                              void* k_out, void* v_out, bool fast, cudaStream_t st) {
  const AppendArgs a{k, v, k_out, v_out, offs, rows, k_stride, v_stride, 1, c};
  switch (dt) {
    case kBF16: launch_append_dt<kBF16>(a, fast, st); break;
    case kF16: launch_append_dt<kF16>(a, fast, st); break;
    default: launch_append_dt<kF32>(a, fast, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

int launch_bound_cache_pages(const PagedCache& c, int64_t new_tokens, void* bounds, bool fast,
                             cudaStream_t st) {
  // the last new_tokens tokens lie in at most this many pages
  int64_t pages = (new_tokens - 1) / c.page + 2;
  if (new_tokens > c.max_pages * c.page || pages > c.max_pages) pages = c.max_pages;
  const BoundArgs a{c, new_tokens, (uint16_t*)bounds};
  // grid.y ends at 65535: longer batches go in parts (heads are at most that)
  for (int64_t b = 0; b < c.n_seqs; b += 65535) {
    BoundArgs part = a;
    part.c.page_table += b * c.max_pages;
    part.c.lengths += b;
    part.c.n_seqs = c.n_seqs - b < 65535 ? c.n_seqs - b : 65535;
    const dim3 grid((unsigned)((pages + 3) / 4), (unsigned)part.c.n_seqs, (unsigned)c.heads);
    switch (c.fmt) {
      case MXQ_FMT_FP8: launch_bound_fmt<MXQ_FMT_FP8>(part, fast, grid, st); break;
      case MXQ_FMT_MXFP4: launch_bound_fmt<MXQ_FMT_MXFP4>(part, fast, grid, st); break;
      default: launch_bound_fmt<MXQ_FMT_NVFP4>(part, fast, grid, st); break;
    }
  }
  return cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

MXQ_DEFINE_CHECK_READER(check_record_cache_paged)

}  // namespace mxq

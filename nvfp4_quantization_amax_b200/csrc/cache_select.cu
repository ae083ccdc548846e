// Selection of the pages that a new token attends to (sm_100a).
//
// The score of a page bounds the logits of its tokens from above: with lo and
// hi the channelwise bounds of its keys, q k <= max(q lo, q hi) in every
// channel.  Summed over the kv head's query heads it is linear in the heads'
// positive and negative parts,
//   score = sum_c lo_c Q-_c + hi_c Q+_c,   Q-+ = sum over heads of min/max(q, 0),
// so a group of any size costs one product of 2 D terms a page; it is taken
// in 64-bit floating point, so that the order of the sum decides no choice
// between pages that differ.  Bound by the read of the bounds (4 D bytes a
// page and head).  The largest scores are then found by their ordered 64-bit
// patterns, digit by digit from the top.
#include "mxq.h"
#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPagesPerWarp = 8;

struct SelectArgs {
  const void* q;
  const uint16_t* bounds;
  PagedCache c;
  int64_t q_stride;
  int group;
  int top, keep_first, keep_last;
  int32_t* selected;
  uint64_t* keys;  // [n_seqs][heads][max_pages]
};

__device__ __forceinline__ float q_at(const void* q, int dt, int64_t i) {
  if (dt == kBF16) return elem_to_f32<kBF16>(((const uint16_t*)q)[i]);
  if (dt == kF16) return elem_to_f32<kF16>(((const uint16_t*)q)[i]);
  return ((const float*)q)[i];
}

// Pages of sequence b, or 0 where its length is out of range (reported).
__device__ __forceinline__ int pages_of(const PagedCache& c, int64_t b) {
  const int64_t len = __ldg(c.lengths + b);
  if (len < 0 || len > c.max_pages * c.page) {
    if (c.status) *c.status = MXQ_ERR_BAD_PAGE;
    return 0;
  }
  return (int)((len + c.page - 1) / c.page);
}

// Ordered pattern of a score: larger scores have larger patterns, both zeros
// the same one.
__device__ __forceinline__ uint64_t ordered(double s) {
  const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// Keys of the pages.  A block takes 64 pages of one (sequence, head), a warp 8
// of them; a lane holds NCH chunks of 8 entries of [Q-, Q+] in registers
// against the same entries of the page's [lo, hi].  VEC: 16-byte loads.
template <int NCH, bool VEC>
__global__ void __launch_bounds__(kThreads) score_kernel(SelectArgs a, int dt) {
  __shared__ double s_q[2 * 512];
  const PagedCache& c = a.c;
  const int64_t b = blockIdx.y;
  const int head = blockIdx.z, D = c.dim, n = pages_of(c, b);
  const int p_block = blockIdx.x * kWarps * kPagesPerWarp;
  if (p_block >= n) return;
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    double neg = 0.0, pos = 0.0;
    const int64_t at = b * a.q_stride + (int64_t)head * a.group * D + ch;
    for (int g = 0; g < a.group; ++g) {
      const double x = (double)q_at(a.q, dt, at + (int64_t)g * D);
      if (x < 0.0) neg += x;
      else pos += x;
    }
    s_q[ch] = neg;
    s_q[D + ch] = pos;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double w[NCH][8];
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (lane + 32 * j) * 8 + i;
      w[j][i] = e < 2 * D ? s_q[e] : 0.0;
    }
  uint64_t* keys = a.keys + (b * c.heads + head) * c.max_pages;
  const int32_t* table = c.page_table + b * c.max_pages;
  [[maybe_unused]] const int64_t n_bounds = c.num_pages * c.heads;
#pragma unroll 2
  for (int i = 0; i < kPagesPerWarp; ++i) {
    const int p = p_block + i * kWarps + warp;
    if (p >= n) break;
    const int64_t page = __ldg(table + p);
    const bool ok = page >= 0 && page < c.num_pages;
    double s = 0.0;
    if (ok && MXQ_IN_RANGE(kChkSelectIn, page * c.heads + head, n_bounds)) {
      const uint16_t* row = a.bounds + (page * c.heads + head) * 2 * D;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int e = (lane + 32 * j) * 8;
        if (e >= 2 * D) continue;
        uint32_t bits[8];
        if constexpr (VEC) {
          load8<kBF16>(row + e, 0, bits);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) bits[x] = e + x < 2 * D ? row[e + x] : 0u;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) s = fma((double)elem_to_f32<kBF16>(bits[x]), w[j][x], s);
      }
    } else if (!ok && lane == 0 && c.status) {
      *c.status = MXQ_ERR_BAD_PAGE;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const bool keep = p < a.keep_first || p >= n - a.keep_last;
    if (lane == 0 && MXQ_IN_RANGE(kChkSelectWs, p, c.max_pages))
      keys[p] = keep ? ~0ull : ok ? ordered(s) : 0ull;
  }
}

// The top largest of n keys, equal ones from the front, in ascending order of
// their places.  The smallest chosen key is found by 8-bit digits from the
// top: after each digit only the keys that share the chosen prefix matter, and
// once that whole prefix is taken the lower digits do not.
__global__ void __launch_bounds__(kThreads) select_kernel(SelectArgs a) {
  __shared__ int s_hist[256];
  __shared__ int s_digit, s_need, s_all;
  __shared__ int s_gt[kWarps], s_eq[kWarps];
  const PagedCache& c = a.c;
  const int64_t b = blockIdx.y;
  const int head = blockIdx.x, n = pages_of(c, b), top = a.top;
  const uint64_t* keys = a.keys + (b * c.heads + head) * c.max_pages;
  int32_t* out = a.selected + (b * c.heads + head) * top;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (n <= top) {
    for (int i = threadIdx.x; i < top; i += kThreads) out[i] = i < n ? i : -1;
    return;
  }
  uint64_t prefix = 0, mask = 0;
  int need = top;  // of the keys that share the prefix
  for (int shift = 56; shift >= 0; shift -= 8) {
    s_hist[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < n; p += kThreads) {
      const uint64_t k = keys[p];
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {  // the digit where the count from above reaches need
      int local[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) local[i] = s_hist[255 - (lane * 8 + i)], sum += local[i];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
      if (before < need && before + sum >= need) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && before + local[i] >= need) {
            s_digit = 255 - (lane * 8 + i);
            s_need = need - before;
            s_all = before + local[i] == need;
          }
          before += local[i];
        }
      }
    }
    __syncthreads();
    prefix |= (uint64_t)s_digit << shift;
    mask |= 255ull << shift;
    need = s_need;
    const bool all = s_all != 0;
    __syncthreads();
    if (all) break;
  }
  // every key above the prefix, and the first `need` that share it
  const int per = (n + kThreads - 1) / kThreads, p0 = min(n, (int)threadIdx.x * per),
            p1 = min(n, p0 + per);
  int gt = 0, eq = 0;
  for (int p = p0; p < p1; ++p) {
    const uint64_t k = keys[p] & mask;
    gt += k > prefix;
    eq += k == prefix;
  }
  int sg = gt, se = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int yg = __shfl_up_sync(0xffffffffu, sg, o), ye = __shfl_up_sync(0xffffffffu, se, o);
    if (lane >= o) sg += yg, se += ye;
  }
  if (lane == 31) s_gt[warp] = sg, s_eq[warp] = se;
  __syncthreads();
  int bg = sg - gt, be = se - eq;
  for (int i = 0; i < warp; ++i) bg += s_gt[i], be += s_eq[i];
  for (int p = p0; p < p1; ++p) {
    const uint64_t k = keys[p] & mask;
    const int at = bg + min(be, need);
    const bool take = k > prefix || (k == prefix && be < need);
    if (take && MXQ_IN_RANGE(kChkSelectOut, at, top)) out[at] = p;
    bg += k > prefix;
    be += k == prefix;
  }
}

template <int NCH>
void launch_score(const SelectArgs& a, int dt, bool vec, dim3 grid, cudaStream_t st) {
  if (vec) score_kernel<NCH, true><<<grid, kThreads, 0, st>>>(a, dt);
  else score_kernel<NCH, false><<<grid, kThreads, 0, st>>>(a, dt);
}

}  // namespace

int launch_select_cache_pages(const void* q, int dt, int64_t q_heads, int64_t q_stride,
                              const void* bounds, const PagedCache& c, int64_t top,
                              int64_t keep_first, int64_t keep_last, int32_t* selected,
                              uint64_t* keys, cudaStream_t st) {
  const SelectArgs all{q,        (const uint16_t*)bounds, c,
                       q_stride, (int)(q_heads / c.heads), (int)top,
                       (int)keep_first, (int)keep_last,   selected,
                       keys};
  const bool vec = c.dim % 4 == 0 && ((uintptr_t)bounds & 15) == 0;
  const int64_t per = kWarps * kPagesPerWarp;
  const int esize = dt == kF32 ? 4 : 2;
  // grid.y ends at 65535: longer batches go in parts
  for (int64_t b = 0; b < c.n_seqs; b += 65535) {
    SelectArgs a = all;
    a.q = (const char*)q + b * q_stride * esize;
    a.c.page_table += b * c.max_pages;
    a.c.lengths += b;
    a.c.n_seqs = c.n_seqs - b < 65535 ? c.n_seqs - b : 65535;
    a.selected += b * c.heads * top;
    a.keys += b * c.heads * c.max_pages;
    const dim3 grid((unsigned)((c.max_pages + per - 1) / per), (unsigned)a.c.n_seqs,
                    (unsigned)c.heads);
    if (c.dim <= 128) launch_score<1>(a, dt, vec, grid, st);
    else if (c.dim <= 256) launch_score<2>(a, dt, vec, grid, st);
    else launch_score<4>(a, dt, vec, grid, st);
    select_kernel<<<dim3((unsigned)c.heads, (unsigned)a.c.n_seqs), kThreads, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

MXQ_DEFINE_CHECK_READER(check_record_cache_select)

}  // namespace mxq

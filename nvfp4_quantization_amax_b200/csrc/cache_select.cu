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
#include "sm100_primitives.cuh"

namespace mxq {

namespace {

constexpr int kThreads = 128;
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

// The bf16 in the upper half of v, times 2^-896: its bits in a double's fields,
// exactly so for every finite one (zeros and subnormals too), without the
// conversion unit, which would bound the kernel.
__device__ __forceinline__ double small_double(uint32_t v) {
  return __hiloint2double((int)((v & 0x80000000u) | ((v >> 3) & 0x0FFFE000u)), 0);
}

// Keys of the pages.  A block takes 32 pages of one (sequence, head), a warp 8
// of them at once; a lane holds NCH chunks of 8 entries of [Q-, Q+] in
// registers against the same entries of the pages' [lo, hi].  The loads of the
// first chunk are under way while the block sums its queries: the chain of
// length, page and bounds is what a block waits for.  VEC: 16-byte loads.
template <int NCH, bool VEC>
__global__ void __launch_bounds__(kThreads) score_kernel(SelectArgs a, int dt) {
  __shared__ double s_q[2 * 512];
  const PagedCache& c = a.c;
  const int64_t b = blockIdx.y;
  const int head = blockIdx.z, D = c.dim, n = pages_of(c, b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x * kWarps * kPagesPerWarp >= n) return;
  uint64_t* keys = a.keys + (b * c.heads + head) * c.max_pages;
  [[maybe_unused]] const int64_t n_bounds = c.num_pages * c.heads;
  const int p0 = (blockIdx.x * kWarps + warp) * kPagesPerWarp;
  int mine = -1;  // the page of p0 + lane, or -1
  if (lane < kPagesPerWarp && p0 + lane < n &&
      MXQ_IN_RANGE(kChkSelectTable, p0 + lane, c.max_pages)) {
    mine = __ldg(c.page_table + b * c.max_pages + p0 + lane);
    if (mine < 0 || mine >= c.num_pages) {
      mine = -1;
      if (c.status) *c.status = MXQ_ERR_BAD_PAGE;
    }
  }
  int page[kPagesPerWarp];
#pragma unroll
  for (int i = 0; i < kPagesPerWarp; ++i) page[i] = __shfl_sync(0xffffffffu, mine, i);
  uint32_t bits[kPagesPerWarp][4];
  auto load = [&](int j) {
    const int e = (lane + 32 * j) * 8;
#pragma unroll
    for (int i = 0; i < kPagesPerWarp; ++i) {
      const int64_t at = (int64_t)page[i] * c.heads + head;
      const bool ok = page[i] >= 0 && e < 2 * D && MXQ_IN_RANGE(kChkSelectIn, at, n_bounds);
      const uint16_t* from = a.bounds + at * 2 * D + e;
      if constexpr (VEC) {
        const uint4 v = ok ? ld_stream_v4(from) : make_uint4(0u, 0u, 0u, 0u);
        bits[i][0] = v.x, bits[i][1] = v.y, bits[i][2] = v.z, bits[i][3] = v.w;
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          bits[i][x] = (ok && e + 2 * x < 2 * D ? from[2 * x] : 0u) |
                       (ok && e + 2 * x + 1 < 2 * D ? (uint32_t)from[2 * x + 1] << 16 : 0u);
      }
    }
  };
  load(0);
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    double neg = 0.0, pos = 0.0;
    const int64_t at = b * a.q_stride + (int64_t)head * a.group * D + ch;
#pragma unroll 4
    for (int g = 0; g < a.group; ++g) {
      if (!MXQ_IN_RANGE(kChkSelectQuery, at + (int64_t)g * D,
                        (c.n_seqs - 1) * a.q_stride + (int64_t)c.heads * a.group * D))
        continue;
      const double x = (double)q_at(a.q, dt, at + (int64_t)g * D);
      neg += x < 0.0 ? x : 0.0;
      pos += x < 0.0 ? 0.0 : x;
    }
    s_q[ch] = neg * 0x1p800;  // against small_double's 2^-896
    s_q[D + ch] = pos * 0x1p800;
  }
  __syncthreads();
  double s[kPagesPerWarp];
#pragma unroll
  for (int i = 0; i < kPagesPerWarp; ++i) s[i] = 0.0;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    if (j > 0) load(j);
    const int e = (lane + 32 * j) * 8;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const double w0 = e + 2 * x < 2 * D ? s_q[e + 2 * x] : 0.0;
      const double w1 = e + 2 * x + 1 < 2 * D ? s_q[e + 2 * x + 1] : 0.0;
#pragma unroll
      for (int i = 0; i < kPagesPerWarp; ++i) {
        s[i] = fma(small_double(bits[i][x] << 16), w0, s[i]);
        s[i] = fma(small_double(bits[i][x]), w1, s[i]);
      }
    }
  }
  // the lanes' sums of 8 pages: three halvings leave a page to each 4 lanes
#pragma unroll
  for (int half = kPagesPerWarp / 2, o = 16; half > 0; half >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const double give = up ? s[i] : s[i + half], keep = up ? s[i + half] : s[i];
      s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
  s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
  const int of = (lane & 16 ? 4 : 0) + (lane & 8 ? 2 : 0) + (lane & 4 ? 1 : 0), p = p0 + of;
  const bool ok = __shfl_sync(0xffffffffu, mine, of) >= 0;
  if ((lane & 3) == 0 && p < n && MXQ_IN_RANGE(kChkSelectWs, p, c.max_pages)) {
    const bool keep = p < a.keep_first || p >= n - a.keep_last;
    keys[p] = keep ? ~0ull : ok ? ordered(s[0]) : 0ull;
  }
}

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHeld = 8;  // keys a thread holds in registers: 4096 pages in all

// The top largest of n keys, equal ones from the front, in ascending order of
// their places.  The smallest chosen key is found by 8-bit digits from the
// highest bit in which keys differ (above it all would count into one place):
// after each digit only the keys that share the chosen prefix matter, and once
// that whole prefix is taken the lower digits do not.  A thread holds the
// keys of kHeld places that follow one another; where there are more, the
// rest are read again for each digit.
__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
  __shared__ int s_hist[2][256];
  __shared__ int s_digit, s_need, s_all;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  __shared__ uint64_t s_differ[kSelWarps];
  const PagedCache& c = a.c;
  const int64_t b = blockIdx.y;
  const int head = blockIdx.x, n = pages_of(c, b), top = a.top;
  const uint64_t* keys = a.keys + (b * c.heads + head) * c.max_pages;
  int32_t* out = a.selected + (b * c.heads + head) * top;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 256) s_hist[0][threadIdx.x] = 0;
  if (n <= top) {
    for (int i = threadIdx.x; i < top; i += kSelThreads) out[i] = i < n ? i : -1;
    sm100::griddep_wait();  // the scores' kernel has its end before this one's
    return;
  }
  sm100::griddep_wait();
  const bool held = n <= kSelThreads * kHeld;
  const int per = held ? kHeld : (n + kSelThreads - 1) / kSelThreads;
  const int p0 = min(n, (int)threadIdx.x * per), p1 = min(n, p0 + per);
  uint64_t k8[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    k8[i] = held && p0 + i < p1 && MXQ_IN_RANGE(kChkSelectWs, p0 + i, c.max_pages) ? keys[p0 + i]
                                                                                   : 0ull;
  auto each = [&](auto f) {  // f(place, key) of this thread's places in order
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (p0 + i < p1) f(p0 + i, k8[i]);
    } else {
      for (int p = p0; p < p1; ++p)
        if (MXQ_IN_RANGE(kChkSelectWs, p, c.max_pages)) f(p, keys[p]);
    }
  };
  // the bits in which the scored keys differ, and how many pages are kept anyway
  const uint64_t some = keys[min(a.keep_first, n - 1)];
  uint64_t differ = 0;
  int kept = 0;
  each([&](int, uint64_t k) {
    if (k == ~0ull) ++kept;
    else differ |= k ^ some;
  });
  const uint32_t dh = __reduce_or_sync(0xffffffffu, (uint32_t)(differ >> 32)),
                 dl = __reduce_or_sync(0xffffffffu, (uint32_t)differ);
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (lane == 0) {
    s_differ[warp] = (uint64_t)dh << 32 | dl;
    s_gt[warp] = kept;
  }
  __syncthreads();
  differ = 0;
  int need = top;  // of the keys that share the prefix
  for (int i = 0; i < kSelWarps; ++i) differ |= s_differ[i], need -= s_gt[i];
  int low = 64 - __clzll((long long)differ);  // bits still open
  uint64_t mask = low == 64 ? 0ull : ~0ull << low, prefix = some & mask;
  if (need <= 0) {  // only pages that are kept anyway
    low = 0;
    mask = prefix = ~0ull;
    need = top;
  }
  for (int turn = 0; low > 0; turn ^= 1) {
    const int width = min(8, low), shift = low - width;
    const uint32_t digits = (1u << width) - 1;
    int* hist = s_hist[turn];
    each([&](int, uint64_t k) {
      if ((k & mask) == prefix && k != ~0ull) atomicAdd(&hist[(uint32_t)(k >> shift) & digits], 1);
    });
    if (threadIdx.x < 256) s_hist[turn ^ 1][threadIdx.x] = 0;
    __syncthreads();
    if (warp == 0) {  // the digit where the count from above reaches need
      int local[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) local[i] = hist[255 - (lane * 8 + i)], sum += local[i];
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
    low = shift;
    mask = ~0ull << low;
    need = s_need;
    if (s_all) break;
  }
  // every key above the prefix, and the first `need` that share it
  int gt = 0, eq = 0;
  each([&](int, uint64_t k) {
    gt += (k & mask) > prefix;
    eq += (k & mask) == prefix;
  });
  int sg = gt, se = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int yg = __shfl_up_sync(0xffffffffu, sg, o), ye = __shfl_up_sync(0xffffffffu, se, o);
    if (lane >= o) sg += yg, se += ye;
  }
  __syncthreads();  // the kept pages' counts have been read
  if (lane == 31) s_gt[warp] = sg, s_eq[warp] = se;
  __syncthreads();
  int bg = sg - gt, be = se - eq;
  for (int i = 0; i < warp; ++i) bg += s_gt[i], be += s_eq[i];
  each([&](int p, uint64_t key) {
    const uint64_t k = key & mask;
    const int at = bg + min(be, need);
    const bool take = k > prefix || (k == prefix && be < need);
    if (take && MXQ_IN_RANGE(kChkSelectOut, at, top)) out[at] = p;
    bg += k > prefix;
    be += k == prefix;
  });
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
    if (cudaGetLastError() != cudaSuccess) return MXQ_ERR_CUDA;  // there are no scores to choose by
    // launched with programmatic stream serialization: it looks up its
    // sequence while the scores' last blocks run
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.heads, (unsigned)a.c.n_seqs);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, select_kernel, a) != cudaSuccess) {
      (void)cudaGetLastError();  // reported here
      return MXQ_ERR_CUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

MXQ_DEFINE_CHECK_READER(check_record_cache_select)

}  // namespace mxq

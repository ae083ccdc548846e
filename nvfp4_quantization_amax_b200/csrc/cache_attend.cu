// Attention of one new token over a paged packed cache (sm_100a): the general
// kernel for any head size, block size, page size and alignment, and the join
// of the parts of pairs that were split (see cache_attend.cuh).
//
// General kernel: a warp takes 4 tokens x 8 heads (8 x 4, 16 x 2 for wide heads)
// at a time, lanes hold channels.  The 32 partial dot products are summed over
// the lanes by halvings, 31 shuffles that leave each lane one (token, head): it
// takes that exponential, and its weight is handed round for the values.  The
// running maximum m, sum l and weighted values o of the softmax are f32:
//   m' = max(m, s), l = l 2^(m-m') + sum 2^(s-m'), o = o 2^(m-m') + sum 2^(s-m') v.
// The warps' sums are joined in shared memory in a fixed order.
#include "cache_attend.cuh"
#include "sm100_primitives.cuh"

namespace mxq {

namespace attend {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Query heads a warp carries, by channels per lane (their queries and sums stay
// in registers), and tokens it has under way: a (token, head) for every lane.
constexpr int general_heads(int dim) { return dim <= 128 ? 8 : dim <= 256 ? 4 : 2; }

// NC channels of a row of codes, as the lane's bytes lie: NC (fp8) or NC / 2
// bytes at once where the sizes allow it (WIDE), else one by one.
template <int FMT, int NC, bool WIDE>
struct Channels {
  static constexpr int BYTES = FMT == MXQ_FMT_FP8 ? NC : NC / 2;
  static constexpr int CODES = WIDE ? (BYTES + 3) / 4 : NC, SCALES = WIDE ? 1 : NC;
  uint32_t code[CODES], scale[SCALES];

  static __device__ __forceinline__ int channel(int lane, int i) {
    return WIDE ? lane * NC + i : lane + 32 * i;
  }
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int lane, int D,
                                       int B) {
    if constexpr (WIDE) {
      if (lane * NC >= D) return;
      const uint8_t* p = codes + lane * BYTES;
      if constexpr (BYTES == 1) code[0] = *p;
      else if constexpr (BYTES == 2) code[0] = *(const uint16_t*)p;
      else if constexpr (BYTES == 4) code[0] = *(const uint32_t*)p;
      else if constexpr (BYTES == 8) *(uint2*)code = *(const uint2*)p;
      else *(uint4*)code = *(const uint4*)p;
      scale[0] = scales[lane * NC / B];
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int ch = min(lane + 32 * i, D - 1);
        code[i] = codes[FMT == MXQ_FMT_FP8 ? ch : ch / 2] >> (FMT == MXQ_FMT_FP8 ? 0 : (ch & 1) * 4);
        scale[i] = scales[ch / B];
      }
    }
  }
  // The values, exact in f32; 0 for a lane past the last channel.
  __device__ __forceinline__ void values(float* v, int lane, int D) const {
    if constexpr (WIDE) {
      const bool in = lane * NC < D;
      const float s = in ? scale_value<FMT>(scale[0]) : 0.0f;
#pragma unroll
      for (int i = 0; i < NC; i += 2) {
        const int bit = (FMT == MXQ_FMT_FP8 ? 8 : 4) * i;  // where the pair begins
        const uint32_t w = in ? code[bit / 32] >> (bit % 32) : 0u;
        const uint32_t h = FMT == MXQ_FMT_FP8 ? e4m3x2_to_f16x2(w & 0xFFFFu) : e2m1x2_to_f16x2(w & 0xFFu);
        v[i] = f16lo(h) * s;
        v[i + 1] = f16hi(h) * s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const float s = scale_value<FMT>(scale[i]);
        const uint32_t h = FMT == MXQ_FMT_FP8 ? e4m3x2_to_f16x2(code[i] & 0xFFu)
                                              : e2m1x2_to_f16x2(code[i] & 15u);
        v[i] = lane + 32 * i < D ? f16lo(h) * s : 0.0f;
      }
    }
  }
};

// NC: channels per lane (head_dim at most 32 NC); HEADS: query heads at once.
template <int FMT, int NC, int HEADS, bool WIDE>
__global__ void __launch_bounds__(kThreads) attend_general_kernel(Args a, int dt) {
  extern __shared__ float s_part[];  // [warps][heads][dim + 2]
  using Ch = Channels<FMT, NC, WIDE>;
  constexpr int TOK = 32 / HEADS;
  const PagedCache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = c.dim;
  const int rb = c.row_bytes(), nb = c.row_scales(), stride = D + 2;
  const int my_tok = lane / HEADS;  // this lane ends up with its logit of head lane % HEADS
  [[maybe_unused]] const int64_t n_rows = c.num_pages * c.heads * c.page;
  walk<kWarps>(a, [&](const Span& s, const Target& t, int v0, int v1) {
    const int r0 = t.tile * HEADS, heads = min(HEADS, a.group - r0);
    float q[HEADS][NC], o[HEADS][NC];
    float m = kLowest, l = 0.0f;  // of head lane % HEADS; l over my_tok's tokens only
#pragma unroll
    for (int r = 0; r < HEADS; ++r)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int ch = Ch::channel(lane, i);
        o[r][i] = q[r][i] = 0.0f;
        if (r < heads && ch < D)
          q[r][i] = a.scale_log2 *
                    load_q(a, dt, t.b * a.q_stride + ((int64_t)t.head * a.group + r0 + r) * D + ch);
      }
    // TOK of a warp's tokens at a time, kWarps apart
    for (int v = v0 + warp; v < v1; v += kWarps * TOK) {
      // every lane looks up its own token's row; -1: none
      int64_t row = -1;
      if (v + my_tok * kWarps < v1) {
        const Token tok = token_at(a, s, t.b, t.head, v + my_tok * kWarps);
        if (tok.row >= 0 && live(a, s, tok.pos) && MXQ_IN_RANGE(kChkAttendIn, tok.row, n_rows))
          row = tok.row;
      }
      float x[32];  // [token][head], this lane's channels' share
      constexpr int AT_ONCE = NC <= 4 ? 4 : NC <= 8 ? 2 : 1;  // tokens whose bytes are under way
      auto rows = [&](int y) { return __shfl_sync(0xffffffffu, row, y * HEADS); };
#pragma unroll
      for (int y0 = 0; y0 < TOK; y0 += AT_ONCE) {
        Ch k[AT_ONCE];
        int64_t at[AT_ONCE];
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          at[y] = max((int64_t)0, rows(y0 + y));  // no token: some row, its weight is 0
          if (v < v1) k[y].load(c.k_codes + at[y] * rb, c.k_scales + at[y] * nb, lane, D, c.block);
        }
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          float kv[NC];
          k[y].values(kv, lane, D);
#pragma unroll
          for (int r = 0; r < HEADS; ++r) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) sum = fmaf(q[r][i], kv[i], sum);
            x[(y0 + y) * HEADS + r] = sum;
          }
        }
      }
      // 32 sums over 32 lanes: halvings leave each lane the total of its own
#pragma unroll
      for (int half = 16; half > 0; half >>= 1) {
        const bool up = lane & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const float give = up ? x[i] : x[i + half], keep = up ? x[i + half] : x[i];
          x[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
        }
      }
      const float mine = row >= 0 ? x[0] : __int_as_float(0xFF800000);
      float mn = fmaxf(m, mine);
#pragma unroll
      for (int w = HEADS; w < 32; w <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
      const float keep = exp2f(m - mn), p = row >= 0 ? exp2f(mine - mn) : 0.0f;
      m = mn;
      l = fmaf(l, keep, p);
      if (__any_sync(0xffffffffu, keep != 1.0f)) {
#pragma unroll
        for (int r = 0; r < HEADS; ++r) {
          const float f = __shfl_sync(0xffffffffu, keep, r);
#pragma unroll
          for (int i = 0; i < NC; ++i) o[r][i] *= f;
        }
      }
#pragma unroll
      for (int y0 = 0; y0 < TOK; y0 += AT_ONCE) {
        Ch val[AT_ONCE];
        bool in[AT_ONCE];
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          const int64_t at = rows(y0 + y);
          in[y] = at >= 0;
          const int64_t from = max((int64_t)0, at);
          val[y].load(c.v_codes + from * rb, c.v_scales + from * nb, lane, D, c.block);
        }
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          float vv[NC];
          val[y].values(vv, lane, D);
#pragma unroll
          for (int r = 0; r < HEADS; ++r) {
            const float w = __shfl_sync(0xffffffffu, p, (y0 + y) * HEADS + r);
            if (!in[y]) continue;  // the same for all lanes
#pragma unroll
            for (int i = 0; i < NC; ++i) o[r][i] = fmaf(w, vv[i], o[r][i]);
          }
        }
      }
    }
#pragma unroll
    for (int w = HEADS; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    __syncthreads();  // the previous pair's sums have been read
#pragma unroll
    for (int r = 0; r < HEADS; ++r)
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (Ch::channel(lane, i) < D)
          s_part[(warp * HEADS + r) * stride + Ch::channel(lane, i)] = o[r][i];
    if (lane < HEADS) {
      s_part[(warp * HEADS + lane) * stride + D] = m;
      s_part[(warp * HEADS + lane) * stride + D + 1] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
      const int r = i / D, ch = i - r * D;
      float top = kLowest, sum = 0.0f, val = 0.0f;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_part[(w * HEADS + r) * stride + D]);
      for (int w = 0; w < kWarps; ++w) {
        const float* p = s_part + (w * HEADS + r) * stride;
        const float f = exp2f(p[D] - top);
        sum = fmaf(p[D + 1], f, sum);
        val = fmaf(p[ch], f, val);
      }
      put(a, dt, t, r, ch, sum > 0.0f ? val / sum : 0.0f);
      if (ch == 0) put_weight(a, t, r, sum > 0.0f ? top + log2f(sum) : kLowest);
    }
  });
}

// Join the parts of a split pair: out = sum_i o_i 2^(l_i - L), L = log2 sum
// 2^l_i.  `per_head` warps share a head's parts (a power of two, set by how
// many there can be), lanes hold VEC channels at a time; the warps' sums are
// added in a fixed order.  One block per (pair, some heads of the tile), which
// finds the pair's parts among the slots, or, where there are more pairs than
// blocks of the line, per (block of the line, some heads): such a block joins
// the split pair that begins there.
template <int VEC, int NC>
__global__ void __launch_bounds__(kThreads)
join_kernel(Args a, int dt, int n_ctas, int per_head, bool by_pair) {
  extern __shared__ float s_part[];  // [warps][dim + 1]
  __shared__ int s_first, s_count;
  const int D = a.c.dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_first = -1, s_count = 0;
  sm100::griddep_wait();
  const int pair1 = by_pair ? (int)blockIdx.x + 1 : a.hdr[2 * blockIdx.x + 1];
  if (pair1 == 0) return;
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < n_ctas; i += kThreads) {
    const int2 h = ((const int2*)a.hdr)[i];
    if (h.y == pair1) s_first = i;
    if (h.x == pair1) atomicAdd(&s_count, 1);
  }
  __syncthreads();
  const int cta = s_first, parts = 1 + s_count;  // the blocks from cta on
  if (cta < 0) return;                           // not split
  const int64_t pairs = (int64_t)a.c.heads * a.head_tiles, pair = pair1 - 1;
  Target t;
  t.b = pair / pairs;
  const int pl = (int)(pair - t.b * pairs);
  t.head = pl / a.head_tiles;
  t.tile = pl - t.head * a.head_tiles;
  t.whole = true;
  t.slot = 0;
  const int r = (blockIdx.y * kWarps + warp) / per_head, share = warp & (per_head - 1);
  const bool have = r < min(a.tile_heads, a.group - t.tile * a.tile_heads);
  auto place = [&](int i) {
    return (int64_t)(i == 0 ? 2 * cta + 1 : 2 * (cta + i)) * a.tile_heads + r;
  };
  float top = kLowest, sum = 0.0f, val[NC][VEC];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k) val[j][k] = 0.0f;
  if (have) {
    // the first parts' sums are under way with all parts' weights
    constexpr int AHEAD = NC <= 2 ? 8 / NC : 2;
    float x[AHEAD][NC][VEC];
    auto load = [&](int i, float (*to)[VEC]) {
      const float* from = a.part_o + place(i) * D;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int ch = (lane + 32 * j) * VEC;
        if (ch >= D) continue;
        if constexpr (VEC == 4) *(float4*)to[j] = *(const float4*)(from + ch);
        else to[j][0] = from[ch];
      }
    };
    auto add = [&](int i, float (*from)[VEC]) {
      const float l = a.part_l[place(i)], f = l <= kLowest ? 0.0f : exp2f(l - top);
      sum += f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if ((lane + 32 * j) * VEC < D) val[j][k] = fmaf(from[j][k], f, val[j][k]);
    };
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, a.part_l[place(i)]);
#pragma unroll
    for (int y = 0; y < AHEAD; ++y)
      if (share + y * per_head < parts) load(share + y * per_head, x[y]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    for (int i = share; i < parts; i += per_head * AHEAD) {
#pragma unroll
      for (int y = 0; y < AHEAD; ++y)
        if (i + y * per_head < parts) add(i + y * per_head, x[y]);
#pragma unroll
      for (int y = 0; y < AHEAD; ++y)
        if (i + (AHEAD + y) * per_head < parts) load(i + (AHEAD + y) * per_head, x[y]);
    }
  }
  float* mine = s_part + warp * (D + 1);
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if ((lane + 32 * j) * VEC < D) mine[(lane + 32 * j) * VEC + k] = val[j][k];
  if (lane == 0) mine[D] = sum;
  __syncthreads();
  if (!have || share != 0) return;
  for (int w = 1; w < per_head; ++w) {
    const float* other = mine + w * (D + 1);
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if ((lane + 32 * j) * VEC < D) val[j][k] += other[(lane + 32 * j) * VEC + k];
    sum += other[D];
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int ch = (lane + 32 * j) * VEC + k;
      if (ch < D) put(a, dt, t, r, ch, val[j][k] * inv);
    }
  if (lane == 0) put_weight(a, t, r, sum > 0.0f ? top + log2f(sum) : kLowest);
}

// Launched with programmatic stream serialization: it takes its place while
// the attention kernel's last blocks run and waits for them on the device.
int launch_join(const Args& a, int dt, int grid, cudaStream_t st) {
  const int64_t pairs = a.c.n_seqs * a.c.heads * a.head_tiles;
  const bool by_pair = pairs <= grid;
  const int64_t parts = grid / pairs + 2;  // of an average pair
  int per_head = 1;
  while (per_head < kWarps && per_head * 4 < parts) per_head *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(by_pair ? pairs : grid),
                     (unsigned)((a.tile_heads * per_head + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWarps * (a.c.dim + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a, dt, grid, per_head, by_pair); };
  cudaError_t err;
  if (a.c.dim % 4 != 0) err = go(join_kernel<1, 16>);
  else if (a.c.dim <= 128) err = go(join_kernel<4, 1>);
  else if (a.c.dim <= 256) err = go(join_kernel<4, 2>);
  else err = go(join_kernel<4, 4>);
  return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

template <int FMT>
int launch_general(const Args& a, int dt, int grid, cudaStream_t st) {
  const int smem = kWarps * a.tile_heads * (a.c.dim + 2) * 4;
  auto go = [&](auto kernel) {
    if (smem > 48 * 1024 && allow_dynamic_smem((const void*)kernel, smem) != cudaSuccess)
      return (int)MXQ_ERR_CUDA;
    kernel<<<grid, kThreads, smem, st>>>(a, dt);
    return (int)MXQ_OK;
  };
  // a lane's channels at once: they lie in one scale block, and their bytes on
  // their own size in every row
  auto wide = [&](int nc) {
    const int bytes = FMT == MXQ_FMT_FP8 ? nc : nc / 2;
    return a.c.dim % nc == 0 && a.c.block % nc == 0 && a.c.row_bytes() % bytes == 0 &&
           ((uintptr_t)a.c.k_codes | (uintptr_t)a.c.v_codes) % bytes == 0;
  };
  if (a.c.dim <= 64)
    return wide(2) ? go(attend_general_kernel<FMT, 2, general_heads(64), true>)
                   : go(attend_general_kernel<FMT, 2, general_heads(64), false>);
  if (a.c.dim <= 128)
    return wide(4) ? go(attend_general_kernel<FMT, 4, general_heads(128), true>)
                   : go(attend_general_kernel<FMT, 4, general_heads(128), false>);
  if (a.c.dim <= 256)
    return wide(8) ? go(attend_general_kernel<FMT, 8, general_heads(256), true>)
                   : go(attend_general_kernel<FMT, 8, general_heads(256), false>);
  return wide(16) ? go(attend_general_kernel<FMT, 16, general_heads(512), true>)
                  : go(attend_general_kernel<FMT, 16, general_heads(512), false>);
}

constexpr int kCtasPerSm = 4;  // at most, of any of the kernels

// Whether the tensor-core kernels have these sizes: see the header's fast path.
bool tc_fits(const Args& a) {
  const PagedCache& c = a.c;
  auto aligned = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
  if (c.dim != 64 && c.dim != 128 && c.dim != 256) return false;
  if (c.page % 16 != 0 || !aligned(c.k_codes) || !aligned(c.k_scales) || !aligned(c.v_codes) ||
      !aligned(c.v_scales))
    return false;
  // tiles of 16 tokens are counted in 31 bits
  if (c.num_pages > (((int64_t)1 << 31) - 1) / ((int64_t)c.heads * (c.page / 16))) return false;
  if (c.fmt == MXQ_FMT_NVFP4) return c.block == 16;
  if (c.fmt == MXQ_FMT_MXFP4) return c.block == 32;
  return c.block >= 32 && (c.block & (c.block - 1)) == 0;
}

int launch_tc_any(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st) {
  if (a.c.fmt == MXQ_FMT_MXFP4) return tc_mxfp4(a, dt, units, grid, st);
  if (a.c.fmt == MXQ_FMT_NVFP4) return tc_nvfp4(a, dt, units, grid, st);
  const int nb = a.c.row_scales();
  if (a.c.dim == 64) return tc_fp8_64(a, dt, nb, units, grid, st);
  if (a.c.dim == 128) return tc_fp8_128(a, dt, nb, units, grid, st);
  return tc_fp8_256(a, dt, nb, units, grid, st);
}

}  // namespace attend

// Slots of partials: two a block, of at most 16 heads of a tile each.
uint64_t attend_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  (void)q_heads, (void)kv_heads;
  const uint64_t slots = 2ull * attend::kCtasPerSm * (uint64_t)num_sms();
  return (slots * 4 + 15) / 16 * 16 + slots * 16 * (uint64_t)(head_dim + 1) * 4;
}

int launch_attend_cache_paged(const void* q, int dt, int64_t q_heads, int64_t q_stride,
                              const PagedCache& c, const int32_t* selected, int64_t top,
                              int64_t window, float softmax_scale, void* out, float* lse,
                              void* workspace, cudaStream_t st) {
  using namespace attend;
  const int64_t lim = c.max_pages * c.page;
  Args a;
  a.q = q;
  a.q_stride = q_stride;
  a.c = c;
  a.selected = selected;
  a.top = (int)top;
  a.window = (int)(window < lim ? window : 0);  // as long as the longest: none
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / c.heads);
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out;
  a.lse = lse;
  const int max_ctas = kCtasPerSm * num_sms();
  const int64_t slots = 2 * max_ctas;
  a.hdr = (int32_t*)workspace;
  a.part_l = (float*)((char*)workspace + (slots * 4 + 15) / 16 * 16);
  a.part_o = a.part_l + slots * 16;  // 16-byte aligned, as are its rows where dim % 4 == 0
  // the tensor-core kernel carries 8 heads, or 16 where that does not overfill
  // its registers (one f16 term, up to 128 channels): K and V are read once
  // for all of a tile
  const bool tc = tc_fits(a);
  a.tile_heads = !tc ? general_heads(c.dim) : a.group > 8 && dt == kBF16 && c.dim <= 128 ? 16 : 8;
  a.head_tiles = (a.group + a.tile_heads - 1) / a.tile_heads;
  // no more blocks than units that there can be
  const int64_t span = selected ? top * c.page : (a.window > 0 ? a.window + 16 : lim);
  const int64_t units = c.n_seqs * c.heads * a.head_tiles * ((span + kUnit - 1) / kUnit);
  int grid = (int)(units < max_ctas ? units : max_ctas);
  int rc;
  if (tc) rc = launch_tc_any(a, dt, units, &grid, st);
  else if (c.fmt == MXQ_FMT_FP8) rc = launch_general<MXQ_FMT_FP8>(a, dt, grid, st);
  else if (c.fmt == MXQ_FMT_MXFP4) rc = launch_general<MXQ_FMT_MXFP4>(a, dt, grid, st);
  else rc = launch_general<MXQ_FMT_NVFP4>(a, dt, grid, st);
  // a span of one unit is never split
  if (rc != MXQ_OK || span <= kUnit) return rc == MXQ_OK && cudaGetLastError() != cudaSuccess ? (int)MXQ_ERR_CUDA : rc;
  return launch_join(a, dt, grid, st);
}

MXQ_DEFINE_CHECK_READER(check_record_cache_attend)

}  // namespace mxq

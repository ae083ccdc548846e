// Attention of one new token over a paged packed cache (sm_100a): the general
// kernel for any head size, block size, page size and alignment, and the join
// of the parts of pairs that were split (see cache_attend.cuh).
//
// General kernel: the arithmetic of the tensor-core kernel (cache_attend_tc.cuh)
// where rows do not lie in whole tiles of it.  A warp takes 16 tokens at a time,
// each row read by the whole warp (as wide as its alignment allows) and decoded
// to f16 in shared memory, padded with zeros to 16 channels: K's values times
// 2^-(the row's largest scale exponent), which returns in f32 on the sums (blocks
// too far below it for f16 are read again, in bands with a largest of their
// own); V's likewise, its exponent in the token's weight (nvfp4: the values
// themselves).
// Then S = K Q^T and O^T = V^T P^T by mma.m16n8k16 from ldmatrix.
#include <type_traits>

#include "cache_attend.cuh"
#include "sm100_primitives.cuh"

namespace mxq {

namespace attend {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// NC channels of a row of codes, as the lane's bytes lie: NC (fp8) or NC / 2
// bytes at once where the sizes allow it (WIDE), else one by one.
template <int FMT, int NC, bool WIDE>
struct Channels {
  static constexpr int BYTES = FMT == MXQ_FMT_FP8 ? NC : NC / 2;
  static constexpr int CODES = WIDE ? (BYTES + 3) / 4 : NC, SCALES = WIDE ? 1 : NC;
  uint32_t code[CODES], scale[SCALES];

  // at: the lane's scale in a row (WIDE)
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int lane, int D,
                                       int B, int at) {
    if constexpr (WIDE) {
      if (lane * NC >= D) return;
      const uint8_t* p = codes + lane * BYTES;
      if constexpr (BYTES == 1) code[0] = __ldg(p);
      else if constexpr (BYTES == 2) code[0] = __ldg((const uint16_t*)p);
      else if constexpr (BYTES == 4) code[0] = __ldg((const uint32_t*)p);
      else if constexpr (BYTES == 8) *(uint2*)code = __ldg((const uint2*)p);
      else *(uint4*)code = __ldg((const uint4*)p);
      scale[0] = __ldg(scales + at);
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int ch = min(lane + 32 * i, D - 1);
        code[i] = __ldg(codes + (FMT == MXQ_FMT_FP8 ? ch : ch / 2)) >>
                  (FMT == MXQ_FMT_FP8 ? 0 : (ch & 1) * 4);
        scale[i] = __ldg(scales + ch / B);
      }
    }
  }
  // The largest scale byte (E8M0), over all lanes; BAND: of those below `lim`,
  // -1 where there is none.
  template <bool BAND = false>
  __device__ __forceinline__ int top_scale(int lane, int D, int lim = 256) const {
    int top = BAND ? -1 : 0;
    auto count = [&](int byte) {
      if (!BAND || byte < lim) top = max(top, byte);
    };
    if constexpr (WIDE) {
      if (lane * NC < D) count((int)scale[0]);
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) count((int)scale[i]);
    }
    return __reduce_max_sync(0xffffffffu, top);
  }
  // Code times 2^(OFF + scale exponent - top's) (E8M0), or times the scale
  // (nvfp4), in f16 at their channels of a row of `pad` channels; 0 behind the
  // last channel.  Factors below 2^-14 count as 0, and BAND: so do blocks whose
  // scale byte is not below `lim`.  Returns whether the lane has left out
  // codes other than zeros because their factor was below 2^-14.
  template <int OFF, bool BAND = false>
  __device__ __forceinline__ bool put(__half* row, int top, int lane, int D, int pad,
                                      int lim = 256) const {
    auto factor = [&](uint32_t byte) -> uint32_t {  // one f16
      if constexpr (FMT == MXQ_FMT_NVFP4) return e4m3x2_to_f16x2(byte) & 0xFFFFu;
      else if (BAND && (int)byte >= lim) return 0u;
      else return (uint32_t)max(0, OFF + 15 + (int)byte - top) << 10;
    };
    constexpr uint32_t kMagnitude = FMT == MXQ_FMT_FP8 ? 0x7F7F7F7Fu : 0x77777777u;
    auto low = [&](uint32_t byte) {
      return FMT != MXQ_FMT_NVFP4 && OFF + 15 + (int)byte - top <= 0;
    };
    if constexpr (WIDE) {
      if (lane * NC >= pad) return false;
      const bool in = lane * NC < D;
      const uint32_t s = in ? factor(scale[0]) * 0x00010001u : 0u;
      uint32_t h[NC / 2 < 2 ? 2 : NC / 2];
      if constexpr (NC == 2) {
        const uint32_t w = in ? code[0] : 0u;
        h[0] = FMT == MXQ_FMT_FP8 ? e4m3x2_to_f16x2(w) : e2m1x2_to_f16x2(w);
      } else {
#pragma unroll
        for (int i = 0; i < CODES; ++i) {
          uint32_t y[4];
          decode_word<FMT>(in ? code[i] : 0u, y);
#pragma unroll
          for (int j = 0; j < Codes<FMT>::kPairs; ++j)
            if (i * Codes<FMT>::kPairs + j < NC / 2) h[i * Codes<FMT>::kPairs + j] = y[j];
        }
      }
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) h[i] = hmul2(h[i], s);
      __half* to = row + lane * NC;
      if constexpr (NC == 2) *(uint32_t*)to = h[0];
      else if constexpr (NC == 4) *(uint2*)to = make_uint2(h[0], h[1]);
      else
#pragma unroll
        for (int i = 0; i < NC / 2; i += 4)
          *(uint4*)(to + 2 * i) = make_uint4(h[i], h[i + 1], h[i + 2], h[i + 3]);
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < CODES; ++i) any |= in ? code[i] & kMagnitude : 0u;
      return any != 0 && low(scale[0]);
    } else {
      bool left = false;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int ch = lane + 32 * i;
        if (ch >= pad) continue;
        const uint32_t h = FMT == MXQ_FMT_FP8 ? e4m3x2_to_f16x2(code[i] & 0xFFu)
                                              : e2m1x2_to_f16x2(code[i] & 15u);
        row[ch] = __ushort_as_half(
            (unsigned short)(ch < D ? hmul2(h & 0xFFFFu, factor(scale[i])) & 0xFFFFu : 0u));
        left |= ch < D && (h & 0x7FFFu) != 0 && low(scale[i]);
      }
      return left;
    }
  }
};

__device__ __forceinline__ void ldmatrix4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// NC: channels per lane (head_dim at most 32 NC).  Shared memory: Q [2 terms][8
// heads][pad + 8] f16, then per warp 16 rows of K or V, [16][pad + 8] f16 (8
// more than the padded channels: the eight rows of an ldmatrix lie in different
// banks), or at the end of a pair the warps' sums [8 heads][dim] f32.
template <int FMT, int NC, bool WIDE>
__global__ void __launch_bounds__(kTcThreads, NC <= 4 ? 4 : NC <= 8 ? 2 : 1)
attend_general_kernel(Args a, int dt, int pad) {
  extern __shared__ __align__(128) uint8_t s_all[];
  __shared__ float s_qf[8], s_m[kTcWarps][8], s_e[kTcWarps][8], s_l[kTcWarps][8];
  using Ch = Channels<FMT, NC, WIDE>;
  constexpr int MT = NC * 2;          // tiles of 16 channels
  constexpr int OFF = FMT == MXQ_FMT_NVFP4 ? 0 : FMT == MXQ_FMT_FP8 ? 7 : 12;
  const PagedCache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = c.dim, stride = pad + 8;
  const int g = lane >> 2, t4 = lane & 3, rb = c.row_bytes(), nb = c.row_scales();
  const int my_scale = WIDE ? min(lane * NC, D - 1) / c.block : 0;
  const bool two = dt != kBF16;  // terms of queries and weights
  [[maybe_unused]] const int64_t n_rows = c.num_pages * c.heads * c.page;
  __half* const s_q = (__half*)s_all;
  __half* const tile = s_q + 16 * stride + warp * 16 * stride;
  const uint32_t q_at = sm100::smem_addr(s_q) +
                        ((lane >> 4) * 8 * stride + (lane & 7) * stride + (lane >> 3 & 1) * 8) * 2;
  const uint32_t k_at = sm100::smem_addr(tile) + ((lane & 15) * stride + (lane >> 4) * 8) * 2;
  const uint32_t v_at = sm100::smem_addr(tile) +
                        (((lane & 7) + (lane >> 4) * 8) * stride + (lane >> 3 & 1) * 8) * 2;
  const float none = __int_as_float(0xFF800000);
  walk<kTcWarps>(a, [&](const Span& s, const Target& tg, int v0, int v1) {
    const int r0 = tg.tile * 8, heads = min(8, a.group - r0);
    // Q, scaled by a power of two to [2^13, 2^14) at its largest
    for (int r = warp; r < 8; r += kTcWarps) {
      float x[NC], top = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int ch = lane + 32 * i;
        x[i] = r < heads && ch < D
                   ? load_q(a, dt, tg.b * a.q_stride + ((int64_t)tg.head * a.group + r0 + r) * D + ch)
                   : 0.0f;
        top = fmaxf(top, fabsf(x[i]));
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const int e = top > 0.0f ? floor_log2_f32bits(__float_as_uint(top)) - 13 : 0;
      const float f1 = exp2i(-(e / 2)), f2 = exp2i(-(e - e / 2));
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int ch = lane + 32 * i;
        if (ch >= pad) continue;
        const float y = x[i] * f1 * f2;
        const __half h = __float2half_rn(y);
        s_q[r * stride + ch] = h;
        s_q[(8 + r) * stride + ch] = __float2half_rn(y - __half2float(h));
      }
      if (lane == 0) s_qf[r] = a.scale_log2 * exp2f((float)e);
    }
    __syncthreads();
    const float qf[2] = {s_qf[2 * t4], s_qf[2 * t4 + 1]};
    float o[MT][4], minus[2] = {0.0f, 0.0f}, E[2] = {kLowest, kLowest}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    bool have = false;

    for (int v = v0 + warp * kTile; v < v1; v += kTcWarps * kTile) {
      // lanes 0 .. 15 look up a token's row each; -1: none
      int64_t row = -1;
      if (lane < kTile && v + lane < v1) {
        const Token tok = token_at(a, s, tg.b, tg.head, v + lane, 1);
        if (tok.row >= 0 && live(a, s, tok.pos) && MXQ_IN_RANGE(kChkAttendIn, tok.row, n_rows))
          row = tok.row;
      }
      const unsigned live_rows = __ballot_sync(0xffffffffu, row >= 0);
      if (live_rows == 0) continue;
      // K or V into the tile; lane y's `tops` is the top scale byte of token y.
      // BAND: only blocks that lay below what token y's f16 reached with the top
      // byte that lane y gives.  Returns whether the lane has left out any.
      bool left;
      auto fetch = [&](auto band, const uint8_t* codes, const uint8_t* scales, int above) {
        constexpr bool BAND = decltype(band)::value;
        // rows whose bytes are under way (8 or 16: 15 to 60 % slower); bands are
        // rare, and take few registers
        constexpr int AT_ONCE = BAND ? 1 : 4;
        int tops = 127;
        left = false;
        __syncwarp();  // the tile's last reads are done
#pragma unroll
        for (int y0 = 0; y0 < kTile; y0 += AT_ONCE) {
          Ch x[AT_ONCE];
#pragma unroll
          for (int y = 0; y < AT_ONCE; ++y) {
            const int64_t at = __shfl_sync(0xffffffffu, row, y0 + y);
            if (at >= 0 && MXQ_IN_RANGE(kChkAttendScale, at * nb + my_scale, n_rows * nb))
              x[y].load(codes + at * rb, scales + at * nb, lane, D, c.block, my_scale);
          }
#pragma unroll
          for (int y = 0; y < AT_ONCE; ++y) {
            __half* to = tile + (y0 + y) * stride;
            if (live_rows >> (y0 + y) & 1) {
              const int lim =
                  BAND ? __shfl_sync(0xffffffffu, above, y0 + y) - OFF - 14 : 256;
              const int top =
                  FMT == MXQ_FMT_NVFP4 ? 127 : x[y].template top_scale<BAND>(lane, D, lim);
              if (lane == y0 + y) tops = top;
              left |= x[y].template put<OFF, BAND>(to, top, lane, D, pad, lim);
            } else {
              for (int ch = lane * 2; ch < pad; ch += 64) *(uint32_t*)(to + ch) = 0u;
            }
          }
        }
        __syncwarp();
        return tops;
      };
      // ---- S = K Q^T, rows tokens g, g + 8, columns heads 2 t, 2 t + 1
      float d[4];
      auto products = [&](int k_tops, float* y) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          if (k * 16 >= pad) continue;
          uint32_t f[4], q[4];
          ldmatrix4(f, k_at + k * 32);
          ldmatrix4(q, q_at + k * 32);
          mma16816(y, f, q[0], q[1]);
          if (two) mma16816(y, f, q[2], q[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float kf = exp2i(max(__shfl_sync(0xffffffffu, k_tops, g + 8 * h), 0) - 127 - OFF);
          y[2 * h] *= kf;
          y[2 * h + 1] *= kf;
        }
      };
      int k_tops = fetch(std::false_type(), c.k_codes, c.k_scales, 256);
      products(k_tops, d);
      // blocks too far below their row's largest for its f16: in bands of their own
      if constexpr (FMT != MXQ_FMT_NVFP4) {
        while (__any_sync(0xffffffffu, left)) {
          k_tops = fetch(std::true_type(), c.k_codes, c.k_scales, k_tops);
          float y[4];
          products(k_tops, y);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] += y[j];
        }
      }
      const int v_tops = fetch(std::false_type(), c.v_codes, c.v_scales, 256);
      float rf[2];  // V's exponent of tokens g and g + 8
#pragma unroll
      for (int h = 0; h < 2; ++h) rf[h] = (float)(__shfl_sync(0xffffffffu, v_tops, g + 8 * h) - 127);
      // ---- d = s - m, and the reference where one exceeds it by 2^4: then the
      // sum of the largest logit
      float over = -1.0f, raw[4];  // s is raw times qf
#pragma unroll
      for (int j = 0; j < 4; ++j) raw[j] = d[j];
      minus_times2(d, raw, minus, qf);
      minus_times2(d + 2, raw + 2, minus, qf);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!(live_rows >> (j < 2 ? g : g + 8) & 1)) d[j] = none;
        over = fmaxf(over, d[j]);
      }
      if (__any_sync(0xffffffffu, over > kLag || !have)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float sign = qf[j] < 0.0f ? -1.0f : 1.0f;
          float top = have ? -sign * minus[j] : none;
#pragma unroll
          for (int h = 0; h < 4; h += 2)
            top = fmaxf(top, d[j + h] == none ? none : sign * raw[j + h]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
          const float to = -sign * top;
          if (have) {
            const float down = (to - minus[j]) * qf[j];
            l[j] *= ex2(down);
            E[j] = fmaxf(kLowest, E[j] + down);
          }
          minus[j] = to;
#pragma unroll
          for (int h = 0; h < 4; h += 2)
            d[j + h] = d[j + h] == none ? none - top : (raw[j + h] + to) * qf[j];
        }
        have = true;
      }
      // ---- weights times 2^(11 + r), x = s - m + r - E + 11
      float x[4];
      auto relate = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = d[j] + (rf[j >> 1] + (kWeightExp - E[j & 1]));
        return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      };
      if (__any_sync(0xffffffffu, relate() > kWeightExp + kLag)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float e = fmaxf(kFloor, fmaxf(d[j] + rf[0], d[j + 2] + rf[1]));
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, w));
          const float En = fmaxf(E[j], e), fo = ex2(E[j] - En);
#pragma unroll
          for (int i = 0; i < MT; ++i) o[i][j] *= fo, o[i][j + 2] *= fo;
          E[j] = En;
        }
        relate();
      }
      uint32_t p[2][2];
      {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = ex2(x[j]);
          l[j & 1] += ex2(d[j]);
        }
        const uint32_t h0 = half2_of(y[0], y[1]), h1 = half2_of(y[2], y[3]);
        p[0][0] = sm100::movmatrix_trans(h0);
        p[0][1] = sm100::movmatrix_trans(h1);
        p[1][0] = sm100::movmatrix_trans(half2_of(y[0] - f16lo(h0), y[1] - f16hi(h0)));
        p[1][1] = sm100::movmatrix_trans(half2_of(y[2] - f16lo(h1), y[3] - f16hi(h1)));
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (i * 16 >= pad) continue;
        uint32_t f[4];
        ldmatrix4_trans(f, v_at + i * 32);
        mma16816(o[i], f, p[0][0], p[0][1]);
        if (two) mma16816(o[i], f, p[1][0], p[1][1]);
      }
    }

    // ---- join the warps: sums [warp][head][dim]
    __syncthreads();
    float* const sums = (float*)(s_all + 16 * stride * 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* to = sums + (warp * 8 + 2 * t4 + j) * D;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (i * 16 + g < D) to[i * 16 + g] = o[i][j];
        if (i * 16 + g + 8 < D) to[i * 16 + g + 8] = o[i][j + 2];
      }
      float lt = l[j];
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, w);
      if (g == 0) {
        s_m[warp][2 * t4 + j] = -minus[j] * qf[j];
        s_e[warp][2 * t4 + j] = E[j];
        s_l[warp][2 * t4 + j] = lt;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * D; i += kTcThreads) {
      const int r = i / D, ch = i - r * D;
      float top = kLowest, ref = kLowest, sum = 0.0f, val = 0.0f;
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w)
        if (s_l[w][r] != 0.0f) top = fmaxf(top, s_m[w][r]);
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w)
        if (s_l[w][r] != 0.0f) ref = fmaxf(ref, s_e[w][r] + (s_m[w][r] - top));
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w) {
        if (s_l[w][r] == 0.0f) continue;  // no token
        const float m = s_m[w][r] - top;
        sum = fmaf(s_l[w][r], exp2f(m), sum);
        val = fmaf(sums[(w * 8 + r) * D + ch], exp2f(s_e[w][r] + m - ref), val);
      }
      const float back = ref - kWeightExp - (float)OFF, half = truncf(back * 0.5f);
      put(a, dt, tg, r, ch, sum != 0.0f ? val / sum * exp2f(half) * exp2f(back - half) : 0.0f);
      if (ch == 0) put_weight(a, tg, r, top, sum);
    }
    __syncthreads();  // the buffers are the next pair's
  });
}

// Join the parts of a split pair: out = sum_i o_i w_i / sum_i w_i, w_i = l_i
// 2^(m_i - the largest m).  `per_head` warps share a head's parts (a power of two, set by how
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
  // the part's place in the workspace; one past the last slot reads the first
  auto place = [&](int i) {
    const int64_t at = (int64_t)(i == 0 ? 2 * cta + 1 : 2 * (cta + i)) * a.tile_heads + r;
    return MXQ_IN_RANGE(kChkAttendWs, at, 2ll * n_ctas * a.tile_heads) ? at : (int64_t)0;
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
      const float2 w = a.part_w[place(i)];
      const float f = w.y != 0.0f ? w.y * exp2f(w.x - top) : 0.0f;
      sum += f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if ((lane + 32 * j) * VEC < D) val[j][k] = fmaf(from[j][k], f, val[j][k]);
    };
    for (int i = lane; i < parts; i += 32) {
      const float2 w = a.part_w[place(i)];
      if (w.y != 0.0f) top = fmaxf(top, w.x);
    }
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
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;  // a NaN stays one
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int ch = (lane + 32 * j) * VEC + k;
      if (ch < D) put(a, dt, t, r, ch, val[j][k] * inv);
    }
  if (lane == 0) put_weight(a, t, r, top, sum);
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
  const cudaError_t last = cudaGetLastError();  // reported here, whichever it is
  return err == cudaSuccess && last == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

template <int FMT>
int launch_general(const Args& a, int dt, int grid, cudaStream_t st) {
  const int pad = (a.c.dim + 15) / 16 * 16;
  const int tiles = kTcWarps * 16 * (pad + 8) * 2, sums = kTcWarps * 8 * a.c.dim * 4;
  const int smem = 16 * (pad + 8) * 2 + (tiles > sums ? tiles : sums);
  auto go = [&](auto kernel) {
    if (smem > 48 * 1024 && allow_dynamic_smem((const void*)kernel, smem) != cudaSuccess)
      return (int)MXQ_ERR_CUDA;
    kernel<<<grid, kTcThreads, smem, st>>>(a, dt, pad);
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
    return wide(2) ? go(attend_general_kernel<FMT, 2, true>) : go(attend_general_kernel<FMT, 2, false>);
  if (a.c.dim <= 128)
    return wide(4) ? go(attend_general_kernel<FMT, 4, true>) : go(attend_general_kernel<FMT, 4, false>);
  if (a.c.dim <= 256)
    return wide(8) ? go(attend_general_kernel<FMT, 8, true>) : go(attend_general_kernel<FMT, 8, false>);
  return wide(16) ? go(attend_general_kernel<FMT, 16, true>) : go(attend_general_kernel<FMT, 16, false>);
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
  return (slots * 4 + 15) / 16 * 16 + slots * 16 * (uint64_t)(head_dim + 2) * 4;
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
  a.part_w = (float2*)((char*)workspace + (slots * 4 + 15) / 16 * 16);
  a.part_o = (float*)(a.part_w + slots * 16);  // 16-byte aligned, as are its rows where dim % 4 == 0
  // the tensor-core kernel carries 8 heads, or 16 where that does not overfill
  // its registers (one f16 term, up to 128 channels): K and V are read once
  // for all of a tile
  const bool tc = tc_fits(a);
  a.tile_heads = tc && a.group > 8 && dt == kBF16 && c.dim <= 128 ? 16 : 8;
  a.head_tiles = (a.group + a.tile_heads - 1) / a.tile_heads;
  a.least = tc ? 2 : 1;  // a unit of the general kernel takes several times as long
  // no more blocks than units that there can be
  const int64_t span = selected ? top * c.page : (a.window > 0 ? a.window + 16 : lim);
  const int64_t units = c.n_seqs * c.heads * a.head_tiles * ((span + kUnit - 1) / kUnit);
  int grid = (int)(units < max_ctas ? units : max_ctas);
  int rc;
  if (tc) rc = launch_tc_any(a, dt, units, &grid, st);
  else if (c.fmt == MXQ_FMT_FP8) rc = launch_general<MXQ_FMT_FP8>(a, dt, grid, st);
  else if (c.fmt == MXQ_FMT_MXFP4) rc = launch_general<MXQ_FMT_MXFP4>(a, dt, grid, st);
  else rc = launch_general<MXQ_FMT_NVFP4>(a, dt, grid, st);
  if (rc != MXQ_OK) return rc;
  if (cudaGetLastError() != cudaSuccess) return MXQ_ERR_CUDA;  // there are no parts to join
  // a span of one unit is never split
  return span <= kUnit ? (int)MXQ_OK : launch_join(a, dt, grid, st);
}

MXQ_DEFINE_CHECK_READER(check_record_cache_attend)

}  // namespace mxq

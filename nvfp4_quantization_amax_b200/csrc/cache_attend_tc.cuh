// Attention of one new token over a paged packed cache on the tensor cores
// (sm_100a): the kernel behind cache_attend_fp8_*.cu and
// cache_attend_fp4.cu.  How the work is laid over the grid is in
// cache_attend.cuh.
//
// A byte of K or V meets the G query heads of its kv head, 4 G flop with fp8:
// at G = 8 and the speed of HBM more than f32 arithmetic gives, and far less
// than the tensor cores'.  So the codes go to f16 in registers (E4M3 and E2M1
// are exact there) and through mma.m16n8k16 with f32 sums.  In fp8 the kernel
// runs at 0.73 of a copy's rate, in mxfp4 at 0.55: there no unit is saturated
// (issue slots 61 % busy, ALU 55 %, DRAM 47 % of peak), with 2.7 warps a
// scheduler each waiting for the chain of its own turn.  (tcgen05's block-scaled
// kinds would take K's codes as they are, with E8M0 scales per 32 channels and
// queries as two E4M3 terms, 128 tokens a tile and the head side, 8 wide, no
// better filled; V's scales lie across its product and leave it to be decoded.)
//
// Per warp, 16 tokens at a time (one tile; a page holds whole tiles):
//  - S = K Q^T: rows are tokens, columns 8 heads.  K comes from shared memory
//    by ldmatrix (four bytes of a row a lane), the order of the channels in the
//    sum is the codes' own and Q is laid out to match.
//  - softmax in base 2 with a running reference m that is moved only when a
//    logit exceeds it by 2^4, so most tiles need no warp maximum and no
//    rescaling of the sums.
//  - O^T = V^T P^T: rows are channels, columns heads.  A lane reads 1/8 of a
//    row of four tokens, two tokens' codes are paired byte by byte (or nibble
//    by nibble) so that one conversion gives the pair the instruction wants,
//    and P turns from S's layout to the operand's by movmatrix.
//
// Scales.  E8M0 scales (fp8, mxfp4) reach 2^+-127, beyond f16.  K: the sum over
// each scale block is multiplied by its scale in f32.  V: an exponent r joins
// the weight, 2^(s - m + r - E), with E the running largest of s - m + r (held
// from m on: beside logits of 2^28 the exponents would be lost): a token of
// huge values and no weight costs no other token its bits.  With one scale a
// row r is the token's.  With several it is the largest of the turn's tokens,
// found by a lane looking at 1/32 of their scale bytes, and what is left of a
// block's scale, 2^(k - r), multiplies the codes in f16 (exactly, as long as
// k - r >= -21); where a scale byte of the turn lies more than 20 (results of
// f16 and f32: 8) below the largest, its tokens are taken in bands of nearly one
// r, each a pass over V.
// E4M3 scales (nvfp4) times E2M1 codes are exact in f16.
//
// Rounding.  Q is scaled by a power of two into f16 and held in TERMS terms
// (one is exact for bf16 and f16; f32: 22 bits), the weights in TERMS terms:
// one f16 (2^-11, below bf16's step) for bf16 results, two (22 bits) for f16
// and f32.
//
// A warp loads its own tiles by 16-byte cp.async through STAGES buffers; the
// chunks of a row are swizzled so that ldmatrix (8 rows, one chunk) and V's
// reads (4 rows, 2 chunks) touch every bank once.
#pragma once

#include "cache_attend.cuh"
#include "sm100_primitives.cuh"

namespace mxq {
namespace attend {

// How far scale bytes of V may lie apart in a band: its tokens' largest ones.
constexpr int kSpan = 4;

// Two E8M0 bytes (low first) as f32.
__device__ __forceinline__ void e8m0x2(uint32_t two, float& lo, float& hi) {
  uint32_t b;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"((uint16_t)two));
  lo = __uint_as_float(b << 16);
  hi = __uint_as_float(b & 0xFFFF0000u);
}

// Place of 16-byte chunk `col` of row `row` in a tile of rows of CH chunks.
// ROWS8: read 8 rows of one chunk at a time (K, ldmatrix); else four rows two
// apart, the whole rows in 32-lane order (V).
template <int CH, bool ROWS8>
__host__ __device__ constexpr int place(int row, int col) {
  if (CH >= 8) return row * CH + (col ^ (row & 7));
  if (CH == 4) {
    const int line = row >> 1;
    return line * 8 + (((row & 1) * 4 + col) ^ (ROWS8 ? (line & 3) : (line & 3) << 1));
  }
  const int line = row >> 2;
  return line * 8 + (((row & 3) * 2 + col) ^ (ROWS8 ? (line & 1) : (line & 1) << 1));
}

// FMT; D: channels; NB: scales of a row; NT: tiles of 8 heads a warp carries;
// TERMS: f16 terms of queries and weights.  A warp takes U tiles of 16 tokens
// at a time: two, so that the loop's own instructions are shared and two chains
// run side by side (32 ragged sequences in fp8, when chosen: 56.0 us replayed
// against 57.8 with one; 56.1 now), or one of fp8 where two would not leave room for two buffers.
template <int FMT, int D, int NB, int NT, int TERMS>
struct Tc {
  static constexpr int RB = FMT == MXQ_FMT_FP8 ? D : D / 2;  // bytes of a row
  static constexpr int U = FMT == MXQ_FMT_FP8 && (D > 128 || NT == 2 || TERMS == 2) ? 1 : 2;
  static constexpr int CH = RB / 16;
  static constexpr int SC = 16 * NB;  // scale bytes of a tile
  static constexpr int SCALES = U * 32 * RB;               // where a buffer's scales begin
  static constexpr int STAGE = U * 2 * (16 * RB + SC);     // [tile][K, V], then their scales
  // Three blocks an SM leave 168 registers a thread: 96 x 8192 in mxfp4 took
  // 117.0 us when this was chosen (119.0 now), with four (128 registers, some
  // spilled) 121.0, with five 132.3.
  static constexpr int MIN_CTAS = NT == 1 && TERMS == 1 && D <= 128 ? 3 : 2;
  static constexpr int SMEM = (MIN_CTAS == 3 ? 74 : 110) * 1024;
  static constexpr int INFO = 32 * 16;  // bytes: a warp's ring of tile places
  static constexpr int QB = TERMS * NT * D * 16;  // bytes of Q: 8 heads of f16 in D channels
  static constexpr int FIT = ((SMEM - QB) / kTcWarps - INFO) / STAGE;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int PER_WARP = INFO + STAGES * STAGE;
  // the warps' sums at the end: [warp][head][group][value], a group's values one
  // word apart from the next's and heads 4 (mod 16) apart, so that the lanes of a
  // warp store to 32 banks
  static constexpr int GROUP = D / 8 + 1, ROW = (8 * GROUP + 11) / 16 * 16 + 4;
  static constexpr int PART = kTcWarps * 8 * NT * ROW * 4;
  static constexpr int BYTES = QB + (kTcWarps * PER_WARP > PART ? kTcWarps * PER_WARP : PART);
  static constexpr int CPL = D / 8;   // channels of V a lane holds
  static constexpr int KS = D / 16;   // k steps of S
  static constexpr int MT = D / 16;   // channel tiles of O
  // how V's scales are met: E4M3 scales that f16 holds; one E8M0 scale a row;
  // several
  static constexpr bool kAbsolute = FMT == MXQ_FMT_NVFP4;
  static constexpr bool kRow = !kAbsolute && NB == 1;
  static constexpr bool kRelative = !kAbsolute && NB > 1;
  static constexpr int B = D / NB;    // channels of a scale
  static constexpr int OFF = !kRelative ? 0 : FMT == MXQ_FMT_FP8 ? 7 : 12;
  // How far a turn's scale bytes of V may lie below its largest to be taken
  // together.  A weight is held to 2^-36 of the largest product of one and a
  // scale, the turn's: 2^-16 of a token's own for bf16 results, 2^-28 for others.
  static constexpr int BAND = TERMS == 1 ? 20 : 8;
  static_assert(STAGES >= 2 && STAGES <= 8, "too few buffers");

  // Channel of the i-th value of V that the lanes of group g hold, and where a
  // channel's sum lies in its row.
  static constexpr bool kHalves = FMT == MXQ_FMT_FP8 && D == 256;  // two reads 128 channels apart
  static __device__ __forceinline__ int channel(int g, int i) {
    return kHalves ? (i >> 4) * 128 + g * 16 + (i & 15) : g * CPL + i;
  }
  static __device__ __forceinline__ int sum_at(int ch) {
    return kHalves ? (ch >> 4 & 7) * GROUP + (ch >> 7) * 16 + (ch & 15)
                   : ch / CPL * GROUP + ch % CPL;
  }
};

template <class T, int FMT, int D, int NB, int NT, int TERMS>
__device__ __forceinline__ void attend_tc_body(const Args& a, int dt) {
  extern __shared__ __align__(128) uint8_t s_all[];
  uint8_t* const smem = s_all + T::QB;  // the warps' buffers, then their sums
  __shared__ float s_m[kTcWarps][8 * NT], s_r[kTcWarps][8 * NT], s_l[kTcWarps][8 * NT];
  __shared__ float s_qf[8 * NT], s_f[kTcWarps][8 * NT], s_back[2][8 * NT];
  constexpr int U = T::U;
  const PagedCache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  uint8_t* const mine = smem + warp * T::PER_WARP;
  int4* const info = (int4*)mine;  // two tiles (or -1), their live tokens
  const uint32_t buf0 = sm100::smem_addr(mine + T::INFO);
  const int tiles_per_page = c.page / kTile;
  [[maybe_unused]] const int64_t n_tiles = c.num_pages * c.heads * tiles_per_page;

  // this lane's places: 16-byte chunks it copies; the rows and chunks of K that
  // ldmatrix reads; tokens 2t and 2t + 1 of V (8 rows on is a constant further)
  uint32_t dst_k[T::CH / 2], dst_v[T::CH / 2], src_k[T::CH / 2], src_v[2];
  constexpr int LB = T::RB / 8 < 16 ? T::RB / 8 : 16;  // bytes of V a lane reads at once
#pragma unroll
  for (int i = 0; i < T::CH / 2; ++i) {
    const int at = lane + 32 * i, row = at / T::CH, col = at % T::CH;
    dst_k[i] = place<T::CH, true>(row, col) * 16;
    dst_v[i] = 16 * T::RB + place<T::CH, false>(row, col) * 16;
    src_k[i] = place<T::CH, true>(lane & 15, 2 * i + (lane >> 4)) * 16;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    src_v[i] = 16 * T::RB + place<T::CH, false>(2 * t4 + i, g * LB / 16) * 16 + g * LB % 16;
  constexpr int EIGHT = place<T::CH, false>(8, 0) * 16;
  const uint32_t q_at = sm100::smem_addr(s_all) + lane * 16;
  // the 16 bytes of scales it copies: [tile][K, V][chunk], over the lanes
  constexpr int SCHUNKS = U * 2 * NB, SROUNDS = (SCHUNKS + 31) / 32;
  const bool copies_scales = SCHUNKS >= 32 || lane < SCHUNKS;
  const int s_tile = SROUNDS > 1 ? 0 : (lane / (2 * NB)) % U;
  const uint8_t* const s_from =
      ((lane / NB) % 2 ? c.v_scales : c.k_scales) + (lane % NB) * 16;

  walk<kTcWarps>(a, [&](const Span& s, const Target& tg, int v0, int v1) {
    // this warp's turns: U tiles each, kTcWarps turns apart
    const int first = v0 / (kTile * U) + warp;
    const int n = max(0, ((v1 + kTile * U - 1) / (kTile * U) - first + kTcWarps - 1) / kTcWarps);
    const int r0 = tg.tile * 8 * NT;  // first head of the tile in its group

    // Places of turns i .. i + 15: the tiles' rows of the cache in tiles (or
    // -1), and the live tokens [lo, hi) of each, lo | hi << 8 in 16 bits.
    auto look_up = [&](int i) {
      if (lane >= 16) return;
      int4 p = make_int4(-1, -1, 0, 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = (first + (i + lane) * kTcWarps) * (kTile * U) + u * kTile;
        if (i + lane >= n || v >= v1) continue;
        const Token tok = token_at(a, s, tg.b, tg.head, v, kTile);
        if (tok.row < 0) continue;
        const int64_t start = a.window > 0 ? s.len - a.window : 0;
        const int lo = (int)max((int64_t)0, min((int64_t)kTile, start - tok.pos));
        const int hi = (int)max((int64_t)0, min((int64_t)kTile, s.len - tok.pos));
        if (lo >= hi || !MXQ_IN_RANGE(kChkAttendIn, tok.row / kTile, n_tiles)) continue;
        (u ? p.y : p.x) = (int)(tok.row / kTile);
        p.z |= (lo | hi << 8) << (16 * u);
      }
      info[(i + lane) & 31] = p;
    };
    uint32_t fill = buf0, use = buf0;  // the buffers to load and to read next
    auto next = [&](uint32_t at) {
      at += T::STAGE;
      return at == buf0 + T::STAGES * T::STAGE ? buf0 : at;
    };
    auto issue = [&](int i) {
      if ((i & 15) == 0) {
        look_up(i);
        __syncwarp();
      }
      const int4 p = info[i & 31];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tile = u ? p.y : p.x;
        const uint32_t bytes = tile >= 0 ? 16 : 0;
        const int64_t at = (int64_t)max(tile, 0) * (16 * T::RB) + lane * 16;
        const uint32_t dst = fill + u * (32 * T::RB);
#pragma unroll
        for (int j = 0; j < T::CH / 2; ++j)
          cp_async16(dst + dst_k[j], c.k_codes + at + 512 * j, bytes);
#pragma unroll
        for (int j = 0; j < T::CH / 2; ++j)
          cp_async16(dst + dst_v[j], c.v_codes + at + 512 * j, bytes);
      }
      if (copies_scales) {
#pragma unroll
        for (int j = 0; j < SROUNDS; ++j) {
          const int tile = (U == 2 && (SROUNDS > 1 ? j : s_tile)) ? p.y : p.x;
          cp_async16(fill + T::SCALES + (lane + 32 * j) * 16,
                     s_from + (int64_t)max(tile, 0) * T::SC, tile >= 0 ? 16 : 0);
        }
      }
      fill = next(fill);
      cp_async_commit();
    };
    // Q in the layout of the second operand of S, in shared memory: lane (g, t)
    // of a warp holds head g's channels, four (fp8) or eight (fp4) a chunk, in
    // the order of the codes; two k steps in 16 bytes.  One warp lays a tile,
    // its loads under way while the first tiles are looked up.
    const int q_head = r0 + warp * 8 + g;
    const int64_t q_from = tg.b * a.q_stride + ((int64_t)tg.head * a.group + q_head) * D;
    const bool q_mine = warp < NT && q_head < a.group;
    const bool q_wide = dt != kF32 && ((uintptr_t)a.q & 7) == 0 && (a.q_stride & 3) == 0;
    auto q_channel = [&](int k) {
      return FMT == MXQ_FMT_FP8 ? k * 16 + t4 * 4 : (k >> 1) * 32 + t4 * 8 + (k & 1) * 4;
    };
    uint2 q_raw[T::KS];  // four channels in 8 bytes
    if (q_mine && q_wide) {
#pragma unroll
      for (int k = 0; k < T::KS; ++k)
        q_raw[k] = is_q(a, q_from + q_channel(k), 4)
                       ? __ldg((const uint2*)((const uint16_t*)a.q + q_from + q_channel(k)))
                       : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < T::STAGES - 1; ++i) issue(i);

    if (warp < NT) {
      float x[T::KS][4], top = 0.0f;
      if (q_mine && q_wide) {
#pragma unroll
        for (int k = 0; k < T::KS; ++k) {
          const uint32_t h[2] = {q_raw[k].x, q_raw[k].y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool bf = TERMS == 1 || dt == kBF16;  // one term: bf16 only
            x[k][2 * j] = bf ? elem_to_f32<kBF16>(h[j] & 0xFFFFu) : f16lo(h[j]);
            x[k][2 * j + 1] = bf ? elem_to_f32<kBF16>(h[j] >> 16) : f16hi(h[j]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < T::KS; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[k][j] = q_mine ? load_q(a, dt, q_from + q_channel(k) + j) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < T::KS; ++k)
        top = max3(top, fmaxf(fabsf(x[k][0]), fabsf(x[k][1])),
                   fmaxf(fabsf(x[k][2]), fabsf(x[k][3])));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // largest magnitude to [2^13, 2^14)
      const int e = top > 0.0f ? floor_log2_f32bits(__float_as_uint(top)) - 13 : 0;
      const float f1 = exp2i(-(e / 2)), f2 = exp2i(-(e - e / 2));
#pragma unroll
      for (int k = 0; k < T::KS; k += 2) {
        uint32_t h[4], low[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = x[k + (j >> 1)][2 * (j & 1)] * f1 * f2,
                      x1 = x[k + (j >> 1)][2 * (j & 1) + 1] * f1 * f2;
          h[j] = half2_of(x0, x1);
          low[j] = half2_of(x0 - f16lo(h[j]), x1 - f16hi(h[j]));
        }
        uint4* to = (uint4*)(s_all + (warp * (T::KS / 2) + k / 2) * 512 + lane * 16);
        *to = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (TERMS == 2)
          to[NT * (T::KS / 2) * 32] = make_uint4(low[0], low[1], low[2], low[3]);
      }
      if (t4 == 0) s_qf[warp * 8 + g] = a.scale_log2 * exp2f((float)e);
    }
    __syncthreads();
    float qf[NT][2];  // of columns 2 t, 2 t + 1: softmax scale x 2^(Q's exponent)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) qf[nt][j] = s_qf[nt * 8 + 2 * t4 + j];

    // sums: l times 2^m, o times 2^(m + E - 11 - OFF); m is -minus times qf
    float o[T::MT][NT][4], minus[NT][2], E[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) minus[nt][j] = 0.0f, E[nt][j] = kLowest, l[nt][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < T::MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
    }

    constexpr uint32_t FULL = U == 2 ? 0x10001000u : 0x1000u;
    const float none = __int_as_float(0xFF800000);
    bool have = false;  // whether a token has been seen: m and E are set
    for (int i = 0; i < n; ++i) {
      cp_async_wait<T::STAGES - 2>();
      __syncwarp();
      issue(i + T::STAGES - 1);
      const uint32_t kb = use, sb = kb + T::SCALES;
      use = next(use);
      const uint32_t live_rows = (uint32_t)info[i & 31].z;
      if (live_rows == 0) continue;
      const bool part = live_rows != FULL;
      // whether a row of tile u is behind the end or before the window
      auto dead = [&](int u, int row) {
        return row < (int)(live_rows >> (16 * u) & 255) ||
               row >= (int)(live_rows >> (16 * u + 8) & 255);
      };
      if (part) {  // no bytes of dead rows count
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int j = 0; j < T::CH / 2; ++j)
            if (dead(u, (lane + 32 * j) / T::CH))
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(kb + u * (32 * T::RB) +
                                                                        dst_v[j]),
                           "r"(0)
                           : "memory");
          if constexpr (T::kAbsolute)
            for (int j = lane; j < T::SC; j += 32)
              if (dead(u, j / NB))
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(sb + (2 * u + 1) * T::SC + j),
                             "h"((uint16_t)0)
                             : "memory");
        }
        __syncwarp();
      }

      // ---- S = K Q^T: rows are tokens g, g + 8, columns heads 2 t, 2 t + 1 of 8
      float d[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t tb = kb + u * (32 * T::RB), ks = sb + 2 * u * T::SC;
        uint32_t sw0[(NB + 3) / 4], sw1[(NB + 3) / 4];  // scale bytes of tokens g, g + 8
        lds_bytes<NB>(sw0, ks + g * NB);
        lds_bytes<NB>(sw1, ks + (g + 8) * NB);
        float tmp[NT][4];
        constexpr int STEPS = Codes<FMT>::kPairs / 2;          // k steps of a chunk
        constexpr int BLK = T::kRelative ? T::B / 16 : T::KS;  // k steps of a scale block
        uint32_t abs0[T::CH], abs1[T::CH];  // nvfp4: this lane's scale of each chunk, twice
        if constexpr (T::kAbsolute) {
#pragma unroll
          for (int q4 = 0; q4 < (T::CH + 3) / 4; ++q4) {
            const uint32_t sel = t4 < 2 ? 0x6420 : 0x7531;  // 8 of a chunk's 32 channels
            constexpr int WORDS = (NB + 3) / 4;
            const int next = 2 * q4 + 1 < WORDS ? 2 * q4 + 1 : 0;  // 0: of no use
            const uint32_t x0 = __byte_perm(sw0[2 * q4], NB > 4 ? sw0[next] : 0u, sel);
            const uint32_t x1 = __byte_perm(sw1[2 * q4], NB > 4 ? sw1[next] : 0u, sel);
            uint32_t y0[2], y1[2];
            decode_word<MXQ_FMT_FP8>(x0, y0);
            decode_word<MXQ_FMT_FP8>(x1, y1);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (q4 * 4 + j < T::CH) {
                abs0[q4 * 4 + j] = __byte_perm(y0[j >> 1], 0, j & 1 ? 0x3232 : 0x1010);
                abs1[q4 * 4 + j] = __byte_perm(y1[j >> 1], 0, j & 1 ? 0x3232 : 0x1010);
              }
          }
        }
#pragma unroll
        for (int c2 = 0; c2 < T::CH; c2 += 2) {
          uint32_t w[4];
          ldmatrix4(w, tb + src_k[c2 / 2]);
          uint32_t q[TERMS][NT][2 * STEPS][2];  // of this pair of chunks' k steps
#pragma unroll
          for (int tm = 0; tm < TERMS; ++tm)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k2 = 0; k2 < STEPS; ++k2)
                lds_bytes<16>(&q[tm][nt][2 * k2][0],
                              q_at + ((tm * NT + nt) * (T::KS / 2) + c2 * STEPS / 2 + k2) * 512);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = c2 + h;
            uint32_t x0[4], x1[4];
            decode_word<FMT>(w[2 * h], x0);
            decode_word<FMT>(w[2 * h + 1], x1);
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
              const int k = col * STEPS + st;
              uint32_t f[4] = {x0[2 * st], x1[2 * st], x0[2 * st + 1], x1[2 * st + 1]};
              if constexpr (T::kAbsolute) {
                f[0] = hmul2(f[0], abs0[col]);
                f[1] = hmul2(f[1], abs1[col]);
                f[2] = hmul2(f[2], abs0[col]);
                f[3] = hmul2(f[3], abs1[col]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int tm = 0; tm < TERMS; ++tm) {
                  const uint32_t* b = q[tm][nt][h * STEPS + st];
                  if (k % BLK == 0 && tm == 0) mma16816_first(tmp[nt], f, b[0], b[1]);
                  else mma16816(tmp[nt], f, b[0], b[1]);
                }
              if (k % BLK == BLK - 1) {
                const int b = k / BLK;
                float f0 = 1.0f, f1 = 1.0f;
                if constexpr (!T::kAbsolute) {
                  float skip;
                  const int at = (b & 3) >> 1;  // half of its word
                  if (b & 1) {
                    e8m0x2(sw0[b >> 2] >> (16 * at), skip, f0);
                    e8m0x2(sw1[b >> 2] >> (16 * at), skip, f1);
                  } else {
                    e8m0x2(sw0[b >> 2] >> (16 * at), f0, skip);
                    e8m0x2(sw1[b >> 2] >> (16 * at), f1, skip);
                  }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float fj = j < 2 ? f0 : f1;
                    if constexpr (T::kAbsolute) d[u][nt][j] = tmp[nt][j];
                    else if (b == 0) d[u][nt][j] = tmp[nt][j] * fj;
                    else d[u][nt][j] = fmaf(tmp[nt][j], fj, d[u][nt][j]);
                  }
              }
            }
          }
        }
      }

      // ---- d = s - m, taken as the difference of the sums times qf: equal sums
      // are 0 apart however large their logits.  The reference moves where one
      // exceeds it by 2^4, to the sum of the largest
      float over = -1.0f, raw[U][NT][4];  // s is raw times qf
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) raw[u][nt][j] = d[u][nt][j];
          minus_times2(d[u][nt], raw[u][nt], minus[nt], qf[nt]);
          minus_times2(d[u][nt] + 2, raw[u][nt] + 2, minus[nt], qf[nt]);
          if (part) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (dead(u, j < 2 ? g : g + 8)) d[u][nt][j] = none;
          }
          over = max3(over, d[u][nt][0], d[u][nt][1]);
          over = max3(over, d[u][nt][2], d[u][nt][3]);
        }
      if (__any_sync(0xffffffffu, over > kLag || !have)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float sign = qf[nt][j] < 0.0f ? -1.0f : 1.0f;
            float top = have ? -sign * minus[nt][j] : none;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                top = fmaxf(top,
                            d[u][nt][j + 2 * h] == none ? none : sign * raw[u][nt][j + 2 * h]);
#pragma unroll
            for (int w = 4; w < 32; w <<= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float to = -sign * top;
            if (have) {
              const float down = (to - minus[nt][j]) * qf[nt][j], f = ex2(down);
              l[nt][j] *= f;
              E[nt][j] = fmaxf(kLowest, E[nt][j] + down);
              if constexpr (T::kAbsolute) {
#pragma unroll
                for (int mt = 0; mt < T::MT; ++mt) o[mt][nt][j] *= f, o[mt][nt][j + 2] *= f;
              }
            }
            minus[nt][j] = to;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                d[u][nt][j + 2 * h] = d[u][nt][j + 2 * h] == none
                                          ? none - top  // NaN where there is nothing else
                                          : (raw[u][nt][j + 2 * h] + to) * qf[nt][j];
          }
        have = true;
      }

      // ---- V's scales.  One a row: its exponent goes into the token's weight.
      // Several: the largest exponent r of the turn's tokens does, and what is
      // left, 2^(k - r), multiplies the codes; where the turn's scale bytes lie
      // far apart (`wide`), its tokens are taken in bands of nearly one r.
      float rf[U][2];                // kRow: r of tokens g and g + 8
      int r = 0, rt[U][2];           // kRelative: the band's r (a byte); tokens' own
      bool wide = false;
      if constexpr (T::kRow) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t y0, y1;
          lds_bytes<1>(&y0, sb + (2 * u + 1) * T::SC + g);
          lds_bytes<1>(&y1, sb + (2 * u + 1) * T::SC + g + 8);
          rf[u][0] = __uint_as_float(y0 | 0x4B000000u) - 8388735.0f;  // 2^23 + byte, exactly
          rf[u][1] = __uint_as_float(y1 | 0x4B000000u) - 8388735.0f;
        }
      }
      if constexpr (T::kRelative) {
        // a lane looks at its share of the turn's scale bytes of V
        constexpr int MY = U * T::SC / 32;
        static_assert(MY >= 1 && MY <= 8, "a lane's share of the scale bytes");
        uint32_t w[(MY + 3) / 4];
        const int at = lane * MY;
        lds_bytes<MY>(w, sb + (2 * (at / T::SC) + 1) * T::SC + at % T::SC);
        uint32_t hi2, lo2;
        if constexpr (MY == 1) {
          hi2 = lo2 = w[0];
        } else if constexpr (MY == 2) {
          hi2 = max(w[0] & 255u, w[0] >> 8);
          lo2 = min(w[0] & 255u, w[0] >> 8);
        } else {
          const uint32_t even = w[0] & 0x00FF00FFu, odd = (w[0] >> 8) & 0x00FF00FFu;
          hi2 = __vmaxu2(even, odd);
          lo2 = __vminu2(even, odd);
          if constexpr (MY == 8) {
            const uint32_t even1 = w[1] & 0x00FF00FFu, odd1 = (w[1] >> 8) & 0x00FF00FFu;
            hi2 = __vmaxu2(hi2, __vmaxu2(even1, odd1));
            lo2 = __vminu2(lo2, __vminu2(even1, odd1));
          }
          hi2 = max(hi2 & 0xFFFFu, hi2 >> 16);
          lo2 = min(lo2 & 0xFFFFu, lo2 >> 16);
        }
        r = (int)__reduce_max_sync(0xffffffffu, hi2);
        wide = part || __any_sync(0xffffffffu, (int)lo2 < r - T::BAND);
        if (wide) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = g + 8 * h;
              int top = -1;
              for (int j = 0; j < NB; ++j) {
                uint32_t y;
                lds_bytes<1>(&y, sb + (2 * u + 1) * T::SC + row * NB + j);
                top = max(top, (int)y);
              }
              rt[u][h] = part && dead(u, row) ? -1 : top;
            }
          int top = rt[0][0];
#pragma unroll
          for (int u = 0; u < U; ++u) top = max(top, max(rt[u][0], rt[u][1]));
          r = __reduce_max_sync(0xffffffffu, top);
        }
      }

      for (;;) {  // once, or once a band
        // ---- weights times 2^(11 + r): x = s - m + r - E + 11
        float x[U][NT][4];
        if constexpr (!T::kAbsolute) {
          auto relate = [&]() {
            float most = -1.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[2];
#pragma unroll
              for (int j = 0; j < 2; ++j)
                c[j] = (kWeightExp + (T::kRow ? 0.0f : (float)(r - 127))) - E[nt][j];
#pragma unroll
              for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  x[u][nt][j] = d[u][nt][j] + (T::kRow ? rf[u][j >> 1] + c[j & 1] : c[j & 1]);
                  if (T::kRelative && wide && (rt[u][j >> 1] > r || rt[u][j >> 1] <= r - kSpan))
                    x[u][nt][j] = none;
                }
                most = max3(most, x[u][nt][0], x[u][nt][1]);
                most = max3(most, x[u][nt][2], x[u][nt][3]);
              }
            }
            return most;
          };
          if (__any_sync(0xffffffffu, relate() > kWeightExp + kLag)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                // the column's largest s - m + r of this band
                float e = kFloor;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const bool out_of =
                        T::kRelative && wide && (rt[u][h] > r || rt[u][h] <= r - kSpan);
                    const float rr = T::kRow ? rf[u][h] : (float)(r - 127);
                    if (!out_of) e = fmaxf(e, d[u][nt][j + 2 * h] + rr);
                  }
#pragma unroll
                for (int w = 4; w < 32; w <<= 1)
                  e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, w));
                const float En = fmaxf(E[nt][j], e), fo = ex2(E[nt][j] - En);
#pragma unroll
                for (int mt = 0; mt < T::MT; ++mt) o[mt][nt][j] *= fo, o[mt][nt][j + 2] *= fo;
                E[nt][j] = En;
              }
            relate();
          }
        }
        const uint32_t rr = (uint32_t)r * 0x00010001u;

#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t vb = kb + u * (32 * T::RB), vs = sb + (2 * u + 1) * T::SC;
          uint32_t p[TERMS][NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (T::kAbsolute) {
                const float e = ex2(d[u][nt][j]);
                l[nt][j & 1] += e;
                y[j] = e * 2048.0f;
              } else {
                y[j] = ex2(x[u][nt][j]);
              }
            }
            const uint32_t h0 = half2_of(y[0], y[1]), h1 = half2_of(y[2], y[3]);
            p[0][nt][0] = sm100::movmatrix_trans(h0);
            p[0][nt][1] = sm100::movmatrix_trans(h1);
            if constexpr (TERMS == 2) {
              p[1][nt][0] = sm100::movmatrix_trans(
                  half2_of(y[0] - f16lo(h0), y[1] - f16hi(h0)));
              p[1][nt][1] = sm100::movmatrix_trans(
                  half2_of(y[2] - f16lo(h1), y[3] - f16hi(h1)));
            }
          }

          // ---- O^T += V^T P^T: tokens 2 t, 2 t + 1 and 8 more; channels of group g
          constexpr int READS = T::RB / 8 / LB, W = LB / 4;
          constexpr int PER_WORD = 2 * Codes<FMT>::kPairs;  // channels
          // words of one scale
          constexpr int SPAN = T::B / PER_WORD < W ? T::B / PER_WORD : W;
#pragma unroll
          for (int rd = 0; rd < READS; ++rd) {
            uint32_t w[4][W];  // tokens 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
            for (int k = 0; k < 4; ++k)
              lds_bytes<LB>(w[k], vb + src_v[k & 1] + (k >> 1) * EIGHT + rd * 128);
            uint32_t sc[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const int ch0 = j * PER_WORD;  // of this read
              // the scales of this lane's block: tokens (2t, 2t+1), (2t+8, 2t+9)
              if constexpr (T::kAbsolute || T::kRelative) {
                if (j % SPAN == 0) {
                  const int b = T::channel(g, rd * W * PER_WORD + ch0) / T::B;
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    uint32_t s0, s1;
                    lds_bytes<1>(&s0, vs + (2 * t4 + 8 * k) * NB + b);
                    lds_bytes<1>(&s1, vs + (2 * t4 + 1 + 8 * k) * NB + b);
                    if constexpr (T::kAbsolute) {
                      sc[k] = e4m3x2_to_f16x2(s1 * 256 + s0);
                    } else {
                      // f16 exponents k - r + OFF + 15 in both halves, within [0, OFF + 15]
                      constexpr uint32_t MOST = (T::OFF + 15) * 0x00010001u;
                      const uint32_t y = s1 * 65536 + s0 + MOST;
                      sc[k] = (wide ? __vminu2(__vmaxu2(y, rr) - rr, MOST) : y - rr) << 10;
                    }
                  }
                }
              }
              uint32_t f[2][PER_WORD];  // token pairs, channels
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t A = w[2 * k][j], Bw = w[2 * k + 1][j];
                if constexpr (FMT == MXQ_FMT_FP8) {
                  decode_word<FMT>(__byte_perm(A, Bw, 0x5140), f[k]);
                  decode_word<FMT>(__byte_perm(A, Bw, 0x7362), f[k] + 2);
                } else {
                  uint32_t even[4], odd[4];
                  decode_word<FMT>((A & 0x0F0F0F0Fu) | ((Bw << 4) & 0xF0F0F0F0u), even);
                  decode_word<FMT>(((A >> 4) & 0x0F0F0F0Fu) | (Bw & 0xF0F0F0F0u), odd);
#pragma unroll
                  for (int h = 0; h < 4; ++h) f[k][2 * h] = even[h], f[k][2 * h + 1] = odd[h];
                }
                if constexpr (T::kAbsolute || T::kRelative) {
#pragma unroll
                  for (int h = 0; h < PER_WORD; ++h) f[k][h] = hmul2(f[k][h], sc[k]);
                }
              }
#pragma unroll
              for (int h = 0; h < PER_WORD / 2; ++h) {  // two channels: one tile of O
                const uint32_t af[4] = {f[0][2 * h], f[0][2 * h + 1], f[1][2 * h], f[1][2 * h + 1]};
                const int mt = (rd * W * PER_WORD + ch0) / 2 + h;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int tm = 0; tm < TERMS; ++tm)
                    mma16816(o[mt][nt], af, p[tm][nt][0], p[tm][nt][1]);
              }
            }
          }
        }
        if constexpr (T::kRelative) {
          if (wide) {  // the next band below this one
            int top = -1;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (rt[u][h] <= r - kSpan) top = max(top, rt[u][h]);
            r = __reduce_max_sync(0xffffffffu, top);
            if (r >= 0) continue;
          }
        }
        break;
      }
      if constexpr (!T::kAbsolute) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) l[nt][j & 1] += ex2(d[u][nt][j]);
      }
    }

    // ---- join the warps
    cp_async_wait<0>();
    __syncthreads();
    float* const sums = (float*)smem;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int head = nt * 8 + 2 * t4 + j;
        float* row = sums + (warp * 8 * NT + head) * T::ROW + g * T::GROUP;
#pragma unroll
        for (int mt = 0; mt < T::MT; ++mt) {
          row[2 * mt] = o[mt][nt][j];
          row[2 * mt + 1] = o[mt][nt][j + 2];
        }
        float lt = l[nt][j];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, w);
        if (g == 0) {
          s_m[warp][head] = -minus[nt][j] * qf[nt][j];
          s_r[warp][head] = T::kAbsolute ? 0.0f : E[nt][j];
          s_l[warp][head] = lt;
        }
      }
    __syncthreads();
    const int heads = min(8 * NT, a.group - r0);
    // a warp's factor 2^(m - top + E - ref); out = sum x 2^(ref - 11 - OFF) / l,
    // the power in two steps.  A sum of 0 has seen no token; one that is not a
    // number (of a logit that is none) stays so
    const int fw = threadIdx.x / (8 * NT), fr = threadIdx.x % (8 * NT);
    if (fw < kTcWarps) {
      float top = kLowest, ref = kLowest, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w)
        if (s_l[w][fr] != 0.0f) top = fmaxf(top, s_m[w][fr]);
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w)
        if (s_l[w][fr] != 0.0f) ref = fmaxf(ref, s_r[w][fr] + (s_m[w][fr] - top));
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w)
        if (s_l[w][fr] != 0.0f) sum = fmaf(s_l[w][fr], exp2f(s_m[w][fr] - top), sum);
      s_f[fw][fr] =
          s_l[fw][fr] != 0.0f ? exp2f(s_r[fw][fr] + (s_m[fw][fr] - top) - ref) : 0.0f;
      if (fw == 0 && fr < heads) {
        const float back = ref - kWeightExp - (float)T::OFF, half = truncf(back * 0.5f);
        s_back[0][fr] = sum != 0.0f ? exp2f(half) / sum : 0.0f;
        s_back[1][fr] = sum != 0.0f ? exp2f(back - half) : 0.0f;
        put_weight(a, tg, fr, top, sum);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * D; i += kTcThreads) {
      const int r = i / D, ch = i - r * D;
      float val = 0.0f;
#pragma unroll
      for (int w = 0; w < kTcWarps; ++w)
        val = fmaf(sums[(w * 8 * NT + r) * T::ROW + T::sum_at(ch)], s_f[w][r], val);
      put(a, dt, tg, r, ch, val * s_back[0][r] * s_back[1][r]);
    }
    __syncthreads();  // the buffers are the next pair's
  });
}

template <int FMT, int D, int NB, int NT, int TERMS>
__global__ void __launch_bounds__(kTcThreads, Tc<FMT, D, NB, NT, TERMS>::MIN_CTAS)
attend_tc_kernel(Args a, int dt) {
  attend_tc_body<Tc<FMT, D, NB, NT, TERMS>, FMT, D, NB, NT, TERMS>(a, dt);
}

// Launch one instance on at most max_ctas blocks.
template <int FMT, int D, int NB, int NT, int TERMS>
int launch_tc(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st) {
  using T = Tc<FMT, D, NB, NT, TERMS>;
  auto kernel = attend_tc_kernel<FMT, D, NB, NT, TERMS>;
  if (allow_dynamic_smem((const void*)kernel, T::BYTES) != cudaSuccess) return MXQ_ERR_CUDA;
  const int64_t ctas = (int64_t)T::MIN_CTAS * num_sms();
  *grid = (int)(units < ctas ? units : ctas);
  kernel<<<*grid, kTcThreads, T::BYTES, st>>>(a, dt);
  return MXQ_OK;
}

// One format's launcher for head size D and NB scales a row.
template <int FMT, int D, int NB>
int launch_tc_dt(const Args& a, int dt, int64_t units, int* grid, cudaStream_t st) {
  if (dt != kBF16) return launch_tc<FMT, D, NB, 1, 2>(a, dt, units, grid, st);
  if constexpr (D <= 128)
    if (a.tile_heads == 16) return launch_tc<FMT, D, NB, 2, 1>(a, dt, units, grid, st);
  return launch_tc<FMT, D, NB, 1, 1>(a, dt, units, grid, st);
}

}  // namespace attend
}  // namespace mxq

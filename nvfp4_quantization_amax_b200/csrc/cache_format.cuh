// The stored cache formats, shared by the packed and the paged cache
// kernels: the scale rule of a group, its scale byte, element codes and
// their values.
#pragma once

#include "mxq_device.cuh"

namespace mxq {

template <int FMT>
struct PackedFormat;
template <>
struct PackedFormat<MXQ_FMT_FP8> {
  static constexpr int kLo = -126, kHi = 127, kQExp = 8;
  static constexpr uint32_t kQFrac = 0x600000u;  // 448 = 1.75 * 2^8
};
template <>
struct PackedFormat<MXQ_FMT_MXFP4> {
  static constexpr int kLo = -126, kHi = 127, kQExp = 2;
  static constexpr uint32_t kQFrac = 0x400000u;  // 6 = 1.5 * 2^2
};
template <>
struct PackedFormat<MXQ_FMT_NVFP4> {
  static constexpr int kLo = -9, kHi = 8, kQExp = 2;
  static constexpr uint32_t kQFrac = 0x400000u;
};

// Least k with 2^k * qmax >= amax, clamped to the format's range.  The
// fraction's excess over qmax's carries into the exponent; zeros and
// subnormals come out below the range's lower end, whatever their fraction.
template <int FMT>
__device__ __forceinline__ int group_scale_exp(uint32_t amax_f32bits) {
  using F = PackedFormat<FMT>;
  const int k = (int)((amax_f32bits + (0x7FFFFFu - F::kQFrac)) >> 23) - 127 - F::kQExp;
  return min(max(k, F::kLo), F::kHi);
}

// 2^k and 2^-k for a group's k: 2^-127, a subnormal, is the one special case.
__device__ __forceinline__ float group_scale(int k) {
  return __uint_as_float((uint32_t)(k + 127) << 23);
}
__device__ __forceinline__ float group_inverse(int k) {
  return __uint_as_float(max((uint32_t)(127 - k) << 23, 0x00400000u));
}

// Scale byte of 2^k.  E4M3 of 2^k, k in [-9, 8]: subnormal 2^(k+9) / 2^-9
// steps below 2^-6, biased exponent (k + 7) above.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(int k) {
  if constexpr (FMT == MXQ_FMT_NVFP4) {
    return k >= -6 ? (uint32_t)(k + 7) << 3 : 1u << (k + 9);
  } else {
    return (uint32_t)(k + 127);
  }
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if constexpr (FMT == MXQ_FMT_NVFP4) {
    return f16lo(e4m3x2_to_f16x2(byte));
  } else {
    return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : exp2i((int)byte - 127);
  }
}

// Element codes of eight values x * 2^-k.  fp8: E4M3 (sign of zero kept);
// fp4: E2M1 with the sign bit iff x < 0 (an addend +0 turns -0 into +0 and
// keeps the sign of a negative product that underflows).  One product an
// instruction: with two (as below, where the values are wanted too) the pack of
// 524288 rows of 512 in bf16 took 164 us against 149 (fp8/128), 149 against
// 134 (nvfp4), and as long in mxfp4.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* x, float inv) {
  if constexpr (FMT == MXQ_FMT_FP8) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = e4m3x2(x[2 * j] * inv, x[2 * j + 1] * inv);
    return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaf(x[j], inv, 0.0f);
    return make_uint2(e2m1x8(v), 0u);
  }
}

// The values of a word of codes as f16 pairs in the codes' order: two of four
// E4M3 bytes, four of eight E2M1 nibbles.  The unpacking of the word inside
// the asm lets each conversion take its byte where it lies.
template <int FMT>
struct Codes {
  static constexpr int kPairs = FMT == MXQ_FMT_FP8 ? 2 : 4;
};
template <int FMT>
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t* r) {
  if constexpr (FMT == MXQ_FMT_FP8) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(r[0]), "=r"(r[1])
        : "r"(w));
  } else {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
  }
}

// The codes and their values as f16 pairs.  Each conversion back takes what its
// conversion made, inside one asm for fp4: unpacking the four bytes of a word
// that e2m1x8 had just packed from four .b8 registers gave zeros for the upper
// bytes (nvcc 12.9; the reason is not known).  decode_word takes words that were
// read from memory or made by operations on whole registers.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* x, float inv, uint32_t* h) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v0, v1;
    if constexpr (FMT == MXQ_FMT_FP8) {
      mul2_rn(v0, v1, x[2 * j], x[2 * j + 1], inv, inv);
      b[j] = e4m3x2(v0, v1);
      h[j] = e4m3x2_to_f16x2(b[j]);
    } else {
      fma2_rn_zero(v0, v1, x[2 * j], x[2 * j + 1], inv, inv);
      asm("{\n\t.reg .b8 t;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 t, %3, %2;\n\t"
          "cvt.rn.f16x2.e2m1x2 %1, t;\n\t"
          "cvt.u32.u8 %0, t;\n\t}"
          : "=r"(b[j]), "=r"(h[j])
          : "f"(v0), "f"(v1));
    }
  }
  if constexpr (FMT == MXQ_FMT_FP8)
    return make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
  else
    return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, 0u);
}

// Eight decoded values, f16 code values (pairs) times the scale, exact in f32.
template <int FMT>
__device__ __forceinline__ void scaled8(const uint32_t* h, float s, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (FMT == MXQ_FMT_FP8)
      mul2_rn(v[2 * j], v[2 * j + 1], f16lo(h[j]), f16hi(h[j]), s, s);
    else  // zero magnitudes give +0
      fma2_rn_zero(v[2 * j], v[2 * j + 1], f16lo(h[j]), f16hi(h[j]), s, s);
  }
}
template <int FMT>
__device__ __forceinline__ void decode8(uint2 c, float s, float* v) {
  uint32_t h[4];
  decode_word<FMT>(c.x, h);
  if constexpr (FMT == MXQ_FMT_FP8) decode_word<FMT>(c.y, h + 2);
  scaled8<FMT>(h, s, v);
}

// Eight values (code times scale, exact in f32) of one (fp4) or two words.
template <int FMT>
__device__ __forceinline__ void values8(const uint32_t* w, float s, float* v) {
  uint32_t h[4];
  decode_word<FMT>(w[0], h);
  if constexpr (FMT == MXQ_FMT_FP8) decode_word<FMT>(w[1], h + 2);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    mul2_rn(v[2 * j], v[2 * j + 1], x.x, x.y, s, s);
  }
}

// The scale of a byte that stands for a finite one.
template <int FMT>
__device__ __forceinline__ float finite_scale(uint32_t byte) {
  if constexpr (FMT == MXQ_FMT_NVFP4) return f16lo(e4m3x2_to_f16x2(byte));
  else return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

template <int FMT>
__device__ __forceinline__ void store_codes(void* codes, int64_t item, uint2 c) {
  if constexpr (FMT == MXQ_FMT_FP8) {
    *(uint2*)((char*)codes + item * 8) = c;
  } else {
    *(uint32_t*)((char*)codes + item * 4) = c.x;
  }
}

template <int FMT>
__device__ __forceinline__ uint2 load_codes(const void* codes, int64_t item) {
  if constexpr (FMT == MXQ_FMT_FP8) {
    return __ldg((const uint2*)((const char*)codes + item * 8));
  } else {
    return make_uint2(__ldg((const uint32_t*)((const char*)codes + item * 4)), 0u);
  }
}

template <int DT>
__device__ __forceinline__ uint32_t elem_bits_at(const void* p, int64_t i) {
  if constexpr (ElemTraits<DT>::kBytes == 2) return ((const uint16_t*)p)[i];
  else return ((const uint32_t*)p)[i];
}

template <int DT>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (ElemTraits<DT>::kBytes == 2) ((uint16_t*)p)[i] = pack2<DT>(v, 0.0f) & 0xFFFFu;
  else ((float*)p)[i] = v;
}

}  // namespace mxq

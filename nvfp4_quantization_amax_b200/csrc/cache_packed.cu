// Packed (stored) form of the cache quantization, and its unpack, for
// sm_100a.
//
// quantize_cache rounds each group of B channels to fp8 or fp4 codes times a
// power-of-two scale 2^k and immediately multiplies back.  These kernels
// keep what that rounding produced instead: the element codes (one E4M3
// byte per element for fp8; two E2M1 nibbles per byte for mxfp4/nvfp4, the
// even channel in the low nibble) and one scale byte per group (E8M0, value
// 2^(byte-127), for fp8 and mxfp4; the E4M3 encoding of 2^k for nvfp4).
// Unpacking multiplies code by scale in f32 and rounds once to the output
// dtype, which is the arithmetic of the fake quantization, so
// unpack(pack(x)) equals quantize_cache(x) bit for bit.
//
// Layout of the fast kernels as in the fake-quantization kernel: an item is
// 8 consecutive channels (one 16-byte bf16/f16 load), B/8 lanes of a warp
// share one group and combine its maximum with xor-shuffles.
//
// Page references (title, then section):
//  "nemo_automodel.components.models.deepseek_v41.quantization":
//   _CacheQuantization.forward (fp8; mxfp4 with E8M0 scale; nvfp4 with E4M3
//   scale), quantize_cache, _power_of_two_ceiling.
//  "nemo_automodel.components.quantization.mxfp4": module docstring (low
//   nibble = even column).
#include <type_traits>

#include "cache_format.cuh"
#include "mxq.h"
#include "mxq_device.cuh"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <int DT, int FMT, int LPB>
__global__ void __launch_bounds__(kThreads)
pack_cache_kernel(const void* __restrict__ in, void* __restrict__ codes,
                  uint8_t* __restrict__ scales, int64_t n_items) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  // The items of a turn: all of them there, whose loads then go out together, or
  // only some (loads that may be left out were not all issued before the first
  // result: 524288 rows of 512 in bf16, fp8/128 183 us against 149 so, mxfp4
  // 140 against 129, nvfp4 144 against 134).
  auto turn = [&](auto all, int64_t base) {
    constexpr bool ALL = decltype(all)::value;
    uint32_t bits[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t item = base + u * stride + lane;
      if ((ALL || item < n_items) && MXQ_IN_RANGE(kChkPackIn, item, n_items))
        load8<DT>(in, item, bits[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t item = base + u * stride + lane;
      const bool valid = ALL || item < n_items;
      uint32_t m = 0;
      if (valid) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, mag_as_f32_bits<DT>(bits[u][j]));
      }
#pragma unroll
      for (int o = 1; o < LPB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (!valid) continue;
      const int k = group_scale_exp<FMT>(m);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = elem_to_f32<DT>(bits[u][j]);
      if (MXQ_IN_RANGE(kChkPackOut, item, n_items))
        store_codes<FMT>(codes, item, encode8<FMT>(x, exp2i(-k)));
      if ((lane & (LPB - 1)) == 0 && MXQ_IN_RANGE(kChkPackScale, item / LPB, n_items / LPB))
        scales[item / LPB] = (uint8_t)scale_byte<FMT>(k);
    }
  };
  for (int64_t base = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); base < n_items;
       base += stride * kUnroll) {
    if (base + (kUnroll - 1) * stride + 32 <= n_items) turn(std::true_type(), base);
    else turn(std::false_type(), base);
  }
}

template <int DT, int FMT, int LPB>
__global__ void __launch_bounds__(kThreads)
unpack_cache_kernel(const void* __restrict__ codes, const uint8_t* __restrict__ scales,
                    void* __restrict__ out, int64_t n_items) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t base = (int64_t)blockIdx.x * kThreads + threadIdx.x; base < n_items;
       base += stride * kUnroll) {
    uint2 c[kUnroll];
    uint32_t sb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t item = base + u * stride;
      if (item < n_items) {
        c[u] = MXQ_IN_RANGE(kChkUnpackIn, item, n_items) ? load_codes<FMT>(codes, item)
                                                         : make_uint2(0u, 0u);
        sb[u] = MXQ_IN_RANGE(kChkUnpackScale, item / LPB, n_items / LPB)
                    ? (uint32_t)__ldg(scales + item / LPB)
                    : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t item = base + u * stride;
      if (item >= n_items) continue;
      float v[8];
      decode8<FMT>(c[u], scale_value<FMT>(sb[u]), v);
      if (MXQ_IN_RANGE(kChkUnpackOut, item, n_items)) store8<DT>(out, item, v);
    }
  }
}

// General kernels: any block size the format allows (even for fp4), any
// alignment; channels % B == 0.  One thread per (row, group).
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads)
pack_cache_general_kernel(const void* __restrict__ in, uint8_t* __restrict__ codes,
                          uint8_t* __restrict__ scales, int64_t n_groups, int B) {
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < n_groups;
       g += (int64_t)gridDim.x * kThreads) {
    const int64_t c0 = g * B;  // groups never straddle rows (channels % B == 0)
    [[maybe_unused]] const int64_t n_el = n_groups * B;
    auto elem = [&](int64_t i) {
      return MXQ_IN_RANGE(kChkPackIn, i, n_el) ? elem_bits_at<DT>(in, i) : 0u;
    };
    uint32_t m = 0;
    for (int c = 0; c < B; ++c) m = max(m, mag_as_f32_bits<DT>(elem(c0 + c)));
    const int k = group_scale_exp<FMT>(m);
    const float inv = exp2i(-k);
    if (MXQ_IN_RANGE(kChkPackScale, g, n_groups)) scales[g] = (uint8_t)scale_byte<FMT>(k);
    for (int c = 0; c < B; c += 2) {
      const float a = elem_to_f32<DT>(elem(c0 + c));
      const float b = c + 1 < B ? elem_to_f32<DT>(elem(c0 + c + 1)) : 0.0f;
      if constexpr (FMT == MXQ_FMT_FP8) {
        const uint32_t two = e4m3x2(a * inv, b * inv);
        if (MXQ_IN_RANGE(kChkPackOut, c0 + c, n_el)) codes[c0 + c] = (uint8_t)two;
        if (c + 1 < B && MXQ_IN_RANGE(kChkPackOut, c0 + c + 1, n_el))
          codes[c0 + c + 1] = (uint8_t)(two >> 8);
      } else {
        if (MXQ_IN_RANGE(kChkPackOut, (c0 + c) / 2, n_el / 2))
          codes[(c0 + c) / 2] = (uint8_t)e2m1x2(fmaf(a, inv, 0.0f), fmaf(b, inv, 0.0f));
      }
    }
  }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads)
unpack_cache_general_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                            void* __restrict__ out, int64_t n_groups, int B) {
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < n_groups;
       g += (int64_t)gridDim.x * kThreads) {
    const int64_t c0 = g * B;
    [[maybe_unused]] const int64_t n_el = n_groups * B;
    const float s = scale_value<FMT>(MXQ_IN_RANGE(kChkUnpackScale, g, n_groups) ? scales[g] : 0u);
    for (int c = 0; c < B; ++c) {
      float v;
      if constexpr (FMT == MXQ_FMT_FP8) {
        v = f16lo(e4m3x2_to_f16x2(MXQ_IN_RANGE(kChkUnpackIn, c0 + c, n_el) ? codes[c0 + c] : 0u)) *
            s;
      } else {
        const uint32_t byte =
            MXQ_IN_RANGE(kChkUnpackIn, (c0 + c) / 2, n_el / 2) ? codes[(c0 + c) / 2] : 0u;
        const uint32_t h2 = e2m1x2_to_f16x2(((c0 + c) & 1) ? (byte >> 4) : (byte & 15u));
        v = fmaf(f16lo(h2), s, 0.0f);
      }
      if (MXQ_IN_RANGE(kChkUnpackOut, c0 + c, n_el)) store_one<DT>(out, c0 + c, v);
    }
  }
}

template <class Kernel>
int grid_over(Kernel kernel, int64_t n_units, int per_block) {
  return wave_grid((const void*)kernel, kThreads, n_units, per_block);
}

template <int DT, int FMT, int LPB>
void launch_fast(const void* in, void* codes, uint8_t* scales, void* out, bool pack,
                 int64_t n_items, cudaStream_t st) {
  const int per = kThreads * kUnroll;
  if (pack)
    pack_cache_kernel<DT, FMT, LPB><<<grid_over(pack_cache_kernel<DT, FMT, LPB>, n_items, per),
                                      kThreads, 0, st>>>(in, codes, scales, n_items);
  else
    unpack_cache_kernel<DT, FMT, LPB><<<grid_over(unpack_cache_kernel<DT, FMT, LPB>, n_items, per),
                                        kThreads, 0, st>>>(codes, scales, out, n_items);
}

template <int DT, int FMT>
void launch_fmt(const void* in, void* codes, uint8_t* scales, void* out, bool pack, int64_t rows,
                int64_t C, int B, bool fast, cudaStream_t st) {
  if (fast) {
    const int64_t n = rows * (C / 8);
    switch (B / 8) {
      case 1: launch_fast<DT, FMT, 1>(in, codes, scales, out, pack, n, st); break;
      case 2: launch_fast<DT, FMT, 2>(in, codes, scales, out, pack, n, st); break;
      case 4: launch_fast<DT, FMT, 4>(in, codes, scales, out, pack, n, st); break;
      case 8: launch_fast<DT, FMT, 8>(in, codes, scales, out, pack, n, st); break;
      case 16: launch_fast<DT, FMT, 16>(in, codes, scales, out, pack, n, st); break;
      default: launch_fast<DT, FMT, 32>(in, codes, scales, out, pack, n, st); break;
    }
    return;
  }
  const int64_t n_groups = rows * (C / B);
  if (pack)
    pack_cache_general_kernel<DT, FMT>
        <<<grid_over(pack_cache_general_kernel<DT, FMT>, n_groups, kThreads), kThreads, 0, st>>>(
            in, (uint8_t*)codes, scales, n_groups, B);
  else
    unpack_cache_general_kernel<DT, FMT>
        <<<grid_over(unpack_cache_general_kernel<DT, FMT>, n_groups, kThreads), kThreads, 0, st>>>(
            (const uint8_t*)codes, scales, out, n_groups, B);
}

template <int DT>
void launch_dt(const void* in, void* codes, uint8_t* scales, void* out, bool pack, int64_t rows,
               int64_t C, int fmt, int B, bool fast, cudaStream_t st) {
  switch (fmt) {
    case MXQ_FMT_FP8:
      launch_fmt<DT, MXQ_FMT_FP8>(in, codes, scales, out, pack, rows, C, B, fast, st);
      break;
    case MXQ_FMT_MXFP4:
      launch_fmt<DT, MXQ_FMT_MXFP4>(in, codes, scales, out, pack, rows, C, B, fast, st);
      break;
    default:
      launch_fmt<DT, MXQ_FMT_NVFP4>(in, codes, scales, out, pack, rows, C, B, fast, st);
      break;
  }
}

int launch_packed(const void* in, void* codes, uint8_t* scales, void* out, bool pack, int dt,
                  int64_t rows, int64_t C, int fmt, int B, bool fast, cudaStream_t st) {
  switch (dt) {
    case kBF16: launch_dt<kBF16>(in, codes, scales, out, pack, rows, C, fmt, B, fast, st); break;
    case kF16: launch_dt<kF16>(in, codes, scales, out, pack, rows, C, fmt, B, fast, st); break;
    default: launch_dt<kF32>(in, codes, scales, out, pack, rows, C, fmt, B, fast, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

}  // namespace

int launch_quantize_cache_packed(const void* in, int dt, int64_t rows, int64_t C, int fmt, int B,
                                 void* codes, void* scales, bool fast, cudaStream_t st) {
  return launch_packed(in, codes, (uint8_t*)scales, nullptr, true, dt, rows, C, fmt, B, fast, st);
}

int launch_dequantize_cache_packed(const void* codes, const void* scales, int64_t rows, int64_t C,
                                   int fmt, int B, void* out, int dt, bool fast, cudaStream_t st) {
  return launch_packed(nullptr, const_cast<void*>(codes), (uint8_t*)const_cast<void*>(scales),
                       out, false, dt, rows, C, fmt, B, fast, st);
}

MXQ_DEFINE_CHECK_READER(check_record_cache_packed)

}  // namespace mxq

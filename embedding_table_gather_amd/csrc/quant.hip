// Quantisation of rows to int8 with one f32 scale each: the ETG_WIRE_I8 definition
// (ADR-0009 "Wire Layout") on any f32, bf16 or f16 matrix, codes and scales in
// separate buffers, as the int8 product (imatmul.hip) reads them.
#include <algorithm>

#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

// scale = max|x| / 127, q = clamp(round-half-even(x / scale), -127, 127), both
// quotients correctly rounded f32 divisions.  A row with scale 0 has codes 0; a row
// that holds a NaN or an infinity has scale NaN and codes 0 (whatever is computed
// from it is then NaN instead of silently wrong).
//
// A row of up to 2,048 loads of 16 bytes, at any alignment, is read once and stays in
// registers until its maximum is known; a longer one is read again for its codes, from the
// caches as a rule.  Bound by the bytes, which needs the arithmetic to be short: a division
// costs about ten operations, so codes come from x * (1 / scale) instead, added to
// 1.5 * 2^23, which leaves the rounded integer in the low byte.  x * (1 / scale) is
// within 127 * 2^-22 of the quotient: where it is that near to a half step (0.02% of the
// values) the vector is divided out.  262,144 rows x 5,376 of bf16 take 745 us, 5.7 TB/s of
// reads and writes (dividing every value 2,758 us, with loads that waited for each other); 64
// rows of 1,024 take 2.7 us.
typedef u32x4 u32x4u __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2u __attribute__((aligned(1)));
typedef uint32_t u32u __attribute__((aligned(1)));

template <int DT>
struct QuantVec {
  static constexpr int N = DT == DT_F32 ? 4 : 8, SIZE = 16 / N;
  // magnitudes as f32 (f16: as f16) bit patterns, which order as the values do
  static __device__ __forceinline__ uint32_t top(const u32x4& w, uint32_t m) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (DT == DT_F32) m = max(m, w[i] & 0x7fffffffu);
      else if constexpr (DT == DT_BF16) m = max(m, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
      else m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    }
    return m;
  }
  static __device__ __forceinline__ float magnitude(uint32_t m) {
    return DT == DT_F16 ? f16_bits_to_f32(m) : __uint_as_float(m);
  }
  static __device__ __forceinline__ float value(const u32x4& w, int j) {
    if constexpr (DT == DT_F32) return __uint_as_float(w[j]);
    if constexpr (DT == DT_BF16) return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
    return f16_bits_to_f32(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
  }
};

// WPR waves per row with R loads per lane; LONG: rows of any length by pieces of that size,
// read for the maximum and again for the codes.
template <int DT, int WPR, int R, bool LONG>
__global__ void __launch_bounds__(WPR == 16 ? 1024 : 256) quantize_i8_kernel(
    const uint8_t* __restrict__ x, int64_t rows, int64_t x_stride, int cols, int8_t* __restrict__ codes,
    int64_t code_stride, float* __restrict__ scale, int64_t scale_stride) {
  using Q = QuantVec<DT>;
  constexpr int N = Q::N, T = 64 * WPR, RPB = WPR == 1 ? 4 : 1;  // rows per workgroup
  __shared__ uint32_t part[WPR == 1 ? 1 : WPR];
  const int t = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  for (int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? threadIdx.x >> 6 : 0); row < rows;
       row += (int64_t)gridDim.x * RPB) {
    const uint8_t* src = x + row * x_stride;
    u32x4 w[R];
    auto load = [&](int from) {
#pragma unroll
      for (int r = 0; r < R; r++) {
        const int c = from + (r * T + t) * N;
        w[r] = u32x4{0, 0, 0, 0};
        if (c + N <= cols) {
          const u32x4u* at = (const u32x4u*)(src + (int64_t)c * Q::SIZE);
          w[r] = LONG ? *at : __builtin_nontemporal_load(at);
        } else if (c < cols) {
#pragma unroll
          for (int j = 0; j < N; j++)
            if (c + j < cols) {
              if constexpr (DT == DT_F32) w[r][j] = ((const uint32_t*)src)[c + j];
              else w[r][j >> 1] |= (uint32_t)((const uint16_t*)src)[c + j] << (16 * (j & 1));
            }
        }
      }
    };
    uint32_t m = 0;
    for (int from = 0; from < (LONG ? cols : 1); from += R * T * N) {
      load(from);
#pragma unroll
      for (int r = 0; r < R; r++) m = Q::top(w[r], m);
    }
    m = wave_minmax_u32<true>(m);
    if constexpr (WPR > 1) {
      __syncthreads();
      if ((t & 63) == 0) part[t >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WPR; i++) m = max(m, part[i]);
    }
    const bool finite = m < (DT == DT_F16 ? 0x7c00u : 0x7f800000u);
    const float sc = finite ? Q::magnitude(m) / 127.0f : __builtin_nanf("");
    if (t == 0) scale[row * scale_stride] = sc;
    const bool some = finite && sc != 0.f;
    const float inv = some ? 1.0f / sc : 0.f;
    const bool rough = some && sc < 1.17549435e-38f;  // a subnormal scale: its reciprocal may be infinite
    int8_t* dst = codes + row * code_stride;
    for (int from = 0; from < (LONG ? cols : 1); from += R * T * N) {
      if constexpr (LONG) load(from);
#pragma unroll
      for (int r = 0; r < R; r++) {
        const int c = from + (r * T + t) * N;
        if (c >= cols) continue;
        float q[N];
        float far = 0.f;
#pragma unroll
        for (int j = 0; j < N; j++) {
          const float v = some ? Q::value(w[r], j) : 0.f;
          q[j] = fmaf(v, inv, 12582912.f);
          far = fmaxf(far, fabsf(fmaf(v, inv, 12582912.f - q[j])));
        }
        if (far > 0.4999f || rough) {
#pragma unroll
          for (int j = 0; j < N; j++)
            q[j] = 12582912.f + fminf(fmaxf(rintf(Q::value(w[r], j) / sc), -127.f), 127.f);
        }
        uint32_t out[N / 4];
#pragma unroll
        for (int j = 0; j < N / 4; j++) {
          // the low bytes of four words
          const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(q[4 * j + 1]), __float_as_uint(q[4 * j]), 0x0c0c0400u);
          const uint32_t hi =
              __builtin_amdgcn_perm(__float_as_uint(q[4 * j + 3]), __float_as_uint(q[4 * j + 2]), 0x04000c0cu);
          out[j] = lo | hi;
        }
        if (c + N <= cols) {
          if constexpr (N == 4) *(u32u*)(dst + c) = out[0];
          else *(u32x2u*)(dst + c) = u32x2{out[0], out[N / 4 - 1]};
        } else {
#pragma unroll
          for (int j = 0; j < N; j++)
            if (c + j < cols) dst[c + j] = (int8_t)(out[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
}

// x_stride in bytes
hipError_t launch_quantize_i8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                              int8_t* codes, int64_t code_stride, float* scale, int64_t scale_stride,
                              hipStream_t stream) {
#define ETG_QUANT(DT, WPR, R, LONG)                                                                                \
  hipLaunchKernelGGL((quantize_i8_kernel<DT, WPR, R, LONG>),                                                       \
                     dim3((unsigned)std::min<int64_t>(cdiv(rows, WPR == 1 ? 4 : 1), 1 << 20)),                     \
                     dim3(WPR == 16 ? 1024 : 256), 0, stream, (const uint8_t*)x, rows, x_stride, (int)cols, codes, \
                     code_stride, scale, scale_stride)
  // Measured (us, bf16): a wave per row against four, 262,144 x 1,024 153 / 295, 64 x 1,024
  // 3.0 / 2.7.  Four waves with 2, 4 or 8 loads per lane, as few as hold the row: 262,144 x
  // 4,096 562 / 671 / 922.  Sixteen waves and pieces against four waves with 8 loads:
  // 65,536 x 16,384 686 / 568; of rows of 65,536, pieces of sixteen against four waves, 1 row
  // 10.4 / 18.0, 16,384 rows 739 / 872.
#define ETG_QUANT_DT(DT)                                                 \
  {                                                                      \
    const int64_t loads = cdiv(cols, QuantVec<DT>::N);                   \
    if (loads <= 128 && rows >= 512) ETG_QUANT(DT, 1, 2, false);         \
    else if (loads <= 512) ETG_QUANT(DT, 4, 2, false);                   \
    else if (loads <= 1024) ETG_QUANT(DT, 4, 4, false);                  \
    else if (loads <= 2048) ETG_QUANT(DT, 4, 8, false);                  \
    else ETG_QUANT(DT, 16, 2, true);                                     \
  }
  if (dtype == DT_F32) ETG_QUANT_DT(DT_F32)
  else if (dtype == DT_BF16) ETG_QUANT_DT(DT_BF16)
  else ETG_QUANT_DT(DT_F16)
#undef ETG_QUANT_DT
#undef ETG_QUANT
  return hipGetLastError();
}

}  // namespace etg

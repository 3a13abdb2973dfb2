// Quantisation of rows to int8 with one f32 scale each: the ETG_WIRE_I8 definition
// (ADR-0009 "Wire Layout") on any f32, bf16 or f16 matrix, codes and scales in
// separate buffers, as the int8 product (imatmul.hip) reads them.
#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

// scale = max|x| / 127, q = clamp(round-half-even(x / scale), -127, 127), both
// quotients correctly rounded f32 divisions.  A row with scale 0 has codes 0; a row
// that holds a NaN or an infinity has scale NaN and codes 0 (whatever is computed
// from it is then NaN instead of silently wrong).
template <int DT>
__device__ __forceinline__ float quant_value(const void* row, int64_t c) {
  if constexpr (DT == DT_F32) return ((const float*)row)[c];
  if constexpr (DT == DT_BF16) return __uint_as_float((uint32_t)((const uint16_t*)row)[c] << 16);
  return f16_bits_to_f32(((const uint16_t*)row)[c]);
}

// One workgroup per row, two reads of it.
template <int DT>
__global__ void __launch_bounds__(256) quantize_i8_kernel(const uint8_t* __restrict__ x, int64_t x_stride, int cols,
                                                          int8_t* __restrict__ codes, int64_t code_stride,
                                                          float* __restrict__ scale, int64_t scale_stride) {
  __shared__ uint32_t part[4];
  const int64_t row = blockIdx.x;
  const uint8_t* src = x + row * x_stride;
  // magnitudes as bit patterns: NaN ranks above infinity, infinity above every finite value
  uint32_t m = 0;
  for (int c = threadIdx.x; c < cols; c += 256) m = max(m, __float_as_uint(quant_value<DT>(src, c)) & 0x7fffffffu);
  m = wave_minmax_u32<true>(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const bool finite = m < 0x7f800000u;
  const float sc = finite ? __uint_as_float(m) / 127.0f : __builtin_nanf("");
  if (threadIdx.x == 0) scale[row * scale_stride] = sc;
  const bool some = finite && sc != 0.f;
  for (int c = threadIdx.x; c < cols; c += 256) {
    const float q = some ? fminf(fmaxf(rintf(quant_value<DT>(src, c) / sc), -127.f), 127.f) : 0.f;
    codes[row * code_stride + c] = (int8_t)q;
  }
}

// x_stride in bytes
hipError_t launch_quantize_i8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                              int8_t* codes, int64_t code_stride, float* scale, int64_t scale_stride,
                              hipStream_t stream) {
#define ETG_QUANT(DT)                                                                                              \
  hipLaunchKernelGGL((quantize_i8_kernel<DT>), dim3((unsigned)rows), dim3(256), 0, stream, (const uint8_t*)x,      \
                     x_stride, (int)cols, codes, code_stride, scale, scale_stride)
  if (dtype == DT_F32) ETG_QUANT(DT_F32);
  else if (dtype == DT_BF16) ETG_QUANT(DT_BF16);
  else ETG_QUANT(DT_F16);
#undef ETG_QUANT
  return hipGetLastError();
}

}  // namespace etg

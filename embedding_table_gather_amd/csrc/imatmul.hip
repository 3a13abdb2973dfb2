// Matrix product in 8-bit integers with a scale per row of each operand (per token
// and per channel): out[m][n] = T( f32(sum_k a[m][k] w[n][k]) * sa[m] * sw[n] ).
// The sum is exact: |sum| <= 65536 * 128 * 128 = 2^30 fits the int32 accumulators.
// Its conversion to f32 and the two multiplications round to nearest (relative
// error at most 3 * 2^-24), the store in T once more.
#include "etg_device.hpp"
#include "etg_internal.hpp"

namespace etg {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Bytes [k, k + 16) of a code row of K bytes at any address, zero past the row.
__device__ __forceinline__ i32x4 load_codes16(const int8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 16; j++)
      if (k + j < K) v[j >> 2] |= (int)((uint32_t)(uint8_t)row[k + j] << (8 * (j & 3)));
  }
  return v;
}

template <int DT>
__device__ __forceinline__ void store_out(void* out, int64_t i, float x) {
  if constexpr (DT == DT_F32) {
    ((float*)out)[i] = x;
  } else if constexpr (DT == DT_BF16) {
    ((__bf16*)out)[i] = (__bf16)x;
  } else {
    // opaque: the compiler would fold the last multiplication into the conversion
    // (one rounding where the definition has two)
    asm volatile("" : "+v"(x));
    ((_Float16*)out)[i] = (_Float16)x;  // past 65504: infinity, as the rounding has it
  }
}

// One wave per tile of 16 w rows x 16 a rows (v_mfma_i32_16x16x64_i8, the w rows as
// the A operand: lane l holds bytes 16 (l / 16) .. + 15 of row l % 16, and result
// register i is w row 4 (l / 16) + i of a row l % 16).  Rows past the end are read
// from the last row and not stored.
template <int DT>
__global__ void __launch_bounds__(256) matmul_i8_kernel(
    const int8_t* __restrict__ a, int64_t a_stride, const float* __restrict__ sa, int64_t sa_stride,
    const int8_t* __restrict__ w, int64_t w_stride, const float* __restrict__ sw, int64_t sw_stride, int64_t M,
    int64_t N, int K, void* __restrict__ out, int64_t out_stride) {
  const int lane = threadIdx.x & 63;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 16, m0 = (int64_t)blockIdx.y * 16;
  if (n0 >= N) return;  // whole wave, no barrier below
  const int8_t* wr = w + min(n0 + (lane & 15), N - 1) * w_stride;
  const int8_t* ar = a + min(m0 + (lane & 15), M - 1) * a_stride;
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 16 * (lane >> 4); k - 16 * (lane >> 4) < K; k += 64)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_codes16(wr, k, K), load_codes16(ar, k, K), acc, 0, 0, 0);
  const int64_t m = m0 + (lane & 15);
  if (m >= M) return;
  const float s = sa[m * sa_stride];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t n = n0 + 4 * (lane >> 4) + i;
    if (n < N) store_out<DT>(out, m * out_stride + n, (float)acc[i] * s * sw[n * sw_stride]);
  }
}

size_t matmul_i8_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_matmul_i8(const MatmulI8& p, void*, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(p.n, 64), (unsigned)cdiv(p.m, 16));
#define ETG_MATMUL(DT)                                                                                             \
  hipLaunchKernelGGL((matmul_i8_kernel<DT>), grid, dim3(256), 0, stream, p.a, p.a_stride, p.a_scale,               \
                     p.a_scale_stride, p.w, p.w_stride, p.w_scale, p.w_scale_stride, p.m, p.n, (int)p.k, p.out,    \
                     p.out_stride)
  if (p.out_dtype == DT_F32) ETG_MATMUL(DT_F32);
  else if (p.out_dtype == DT_BF16) ETG_MATMUL(DT_BF16);
  else ETG_MATMUL(DT_F16);
#undef ETG_MATMUL
  return hipGetLastError();
}

}  // namespace etg

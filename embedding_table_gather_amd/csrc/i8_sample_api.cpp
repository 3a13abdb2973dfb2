// C-ABI of the int8 lm_head (row quantisation, int8 product) and of sampling:
// argument checks, error messages, dispatch.  The public contract is in etg.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/etg.h"
#include "etg_internal.hpp"

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxCols = 65536;              // |sum of k int8 products| <= 2^30 fits int32
constexpr int64_t kMaxRows = 2147483647;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxSpan = (int64_t)1 << 57;   // bytes from a first row to a last: more than an address space holds
constexpr int64_t kMaxTokens = 65536;
constexpr int64_t kMaxSampleVocab = 1 << 20;      // a total in 64-bit fixed point stays within 2^-24 of itself

// bytes of one f32 / bf16 / f16 value, 0 for any other dtype
size_t float_bytes(int32_t dtype) { return dtype == ETG_F32 ? 4 : dtype == ETG_BF16 || dtype == ETG_F16 ? 2 : 0; }

// Rows (at least 0 of them) stride values of `size` bytes apart: kernels compute row * stride
// * size in 64 bits, so it has to stay inside them.
int32_t check_stride(const char* what, int64_t stride, int64_t least, int64_t rows, size_t size) {
  if (stride < least || stride > kMaxStride)
    return etg::set_error(ETG_ESHAPE, "%s stride %lld outside [%lld, 2^40]", what, (long long)stride,
                          (long long)least);
  if (rows > 1 && rows - 1 > kMaxSpan / (stride * (int64_t)size))
    return etg::set_error(ETG_ESHAPE, "%s stride %lld over %lld rows spans more than 2^57 bytes", what,
                          (long long)stride, (long long)rows);
  return ETG_OK;
}

int32_t check_matmul_shape(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || m > kMaxTokens)
    return etg::set_error(ETG_ESHAPE, "m %lld outside [0, %lld]", (long long)m, (long long)kMaxTokens);
  if (n < 0 || n > kMaxRows) return etg::set_error(ETG_ESHAPE, "n %lld outside [0, 2^31 - 1]", (long long)n);
  if (k < 1 || k > kMaxCols)
    return etg::set_error(ETG_ESHAPE, "k %lld outside [1, %lld]", (long long)k, (long long)kMaxCols);
  return ETG_OK;
}

// Every argument of a product but its workspace; with m or n 0 the pointers are not looked at.
int32_t check_matmul(const int8_t* d_a, int64_t a_stride, const float* d_a_scale, int64_t a_scale_stride,
                     const int8_t* d_w, int64_t w_stride, const float* d_w_scale, int64_t w_scale_stride, int64_t m,
                     int64_t n, int64_t k, const void* d_out, int32_t out_dtype, int64_t out_stride) {
  const size_t esize = float_bytes(out_dtype);
  if (esize == 0) return etg::set_error(ETG_EDTYPE, "output dtype %d is not f32, bf16 or f16", out_dtype);
  int32_t st = check_matmul_shape(m, n, k);
  if (st == ETG_OK) st = check_stride("a", a_stride, k, m, 1);
  if (st == ETG_OK) st = check_stride("w", w_stride, k, n, 1);
  if (st == ETG_OK) st = check_stride("a scale", a_scale_stride, 1, m, 4);
  if (st == ETG_OK) st = check_stride("w scale", w_scale_stride, 1, n, 4);
  if (st == ETG_OK) st = check_stride("output", out_stride, n > 1 ? n : 1, m, esize);
  if (st != ETG_OK) return st;
  if (m == 0 || n == 0) return ETG_OK;
  if (d_a == nullptr || d_a_scale == nullptr || d_w == nullptr || d_w_scale == nullptr || d_out == nullptr)
    return etg::set_error(ETG_EINVAL, "an operand, scale or output pointer is NULL");
  if (!aligned(d_a_scale, 4) || !aligned(d_w_scale, 4))
    return etg::set_error(ETG_EALIGN, "a scale pointer is not 4-byte aligned");
  if (!aligned(d_out, esize)) return etg::set_error(ETG_EALIGN, "output pointer is not %zu-byte aligned", esize);
  return ETG_OK;
}

int32_t check_sample_shape(int64_t batch, int64_t vocab) {
  if (batch < 0 || batch > kMaxTokens)
    return etg::set_error(ETG_ESHAPE, "batch %lld outside [0, %lld]", (long long)batch, (long long)kMaxTokens);
  if (vocab < 1 || vocab > kMaxSampleVocab)
    return etg::set_error(ETG_ESHAPE, "vocab %lld outside [1, %lld]", (long long)vocab, (long long)kMaxSampleVocab);
  return ETG_OK;
}

}  // namespace

extern "C" {

int32_t etg_quantize_i8(const void* d_x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                        int8_t* d_codes, int64_t code_stride, float* d_scale, int64_t scale_stride, void* stream) {
  const size_t esize = float_bytes(dtype);
  if (esize == 0) return etg::set_error(ETG_EDTYPE, "dtype %d is not f32, bf16 or f16", dtype);
  if (rows < 0 || rows > kMaxRows)
    return etg::set_error(ETG_ESHAPE, "rows %lld outside [0, 2^31 - 1]", (long long)rows);
  if (cols < 1 || cols > kMaxCols)
    return etg::set_error(ETG_ESHAPE, "cols %lld outside [1, %lld]", (long long)cols, (long long)kMaxCols);
  int32_t st = check_stride("input", x_stride, cols, rows, esize);
  if (st == ETG_OK) st = check_stride("code", code_stride, cols, rows, 1);
  if (st == ETG_OK) st = check_stride("scale", scale_stride, 1, rows, 4);
  if (st != ETG_OK) return st;
  if (rows == 0) return ETG_OK;
  if (d_x == nullptr || d_codes == nullptr || d_scale == nullptr)
    return etg::set_error(ETG_EINVAL, "an input, code or scale pointer is NULL");
  if (!aligned(d_x, esize)) return etg::set_error(ETG_EALIGN, "input pointer is not %zu-byte aligned", esize);
  if (!aligned(d_scale, 4)) return etg::set_error(ETG_EALIGN, "scale pointer is not 4-byte aligned");
  const hipError_t e = etg::launch_quantize_i8(d_x, dtype, rows, cols, x_stride * (int64_t)esize, d_codes,
                                               code_stride, d_scale, scale_stride, (hipStream_t)stream);
  if (e != hipSuccess) return etg::set_error(ETG_EHIP, "quantize launch failed: %s", hipGetErrorString(e));
  return ETG_OK;
}

int64_t etg_matmul_i8_workspace(int64_t m, int64_t n, int64_t k) {
  const int32_t st = check_matmul_shape(m, n, k);
  return st != ETG_OK ? st : (int64_t)etg::matmul_i8_workspace(m, n, k);
}

int32_t etg_matmul_i8(const int8_t* d_a, int64_t a_stride, const float* d_a_scale, int64_t a_scale_stride,
                      const int8_t* d_w, int64_t w_stride, const float* d_w_scale, int64_t w_scale_stride, int64_t m,
                      int64_t n, int64_t k, void* d_out, int32_t out_dtype, int64_t out_stride, void* d_workspace,
                      size_t workspace_bytes, void* stream) {
  const int32_t st =
      check_matmul(d_a, a_stride, d_a_scale, a_scale_stride, d_w, w_stride, d_w_scale, w_scale_stride, m, n, k, d_out,
                   out_dtype, out_stride);
  if (st != ETG_OK || m == 0 || n == 0) return st;
  const size_t need = etg::matmul_i8_workspace(m, n, k);
  if (need != 0) {
    if (d_workspace == nullptr) return etg::set_error(ETG_EINVAL, "workspace pointer is NULL");
    if (!aligned(d_workspace, 256)) return etg::set_error(ETG_EALIGN, "workspace pointer is not 256-byte aligned");
    if (workspace_bytes < need)
      return etg::set_error(ETG_EWORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  }
  const etg::MatmulI8 p = {d_a,        a_stride, d_a_scale, a_scale_stride, d_w, w_stride, d_w_scale, w_scale_stride,
                           m,          n,        k,         d_out,          out_dtype,     out_stride};
  const hipError_t e = etg::launch_matmul_i8(p, d_workspace, (hipStream_t)stream);
  if (e != hipSuccess) return etg::set_error(ETG_EHIP, "int8 product launch failed: %s", hipGetErrorString(e));
  return ETG_OK;
}

}  // extern "C"

namespace {

// Workspace of etg_logits_i8: the residual rows' codes (rows 16-byte aligned), their
// scales, then the product's own workspace.
struct LogitsI8Ws {
  int64_t code_stride;
  size_t scale_offset, product_offset, bytes;
};
LogitsI8Ws logits_i8_ws(int64_t batch, int64_t vocab, int64_t hidden) {
  LogitsI8Ws w;
  w.code_stride = (int64_t)etg::align_up((size_t)hidden, 16);
  w.scale_offset = etg::align_up((size_t)(batch * w.code_stride), 256);
  w.product_offset = etg::align_up(w.scale_offset + (size_t)batch * 4, 256);
  w.bytes = w.product_offset + etg::matmul_i8_workspace(batch, vocab, hidden);
  return w;
}

}  // namespace

extern "C" {

int64_t etg_logits_i8_workspace(int64_t batch, int64_t vocab, int64_t hidden) {
  const int32_t st = check_matmul_shape(batch, vocab, hidden);
  return st != ETG_OK ? st : (int64_t)logits_i8_ws(batch, vocab, hidden).bytes;
}

int32_t etg_logits_i8(const int8_t* d_codes, int64_t code_stride, const float* d_scale, int64_t scale_stride,
                      int64_t vocab, int64_t hidden, const void* d_residual, int32_t dtype, int64_t residual_stride,
                      int64_t batch, void* d_out, int32_t out_dtype, int64_t out_stride, void* d_workspace,
                      size_t workspace_bytes, void* stream) {
  int32_t st = check_matmul_shape(batch, vocab, hidden);
  if (st != ETG_OK) return st;
  const LogitsI8Ws w = logits_i8_ws(batch, vocab, hidden);
  if (batch > 0 && vocab > 0) {
    if (d_workspace == nullptr) return etg::set_error(ETG_EINVAL, "workspace pointer is NULL");
    if (!aligned(d_workspace, 256)) return etg::set_error(ETG_EALIGN, "workspace pointer is not 256-byte aligned");
    if (workspace_bytes < w.bytes)
      return etg::set_error(ETG_EWORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, w.bytes);
  }
  uint8_t* ws = (uint8_t*)d_workspace;
  int8_t* a = (int8_t*)ws;
  float* a_scale = ws != nullptr ? (float*)(ws + w.scale_offset) : nullptr;
  // the product's own checks, before anything is enqueued
  st = check_matmul(a, w.code_stride, a_scale, 1, d_codes, code_stride, d_scale, scale_stride, batch, vocab, hidden,
                    d_out, out_dtype, out_stride);
  if (st != ETG_OK) return st;
  if (batch == 0 || vocab == 0) return ETG_OK;
  st = etg_quantize_i8(d_residual, dtype, batch, hidden, residual_stride, a, w.code_stride, a_scale, 1, stream);
  if (st != ETG_OK) return st;
  return etg_matmul_i8(a, w.code_stride, a_scale, 1, d_codes, code_stride, d_scale, scale_stride, batch, vocab, hidden,
                       d_out, out_dtype, out_stride, ws + w.product_offset, w.bytes - w.product_offset, stream);
}

int64_t etg_sample_workspace(int64_t batch, int64_t vocab) {
  const int32_t st = check_sample_shape(batch, vocab);
  return st != ETG_OK ? st : (int64_t)etg::sample_workspace(batch, vocab);
}

int32_t etg_sample(const void* d_logits, int32_t dtype, int64_t batch, int64_t vocab, int64_t logits_stride,
                   const etg_sampling* how, const float* d_uniform, int32_t* d_ids, float* d_probs,
                   void* d_workspace, size_t workspace_bytes, void* stream) {
  const size_t esize = float_bytes(dtype);
  if (esize == 0) return etg::set_error(ETG_EDTYPE, "logits dtype %d is not f32, bf16 or f16", dtype);
  int32_t st = check_sample_shape(batch, vocab);
  if (st == ETG_OK) st = check_stride("logits", logits_stride, vocab, batch, esize);
  if (st != ETG_OK) return st;
  if (how == nullptr) return etg::set_error(ETG_EINVAL, "sampling settings are NULL");
  // written so that a NaN fails; a per-row array replaces its scalar
  if (how->d_temperature == nullptr && !(how->temperature >= 0.f && std::isfinite(how->temperature)))
    return etg::set_error(ETG_ERANGE, "temperature %g is not a finite value >= 0", (double)how->temperature);
  if (how->d_top_k == nullptr && how->top_k < 0) return etg::set_error(ETG_ERANGE, "top_k %d is negative", how->top_k);
  if (how->d_top_p == nullptr && !(how->top_p > 0.f && how->top_p <= 1.f))
    return etg::set_error(ETG_ERANGE, "top_p %g outside (0, 1]", (double)how->top_p);
  if (how->d_min_p == nullptr && !(how->min_p >= 0.f && how->min_p <= 1.f))
    return etg::set_error(ETG_ERANGE, "min_p %g outside [0, 1]", (double)how->min_p);
  const int64_t words = (vocab + 31) / 32;
  if (how->d_allowed != nullptr && how->allowed_stride != 0) {
    st = check_stride("allowed", how->allowed_stride, words, batch, 4);
    if (st != ETG_OK) return st;
  }
  if (batch == 0) return ETG_OK;
  if (d_logits == nullptr || d_uniform == nullptr || d_ids == nullptr || d_probs == nullptr)
    return etg::set_error(ETG_EINVAL, "a logits, uniform or output pointer is NULL");
  if (!aligned(d_logits, esize)) return etg::set_error(ETG_EALIGN, "logits pointer is not %zu-byte aligned", esize);
  if (!aligned(d_uniform, 4) || !aligned(d_ids, 4) || !aligned(d_probs, 4) || !aligned(how->d_temperature, 4) ||
      !aligned(how->d_top_k, 4) || !aligned(how->d_top_p, 4) || !aligned(how->d_min_p, 4) ||
      !aligned(how->d_allowed, 4))
    return etg::set_error(ETG_EALIGN, "uniform, setting, mask and output pointers must be 4-byte aligned");
  const size_t need = etg::sample_workspace(batch, vocab);
  if (need != 0) {
    if (d_workspace == nullptr) return etg::set_error(ETG_EINVAL, "workspace pointer is NULL");
    if (!aligned(d_workspace, 256)) return etg::set_error(ETG_EALIGN, "workspace pointer is not 256-byte aligned");
    if (workspace_bytes < need)
      return etg::set_error(ETG_EWORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  }
  const etg::Sample s = {d_logits,          dtype,        batch,        vocab,        logits_stride,
                         d_uniform,         how->temperature, how->top_p, how->min_p,  how->top_k,
                         how->d_temperature, how->d_top_p, how->d_min_p, how->d_top_k, how->d_allowed,
                         how->allowed_stride, d_ids,       d_probs};
  const hipError_t e = etg::launch_sample(s, d_workspace, (hipStream_t)stream);
  if (e != hipSuccess) return etg::set_error(ETG_EHIP, "sample launch failed: %s", hipGetErrorString(e));
  return ETG_OK;
}

}  // extern "C"

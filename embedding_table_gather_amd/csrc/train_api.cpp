// C-ABI of the tied table's training operators (cross entropy, its gradients, the gather's
// gradient): argument checks, error messages, dispatch.  The public contract is in etg.h.
#include <hip/hip_runtime.h>

#include "../../include/etg.h"
#include "etg_internal.hpp"

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxBatch = 65536;
constexpr int64_t kMaxIds = 1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxSpan = (int64_t)1 << 57;  // bytes from a first row to a last: more than an address space holds

size_t float_bytes(int32_t dtype) { return dtype == ETG_F32 ? 4 : dtype == ETG_BF16 || dtype == ETG_F16 ? 2 : 0; }

int32_t check_table(const etg_table* t) {
  if (t == nullptr) return etg::set_error(ETG_EINVAL, "table handle is NULL");
  if (float_bytes(t->d.dtype) == 0) return etg::set_error(ETG_EDTYPE, "a Q8_0 table has no gradients");
  return ETG_OK;
}

int32_t check_stride(const char* what, int64_t stride, int64_t least, int64_t rows, size_t size) {
  if (stride < least || stride > kMaxStride)
    return etg::set_error(ETG_ESHAPE, "%s stride %lld outside [%lld, 2^40]", what, (long long)stride,
                          (long long)least);
  if (rows > 1 && rows - 1 > kMaxSpan / (stride * (int64_t)size))
    return etg::set_error(ETG_ESHAPE, "%s stride %lld over %lld rows spans more than 2^57 bytes", what,
                          (long long)stride, (long long)rows);
  return ETG_OK;
}

int32_t check_batch(const etg_table* t, int64_t batch) {
  const int32_t st = check_table(t);
  if (st != ETG_OK) return st;
  if (batch < 0 || batch > kMaxBatch)
    return etg::set_error(ETG_ESHAPE, "batch %lld outside [0, %lld]", (long long)batch, (long long)kMaxBatch);
  return ETG_OK;
}

int32_t check_ids(const etg_table* t, int64_t seq_len) {
  const int32_t st = check_table(t);
  if (st != ETG_OK) return st;
  if (seq_len < 0 || seq_len > kMaxIds)
    return etg::set_error(ETG_ESHAPE, "seq_len %lld outside [0, 2^24]", (long long)seq_len);
  return ETG_OK;
}

int32_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return ETG_OK;
  if (ws == nullptr) return etg::set_error(ETG_EINVAL, "workspace pointer is NULL");
  if (!aligned(ws, 256)) return etg::set_error(ETG_EALIGN, "workspace pointer is not 256-byte aligned");
  if (bytes < need) return etg::set_error(ETG_EWORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  return ETG_OK;
}

}  // namespace

extern "C" {

int64_t etg_cross_entropy_workspace(const etg_table* t, int64_t batch) {
  const int32_t st = check_batch(t, batch);
  return st != ETG_OK ? st : (int64_t)etg::xent_workspace(t->d, batch);
}

int32_t etg_cross_entropy(const etg_table* t, const void* d_residual, int64_t residual_stride, int64_t batch,
                          const int32_t* d_labels, float* d_loss, float* d_lse, void* d_workspace,
                          size_t workspace_bytes, void* stream) {
  int32_t st = check_batch(t, batch);
  if (st != ETG_OK) return st;
  const size_t esize = float_bytes(t->d.dtype);
  if ((st = check_stride("residual", residual_stride, t->d.hidden, batch, esize)) != ETG_OK) return st;
  if (batch == 0) return ETG_OK;
  if (d_residual == nullptr || d_labels == nullptr || d_loss == nullptr || d_lse == nullptr)
    return etg::set_error(ETG_EINVAL, "a residual, labels, loss or lse pointer is NULL");
  if (!aligned(d_residual, esize))
    return etg::set_error(ETG_EALIGN, "residual pointer is not %zu-byte aligned", esize);
  if (!aligned(d_labels, 4) || !aligned(d_loss, 4) || !aligned(d_lse, 4))
    return etg::set_error(ETG_EALIGN, "labels, loss and lse pointers must be 4-byte aligned");
  if ((st = check_workspace(d_workspace, workspace_bytes, etg::xent_workspace(t->d, batch))) != ETG_OK) return st;
  etg::XentCall c = {};
  c.x = d_residual, c.x_pitch = residual_stride * (int64_t)esize, c.n = batch, c.labels = d_labels;
  c.loss = d_loss, c.lse_out = d_lse;
  const hipError_t e = etg::launch_xent(t->d, c, d_workspace, (hipStream_t)stream);
  if (e != hipSuccess) return etg::set_error(ETG_EHIP, "cross entropy launch failed: %s", hipGetErrorString(e));
  return ETG_OK;
}

int64_t etg_cross_entropy_grad_workspace(const etg_table* t, int64_t batch) {
  const int32_t st = check_batch(t, batch);
  return st != ETG_OK ? st : (int64_t)etg::xent_grad_workspace(t->d, batch);
}

int32_t etg_cross_entropy_grad(const etg_table* t, const void* d_residual, int64_t residual_stride, int64_t batch,
                               const int32_t* d_labels, const float* d_lse, float grad_loss, const float* d_grad_loss,
                               const float* d_grad_lse, void* d_residual_grad, int64_t residual_grad_stride,
                               void* d_table_grad, int32_t accumulate, void* d_workspace, size_t workspace_bytes,
                               void* stream) {
  int32_t st = check_batch(t, batch);
  if (st != ETG_OK) return st;
  const size_t esize = float_bytes(t->d.dtype);
  if ((st = check_stride("residual", residual_stride, t->d.hidden, batch, esize)) != ETG_OK) return st;
  if (d_residual_grad != nullptr &&
      (st = check_stride("residual gradient", residual_grad_stride, t->d.hidden, batch, esize)) != ETG_OK)
    return st;
  if (!aligned(d_table_grad, 16))
    return etg::set_error(ETG_EALIGN, "table gradient pointer is not 16-byte aligned");
  if (batch > 0) {
    if (d_residual == nullptr || d_labels == nullptr || d_lse == nullptr)
      return etg::set_error(ETG_EINVAL, "a residual, labels or lse pointer is NULL");
    if (!aligned(d_residual, esize) || !aligned(d_residual_grad, esize))
      return etg::set_error(ETG_EALIGN, "residual and residual gradient pointers must be %zu-byte aligned", esize);
    if (!aligned(d_labels, 4) || !aligned(d_lse, 4) || !aligned(d_grad_loss, 4) || !aligned(d_grad_lse, 4))
      return etg::set_error(ETG_EALIGN, "labels, lse and gradient pointers must be 4-byte aligned");
  }
  if (d_residual_grad == nullptr && d_table_grad == nullptr) return ETG_OK;
  if ((st = check_workspace(d_workspace, workspace_bytes, etg::xent_grad_workspace(t->d, batch))) != ETG_OK) return st;
  etg::XentCall c = {};
  c.x = d_residual, c.x_pitch = residual_stride * (int64_t)esize, c.n = batch, c.labels = d_labels, c.lse = d_lse;
  c.grad_loss_all = grad_loss, c.grad_loss = d_grad_loss, c.grad_lse = d_grad_lse;
  c.d_x = d_residual_grad, c.d_x_pitch = residual_grad_stride * (int64_t)esize;
  c.d_rows = d_table_grad, c.add = accumulate != 0;
  const hipError_t e = etg::launch_xent_grad(t->d, c, d_workspace, (hipStream_t)stream);
  if (e != hipSuccess)
    return etg::set_error(ETG_EHIP, "cross entropy gradient launch failed: %s", hipGetErrorString(e));
  return ETG_OK;
}

int64_t etg_embed_gather_grad_workspace(const etg_table* t, int64_t seq_len) {
  const int32_t st = check_ids(t, seq_len);
  return st != ETG_OK ? st : (int64_t)etg::rowgrad_workspace(seq_len, t->d.V, t->d.hidden);
}

int32_t etg_embed_gather_grad(const etg_table* t, const int32_t* d_ids, int64_t seq_len, const void* d_grad,
                              int32_t grad_dtype, int64_t grad_stride, float scale, void* d_out, int32_t out_dtype,
                              int32_t accumulate, void* d_workspace, size_t workspace_bytes, void* stream) {
  int32_t st = check_ids(t, seq_len);
  if (st != ETG_OK) return st;
  const size_t esize = float_bytes(grad_dtype);
  if (esize == 0) return etg::set_error(ETG_EDTYPE, "gradient dtype %d is not f32, bf16 or f16", grad_dtype);
  if (out_dtype != t->d.dtype && out_dtype != ETG_F32)
    return etg::set_error(ETG_EDTYPE, "output dtype %d is neither the table's (%d) nor f32", out_dtype, t->d.dtype);
  if ((st = check_stride("gradient", grad_stride, t->d.hidden, seq_len, esize)) != ETG_OK) return st;
  if (d_out == nullptr) return etg::set_error(ETG_EINVAL, "output pointer is NULL");
  if (!aligned(d_out, 16)) return etg::set_error(ETG_EALIGN, "output pointer is not 16-byte aligned");
  if (seq_len > 0) {
    if (d_ids == nullptr || d_grad == nullptr) return etg::set_error(ETG_EINVAL, "an ids or gradient pointer is NULL");
    if (!aligned(d_ids, 4)) return etg::set_error(ETG_EALIGN, "ids pointer is not 4-byte aligned");
    if (!aligned(d_grad, esize))
      return etg::set_error(ETG_EALIGN, "gradient pointer is not %zu-byte aligned", esize);
  }
  st = check_workspace(d_workspace, workspace_bytes, etg::rowgrad_workspace(seq_len, t->d.V, t->d.hidden));
  if (st != ETG_OK) return st;
  etg::RowGrad g = {};
  g.ids = d_ids, g.n = seq_len, g.V = t->d.V, g.hidden = t->d.hidden;
  g.grad = d_grad, g.grad_dtype = grad_dtype, g.pitch = grad_stride * (int64_t)esize;
  g.scale = scale, g.out = d_out, g.out_dtype = out_dtype, g.add = accumulate != 0;
  const hipError_t e = etg::launch_rowgrad(g, d_workspace, (hipStream_t)stream);
  if (e != hipSuccess) return etg::set_error(ETG_EHIP, "gather gradient launch failed: %s", hipGetErrorString(e));
  return ETG_OK;
}

}  // extern "C"

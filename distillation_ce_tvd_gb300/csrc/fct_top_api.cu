// C ABI of distillation from a teacher's top logits: argument checks and
// dispatch.  The operations are described in include/fused_ce_tvd.h.
#include "fct_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A (rows, cols) array of e-byte elements with row stride ld.
struct Array {
  const void* p;
  int64_t rows, cols, ld;
  int64_t e;
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const { return lo() + static_cast<uintptr_t>(((rows - 1) * ld + cols) * e); }
};

// FCT_OK if x is there, its rows do not overlap each other, it spans at most
// 2^62 bytes and is aligned to its element.
int check_array(const Array& x) {
  if (x.p == nullptr || x.ld < x.cols) return FCT_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 62) / x.e;
  if (x.cols > lim || x.rows - 1 > (lim - x.cols) / x.ld) return FCT_ERR_UNSUPPORTED;
  return aligned(x.p, static_cast<size_t>(x.e)) ? FCT_OK : FCT_ERR_ALIGNMENT;
}

bool overlap(const Array& a, const Array& b) { return a.lo() < b.hi() && b.lo() < a.hi(); }

// Checks every array, and that no output overlaps an input or another output.
int check_arrays(const Array* in, int n_in, const Array* out, int n_out) {
  int rc;
  for (int i = 0; i < n_in; ++i)
    if ((rc = check_array(in[i])) != FCT_OK) return rc;
  for (int i = 0; i < n_out; ++i)
    if ((rc = check_array(out[i])) != FCT_OK) return rc;
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return FCT_ERR_INVALID_ARG;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(out[i], out[j])) return FCT_ERR_INVALID_ARG;
  }
  return FCT_OK;
}

int check_status(const int32_t* dev_status) {
  return dev_status && !aligned(dev_status, 4) ? FCT_ERR_ALIGNMENT : FCT_OK;
}

int launched(cudaError_t e) { return e == cudaSuccess ? FCT_OK : FCT_ERR_CUDA; }

int element_size(int dtype) { return dtype == FCT_BF16 ? 2 : 4; }

int check_list(const fct_top_list* t) {
  if (t == nullptr || t->K <= 0 || t->reserved[0] != 0 || t->reserved[1] != 0)
    return FCT_ERR_INVALID_ARG;
  return t->K > FCT_TOP_MAX ? FCT_ERR_UNSUPPORTED : FCT_OK;
}

int check_sizes(int dtype, int64_t V, int64_t max_v) {
  if (dtype != FCT_F32 && dtype != FCT_BF16) return FCT_ERR_UNSUPPORTED;
  if (V <= 0) return FCT_ERR_INVALID_ARG;
  return V > max_v ? FCT_ERR_UNSUPPORTED : FCT_OK;
}

constexpr int64_t kMaxSelectV = (int64_t(1) << 31) - (1 << 16);

// The loss on logits: forward (forward true), backward (grad given) or both.
int loss_impl(const void* student, int64_t ld, int dtype, const int64_t* target,
              const fct_top_list* t, int64_t BT, int64_t V, int64_t ignore_index, float* ce,
              float* tvd, float* lse, float* rest, float* t_lse, float* sigma, bool forward,
              bool backward, const float* grad_ce, const float* grad_tvd, int64_t grad_stride,
              void* grad, int64_t ld_g, int32_t* dev_status, void* stream) {
  if (BT < 0) return FCT_ERR_INVALID_ARG;
  int rc = check_sizes(dtype, V, fct::kTopMaxV);
  if (rc != FCT_OK) return rc;
  if ((rc = check_list(t)) != FCT_OK) return rc;
  if (BT == 0) return FCT_OK;
  if (backward && grad_stride != 0 && grad_stride != 1) return FCT_ERR_INVALID_ARG;
  const int64_t e = element_size(dtype);
  auto row = [&](const void* p, int64_t n = -1, int64_t size = 4) {
    return Array{p, 1, n < 0 ? BT : n, n < 0 ? BT : n, size};
  };
  Array in[12], out[8];
  int n_in = 0, n_out = 0;
  const Array logits{student, BT, V, ld, e};
  const bool inplace = backward && grad == student;
  if (inplace && ld_g != ld) return FCT_ERR_INVALID_ARG;
  if (!inplace) in[n_in++] = logits;
  in[n_in++] = row(target, -1, 8);
  in[n_in++] = Array{t->index, BT, t->K, t->ld_index, 4};
  in[n_in++] = Array{t->values, BT, t->K, t->ld_values, 4};
  if (t->rest_lse) in[n_in++] = row(t->rest_lse);
  if (forward) {
    for (float* p : {ce, tvd, lse, rest, t_lse, sigma}) out[n_out++] = row(p);
  } else {
    for (float* p : {lse, rest, t_lse, sigma}) in[n_in++] = row(p);
  }
  if (backward) {
    const int64_t n = grad_stride ? BT : 1;
    in[n_in++] = row(grad_ce, n);
    in[n_in++] = row(grad_tvd, n);
    out[n_out++] = Array{grad, BT, V, ld_g, e};
  }
  if ((rc = check_arrays(in, n_in, out, n_out)) != FCT_OK) return rc;
  if ((rc = check_status(dev_status)) != FCT_OK) return rc;
  int sms = 0, device = 0, l2 = 0;
  if ((rc = fct::current_device_sms(&sms, &device, &l2)) != FCT_OK) return rc;
  fct::TopArgs a{student, ld, dtype, target, t->values, t->ld_values, t->index, t->ld_index,
                 t->rest_lse, BT, V, t->K, ignore_index, ce, tvd, lse, rest, t_lse, sigma,
                 dev_status};
  if (backward) {
    a.grad_ce = grad_ce;
    a.grad_tvd = grad_tvd;
    a.grad_stride = grad_stride;
    a.grad = grad;
    a.ld_g = ld_g;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launched(forward ? fct::launch_top_forward(a, sms, device, l2, st)
                          : fct::launch_top_backward(a, st));
}

}  // namespace

extern "C" {

int fct_top_logits(const void* logits, int64_t ld, fct_dtype dtype, int64_t BT, int64_t V,
                   int64_t K, float* values, int64_t ld_values, int32_t* index, int64_t ld_index,
                   float* rest_lse, int32_t* dev_status, void* stream) {
  if (BT < 0 || K <= 0) return FCT_ERR_INVALID_ARG;
  int rc = check_sizes(dtype, V, kMaxSelectV);
  if (rc != FCT_OK) return rc;
  if (K > FCT_TOP_MAX) return FCT_ERR_UNSUPPORTED;
  if (BT == 0) return FCT_OK;
  const Array in[1] = {{logits, BT, V, ld, element_size(dtype)}};
  const Array out[3] = {{values, BT, K, ld_values, 4}, {index, BT, K, ld_index, 4},
                        {rest_lse, 1, BT, BT, 4}};
  if ((rc = check_arrays(in, 1, out, 3)) != FCT_OK) return rc;
  if ((rc = check_status(dev_status)) != FCT_OK) return rc;
  int sms = 0, device = 0;
  if ((rc = fct::current_device_sms(&sms, &device)) != FCT_OK) return rc;
  return launched(fct::launch_top_select(
      fct::TopSelectArgs{logits, ld, dtype, BT, V, K, values, ld_values, index, ld_index, rest_lse,
                         dev_status},
      sms, device, static_cast<cudaStream_t>(stream)));
}

int fused_ce_tvd_top_forward(const void* student, int64_t ld_student, fct_dtype dtype,
                             const int64_t* target, const fct_top_list* teacher, int64_t BT,
                             int64_t V, int64_t ignore_index, float* ce, float* tvd,
                             float* student_lse, float* student_rest, float* teacher_lse,
                             float* sigma, int32_t* dev_status, void* stream) {
  return loss_impl(student, ld_student, dtype, target, teacher, BT, V, ignore_index, ce, tvd,
                   student_lse, student_rest, teacher_lse, sigma, true, false, nullptr, nullptr, 0,
                   nullptr, 0, dev_status, stream);
}

int fused_ce_tvd_top_backward(const void* student, int64_t ld_student, fct_dtype dtype,
                              const int64_t* target, const fct_top_list* teacher, int64_t BT,
                              int64_t V, int64_t ignore_index, const float* student_lse,
                              const float* student_rest, const float* teacher_lse,
                              const float* sigma, const float* grad_ce, const float* grad_tvd,
                              int64_t grad_stride, void* grad_student, int64_t ld_grad,
                              int32_t* dev_status, void* stream) {
  // the four saved vectors are only read
  return loss_impl(student, ld_student, dtype, target, teacher, BT, V, ignore_index, nullptr,
                   nullptr, const_cast<float*>(student_lse), const_cast<float*>(student_rest),
                   const_cast<float*>(teacher_lse), const_cast<float*>(sigma), false, true,
                   grad_ce, grad_tvd, grad_stride, grad_student, ld_grad, dev_status, stream);
}

int fused_ce_tvd_top_forward_backward(const void* student, int64_t ld_student, fct_dtype dtype,
                                      const int64_t* target, const fct_top_list* teacher,
                                      int64_t BT, int64_t V, int64_t ignore_index,
                                      const float* grad_ce, const float* grad_tvd,
                                      int64_t grad_stride, float* ce, float* tvd,
                                      float* student_lse, float* student_rest, float* teacher_lse,
                                      float* sigma, void* grad_student, int64_t ld_grad,
                                      int32_t* dev_status, void* stream) {
  return loss_impl(student, ld_student, dtype, target, teacher, BT, V, ignore_index, ce, tvd,
                   student_lse, student_rest, teacher_lse, sigma, true, true, grad_ce, grad_tvd,
                   grad_stride, grad_student, ld_grad, dev_status, stream);
}

}  // extern "C"

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

// From hidden states: forward (grad false) or backward; t nullptr is
// cross-entropy alone, whose tvd, rest, t_lse, sigma and grad_tvd are nullptr.
int linear_impl(const void* h, int64_t ld_h, const void* w, int64_t ld_w, int64_t d,
                const int64_t* target, const fct_top_list* t, bool list, int64_t BT, int64_t V,
                int64_t ignore_index, float* ce, float* tvd, float* lse, float* rest,
                float* t_lse, float* sigma, bool grad, const float* grad_ce,
                const float* grad_tvd, int64_t grad_stride, void* grad_h, int64_t ld_gh,
                void* grad_w, int64_t ld_gw, int grad_w_kind, void* workspace,
                size_t workspace_bytes, int64_t piece_cols, int32_t* dev_status, void* stream) {
  if (BT < 0 || V <= 0 || d <= 0 || piece_cols < 0) return FCT_ERR_INVALID_ARG;
  int rc;
  if (list && (rc = check_list(t)) != FCT_OK) return rc;
  const int64_t K = list ? t->K : 0, most = fct::kGemmMaxDim;
  if (grad) {
    if (grad_stride != 0 && grad_stride != 1) return FCT_ERR_INVALID_ARG;
    if (grad_w_kind != FCT_GEMM_F32 && grad_w_kind != FCT_GEMM_BF16 &&
        grad_w_kind != FCT_GEMM_ADD_F32)
      return FCT_ERR_UNSUPPORTED;
  }
  if (BT == 0 && !(grad && grad_w)) return FCT_OK;
  if (BT > most || V > most || d > most || ld_h > most || ld_w > most || piece_cols > most ||
      (grad_h && ld_gh > most) || (grad_w && ld_gw > most))
    return FCT_ERR_UNSUPPORTED;
  auto row = [&](const void* p, int64_t n = -1, int64_t size = 4) {
    return Array{p, 1, n < 0 ? BT : n, n < 0 ? BT : n, size};
  };
  Array in[14], out[8];
  int n_in = 0, n_out = 0;
  const int64_t ew = grad_w_kind == FCT_GEMM_BF16 ? 2 : 4;
  if (BT > 0) {
    in[n_in++] = Array{h, BT, d, ld_h, 2};
    in[n_in++] = Array{w, V, d, ld_w, 2};
    in[n_in++] = row(target, -1, 8);
    if (list) {
      in[n_in++] = Array{t->index, BT, K, t->ld_index, 4};
      in[n_in++] = Array{t->values, BT, K, t->ld_values, 4};
      if (t->rest_lse) in[n_in++] = row(t->rest_lse);
    }
    Array* stats = grad ? in : out;
    int& n = grad ? n_in : n_out;
    if (!grad) stats[n++] = row(ce);
    stats[n++] = row(lse);
    if (list) {
      if (!grad) stats[n++] = row(tvd);
      for (float* p : {rest, t_lse, sigma}) stats[n++] = row(p);
    }
    if (grad) {
      in[n_in++] = row(grad_ce, grad_stride ? BT : 1);
      if (list) in[n_in++] = row(grad_tvd, grad_stride ? BT : 1);
      if (grad_h) out[n_out++] = Array{grad_h, BT, d, ld_gh, 2};
    }
  }
  if (grad && grad_w) out[n_out++] = Array{grad_w, V, d, ld_gw, ew};
  const size_t need = BT == 0 ? 0
                      : grad  ? fct::top_linear_backward_bytes(BT, V, d, K, piece_cols)
                              : fct::top_linear_forward_bytes(BT, V, K);
  if (need == SIZE_MAX) return FCT_ERR_UNSUPPORTED;
  if (BT > 0) {
    if (workspace == nullptr || workspace_bytes < need) return FCT_ERR_INVALID_ARG;
    const int64_t n = static_cast<int64_t>(need);
    out[n_out++] = Array{workspace, 1, n, n, 1};
  }
  if ((rc = check_arrays(in, n_in, out, n_out)) != FCT_OK) return rc;
  if (BT > 0 && (!fct::gemm_operand_ok(h, ld_h) || !fct::gemm_operand_ok(w, ld_w) ||
                 !aligned(workspace, 256)))
    return FCT_ERR_ALIGNMENT;
  if ((rc = check_status(dev_status)) != FCT_OK) return rc;
  int sms = 0, device = 0;
  if ((rc = fct::current_device_sms(&sms, &device)) != FCT_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (BT == 0) {  // a weight gradient of no rows
    if (grad_w_kind != FCT_GEMM_ADD_F32 &&
        cudaMemset2DAsync(grad_w, size_t(ld_gw) * ew, 0, size_t(d) * ew, size_t(V), st) !=
            cudaSuccess)
      return FCT_ERR_CUDA;
    return FCT_OK;
  }
  fct::TopLinearArgs a{h, ld_h, w, ld_w, d, target, list ? t->values : nullptr,
                       list ? t->ld_values : 0, list ? t->index : nullptr, list ? t->ld_index : 0,
                       list ? t->rest_lse : nullptr, BT, V, K, ignore_index, ce, tvd, lse, rest,
                       t_lse, sigma, workspace, dev_status};
  if (!grad) return launched(fct::launch_top_linear_forward(a, sms, device, st));
  a.grad_ce = grad_ce;
  a.grad_tvd = grad_tvd;
  a.grad_stride = grad_stride;
  a.grad_h = grad_h;
  a.ld_gh = ld_gh;
  a.grad_w = grad_w;
  a.ld_gw = ld_gw;
  a.grad_w_kind = grad_w_kind;
  a.piece_cols = piece_cols;
  if (grad_h == nullptr && grad_w == nullptr) return FCT_OK;
  return launched(fct::launch_top_linear_backward(a, sms, device, st));
}

bool sizes_ok(int64_t BT, int64_t V, int64_t d, int64_t K, int64_t piece) {
  const int64_t most = fct::kGemmMaxDim;
  return BT > 0 && V > 0 && d > 0 && K >= 0 && piece >= 0 && BT <= most && V <= most &&
         d <= most && K <= FCT_TOP_MAX && piece <= most;
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

size_t fused_linear_ce_tvd_top_forward_workspace_size(int64_t BT, int64_t V, int64_t K) {
  if (!sizes_ok(BT, V, 1, K, 0)) return 0;
  const size_t b = fct::top_linear_forward_bytes(BT, V, K);
  return b == SIZE_MAX ? 0 : b;
}

size_t fused_linear_ce_tvd_top_backward_workspace_size(int64_t BT, int64_t V, int64_t d, int64_t K,
                                                       int64_t piece_cols) {
  if (!sizes_ok(BT, V, d, K, piece_cols)) return 0;
  const size_t b = fct::top_linear_backward_bytes(BT, V, d, K, piece_cols);
  return b == SIZE_MAX ? 0 : b;
}

int fused_linear_ce_tvd_top_forward(const void* h, int64_t ld_h, const void* w, int64_t ld_w,
                                    int64_t d, const int64_t* target, const fct_top_list* teacher,
                                    int64_t BT, int64_t V, int64_t ignore_index, float* ce,
                                    float* tvd, float* student_lse, float* student_rest,
                                    float* teacher_lse, float* sigma, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return linear_impl(h, ld_h, w, ld_w, d, target, teacher, true, BT, V, ignore_index, ce, tvd,
                     student_lse, student_rest, teacher_lse, sigma, false, nullptr, nullptr, 0,
                     nullptr, 0, nullptr, 0, 0, workspace, workspace_bytes, 0, dev_status, stream);
}

int fused_linear_ce_tvd_top_backward(const void* h, int64_t ld_h, const void* w, int64_t ld_w,
                                     int64_t d, const int64_t* target, const fct_top_list* teacher,
                                     int64_t BT, int64_t V, int64_t ignore_index,
                                     const float* student_lse, const float* student_rest,
                                     const float* teacher_lse, const float* sigma,
                                     const float* grad_ce, const float* grad_tvd,
                                     int64_t grad_stride, void* grad_h, int64_t ld_grad_h,
                                     void* grad_w, int64_t ld_grad_w, int32_t grad_w_kind,
                                     void* workspace, size_t workspace_bytes, int64_t piece_cols,
                                     int32_t* dev_status, void* stream) {
  return linear_impl(h, ld_h, w, ld_w, d, target, teacher, true, BT, V, ignore_index, nullptr,
                     nullptr, const_cast<float*>(student_lse), const_cast<float*>(student_rest),
                     const_cast<float*>(teacher_lse), const_cast<float*>(sigma), true, grad_ce,
                     grad_tvd, grad_stride, grad_h, ld_grad_h, grad_w, ld_grad_w, grad_w_kind,
                     workspace, workspace_bytes, piece_cols, dev_status, stream);
}

int fused_linear_ce_forward(const void* h, int64_t ld_h, const void* w, int64_t ld_w, int64_t d,
                            const int64_t* target, int64_t BT, int64_t V, int64_t ignore_index,
                            float* ce, float* lse, void* workspace, size_t workspace_bytes,
                            int32_t* dev_status, void* stream) {
  return linear_impl(h, ld_h, w, ld_w, d, target, nullptr, false, BT, V, ignore_index, ce, nullptr,
                     lse, nullptr, nullptr, nullptr, false, nullptr, nullptr, 0, nullptr, 0,
                     nullptr, 0, 0, workspace, workspace_bytes, 0, dev_status, stream);
}

int fused_linear_ce_backward(const void* h, int64_t ld_h, const void* w, int64_t ld_w, int64_t d,
                             const int64_t* target, int64_t BT, int64_t V, int64_t ignore_index,
                             const float* lse, const float* grad_ce, int64_t grad_stride,
                             void* grad_h, int64_t ld_grad_h, void* grad_w, int64_t ld_grad_w,
                             int32_t grad_w_kind, void* workspace, size_t workspace_bytes,
                             int64_t piece_cols, int32_t* dev_status, void* stream) {
  return linear_impl(h, ld_h, w, ld_w, d, target, nullptr, false, BT, V, ignore_index, nullptr,
                     nullptr, const_cast<float*>(lse), nullptr, nullptr, nullptr, true, grad_ce,
                     nullptr, grad_stride, grad_h, ld_grad_h, grad_w, ld_grad_w, grad_w_kind,
                     workspace, workspace_bytes, piece_cols, dev_status, stream);
}

}  // extern "C"

// api_layer.cu -- the C ABI of a layer's operators between its hidden states and the
// attention: argument checks of the norm with rotation (norm_rope.cu).
#include <cmath>
#include <string>

#include "internal.h"

using namespace tsr;

namespace {

tsr_status check_norm_rope(const tsr_rope_desc* d, double eps, const tsr_norm_rope_tensor* t, int32_t n, bool grad) {
  if (!d || !t) return fail(TSR_ERR_INVALID_ARG, "desc / tensors is NULL");
  if (n < 1 || n > 4) return fail(TSR_ERR_INVALID_ARG, "1 to 4 tensors per call");
  if (tsr_status e = check_rope_desc(d)) return e;
  if (!(static_cast<float>(eps) > 0.f) || !std::isfinite(static_cast<float>(eps)))
    return fail(TSR_ERR_INVALID_ARG, "eps must be > 0 and finite in fp32");
  const size_t es = d->dtype == TSR_DTYPE_F32 ? 4 : 2;
  int64_t heads = 0;
  for (int i = 0; i < n; ++i) {
    const std::string at = "tensor " + std::to_string(i) + ": ";
    if (!t[i].x || !t[i].out || (grad && !t[i].dout)) return fail(TSR_ERR_INVALID_ARG, at + "NULL pointer");
    if (!aligned(t[i].x, es) || !aligned(t[i].out, es) || (grad && !aligned(t[i].dout, es)))
      return fail(TSR_ERR_INVALID_ARG, at + "pointers must be aligned to the element type");
    if (t[i].weight_dtype != d->dtype && t[i].weight_dtype != TSR_DTYPE_F32)
      return fail(TSR_ERR_INVALID_ARG, at + "weight_dtype must be the tensors' type or fp32");
    if (t[i].weight_dtype != t[0].weight_dtype)
      return fail(TSR_ERR_INVALID_ARG, at + "the weights of a call have one type");
    const size_t ws = t[i].weight_dtype == TSR_DTYPE_F32 ? 4 : 2;
    if (!aligned(t[i].weight, ws) || (grad && !aligned(t[i].dweight, ws)))
      return fail(TSR_ERR_INVALID_ARG, at + "weights must be aligned to their type");
    if (grad && t[i].dweight && !t[i].weight) return fail(TSR_ERR_INVALID_ARG, at + "dweight without a weight");
    if (grad && t[i].dweight && (t[i].dweight == t[i].weight || t[i].dweight == t[i].x || t[i].dweight == t[i].dout ||
                                 t[i].dweight == t[i].out))
      return fail(TSR_ERR_INVALID_ARG, at + "dweight shares memory with another tensor");
    if (t[i].H <= 0) return fail(TSR_ERR_INVALID_ARG, at + "H must be > 0");
    heads += t[i].H;
    bool same = true;
    if (tsr_status e = check_rope_strides(*d, t[i].H, t[i].x_stride, t[i].out_stride, at, &same)) return e;
    if (t[i].x == t[i].out && !same) return fail(TSR_ERR_INVALID_ARG, at + "in place needs equal strides");
    if (grad) {
      if (tsr_status e = check_rope_strides(*d, t[i].H, t[i].dout_stride, t[i].out_stride, at, &same)) return e;
      if (t[i].dout == t[i].out && !same) return fail(TSR_ERR_INVALID_ARG, at + "in place needs equal strides");
    }
    for (int j = 0; j < i; ++j) {
      if (t[i].out == t[j].out || t[i].x == t[j].out || t[i].out == t[j].x ||
          (grad && (t[i].dout == t[j].out || t[i].out == t[j].dout)))
        return fail(TSR_ERR_INVALID_ARG, at + "shares memory with an earlier tensor's output");
      if (grad && t[i].dweight && t[i].dweight == t[j].dweight)
        return fail(TSR_ERR_INVALID_ARG, at + "shares dweight with an earlier tensor");
    }
  }
  if (heads > (1 << 20)) return fail(TSR_ERR_UNSUPPORTED, "more than 2^20 heads");
  return TSR_OK;
}

}  // namespace

extern "C" {

tsr_status tsr_norm_rope(const tsr_rope_desc* desc, double eps, const tsr_norm_rope_tensor* tensors, int32_t n_tensors,
                         void* stream) {
  set_error("");
  if (tsr_status e = check_norm_rope(desc, eps, tensors, n_tensors, false)) return e;
  return launch_norm_rope(*desc, eps, tensors, n_tensors, static_cast<cudaStream_t>(stream));
}

tsr_status tsr_norm_rope_backward_workspace(const tsr_rope_desc* desc, int32_t n_tensors, size_t* bytes) {
  set_error("");
  if (!desc || !bytes) return fail(TSR_ERR_INVALID_ARG, "desc / bytes is NULL");
  if (n_tensors < 1 || n_tensors > 4) return fail(TSR_ERR_INVALID_ARG, "1 to 4 tensors per call");
  if (tsr_status e = check_rope_desc(desc)) return e;
  *bytes = norm_rope_workspace(*desc, n_tensors);
  return TSR_OK;
}

tsr_status tsr_norm_rope_backward(const tsr_rope_desc* desc, double eps, const tsr_norm_rope_tensor* tensors,
                                  int32_t n_tensors, void* workspace, size_t workspace_bytes, void* stream) {
  set_error("");
  if (tsr_status e = check_norm_rope(desc, eps, tensors, n_tensors, true)) return e;
  bool any = false;
  for (int i = 0; i < n_tensors; ++i) any = any || tensors[i].dweight;
  if (any) {
    if (!workspace || !aligned(workspace, 256)) return fail(TSR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < norm_rope_workspace(*desc, n_tensors))
      return fail(TSR_ERR_INVALID_ARG, "workspace too small");
  }
  return launch_norm_rope_backward(*desc, eps, tensors, n_tensors, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

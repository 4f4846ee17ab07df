// api_layer.cu -- the C ABI of a layer's operators between its hidden states and the
// attention: argument checks of the norm with rotation (norm_rope.cu) and of the linear
// layers (linear.cu).
#include <cmath>
#include <string>
#include <utility>

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

// Sizes, and the products of them that the kernels index with.
tsr_status check_linear(const tsr_linear_desc* d) {
  if (!d) return fail(TSR_ERR_INVALID_ARG, "desc is NULL");
  if (d->B <= 0 || d->N <= 0) return fail(TSR_ERR_INVALID_ARG, "B, N must be > 0");
  const int32_t heads[2] = {d->in_heads, d->out_heads}, dim[2] = {d->in_dim, d->out_dim};
  for (int i = 0; i < 2; ++i) {
    const std::string at = i ? "out: " : "in: ";
    if (heads[i] <= 0 || dim[i] <= 0) return fail(TSR_ERR_INVALID_ARG, at + "heads and dim must be > 0");
    if (dim[i] % 8) return fail(TSR_ERR_INVALID_ARG, at + "features must be a multiple of 8");
    if (heads[i] > 1 && dim[i] % 64) return fail(TSR_ERR_INVALID_ARG, at + "dim must be a multiple of 64 with heads");
    if (static_cast<int64_t>(heads[i]) * dim[i] > (1 << 20)) return fail(TSR_ERR_UNSUPPORTED, at + "features above 2^20");
  }
  if (d->dtype != TSR_DTYPE_BF16 && d->dtype != TSR_DTYPE_F16) return fail(TSR_ERR_INVALID_ARG, "dtype must be bf16 or fp16");
  if (d->activation < TSR_ACT_NONE || d->activation > TSR_ACT_SILU) return fail(TSR_ERR_INVALID_ARG, "unknown activation");
  if (static_cast<int64_t>(d->B) * d->N > (1 << 24)) return fail(TSR_ERR_UNSUPPORTED, "B*N above 2^24");
  return TSR_OK;
}

// A tensor of token rows: [B][heads][N][dim] by strides.  `written`: its rows must not run
// into each other.
tsr_status check_rows(const tsr_linear_desc& d, const char* name, const void* p, const int64_t* stride, int32_t heads,
                      int32_t dim, bool written) {
  const std::string at = std::string(name) + ": ";
  if (!p) return fail(TSR_ERR_INVALID_ARG, at + "NULL pointer");
  if (!aligned(p, 16)) return fail(TSR_ERR_INVALID_ARG, at + "must be 16-byte aligned");
  const int64_t size[3] = {d.B, heads, d.N};
  int order[3] = {0, 1, 2};
  for (int k = 0; k < 3; ++k) {
    if (size[k] == 1) continue;
    if (stride[k] <= 0 || stride[k] % 8) return fail(TSR_ERR_INVALID_ARG, at + "strides must be multiples of 8 and > 0");
    if (stride[k] >= (int64_t{1} << 38)) return fail(TSR_ERR_UNSUPPORTED, at + "strides of 2^38 and more");
  }
  if (!written) return TSR_OK;
  for (int a = 0; a < 2; ++a)
    for (int b = a + 1; b < 3; ++b)
      if (stride[order[b]] < stride[order[a]]) std::swap(order[a], order[b]);
  int64_t reach = dim;
  for (int k : order) {
    if (size[k] == 1) continue;
    if (stride[k] < reach) return fail(TSR_ERR_INVALID_ARG, at + "rows overlap");
    reach += stride[k] * (size[k] - 1);
  }
  return TSR_OK;
}

tsr_status check_array(const char* name, const void* p, bool needed) {
  if (!p && needed) return fail(TSR_ERR_INVALID_ARG, std::string(name) + ": NULL pointer");
  if (!aligned(p, 16)) return fail(TSR_ERR_INVALID_ARG, std::string(name) + ": must be 16-byte aligned");
  return TSR_OK;
}

tsr_status check_workspace(const void* p, size_t bytes, size_t need) {
  if (!need) return TSR_OK;
  if (!p || !aligned(p, 256)) return fail(TSR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (bytes < need) return fail(TSR_ERR_INVALID_ARG, "workspace too small");
  return TSR_OK;
}

}  // namespace

extern "C" {

tsr_status tsr_linear_workspace(const tsr_linear_desc* desc, size_t* bytes) {
  set_error("");
  if (!bytes) return fail(TSR_ERR_INVALID_ARG, "bytes is NULL");
  if (tsr_status e = check_linear(desc)) return e;
  *bytes = linear_workspace(*desc);
  return TSR_OK;
}

tsr_status tsr_linear(const tsr_linear_desc* desc, const tsr_linear_args* a, void* workspace, size_t workspace_bytes,
                      void* stream) {
  set_error("");
  if (tsr_status e = check_linear(desc)) return e;
  if (!a) return fail(TSR_ERR_INVALID_ARG, "args is NULL");
  const tsr_linear_desc& d = *desc;
  if (tsr_status e = check_rows(d, "x", a->x, a->x_stride, d.in_heads, d.in_dim, false)) return e;
  if (tsr_status e = check_rows(d, "out", a->out, a->out_stride, d.out_heads, d.out_dim, true)) return e;
  if (tsr_status e = check_array("weight", a->weight, true)) return e;
  if (tsr_status e = check_array("bias", a->bias, false)) return e;
  if (a->residual) {
    if (tsr_status e = check_rows(d, "residual", a->residual, a->residual_stride, d.out_heads, d.out_dim, false)) return e;
    if (a->residual == a->out)
      for (int k = 0; k < 3; ++k)
        if ((k == 0 ? d.B : k == 1 ? d.out_heads : d.N) > 1 && a->residual_stride[k] != a->out_stride[k])
          return fail(TSR_ERR_INVALID_ARG, "residual: in place needs equal strides");
  }
  if (a->pre) {
    if (tsr_status e = check_rows(d, "pre", a->pre, a->pre_stride, d.out_heads, d.out_dim, true)) return e;
    if (a->pre == a->out || a->pre == a->residual) return fail(TSR_ERR_INVALID_ARG, "pre shares memory with another tensor");
  }
  for (const void* w : {static_cast<const void*>(a->out), static_cast<const void*>(a->pre)})
    if (w && (w == a->x || w == a->weight || w == a->bias))
      return fail(TSR_ERR_INVALID_ARG, "an output shares memory with an input");
  if (tsr_status e = check_workspace(workspace, workspace_bytes, linear_workspace(d))) return e;
  return launch_linear(d, *a, workspace, static_cast<cudaStream_t>(stream));
}

tsr_status tsr_linear_backward_workspace(const tsr_linear_desc* desc, size_t* bytes) {
  set_error("");
  if (!bytes) return fail(TSR_ERR_INVALID_ARG, "bytes is NULL");
  if (tsr_status e = check_linear(desc)) return e;
  *bytes = linear_backward_workspace(*desc);
  return TSR_OK;
}

tsr_status tsr_linear_backward(const tsr_linear_desc* desc, const tsr_linear_grads* a, void* workspace,
                               size_t workspace_bytes, void* stream) {
  set_error("");
  if (tsr_status e = check_linear(desc)) return e;
  if (!a) return fail(TSR_ERR_INVALID_ARG, "args is NULL");
  const tsr_linear_desc& d = *desc;
  if (!a->dx && !a->dweight && !a->dbias) return fail(TSR_ERR_INVALID_ARG, "no gradient is asked for");
  if (tsr_status e = check_rows(d, "dout", a->dout, a->dout_stride, d.out_heads, d.out_dim, false)) return e;
  if (d.activation)
    if (tsr_status e = check_rows(d, "pre", a->pre, a->pre_stride, d.out_heads, d.out_dim, false)) return e;
  if (a->dx) {
    if (tsr_status e = check_rows(d, "dx", a->dx, a->dx_stride, d.in_heads, d.in_dim, true)) return e;
    if (tsr_status e = check_array("weight", a->weight, true)) return e;
  }
  if (a->dweight) {
    if (tsr_status e = check_rows(d, "x", a->x, a->x_stride, d.in_heads, d.in_dim, false)) return e;
    if (tsr_status e = check_array("dweight", a->dweight, true)) return e;
  }
  if (tsr_status e = check_array("dbias", a->dbias, false)) return e;
  const void* outs[3] = {a->dx, a->dweight, a->dbias};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i]) continue;
    for (const void* in : {a->dout, a->x, a->weight, a->pre})
      if (outs[i] == in) return fail(TSR_ERR_INVALID_ARG, "a gradient shares memory with an input");
    for (int j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return fail(TSR_ERR_INVALID_ARG, "two gradients share memory");
  }
  if (tsr_status e = check_workspace(workspace, workspace_bytes, linear_backward_workspace(d))) return e;
  return launch_linear_backward(d, *a, workspace, static_cast<cudaStream_t>(stream));
}

tsr_status tsr_linear_test_stall(int32_t on) {
  set_error("");
  if (on != 0 && on != 1) return fail(TSR_ERR_INVALID_ARG, "on must be 0 or 1");
  linear_test_stall(on);
  return TSR_OK;
}

tsr_status tsr_linear_device_status(void* stream) {
  set_error("");
  return linear_device_status(static_cast<cudaStream_t>(stream));
}

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

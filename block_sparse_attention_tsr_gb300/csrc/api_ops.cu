// api_ops.cu -- the C ABI of the operators beside the attention forward: argument
// checks of the position rotation (rope.cu) and the block selection (select.cu).
#include <cmath>
#include <string>

#include "internal.h"

using namespace tsr;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tsr_status check_select(const tsr_select_desc* s) {
  if (!s) return fail(TSR_ERR_INVALID_ARG, "desc is NULL");
  if (s->B <= 0 || s->H <= 0 || s->N <= 0) return fail(TSR_ERR_INVALID_ARG, "B, H, N must be > 0");
  if (s->d != 64 && s->d != 128) return fail(TSR_ERR_INVALID_ARG, "d must be 64 or 128");
  if (s->bq < 16 || s->bk < 16) return fail(TSR_ERR_INVALID_ARG, "bq, bk must be >= 16");
  if (s->keep < 1) return fail(TSR_ERR_INVALID_ARG, "keep must be >= 1");
  if (s->first < 0) return fail(TSR_ERR_INVALID_ARG, "first must be >= 0");
  if (s->N > (1 << 24)) return fail(TSR_ERR_UNSUPPORTED, "N above 2^24");
  if (static_cast<int64_t>(s->B) * s->H > (1 << 20)) return fail(TSR_ERR_UNSUPPORTED, "B*H above 2^20");
  return TSR_OK;
}

}  // namespace

extern "C" {

tsr_status tsr_rope(const tsr_rope_desc* d, const tsr_rope_tensor* t, int32_t n, void* stream) {
  set_error("");
  if (!d || !t) return fail(TSR_ERR_INVALID_ARG, "desc / tensors is NULL");
  if (n < 1 || n > 4) return fail(TSR_ERR_INVALID_ARG, "1 to 4 tensors per call");
  if (d->B <= 0 || d->N <= 0) return fail(TSR_ERR_INVALID_ARG, "B, N must be > 0");
  if (d->d < 2 || d->d > 256 || d->d % 2) return fail(TSR_ERR_INVALID_ARG, "d must be even, 2 to 256");
  if (d->dtype < TSR_DTYPE_BF16 || d->dtype > TSR_DTYPE_F32) return fail(TSR_ERR_INVALID_ARG, "unknown dtype");
  if (d->n_axes < 1 || d->n_axes > 4) return fail(TSR_ERR_INVALID_ARG, "n_axes must be 1 to 4");
  int64_t width = 0, cells = 1;
  for (int a = 0; a < d->n_axes; ++a) {
    if (d->axis_dim[a] <= 0 || d->axis_dim[a] % 2)
      return fail(TSR_ERR_INVALID_ARG, "axis_dim must be even and > 0");
    width += d->axis_dim[a];
    if (!d->positions) {
      if (d->grid[a] <= 0 || d->grid[a] > d->N) return fail(TSR_ERR_INVALID_ARG, "grid does not hold N tokens");
      cells *= d->grid[a];
      if (cells > d->N) return fail(TSR_ERR_INVALID_ARG, "grid does not hold N tokens");
    }
  }
  if (width > d->d) return fail(TSR_ERR_INVALID_ARG, "axis_dim sums to more than d");
  if (!d->positions && cells != d->N) return fail(TSR_ERR_INVALID_ARG, "grid does not hold N tokens");
  if (!(d->theta > 0.0) || !std::isfinite(d->theta)) return fail(TSR_ERR_INVALID_ARG, "theta must be > 0");
  if (d->N > (1 << 24)) return fail(TSR_ERR_UNSUPPORTED, "N above 2^24");
  if (d->B > 65535) return fail(TSR_ERR_UNSUPPORTED, "B above 65535");
  if (d->positions && !aligned(d->positions, 4)) return fail(TSR_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  const size_t es = d->dtype == TSR_DTYPE_F32 ? 4 : 2;
  int64_t heads = 0;
  for (int i = 0; i < n; ++i) {
    const std::string at = "tensor " + std::to_string(i) + ": ";
    if (!t[i].x || !t[i].out) return fail(TSR_ERR_INVALID_ARG, at + "NULL pointer");
    if (!aligned(t[i].x, es) || !aligned(t[i].out, es))
      return fail(TSR_ERR_INVALID_ARG, at + "pointers must be aligned to the element type");
    if (t[i].H <= 0) return fail(TSR_ERR_INVALID_ARG, at + "H must be > 0");
    heads += t[i].H;
    const int64_t size[3] = {d->B, t[i].H, d->N};
    bool same = true;
    for (int k = 0; k < 3; ++k) {
      const int64_t xs = t[i].x_stride[k], os = t[i].out_stride[k];
      if (size[k] == 1) continue;
      same = same && xs == os;
      if (xs < 0 || os < d->d) return fail(TSR_ERR_INVALID_ARG, at + "strides: x >= 0, out >= d");
      if (xs > INT64_MAX / 8 / size[k] || os > INT64_MAX / 8 / size[k])
        return fail(TSR_ERR_INVALID_ARG, at + "strides too large");
    }
    if (t[i].x == t[i].out && !same) return fail(TSR_ERR_INVALID_ARG, at + "in place needs equal strides");
    for (int j = 0; j < i; ++j)
      if (t[i].out == t[j].out || t[i].x == t[j].out || t[i].out == t[j].x)
        return fail(TSR_ERR_INVALID_ARG, at + "shares memory with an earlier tensor's output");
  }
  if (heads > (1 << 20)) return fail(TSR_ERR_UNSUPPORTED, "more than 2^20 heads");
  return launch_rope(*d, t, n, static_cast<cudaStream_t>(stream));
}

tsr_status tsr_block_select_workspace(const tsr_select_desc* desc, size_t* bytes) {
  set_error("");
  if (!bytes) return fail(TSR_ERR_INVALID_ARG, "bytes is NULL");
  if (tsr_status e = check_select(desc)) return e;
  *bytes = select_workspace(*desc);
  return TSR_OK;
}

tsr_status tsr_block_select(const tsr_select_desc* desc, const void* q, const void* k, uint8_t* blocks,
                            void* workspace, size_t workspace_bytes, void* stream) {
  set_error("");
  if (tsr_status e = check_select(desc)) return e;
  if (!q || !k || !blocks || !workspace) return fail(TSR_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(q, 16) || !aligned(k, 16)) return fail(TSR_ERR_INVALID_ARG, "q, k must be 16-byte aligned");
  if (!aligned(workspace, 256)) return fail(TSR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < select_workspace(*desc)) return fail(TSR_ERR_INVALID_ARG, "workspace too small");
  return launch_select(*desc, q, k, blocks, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

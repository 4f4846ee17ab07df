// api_ops.cu -- the C ABI of the operators beside the attention forward: argument
// checks of the position rotation (rope.cu), the block selection (select.cu) and
// the attention backward (bwd.cu) with its plans.
#include <cmath>
#include <cstring>
#include <new>
#include <string>
#include <utility>

#include "internal.h"

using namespace tsr;

// The mask's tiles by query (q: the mask's plan) and by key (k: the plan of its
// transpose, whose block array is held here).
struct tsr_backward_plan_s {
  tsr_plan_t q = nullptr, k = nullptr;
  DevBuf blocks_t;
  bool ready = false;
  int32_t stall = 0;            // test only
};

namespace {

void free_backward(tsr_backward_plan_s* p) {
  if (!p) return;
  if (p->q) tsr_plan_destroy(p->q);
  if (p->k) tsr_plan_destroy(p->k);
  devbuf_free(p->blocks_t);
  delete p;
}

// Both plans for `mask`, made or rebuilt in place.
tsr_status fill_backward(tsr_backward_plan_s* p, const tsr_mask* mask, cudaStream_t st) {
  p->ready = false;
  tsr_plan_opts opts;
  memset(&opts, 0, sizeof opts);
  opts.bn = 64;
  opts.orient = TSR_ORIENT_ROWS;
  opts.kv_split = 1;
  // the mask first: its checks cover the transpose's arguments
  if (tsr_status e = p->q ? tsr_plan_update(p->q, mask, st) : tsr_plan(mask, &opts, &p->q, st)) return e;
  tsr_mask t = *mask;
  int64_t nq, nk;
  if (mask->kind == TSR_MASK_UNIFORM) {
    nq = n_blocks(mask->N, mask->bq);
    nk = n_blocks(mask->N, mask->bk);
    t.bq = mask->bk;
    t.bk = mask->bq;
  } else {
    nq = mask->n_qseg;
    nk = mask->n_kseg;
    t.n_qseg = mask->n_kseg;
    t.n_kseg = mask->n_qseg;
    t.q_bounds = mask->k_bounds;
    t.k_bounds = mask->q_bounds;
  }
  const int64_t heads = static_cast<int64_t>(mask->B) * mask->H;
  if (tsr_status e = devbuf_reserve(p->blocks_t, static_cast<size_t>(heads * nq * nk))) return e;
  t.blocks = static_cast<const uint8_t*>(p->blocks_t.p);
  if (tsr_status e = launch_transpose_blocks(mask->blocks, static_cast<uint8_t*>(p->blocks_t.p), heads,
                                             static_cast<int32_t>(nq), static_cast<int32_t>(nk), st))
    return e;
  if (tsr_status e = p->k ? tsr_plan_update(p->k, &t, st) : tsr_plan(&t, &opts, &p->k, st)) return e;
  p->ready = true;
  return TSR_OK;
}

tsr_status check_backward_kind(const tsr_mask* mask) {
  if (!mask) return fail(TSR_ERR_INVALID_ARG, "mask is NULL");
  if (mask->kind == TSR_MASK_SVG || mask->kind == TSR_MASK_KEYLIST)
    return fail(TSR_ERR_UNSUPPORTED, "the backward pass takes UNIFORM and SEGMENTS masks");
  return TSR_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tsr_status check_select(const tsr_select_desc* s) {
  if (!s) return fail(TSR_ERR_INVALID_ARG, "desc is NULL");
  if (s->B <= 0 || s->H <= 0 || s->N <= 0) return fail(TSR_ERR_INVALID_ARG, "B, H, N must be > 0");
  if (s->d != 64 && s->d != 128) return fail(TSR_ERR_INVALID_ARG, "d must be 64 or 128");
  if (s->bq < 16 || s->bk < 16) return fail(TSR_ERR_INVALID_ARG, "bq, bk must be >= 16");
  if (s->keep < 1) return fail(TSR_ERR_INVALID_ARG, "keep must be >= 1");
  if (s->first < 0) return fail(TSR_ERR_INVALID_ARG, "first must be >= 0");
  if (s->N > (1 << 24)) return fail(TSR_ERR_UNSUPPORTED, "N above 2^24");
  const int64_t heads = static_cast<int64_t>(s->B) * s->H;
  if (heads > (1 << 20)) return fail(TSR_ERR_UNSUPPORTED, "B*H above 2^20");
  if (heads * (static_cast<int64_t>(n_blocks(s->N, s->bq)) + n_blocks(s->N, s->bk)) >= (int64_t{1} << 31))
    return fail(TSR_ERR_UNSUPPORTED, "more than 2^31 blocks");
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
  for (int a = 0; a < d->n_axes; ++a)      // theta^(-2 j / axis_dim) of the last pair
    if (!std::isfinite(std::pow(d->theta, -(d->axis_dim[a] - 2.0) / d->axis_dim[a])))
      return fail(TSR_ERR_INVALID_ARG, "theta is so small that a frequency is not finite");
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
    // the output's rows must not run into each other: each dimension, in order of its
    // stride, steps over all that the smaller ones reach
    int order[3] = {0, 1, 2};
    for (int a = 0; a < 2; ++a)
      for (int b = a + 1; b < 3; ++b)
        if (t[i].out_stride[order[b]] < t[i].out_stride[order[a]]) std::swap(order[a], order[b]);
    int64_t reach = d->d;
    for (int k : order) {
      if (size[k] == 1) continue;
      if (t[i].out_stride[k] < reach) return fail(TSR_ERR_INVALID_ARG, at + "elements of out overlap");
      reach += t[i].out_stride[k] * (size[k] - 1);
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

tsr_status tsr_backward_plan(const tsr_mask* mask, tsr_backward_plan_t* out, void* stream) {
  set_error("");
  if (!out) return fail(TSR_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (tsr_status e = check_backward_kind(mask)) return e;
  tsr_backward_plan_s* p = new (std::nothrow) tsr_backward_plan_s();
  if (!p) return fail(TSR_ERR_OOM, "host allocation failed");
  if (tsr_status e = fill_backward(p, mask, static_cast<cudaStream_t>(stream))) {
    const std::string why = last_error_cstr();
    free_backward(p);
    return fail(e, why);
  }
  *out = p;
  return TSR_OK;
}

tsr_status tsr_backward_plan_update(tsr_backward_plan_t plan, const tsr_mask* mask, void* stream) {
  set_error("");
  if (!plan) return fail(TSR_ERR_INVALID_ARG, "plan is NULL");
  if (tsr_status e = check_backward_kind(mask)) return e;
  // a mask that the plan cannot take leaves it as it was
  const tsr_plan_s* q = plan->q;
  if (mask->B != q->B || mask->H != q->H || mask->N != q->N || mask->d != q->d)
    return fail(TSR_ERR_INVALID_ARG, "tsr_backward_plan_update needs the plan's B, H, N and d");
  return fill_backward(plan, mask, static_cast<cudaStream_t>(stream));
}

tsr_status tsr_backward_plan_destroy(tsr_backward_plan_t plan) {
  free_backward(plan);
  return TSR_OK;
}

tsr_status tsr_backward_plan_device_status(tsr_backward_plan_t plan, void* stream) {
  set_error("");
  if (!plan) return fail(TSR_ERR_INVALID_ARG, "plan is NULL");
  return tsr_plan_device_status(plan->q, stream);
}

tsr_status tsr_backward_plan_test_stall(tsr_backward_plan_t plan, int32_t where) {
  set_error("");
  if (!plan) return fail(TSR_ERR_INVALID_ARG, "plan is NULL");
  if (where < 0 || where > 15) return fail(TSR_ERR_INVALID_ARG, "where must be TSR_BACKWARD_STALL_* bits");
  plan->stall = where;
  return TSR_OK;
}

tsr_status tsr_bsa_backward_workspace(tsr_backward_plan_t plan, size_t* bytes) {
  set_error("");
  if (!plan || !bytes) return fail(TSR_ERR_INVALID_ARG, "plan / bytes is NULL");
  if (!plan->k) return fail(TSR_ERR_INVALID_ARG, "the plan's last update failed");
  *bytes = backward_workspace(plan->q, plan->k);
  return TSR_OK;
}

tsr_status tsr_bsa_backward(const void* q, const void* k, const void* v, const void* out, const float* lse,
                            const void* dout, tsr_backward_plan_t plan, void* dq, void* dk, void* dv,
                            void* workspace, size_t workspace_bytes, void* stream) {
  set_error("");
  if (!plan) return fail(TSR_ERR_INVALID_ARG, "plan is NULL");
  if (!plan->ready) return fail(TSR_ERR_INVALID_ARG, "the plan's last update failed");
  const void* in[6] = {q, k, v, out, dout, lse};
  void* grad[3] = {dq, dk, dv};
  for (const void* t : in) {
    if (!t) return fail(TSR_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned(t, 16)) return fail(TSR_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  }
  for (int i = 0; i < 3; ++i) {
    if (!grad[i]) return fail(TSR_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned(grad[i], 16)) return fail(TSR_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    for (const void* t : in)
      if (grad[i] == t) return fail(TSR_ERR_INVALID_ARG, "a gradient aliases an input");
    for (int j = 0; j < i; ++j)
      if (grad[i] == grad[j]) return fail(TSR_ERR_INVALID_ARG, "two gradients alias");
  }
  if (!workspace || !aligned(workspace, 256))
    return fail(TSR_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < backward_workspace(plan->q, plan->k)) return fail(TSR_ERR_INVALID_ARG, "workspace too small");
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  if (dev != plan->q->device) return fail(TSR_ERR_INVALID_ARG, "plan was made on another device");
  BwdArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.workspace = workspace;
  a.stall = plan->stall;
  a.plan_q = plan->q;
  a.plan_k = plan->k;
  return launch_backward(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

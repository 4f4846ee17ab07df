// internal.h -- library-private declarations shared by the .cu files.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>
#include <string>
#include <vector>

#include "../../include/tsr.h"

namespace tsr {

constexpr int kBM = 128;  // query rows per physical tile (the tcgen05 M = 128 datapath)

void set_error(const std::string& msg);
const char* last_error_cstr();
tsr_status fail(tsr_status s, const std::string& msg);
tsr_status cuda_fail(cudaError_t e, const char* what);

#define TSR_CUDA(expr)                                  \
  do {                                                  \
    cudaError_t e_ = (expr);                            \
    if (e_ != cudaSuccess) return cuda_fail(e_, #expr); \
  } while (0)

// Logical mask as the planner kernels see it (device pointers).
struct MaskDev {
  int32_t kind, B, H, N;
  int32_t bq, bk;
  int32_t n_qseg, n_kseg;
  const int32_t* q_bounds;
  const int32_t* k_bounds;
  const uint8_t* blocks;
  int32_t F, S;
  int32_t R;                 // SVG temporal radius
  const int8_t* head_kind;   // device copy, [H]
  int32_t slice_m;
  const int64_t* indptr;
  const int32_t* indices;
};

// Blocks of b tokens in N (N + b - 1 may pass 2^31).
__host__ __device__ constexpr int32_t n_blocks(int32_t N, int32_t b) { return (N - 1) / b + 1; }

// A UNIFORM mask's block size as MaskDev holds it: a block of 2^24 tokens holds any
// sequence (N <= 2^24), and the planner's products of block sizes and indices (up to
// 8 past the last block) stay in 32 bits.
constexpr int32_t planned_block(int32_t b) { return b < (1 << 24) ? b : (1 << 24); }

struct Regime {
  int32_t bn, stages, ctas, id;
  int32_t orient = TSR_ORIENT_ROWS;   // TSR_ORIENT_ROWS or TSR_ORIENT_KEYS
};

// Query rows per physical tile of an orientation.
constexpr int32_t bm_of(int32_t orient) { return orient == TSR_ORIENT_KEYS ? 64 : kBM; }

// A grow-only device buffer owned by a plan.
struct DevBuf {
  void* p = nullptr;
  size_t cap = 0;
};

struct tsr_plan_impl {
  int device = 0;
  int32_t B = 0, H = 0, N = 0, d = 0;
  int32_t kind = 0;
  int32_t bn = 128, stages = 3, ctas = 1, regime_id = -1;
  int32_t orient = TSR_ORIENT_ROWS, bm = kBM;   // tile orientation and query rows per tile
  int32_t gathered = 0, slice_m = 0;
  int32_t F = 0, S = 0, R = 0;
  int32_t flags = 0;
  int64_t n_items = 0, n_entries = 0, n_desc = 0, n_gidx = 0;
  int64_t n_logical_on = 0, n_logical_total = 0, max_item_len = 0;
  std::vector<int8_t> head_layout;  // host copy: 1 = temporal-major
  int32_t n_temporal = 0;
  int32_t group_heads = 0;    // > 0: heads per longest-first scheduling group (else sized for L2)
  // split-KV: each work item's tile list cut into kv_split parts (1 = off); the
  // parts are the launch's work units, written to `units` in item order
  int32_t kv_split = 1;
  void* units = nullptr;      // tsr_plan_item [n_launch * kv_split] (kv_split > 1)
  // SVG temporal heads of radius 0 with at most 32 frames run as one F x F block
  // per spatial position (svg_temporal.cu); the attention kernels then take the
  // spatial heads' items only: `launch`, the items without the temporal heads'
  // in their scheduled order.  Otherwise launch = items, n_launch = n_items.
  int32_t temporal_band = 0;
  void* launch = nullptr;
  int64_t n_launch = 0;
  std::vector<int64_t> spatial_before;   // [B*H + 1]: spatial heads among bh < i
  // the per-position kernel's stream, forked from the caller's stream before
  // the attention launch and joined after it (created with the first such plan)
  cudaStream_t band_stream = nullptr;
  cudaEvent_t band_fork = nullptr, band_join = nullptr;
  // device buffers (owned)
  void* items = nullptr;     // tsr_plan_item [n_items]
  void* entries = nullptr;   // tsr_plan_entry [n_entries]
  void* descs = nullptr;     // 32 B [n_desc]
  int32_t* gidx = nullptr;   // [n_gidx]
  int32_t* counter = nullptr;
  uint32_t* err = nullptr;
  int8_t* head_kind_dev = nullptr;
  // storage reused when the plan is rebuilt for a new mask (tsr_plan_update)
  DevBuf b_items, b_entries, b_descs, b_cnt, b_tot, b_ebegin, b_dbegin, b_hist, b_gidx;
  // split-KV storage: units, each unit's partial O (fp32 [bm][d]) and lse (base 2,
  // [bm]), one arrival counter per work item
  DevBuf b_units, b_part_o, b_part_lse, b_part_cnt;
  DevBuf b_launch;
  unsigned long long* host_tot = nullptr;   // pinned: 8 totals + the error word
  int8_t* host_kinds = nullptr;             // pinned: SVG head kinds, read after the count sync
  bool has_opts = false;
  tsr_plan_opts opts{};
};

// Make `b` hold at least `bytes` (contents are not preserved when it grows).
tsr_status devbuf_reserve(DevBuf& b, size_t bytes);
void devbuf_free(DevBuf& b);

// planner (plan.cu)
tsr_status plan_build(const tsr_mask* mask, const tsr_plan_opts* opts, tsr_plan_impl* P,
                      cudaStream_t stream);

tsr_status plan_build_keylist(const tsr_mask* mask, const tsr_plan_opts* opts, tsr_plan_impl* P,
                              cudaStream_t stream);
tsr_status plan_schedule_into(const int32_t* cnt_e, const int32_t* cnt_b, int64_t n_items,
                              int32_t nqt, int32_t H, int32_t lpt, int32_t max_len,
                              int32_t group_heads, int32_t* ebegin, int32_t* dbegin,
                              int32_t* hist, void* items, cudaStream_t stream);
// Heads per longest-first scheduling group: as many (b, h) as keep their K and
// V (plus extra_per_head bytes that stream through L2 with them, e.g. gathered
// key indices) within ~96 MB of the L2.
int32_t heads_per_group(int32_t N, int32_t d, int64_t n_heads, double extra_per_head = 0.0);
tsr_status plan_count_into(const MaskDev& m, int32_t nqt, int32_t* cnt, unsigned long long* tot,
                           uint32_t* err, int64_t n_grid, cudaStream_t stream);
tsr_status plan_finish_into(const MaskDev& m, int32_t nqt, int32_t bn, const int32_t* cnt_e,
                            const int32_t* cnt_b, int32_t max_len, int32_t* ebegin,
                            int32_t* dbegin, int32_t* hist, void* items, void* entries,
                            void* descs, cudaStream_t stream);

// The attention launch list (plan.cu): the spatial heads' items when the SVG
// temporal heads go to the per-position kernel, else the items themselves.
tsr_status plan_launch_list(tsr_plan_impl* P, cudaStream_t stream);

// split-KV (plan.cu): the number of parts per work item (the caller's
// opts->kv_split, else enough parts for about eight work units per CTA slot,
// at most 4), and the units and partial-result storage of a split plan
tsr_status plan_split(tsr_plan_impl* P, const tsr_plan_opts* opts, cudaStream_t stream);

// device-side plan consistency checks (check.cu)
tsr_status plan_check(const tsr_plan_impl* P, cudaStream_t stream);

// forward kernels (fwd.cu)
struct FwdArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const tsr_plan_impl* plan;
  // Work items [item_lo, item_hi) of the plan (item_hi < 0: all of them), and
  // the launch's own work counter (null: the plan's).  Launches of one plan
  // that may run at the same time need disjoint item ranges and their own
  // counters, and no debug tile counting.
  int64_t item_lo = 0, item_hi = -1;
  int32_t* counter = nullptr;
};
tsr_status launch_forward(const FwdArgs& a, cudaStream_t stream);
// Up to 16 requests in one launch (same d, regime and mask family).
tsr_status launch_forward_batch(const FwdArgs* reqs, int n_req, cudaStream_t stream);
bool variant_exists(int d, int bn, int stages, int ctas, bool gathered);
bool variant_pick(int d, bool gathered, int bn, int stages, int ctas, int* out_bn, int* out_st,
                  int* out_ct);
// The regime for a plan: the table's choice, with the caller's overrides (opts
// fields that are nonzero) taking precedence; completed to a compiled variant.
tsr_status resolve_regime(Regime table, const tsr_plan_opts* opts, int d, bool gathered,
                          Regime* out);

// SVG head routing (route.cu)
tsr_status launch_route(const void* q, const void* k, const void* v, int32_t B, int32_t H,
                        int32_t F, int32_t S, int32_t d, int32_t R, const int32_t* samples,
                        int32_t n_samples, float* stats, int8_t* head_kind, cudaStream_t stream);

// SVG temporal heads, one F x F block per spatial position (svg_temporal.cu):
// radius 0, 1 <= F <= 32, d in {64, 128}.  Heads bh in [bh_lo, bh_hi) whose kind
// is temporal; the others are left alone.
bool svg_temporal_eligible(int32_t F, int32_t R, int32_t d);
tsr_status launch_svg_temporal(const void* q, const void* k, const void* v, void* out, float* lse,
                               int32_t H, int32_t N, int32_t d, int32_t F, int32_t S,
                               const int8_t* head_kind, int64_t bh_lo, int64_t bh_hi,
                               cudaStream_t stream);

// argument checks that several operators share (api_ops.cu)
bool aligned(const void* p, size_t a);
tsr_status check_rope_desc(const tsr_rope_desc* d);
tsr_status check_rope_strides(const tsr_rope_desc& d, int32_t H, const int64_t* x_stride, const int64_t* out_stride,
                              const std::string& at, bool* same);

// multi-axis rotary positions (rope.cu)
tsr_status launch_rope(const tsr_rope_desc& d, const tsr_rope_tensor* t, int32_t n, cudaStream_t stream);

// norm of every head's row and rotation (norm_rope.cu)
tsr_status launch_norm_rope(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n,
                            cudaStream_t st);
size_t norm_rope_workspace(const tsr_rope_desc& d, int32_t n);
tsr_status launch_norm_rope_backward(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n,
                                     void* ws, cudaStream_t st);

// linear layers (linear.cu)
size_t linear_workspace(const tsr_linear_desc& d);
size_t linear_backward_workspace(const tsr_linear_desc& d);
tsr_status launch_linear(const tsr_linear_desc& d, const tsr_linear_args& a, void* ws, cudaStream_t st);
tsr_status launch_linear_backward(const tsr_linear_desc& d, const tsr_linear_grads& a, void* ws, cudaStream_t st);
tsr_status linear_device_status(cudaStream_t st);
void linear_test_stall(int32_t on);

// block selection (select.cu)
size_t select_workspace(const tsr_select_desc& s);
tsr_status launch_select(const tsr_select_desc& s, const void* q, const void* k, uint8_t* blocks, void* ws,
                         cudaStream_t stream);

// backward pass (bwd.cu): the mask's plan (query items) and its transpose's (key
// items), both 128-row tiles 64 wide
struct BwdArgs {
  const void *q, *k, *v, *out;
  const float* lse;
  const void* dout;
  void *dq, *dk, *dv;
  void* workspace;              // backward_workspace() bytes
  int32_t stall;                // test only: TSR_BACKWARD_STALL_* bits
  const tsr_plan_impl *plan_q, *plan_k;
};
tsr_status launch_backward(const BwdArgs& a, cudaStream_t stream);
size_t backward_workspace(const tsr_plan_impl* plan_q, const tsr_plan_impl* plan_k);
// blocks uint8 [heads][nq][nk] -> [heads][nk][nq]
tsr_status launch_transpose_blocks(const uint8_t* src, uint8_t* dst, int64_t heads, int32_t nq, int32_t nk,
                                   cudaStream_t stream);

// permutation (permute.cu)
tsr_status launch_permute(const void* src, void* dst, int32_t B, int32_t H, int32_t F, int32_t S,
                          int32_t row_bytes, const int8_t* head_kind_host, int32_t inverse,
                          cudaStream_t stream);

// regime table (api.cu)
Regime regime_lookup(int32_t kind, int32_t bq, int32_t bk, int32_t N, double density, int32_t d);

// tensor maps (fwd.cu)
bool encode_tmap_3d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows,
                    uint64_t outer, uint32_t box_inner, uint32_t box_rows);

int num_sms(int device);

// What has been done on each device (an attribute of a function is its own on each).  Calls
// of several threads may both find it undone: it is done twice then, to the same end.
class OncePerDevice {
 public:
  bool done(int device) const { return device >= 0 && device < 64 && done_[device].load(std::memory_order_acquire); }
  void mark(int device) {
    if (device >= 0 && device < 64) done_[device].store(true, std::memory_order_release);
  }

 private:
  std::atomic<bool> done_[64] = {};
};

// The limit of a kernel's dynamic shared memory; `once`: the kernel's own.
template <typename Kern>
tsr_status allow_smem(Kern kern, size_t bytes, int device, OncePerDevice& once) {
  if (once.done(device)) return TSR_OK;
  TSR_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)));
  once.mark(device);
  return TSR_OK;
}

// Launch a kernel that may start while the stream's previous kernel finishes
// (programmatic dependent launch): it has to call grid_wait() before it touches
// anything that kernel reads or writes, and then reads what that kernel wrote with
// plain loads (__ldg may be moved above the wait).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                             A&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<A&&>(args)...);
}

}  // namespace tsr

struct tsr_plan_s : tsr::tsr_plan_impl {};

// linear.cu -- linear layers y = act(x W^T + b) + residual and their gradients: the host
// side of the products (linear_gemm.cuh), the sum of a split product's parts, and the pass
// over the output's gradient that comes before the products of the backward,
//     dz = dout o act'(pre),   dbias = sum of dz over the tokens.
// dz is rounded to the tensors' type: the tensor cores take 16-bit operands, and dz in two of
// them (its rounding and the rest) would be twice the products.  That rounding is as large as
// the output's own, so the gradients' errors are 1.4 times those of one rounding (bf16 0.0024
// for 0.0017 of their norm, fp16 0.00029 for 0.00021); in fp16 a dz past 65,504 is an infinity.
// dbias is summed in fp32 from the unrounded dz, in a fixed order.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "internal.h"
#include "linear_gemm.cuh"

namespace tsr {

namespace linear {

namespace {

constexpr int kSms = 152;              // what the choice of tiles is made for
constexpr uint64_t kStallNs = 20000000;    // bound of the waits of a stalled product (test only)
thread_local int32_t g_stall = 0;

// D's values of the tiles that were cut along k, from their parts, in their order.  L2-bound;
// of eight parts and more, eight groups of threads add up an eighth each (a loop over 76 of
// them alone took 10 us of 20, 128 x 128 from 32,760 tokens; 10 to 14 in all now).
constexpr int kGroupedParts = 8;
template <int BN, int G>
__global__ void __launch_bounds__(256) linear_finish_kernel(const __grid_constant__ GemmParams p) {
  constexpr int VECS = BN / 8, EACH = 256 / G;
  __shared__ F2 red[G > 1 ? G : 1][G > 1 ? EACH : 1][4];
  const int at = threadIdx.x % EACH, g = threadIdx.x / EACH;
  const int64_t i = blockIdx.x * static_cast<int64_t>(EACH) + at;
  const int64_t rest = p.by_cut.d, cut = i / (256 * VECS);
  const int32_t row = static_cast<int32_t>(i / VECS) % 256, c = static_cast<int32_t>(i % VECS) * 8;
  grid_wait();
  const int2 rc = tile_of(p, p.whole + static_cast<uint32_t>(min(cut, rest - 1)));
  const int32_t b = p.by_batch(rc.x), n = (rc.x - b * static_cast<int32_t>(p.by_batch.d)) * 256 + row, f = rc.y * BN + c;
  const bool on = cut < rest && n < p.n_rows && f < p.cols;
  // a CTA that gave up has not stored its parts: nothing is added then
  static_assert(kMostCtas == 32 * sizeof(uint2), "a warp reads them");
  const uint2 gave_up = reinterpret_cast<const uint2*>(p.gave_up)[threadIdx.x & 31];
  F2 v[4] = {};
  if (on) {
    const int32_t s1 = p.splits * (g + 1) / G;
#pragma unroll 4
    for (int32_t s = p.splits * g / G; s < s1; ++s) {
      const float4* src = reinterpret_cast<const float4*>(p.part + ((s * rest + cut) * 256 + row) * BN + c);
      const float4 x = src[0], y = src[1];
      v[0] = add2(v[0], pack2(x.x, x.y));
      v[1] = add2(v[1], pack2(x.z, x.w));
      v[2] = add2(v[2], pack2(y.x, y.y));
      v[3] = add2(v[3], pack2(y.z, y.w));
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) red[g][at][k] = v[k];
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      for (int h = 1; h < G; ++h) v[k] = add2(v[k], red[h][at][k]);
  }
  if (__any_sync(0xFFFFFFFFu, gave_up.x | gave_up.y)) return;
  if (on) by_kind(p.epi.f16, p.epi.act, [&](auto f16, auto act) { finish8<f16.value, act.value>(p.epi, v, b, n, f); });
}

struct DzParams {
  const uint16_t *dout, *pre;          // pre: null without activation
  uint16_t* dz;                        // [rows][cols], null: dout itself is the operand
  float* part;                         // [row blocks][cols], null: no dbias
  View vdout, vpre;
  int64_t rows;
  int32_t n_rows, cols, rows_per_block, lanes_log2, act, f16;
};

// 8, 16 or 32 lanes of 8 columns, 32, 16 or 8 rows at a time.
__global__ void __launch_bounds__(256, 4) linear_dz_kernel(const __grid_constant__ DzParams p) {
  __shared__ float red[256][8];
  const int lanes = 1 << p.lanes_log2, rows = 256 >> p.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1), ty = threadIdx.x >> p.lanes_log2;
  const int32_t f = (blockIdx.x * lanes + lane) * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per_block;
  const int64_t r1 = min(r0 + p.rows_per_block, p.rows);
  grid_launch_dependents();
  F2 sum[4] = {};
  if (f < p.cols)
    by_kind(p.f16, p.act, [&](auto f16, auto act) {
      constexpr int kRows = act.value == TSR_ACT_NONE ? 8 : 4;      // in flight
#pragma unroll kRows
      for (int64_t r = r0 + ty; r < r1; r += rows) {
        int64_t b = 0, n = r;
        if (p.n_rows < p.rows) {
          b = r / p.n_rows;
          n = r - b * p.n_rows;
        }
        F2 g[4];
        unpack8<f16.value>(*reinterpret_cast<const uint4*>(p.dout + at(p.vdout, b, n, f)), g);
        if constexpr (act.value != TSR_ACT_NONE) {
          F2 z[4];
          unpack8<f16.value>(*reinterpret_cast<const uint4*>(p.pre + at(p.vpre, b, n, f)), z);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], slope<act.value>(z[i]));
        }
        if (p.dz) *reinterpret_cast<uint4*>(p.dz + r * p.cols + f) = pack8<f16.value>(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = add2(sum[i], g[i]);
      }
    });
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2(sum[i]);
    red[threadIdx.x][2 * i] = x.x;
    red[threadIdx.x][2 * i + 1] = x.y;
  }
  __syncthreads();
  const int c = threadIdx.x;           // a column of the block's
  const int32_t col = blockIdx.x * lanes * 8 + c;
  float s = 0.f;
  if (c >= lanes * 8 || col >= p.cols) return;
  for (int k = 0; k < rows; ++k) s += red[k * lanes + (c >> 3)][c & 7];
  p.part[static_cast<int64_t>(blockIdx.y) * p.cols + col] = s;
}

// Column sums of the row blocks' sums: 32 columns a CTA, 32 rows at a time.
__global__ void __launch_bounds__(1024) linear_bias_kernel(const float* part, int32_t blocks, int32_t cols, void* out,
                                                           int32_t f16) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  grid_wait();
  grid_pass_on();                      // dz, to the products, which do not wait for this grid
  grid_launch_dependents();
  float s = 0.f;
  if (c < cols)
    for (int i = slice; i < blocks; i += 32) s += part[static_cast<int64_t>(i) * cols + c];
  red[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    if (f16) static_cast<__half*>(out)[c] = __float2half_rn(s);
    else static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
  }
}

size_t round256(size_t x) { return (x + 255) & ~size_t{255}; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ----------------------------------------------------------- choice of tiles
enum Kind { FORWARD, DX, DWEIGHT };
enum Variant { PAIR_256, PAIR_128, FEW_32, FEW_128 };

struct Choice {
  Variant variant;
  int32_t splits;
  int64_t whole;                       // tiles that are not cut along k (pairs)
};

// Rows, columns and k of a product: D is [batches x n_rows][cols].
struct Product {
  int64_t batches, n_rows, cols, k_steps;
  Kind kind;
};

// The fastest by a model in microseconds: waves of units, each its k steps and a fill and an
// epilogue; where pairs' tiles are cut a launch and the parts' traffic.  With 32 tokens 70 CTAs
// take what the L2 gives; clusters of 4 and 8 CTAs leave SMs free.  Each part has four steps at
// least.  The constants are a fit to timed products; of 270 (forward, dx and dweight, 1 to 44,340
// tokens, 64 to 8,192 features, profiles/linear_choice.txt) the choice is on average 1.6% behind
// the fastest (up to 300 tokens 2.9%, up to 512 1.1%, above 0.6%), 33% at most.  For example
// 666 x 4096 -> 2048: 14 us on 256 x 128 tiles, 22 on 256 x 256, 18 with k in three parts; 1 x
// 4096 -> 4096: 10 us (8.2 with the weight in L2) with the token on 32 columns and k in four
// parts, 27 on 256 x 128.
Choice choose(const Product& q) {
  constexpr double kStep[4] = {0.298, 0.18, 0.156, 0.188}, kUnit[4] = {1.5, 1.27, 3.35, 4.4};
  constexpr int kTok[4] = {256, 256, 32, 128}, kFeat[4] = {256, 128, 128, 128};
  Choice best{PAIR_256, 1, 0};
  double least = 1e30;
  for (int v = PAIR_256; v <= FEW_128; ++v) {
    const bool few = v >= FEW_32;
    if (few && (q.kind == DWEIGHT || q.batches * q.n_rows > 512)) continue;   // above, clusters were not timed
    const int64_t tiles = q.batches * cdiv(q.n_rows, kTok[v]) * cdiv(q.cols, kFeat[v]);
    // more than 16 parts only of tiles that are too few for the pairs
    for (int64_t s = 1; s <= (few ? 8 : std::max<int64_t>(16, kSms / 2 / tiles)) && (s == 1 || q.k_steps >= 4 * s);
         s += few ? s : 1) {
      const int64_t slots = !few ? kSms / 2 : v == FEW_32 ? (s < 4 ? 300 : 256) : s == 8 ? 96 : s == 4 ? 128 : 150;
      const int64_t whole = s == 1 ? tiles : few ? 0 : tiles / slots * slots, rest = tiles - whole;
      if (s > 1 && !rest) continue;
      const double crowd = v == FEW_32 ? std::max(1.0, std::min<double>(static_cast<double>(tiles * s), slots) / 70) : 1.0;
      double t = cdiv(whole, slots) * (q.k_steps * kStep[v] * crowd + kUnit[v]) +
                 cdiv(rest * s, slots) * (cdiv(q.k_steps, s) * kStep[v] * crowd + kUnit[v]);
      if (few) t += 0.11 * s + (v == FEW_128 && s > 1 ? 2.4 : 0.0);
      else t += 2.75 + (s > 1 ? 2.6 + 0.66e-6 * s * rest * kTok[v] * kFeat[v] : 0.0);
      if (t < least) {
        least = t;
        best = {static_cast<Variant>(v), static_cast<int32_t>(s), whole};
      }
    }
  }
  return best;
}

// Row tiles of a group.  A B that stays in L2 is read again at no cost: two, so that A's rows
// are through soonest (2048 -> 6144, 32,760 tokens: 482 us, of eight 490; its dx 490 for 505).
// Else eight by some nine columns run together on 76 pairs, the fewest rows and columns of
// all shapes (8192 -> 2048, dweight, 8 x 32 tiles: of eight 654 us, of two 695; 5120 -> 5120,
// 9,000 tokens: 291, of two 294); two where there are no more columns than that anyway (2048
// -> 8192, dweight, 32 x 8 tiles: of two 654, of eight 672).
uint32_t group_log2(const Product& q, int64_t col_tiles) {
  return q.cols * q.k_steps * BK * 2 <= 40 << 20 || col_tiles < 10 ? 1 : 3;
}

// The parts of a product, and behind them a byte for each CTA.
size_t part_bytes(const Product& q, const Choice& c) {
  if (c.splits == 1 || c.variant >= FEW_32) return 0;
  const int bn = c.variant == PAIR_256 ? 256 : 128;
  return static_cast<size_t>(q.batches * cdiv(q.n_rows, 256) * cdiv(q.cols, bn) - c.whole) * c.splits * 256 * bn * 4;
}
size_t part_space(const Product& q) {
  const size_t parts = part_bytes(q, choose(q));
  return parts ? parts + kMostCtas : 0;
}

// ---------------------------------------------------------------- the layer
struct Layer {
  int64_t B, N, K, M;                  // tokens B x N, in and out features
  int32_t in_heads, in_dim, out_heads, out_dim;
  bool f16;
};
Layer layer_of(const tsr_linear_desc& d) {
  return {d.B, d.N, static_cast<int64_t>(d.in_heads) * d.in_dim, static_cast<int64_t>(d.out_heads) * d.out_dim,
          d.in_heads, d.in_dim, d.out_heads, d.out_dim, d.dtype == TSR_DTYPE_F16};
}
Product product(const Layer& y, Kind kind) {
  if (kind == DWEIGHT) return {1, y.M, y.K, y.B * cdiv(y.N, BK), kind};
  return {y.B, y.N, kind == FORWARD ? y.M : y.K, cdiv(kind == FORWARD ? y.K : y.M, BK), kind};
}
// Tokens of all batches as one row of tokens, where every tensor of the call allows it.
bool flat(const Layer& y, const View& v) { return y.B == 1 || y.N == 1 || v.sb == y.N * v.sn; }
void flatten(Layer& y, View* const* views, int n) {
  for (int i = 0; i < n; ++i)
    if (!flat(y, *views[i])) return;
  for (int i = 0; i < n; ++i)
    if (y.N == 1) views[i]->sn = views[i]->sb;
  y.N *= y.B;
  y.B = 1;
}
size_t most_parts(const tsr_linear_desc& d, Kind kind) {
  Layer y = layer_of(d);
  const size_t a = part_space(product(y, kind));
  if (y.B == 1) return a;
  y.N *= y.B;
  y.B = 1;
  return std::max(a, part_space(product(y, kind)));
}

View view(const int64_t* stride, int32_t dim) { return {stride[0], stride[1], stride[2], dim}; }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// A 4-D tensor map, 128-byte swizzle; strides in elements, of dimensions 1 to 3.
tsr_status encode(CUtensorMap* m, const void* p, CUtensorMapDataType type, int size, const int64_t (&dims)[4],
                  const int64_t (&strides)[3], int box0, int box1) {
  // no promotion of misses to longer L2 fetches: it cost up to 6% where rows are not lines
  // the box's row of 128 or 64 bytes is the swizzle's
  if (!encoder()) return fail(TSR_ERR_CUDA, "cuTensorMapEncodeTiled is missing");
  cuuint64_t d[4], s[3];
  for (int i = 0; i < 4; ++i) d[i] = static_cast<cuuint64_t>(dims[i]);
  for (int i = 0; i < 3; ++i) s[i] = static_cast<cuuint64_t>(dims[i + 1] > 1 ? size * strides[i] : 16);
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box0), static_cast<cuuint32_t>(box1), 1, 1}, es[4] = {1, 1, 1, 1};
  if (encoder()(m, type, 4, const_cast<void*>(p), d, s, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                box0 * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(TSR_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  return TSR_OK;
}
// {channel, token, head, batch} boxes of `channels` x `rows` tokens.
tsr_status encode(CUtensorMap* m, const void* p, const View& v, int64_t heads, int64_t n, int64_t b, int channels,
                  int rows, bool f16) {
  return encode(m, p, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                {v.dim, n, heads, b}, {v.sn, v.sh, v.sb}, channels, rows);
}

// A kernel that may set itself up while what is before it on the stream ends (it waits for
// that before it touches memory), in clusters of `cluster` CTAs.
tsr_status launch_clusters(void (*kern)(GemmParams), OncePerDevice& once, int smem, int64_t ctas, int cluster,
                           const GemmParams& p, cudaStream_t st) {
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  if (tsr_status e = allow_smem(kern, smem, dev, once)) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  TSR_CUDA(cudaLaunchKernelEx(&cfg, kern, p));
  return TSR_OK;
}

template <int BN, bool A_MN, bool B_MN>
tsr_status launch_pairs(const GemmParams& p, cudaStream_t st) {
  static OncePerDevice once;
  const int64_t rest = static_cast<int64_t>(p.row_tiles) * p.col_tiles - p.whole;
  if (tsr_status e = launch_clusters(linear_gemm_kernel<BN, A_MN, B_MN>, once, Cfg<BN>::SMEM, p.ctas, 2, p, st)) return e;
  if (rest) {
    const bool many = p.splits >= kGroupedParts;
    TSR_CUDA(launch_dependent(many ? linear_finish_kernel<BN, 8> : linear_finish_kernel<BN, 1>,
                              static_cast<unsigned>(rest * BN / 8 * (many ? 8 : 1)), 256u, 0, st, p));
  }
  return TSR_OK;
}
template <int BN, bool W_MN>
tsr_status launch_few(const GemmParams& p, cudaStream_t st) {
  static OncePerDevice once;
  return launch_clusters(linear_few_kernel<BN, W_MN>, once, FewCfg<BN>::SMEM,
                         static_cast<int64_t>(p.row_tiles) * p.col_tiles * p.splits, p.splits, p, st);
}

template <bool A_MN, bool B_MN>
tsr_status launch_kind(Variant v, const GemmParams& p, cudaStream_t st) {
  if (v == PAIR_256) return launch_pairs<256, A_MN, B_MN>(p, st);
  if (v == PAIR_128) return launch_pairs<128, A_MN, B_MN>(p, st);
  if constexpr (!A_MN) {
    if (v == FEW_32) return launch_few<32, B_MN>(p, st);
    return launch_few<128, B_MN>(p, st);
  }
  return fail(TSR_ERR_INTERNAL, "no kernel for this product");
}

// One product with its epilogue.  `tok`: the tensor whose rows are tokens (x or dz),
// `other`: the weight, or x for the weight's gradient.
tsr_status run(const Layer& y, Kind kind, const void* tok, const View& vtok, int64_t tok_heads, const void* other,
               const View& vother, int64_t other_heads, const Epilogue& e, float* ws, bool late, bool pass_on,
               cudaStream_t st) {
  const Product q = product(y, kind);
  const Choice c = choose(q);
  const bool few = c.variant >= FEW_32;
  GemmParams p;
  memset(&p, 0, sizeof p);
  p.epi = e;
  p.part = ws;
  p.n_rows = static_cast<int32_t>(q.n_rows);
  p.cols = static_cast<int32_t>(q.cols);
  p.splits = c.splits;
  p.k_steps = static_cast<int32_t>(q.k_steps);
  p.k_each = static_cast<uint32_t>(q.k_steps / c.splits);
  p.k_more = static_cast<uint32_t>(q.k_steps % c.splits);
  p.k_steps_per_batch = static_cast<int32_t>(cdiv(y.N, BK));
  p.late = late;
  p.pass_on = pass_on;
  p.stall = g_stall;
  p.timeout_ns = g_stall ? kStallNs : kWaitTimeoutNs;
  const int bn = c.variant == PAIR_256 ? 256 : c.variant == FEW_32 ? 32 : 128;
  const int64_t per_batch = cdiv(q.n_rows, few ? bn : 256), col_tiles = cdiv(q.cols, few ? 128 : bn);
  const int64_t tiles = per_batch * q.batches * col_tiles, rest = tiles - c.whole;
  if (c.whole + rest * c.splits > INT32_MAX) return fail(TSR_ERR_UNSUPPORTED, "a linear layer of too many tiles");
  p.row_tiles = static_cast<int32_t>(per_batch * q.batches);
  p.col_tiles = static_cast<int32_t>(col_tiles);
  p.by_batch = div_by(static_cast<uint32_t>(per_batch));
  if (few) {
    std::swap(p.row_tiles, p.col_tiles);
  } else {
    p.whole = static_cast<uint32_t>(c.whole);
    p.units = static_cast<uint32_t>(c.whole + rest * c.splits);
    p.group_log2 = group_log2(q, col_tiles);
    // of one group that holds all tiles only the remainders are taken
    p.by_group = div_by(static_cast<uint32_t>(std::min<int64_t>(col_tiles << p.group_log2, INT32_MAX)));
    p.by_cut = div_by(static_cast<uint32_t>(std::max<int64_t>(rest, 1)));
    p.out_dim = div_by(e.vout.dim);
    int dev = 0;
    TSR_CUDA(cudaGetDevice(&dev));
    p.ctas = 2 * std::min<uint32_t>(p.units, std::min(num_sms(dev), kMostCtas) / 2);
    if (rest) p.gave_up = reinterpret_cast<uint8_t*>(ws) + part_bytes(q, c);
  }
  CUtensorMap *mt = few ? &p.tb : &p.ta, *mo = few ? &p.ta : &p.tb;
  (few ? p.b_dim : p.a_dim) = div_by(vtok.dim);
  (few ? p.a_dim : p.b_dim) = div_by(vother.dim);
  const bool tok_mn = kind == DWEIGHT, other_mn = kind != FORWARD;
  const int tok_rows = tok_mn ? BK : few ? bn : 128, other_rows = other_mn ? BK : few ? 128 : bn / 2;
  if (tsr_status s = encode(mt, tok, vtok, tok_heads, y.N, y.B, BK, tok_rows, y.f16)) return s;
  const int64_t on = kind == DWEIGHT ? y.N : y.M, ob = kind == DWEIGHT ? y.B : 1;
  if (tsr_status s = encode(mo, other, vother, other_heads, on, ob, BK, other_rows, y.f16)) return s;
  p.idesc = idesc_16bit(y.f16, few ? 128 : 256, bn, few ? other_mn : tok_mn, few ? tok_mn : other_mn);
  if (!few) {
    // out's rows: tokens, or the weight's for its gradient
    const int64_t rows = q.n_rows, heads = q.cols / e.vout.dim;
    if (c.whole) {
      const int width = e.pre ? 32 : 64;
      if (tsr_status s = encode(&p.tout, e.out, e.vout, heads, rows, q.batches, width, 32, y.f16)) return s;
      if (e.pre)
        if (tsr_status s = encode(&p.tpre, e.pre, e.vpre, heads, rows, q.batches, width, 32, y.f16)) return s;
      if (e.res)
        if (tsr_status s = encode(&p.tres, e.res, e.vres, heads, rows, q.batches, width, 32, y.f16)) return s;
    }
    if (rest)
      if (tsr_status s = encode(&p.tpart, p.part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, {bn, 256, rest, c.splits},
                                {bn, 256 * bn, rest * 256 * bn}, 32, 32))
        return s;
  }
  if (kind == FORWARD) return launch_kind<false, false>(c.variant, p, st);
  if (kind == DX) return launch_kind<false, true>(c.variant, p, st);
  return launch_kind<true, true>(c.variant, p, st);
}

// Lanes of a row in the pass over dz: as many as leave the fewest idle.
int dz_lanes_log2(int64_t M) {
  int best = 5;
  for (int l = 4; l >= 3; --l)
    if (cdiv(M, 8 << l) << l < cdiv(M, 8 << best) << best) best = l;
  return best;
}
// Blocks of rows of it: one wave of the four CTAs that an SM holds (dbias alone of 32,760 x
// 8,192 with the tanh GELU, 1.07 GB read, 208 us; twice as many and one more 245).
int64_t dz_blocks(int64_t T, int64_t M) {
  return std::max<int64_t>(1, std::min(cdiv(T, 32), kSms * 4 / cdiv(M, 8 << dz_lanes_log2(M))));
}

struct BackwardSpace {
  size_t dz, sums, parts, total;
};
BackwardSpace backward_space(const tsr_linear_desc& d) {
  const Layer y = layer_of(d);
  BackwardSpace s;
  s.dz = 0;
  s.sums = s.dz + (d.activation ? round256(static_cast<size_t>(y.B * y.N * y.M) * 2) : 0);
  s.parts = s.sums + round256(static_cast<size_t>(dz_blocks(y.B * y.N, y.M) * y.M) * 4);
  s.total = s.parts + round256(std::max(most_parts(d, DX), most_parts(d, DWEIGHT)));
  return s;
}

}  // namespace

}  // namespace linear

using namespace linear;

size_t linear_workspace(const tsr_linear_desc& d) { return round256(most_parts(d, FORWARD)); }
size_t linear_backward_workspace(const tsr_linear_desc& d) { return backward_space(d).total; }

// The arguments of both have been checked (api_layer.cu).
tsr_status launch_linear(const tsr_linear_desc& d, const tsr_linear_args& a, void* ws, cudaStream_t st) {
  Layer y = layer_of(d);
  View vx = view(a.x_stride, y.in_dim);
  Epilogue e;
  memset(&e, 0, sizeof e);
  e.bias = a.bias;
  e.res = a.residual;
  e.out = a.out;
  e.pre = a.pre;
  e.vout = view(a.out_stride, y.out_dim);
  e.vres = view(a.residual_stride, y.out_dim);
  e.vpre = view(a.pre_stride, y.out_dim);
  e.act = d.activation;
  e.f16 = y.f16;
  View* views[4] = {&vx, &e.vout};
  int n = 2;
  if (a.residual) views[n++] = &e.vres;
  if (a.pre) views[n++] = &e.vpre;
  flatten(y, views, n);
  const View vw{0, 0, y.K, static_cast<int32_t>(y.K)};
  return run(y, FORWARD, a.x, vx, y.in_heads, a.weight, vw, 1, e, static_cast<float*>(ws), false, false, st);
}

tsr_status launch_linear_backward(const tsr_linear_desc& d, const tsr_linear_grads& a, void* ws, cudaStream_t st) {
  Layer y = layer_of(d);
  const BackwardSpace space = backward_space(d);
  char* base = static_cast<char*>(ws);
  View vx = view(a.x_stride, y.in_dim), vdx = view(a.dx_stride, y.in_dim);
  View vdout = view(a.dout_stride, y.out_dim), vpre = view(a.pre_stride, y.out_dim);
  View* views[4] = {&vdout};
  int n = 1;
  if (a.dweight) views[n++] = &vx;
  if (a.dx) views[n++] = &vdx;
  if (d.activation) views[n++] = &vpre;
  flatten(y, views, n);
  const void* dz = a.dout;
  View vdz = vdout;
  int64_t dz_heads = y.out_heads;
  const bool operands = a.dx || a.dweight;
  if ((d.activation && operands) || a.dbias) {
    DzParams p;
    memset(&p, 0, sizeof p);
    p.dout = static_cast<const uint16_t*>(a.dout);
    p.pre = d.activation ? static_cast<const uint16_t*>(a.pre) : nullptr;
    p.dz = d.activation && operands ? reinterpret_cast<uint16_t*>(base + space.dz) : nullptr;
    p.part = a.dbias ? reinterpret_cast<float*>(base + space.sums) : nullptr;
    p.vdout = vdout;
    p.vpre = vpre;
    p.rows = y.B * y.N;
    p.n_rows = static_cast<int32_t>(y.N);
    p.cols = static_cast<int32_t>(y.M);
    p.act = d.activation;
    p.f16 = y.f16;
    int64_t blocks = dz_blocks(p.rows, y.M);
    p.lanes_log2 = dz_lanes_log2(y.M);
    p.rows_per_block = static_cast<int32_t>(cdiv(p.rows, blocks));
    blocks = cdiv(p.rows, p.rows_per_block);
    linear_dz_kernel<<<dim3(static_cast<unsigned>(cdiv(y.M, 8 << p.lanes_log2)), static_cast<unsigned>(blocks)), 256, 0, st>>>(p);
    TSR_CUDA(cudaGetLastError());
    if (a.dbias)
      TSR_CUDA(launch_dependent(linear_bias_kernel, static_cast<unsigned>(cdiv(y.M, 32)), 1024u, 0, st,
                                static_cast<const float*>(p.part), static_cast<int32_t>(blocks), p.cols, a.dbias,
                                p.f16));
    if (p.dz) {
      dz = p.dz;
      vdz = View{y.N * y.M, 0, y.M, static_cast<int32_t>(y.M)};
      dz_heads = 1;
    }
  }
  float* part = reinterpret_cast<float*>(base + space.parts);
  Epilogue e;
  memset(&e, 0, sizeof e);
  e.f16 = y.f16;
  // A product's CTAs may start as those of the kernel before leave, where that kernel has
  // waited for the products' inputs, passed them on (grid_pass_on) and writes nothing that the
  // product touches: behind the sum of dbias, and dweight behind a dx whose tiles are not cut
  // (its parts would share their memory).
  bool late = a.dbias != nullptr;
  if (a.dx) {
    e.out = a.dx;
    e.vout = vdx;
    const View vw{0, 0, y.K, static_cast<int32_t>(y.K)};
    const bool uncut = part_space(product(y, DX)) == 0;
    if (tsr_status s = run(y, DX, dz, vdz, dz_heads, a.weight, vw, 1, e, part, late, late || (a.dweight && uncut), st))
      return s;
    late = uncut;
  }
  if (a.dweight) {
    e.out = a.dweight;
    e.vout = View{0, 0, y.K, static_cast<int32_t>(y.K)};
    return run(y, DWEIGHT, dz, vdz, dz_heads, a.x, vx, y.in_heads, e, part, late, late, st);
  }
  return TSR_OK;
}

void linear_test_stall(int32_t on) { g_stall = on; }

tsr_status linear_device_status(cudaStream_t st) {
  uint32_t word = 0;
  void* at = nullptr;
  TSR_CUDA(cudaGetSymbolAddress(&at, g_err));
  TSR_CUDA(cudaMemcpyAsync(&word, at, sizeof word, cudaMemcpyDeviceToHost, st));
  TSR_CUDA(cudaMemsetAsync(at, 0, sizeof word, st));
  TSR_CUDA(cudaStreamSynchronize(st));
  if (word & DEV_ERR_TIMEOUT) return fail(TSR_ERR_TIMEOUT, "a wait in a linear layer's product gave up");
  if (word) return fail(TSR_ERR_INTERNAL, "a linear layer's product found its memory misaligned");
  return TSR_OK;
}

}  // namespace tsr

// tara_layer.cu -- C entry points of the operators around the attention: argument checks and
// launches of the rotary table, the norm and rotation of Q and K, the linear layer and the
// Q/K/V projection.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "tara_attn.h"
#include "forward_internal.h"
#include "layer_checks.h"
#include "linear_pair.cuh"
#include "linear_simt.cuh"
#include "linear_skinny.cuh"
#include "norm_rope.cuh"

namespace tara {
namespace {

int launched() { return cudaGetLastError() == cudaSuccess ? TARA_OK : TARA_ERR_CUDA; }

// ---------------------------------------------------------------------------------------
// norm and rotation
// ---------------------------------------------------------------------------------------
// CTAs that keep every SM of the device busy through a few rounds.
constexpr long long kNormRopeFill = 148 * 16;

template <typename T, int LANES>
int launch_norm_rope(NormRopeArgs a, int B, int n_tensors, bool halves, cudaStream_t stream) {
  const int rows = kNormRopeThreads / LANES;
  const long long gx = ((long long)a.N + rows - 1) / rows;
  // one CTA walks as many heads as leave the device a few CTAs per SM (the table is read once
  // per CTA and token), at least one batch
  const long long want = (kNormRopeFill + gx * B * n_tensors - 1) / (gx * B * n_tensors);
  a.heads_per_cta = (int)std::max<long long>(4, (a.H + want - 1) / want);
  a.chunks = (a.H + a.heads_per_cta - 1) / a.heads_per_cta;
  const dim3 grid((unsigned)gx, (unsigned)(n_tensors * a.chunks), (unsigned)B);
  if (halves)
    norm_rope_kernel<T, LANES, true><<<grid, kNormRopeThreads, 0, stream>>>(a);
  else
    norm_rope_kernel<T, LANES, false><<<grid, kNormRopeThreads, 0, stream>>>(a);
  return launched();
}

template <typename T>
int launch_norm_rope_t(const NormRopeArgs& a, int B, int nt, bool halves, cudaStream_t stream) {
  if (a.D <= 64) return launch_norm_rope<T, 8>(a, B, nt, halves, stream);
  if (a.D <= 128) return launch_norm_rope<T, 16>(a, B, nt, halves, stream);
  return launch_norm_rope<T, 32>(a, B, nt, halves, stream);
}

int run_norm_rope(const tara_view* q, const tara_view* k, const tara_norm_rope* p,
                  const tara_view* q_out, const tara_view* k_out, cudaStream_t stream) {
  NormRopeArgs a{};
  const tara_view* in[2] = {q, k};
  const tara_view* out[2] = {q_out, k_out};
  const void* weight[2] = {p->q_weight, p->k_weight};
  const int nt = k ? 2 : 1;
  for (int i = 0; i < nt; ++i) {
    const tara_view vi = normalised(*in[i]), vo = normalised(*out[i]);
    a.t[i] = NormRopeTensor{vi.ptr, vo.ptr, weight[i], vi.stride_b, vi.stride_h, vi.stride_n,
                            vo.stride_b, vo.stride_h, vo.stride_n};
  }
  a.table = p->table;
  a.table_b = p->table_batch_stride;
  a.weight_h = p->weight_head_stride;
  a.H = q->H;
  a.N = q->N;
  a.D = q->D;
  a.rot = p->table ? p->rot_dim : 0;
  a.norm = p->norm;
  a.eps = p->eps;
  a.inv_d = 1.0f / (float)q->D;
  const bool halves = p->pairing == TARA_ROPE_HALVES;
  if (q->dtype == TARA_BF16) return launch_norm_rope_t<__nv_bfloat16>(a, q->B, nt, halves, stream);
  if (q->dtype == TARA_FP16) return launch_norm_rope_t<__half>(a, q->B, nt, halves, stream);
  return launch_norm_rope_t<float>(a, q->B, nt, halves, stream);
}

// ---------------------------------------------------------------------------------------
// linear
// ---------------------------------------------------------------------------------------
RowView row_view(const tara_view& v) {
  const tara_view n = normalised(v);
  return RowView{n.ptr, n.stride_b, n.stride_h, n.stride_n, n.D};
}

// A view of the linear layer: 16-bit views are read and written by 16-byte chunks, x by 64-column
// boxes of a tensor map (whose strides may not be 0); the fp32 kernels take anything.  The kernels
// count x's columns in int and step past the last one, by less than kLinearStep.
constexpr int64_t kLinearStep = 256;

int check_linear_view(const tara_view* v, bool out, bool is_x) {
  if (!v) return TARA_ERR_NULL;
  const int align = v->dtype == TARA_FP32 ? 0 : 16;
  const int rc = out ? check_out_view(v, align) : check_view(v, align);
  if (rc != TARA_OK) return rc;
  if (is_x && (int64_t)v->H * v->D > ((int64_t)1 << 31) - kLinearStep) return TARA_ERR_TOO_LARGE;
  if (v->dtype == TARA_FP32) return TARA_OK;
  if (v->D % 8 != 0 || (v->H > 1 && v->D % 64 != 0)) return TARA_ERR_SHAPE;
  if (is_x && ((v->B > 1 && v->stride_b == 0) || (v->H > 1 && v->stride_h == 0) ||
               (v->N > 1 && v->stride_n == 0)))
    return TARA_ERR_PARAM;
  return TARA_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map of a row-major 16-bit array of up to 4 dimensions (innermost first; strides of
// dimensions 1.. in elements): 128-byte-swizzled boxes of 64 columns x box_rows.
int encode_map(const DeviceInfo& dev, CUtensorMap* map, tara_dtype dt, const void* ptr, int rank,
               const long long* dims, const long long* strides, int box_rows) {
  cuuint64_t gdim[4], gstr[3];
  cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, estr[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) gdim[i] = (cuuint64_t)dims[i];
  // the stride of a dimension of size 1 is never used, but has to be a valid one
  for (int i = 1; i < rank; ++i)
    gstr[i - 1] = dims[i] == 1 ? (cuuint64_t)((dims[0] + 7) / 8 * 16) : (cuuint64_t)strides[i] * 2;
  const CUresult r = reinterpret_cast<EncodeTiledFn>(dev.encode_tiled)(
      map, dt == TARA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      (cuuint32_t)rank, const_cast<void*>(ptr), gdim, gstr, box, estr,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TARA_OK : TARA_ERR_CUDA;
}

// [B][H][N][D] view with `cols` columns of rows in all.
int encode_view(const DeviceInfo& dev, CUtensorMap* map, tara_dtype dt, const RowView& v, int B,
                int N, int cols, int box_rows) {
  const long long dims[4] = {v.D, N, cols / v.D, B}, strides[4] = {1, v.n, v.h, v.b};
  return encode_map(dev, map, dt, v.ptr, 4, dims, strides, box_rows);
}

int encode_weights(const DeviceInfo& dev, CUtensorMap* map, tara_dtype dt, const void* w, int C,
                   int K, int box_rows) {
  const long long dims[2] = {K, C}, strides[2] = {1, K};
  return encode_map(dev, map, dt, w, 2, dims, strides, box_rows);
}

template <bool kBF16, int BN, int kSubs, int kEpi>
struct PairLauncher {
  static int allow(const DeviceInfo& dev) {
    static std::mutex mu;
    static uint64_t done = 0;   // one bit per device
    std::lock_guard<std::mutex> lock(mu);
    if (done >> dev.index & 1) return TARA_OK;
    // the kernel's register split draws on exactly this many registers a thread
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, linear_pair_kernel<kBF16, BN, kSubs, kEpi>) != cudaSuccess ||
        fa.numRegs != kPairLinRegs)
      return TARA_ERR_CUDA;
    if (cudaFuncSetAttribute(linear_pair_kernel<kBF16, BN, kSubs, kEpi>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PairLin<BN, kSubs>::kSmemBytes) != cudaSuccess)
      return TARA_ERR_CUDA;
    done |= (uint64_t)1 << dev.index;
    return TARA_OK;
  }
  static int launch(const DeviceInfo& dev, const PairLinArgs& args, tara_dtype dt,
                    cudaStream_t stream) {
    int rc;
    if ((rc = allow(dev)) != TARA_OK) return rc;
    const LinearArgs& a = args.lin;
    PairLinArgs p = args;
    PairLinMaps maps;
    if ((rc = encode_view(dev, &maps.x, dt, a.x, a.B, a.N, a.K, 128)) != TARA_OK ||
        (rc = encode_weights(dev, &maps.w, dt, a.w, a.C, a.K, p.bn / 2)) != TARA_OK)
      return rc;
    constexpr int rows = 256 * kSubs;
    p.m_tiles = (int)(((long long)a.N + rows - 1) / rows);
    p.n_tiles = (int)(((long long)a.C + p.bn - 1) / p.bn);
    p.group = 8 / kSubs;
    const long long tiles = (long long)a.B * p.m_tiles * p.n_tiles;
    const long long clusters = std::min<long long>(tiles, std::max(1, dev.sms / 2));
    linear_pair_kernel<kBF16, BN, kSubs, kEpi>
        <<<(unsigned)(2 * clusters), kPairLinThreads, PairLin<BN, kSubs>::kSmemBytes, stream>>>(maps, p);
    return launched();
  }
};

// Folds the branches into one run of rows where every view allows it and nothing is per branch.
void merge_branches(LinearArgs* a) {
  if (a->B == 1 || a->gate_b != 0 || (long long)a->B * a->N > 0x7fffffffLL) return;
  auto runs_on = [a](const RowView& v) { return a->N == 1 ? true : v.b == v.n * a->N; };
  const int parts = a->C / a->part_cols;
  if (!runs_on(a->x) || (a->residual.ptr && !runs_on(a->residual))) return;
  for (int i = 0; i < parts; ++i)
    if (!runs_on(a->y[i])) return;
  if (a->N == 1) {
    a->x.n = a->x.b;
    a->residual.n = a->residual.b;
    for (int i = 0; i < parts; ++i) a->y[i].n = a->y[i].b;
  }
  a->N *= a->B;
  a->B = 1;
}

template <bool kBF16, int BN, int kSubs>
int launch_pair(const DeviceInfo& dev, const PairLinArgs& p, bool heads, tara_dtype dt,
                cudaStream_t stream) {
  if (heads) return PairLauncher<kBF16, BN, kSubs, kEpiHeads>::launch(dev, p, dt, stream);
  switch (p.lin.act) {
    case 1: return PairLauncher<kBF16, BN, kSubs, 1>::launch(dev, p, dt, stream);
    case 2: return PairLauncher<kBF16, BN, kSubs, 2>::launch(dev, p, dt, stream);
    case 3: return PairLauncher<kBF16, BN, kSubs, 3>::launch(dev, p, dt, stream);
    default: return PairLauncher<kBF16, BN, kSubs, 0>::launch(dev, p, dt, stream);
  }
}

template <bool kBF16, int kT, bool kQkv>
int launch_skinny(const DeviceInfo& dev, SkinnyArgs p, int zs, tara_dtype dt, cudaStream_t stream) {
  using S = SkinnyLin<kT>;
  static std::mutex mu;
  static uint64_t done = 0;   // one bit per device
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(done >> dev.index & 1)) {
      if (cudaFuncSetAttribute(linear_skinny_kernel<kBF16, kT, kQkv>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               S::kSmemBytes) != cudaSuccess)
        return TARA_ERR_CUDA;
      done |= (uint64_t)1 << dev.index;
    }
  }
  const LinearArgs& a = p.lin;
  PairLinMaps maps;
  RowView x = a.x;
  if (p.rows != a.N && a.N == 1) x.n = x.b;            // the branches run on as rows
  int rc;
  if ((rc = encode_view(dev, &maps.x, dt, x, zs, p.rows, a.K, kT)) != TARA_OK ||
      (rc = encode_weights(dev, &maps.w, dt, a.w, a.C, a.K, 128)) != TARA_OK)
    return rc;
  const long long c_tiles = ((long long)a.C + 127) / 128, t_tiles = ((long long)p.rows + kT - 1) / kT;
  // The split of K by the estimated time, in K steps of a CTA by itself.  CTAs that share an SM
  // wait for memory much of the time: two of them take about 1.4 times as long as one.  Each CTA
  // an SM runs costs about 4 steps beyond its own (start, the join over the cluster, the end).
  // (7,168 -> 7,168, 1 row: 1 to 8 CTAs a tile take 36, 22, 16 and 20 us; 1,024 -> 4,096, 128 rows:
  // 11.7, 10.8, 9.4 and 13.7; 4,096 -> 1,024, 1 row: 18.7, 12.2, 8.5 and 6.7.)
  const long long tiles = c_tiles * t_tiles * zs, steps = (a.K + 63) / 64;
  const double sms = dev.sms, room = (double)S::kCtas * dev.sms;
  double best = 0.0;
  for (int s = 1; s <= 8 && s <= steps; s *= 2) {
    const double ctas = (double)(tiles * s);
    const double share = std::max(1.0, 0.7 * std::min(ctas, room) / sms);
    const double cost = std::ceil(ctas / room) * std::ceil((double)steps / s) * share +
                        4.0 * std::ceil(ctas / sms);
    if (s == 1 || cost < best) {
      best = cost;
      p.splits = s;
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(c_tiles * p.splits), (unsigned)t_tiles, (unsigned)zs);
  cfg.blockDim = dim3(kSkinnyThreads);
  cfg.dynamicSmemBytes = S::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, linear_skinny_kernel<kBF16, kT, kQkv>, maps, p) != cudaSuccess) {
    cudaGetLastError();   // a refused launch leaves nothing behind for the next call's check
    return TARA_ERR_CUDA;
  }
  return TARA_OK;
}

template <bool kBF16, bool kQkv>
int launch_skinny_rows(const DeviceInfo& dev, const SkinnyArgs& p, int zs, tara_dtype dt,
                       cudaStream_t stream) {
  if (p.rows <= 16) return launch_skinny<kBF16, 16, kQkv>(dev, p, zs, dt, stream);
  if (p.rows <= 32) return launch_skinny<kBF16, 32, kQkv>(dev, p, zs, dt, stream);
  if (p.rows <= 64) return launch_skinny<kBF16, 64, kQkv>(dev, p, zs, dt, stream);
  if (p.rows <= 128) return launch_skinny<kBF16, 128, kQkv>(dev, p, zs, dt, stream);
  return launch_skinny<kBF16, 256, kQkv>(dev, p, zs, dt, stream);
}

// Whether the kernel that streams W takes a call of `rows` rows: up to 128 (7,168 -> 7,168, 128
// rows: 26 us against 34), and up to 256 where the output is too narrow to give the pair kernel's
// tiles to many SMs but K is long enough to split (4,096 -> 1,024, 129 to 256 rows: 11 to 14 us
// against 21; at 7,168 -> 7,168 31 to 38 against 35, at 7,168 -> 21,504 115 to 130 against 72 to 77).
bool streams_weights(long long rows, int C, int K, int sms) {
  return rows <= 128 || (rows <= 256 && (C + 127LL) / 128 * 8 <= sms && K >= 2048);
}

// head: the norm and rotation of a projection's q and k, or nullptr.
int run_linear(LinearArgs a, const HeadArgs* head, tara_dtype dt, cudaStream_t stream) {
  if (dt == TARA_FP32) {
    if (a.N <= kSimtRows) {
      const int cols_cta = kSimtLinThreads / 32 * kRowsCols;
      const dim3 grid((unsigned)(((long long)a.C + cols_cta - 1) / cols_cta), (unsigned)a.B);
      if (a.N == 1)
        linear_simt_rows_kernel<1><<<grid, kSimtLinThreads, 0, stream>>>(a);
      else if (a.N == 2)
        linear_simt_rows_kernel<2><<<grid, kSimtLinThreads, 0, stream>>>(a);
      else if (a.N <= 4)
        linear_simt_rows_kernel<4><<<grid, kSimtLinThreads, 0, stream>>>(a);
      else
        linear_simt_rows_kernel<kSimtRows><<<grid, kSimtLinThreads, 0, stream>>>(a);
      return launched();
    }
    auto tiles = [&a](long long m) { return dim3((unsigned)((a.N + m - 1) / m),
                                                 (unsigned)((a.C + m - 1) / m), (unsigned)a.B); };
    // the large tiles as soon as they give every other SM one
    const dim3 big = tiles(128), small = tiles(32);
    const bool large = (long long)big.x * big.y * big.z >= 74;
    if ((large ? big.y : small.y) > 65535) return TARA_ERR_TOO_LARGE;
    if (large)
      linear_simt_kernel<128, 16><<<big, kSimtLinThreads, 0, stream>>>(a);
    else
      linear_simt_kernel<32, 64><<<small, kSimtLinThreads, 0, stream>>>(a);
    return launched();
  }
  DeviceInfo dev;
  int rc = device_info(&dev);
  if (rc != TARA_OK) return rc;
  a.status = dev.status;
  const bool heads = head != nullptr;
  if (streams_weights((long long)a.B * a.N, a.C, a.K, dev.sms)) {
    SkinnyArgs p{};
    p.lin = a;
    if (head) p.head = *head;
    // one run of rows over all branches where x allows it: W is read once
    const bool runs_on = a.B == 1 || a.N == 1 || a.x.b == a.x.n * a.N;
    p.rows = runs_on ? a.B * a.N : a.N;
    const int zs = runs_on ? 1 : a.B;
    if (dt == TARA_BF16)
      return heads ? launch_skinny_rows<true, true>(dev, p, zs, dt, stream)
                   : launch_skinny_rows<true, false>(dev, p, zs, dt, stream);
    return heads ? launch_skinny_rows<false, true>(dev, p, zs, dt, stream)
                 : launch_skinny_rows<false, false>(dev, p, zs, dt, stream);
  }
  if (!head || !head->table) merge_branches(&a);
  // the kernel numbers its tiles in int
  const long long tiles128 = (long long)a.B * (((long long)a.N + 255) / 256) *
                             (((long long)a.C + 127) / 128);
  if (tiles128 > 0x3fffffffLL) return TARA_ERR_TOO_LARGE;
  PairLinArgs p{};
  p.lin = a;
  if (head) p.head = *head;
  // Tile width by the estimated cycles of a cluster's rounds.  A 64-column K step of a 256 x bn
  // tile takes 2 * bn cycles of the tensor cores, and its (256 + bn) * 64 bytes an SM arrive at
  // about 64 bytes a cycle, which is the larger up to 256 columns.  What a call costs beyond its
  // products (filling the ring, the last tile's epilogue; the epilogues of earlier rounds run
  // under the next products) counts as 8 K steps.  Widths between
  // 128 and 256 are for rows of one head and one part, where a tile may end anywhere (512 x 7,168
  // -> 7,168 on 74 SM pairs: 70 tiles of 208 columns, 42 us, instead of 56 of 256, 44 us).
  const int pairs = std::max(1, dev.sms / 2);
  const long long k_steps = ((long long)a.K + 63) / 64;
  const long long m_tiles = (long long)a.B * (((long long)a.N + 255) / 256);
  const bool any_width = !heads && a.part_cols == a.C && a.y[0].D == a.C &&
                         (!a.residual.ptr || a.residual.D == a.C);
  long long best = 0;
  for (int bn = 256; bn >= 128; bn -= any_width ? 16 : 128) {
    const long long tiles = m_tiles * (((long long)a.C + bn - 1) / bn);
    const long long cost = (tiles + pairs - 1) / pairs * k_steps * (256 + bn) + 8 * (256 + bn);
    if (best == 0 || cost < best) {
      best = cost;
      p.bn = bn;
    }
  }
  // 512 x 256 reads a quarter less through L2 than 256 x 256, but its accumulators fill tensor
  // memory, so part of every epilogue is exposed (about 5,000 cycles).  Long calls run at the
  // power cap, where the saved traffic counts for more.  Back to back for half a second each,
  // 512-row against 256-row tiles, by K steps and rounds of 256 x 256 tiles:
  //   112 steps: 24 rounds 1.33 and 1.35 ms, 48 rounds 2.63 and 2.72, 78 rounds 4.34 and 4.5,
  //     158 rounds 9.2 and 10.2, 475 rounds 28.0 and 33.4;
  //   88 steps, 158 rounds: 6.9 and 7.5 ms;
  //   64 steps: 34 rounds 1.10 and 1.06 ms, 78 rounds 2.49 and 2.47, 158 rounds 5.0 and 5.1,
  //     475 rounds 14.9 and 17.8;
  //   32 steps, 78 rounds: 1.31 and 1.21 ms.
  // The rule starts where the two meet.
  const bool tall = k_steps >= 64 && tiles128 / 2 >= 32LL * pairs;
  if (tall) p.bn = 256;
  const bool narrow = p.bn == 128;
  if (dt == TARA_BF16) {
    if (tall) return launch_pair<true, 256, 2>(dev, p, heads, dt, stream);
    if (!narrow) return launch_pair<true, 256, 1>(dev, p, heads, dt, stream);
    return launch_pair<true, 128, 1>(dev, p, heads, dt, stream);
  }
  if (tall) return launch_pair<false, 256, 2>(dev, p, heads, dt, stream);
  if (!narrow) return launch_pair<false, 256, 1>(dev, p, heads, dt, stream);
  return launch_pair<false, 128, 1>(dev, p, heads, dt, stream);
}

// The whole per-token column count of a view.
int64_t columns(const tara_view& v) { return (int64_t)v.H * v.D; }

}  // namespace
}  // namespace tara

using namespace tara;

extern "C" {

int tara_rope_table(const float* pos, int64_t n_rows, const tara_rope* rope, float* table,
                    void* stream) {
  if (!pos || !rope || !table) return TARA_ERR_NULL;
  if (rope->n_axes < 1 || rope->n_axes > TARA_ROPE_MAX_AXES) return TARA_ERR_PARAM;
  if (n_rows < 1) return TARA_ERR_SHAPE;
  int R = 0;
  for (int a = 0; a < rope->n_axes; ++a) {
    if (!(rope->theta[a] > 0.0) || !std::isfinite(rope->theta[a])) return TARA_ERR_PARAM;
    if (rope->dim[a] < 2 || rope->dim[a] % 2 != 0 || rope->dim[a] > 2 * kRopeMaxPairs)
      return TARA_ERR_SHAPE;
    R += rope->dim[a];
  }
  if (R > 2 * kRopeMaxPairs || R % 4 != 0) return TARA_ERR_SHAPE;
  if (!ptr_aligned(pos, 4) || !ptr_aligned(table, 16)) return TARA_ERR_ALIGN;
  RopeFreqs fr{};
  fr.n_axes = rope->n_axes;
  for (int a = 0; a < rope->n_axes; ++a)
    for (int i = 0; i < rope->dim[a] / 2; ++i) {
      fr.axis[fr.n_pairs] = (uint8_t)a;
      fr.quarter_turns[fr.n_pairs++] =
          std::pow(rope->theta[a], -2.0 * i / rope->dim[a]) * 0.63661977236758134308;   // 2/pi
    }
  // one row a thread, up to the CTAs that run together
  const long long rows_step = kRopeThreads / (fr.n_pairs / 2);
  const long long grid = std::min<long long>((n_rows - 1) / rows_step + 1, 148 * kRopeCtas);
  if (n_rows > ((int64_t)1 << 40)) return TARA_ERR_TOO_LARGE;
  rope_table_kernel<<<(unsigned)grid, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      pos, n_rows, fr, reinterpret_cast<float4*>(table));
  return launched();
}

int tara_qk_norm_rope(const tara_view* q, const tara_view* k, const tara_norm_rope* p,
                      tara_view* q_out, tara_view* k_out, void* stream) {
  if (!q || !p || !q_out || (k == nullptr) != (k_out == nullptr)) return TARA_ERR_NULL;
  int rc;
  if ((rc = check_view(q, 16)) != TARA_OK || (rc = check_out_view(q_out, 16)) != TARA_OK)
    return rc;
  if (k && ((rc = check_view(k, 16)) != TARA_OK || (rc = check_out_view(k_out, 16)) != TARA_OK))
    return rc;
  const tara_view* all[4] = {q, q_out, k, k_out};
  for (const tara_view* v : all) {
    if (!v) continue;
    if (v->dtype != q->dtype) return TARA_ERR_DTYPE;
    if (!same_shape(*v, *q)) return TARA_ERR_SHAPE;
  }
  if (q->D % 8 != 0 || q->D > 256) return TARA_ERR_HEAD_DIM;
  if (2LL * q->H > 65535) return TARA_ERR_TOO_LARGE;
  if ((rc = check_norm_rope(p, q->D, q->N, q->dtype)) != TARA_OK) return rc;
  // an output is its own input, or starts elsewhere than every other view
  if (q_out->ptr == q->ptr && !same_layout(*q_out, *q)) return TARA_ERR_PARAM;
  if (k) {
    if (k_out->ptr == k->ptr && !same_layout(*k_out, *k)) return TARA_ERR_PARAM;
    if (q_out->ptr == k->ptr || k_out->ptr == q->ptr || q_out->ptr == k_out->ptr)
      return TARA_ERR_PARAM;
  }
  return run_norm_rope(q, k, p, q_out, k_out, static_cast<cudaStream_t>(stream));
}

int tara_linear(const tara_view* x, const void* w, const tara_epilogue* e, tara_view* y,
                void* stream) {
  if (!x || !w || !y) return TARA_ERR_NULL;
  int rc;
  if ((rc = check_linear_view(x, false, true)) != TARA_OK || (rc = check_linear_view(y, true, false)) != TARA_OK)
    return rc;
  if (x->dtype != y->dtype) return TARA_ERR_DTYPE;
  if (x->B != y->B || x->N != y->N) return TARA_ERR_SHAPE;
  const uintptr_t align = x->dtype == TARA_FP32 ? 4 : 16;
  if (!ptr_aligned(w, align)) return TARA_ERR_ALIGN;
  if (y->ptr == x->ptr || y->ptr == w) return TARA_ERR_PARAM;
  LinearArgs a{};
  a.x = row_view(*x);
  a.y[0] = row_view(*y);
  a.w = w;
  a.B = x->B;
  a.N = x->N;
  a.K = (int)columns(*x);
  a.C = (int)columns(*y);
  a.part_cols = a.C;
  if (e) {
    if (e->act < TARA_ACT_NONE || e->act > TARA_ACT_SILU) return TARA_ERR_PARAM;
    if (e->gate && e->gate_stride != 0 && e->gate_stride < a.C) return TARA_ERR_PARAM;
    if (!ptr_aligned(e->bias, align) || !ptr_aligned(e->gate, align)) return TARA_ERR_ALIGN;
    if (e->gate && (e->gate_stride * elem_size(x->dtype)) % (int)align != 0) return TARA_ERR_ALIGN;
    a.bias = e->bias;
    a.act = e->act;
    a.gate = e->gate;
    a.gate_b = e->gate_stride;
    if (e->residual) {
      const tara_view* r = e->residual;
      if ((rc = check_linear_view(r, false, false)) != TARA_OK) return rc;
      if (r->dtype != x->dtype) return TARA_ERR_DTYPE;
      if (r->B != y->B || r->N != y->N || columns(*r) != columns(*y)) return TARA_ERR_SHAPE;
      if (r->ptr == y->ptr && !same_layout(*r, *y)) return TARA_ERR_PARAM;
      a.residual = row_view(*r);
    }
  }
  return run_linear(a, nullptr, x->dtype, static_cast<cudaStream_t>(stream));
}

int tara_qkv_project(const tara_view* x, const void* w, const void* bias,
                     const tara_norm_rope* p, tara_view* q, tara_view* k, tara_view* v,
                     void* stream) {
  if (!x || !w || !q || !k || !v) return TARA_ERR_NULL;
  int rc;
  if ((rc = check_linear_view(x, false, true)) != TARA_OK) return rc;
  const tara_view* outs[3] = {q, k, v};
  for (const tara_view* o : outs) {
    if ((rc = check_out_view(o, 16)) != TARA_OK) return rc;
    if (o->dtype != x->dtype) return TARA_ERR_DTYPE;
    if (!same_shape(*o, *q) || o->B != x->B || o->N != x->N) return TARA_ERR_SHAPE;
    if (o->ptr == x->ptr || o->ptr == w) return TARA_ERR_PARAM;
  }
  if (q->ptr == k->ptr || q->ptr == v->ptr || k->ptr == v->ptr) return TARA_ERR_PARAM;
  if (q->dtype == TARA_FP32 ? (q->D % 8 != 0 || q->D > 256) : (q->D != 64 && q->D != 128))
    return TARA_ERR_HEAD_DIM;
  if (2LL * q->H > 65535 || 3 * columns(*q) > 0x7fffffffLL) return TARA_ERR_TOO_LARGE;
  const uintptr_t align = x->dtype == TARA_FP32 ? 4 : 16;
  if (!ptr_aligned(w, align) || !ptr_aligned(bias, align)) return TARA_ERR_ALIGN;
  if (p && (rc = check_norm_rope(p, q->D, q->N, q->dtype)) != TARA_OK) return rc;
  LinearArgs a{};
  a.x = row_view(*x);
  for (int i = 0; i < 3; ++i) a.y[i] = row_view(*outs[i]);
  a.w = w;
  a.bias = bias;
  a.B = x->B;
  a.N = x->N;
  a.K = (int)columns(*x);
  a.part_cols = (int)columns(*q);
  a.C = 3 * a.part_cols;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (x->dtype == TARA_FP32) {
    if ((rc = run_linear(a, nullptr, x->dtype, st)) != TARA_OK || !p) return rc;
    return run_norm_rope(q, k, p, q, k, st);
  }
  HeadArgs head{};
  if (p) {
    head.weight[0] = p->norm ? p->q_weight : nullptr;
    head.weight[1] = p->norm ? p->k_weight : nullptr;
    head.weight_h = p->weight_head_stride;
    head.table = p->table;
    head.table_b = p->table_batch_stride;
    head.D = q->D;
    head.rot = p->table ? p->rot_dim : 0;
    head.halves = p->pairing == TARA_ROPE_HALVES;
    head.norm = p->norm;
    head.eps = p->eps;
    head.inv_d = 1.0f / (float)q->D;
  }
  return run_linear(a, p ? &head : nullptr, x->dtype, st);
}

}  // extern "C"

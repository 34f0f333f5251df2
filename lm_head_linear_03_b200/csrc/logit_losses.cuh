// Post-training losses on given logits, and the row steps that they share with
// the fused head.
//
// The post-training part of the library the pages describe ("Liger-Kernel:
// Triton kernels that replace HF training ops", section "Installation and the
// one-line patch") takes the output layer's logits or its inputs and returns a
// loss.  Two of these losses live here:
//
//   clipped policy loss with a KL term.  With x = z/T and lp = x_y - lse(x),
//     r = exp(lp - old),  kl = exp(ref - lp) - (ref - lp) - 1,
//     L = -min(r A, clip(r, 1 - lo, 1 + hi) A) + beta kl - eta H,
//     H = lse(x) - sum_j p_j x_j                      (the row's entropy)
//     dL/dlp = -A r [r not clipped away] + beta (1 - exp(ref - lp)) = g
//     dL/dz_j = (g ([j == y] - p_j) + eta p_j (log p_j + H)) / T
//
//   distillation from a teacher's K largest logits u_k at entries t_k,
//     q = softmax_K(u/T), or exp(u/T - lse_teacher) with the teacher's own
//     normaliser,  Q = sum_k q_k,
//     L = kd sum_k q_k (log q_k - log p_{t_k}) + ce (lse(z) - z_y),  p = softmax(z/T),
//     dL/dz_j = kd/T (Q p_j - sum_{k: t_k = j} q_k) + ce (softmax(z)_j - [j == y]).
//
// Both gradients are a dense part that depends on the row's softmax alone and a
// few sparse entries, so one kernel serves both.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "flce_kernels.cuh"

namespace flce {

constexpr int DISTILL_MAX_K = 1024;
// Lower logits count as LOGIT_LOWEST in the policy loss, whose sums hold e (z - m):
// the difference is finite whatever finite m is, so that a probability of 0 adds
// 0.  A register without a logit holds LOGIT_NONE, which has probability 0 beside
// any logit.  Powers of two: the same value in bf16.
constexpr float LOGIT_LOWEST = -0x1p40f, LOGIT_NONE = -0x1p42f;
constexpr double NEG_BIG = -1e4;  // a power of two of this exponent is 0 in every format

// ------------------------------------------------------- logits by type --

template <typename T>
struct LogitTraits;  // a 16-byte chunk of logits: unpacked in pairs, packed, its maximum
template <>
struct LogitTraits<__nv_bfloat16> {
  static constexpr int EPC = 8;  // elements of a chunk
  __device__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
  __device__ static uint64_t pair(const uint4& v, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i];
    return f32x2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  }
  __device__ static void put(uint4& v, int i, float lo, float hi) { reinterpret_cast<uint32_t*>(&v)[i] = pack_bf16x2(lo, hi); }
  // CLAMPS: the type can hold LOGIT_LOWEST; clamp raises a chunk to it (a NaN stays)
  static constexpr bool CLAMPS = true;
  __device__ static void clamp(uint4& v) {
    const __nv_bfloat162 lowest = __float2bfloat162_rn(LOGIT_LOWEST);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162& h = reinterpret_cast<__nv_bfloat162*>(&v)[i];
      h = __hmax2_nan(h, lowest);
    }
  }
  // running maximum of pairs; a NaN is passed over here and met again in the sum
  using Max = __nv_bfloat162;
  __device__ static Max max_init() { return __float2bfloat162_rn(-INFINITY); }
  __device__ static void max_add(Max& m, const uint4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2(m, reinterpret_cast<const __nv_bfloat162*>(&v)[i]);
  }
  __device__ static float max_get(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct LogitTraits<__half> {
  static constexpr int EPC = 8;
  __device__ static float load(const __half* p) { return __half2float(*p); }
  __device__ static __half round(float v) { return __float2half_rn(v); }
  __device__ static uint64_t pair(const uint4& v, int i) {
    const float2 f = __half22float2(reinterpret_cast<const __half2*>(&v)[i]);
    return f32x2(f.x, f.y);
  }
  static constexpr bool CLAMPS = false;  // 65504 is too near for that at a high temperature: raised in fp32
  __device__ static void clamp(uint4&) {}
  __device__ static void put(uint4& v, int i, float lo, float hi) { reinterpret_cast<__half2*>(&v)[i] = __floats2half2_rn(lo, hi); }
  using Max = __half2;
  __device__ static Max max_init() { return __float2half2_rn(-INFINITY); }
  __device__ static void max_add(Max& m, const uint4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2(m, reinterpret_cast<const __half2*>(&v)[i]);
  }
  __device__ static float max_get(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct LogitTraits<float> {
  static constexpr int EPC = 4;
  __device__ static float load(const float* p) { return *p; }
  __device__ static float round(float v) { return v; }
  __device__ static uint64_t pair(const uint4& v, int i) {
    return i == 0 ? f32x2(__uint_as_float(v.x), __uint_as_float(v.y)) : f32x2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static constexpr bool CLAMPS = true;
  __device__ static void clamp(uint4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t& w = reinterpret_cast<uint32_t*>(&v)[i];
      w = __float_as_uint(max_nan(__uint_as_float(w), LOGIT_LOWEST));
    }
  }
  __device__ static void put(uint4& v, int i, float lo, float hi) {
    reinterpret_cast<uint32_t*>(&v)[2 * i] = __float_as_uint(lo);
    reinterpret_cast<uint32_t*>(&v)[2 * i + 1] = __float_as_uint(hi);
  }
  using Max = float;
  __device__ static Max max_init() { return -INFINITY; }
  __device__ static void max_add(Max& m, const uint4& v) {
    m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))));
  }
  __device__ static float max_get(Max m) { return m; }
};

enum : int { DT_BF16 = 0, DT_FP16 = 1, DT_FP32 = 2 };

__device__ __forceinline__ float load_as_f32(const void* p, int dtype, size_t i) {
  if (dtype == DT_FP32) return static_cast<const float*>(p)[i];
  if (dtype == DT_FP16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// ------------------------------------------------------------ setup, sums --

// The first launch of a call: sets its ticket and status word, and counts the
// valid rows of each block's range.  The next launch adds the blocks' counts
// (count_rows), so nothing has to be zeroed ahead.  It costs its launch: in a
// graph a clipped-policy call takes 8.2 us at 4096 rows with it and 4.2 us at 512
// without.  Counting in every CTA of the next launch instead would read the
// targets once per CTA, which a few rows could bear; the ticket would still have to
// be zero before that launch.  Not built, nor a launch that overlaps the next.
constexpr int BEGIN_THREADS = 512;
constexpr int BEGIN_ROWS = 16 * BEGIN_THREADS;  // per block; more when that would take over BEGIN_BLOCKS blocks
constexpr int BEGIN_BLOCKS = 256;
__global__ void __launch_bounds__(BEGIN_THREADS)
    flce_begin_kernel(const int32_t* y, int N, int ignore_index, int per, unsigned int* ticket, int* counts, int* status) {
  const int lo = blockIdx.x * per, hi = min(N, lo + per);
  int c = 0;
#pragma unroll 4
  for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += BEGIN_THREADS) c += y[i] != ignore_index ? 1 : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_down_sync(0xffffffffu, c, o);
  __shared__ int w[BEGIN_THREADS / 32];
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
    for (int k = 0; k < BEGIN_THREADS / 32; ++k) t += w[k];
    counts[blockIdx.x] = t;
    if (blockIdx.x == 0) {
      *ticket = 0u;
      *status = 0;
    }
  }
}

// The valid rows of the call, from the first launch's counts (every warp for itself).
struct RowCounts {
  const int* counts;
  int blocks;
};
__device__ __forceinline__ int count_rows(const RowCounts& r) {
  int n = 0;
  for (int i = threadIdx.x & 31; i < r.blocks; i += 32) n += r.counts[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// The last block to finish adds the blocks' sums: a fixed tree over a fixed
// assignment, in fp64.
template <int THREADS>
__device__ __forceinline__ double ordered_sum(const double* v, int n, double* scratch) {
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += THREADS) s += __ldcg(v + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_down_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = s;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int k = 0; k < THREADS / 32; ++k) t += scratch[k];
  return t;  // thread 0's
}

// ------------------------------------------------------ teacher's softmax --

// A warp's view of one row's teacher distribution over the K entries of s_u
// (-inf: no entry): log q_k = u_k / T - shift.  `any` is false when the row has
// no entry.  Differences are taken in fp64 before they are rounded for expf,
// so large teacher logits cost no precision; the sum is fp32.
struct TeacherShift {
  double shift;
  bool any;
};
__device__ __forceinline__ TeacherShift teacher_shift(const float* s_u, int K, int lane, double inv_T,
                                                      const float* teacher_lse, size_t row) {
  float um = -INFINITY;
  bool any = false;
  for (int k = lane; k < K; k += 32) {
    um = fmaxf(um, s_u[k]);
    any = any || !(s_u[k] == -INFINITY);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, o));
  TeacherShift t;
  t.any = __any_sync(0xffffffffu, any);
  t.shift = static_cast<double>(um) * inv_T;
  if (teacher_lse) {
    t.shift = static_cast<double>(teacher_lse[row]);
  } else if (t.any) {
    float S = 0.f;
    for (int k = lane; k < K; k += 32) S += expf(static_cast<float>(static_cast<double>(s_u[k]) * inv_T - t.shift));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    t.shift += log(static_cast<double>(S));
  }
  return t;
}

// ------------------------------------------------------ clipped policy rows --

struct PolicyRowsArgs {
  PolicyArgs pol;
  const float* row_loss;  // [N] l_i = -lp_i
  const int32_t* y;
  int N, ignore_index, reduction;
  const float* row_scale;
  RowCounts valid;      // several blocks: the first launch's counts
  unsigned int* ticket;
  double* blk_sum;      // [gridDim.x]
  double* loss;
  int* status;
  float* out_rows;      // [N] policy loss per row
  float* out_kl;        // [N]
  float* out_weight;    // [N] s_i dL_i/dl_i
};

// Elementwise over the rows, with two fp64 exponentials (the ratio, the KL term) in
// each.  A thread takes four neighbouring rows, so that the loads of each of its up
// to six streams are one 16-byte access where the stream allows it.  Measured, both
// launches in a graph: 1,048,576 rows (34 MB) 16.7 us, 4,194,304 rows 43 to 47 us,
// 3.1 to 2.8 TB/s.
// No unit is full (52% of the issue slots, the fp64 pipe 23%): what bounds it is
// latency, of the loads and of the exponentials' chains, which run one after the
// other because each of a thread's rows lies behind a branch.  Fewer registers for
// 5, 6 or 8 CTAs on an SM: 44.0, 45.3, 46.5 us against 43.0.
constexpr int POLICY_THREADS = 256;
constexpr int POLICY_ROWS = 4;

__device__ __forceinline__ void load_rows4(const float* p, int i, int n, float (&v)[POLICY_ROWS]) {
  if (!p) return;
  if (n == POLICY_ROWS && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const float4 t = *reinterpret_cast<const float4*>(p + i);
    v[0] = t.x;
    v[1] = t.y;
    v[2] = t.z;
    v[3] = t.w;
  } else {
    for (int k = 0; k < n; ++k) v[k] = p[i + k];
  }
}
__device__ __forceinline__ void store_rows4(float* p, int i, int n, const float (&v)[POLICY_ROWS]) {
  if (n == POLICY_ROWS && (reinterpret_cast<uintptr_t>(p) & 15) == 0)
    *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
  else
    for (int k = 0; k < n; ++k) p[i + k] = v[k];
}

// ONE: a single block, which counts the valid rows itself; its only launch.
// Otherwise the last block to finish adds the blocks' sums in order.
template <bool ONE>
__global__ void __launch_bounds__(POLICY_THREADS) flce_policy_rows_kernel(const PolicyRowsArgs a) {
  __shared__ double w[POLICY_THREADS / 32];
  __shared__ bool is_last;
  int n_valid;
  if constexpr (ONE) {
    int c = 0;
    for (int i0 = 0; i0 < a.N; i0 += POLICY_THREADS) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      c += __syncthreads_count(i < a.N && a.y[i] != a.ignore_index);
    }
    n_valid = c;
  } else {
    n_valid = count_rows(a.valid);
  }
  const double inv_n = n_valid > 0 ? 1.0 / static_cast<double>(n_valid) : 0.0;
  double acc = 0.0;
  for (int i = (blockIdx.x * POLICY_THREADS + threadIdx.x) * POLICY_ROWS; i < a.N;
       i += gridDim.x * (POLICY_THREADS * POLICY_ROWS)) {
    const int n = min(POLICY_ROWS, a.N - i);
    float l[POLICY_ROWS], yf[POLICY_ROWS], scale[POLICY_ROWS];
    PolicyIn in[POLICY_ROWS];
    float old[POLICY_ROWS] = {}, adv[POLICY_ROWS] = {}, ref[POLICY_ROWS] = {};
    load_rows4(reinterpret_cast<const float*>(a.y), i, n, yf);
    load_rows4(a.row_loss, i, n, l);
    load_rows4(a.pol.old_logp, i, n, old);
    load_rows4(a.pol.adv, i, n, adv);
    load_rows4(a.pol.ref_logp, i, n, ref);
    load_rows4(a.row_scale, i, n, scale);
    float rows[POLICY_ROWS] = {}, kl[POLICY_ROWS] = {}, weight[POLICY_ROWS] = {};
#pragma unroll
    for (int k = 0; k < POLICY_ROWS; ++k) {
      if (k < n && __float_as_int(yf[k]) != a.ignore_index) {
        in[k] = {old[k], adv[k], ref[k]};
        const PolicyRow p = policy_row(a.pol, in[k], -static_cast<double>(l[k]));
        const double s = a.reduction == RED_MEAN ? inv_n
                         : a.reduction == RED_NONE && a.row_scale ? static_cast<double>(scale[k]) : 1.0;
        rows[k] = static_cast<float>(p.loss);
        kl[k] = static_cast<float>(p.kl);
        weight[k] = static_cast<float>(-p.dlogp * s);
        acc += a.reduction == RED_MEAN ? p.loss : p.loss * s;
      }
    }
    store_rows4(a.out_rows, i, n, rows);
    store_rows4(a.out_kl, i, n, kl);
    store_rows4(a.out_weight, i, n, weight);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_down_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int k = 0; k < POLICY_THREADS / 32; ++k) t += w[k];
    if constexpr (ONE) {
      *a.loss = a.reduction == RED_MEAN ? t * inv_n : t;
      *a.status = 0;
    } else {
      a.blk_sum[blockIdx.x] = t;
      __threadfence();
      is_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
  }
  if constexpr (!ONE) {
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    const double t = ordered_sum<POLICY_THREADS>(a.blk_sum, gridDim.x, w);
    if (threadIdx.x == 0) *a.loss = a.reduction == RED_MEAN ? t * inv_n : t;
  }
}

// --------------------------------------------------- losses on the logits --

enum : int {
  LOSS_POLICY = 0,    // clipped policy loss
  LOSS_DISTILL = 1,   // distillation, one softmax (ce == 0 or T == 1)
  LOSS_DISTILL2 = 2,  // distillation at T != 1 mixed with hard labels: a second softmax at T = 1
  LOSS_POLICY_ENT = 3 // clipped policy loss with an entropy term in its gradient
};
__host__ __device__ constexpr bool is_policy(int loss) { return loss == LOSS_POLICY || loss == LOSS_POLICY_ENT; }

struct LogitArgs {
  const void* z;          // [N][V], row stride ld elements
  void* g;                // gradient, row stride ldg, or null; may be z itself
  long long ld, ldg;
  const int32_t* y;
  int N, V, ignore_index, reduction;
  const float* row_scale;
  RowCounts valid;
  unsigned int* ticket;
  double* sums;           // [clusters], at most N
  float* loss;
  int* status;
  double inv_T;
  float zs;               // log2(e) / T
  double zs_off;          // its rounding: zs / (log2(e) / T) - 1
  unsigned long long timeout_ns;
  // policy
  PolicyArgs pol;
  double ent_coef;
  float* out_logp;        // [N]
  float* out_entropy;     // [N]
  float* out_kl;          // [N]
  // distillation
  const int32_t* ids;     // [N][K], negative: no entry
  const void* u;          // [N][K] teacher logits
  int u_dtype, K;
  const float* teacher_lse;  // [N] or null
  double kd, ce;
  float* out_rows;        // [N] or null
};

// A row's running statistics under a reference m, which is the maximum to
// within RAISE in the exponent: sum of e = 2^((z - m) zs), and for the policy loss
// the first moment sum e (z - m), for DISTILL2 the sum of 2^((z - m) log2 e).  The
// moment takes z - m, which is finite, not the exponent, which a large m or a
// small temperature takes beyond fp32: e is 0 there, and 0 times infinity is NaN.
struct RowStat {
  float m, l, t;
};
// How far a logit may lie above the reference, in the exponent, before the
// reference moves: rarely, because each move rounds the sums.
constexpr float RAISE = 60.f;

// What the gradient needs of a row.
struct RowCoef {
  float m;       // the row's reference
  float a, b;    // dense part: e a + e (z - m) b, or e a + e1 b with two softmaxes
  float c, zy;   // policy: subtracted at the target, and the logit there
};

template <bool B>
struct Flag {  // a compile-time truth value to pass to a lambda
  static constexpr bool value = B;
};

constexpr int LOGIT_THREADS = 256;  // of a CTA; fewer for short rows (see the launch)
constexpr int LOGIT_MAX_CLUSTER = 8;
constexpr int TILE_CHUNKS = 256;  // 16-byte chunks of a warp's tile (4 KB), eight per lane
constexpr int TILE_STAGES = 3;    // tiles per warp in shared memory
constexpr int WARP_RING_BYTES = TILE_STAGES * TILE_CHUNKS * 16;

// Where row `row` lies, and which of it is CTA `rank`'s part.  Bulk copies move
// 16-byte chunks on 16-byte boundaries: the up to 2 * (EPC - 1) elements in
// front of the first and behind the last boundary ("edges") are held one per
// thread by the cluster's first CTA.
template <typename T, int WARPS>
struct RowPart {
  static constexpr int EPC = LogitTraits<T>::EPC;
  const T* z;
  T* g;
  int head, edges;  // elements before the first boundary, elements outside chunks
  int n;            // this CTA's chunks
  int col0;         // column of the first one
  int tiles;        // tiles of the calling warp: those j < ceil(n / TILE_CHUNKS) with j % WARPS == warp
  bool vec_out;     // the gradient row shares the logits' alignment
  __device__ RowPart(const LogitArgs& a, int row, int rank, int cs, int warp) {
    z = static_cast<const T*>(a.z) + static_cast<long long>(row) * a.ld;
    g = a.g ? static_cast<T*>(a.g) + static_cast<long long>(row) * a.ldg : nullptr;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    head = min(a.V, mis ? EPC - mis : 0);
    const int chunks = (a.V - head) / EPC;
    edges = a.V - chunks * EPC;
    const int per = (chunks + cs - 1) / cs;
    const int c0 = min(chunks, rank * per);
    n = min(per, chunks - c0);
    col0 = head + c0 * EPC;
    const int all = (n + TILE_CHUNKS - 1) / TILE_CHUNKS;
    tiles = all > warp ? (all - warp + WARPS - 1) / WARPS : 0;
    vec_out = g && ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
  }
  __device__ bool has(int id) const { return id >= col0 && id < col0 + n * EPC; }
  // first chunk and chunk count of the calling warp's k-th tile
  __device__ int tile_at(int k, int warp) const { return (k * WARPS + warp) * TILE_CHUNKS; }
  __device__ int tile_size(int at) const { return min(TILE_CHUNKS, n - at); }
  __device__ int edge_col(const LogitArgs& a, int rank, int tid) const {
    return rank == 0 && tid < edges ? (tid < head ? tid : a.V - edges + tid) : -1;
  }
};

__device__ __forceinline__ bool row_counts(const LogitArgs& a, int y) {
  return y != a.ignore_index && y >= 0 && y < a.V;
}

// Persistent CTAs, each with a row (or, in clusters, its part of a row) at a
// time.  A row is walked twice: forwards for its maximum and sums, backwards
// for the gradient.  The second read finds most of the row in L2, where the first
// one's policy keeps it: the rows under way on all SMs are some 80 MB at most, as
// the host gives rows of over 256 KB to clusters; from 2 MB on, the largest
// cluster's parts grow again.  Memory is thus read and written about once,
// and what a row costs beside its elements (two exchanges, the fp64 of its
// scalars) is paid once per 100,000 elements or so.
//
// Every warp moves its own tiles of 4 KB through a ring of its own in shared
// memory: one lane issues the bulk copies, the next tiles (of the second walk,
// and of the next row) are under way while this one is worked on, and a tile
// waits for no other warp.  Gradient tiles are written in place of the logits
// and leave by bulk copies too.
//
// Statistics: every warp folds its elements under a reference near its maximum
// and writes one record into every CTA of the cluster; behind one barrier warp 0
// of each CTA merges the records in a fixed order, so all CTAs find the same
// totals, and turns them into the row's outputs (first CTA) and the gradient's
// coefficients.
//
// Two exponentials per element, one per walk: probabilities kept from the first
// walk would be a second array to write and read.  Measured in a graph, with the
// first launch: policy loss, bf16 4096 x 128256 427 us (2.10 GB, 4.9 TB/s), with an
// entropy term 447 us, with a quarter of the rows ignored (not read) 408 us;
// distillation, bf16 2048 x 256000, 64 entries 470 us and 432 us; fp16 1023 x
// 50021, a fifth ignored, 60 us.  On 1184 x 128256 alone, with an entropy term, 133
// us: 4.6 TB/s from and to DRAM, 58% of the issue slots, 56% of the exponential
// unit.  No unit is full; with 16 warps on an SM (128 registers each, for eight
// chunks of a tile in flight) what remains is latency.  Three CTAs on an SM (80
// registers), tiles of 2 KB, a gradient stored from registers and refills in
// another order measured the same or slower.
template <typename T, int LOSS, int THREADS>
__global__ void __launch_bounds__(THREADS, 2 * LOGIT_THREADS / THREADS) flce_logit_loss_kernel(const LogitArgs a) {
  using L = LogitTraits<T>;
  constexpr int EPC = L::EPC;
  constexpr int LANE_CHUNKS = TILE_CHUNKS / 32;
  constexpr int WARPS = THREADS / 32;
  extern __shared__ __align__(128) uint8_t dyn_tiles[];
  const int K1 = is_policy(LOSS) ? 0 : a.K + 1;
  // the warps' rings, then twice (for two rows) the sparse entries: vocabulary
  // ids (-1: none), coefficients subtracted there, the student's logits, the teacher's
  int* entries = reinterpret_cast<int*>(dyn_tiles + WARPS * WARP_RING_BYTES);
  __shared__ float4 rec[2][LOGIT_MAX_CLUSTER * WARPS];
  __shared__ RowCoef coefs[2];
  __shared__ double dsum[WARPS];
  __shared__ uint64_t bars[WARPS * TILE_STAGES];
  __shared__ int abort_flag;
  __shared__ bool is_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  const int clusters = gridDim.x / cs;
  const uint64_t keep = l2_evict_last(), last = l2_evict_first();
  uint4* ring = reinterpret_cast<uint4*>(dyn_tiles) + warp * (TILE_STAGES * TILE_CHUNKS);
  const uint32_t bar0 = smem_u32(bars + warp * TILE_STAGES);
  if (lane < TILE_STAGES) mbar_init(bar0 + 8u * lane, 1);
  if (tid == 0) abort_flag = 0;
  fence_mbar_init();
  __syncthreads();
  if (cs > 1) cluster_sync_all();  // the others run before a record is written into their shared memory
  const int n_valid = count_rows(a.valid);
  const double inv_n = n_valid > 0 ? 1.0 / static_cast<double>(n_valid) : 0.0;
  const int walks = a.g ? 2 : 1;
  // ---- the warp's ring: tiles are issued and used in the same order
  const int first = blockIdx.x / cs;
  // Targets are read a row ahead of the question whether the row counts.
  auto target = [&](int r) { return r < a.N ? a.y[r] : a.ignore_index; };
  int ahead = first;  // row of the next tile to issue; `then` follows it
  while (ahead < a.N && !row_counts(a, a.y[ahead])) ahead += clusters;
  int then = ahead + clusters, then_y = target(then);
  RowPart<T, WARPS> ap(a, min(ahead, a.N - 1), rank, cs, warp);
  int ahead_k = 0;                   // its number in the row's 2 * tiles (or tiles) ones
  int in_stage = 0;
  auto issue = [&]() {
    while (ahead < a.N && ahead_k == walks * ap.tiles) {
      while (then < a.N && !row_counts(a, then_y)) {
        then += clusters;
        then_y = target(then);
      }
      ahead = then;
      then += clusters;
      then_y = target(then);
      ahead_k = 0;
      if (ahead < a.N) ap = RowPart<T, WARPS>(a, ahead, rank, cs, warp);
    }
    if (ahead >= a.N || *const_cast<volatile int*>(&abort_flag)) return;
    const bool again = ahead_k >= ap.tiles;
    const int at = ap.tile_at(again ? 2 * ap.tiles - 1 - ahead_k : ahead_k, warp);
    if (lane == 0) {
      const uint32_t bytes = static_cast<uint32_t>(ap.tile_size(at)) * 16u;
      mbar_arrive_expect_tx(bar0 + 8u * in_stage, bytes);
      bulk_load(smem_u32(ring + in_stage * TILE_CHUNKS), reinterpret_cast<const uint4*>(ap.z + ap.col0) + at, bytes,
                bar0 + 8u * in_stage, again || walks == 1 ? last : keep);
    }
    ++ahead_k;
    if (++in_stage == TILE_STAGES) in_stage = 0;
  };
  int stage = 0;          // of the tile in use
  uint32_t phase = 0;
  bool freed_late = false;  // the last tile's stage is free once its gradient has been read out
  auto arrived = [&]() {
    if (freed_late) {
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      issue();
      freed_late = false;
    }
    if (!mbar_wait(bar0 + 8u * stage, phase, &abort_flag, a.timeout_ns)) {
      *const_cast<volatile int*>(&abort_flag) = 1;
      raise_status(a.status, ST_TIMEOUT);
    }
    __syncwarp();
  };
  auto advance = [&]() {
    if (++stage == TILE_STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  };
  for (int k = 0; k < TILE_STAGES; ++k) issue();

  auto lifted = [&](float x) { return is_policy(LOSS) ? max_nan(x, LOGIT_LOWEST) : x; };
  // a pair of logits from a chunk, raised where the packed form could not be
  auto raised = [&](uint64_t x) {
    if constexpr (!is_policy(LOSS) || L::CLAMPS) return x;
    float lo, hi;
    f32x2_split(x, lo, hi);
    return f32x2(lifted(lo), lifted(hi));
  };
  const float none = is_policy(LOSS) ? LOGIT_NONE : -INFINITY;
  const uint64_t zs2 = f32x2(a.zs, a.zs), one2 = f32x2(LOG2E, LOG2E);
  int parity = 0;
  double sum = 0.0;  // thread 0: the losses of this CTA's rows, in their order
  int next_y = target(first);
  for (int row = first; row < a.N; row += clusters) {
    const int y = next_y;
    next_y = target(row + clusters);
    const RowPart<T, WARPS> p(a, row, rank, cs, warp);
    const int edge_col = p.edge_col(a, rank, tid);
    if (!row_counts(a, y)) {
      if (rank == 0 && tid == 0) {
        if (y != a.ignore_index) raise_status(a.status, ST_TARGET_OUT_OF_RANGE);
        if constexpr (is_policy(LOSS)) {
          a.out_logp[row] = a.out_entropy[row] = a.out_kl[row] = 0.f;
        } else if (a.out_rows) {
          a.out_rows[row] = 0.f;
        }
      }
      if (p.g) {
        if ((reinterpret_cast<uintptr_t>(p.g + p.col0) & 15) == 0) {
          uint4* gv = reinterpret_cast<uint4*>(p.g + p.col0);
          for (int c = tid; c < p.n; c += THREADS) st_l2hint_v4(gv + c, make_uint4(0u, 0u, 0u, 0u), last);
        } else {
          for (int e = tid; e < p.n * EPC; e += THREADS) p.g[p.col0 + e] = L::round(0.f);
        }
        if (edge_col >= 0) p.g[edge_col] = L::round(0.f);
      }
      continue;
    }

    // ---- what the row has besides its tiles, read ahead of its use
    float edge = edge_col >= 0 ? L::load(p.z + edge_col) : -INFINITY;
    PolicyIn pin{};
    T zy_raw{};
    double scale = 1.0;
    if (tid < 32) {
      if (is_policy(LOSS)) pin = policy_load(a.pol, row);
      zy_raw = p.z[y];
      scale = a.reduction == RED_MEAN ? inv_n
              : a.reduction == RED_NONE && a.row_scale ? static_cast<double>(a.row_scale[row]) : 1.0;
    }
    int* s_id = entries + parity * 4 * K1;
    float* s_c = reinterpret_cast<float*>(s_id + K1);
    float *s_z = s_c + K1, *s_u = s_z + K1;
    // The teacher's entries, then the target.  A thread's first one is read in
    // three steps, each waited for only at the next: id and teacher logit here,
    // the student's logit behind the first tile, its use behind the last.
    auto teacher_id = [&](int k) { return k < a.K ? a.ids[static_cast<size_t>(row) * a.K + k] : y; };
    auto teacher_u = [&](int k) {
      return k < a.K ? load_as_f32(a.u, a.u_dtype, static_cast<size_t>(row) * a.K + k) : -INFINITY;
    };
    auto wanted = [&](int id) { return id >= 0 && (rank == 0 || p.has(id)); };
    auto checked = [&](int id) {
      if (id >= a.V) raise_status(a.status, ST_TARGET_OUT_OF_RANGE);
      return id < 0 || id >= a.V ? -1 : id;
    };
    int my_id = -1;
    float my_u = -INFINITY;
    T my_z{};
    if (!is_policy(LOSS) && tid < K1) {
      my_id = teacher_id(tid);
      my_u = teacher_u(tid);
    }
    auto read_entries = [&]() {
      if constexpr (!is_policy(LOSS)) {
        for (int k = tid; k < K1; k += THREADS) {
          const int id = checked(k == tid ? my_id : teacher_id(k));
          const float u = k == tid ? my_u : teacher_u(k);
          s_id[k] = id;
          s_u[k] = id < 0 ? -INFINITY : u;
          if (k == tid) {
            my_id = id;
            if (wanted(id)) my_z = p.z[id];
          } else {
            s_z[k] = wanted(id) ? L::load(p.z + id) : 0.f;
          }
        }
      }
    };

    // ---- first walk: the sums, each warp under a reference of its own
    float top = edge;  // this lane's largest logit as it stands
    if (is_policy(LOSS)) edge = edge_col >= 0 ? lifted(edge) : none;
    float ref = is_policy(LOSS) ? LOGIT_LOWEST : -FLT_MAX;  // the warp's reference
    uint64_t l2 = 0ull, t2 = 0ull;                          // this lane's sums, in two parts each
    // in the exponents of the sharper softmax, where there are two
    const float steep = LOSS == LOSS_DISTILL2 ? fmaxf(a.zs, LOG2E) : a.zs;
    auto raise = [&](float lane_top) {  // the reference, where some lane's logits need it
      if (!__any_sync(0xffffffffu, (lane_top - ref) * steep > RAISE)) return;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) lane_top = fmaxf(lane_top, __shfl_xor_sync(0xffffffffu, lane_top, s));
      const float d = ref - lane_top, f = ex2_approx(d * a.zs);
      const uint64_t f2 = f32x2(f, f);
      if constexpr (is_policy(LOSS)) {
        const float df = f == 0.f ? 0.f : d;  // l2 d might overflow, and what it is added to ends as 0
        t2 = mul2(f2, fma2(l2, f32x2(df, df), t2));
      }
      if constexpr (LOSS == LOSS_DISTILL2) {
        const float f1 = ex2_approx((ref - lane_top) * LOG2E);
        t2 = mul2(t2, f32x2(f1, f1));
      }
      l2 = mul2(l2, f2);
      ref = lane_top;
    };
    auto fold = [&](uint64_t x) {
      const uint64_t d0 = add2(x, f32x2(-ref, -ref));
      float lo, hi;
      f32x2_split(mul2(d0, zs2), lo, hi);
      const uint64_t e = f32x2(ex2_approx(lo), ex2_approx(hi));
      l2 = add2(l2, e);
      if constexpr (is_policy(LOSS)) t2 = fma2(e, d0, t2);
      if constexpr (LOSS == LOSS_DISTILL2) {
        f32x2_split(mul2(d0, one2), lo, hi);
        t2 = add2(t2, f32x2(ex2_approx(lo), ex2_approx(hi)));
      }
    };
    auto fold_tile = [&](auto full, int size) {
      auto has = [&](int u) { return decltype(full)::value || u * 32 + lane < size; };
      uint4 v[LANE_CHUNKS];
      const uint4* tile = ring + stage * TILE_CHUNKS + lane;
#pragma unroll
      for (int u = 0; u < LANE_CHUNKS; ++u)
        if (has(u)) v[u] = tile[u * 32];
      __syncwarp();
      issue();  // the tile is in registers
      advance();
      typename L::Max vmax = L::max_init();
#pragma unroll
      for (int u = 0; u < LANE_CHUNKS; ++u)
        if (has(u)) L::max_add(vmax, v[u]);
      const float tile_top = L::max_get(vmax);
      top = fmaxf(top, tile_top);
      raise(tile_top);
#pragma unroll
      for (int u = 0; u < LANE_CHUNKS; ++u) {
        if (has(u)) {
          if constexpr (is_policy(LOSS)) L::clamp(v[u]);
#pragma unroll
          for (int i = 0; i < EPC / 2; ++i) fold(raised(L::pair(v[u], i)));
        }
      }
    };
    for (int k = 0; k < p.tiles; ++k) {
      const int size = p.tile_size(p.tile_at(k, warp));
      arrived();
      if (size == TILE_CHUNKS)
        fold_tile(Flag<true>{}, size);
      else
        fold_tile(Flag<false>{}, size);
      if (k == 0) read_entries();
    }
    if (p.tiles == 0) read_entries();
    if (!is_policy(LOSS) && tid < K1) s_z[tid] = wanted(my_id) ? L::load(&my_z) : 0.f;
    raise(edge);
    fold(f32x2(edge, none));
    RowStat w{ref, 0.f, 0.f};
    {
      float lo, hi;
      f32x2_split(l2, lo, hi);
      w.l = lo + hi;
      f32x2_split(t2, lo, hi);
      w.t = lo + hi;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) {
        w.l += __shfl_xor_sync(0xffffffffu, w.l, s);
        w.t += __shfl_xor_sync(0xffffffffu, w.t, s);
      }
      top = __any_sync(0xffffffffu, top > -INFINITY) ? 1.f : 0.f;  // some logit is above -infinity
    }
    if (cs == 1) {
      if (lane == 0) rec[parity][warp] = make_float4(w.m, w.l, w.t, top);
      __syncthreads();
    } else {
      if (lane < cs)
        st_cluster_f4(mapa_shared(smem_u32(&rec[parity][rank * WARPS + warp]), lane),
                      make_float4(w.m, w.l, w.t, top));
      cluster_sync_all();
    }

    // ---- the row's totals and scalars
    if (warp == 0) {
      // The records under the largest reference, in fp64: a rounded factor
      // would put the same error on a whole warp's sum.
      const int records = cs * WARPS;
      float ref_max = -FLT_MAX;
      for (int r = lane; r < records; r += 32) ref_max = fmaxf(ref_max, rec[parity][r].x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) ref_max = fmaxf(ref_max, __shfl_xor_sync(0xffffffffu, ref_max, s));
      double sum_l = 0.0, sum_t = 0.0;
      top = 0.f;
      for (int r = lane; r < records; r += 32) {
        const float4 v = rec[parity][r];
        const double gap = static_cast<double>(v.x) - static_cast<double>(ref_max);
        const double f = exp2(fmax(gap * static_cast<double>(a.zs), NEG_BIG));
        sum_l += f * static_cast<double>(v.y);
        if constexpr (is_policy(LOSS)) sum_t += f * (static_cast<double>(v.z) + gap * static_cast<double>(v.y));
        if constexpr (LOSS == LOSS_DISTILL2)
          sum_t += exp2(fmax(gap * static_cast<double>(LOG2E), NEG_BIG)) * static_cast<double>(v.z);
        top = fmaxf(top, v.w);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) {
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, s);
        sum_t += __shfl_xor_sync(0xffffffffu, sum_t, s);
      }
      if (is_policy(LOSS) && !__any_sync(0xffffffffu, top > 0.f)) sum_l = 0.0;  // every logit is -infinity: NaN
      // Log-probabilities as (z - m)/T - ln L: the difference first, so that a
      // row whose every logit is the type's lowest value still has one.
      const double m = static_cast<double>(ref_max);
      const double inv_l = 1.0 / sum_l;
      double lnL = log(sum_l);
      const double mean = sum_t * inv_l;  // policy: E[z - m]
      // zs is off by zs_off of itself: d ln L / d ln zs = E[z - m] / T.  Distillation has
      // no such mean; it keeps an error of 2^-25 of it, some 1e-6 where the row's
      // logits lie tens of T below their maximum.
      if (is_policy(LOSS)) lnL -= a.zs_off * a.inv_T * mean;
      const float zy = L::load(&zy_raw);
      double total = 0.0;
      RowCoef c{ref_max, 0.f, 0.f, 0.f, 0.f};
      if constexpr (is_policy(LOSS)) {
        const double lp = (static_cast<double>(zy == -INFINITY ? zy : lifted(zy)) - m) * a.inv_T - lnL;
        const double H = lnL - mean * a.inv_T;
        const PolicyRow r = policy_row(a.pol, pin, lp);
        total = r.loss;
        double a0 = -r.dlogp, a1 = 0.0;
        if (a.ent_coef != 0.0) {
          total -= a.ent_coef * H;
          a0 += a.ent_coef * (H - lnL);
          a1 = a.ent_coef * a.inv_T;
        }
        const double f = scale * a.inv_T;
        c.a = static_cast<float>(a0 * f * inv_l);
        c.b = static_cast<float>(a1 * f * inv_l);
        c.c = static_cast<float>(-r.dlogp * f);
        c.zy = lifted(zy);
        if (rank == 0 && lane == 0) {
          a.out_logp[row] = static_cast<float>(lp);
          a.out_entropy[row] = static_cast<float>(H);
          a.out_kl[row] = static_cast<float>(r.kl);
        }
      } else {
        const TeacherShift ts = teacher_shift(s_u, a.K, lane, a.inv_T, a.teacher_lse, row);
        double Q = 0.0, kl = 0.0;
        for (int k = lane; k < a.K; k += 32) {
          const double lq = static_cast<double>(s_u[k]) * a.inv_T - ts.shift;
          const float q = ts.any ? expf(static_cast<float>(lq)) : 0.f;
          s_c[k] = static_cast<float>(static_cast<double>(q) * a.kd * a.inv_T * scale);
          Q += q;
          if (rank == 0 && !(q == 0.f))
            kl += static_cast<double>(q) * (lq - ((static_cast<double>(s_z[k]) - m) * a.inv_T - lnL));
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
          Q += __shfl_xor_sync(0xffffffffu, Q, s);
          kl += __shfl_xor_sync(0xffffffffu, kl, s);
        }
        if (a.kd != 0.0) total = a.kd * kl;
        double da = a.kd * Q * a.inv_T, db = 0.0;
        if (a.ce != 0.0) {
          const double ln1 = LOSS == LOSS_DISTILL2 ? log(sum_t) : lnL;
          total += a.ce * (m - static_cast<double>(zy) + ln1);
          if constexpr (LOSS == LOSS_DISTILL2)
            db = a.ce / sum_t;
          else
            da += a.ce;
        }
        c.a = static_cast<float>(da * scale * inv_l);
        c.b = static_cast<float>(db * scale);
        if (lane == 0) {
          s_c[a.K] = static_cast<float>(a.ce * scale);
          if (rank == 0 && a.out_rows) a.out_rows[row] = static_cast<float>(total);
        }
      }
      if (lane == 0) {
        coefs[parity] = c;
        sum += a.reduction == RED_MEAN ? total : total * scale;
      }
    }

    // ---- second walk, backwards: the gradient
    if (a.g) {
      __syncthreads();
      const RowCoef c = coefs[parity];
      const uint64_t neg_m2 = f32x2(-c.m, -c.m), a2 = f32x2(c.a, c.a), b2 = f32x2(c.b, c.b);
      auto dense2 = [&](uint64_t x) {
        const uint64_t d0 = add2(LOSS == LOSS_POLICY_ENT ? raised(x) : x, neg_m2);
        float lo, hi;
        f32x2_split(mul2(d0, zs2), lo, hi);
        const uint64_t e = f32x2(ex2_approx(lo), ex2_approx(hi));
        // b (z - m) may overflow where e is 0, with a logit near the largest fp32 value:
        // e (z - m) comes first.  4096 x 128256 takes 444 -> 452 us for it, and 1% longer
        // than before with a choice between the two per row.  fp16 has no such logits.
        if constexpr (LOSS == LOSS_POLICY_ENT && L::CLAMPS) return fma2(mul2(e, d0), b2, mul2(e, a2));
        if constexpr (LOSS == LOSS_POLICY_ENT) return mul2(e, fma2(b2, d0, a2));
        if constexpr (LOSS == LOSS_DISTILL2) {
          f32x2_split(mul2(d0, one2), lo, hi);
          return fma2(f32x2(ex2_approx(lo), ex2_approx(hi)), b2, mul2(e, a2));
        }
        return mul2(e, a2);
      };
      auto dense = [&](float x) {
        float lo, hi;
        f32x2_split(dense2(f32x2(x, x)), lo, hi);
        return lo;
      };
      // what is subtracted at column id: equal ids add up
      auto sparse = [&](int id) {
        if (is_policy(LOSS)) return id == y ? c.c : 0.f;
        float sum = 0.f;
#pragma unroll 4
        for (int k = 0; k < K1; ++k) sum += s_id[k] == id ? s_c[k] : 0.f;
        return sum;
      };
      if constexpr (!is_policy(LOSS)) {  // every entry's, in place of the teacher's logits (equal ids: the same sum)
        for (int k = tid; k < K1; k += THREADS) s_u[k] = sparse(s_id[k]);
        __syncthreads();
      }
      if (edge_col >= 0) p.g[edge_col] = L::round(dense(edge) - sparse(edge_col));
      for (int k = p.tiles - 1; k >= 0; --k) {
        const int at = p.tile_at(k, warp), size = p.tile_size(at);
        const int col = p.col0 + at * EPC, end = col + size * EPC;
        arrived();
        uint4* tile = ring + stage * TILE_CHUNKS;
        auto write_tile = [&](auto full) {
#pragma unroll
          for (int u = 0; u < LANE_CHUNKS; ++u) {
            if (decltype(full)::value || u * 32 + lane < size) {
              uint4 v = tile[u * 32 + lane], o;
              if constexpr (is_policy(LOSS)) L::clamp(v);
#pragma unroll
              for (int i = 0; i < EPC / 2; ++i) {
                float lo, hi;
                f32x2_split(dense2(L::pair(v, i)), lo, hi);
                L::put(o, i, lo, hi);
              }
              tile[u * 32 + lane] = o;
            }
          }
        };
        if (size == TILE_CHUNKS)
          write_tile(Flag<true>{});
        else
          write_tile(Flag<false>{});
        if constexpr (is_policy(LOSS)) {
          if (y >= col && y < end) {
            __syncwarp();
            if (lane == 0) reinterpret_cast<T*>(tile)[y - col] = L::round(dense(c.zy) - c.c);
          }
        } else {
          __syncwarp();
          for (int i = lane; i < K1; i += 32) {
            const int id = s_id[i];
            if (id >= col && id < end) reinterpret_cast<T*>(tile)[id - col] = L::round(dense(s_z[i]) - s_u[i]);
          }
        }
        if (p.vec_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            bulk_store(p.g + col, smem_u32(tile), static_cast<uint32_t>(size) * 16u, last);
            bulk_commit();
          }
          freed_late = true;
        } else {
          __syncwarp();
          for (int e = lane; e < size * EPC; e += 32) p.g[col + e] = reinterpret_cast<const T*>(tile)[e];
          fence_proxy_async_smem();
          __syncwarp();
          issue();
        }
        advance();
      }
    }
    parity ^= 1;
  }
  if (lane == 0) {
    if (*const_cast<volatile int*>(&abort_flag)) {  // a late copy must not outlive the CTA (again with a limit)
      int no = 0;
      for (int k = 0; k < TILE_STAGES; ++k) mbar_wait(bar0 + 8u * k, phase ^ (k < stage ? 1u : 0u), &no, a.timeout_ns);
    }
    bulk_wait_read<0>();
  }
  __syncwarp();
  if (cs > 1) cluster_sync_all();  // no CTA leaves while another may still write a record into it
  // the loss, by the last cluster to finish
  if (rank != 0) return;
  if (tid == 0) {
    a.sums[first] = sum;
    __threadfence();
    is_last = atomicAdd(a.ticket, 1u) == static_cast<unsigned>(clusters - 1);
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  const double t = ordered_sum<THREADS>(a.sums, clusters, dsum);
  if (tid == 0) *a.loss = static_cast<float>(a.reduction == RED_MEAN ? t * inv_n : t);
}

// ------------------------------------------- distillation through the head --

struct TeacherArgs {
  const int32_t* ids;     // [N][K], the caller's row order
  const void* u;
  int u_dtype, K, N, V, ignore_index;
  const float* teacher_lse;
  double inv_T, kd, ce;
  const int* perm;        // row of the caller behind each row
  const int32_t* y;       // targets in the rows' order
  // outputs, in the rows' order
  int2* list;             // [N][K + 1]
  int* list_count;
  float* list_dense;
  double* list_const;
  double* list_lse;
  double* list_sum;
  int* status;
};

// Each row's entries (the teacher's, and the target when hard labels are mixed
// in) ascending by id, with the coefficients that the G tiles subtract there,
// and the row's constants:
//   L = kd sum q log q + (kd Q + ce) ln L + sum_k c_k (m - z_k),  c_k = kd q_k / T + ce [target],
//   G = s ((kd Q / T + ce) p - c),
// with the student's maximum m and its sum L of e^((z - m) / T) (ce needs T = 1).
// Entries are ranked by counting (id, position) pairs below their own, so the
// order is the same on every call; equal ids stay separate entries, which the
// G tiles subtract one after the other.  One CTA per row: counting is K^2 / 128
// comparisons a thread, in shared memory.  2048 rows of 64 entries take 12 us beside
// the head's 7 ms, 300 rows of 16 entries 6 us.
constexpr int TEACHER_THREADS = 128;
__global__ void __launch_bounds__(TEACHER_THREADS) flce_teacher_lists_kernel(const TeacherArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  const int K1 = a.K + 1;
  int* s_id = reinterpret_cast<int*>(dyn);
  float* s_u = reinterpret_cast<float*>(s_id + K1);
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = blockIdx.x; i < a.N; i += gridDim.x) {
    const int y = a.y[i];
    if (y == a.ignore_index) {
      if (tid == 0) {
        a.list_count[i] = 0;
        a.list_dense[i] = 0.f;
        a.list_const[i] = a.list_lse[i] = a.list_sum[i] = 0.0;
      }
      continue;
    }
    const size_t src = static_cast<size_t>(a.perm[i]);
    const size_t out = static_cast<size_t>(i) * K1;
    for (int k = tid; k < K1; k += TEACHER_THREADS) {
      int id = 0x7fffffff;
      float u = -INFINITY;
      if (k < a.K) {
        const int t = a.ids[src * a.K + k];
        if (t >= a.V) raise_status(a.status, ST_TARGET_OUT_OF_RANGE);
        if (t >= 0 && t < a.V) {
          id = t;
          u = load_as_f32(a.u, a.u_dtype, src * a.K + k);
        }
      } else if (a.ce != 0.0 && y >= 0 && y < a.V) {
        id = y;
      }
      s_id[k] = id;
      s_u[k] = u;
    }
    __syncthreads();
    const TeacherShift ts = teacher_shift(s_u, a.K, lane, a.inv_T, a.teacher_lse, src);
    auto log_q = [&](int k) { return static_cast<double>(s_u[k]) * a.inv_T - ts.shift; };
    auto prob = [&](int k) { return expf(static_cast<float>(log_q(k))); };
    auto coef = [&](int k) {  // c of an entry, as the list holds it
      return static_cast<float>(k == a.K ? a.ce : ts.any ? static_cast<double>(prob(k)) * a.kd * a.inv_T : 0.0);
    };
    double Q = 0.0, qlogq = 0.0, csum = 0.0;
    int count = 0;
    if (tid < 32) {
      for (int k = lane; k < K1; k += 32) {
        if (s_id[k] != 0x7fffffff) {
          ++count;
          csum += static_cast<double>(coef(k));
        }
        if (k < a.K && ts.any) {
          const double lq = log_q(k);
          const float q = prob(k);
          Q += q;
          if (!(q == 0.f)) qlogq += static_cast<double>(q) * lq;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        Q += __shfl_xor_sync(0xffffffffu, Q, o);
        qlogq += __shfl_xor_sync(0xffffffffu, qlogq, o);
        csum += __shfl_xor_sync(0xffffffffu, csum, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
      }
      if (lane == 0) {
        a.list_count[i] = count;
        a.list_dense[i] = static_cast<float>(a.kd * Q * a.inv_T + a.ce);
        a.list_const[i] = a.kd * qlogq;
        a.list_lse[i] = a.kd * Q + a.ce;
        a.list_sum[i] = csum;
      }
    }
    for (int k = tid; k < K1; k += TEACHER_THREADS) {
      const int id = s_id[k];
      if (id == 0x7fffffff) continue;
      int rank = 0;
      for (int j = 0; j < K1; ++j) rank += s_id[j] < id || (s_id[j] == id && j < k) ? 1 : 0;
      a.list[out + rank] = make_int2(id, __float_as_int(coef(k)));
    }
    __syncthreads();
  }
}

}  // namespace flce

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
// the difference stays finite, so that a probability of 0 adds 0.  Registers
// without a logit hold LOGIT_NONE, which has probability 0 beside any logit.
// Powers of two: the same value in bf16.
constexpr float LOGIT_LOWEST = -0x1p100f, LOGIT_NONE = -0x1p102f;
constexpr float NEG_BIG = -1e4f;  // exponents below this are 0 in every format; finite, so that 0 * it is 0

// ------------------------------------------------------- logits by type --

template <typename T>
struct LogitTraits;  // a 16-byte chunk of logits: unpacked in pairs, packed, its maximum
template <>
struct LogitTraits<__nv_bfloat16> {
  static constexpr int EPC = 8;  // elements of a chunk
  static constexpr uint32_t NEG_INF = 0xff80ff80u;
  __device__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
  __device__ static uint64_t pair(const uint4& v, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i];
    return f32x2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  }
  __device__ static void put(uint4& v, int i, float lo, float hi) { reinterpret_cast<uint32_t*>(&v)[i] = pack_bf16x2(lo, hi); }
  // CLAMPS: the type can hold LOGIT_LOWEST.  clamp raises a chunk to it (a NaN
  // stays), none() is a chunk without logits.
  static constexpr bool CLAMPS = true;
  __device__ static void clamp(uint4& v) {
    const __nv_bfloat162 lowest = __float2bfloat162_rn(LOGIT_LOWEST);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162& h = reinterpret_cast<__nv_bfloat162*>(&v)[i];
      h = __hmax2_nan(h, lowest);
    }
  }
  __device__ static uint4 none() {
    const uint32_t w = pack_bf16x2(LOGIT_NONE, LOGIT_NONE);
    return make_uint4(w, w, w, w);
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
  static constexpr uint32_t NEG_INF = 0xfc00fc00u;
  __device__ static float load(const __half* p) { return __half2float(*p); }
  __device__ static __half round(float v) { return __float2half_rn(v); }
  __device__ static uint64_t pair(const uint4& v, int i) {
    const float2 f = __half22float2(reinterpret_cast<const __half2*>(&v)[i]);
    return f32x2(f.x, f.y);
  }
  static constexpr bool CLAMPS = false;  // 65504 is too near for that at a high temperature
  __device__ static void clamp(uint4&) {}
  __device__ static uint4 none() { return make_uint4(NEG_INF, NEG_INF, NEG_INF, NEG_INF); }
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
  static constexpr uint32_t NEG_INF = 0xff800000u;
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
  __device__ static uint4 none() {
    const uint32_t w = __float_as_uint(LOGIT_NONE);
    return make_uint4(w, w, w, w);
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

// Counters and the status word of a call, and its number of valid rows
// (one CTA: short enough for the row counts it is launched for).
constexpr int BEGIN_THREADS = 1024;
__global__ void __launch_bounds__(BEGIN_THREADS)
    flce_begin_kernel(const int32_t* y, int N, int ignore_index, unsigned int* ticket, int* n_valid, int* status) {
  int c = 0;
  for (int i = threadIdx.x; i < N; i += BEGIN_THREADS) c += y[i] != ignore_index ? 1 : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_down_sync(0xffffffffu, c, o);
  __shared__ int w[BEGIN_THREADS / 32];
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
    for (int k = 0; k < BEGIN_THREADS / 32; ++k) t += w[k];
    *n_valid = t;
    *ticket = 0u;
    *status = 0;
  }
}

// The last block to finish adds the rows' contributions in row order: a fixed
// tree over a fixed assignment, in fp64.
template <int THREADS>
__device__ __forceinline__ double ordered_sum(const double* v, int n, double* scratch) {
  double s = 0.0;
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
  const int* n_valid;
  unsigned int* ticket;
  double* blk_sum;      // [gridDim.x]
  double* loss;
  float* out_rows;      // [N] policy loss per row
  float* out_kl;        // [N]
  float* out_weight;    // [N] s_i dL_i/dl_i
};

constexpr int POLICY_THREADS = 256;
__global__ void __launch_bounds__(POLICY_THREADS) flce_policy_rows_kernel(const PolicyRowsArgs a) {
  const int n = *a.n_valid;
  const double inv_n = n > 0 ? 1.0 / static_cast<double>(n) : 0.0;
  double acc = 0.0;
  for (int i = blockIdx.x * POLICY_THREADS + threadIdx.x; i < a.N; i += gridDim.x * POLICY_THREADS) {
    float rows = 0.f, kl = 0.f, weight = 0.f;
    if (a.y[i] != a.ignore_index) {
      const PolicyRow p = policy_row(a.pol, policy_load(a.pol, i), -static_cast<double>(a.row_loss[i]));
      const double s = a.reduction == RED_MEAN ? inv_n
                       : a.reduction == RED_NONE && a.row_scale ? static_cast<double>(a.row_scale[i]) : 1.0;
      rows = static_cast<float>(p.loss);
      kl = static_cast<float>(p.kl);
      weight = static_cast<float>(-p.dlogp * s);
      acc += a.reduction == RED_MEAN ? p.loss : p.loss * s;
    }
    a.out_rows[i] = rows;
    a.out_kl[i] = kl;
    a.out_weight[i] = weight;
  }
  __shared__ double w[POLICY_THREADS / 32];
  __shared__ bool is_last;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_down_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int k = 0; k < POLICY_THREADS / 32; ++k) t += w[k];
    a.blk_sum[blockIdx.x] = t;
    __threadfence();
    is_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  const double t = ordered_sum<POLICY_THREADS>(a.blk_sum, gridDim.x, w);
  if (threadIdx.x == 0) *a.loss = a.reduction == RED_MEAN ? t * inv_n : t;
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
  const int* n_valid;
  unsigned int* ticket;
  double* row_acc;        // [N]
  float* loss;
  int* status;
  double inv_T;
  float zs;               // log2(e) / T
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

// A row's running statistics: max of z, sum of e = 2^((z - m) zs), and for the
// policy loss the first moment sum e (z - m) zs, for DISTILL2 the sum of
// 2^((z - m) log2 e).
struct RowStat {
  float m, l, t;
};

template <int LOSS>
__device__ __forceinline__ void stat_add(RowStat& s, float z, float zs) {
  if (z > s.m) {  // move to the new maximum
    const float d = (s.m - z) * zs, f = ex2_approx(d);
    if constexpr (is_policy(LOSS)) s.t = f * (s.t + s.l * fmaxf(d, NEG_BIG));
    if constexpr (LOSS == LOSS_DISTILL2) s.t *= ex2_approx((s.m - z) * LOG2E);
    s.l *= f;
    s.m = z;
  }
  const float d = (z - s.m) * zs, e = ex2_approx(d);
  s.l += e;
  if constexpr (is_policy(LOSS)) s.t += e * fmaxf(d, NEG_BIG);
  if constexpr (LOSS == LOSS_DISTILL2) s.t += ex2_approx((z - s.m) * LOG2E);
}

template <int LOSS>
__device__ __forceinline__ void stat_merge(RowStat& s, const RowStat& o, float zs) {
  const float m = fmaxf(s.m, o.m);
  const float d1 = (s.m - m) * zs, d2 = (o.m - m) * zs;
  const float f1 = ex2_approx(d1), f2 = ex2_approx(d2);
  if constexpr (is_policy(LOSS))
    s.t = f1 * (s.t + s.l * fmaxf(d1, NEG_BIG)) + f2 * (o.t + o.l * fmaxf(d2, NEG_BIG));
  if constexpr (LOSS == LOSS_DISTILL2)
    s.t = s.t * ex2_approx((s.m - m) * LOG2E) + o.t * ex2_approx((o.m - m) * LOG2E);
  s.l = s.l * f1 + o.l * f2;
  s.m = m;
}

// What the gradient pass needs of a row.
struct RowCoef {
  float a, b;    // dense part: e (a + b arg), or a e + b e1 with two softmaxes
};

constexpr int LOGIT_MAX_CLUSTER = 8;

// A row is split over the CTAs of a cluster, each of which holds its part in
// registers: 16-byte chunks on 16-byte boundaries, NCH per thread, so the
// logits are read from memory once and all of a thread's loads are in flight
// together.  (What lies beyond the registers, in rows longer than
// cluster * THREADS * NCH chunks, is read a second time for the gradient.)
// The up to 2 * (EPC - 1) elements in front of the first and behind the last
// boundary are held one per thread by the cluster's first CTA.
//
// Statistics: each warp folds its elements under its own maximum and writes one
// record into every CTA of the cluster; after one cluster barrier every warp
// merges all records in a fixed order, so all CTAs know the row's totals
// without a second exchange.  Warp 0 turns them into the row's outputs (first
// CTA) and the gradient's coefficients; then each CTA writes its part of the
// gradient and, behind a CTA barrier, the sparse entries that lie in it.
template <typename T, int LOSS, int THREADS, int NCH>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) flce_logit_loss_kernel(const LogitArgs a) {
  using L = LogitTraits<T>;
  constexpr int EPC = L::EPC;
  constexpr int WARPS = THREADS / 32;
  extern __shared__ __align__(16) uint8_t dyn[];
  const int K1 = is_policy(LOSS) ? 1 : a.K + 1;
  int* s_id = reinterpret_cast<int*>(dyn);           // sparse entries' vocabulary ids (-1: none)
  float* s_u = reinterpret_cast<float*>(s_id + K1);  // teacher logits
  float* s_c = s_u + K1;                             // coefficient subtracted at the entry
  float* s_z = s_c + K1;                             // the student's logit there
  __shared__ float4 rec[2][LOGIT_MAX_CLUSTER * WARPS];
  __shared__ RowCoef coef;
  __shared__ double dsum[WARPS];
  __shared__ bool is_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  const int clusters = gridDim.x / cs;
  const int n_valid = *a.n_valid;
  const double inv_n = n_valid > 0 ? 1.0 / static_cast<double>(n_valid) : 0.0;
  const uint64_t once = l2_evict_first();
  int parity = 0;
  for (int row = blockIdx.x / cs; row < a.N; row += clusters) {
    const T* z = static_cast<const T*>(a.z) + static_cast<long long>(row) * a.ld;
    T* g = a.g ? static_cast<T*>(a.g) + static_cast<long long>(row) * a.ldg : nullptr;
    // elements in front of the first 16-byte boundary, chunks, elements behind the last one
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const int head = min(a.V, mis ? EPC - mis : 0);
    const int chunks = (a.V - head) / EPC;
    const int edges = a.V - chunks * EPC;
    const int per = (chunks + cs - 1) / cs;
    const int c0 = min(chunks, rank * per), c1 = min(chunks, c0 + per);
    const T* zc = z + head;
    // the gradient row shares the logits' alignment, or its elements are stored one by one
    const bool vec_out = g && ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    const int edge_col = rank == 0 && tid < edges ? (tid < head ? tid : a.V - edges + tid) : -1;
    auto put = [&](int c, const uint4& o) {
      if (vec_out) {
        st_l2hint_v4(reinterpret_cast<uint4*>(g + head) + c, o, once);
      } else {
#pragma unroll
        for (int e = 0; e < EPC; ++e) g[head + c * EPC + e] = reinterpret_cast<const T*>(&o)[e];
      }
    };

    const int y = a.y[row];
    const bool in_range = y >= 0 && y < a.V;
    if (y == a.ignore_index || !in_range) {
      if (rank == 0 && tid == 0) {
        if (y != a.ignore_index) raise_status(a.status, ST_TARGET_OUT_OF_RANGE);
        a.row_acc[row] = 0.0;
        if constexpr (is_policy(LOSS)) {
          a.out_logp[row] = a.out_entropy[row] = a.out_kl[row] = 0.f;
        } else if (a.out_rows) {
          a.out_rows[row] = 0.f;
        }
      }
      if (g) {
        for (int c = c0 + tid; c < c1; c += THREADS) put(c, make_uint4(0u, 0u, 0u, 0u));
        if (edge_col >= 0) g[edge_col] = L::round(0.f);
      }
      continue;
    }

    // ---- the row's part of this CTA
    const uint4* zt = reinterpret_cast<const uint4*>(zc) + (c0 + tid);
    const int mine = c1 - c0 - tid;  // chunks from this thread's first on: u * THREADS < mine
    uint4 raw[NCH];
#pragma unroll
    for (int u = 0; u < NCH; ++u)
      raw[u] = u * THREADS < mine ? ld_l2hint_v4(zt + u * THREADS, once)
                                  : make_uint4(L::NEG_INF, L::NEG_INF, L::NEG_INF, L::NEG_INF);
    auto lifted = [&](float x) { return is_policy(LOSS) ? max_nan(x, LOGIT_LOWEST) : x; };
    const float none = is_policy(LOSS) ? LOGIT_NONE : -INFINITY;
    float edge = edge_col >= 0 ? L::load(z + edge_col) : -INFINITY;
    PolicyIn pin{};
    if (is_policy(LOSS) && tid == 0) pin = policy_load(a.pol, row);
    // the sparse entries: the teacher's, then the target
    for (int k = tid; k < K1; k += THREADS) {
      int id = y;
      float u = -INFINITY;
      if (k < K1 - 1) {
        const size_t at = static_cast<size_t>(row) * a.K + k;
        id = a.ids[at];
        if (id >= a.V) {
          raise_status(a.status, ST_TARGET_OUT_OF_RANGE);
          id = -1;
        }
        if (id >= 0) u = load_as_f32(a.u, a.u_dtype, at);
      }
      s_id[k] = id < 0 ? -1 : id;
      s_u[k] = u;
      s_z[k] = id < 0 ? 0.f : L::load(z + id);
    }

    // ---- statistics
    float top = edge;  // this thread's largest logit as it stands
    RowStat st{-FLT_MAX, 0.f, 0.f};
    for (int c = c0 + NCH * THREADS + tid; c < c1; c += THREADS) {  // beyond the registers
      const uint4 v = ld_l2hint_v4(reinterpret_cast<const uint4*>(zc) + c, l2_evict_normal());
#pragma unroll
      for (int i = 0; i < EPC / 2; ++i) {
        float lo, hi;
        f32x2_split(L::pair(v, i), lo, hi);
        top = fmaxf(top, fmaxf(lo, hi));
        stat_add<LOSS>(st, lifted(lo), a.zs);
        stat_add<LOSS>(st, lifted(hi), a.zs);
      }
    }
    typename L::Max vmax = L::max_init();
#pragma unroll
    for (int u = 0; u < NCH; ++u) L::max_add(vmax, raw[u]);
    top = fmaxf(top, L::max_get(vmax));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // -FLT_MAX, not -infinity, so that the differences below are never NaN for it
    RowStat w{fmaxf(top, is_policy(LOSS) ? LOGIT_LOWEST : -FLT_MAX), 0.f, 0.f};
    if constexpr (is_policy(LOSS)) {
#pragma unroll
      for (int u = 0; u < NCH; ++u) {
        if (u * THREADS < mine)
          L::clamp(raw[u]);
        else
          raw[u] = L::none();
      }
      edge = edge_col >= 0 ? lifted(edge) : none;
    }
    const uint64_t zs2 = f32x2(a.zs, a.zs), one2 = f32x2(LOG2E, LOG2E);
    {
      const uint64_t neg_m2 = f32x2(-w.m, -w.m);
      uint64_t l2 = 0ull, t2 = 0ull;  // two partial sums each
      auto fold = [&](uint64_t x) {
        const uint64_t d0 = add2(x, neg_m2);
        uint64_t d = mul2(d0, zs2);
        float lo, hi;
        f32x2_split(d, lo, hi);
        if constexpr (is_policy(LOSS) && !L::CLAMPS) {  // finite, so that a probability of 0 adds 0 to the entropy
          lo = max_nan(lo, NEG_BIG);
          hi = max_nan(hi, NEG_BIG);
          d = f32x2(lo, hi);
        }
        const uint64_t e = f32x2(ex2_approx(lo), ex2_approx(hi));
        l2 = add2(l2, e);
        if constexpr (is_policy(LOSS)) t2 = fma2(e, d, t2);
        if constexpr (LOSS == LOSS_DISTILL2) {
          f32x2_split(mul2(d0, one2), lo, hi);
          t2 = add2(t2, f32x2(ex2_approx(lo), ex2_approx(hi)));
        }
      };
#pragma unroll
      for (int u = 0; u < NCH; ++u) {
#pragma unroll
        for (int i = 0; i < EPC / 2; ++i) fold(L::pair(raw[u], i));
      }
      fold(f32x2(edge, none));
      float lo, hi;
      f32x2_split(l2, lo, hi);
      w.l = lo + hi;
      f32x2_split(t2, lo, hi);
      w.t = lo + hi;
    }
    if (c1 - c0 > NCH * THREADS) stat_merge<LOSS>(w, st, a.zs);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      w.l += __shfl_xor_sync(0xffffffffu, w.l, o);
      w.t += __shfl_xor_sync(0xffffffffu, w.t, o);
    }
    if (cs == 1) {
      if (lane == 0) rec[parity][warp] = make_float4(w.m, w.l, w.t, top);
      __syncthreads();
    } else {
      if (lane < cs)
        st_cluster_f4(mapa_shared(smem_u32(&rec[parity][rank * WARPS + warp]), lane), make_float4(w.m, w.l, w.t, top));
      cluster_sync_all();
    }

    // ---- the row's totals (every warp, the same order everywhere)
    const int records = cs * WARPS;
    w.m = -FLT_MAX;
    for (int r = lane; r < records; r += 32) w.m = fmaxf(w.m, rec[parity][r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w.m = fmaxf(w.m, __shfl_xor_sync(0xffffffffu, w.m, o));
    if (warp == 0) {
      w.l = w.t = 0.f;
      top = -INFINITY;
      for (int r = lane; r < records; r += 32) {
        const float4 v = rec[parity][r];
        top = fmaxf(top, v.w);
        RowStat o{w.m, 0.f, 0.f};
        stat_merge<LOSS>(o, RowStat{v.x, v.y, v.z}, a.zs);
        w.l += o.l;
        w.t += o.t;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        w.l += __shfl_xor_sync(0xffffffffu, w.l, o);
        w.t += __shfl_xor_sync(0xffffffffu, w.t, o);
      }
      if (is_policy(LOSS) && !__any_sync(0xffffffffu, top > -INFINITY)) w.l = 0.f;  // every logit is -infinity: NaN
      // Log-probabilities as (z - m)/T - ln L: the difference first, so that a
      // row whose every logit is the type's lowest value still has one.
      const double m = static_cast<double>(w.m);
      const double lnL = log(static_cast<double>(w.l));
      const double s = a.reduction == RED_MEAN ? inv_n
                       : a.reduction == RED_NONE && a.row_scale ? static_cast<double>(a.row_scale[row]) : 1.0;
      double total = 0.0;
      if constexpr (is_policy(LOSS)) {
        if (lane == 0) {
          const float zy = s_z[0] == -INFINITY ? s_z[0] : lifted(s_z[0]);
          const double lp = (static_cast<double>(zy) - m) * a.inv_T - lnL;
          const double inv_l = 1.0 / static_cast<double>(w.l);
          const double H = lnL - static_cast<double>(w.t) * inv_l * LN2;
          const PolicyRow p = policy_row(a.pol, pin, lp);
          total = p.loss;
          double a0 = -p.dlogp, a1 = 0.0;
          if (a.ent_coef != 0.0) {
            total -= a.ent_coef * H;
            a0 += a.ent_coef * (H - lnL);
            a1 = a.ent_coef * LN2;
          }
          const double f = s * a.inv_T;
          s_c[0] = static_cast<float>(-p.dlogp * f);
          coef.a = static_cast<float>(a0 * f * inv_l);
          coef.b = static_cast<float>(a1 * f * inv_l);
          if (rank == 0) {
            a.out_logp[row] = static_cast<float>(lp);
            a.out_entropy[row] = static_cast<float>(H);
            a.out_kl[row] = static_cast<float>(p.kl);
          }
        }
      } else {
        const TeacherShift ts = teacher_shift(s_u, a.K, lane, a.inv_T, a.teacher_lse, row);
        double Q = 0.0, kl = 0.0;
        if (ts.any) {
          for (int k = lane; k < a.K; k += 32) {
            const double lq = static_cast<double>(s_u[k]) * a.inv_T - ts.shift;
            const float q = expf(static_cast<float>(lq));
            s_c[k] = static_cast<float>(static_cast<double>(q) * a.kd * a.inv_T * s);
            Q += q;
            if (!(q == 0.f)) kl += static_cast<double>(q) * (lq - ((static_cast<double>(s_z[k]) - m) * a.inv_T - lnL));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            Q += __shfl_xor_sync(0xffffffffu, Q, o);
            kl += __shfl_xor_sync(0xffffffffu, kl, o);
          }
        } else {
          for (int k = lane; k < a.K; k += 32) s_c[k] = 0.f;
        }
        if (lane == 0) {
          if (a.kd != 0.0) total = a.kd * kl;
          double da = a.kd * Q * a.inv_T, db = 0.0;
          if (a.ce != 0.0) {
            const double ln1 = LOSS == LOSS_DISTILL2 ? log(static_cast<double>(w.t)) : lnL;
            total += a.ce * (m - static_cast<double>(s_z[a.K]) + ln1);
            if constexpr (LOSS == LOSS_DISTILL2)
              db = a.ce / static_cast<double>(w.t);
            else
              da += a.ce;
          }
          s_c[a.K] = static_cast<float>(a.ce * s);
          coef.a = static_cast<float>(da * s / static_cast<double>(w.l));
          coef.b = static_cast<float>(db * s);
          if (rank == 0 && a.out_rows) a.out_rows[row] = static_cast<float>(total);
        }
      }
      if (rank == 0 && lane == 0) a.row_acc[row] = a.reduction == RED_MEAN ? total : total * s;
    }
    __syncthreads();

    // ---- the gradient
    if (g) {
      // Unpack the chunks anew here: values kept unpacked since the sums would
      // take twice the registers, and spill.
#pragma unroll
      for (int u = 0; u < NCH; ++u)
        asm volatile("" : "+r"(raw[u].x), "+r"(raw[u].y), "+r"(raw[u].z), "+r"(raw[u].w));
      const RowCoef c = coef;
      const float m = w.m;
      const uint64_t neg_m2 = f32x2(-m, -m), a2 = f32x2(c.a, c.a), b2 = f32x2(c.b, c.b);
      auto dense2 = [&](uint64_t x) {
        const uint64_t d0 = add2(x, neg_m2);
        uint64_t d = mul2(d0, zs2);
        float lo, hi;
        f32x2_split(d, lo, hi);
        if constexpr (LOSS == LOSS_POLICY_ENT && !L::CLAMPS) {
          lo = max_nan(lo, NEG_BIG);
          hi = max_nan(hi, NEG_BIG);
          d = f32x2(lo, hi);
        }
        const uint64_t e = f32x2(ex2_approx(lo), ex2_approx(hi));
        if constexpr (LOSS == LOSS_POLICY_ENT) return mul2(e, fma2(b2, d, a2));
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
      auto grad_chunk = [&](const uint4& v) {
        uint4 o;
#pragma unroll
        for (int i = 0; i < EPC / 2; ++i) {
          float lo, hi;
          f32x2_split(dense2(L::pair(v, i)), lo, hi);
          L::put(o, i, lo, hi);
        }
        return o;
      };
      if (vec_out) {
        uint4* gt = reinterpret_cast<uint4*>(g + head) + (c0 + tid);
#pragma unroll
        for (int u = 0; u < NCH; ++u)
          if (u * THREADS < mine) st_l2hint_v4(gt + u * THREADS, grad_chunk(raw[u]), once);
      } else {
#pragma unroll
        for (int u = 0; u < NCH; ++u)
          if (u * THREADS < mine) put(c0 + u * THREADS + tid, grad_chunk(raw[u]));
      }
      for (int ch = c0 + NCH * THREADS + tid; ch < c1; ch += THREADS) {
        uint4 v = ld_l2hint_v4(reinterpret_cast<const uint4*>(zc) + ch, once);
        if constexpr (is_policy(LOSS)) L::clamp(v);
        put(ch, grad_chunk(v));
      }
      if (edge_col >= 0) g[edge_col] = L::round(dense(edge));
      __syncthreads();
      // The sparse entries of this CTA's part; equal ids add up, and each of
      // them writes the same sum.
      const int lo = head + c0 * EPC, hi = head + c1 * EPC;
      for (int k = tid; k < K1; k += THREADS) {
        const int id = s_id[k];
        const bool mine = id >= lo && id < hi ? true : rank == 0 && id >= 0 && (id < head || id >= head + chunks * EPC);
        if (!mine) continue;
        float c_sum = 0.f;
        for (int i = 0; i < K1; ++i)
          if (s_id[i] == id) c_sum += s_c[i];
        g[id] = L::round(dense(lifted(s_z[k])) - c_sum);
      }
    }
    __syncthreads();  // the shared row data is reused
    parity ^= 1;
  }
  // the loss, by the last cluster to finish
  if (rank != 0) return;
  if (tid == 0) {
    __threadfence();
    is_last = atomicAdd(a.ticket, 1u) == static_cast<unsigned>(clusters - 1);
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  const double t = ordered_sum<THREADS>(a.row_acc, a.N, dsum);
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
  int32_t* list_ids;      // [N][K + 1]
  float* list_c;
  float* list_z;          // read by flce_list_dot_kernel
  int* list_count;
  float* list_dense;
  double* list_const;
  double* list_lse;
  double* list_dot;
  int* status;
};

// Each row's entries (the teacher's, and the target when hard labels are mixed
// in) ascending by id, with the coefficients that the G tiles subtract there,
// and the row's constants:
//   L = kd sum q log q + (kd Q + ce) lse - sum_k c_k z_k,  c_k = kd q_k / T + ce [target],
//   G = s ((kd Q / T + ce) p - c).
// Entries are ranked by counting (id, position) pairs below their own, so the
// order is the same on every call; equal ids stay separate entries, which the
// G tiles subtract one after the other.  One CTA per row.
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
        a.list_const[i] = a.list_lse[i] = 0.0;
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
    double Q = 0.0, qlogq = 0.0;
    int count = 0;
    if (tid < 32) {
      for (int k = lane; k < K1; k += 32) {
        if (s_id[k] != 0x7fffffff) ++count;
        if (k < a.K && ts.any) {
          const double lq = static_cast<double>(s_u[k]) * a.inv_T - ts.shift;
          const float q = expf(static_cast<float>(lq));
          Q += q;
          if (!(q == 0.f)) qlogq += static_cast<double>(q) * lq;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        Q += __shfl_xor_sync(0xffffffffu, Q, o);
        qlogq += __shfl_xor_sync(0xffffffffu, qlogq, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
      }
      if (lane == 0) {
        a.list_count[i] = count;
        a.list_dense[i] = static_cast<float>(a.kd * Q * a.inv_T + a.ce);
        a.list_const[i] = a.kd * qlogq;
        a.list_lse[i] = a.kd * Q + a.ce;
      }
    }
    for (int k = tid; k < K1; k += TEACHER_THREADS) {
      const int id = s_id[k];
      if (id == 0x7fffffff) continue;
      int rank = 0;
      for (int j = 0; j < K1; ++j) rank += s_id[j] < id || (s_id[j] == id && j < k) ? 1 : 0;
      double c = a.ce;
      if (k < a.K) c = ts.any ? static_cast<double>(expf(static_cast<float>(static_cast<double>(s_u[k]) * a.inv_T - ts.shift))) * a.kd * a.inv_T : 0.0;
      a.list_ids[out + rank] = id;
      a.list_c[out + rank] = static_cast<float>(c);
    }
    __syncthreads();
  }
}

// sum_k c_k z_k of each row, in fp64 (one warp per row, fixed order).
__global__ void __launch_bounds__(256) flce_list_dot_kernel(const TeacherArgs a) {
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < a.N; i += gridDim.x * 8) {
    const size_t at = static_cast<size_t>(i) * (a.K + 1);
    const int n = a.list_count[i];
    double s = 0.0;
    for (int k = lane; k < n; k += 32) {
      const float c = a.list_c[at + k];
      if (!(c == 0.f)) s += static_cast<double>(c) * static_cast<double>(a.list_z[at + k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) a.list_dot[i] = s;
  }
}

}  // namespace flce

// Router kernels: logits -> route IDs and weights, the balance loss of a
// routing with its per-expert counts, and the gradient of both with respect to
// the logits. Every one reads each logit once.
//
// Layout: 16 lanes hold one row, four rows to a wave (a few rows of the top-k: 64). Lane i of a row holds
// experts 64 j + 4 i + v (v = 0..3) of block j in l[4 j + v]: 16 bytes of fp32
// or 8 of a 16-bit type in one load, and a block of a row is one run of 256 or
// 128 bytes. Reductions over a row are four rotations inside the 16 lanes of a
// DPP row, with no LDS traffic.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace exl3 {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kRowsPerWg = 16;  // 256 threads
// balance_kernel: 32 rows at a time, 16 above 512 experts (its sums are
// registers, and eight waves would not have enough)
constexpr int balance_threads(int I) { return I <= 8 ? 512 : 256; }
constexpr float kFltMax = 3.40282346638528859812e+38f;
constexpr float kNegInf = -__builtin_inff();

// ------------------------------------------------- 16-lane row reductions
// ror16<N>(v): the value of the lane N places on inside the 16-lane DPP row.
template <int N>
__device__ __forceinline__ int ror16(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ float ror16(float v) {
  return __builtin_bit_cast(float, ror16<N>(__builtin_bit_cast(int, v)));
}
template <int N>
__device__ __forceinline__ double ror16(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)ror16<N>((int)(uint32_t)u);
  const uint32_t hi = (uint32_t)ror16<N>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float kmax(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double kmax(double a, double b) { return fmax(a, b); }
// Every lane gets the result; sums add the same pairs in every lane.
template <typename T>
__device__ __forceinline__ T row_max(T v) {
  v = kmax(v, ror16<8>(v));
  v = kmax(v, ror16<4>(v));
  v = kmax(v, ror16<2>(v));
  return kmax(v, ror16<1>(v));
}
__device__ __forceinline__ int row_min(int v) {
  v = min(v, ror16<8>(v));
  v = min(v, ror16<4>(v));
  v = min(v, ror16<2>(v));
  return min(v, ror16<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += ror16<8>(v);
  v += ror16<4>(v);
  v += ror16<2>(v);
  return v + ror16<1>(v);
}
// Rows of L = 16 or 64 lanes. A swap of v with itself leaves each 16 (32) lanes
// and their neighbours in the same lanes of two registers.
template <int N>
__device__ __forceinline__ void swap_rows(uint32_t v, uint32_t &a, uint32_t &b) {
  typedef uint32_t pair __attribute__((ext_vector_type(2)));
  pair r;
  if constexpr (N == 16) r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  else r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
template <int N>
__device__ __forceinline__ float pair_max(float v) {
  uint32_t a, b;
  swap_rows<N>(__builtin_bit_cast(uint32_t, v), a, b);
  return kmax(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
template <int N>
__device__ __forceinline__ double pair_max(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t la, lb, ha, hb;
  swap_rows<N>((uint32_t)u, la, lb);
  swap_rows<N>((uint32_t)(u >> 32), ha, hb);
  return kmax(__builtin_bit_cast(double, ((uint64_t)ha << 32) | la),
              __builtin_bit_cast(double, ((uint64_t)hb << 32) | lb));
}
template <int N>
__device__ __forceinline__ int pair_min(int v) {
  uint32_t a, b;
  swap_rows<N>((uint32_t)v, a, b);
  return min((int)a, (int)b);
}
template <int L, typename T>
__device__ __forceinline__ T wide_max(T v) {
  v = row_max(v);
  if constexpr (L == 64) v = pair_max<32>(pair_max<16>(v));
  return v;
}
template <int L>
__device__ __forceinline__ int wide_min(int v) {
  v = row_min(v);
  if constexpr (L == 64) v = pair_min<32>(pair_min<16>(v));
  return v;
}
__device__ __forceinline__ bool row_any(bool b) {
  const int shift = (threadIdx.x & 48);
  return ((__ballot(b) >> shift) & 0xffffull) != 0;
}

// ------------------------------------------------------------------ loads
// dtype codes of the launch parameters: 1 fp16, 2 bf16, 3 fp32
__device__ __forceinline__ float load_as_f32(const void *p, int dtype, int64_t i) {
  if (dtype == 3) return ((const float *)p)[i];
  const uint16_t b = ((const uint16_t *)p)[i];
  return dtype == 2 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}
// NaN and -inf -> -inf (the expert takes no part), +inf -> the largest finite
// fp32 (exp(l - max) stays defined).
__device__ __forceinline__ float clean(float l) {
  return l == l ? fminf(l, kFltMax) : kNegInf;
}

// The lane's share of a row as loaded: four fp32 or four 16-bit logits a block.
template <int DT>
struct Raw {
  typedef uint32_t type __attribute__((ext_vector_type(2)));
};
template <>
struct Raw<3> {
  typedef u32x4 type;
};
template <int I, int DT>
using RawRow = typename Raw<DT>::type[I];

// Loads of the row whose first element has index `at` (not waited for). vec4:
// E is a multiple of four and every group of four starts on one, so a group is
// one load. Groups and values past E read the last ones again: no branch stands
// between the loads, which would make each wait for the one before.
template <int I, int DT, int L = 16>
__device__ __forceinline__ void load_raw(const RouterParams &p, int64_t at, int lane,
                                         RawRow<I, DT> &raw) {
  typedef typename Raw<DT>::type raw_t;
  if (p.vec4) {
    const char *q = (const char *)p.logits + at * (DT == 3 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < I; ++j)
      raw[j] = *(const raw_t *)(q + min(4 * L * j + 4 * lane, p.E - 4) * (DT == 3 ? 4 : 2));
  } else {
    asm volatile("" : "+v"(lane));  // 4 I indexes are computed here, not kept in registers
#pragma unroll
    for (int j = 0; j < I; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t e = at + min(4 * L * j + 4 * lane + v, p.E - 1);
        if constexpr (DT == 3) w[v] = ((const uint32_t *)p.logits)[e];
        else w[v] = ((const uint16_t *)p.logits)[e];
      }
      if constexpr (DT == 3) raw[j] = (raw_t){w[0], w[1], w[2], w[3]};
      else raw[j] = (raw_t){w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
    }
  }
}
template <int I, int DT, int L = 16>
__device__ __forceinline__ void unpack_row(const RouterParams &p, int lane,
                                           const RawRow<I, DT> &raw, float (&l)[4 * I]) {
#pragma unroll
  for (int j = 0; j < I; ++j) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if constexpr (DT == 3) {
        const uint32_t b = raw[j][v];
        l[4 * j + v] = clean(__builtin_bit_cast(float, b));
      } else {
        const uint32_t w = raw[j][v >> 1];
        const uint16_t b = (uint16_t)(w >> (16 * (v & 1)));
        l[4 * j + v] = clean(DT == 2 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b));
      }
    }
    if (4 * L * (j + 1) > p.E) {  // the block that E ends in
#pragma unroll
      for (int v = 0; v < 4; ++v)
        l[4 * j + v] = 4 * L * j + 4 * lane + v < p.E ? l[4 * j + v] : kNegInf;
    }
  }
}

template <int N>
__device__ __forceinline__ float max_of(const float (&l)[N]) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = fmaxf(m, l[j]);
  return m;
}

// ------------------------------------------------------------------ scores
// A row's t_e up to one factor per row (it cancels wherever t is divided by a
// sum of t). Softmax: exp(l - m), m the row's largest logit. Sigmoid:
// 1 / (1 + exp(-l)) times exp(-m), m = min(0, largest logit), as
// exp(l - m) / (1 + exp(l)) for l < 0 (m = 0 where any l is not): the largest
// t is at least 1/2, so no sum of t underflows however far below zero the
// logits lie. shift() maps the largest logit to m; a row without experts
// (largest logit -inf) gets m = 0 and t = 0 throughout.
__device__ __forceinline__ float shift(bool sigmoid, float largest) {
  if (largest == kNegInf) return 0.0f;
  return sigmoid ? fminf(0.0f, largest) : largest;
}
__device__ __forceinline__ float strength(bool sigmoid, float l, float m) {
  if (!sigmoid) return expf(l - m);
  const float z = expf(-fabsf(l));
  return (l < 0.0f ? expf(l - m) : 1.0f) / (1.0f + z);
}
// t of every expert of a row, for sums, probabilities and gradients: the
// hardware's exp2 and reciprocal (1 ulp each) instead of the full functions.
// (l - m) log2(e) is rounded once more than l - m is, so t is off by
// 2 |l - m| 2^-24 rather than |l - m| 2^-24 at most; a t below 2^-126 counts
// as 0. Chosen experts' weights, two to a lane, take strength().
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}
template <int N>
__device__ __forceinline__ void fast_strengths(bool sigmoid, const float (&l)[N], float m,
                                               float (&t)[N]) {
  if (!sigmoid) {
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = fast_exp(l[j] - m);
  } else if (m == 0.0f) {  // the row's own: its bytes do not depend on the wave's other rows
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[j]));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      t[j] = fast_exp(fminf(l[j], 0.0f) - m) * __builtin_amdgcn_rcpf(1.0f + fast_exp(-fabsf(l[j])));
  }
}
// The same of sigmoid scores, with h = d log t / d l = 1 - sigmoid(l).
template <int N>
__device__ __forceinline__ void fast_strengths_slopes(const float (&l)[N], float m, float (&t)[N],
                                                      float (&h)[N]) {
  if (m == 0.0f) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float z = fast_exp(-l[j]);  // infinite where t is 0
      t[j] = __builtin_amdgcn_rcpf(1.0f + z);
      h[j] = fminf(z, kFltMax) * t[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float z = fast_exp(-fabsf(l[j])), r = __builtin_amdgcn_rcpf(1.0f + z);
      t[j] = fast_exp(fminf(l[j], 0.0f) - m) * r;
      h[j] = (l[j] < 0.0f ? 1.0f : z) * r;
    }
  }
}
// d log t / d l: 1, or 1 - sigmoid(l) computed without cancellation.
__device__ __forceinline__ float slope(bool sigmoid, float l) {
  if (!sigmoid) return 1.0f;
  const float z = expf(-fabsf(l));
  return (l < 0.0f ? 1.0f : z) / (1.0f + z);
}
// 1 / x, 0 for an empty sum.
__device__ __forceinline__ float inv_or_0(float x) { return x > 0.0f ? 1.0f / x : 0.0f; }

__device__ __forceinline__ void store_as(void *p, int dtype, int64_t i, float v) {
  if (dtype == 3) ((float *)p)[i] = v;
  else ((uint16_t *)p)[i] = f32_to_out16(v, dtype == 2);
}

// ------------------------------------------------------------------- top-k
// Selection keys: the logit itself, or with a bias sigmoid(l) + bias in fp64.
// fp32 would round the sum to 2^-24 and order near-equal experts by their
// index rather than their score.
template <bool BIAS>
struct Key {
  typedef float type;
};
template <>
struct Key<true> {
  typedef double type;
};

// L = 16 or 64 lanes to a row. Bound by the chain of k selections, not by bytes:
// 8192 x 192 fp32 (6.7 MB, 1.3 us at 5 TB/s), k = 8: 6.4 us; a few rows 4 (an
// empty launch: 2.5), with a bias, for the fp64 scores, 6.
template <int I, int DT, bool BIAS, int L>
__global__ void __launch_bounds__(256) route_topk_kernel(RouterParams p) {
  typedef typename Key<BIAS>::type key_t;
  const int lane = threadIdx.x & (L - 1);
  const int64_t row =
      ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (256 / L) + threadIdx.x / L;
  const bool in = row < p.rows;
  const bool live = in && (!p.row_mask || p.row_mask[row] != 0);
  const int64_t at = (live ? row : 0) * p.ld_logits;
  RawRow<I, DT> raw;
  load_raw<I, DT, L>(p, at, lane, raw);
  float l[4 * I];
  unpack_row<I, DT, L>(p, lane, raw, l);
  if (!live) {
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) l[j] = kNegInf;
  }
  const bool sig = p.sigmoid;
  // softmax over all experts: its sum, while the logits are at hand. Rows of 64
  // lanes have no such form (launch_route_topk).
  const bool over_all = L == 16 && !sig && !p.renorm;
  float m_all = 0.0f, total = 0.0f;
  if (over_all) {
    m_all = shift(false, row_max(max_of(l)));
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) total += fast_exp(l[j] - m_all);
    total = row_sum(total);
  }
  key_t s[4 * I];
#pragma unroll
  for (int j = 0; j < 4 * I; ++j) {
    const int e = 4 * L * (j >> 2) + 4 * lane + (j & 3);
    if constexpr (BIAS) {
      const double b = e < p.E ? (double)p.bias[e] : 0.0;
      const double v = 1.0 / (1.0 + exp(-(double)l[j])) + b;
      s[j] = l[j] > kNegInf && v == v ? v : (double)kNegInf;
    } else {
      s[j] = l[j];
    }
  }
  // k times: the largest key of the row, then the lowest expert holding it.
  // Lane j keeps picks j and j + 16.
  int pick[2] = {-1, -1};
  for (int k = 0; k < p.topk; ++k) {
    // four chains side by side: one chain of 4 I dependent steps is most of a
    // small call's time
    key_t top[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      top[v] = s[v];
#pragma unroll
      for (int j = 1; j < I; ++j) top[v] = kmax(top[v], s[4 * j + v]);
    }
    const key_t best = wide_max<L>(kmax(kmax(top[0], top[1]), kmax(top[2], top[3])));
    int first[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      first[v] = 0x7fffffff;
#pragma unroll
      for (int j = I - 1; j >= 0; --j)
        first[v] = s[4 * j + v] == best ? 4 * L * j + 4 * lane + v : first[v];
    }
    const int e = wide_min<L>(min(min(first[0], first[1]), min(first[2], first[3])));
    const bool some = best > (key_t)kNegInf;
#pragma unroll
    for (int j = 0; j < 4 * I; ++j)
      s[j] = 4 * L * (j >> 2) + 4 * lane + (j & 3) == e ? (key_t)kNegInf : s[j];
    if ((k & 15) == lane) pick[k >> 4] = some ? e : -1;
  }
  // weights of the picks, from their logits
  float lp[2], t[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    lp[h] = pick[h] >= 0 ? clean(load_as_f32(p.logits, DT, at + pick[h])) : kNegInf;
  const float m = p.renorm ? shift(sig, row_max(fmaxf(lp[0], lp[1]))) : m_all;
#pragma unroll
  for (int h = 0; h < 2; ++h) t[h] = pick[h] >= 0 ? strength(sig, lp[h], m) : 0.0f;
  if (p.renorm) total = row_sum(t[0] + t[1]);
  if (!in || lane >= 16) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = lane + 16 * h;
    if (k >= p.topk) continue;
    const int64_t o = row * p.topk + k;
    const float w = pick[h] < 0 ? 0.0f : (sig && !p.renorm) ? p.scale * t[h]
                                                            : p.scale * (t[h] / total);
    if (p.ids_i64) ((int64_t *)p.ids)[o] = pick[h];
    else ((int32_t *)p.ids)[o] = pick[h];
    store_as(p.w, p.w_dtype, o, w);
  }
}

// The row's IDs j = lane and lane + 16, as loaded (a lane without one reads
// the row's last) and as experts: -1 for none, outside [0, E), or past the
// row's topk. At most 16 IDs leave the second one out. Nothing is made of a
// loaded value here, behind a branch on its type: the wait for it would come
// before the loads that follow.
__device__ __forceinline__ void load_ids(const RouterParams &p, int64_t row, int lane,
                                         uint32_t (&raw)[4]) {
  const int64_t at = row * p.topk;
  auto one = [&](int64_t i, uint32_t &lo, uint32_t &hi) {
    if (p.ids_i64) {
      const u32x2 v = ((const u32x2 *)p.ids)[i];
      lo = v[0];
      hi = v[1];
    } else {
      lo = ((const uint32_t *)p.ids)[i];
    }
  };
  one(at + min(lane, p.topk - 1), raw[0], raw[1]);
  if (p.topk > 16) one(at + min(lane + 16, p.topk - 1), raw[2], raw[3]);
}
__device__ __forceinline__ void take_ids(const RouterParams &p, bool in, int lane,
                                         const uint32_t (&raw)[4], int (&id)[2]) {
  auto one = [&](int k, uint32_t lo, uint32_t hi) {
    const bool ok = lo < (uint32_t)p.E && (!p.ids_i64 || hi == 0);
    return in && k < p.topk && ok ? (int)lo : -1;
  };
  id[0] = one(lane, raw[0], raw[1]);
  id[1] = one(lane + 16, raw[2], raw[3]);
}
// A value of a [rows][topk] array, as loaded and as fp32.
__device__ __forceinline__ uint32_t load_bits(const void *p, int dtype, int64_t i) {
  return dtype == 3 ? ((const uint32_t *)p)[i] : ((const uint16_t *)p)[i];
}
__device__ __forceinline__ float bits_to_f32(uint32_t b, int dtype) {
  return dtype == 3   ? __builtin_bit_cast(float, b)
         : dtype == 2 ? bf16_bits_to_f32((uint16_t)b)
                      : f16_bits_to_f32((uint16_t)b);
}

// ----------------------------------------------------------------- balance
// Workgroup b sums every gridDim-th 32 rows from the 32 b-th on: probabilities
// in registers, counts by LDS integer atomics (exact in any order). Its sums
// go to part_prob[b][E], part_count[b][E] and part_tokens[b]; they are added
// in the order of b by balance_sum_kernel, so the same call gives the same
// bytes.
// The next rows' loads are under way while a row is summed up. 65536 x 256 bf16,
// sigmoid (35.7 MB): 14.8 us, 2.4 TB/s. The counters show 22 vector instructions
// a logit, two of them (exp2, rcp) at a quarter of the rate, and the vector units
// at work for 10 us of it; the rest is filling up and the last sums. With expf,
// division and no rows ahead 50 us.
template <int I, int DT>
__global__ void __launch_bounds__(balance_threads(I)) balance_kernel(RouterParams p) {
  constexpr int kThreads = balance_threads(I), kWaves = kThreads / 64, kRows = kThreads / 16;
  __shared__ int s_count[64 * I];
  __shared__ float s_prob[kWaves][64 * I];
  __shared__ int s_tokens;
  const int lane = threadIdx.x & 15, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < 64 * I; e += kThreads) s_count[e] = 0;
  if (threadIdx.x == 0) s_tokens = 0;
  __syncthreads();
  float acc[4 * I];
#pragma unroll
  for (int j = 0; j < 4 * I; ++j) acc[j] = 0.0f;
  const bool sig = p.sigmoid;
  int tokens = 0;
  int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 4);
  const int64_t step = (int64_t)gridDim.x * kRows;
  const int64_t last = p.rows - 1;
  uint32_t next_id[4] = {0, 0, 0, 0};
  RawRow<I, DT> next;
  if (last >= 0) {
    load_ids(p, min(row, last), lane, next_id);
    load_raw<I, DT>(p, min(row, last) * p.ld_logits, lane, next);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 <= last; r0 += step, row += step) {
    int id[2];
    take_ids(p, row <= last, lane, next_id, id);
    float l[4 * I];
    unpack_row<I, DT>(p, lane, next, l);
    if (r0 + step <= last) {
      load_ids(p, min(row + step, last), lane, next_id);
      load_raw<I, DT>(p, min(row + step, last) * p.ld_logits, lane, next);
    }
    const bool live = row_any(id[0] >= 0 || id[1] >= 0);
    const float m = shift(sig, row_max(max_of(l)));
    float t[4 * I], sum = 0.0f;
    fast_strengths(sig, l, m, t);
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) sum += t[j];
    const float inv = live ? inv_or_0(row_sum(sum)) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) acc[j] += t[j] * inv;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && p.topk <= 16) break;
      if (id[h] >= 0) atomicAdd(&s_count[id[h]], 1);
    }
    tokens += live ? 1 : 0;
  }
  if (lane == 0 && tokens) atomicAdd(&s_tokens, tokens);
  // the wave's four rows, then the waves
#pragma unroll
  for (int j = 0; j < 4 * I; ++j) {
    acc[j] += __shfl_xor(acc[j], 16, 64);
    acc[j] += __shfl_xor(acc[j], 32, 64);
    if ((threadIdx.x & 48) == 0) s_prob[wave][64 * (j >> 2) + 4 * lane + (j & 3)] = acc[j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    float sum = s_prob[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += s_prob[w][e];
    p.part_prob[(int64_t)blockIdx.x * p.E + e] = sum;
    p.part_count[(int64_t)blockIdx.x * p.E + e] = s_count[e];
  }
  if (threadIdx.x == 0) {
    p.part_tokens[blockIdx.x] = s_tokens;
    if (blockIdx.x == 0) *p.part_arrived = 0;
  }
}

// Adds the partial sums and forms the loss. Workgroup b takes experts 16 b ..
// 16 b + 15: 64 threads to an expert, each over every 64th partial sum, then
// the 64 in order. The workgroup that arrives last (part_arrived, zeroed by
// balance_kernel) adds the workgroups' shares of the loss in their order.
// One workgroup for all experts took 66 us on 256 partial sums of 256 experts,
// a chain of dependent loads; 16 threads to an expert 7.5 us on 512, these 6.6,
// of which a launch that does nothing is 2.5.
constexpr int kSumSlices = 64;

__global__ void __launch_bounds__(16 * kSumSlices) balance_sum_kernel(RouterParams p) {
  __shared__ float s_prob[kSumSlices][17];
  __shared__ int s_count[kSumSlices][17];
  __shared__ float s_share[16];
  __shared__ int s_tokens, s_last;
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + c;
  if (threadIdx.x == 0) s_tokens = 0;
  __syncthreads();
  float prob = 0.0f;
  int count = 0, tokens = 0;
  for (int b = threadIdx.x; b < p.nblk; b += 16 * kSumSlices) tokens += p.part_tokens[b];
  if (e < p.E) {
#pragma unroll 8
    for (int b = slice; b < p.nblk; b += kSumSlices) {
      prob += p.part_prob[(int64_t)b * p.E + e];
      count += p.part_count[(int64_t)b * p.E + e];
    }
  }
  if (tokens) atomicAdd(&s_tokens, tokens);
  s_prob[slice][c] = prob;
  s_count[slice][c] = count;
  __syncthreads();
  const int T = s_tokens;
  if (threadIdx.x < 16) {
    prob = 0.0f;
    count = 0;
#pragma unroll 16
    for (int i = 0; i < kSumSlices; ++i) {
      prob += s_prob[i][c];
      count += s_count[i][c];
    }
    prob = T > 0 ? prob / (float)T : 0.0f;
    if (e < p.E) {
      p.count[e] = count;
      p.prob[e] = prob;
    }
    s_share[c] = T > 0 ? (float)count / ((float)T * (float)p.topk) * prob : 0.0f;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float share = 0.0f;
    for (int i = 0; i < 16; ++i) share += s_share[i];
    __hip_atomic_store(p.part_share + blockIdx.x, share, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    s_last = __hip_atomic_fetch_add(p.part_arrived, 1, __ATOMIC_ACQ_REL,
                                    __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last || threadIdx.x >= 64) return;
  // at most 64 shares (1024 experts): one to a lane
  float v = threadIdx.x < gridDim.x ? __hip_atomic_load(p.part_share + threadIdx.x,
                                                        __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT)
                                    : 0.0f;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  if (threadIdx.x == 0) {
    p.tokens[0] = T;
    p.loss[0] = p.coef * (float)p.E * v;
  }
}

// ---------------------------------------------------------------- backward
// With g the incoming gradient and p, q = t over its sum over all experts,
// over the chosen:
//   weights  renorm         dl_e = scale q_e h_e (g_e - sum q g)
//            softmax, all   dl_e = scale p_e (g_e - sum p g)
//            sigmoid        dl_e = scale t_e h_e g_e
//   balance  dl_e = c p_e h_e (f_e - sum f p),  c = dloss coef E / T
// (h = slope, g = 0 where not chosen). Both in one pass over the row.
//
// The chosen entries reach the lanes that hold their experts through LDS, one
// [E] row per 16 lanes, zeroed and filled by the row's own lanes (a wave's LDS
// operations stay in order: lds_exchange() between the steps, no barrier). Comparing
// every chosen expert with every lane's experts took 24 of 45 instructions
// per logit and 28 us on 32768 x 256.
//
// SIG, the scores, is a template argument: with a branch on it 32768 x 256 took
// 20 us in bf16 (softmax), 22 in fp32 and 23 with sigmoid scores; so it is 18.2,
// 19.3 and 19.3, and 131072 rows of bf16 48 (2.8 TB/s). The counters show 33
// vector instructions a logit: the vector units are at work for 29 us of those 48
// and for 7 of the 18, where reading, working and writing are done by all waves
// at the same time and a row's entries cross LDS three times. More than 128
// registers cost more than they give (sigmoid slopes kept beside the logits: 72
// instead of 54).
template <int I, int DT, bool SIG>
__global__ void __launch_bounds__(256) route_backward_kernel(RouterParams p) {
  __shared__ __align__(16) float s_add[kRowsPerWg][64 * I];
  const int lane = threadIdx.x & 15;
  constexpr bool sig = SIG;
  const bool need_all = p.count != nullptr || (!sig && !p.renorm);
  const bool two = p.topk > 16;  // else no lane has a second entry
  float *add = s_add[threadIdx.x >> 4];

  int64_t row = (int64_t)blockIdx.x * kRowsPerWg + (threadIdx.x >> 4);
  const int64_t step = (int64_t)gridDim.x * kRowsPerWg;
  const int64_t last = p.rows - 1;
  // the next rows' loads are under way while a row is worked on
  uint32_t next_id[4] = {0, 0, 0, 0};
  uint32_t next_g[2] = {0, 0};
  RawRow<I, DT> next;
  auto fetch = [&](int64_t r) {
    load_raw<I, DT>(p, r * p.ld_logits, lane, next);
    load_ids(p, r, lane, next_id);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!p.dw || (h == 1 && !two)) break;
      next_g[h] = load_bits(p.dw, p.dw_dtype, r * p.topk + min(lane + 16 * h, p.topk - 1));
    }
  };
  fetch(min(row, last));
  // the balance loss: c f_e
  float cf[4 * I];
#pragma unroll
  for (int j = 0; j < 4 * I; ++j) cf[j] = 0.0f;
  if (p.count) {
#pragma unroll
    for (int j = 0; j < 4 * I; ++j)  // past E: the last expert's, times p = 0
      cf[j] = (float)p.count[min(64 * (j >> 2) + 4 * lane + (j & 3), p.E - 1)];
    const float T = (float)*p.tokens;
    const float c = T > 0.0f ? (p.dloss ? *p.dloss : 1.0f) * p.coef * (float)p.E / T : 0.0f;
    const float cn = T > 0.0f ? c / (T * (float)p.topk) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * I; ++j) cf[j] *= cn;
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kRowsPerWg; r0 <= last; r0 += step, row += step) {
    int id[2];
    take_ids(p, row <= last, lane, next_id, id);
    float g[2] = {bits_to_f32(next_g[0], p.dw_dtype), bits_to_f32(next_g[1], p.dw_dtype)};
    float l[4 * I];
    unpack_row<I, DT>(p, lane, next, l);
    if (r0 + step <= last) fetch(min(row + step, last));
    const bool live = row_any(id[0] >= 0 || id[1] >= 0);
    const float m = shift(sig, row_max(max_of(l)));
    // the chosen entries' logits, from the lanes that hold them (before the
    // probabilities, which then take the logits' registers)
    float lp[2] = {kNegInf, kNegInf};
    if (p.dw) {
#pragma unroll
      for (int j = 0; j < I; ++j)
        *(f32x4 *)(add + 64 * j + 4 * lane) =
            (f32x4){l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]};
      lds_exchange();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) break;
        if (id[h] >= 0) lp[h] = add[id[h]];
        if (lp[h] == kNegInf) g[h] = 0.0f;  // an expert that takes no part
      }
      lds_exchange();
#pragma unroll
      for (int j = 0; j < I; ++j)
        *(f32x4 *)(add + 64 * j + 4 * lane) = (f32x4){0.f, 0.f, 0.f, 0.f};
      lds_exchange();
    }
    float pe[4 * I], h[4 * I], inv = 0.0f;  // p_e, and with sigmoid scores h_e
    float mean = 0.0f;  // c sum f p, and for softmax over all experts scale sum p g
    if (need_all) {
      float total = 0.0f;
      if constexpr (sig) fast_strengths_slopes(l, m, pe, h);
      else fast_strengths(false, l, m, pe);
#pragma unroll
      for (int j = 0; j < 4 * I; ++j) total += pe[j];
      inv = live ? inv_or_0(row_sum(total)) : 0.0f;
#pragma unroll
      for (int j = 0; j < 4 * I; ++j) {
        pe[j] *= inv;
        mean += cf[j] * pe[j];
      }
      mean = row_sum(mean);
    } else {
#pragma unroll
      for (int j = 0; j < 4 * I; ++j) pe[j] = h[j] = 0.0f;
    }

    if (p.dw) {
      // v: what each chosen entry adds to its expert's gradient
      float v[2] = {0.0f, 0.0f};
      if (p.renorm) {
        const float mc = shift(sig, row_max(fmaxf(lp[0], lp[1])));
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          q[h] = strength(sig, lp[h], mc);
        }
        const float iq = inv_or_0(row_sum(q[0] + q[1]));
        const float gm = row_sum(q[0] * g[0] + q[1] * g[1]) * iq;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          if (lp[h] > kNegInf) v[h] = p.scale * (q[h] * iq) * slope(sig, lp[h]) * (g[h] - gm);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          v[h] = p.scale * g[h] *
                 (sig ? strength(true, lp[h], 0.0f) * slope(true, lp[h]) : fast_exp(lp[h] - m) * inv);
        }
        if (!sig) mean += row_sum(v[0] + v[1]);
      }
      // an expert named twice: its entry holds the tag of only one of them
      bool twice = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) break;
        if (id[h] >= 0) add[id[h]] = (float)(lane + 16 * h);
      }
      lds_exchange();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) break;
        if (id[h] >= 0) twice |= add[id[h]] != (float)(lane + 16 * h);
      }
      lds_exchange();
      if (!row_any(twice)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          if (id[h] >= 0) add[id[h]] = v[h];
        }
      } else {  // one entry after the other, in the order of the row's IDs
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (id[h] >= 0) add[id[h]] = 0.0f;
        for (int k = 0; k < p.topk; ++k) {
          const int i = k < 16 ? id[0] : id[1];
          const float a = k < 16 ? v[0] : v[1];
          lds_exchange();
          if ((k & 15) == lane && i >= 0) add[i] += a;
        }
      }
      lds_exchange();
    }

    // A row or an expert that takes no part has gradient 0: its p and its
    // added value are 0, so only a row whose mean is not finite needs to look
    // (0 times infinity).
    const bool odd = !(fabsf(mean) < __builtin_inff());
    if (row > last) continue;
    const int64_t to = row * p.ld_dlogits;
#pragma unroll
    for (int j = 0; j < I; ++j) {
      const int e0 = 64 * j + 4 * lane;
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
      if (p.dw) d = *(const f32x4 *)(add + e0);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float x = cf[4 * j + v] - mean;
        const float y = pe[4 * j + v] * (sig ? h[4 * j + v] * x : x);
        d[v] += odd && pe[4 * j + v] == 0.0f ? 0.0f : y;
      }
      if (p.dvec4 && e0 + 4 <= p.E) {
        if (p.dlogits_dtype == 3)
          *(f32x4 *)((float *)p.dlogits + to + e0) = d;
        else
          *(uint2 *)((uint16_t *)p.dlogits + to + e0) =
              make_uint2(f32x2_to_out16(d[0], d[1], p.dlogits_dtype == 2),
                         f32x2_to_out16(d[2], d[3], p.dlogits_dtype == 2));
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (e0 + v < p.E) store_as(p.dlogits, p.dlogits_dtype, to + e0 + v, d[v]);
      }
    }
  }
}

// f(blocks of 64 (rows of 64 lanes: 256) experts a kernel instance holds per
// row, logit type)
template <typename F>
hipError_t by_row(const RouterParams &p, int block, F f) {
  auto typed = [&](auto I) {
    if (p.logits_dtype == 1) f(I, std::integral_constant<int, 1>());
    else if (p.logits_dtype == 2) f(I, std::integral_constant<int, 2>());
    else f(I, std::integral_constant<int, 3>());
    return hipGetLastError();
  };
  const int blocks = (p.E + block - 1) / block;
  if (blocks <= 1) return typed(std::integral_constant<int, 1>());
  if (blocks <= 2) return typed(std::integral_constant<int, 2>());
  if (blocks <= 3) return typed(std::integral_constant<int, 3>());
  if (blocks <= 4) return typed(std::integral_constant<int, 4>());
  if (blocks <= 8) return typed(std::integral_constant<int, 8>());
  if (blocks <= 16) return typed(std::integral_constant<int, 16>());
  return hipErrorInvalidValue;
}

unsigned row_groups(int rows) { return ((unsigned)rows + kRowsPerWg - 1) / kRowsPerWg; }

}  // namespace

hipError_t launch_route_topk(const RouterParams &p, hipStream_t s) {
  // Rows of 64 lanes while there are waves to spare (in us, 64 lanes and 16: 256
  // rows of 256 experts 4.5 and 5.4, with a bias 6.0 and 9.6; 1024 rows 4.7 and
  // 5.5, 6.0 and 9.7; 4096 rows 7.2 and 5.7, 10.1 and 10.0; 1024 experts, k = 16,
  // 256 rows 8.3 and 19.9). The sum of a softmax over all experts would change
  // its order, and a row's bytes with the number of rows: it stays with 16.
  if (p.E > 64 && p.rows <= 1024 && (p.sigmoid || p.renorm)) {
    const dim3 grid((p.rows + 3) / 4);
    return by_row(p, 256, [&](auto I, auto D) {
      constexpr int i = decltype(I)::value, d = decltype(D)::value;
      if constexpr (i <= 4) {
        if (p.bias) hipLaunchKernelGGL((route_topk_kernel<i, d, true, 64>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((route_topk_kernel<i, d, false, 64>), grid, dim3(256), 0, s, p);
      }
    });
  }
  // an axis of a launch holds fewer than 2^32 threads
  const unsigned groups = row_groups(p.rows), x = min(groups, 1u << 22);
  const dim3 grid(x, (groups + x - 1) / x);
  return by_row(p, 64, [&](auto I, auto D) {
    constexpr int i = decltype(I)::value, d = decltype(D)::value;
    if (p.bias) hipLaunchKernelGGL((route_topk_kernel<i, d, true, 16>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((route_topk_kernel<i, d, false, 16>), grid, dim3(256), 0, s, p);
  });
}

int balance_blocks(int rows) {
  return (int)max(1u, min((row_groups(rows) + 1) / 2, 512u));  // two workgroups to a CU
}

hipError_t launch_balance(const RouterParams &p, hipStream_t s) {
  return by_row(p, 64, [&](auto I, auto D) {
    hipLaunchKernelGGL((balance_kernel<decltype(I)::value, decltype(D)::value>), dim3(p.nblk),
                       dim3(balance_threads(decltype(I)::value)), 0, s, p);
  });
}

hipError_t launch_balance_sum(const RouterParams &p, hipStream_t s) {
  hipLaunchKernelGGL(balance_sum_kernel, dim3((p.E + 15) / 16), dim3(16 * kSumSlices), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouterParams &p, hipStream_t s) {
  return by_row(p, 64, [&](auto I, auto D) {
    constexpr int i = decltype(I)::value, d = decltype(D)::value;
    const dim3 grid(min(row_groups(p.rows), 1024u));
    if (p.sigmoid) hipLaunchKernelGGL((route_backward_kernel<i, d, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((route_backward_kernel<i, d, false>), grid, dim3(256), 0, s, p);
  });
}

}  // namespace exl3

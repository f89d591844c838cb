// Rows carried to experts and back. Row t has topk choices; choice (t, j) stands
// at position pos(t, j) of the packed rows (pos_of_pair, -1: dropped).
//   permute    xs[pos(t, j)] = x[t]
//   unpermute  out[t] = sum_j w[t, j] y[pos(t, j)]     in fp32, j ascending
//   backward   dy[pos(t, j)] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[pos(t, j)]>
// Nothing is computed that costs time: all three are bound by the bytes they
// move. Work is cut by row t, so that the side that has one row per token (x,
// out, dout) is moved once, and its topk packed rows are whole rows wherever
// they stand. A lane moves 16 bytes (8 values) at a time; a row takes the lanes
// it fills (up to 256), so short rows share a wave. Measured (a large copy: 5.15
// TB/s): 8192 rows of 6144 to 8 places each in bf16, 816 MB, 157 us; 4001 rows
// summed from 8 in fp32, 757 MB, 148; gradients of 8192 rows of 6144 with 4
// choices in fp16, 1007 MB, 206. One row: 3 us, an empty launch 2.5.
#include "common.hpp"
#include "kernels.hpp"

namespace exl3 {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;  // choices whose packed rows are in flight together

// Eight consecutive values as stored (dtype codes: 1 fp16, 2 bf16, 3 fp32).
template <int DT>
struct Eight {
  u32x4 v[DT == 3 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Eight<DT> load_eight(const char *p) {
  Eight<DT> r;
  r.v[0] = *(const u32x4 *)p;
  if constexpr (DT == 3) r.v[1] = *(const u32x4 *)(p + 16);
  return r;
}
template <int DT>
__device__ __forceinline__ void unpack(const Eight<DT> &e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == 3) {
      const uint32_t b = e.v[i >> 2][i & 3];
      f[i] = __builtin_bit_cast(float, b);
    } else {
      const uint16_t b = (uint16_t)(e.v[0][i >> 1] >> (16 * (i & 1)));
      f[i] = DT == 2 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
    }
  }
}
// Results that the L2s cannot hold go past them (stream): 8 x 4 MB. us of one and
// the other: 5284 rows x 13 x 2048 carried in bf16 (281 MB) 51 and 57, 4001 rows
// of 6144 summed from 8 in fp32 149 and 153; at 5 MB no difference.
template <bool STREAM>
__device__ __forceinline__ void store16(void *p, u32x4 v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, (u32x4 *)p);
  else *(u32x4 *)p = v;
}
template <int DT, bool STREAM>
__device__ __forceinline__ void store_eight(char *p, const float (&f)[8]) {
  if constexpr (DT == 3) {
    store16<STREAM>(p, __builtin_bit_cast(u32x4, (f32x4){f[0], f[1], f[2], f[3]}));
    store16<STREAM>(p + 16, __builtin_bit_cast(u32x4, (f32x4){f[4], f[5], f[6], f[7]}));
  } else {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f32x2_to_out16(f[2 * i], f[2 * i + 1], DT == 2);
    store16<STREAM>(p, v);
  }
}
__device__ __forceinline__ float load_weight(const void *w, int dtype, int64_t i) {
  if (dtype == 3) return ((const float *)w)[i];
  const uint16_t b = ((const uint16_t *)w)[i];
  return dtype == 2 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// A block holds blockDim.y rows of blockDim.x lanes; blocks step over groups of
// rows, since one axis of a launch is shorter than the longest call.
__device__ __forceinline__ int64_t row_groups(const MoveParams &p) {
  return ((int64_t)p.rows + blockDim.y - 1) / blockDim.y;
}

// Choices j0 .. j0 + B - 1 of row t: packed positions (-1: dropped, or past topk)
// and weights. All loads are asked for before the first is needed.
template <int B>
__device__ __forceinline__ void load_choices(const MoveParams &p, int64_t t, int j0, int (&q)[B],
                                             float (&w)[B]) {
#pragma unroll
  for (int i = 0; i < B; ++i) q[i] = p.pos[t * p.topk + min(j0 + i, p.topk - 1)];
  if (p.w) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      w[i] = load_weight(p.w, p.w_dtype, t * p.topk + min(j0 + i, p.topk - 1));
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = 1.f;
  }
#pragma unroll
  for (int i = 0; i < B; ++i)
    q[i] = j0 + i < p.topk && (uint32_t)q[i] < (uint32_t)p.pairs ? q[i] : -1;
}

template <bool STREAM>
__global__ void __launch_bounds__(kThreads) permute_kernel(MoveParams p) {
  const int units = (int)((int64_t)p.features * p.esize / 16);
  const int u = blockIdx.y * blockDim.x + threadIdx.x;
  for (int64_t g = blockIdx.x; g < row_groups(p); g += gridDim.x) {
    const int64_t t = g * blockDim.y + threadIdx.y;
    if (t >= p.rows || u >= units) continue;
    const u32x4 v = *(const u32x4 *)((const char *)p.x + t * p.ldx * p.esize + 16 * (int64_t)u);
    for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
      int q[kBatch];
      float w[kBatch];  // none here
      load_choices(p, t, j0, q, w);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (q[i] >= 0)
          store16<STREAM>((char *)p.out + q[i] * p.ldout * p.esize + 16 * (int64_t)u, v);
    }
  }
}

// DY: type of y, DO: of out. B choices at once: their loads are all in flight
// before the first is added (one after the other, 8 choices wait 8 times).
template <int DY, int DO, int B, bool STREAM>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(MoveParams p) {
  constexpr int SY = DY == 3 ? 4 : 2, SO = DO == 3 ? 4 : 2;
  const int u = blockIdx.y * blockDim.x + threadIdx.x;
  for (int64_t g = blockIdx.x; g < row_groups(p); g += gridDim.x) {
    const int64_t t = g * blockDim.y + threadIdx.y;
    if (t >= p.rows || 8 * u >= p.features) continue;
    float acc[8] = {};
    for (int j0 = 0; j0 < p.topk; j0 += B) {
      Eight<DY> raw[B];
      int q[B];
      float w[B];
      load_choices(p, t, j0, q, w);
      int some = -1;  // a row that may be read
      uint32_t taken = 0;  // bit i: choice i takes part (keeping q: 7 registers more)
#pragma unroll
      for (int i = 0; i < B; ++i) {
        taken |= (uint32_t)(q[i] >= 0) << i;
        some = max(some, q[i]);
      }
      if (some < 0) continue;
#pragma unroll
      for (int i = 0; i < B; ++i) {  // a dropped choice reads another's row and is not added
        const int row = q[i] >= 0 ? q[i] : some;
        raw[i] = load_eight<DY>((const char *)p.x + (row * p.ldx + 8 * u) * SY);
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        float y[8];
        unpack<DY>(raw[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = taken >> i & 1 ? fmaf(w[i], y[k], acc[k]) : acc[k];
      }
    }
    store_eight<DO, STREAM>((char *)p.out + (t * p.ldout + 8 * u) * SO, acc);
  }
}

// DY: type of y and dy, DO: of dout. WITH_DW: y is read and dw written. A
// block's lanes cover a whole row, so that <dout, y> needs no second launch; the
// 8 sums of a batch cross the wave together (one after the other, 2 rows of 13
// choices took 13 us instead of 9).
template <int DY, int DO, bool WITH_DW, bool STREAM>
__global__ void __launch_bounds__(kThreads) unpermute_backward_kernel(MoveParams p) {
  constexpr int SY = DY == 3 ? 4 : 2, SO = DO == 3 ? 4 : 2;
  __shared__ float part[kThreads / 64][kBatch];
  const int lanes = blockDim.x;  // a power of two
  const int units = p.features / 8;
  for (int64_t g = blockIdx.x; g < row_groups(p); g += gridDim.x) {
    const int64_t t = g * blockDim.y + threadIdx.y;
    const bool in = t < p.rows;
    for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
      float dot[kBatch] = {};
      int at[kBatch];
      float w[kBatch];
      load_choices(p, in ? t : 0, j0, at, w);
      if (in) {
        for (int u = threadIdx.x; u < units; u += lanes) {
          float d[8];
          unpack<DO>(load_eight<DO>((const char *)p.dout + (t * p.lddout + 8 * u) * SO), d);
          Eight<DY> raw[kBatch];
          if constexpr (WITH_DW) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (at[i] >= 0)
                raw[i] = load_eight<DY>((const char *)p.x + (at[i] * p.ldx + 8 * u) * SY);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (at[i] < 0) continue;
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = w[i] * d[k];
            store_eight<DY, STREAM>((char *)p.out + (at[i] * p.ldout + 8 * u) * SY, o);
            if constexpr (WITH_DW) {
              float y[8];
              unpack<DY>(raw[i], y);
#pragma unroll
              for (int k = 0; k < 8; ++k) dot[i] = fmaf(d[k], y[k], dot[i]);
            }
          }
        }
      }
      if constexpr (WITH_DW) {
#pragma unroll
        for (int s = 32; s; s >>= 1)
          if (s < lanes) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) dot[i] += __shfl_xor(dot[i], s, 64);
          }
        if (lanes > 64) {
          // a row takes all of the block: one value per wave and choice
          __syncthreads();
          if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) part[threadIdx.x >> 6][i] = dot[i];
          }
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            dot[i] = part[0][i];
            for (int v = 1; v < lanes / 64; ++v) dot[i] += part[v][i];
          }
        }
        if (in && threadIdx.x == 0) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (j0 + i >= p.topk) break;
            const int64_t pair = t * p.topk + j0 + i;
            const float v = at[i] >= 0 ? dot[i] : 0.f;
            if (p.dw_dtype == 3) ((float *)p.dw)[pair] = v;
            else ((uint16_t *)p.dw)[pair] = f32_to_out16(v, p.dw_dtype == 2);
          }
        }
      }
    }
  }
}

// Lanes of a row of `units` pieces: the power of two that holds them, at most a
// block; a row of more than a wave takes the block.
struct Shape {
  dim3 grid, block;
};
Shape shape(const MoveParams &p, int units, bool whole_row) {
  int lanes = 1;
  while (lanes < units && lanes < kThreads) lanes *= 2;
  if (lanes > 64) lanes = kThreads;  // the backward pass's barriers are one row's
  const int per = kThreads / lanes;
  const int64_t groups = ((int64_t)p.rows + per - 1) / per;
  Shape s;
  s.block = dim3(lanes, per);
  s.grid = dim3((unsigned)(groups < (1 << 22) ? groups : 1 << 22),
                whole_row ? 1 : (units + lanes - 1) / lanes);
  return s;
}

template <int DY, int DO, int B>
void unpermute_batch(const MoveParams &p, const Shape &s, hipStream_t st) {
  if (p.stream) unpermute_kernel<DY, DO, B, true><<<s.grid, s.block, 0, st>>>(p);
  else unpermute_kernel<DY, DO, B, false><<<s.grid, s.block, 0, st>>>(p);
}
template <int DY, int DO>
void unpermute(const MoveParams &p, const Shape &s, hipStream_t st) {
  if (p.topk == 1) unpermute_batch<DY, DO, 1>(p, s, st);
  else if (p.topk == 2) unpermute_batch<DY, DO, 2>(p, s, st);
  else if (p.topk <= 4) unpermute_batch<DY, DO, 4>(p, s, st);
  else unpermute_batch<DY, DO, kBatch>(p, s, st);
}
template <int DY, int DO, bool WITH_DW>
void backward_of(const MoveParams &p, const Shape &s, hipStream_t st) {
  if (p.stream) unpermute_backward_kernel<DY, DO, WITH_DW, true><<<s.grid, s.block, 0, st>>>(p);
  else unpermute_backward_kernel<DY, DO, WITH_DW, false><<<s.grid, s.block, 0, st>>>(p);
}
template <int DY, int DO>
void backward(const MoveParams &p, const Shape &s, hipStream_t st) {
  if (p.dw) backward_of<DY, DO, true>(p, s, st);
  else backward_of<DY, DO, false>(p, s, st);
}

}  // namespace

hipError_t launch_permute(const MoveParams &p, hipStream_t st) {
  const Shape s = shape(p, (int)((int64_t)p.features * p.esize / 16), false);
  if (p.stream) permute_kernel<true><<<s.grid, s.block, 0, st>>>(p);
  else permute_kernel<false><<<s.grid, s.block, 0, st>>>(p);
  return hipGetLastError();
}

// Calls F<x_dtype, o_dtype>(p, s, st).
#define EXL3_BY_TYPES(F)                                  \
  switch (4 * p.x_dtype + p.o_dtype) {                    \
    case 5: F<1, 1>(p, s, st); break;                     \
    case 6: F<1, 2>(p, s, st); break;                     \
    case 7: F<1, 3>(p, s, st); break;                     \
    case 9: F<2, 1>(p, s, st); break;                     \
    case 10: F<2, 2>(p, s, st); break;                    \
    case 11: F<2, 3>(p, s, st); break;                    \
    case 13: F<3, 1>(p, s, st); break;                    \
    case 14: F<3, 2>(p, s, st); break;                    \
    default: F<3, 3>(p, s, st); break;                    \
  }

hipError_t launch_unpermute(const MoveParams &p, hipStream_t st) {
  const Shape s = shape(p, p.features / 8, false);
  EXL3_BY_TYPES(unpermute)
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const MoveParams &p, hipStream_t st) {
  const Shape s = shape(p, p.features / 8, true);
  EXL3_BY_TYPES(backward)
  return hipGetLastError();
}
#undef EXL3_BY_TYPES

}  // namespace exl3

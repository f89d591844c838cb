// Low-rank adapters of many requests beside a shared projection:
//   out_t = base_t + scale_a (x_t A_a^T) B_a^T,   a = ids[t]
// in two launches. lora_a writes s = x A^T (fp32, R values a row) to the
// workspace; lora_b multiplies s by B^T, adds the base and stores.
//
// Tiles. A tile is up to 64 rows of one adapter. Every workgroup finds its
// tile by itself: rows are taken in windows of 2048, and the workgroup counts
// its window's IDs per adapter, scans the tile counts and collects its rows
// (plan_tile). No launch and no table go before the products, and rows need
// not be sorted. Rows without an adapter are one more bucket, whose tiles
// lora_b copies.
//
// A row's bytes depend on that row alone: the K axis is cut the same way in
// every call (512 inputs to a wave, four waves to a group, groups in
// ascending order), a row is one column of the MFMA tiles whichever row it
// shares them with, and the second product's scaling is per row.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace exl3 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWindow = 2048;     // rows planned together
constexpr int kTileRows = 64;     // rows of a tile
constexpr int kSlice = 512;       // inputs a wave of lora_a sums
constexpr int kGroup = 4 * kSlice;  // inputs a workgroup of lora_a sums
constexpr int kMaxBuckets = 1025;  // EXL3_MAX_ADAPTERS and "none"
constexpr int kBucketsPerThread = (kMaxBuckets + 255) / 256;

struct PlanLds {
  int count[256 * kBucketsPerThread];
  int wave_tiles[4];
  int4 rank[kWindow / 256];  // [chunk] -> per wave
  int rows[kTileRows];
  int found[3];  // bucket (-1: none), tile within it, rows in the bucket
};

// Tile `tile` of window `win`: its adapter (p.adapters: rows without one; -1:
// the window has fewer tiles) and its rows in L.rows[0 .. nrows). Called by
// all 256 threads.
__device__ __forceinline__ int plan_tile(const LoraParams &p, int win, int tile, PlanLds &L,
                                         int &nrows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row0 = win * kWindow;
  const int n = min(p.rows - row0, kWindow);
  const int chunks = (n + 255) >> 8;
  int a[kWindow / 256];
#pragma unroll
  for (int i = 0; i < kWindow / 256; ++i) {
    a[i] = -1;
    if (i * 256 + tid < n) {
      const int64_t id = p.ids_i64 ? ((const int64_t *)p.ids)[row0 + i * 256 + tid]
                                   : (int64_t)((const int32_t *)p.ids)[row0 + i * 256 + tid];
      a[i] = id >= 0 && id < p.adapters ? (int)id : p.adapters;
    }
  }
  for (int b = tid; b <= p.adapters; b += 256) L.count[b] = 0;
  if (tid == 0) L.found[0] = -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWindow / 256; ++i) {
    if (i >= chunks) break;
    // a prompt's rows share one adapter: one addition for the wave
    const int first = __builtin_amdgcn_readfirstlane(a[i]);
    const uint64_t same = __ballot(a[i] == first), valid = __ballot(a[i] >= 0);
    if (same == valid) {
      if (lane == 0 && first >= 0) atomicAdd(&L.count[first], __popcll(same));
    } else if (a[i] >= 0) {
      atomicAdd(&L.count[a[i]], 1);
    }
  }
  __syncthreads();
  // exclusive scan of the buckets' tiles
  int cnt[kBucketsPerThread], mine = 0;
#pragma unroll
  for (int j = 0; j < kBucketsPerThread; ++j) {
    const int b = tid * kBucketsPerThread + j;
    cnt[j] = b <= p.adapters ? L.count[b] : 0;
    mine += (cnt[j] + kTileRows - 1) / kTileRows;
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    incl += lane >= d ? o : 0;
  }
  if (lane == 63) L.wave_tiles[wave] = incl;
  __syncthreads();
  int first_tile = incl - mine;
  for (int w = 0; w < wave; ++w) first_tile += L.wave_tiles[w];
#pragma unroll
  for (int j = 0; j < kBucketsPerThread; ++j) {
    const int t = (cnt[j] + kTileRows - 1) / kTileRows;
    if (tile >= first_tile && tile < first_tile + t) {
      L.found[0] = tid * kBucketsPerThread + j;
      L.found[1] = tile - first_tile;
      L.found[2] = cnt[j];
    }
    first_tile += t;
  }
  __syncthreads();
  const int ad = __builtin_amdgcn_readfirstlane(L.found[0]);
  if (ad < 0) return -1;
  const int skip = __builtin_amdgcn_readfirstlane(L.found[1]) * kTileRows;
  nrows = min(kTileRows, __builtin_amdgcn_readfirstlane(L.found[2]) - skip);
  // the bucket's rows in order, from number `skip` on
#pragma unroll
  for (int i = 0; i < kWindow / 256; ++i) {
    if (i >= chunks) break;
    const uint64_t hit = __ballot(a[i] == ad);
    if (lane == 0) ((int *)&L.rank[i])[wave] = __popcll(hit);
  }
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < kWindow / 256; ++i) {
    if (i >= chunks) break;
    const int4 r = L.rank[i];
    const uint64_t hit = __ballot(a[i] == ad);
    const int at = before + (wave > 0 ? r.x : 0) + (wave > 1 ? r.y : 0) + (wave > 2 ? r.z : 0) +
                   __popcll(hit & ((1ull << lane) - 1)) - skip;
    if (a[i] == ad && at >= 0 && at < kTileRows) L.rows[at] = row0 + i * 256 + tid;
    before += r.x + r.y + r.z + r.w;
  }
  __syncthreads();
  return ad;
}

// Ranks the adapter uses.
__device__ __forceinline__ int used_rank(const LoraParams &p, int ad) {
  return p.ranks ? max(0, min(p.R, uload_i32(p.ranks + ad))) : p.R;
}

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// ------------------------------------------------------------------ x A^T
// One wave: s[r][t] of RT * 16 ranks and TT * 16 rows over one slice. Ranks
// are the MFMA rows, tile rows its columns; both operands are contiguous along
// K, so each lane's 16-byte loads are MFMA operands as they come and nothing
// goes through LDS on the way in.
template <int RT, int TT, bool BF16>
__device__ __forceinline__ void lora_a_tile(const LoraParams &p, const PlanLds &L, int nrows,
                                            int ad, int r0, int ra, int k0, float *red) {
  constexpr int kLd = RT * 16 + 4;
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int k1 = min(k0 + kSlice, p.K);
  f32x4 acc[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  if (k0 < k1) {
    const uint16_t *px[TT], *pa[RT];
    // lanes past the last row or rank repeat it; their sums are not used
#pragma unroll
    for (int j = 0; j < TT; ++j)
      px[j] = p.x + (int64_t)L.rows[min(j * 16 + c, nrows - 1)] * p.ldx + 8 * g;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      pa[i] = p.a + ((int64_t)ad * p.R + min(r0 + i * 16 + c, ra - 1)) * p.K + 8 * g;
    int k = k0;
#pragma unroll 4
    for (; k + 32 <= k1; k += 32) {
      u32x4 x[TT], a[RT];
#pragma unroll
      for (int j = 0; j < TT; ++j) x[j] = *(gu32x4p)(uintptr_t)(px[j] + k);
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i] = *(gu32x4p)(uintptr_t)(pa[i] + k);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = mfma16<BF16>(a[i], x[j], acc[i][j]);
    }
    if (k < k1) {  // K is a multiple of 8: a lane's eight inputs are all there or none is
      const bool ok = k + 8 * g < k1;
      const u32x4 zero = {0, 0, 0, 0};
      u32x4 x[TT], a[RT];
#pragma unroll
      for (int j = 0; j < TT; ++j) x[j] = ok ? *(gu32x4p)(uintptr_t)(px[j] + k) : zero;
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i] = ok ? *(gu32x4p)(uintptr_t)(pa[i] + k) : zero;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = mfma16<BF16>(a[i], x[j], acc[i][j]);
    }
  }
  // lane: ranks 4 g .. 4 g + 3 of row c
  float *to = red + (threadIdx.x >> 6) * kTileRows * kLd;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j)
      *(f32x4 *)(to + (j * 16 + c) * kLd + i * 16 + 4 * g) = acc[i][j];
}

// Workgroup (tile, group and rank chunk, window).
template <int RT, bool BF16>
__global__ void __launch_bounds__(256) lora_a_kernel(LoraParams p, int chunks) {
  constexpr int kLd = RT * 16 + 4;
  __shared__ PlanLds L;
  __shared__ __align__(16) float red[4 * kTileRows * kLd];
  int nrows = 0;
  const int ad = plan_tile(p, blockIdx.z, blockIdx.x, L, nrows);
  if (ad < 0 || ad == p.adapters) return;
  const int group = blockIdx.y / chunks;
  const int r0 = (blockIdx.y - group * chunks) * RT * 16;
  const int ra = used_rank(p, ad);
  if (r0 >= ra) return;
  const int k0 = group * kGroup + wave_id() * kSlice;
  if (nrows <= 16) lora_a_tile<RT, 1, BF16>(p, L, nrows, ad, r0, ra, k0, red);
  else if (nrows <= 32) lora_a_tile<RT, 2, BF16>(p, L, nrows, ad, r0, ra, k0, red);
  else lora_a_tile<RT, 4, BF16>(p, L, nrows, ad, r0, ra, k0, red);
  __syncthreads();
  const int rp = (p.R + 15) & ~15;
  for (int i = threadIdx.x; i < nrows * RT * 4; i += 256) {
    const int t = i / (RT * 4), r = (i - t * RT * 4) * 4;
    const float *from = red + t * kLd + r;
    f32x4 s = *(const f32x4 *)from;
#pragma unroll
    for (int w = 1; w < 4; ++w) s += *(const f32x4 *)(from + w * kTileRows * kLd);
    if (r0 + r < rp)
      *(f32x4 *)(p.part + ((int64_t)group * p.rows + L.rows[t]) * rp + r0 + r) = s;
  }
}

// ------------------------------------------------------------------ s B^T
__device__ __forceinline__ uint16_t to16(float v, bool bf16) {
  return bf16 ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
}
__device__ __forceinline__ float from16(uint16_t b, bool bf16) {
  return bf16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// Eight consecutive columns of a row as fp32, and back.
__device__ __forceinline__ void load8(const void *p, int dtype, int64_t i, float (&v)[8]) {
  if (dtype == 3) {
    const f32x4 lo = *(const f32x4 *)((const float *)p + i);
    const f32x4 hi = *(const f32x4 *)((const float *)p + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = lo[j];
      v[4 + j] = hi[j];
    }
  } else {
    const u32x4 q = *(const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = from16((uint16_t)(q[j >> 1] >> (16 * (j & 1))), dtype == 2);
  }
}
__device__ __forceinline__ void store8(void *p, int dtype, int64_t i, const float (&v)[8]) {
  if (dtype == 3) {
    *(f32x4 *)((float *)p + i) = (f32x4){v[0], v[1], v[2], v[3]};
    *(f32x4 *)((float *)p + i + 4) = (f32x4){v[4], v[5], v[6], v[7]};
  } else {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = (uint32_t)to16(v[2 * j], dtype == 2) |
             ((uint32_t)to16(v[2 * j + 1], dtype == 2) << 16);
    *(u32x4 *)((uint16_t *)p + i) = q;
  }
}

// s as MFMA operands. The matrix cores take 16-bit inputs, so s is written as
// a sum of 16-bit terms, each the rounded rest of the ones before: two fp16
// terms hold 2^-23 of the row's largest entry, two bf16 terms 2^-17 (enough
// below the last bit of a 16-bit output: 2^-8 or 2^-11), three 2^-26 (fp32
// outputs). The row is first scaled by a power of two to [2^13, 2^14), so
// fp16 terms neither overflow nor lose small entries; exact, and undone on the
// fp32 sum. An infinite or NaN entry is its first term alone.
//
// One MFMA takes 32 inner values: the first term of 16 ranks and the second
// term of the same 16, against B given twice. The third term, if any, is a
// second MFMA with zeros in the other half.
template <int RT, int TERMS>
struct SLds {
  static constexpr int kLd = RT * 16 + 8;  // 16-byte rows, spread over the banks
  uint16_t s[TERMS][kTileRows][kLd];
  int e[kTileRows];
};

template <int RT, int TERMS, bool BF16>
__device__ __forceinline__ void load_s(const LoraParams &p, const PlanLds &L, int nrows, int ad,
                                       int ra, int groups, SLds<RT, TERMS> &S) {
  const int t = threadIdx.x >> 2, q = threadIdx.x & 3;
  if (t >= nrows) return;  // columns of the tile past its rows are not used
  const int rp = (p.R + 15) & ~15;
  const float scale = p.scale ? p.scale[ad] : 1.0f;
  const float *from = p.part + (int64_t)L.rows[t] * rp;
  float v[RT][4];
  float big = 0.0f;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int r = 4 * (q + 4 * j);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (r < ra) {  // written by lora_a: whole chunks of 16 ranks below ra
      s = *(const f32x4 *)(from + r);
      for (int i = 1; i < groups; ++i) s += *(const f32x4 *)(from + (int64_t)i * p.rows * rp + r);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[j][u] = r + u < ra ? s[u] * scale : 0.0f;
      big = fmaxf(big, fabsf(v[j][u]));
    }
  }
  big = fmaxf(big, __shfl_xor(big, 1, 64));
  big = fmaxf(big, __shfl_xor(big, 2, 64));
  // fmaxf passes over NaN; the row's finite entries are scaled by the largest
  // (an infinity counts as exponent 255: everything finite stays below 2^14)
  const int e = (int)((__builtin_bit_cast(uint32_t, big) >> 23) & 255u) - 140;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    uint32_t w[TERMS][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float rest = ldexpf(v[j][u], -e);
#pragma unroll
      for (int m = 0; m < TERMS; ++m) {
        const uint16_t b = to16(rest, BF16);
        if (u & 1) w[m][u >> 1] |= (uint32_t)b << 16;
        else w[m][u >> 1] = b;
        rest = fabsf(rest) < __builtin_inff() ? rest - from16(b, BF16) : 0.0f;
      }
    }
#pragma unroll
    for (int m = 0; m < TERMS; ++m)
      *(uint2 *)&S.s[m][t][4 * (q + 4 * j)] = make_uint2(w[m][0], w[m][1]);
  }
  if (q == 0) S.e[t] = e;
}

// B operand: eight ranks from r of output row n (rows of B past N repeat the
// last one). Ranks at or above ra give zero whatever B holds there.
template <bool VEC>
__device__ __forceinline__ u32x4 load_b(const LoraParams &p, const uint16_t *b, int n, int r,
                                        int ra) {
  u32x4 v = {0, 0, 0, 0};
  if (r >= ra) return v;
  const uint16_t *at = b + (int64_t)min(n, p.N - 1) * p.R + r;
  if constexpr (VEC) {  // R is a multiple of 8
    v = *(gu32x4p)(uintptr_t)at;
    if (r + 8 > ra) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r + j >= ra) v[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (r + j < ra) v[j >> 1] |= (uint32_t)at[j] << (16 * (j & 1));
  }
  return v;
}

// One wave: 64 columns from n0 of TT * 16 rows. Columns are the MFMA rows:
// row m of MFMA i is column n0 + 16 (m / 4) + 4 i + m % 4, so that a lane's
// results of the four MFMAs are 16 consecutive columns of one row, and a row's
// 64 columns are one run of 128 bytes (16-bit) or 256 (fp32).
template <int RT, int TT, int TERMS, bool BF16, bool VEC>
__device__ __forceinline__ void lora_b_block(const LoraParams &p, const PlanLds &L, int nrows,
                                             const uint16_t *b, int ra, int n0,
                                             const SLds<RT, TERMS> &S) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int nc = n0 + 16 * (c >> 2) + (c & 3);
  const int rg = 8 * (g & 1);
  f32x4 acc[4][TT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt * 16 >= ra) break;
    u32x4 bv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bv[i] = load_b<VEC>(p, b, nc + 4 * i, rt * 16 + rg, ra);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const u32x4 s = *(const u32x4 *)&S.s[g >> 1][j * 16 + c][rt * 16 + rg];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][j] = mfma16<BF16>(bv[i], s, acc[i][j]);
      if constexpr (TERMS == 3) {
        u32x4 s3 = *(const u32x4 *)&S.s[2][j * 16 + c][rt * 16 + rg];
        if (g >> 1) s3 = (u32x4){0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = mfma16<BF16>(bv[i], s3, acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = j * 16 + c;
    if (t >= nrows) continue;
    const int64_t row = L.rows[t];
    const int e = S.e[t];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + 16 * g + 8 * h;
      if (n >= p.N) continue;
      float v[8];
      if (p.base) load8(p.base, p.base_dtype, row * p.ldbase + n, v);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = ldexpf(acc[2 * h + (u >> 2)][j][u & 3], e) + (p.base ? v[u] : 0.0f);
      store8(p.out, p.out_dtype, row * p.ldout + n, v);
    }
  }
}

// Rows without an adapter: out = base (or zeros).
__device__ __forceinline__ void copy_rows(const LoraParams &p, const PlanLds &L, int nrows, int n0,
                                          int n1) {
  if (p.base == p.out) return;
  const int per_row = (n1 - n0) / 8;
  for (int i = threadIdx.x; i < nrows * per_row; i += 256) {
    const int t = i / per_row, n = n0 + (i - t * per_row) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (p.base) load8(p.base, p.base_dtype, (int64_t)L.rows[t] * p.ldbase + n, v);
    store8(p.out, p.out_dtype, (int64_t)L.rows[t] * p.ldout + n, v);
  }
}

// Workgroup (tile, `cols` columns, window).
template <int RT, int TERMS, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) lora_b_kernel(LoraParams p, int cols, int groups) {
  __shared__ PlanLds L;
  __shared__ __align__(16) SLds<RT, TERMS> S;
  int nrows = 0;
  const int ad = plan_tile(p, blockIdx.z, blockIdx.x, L, nrows);
  if (ad < 0) return;
  const int c0 = blockIdx.y * cols, c1 = min(c0 + cols, p.N);
  const int ra = ad < p.adapters ? used_rank(p, ad) : 0;
  if (ra == 0) {
    copy_rows(p, L, nrows, c0, c1);
    return;
  }
  load_s<RT, TERMS, BF16>(p, L, nrows, ad, ra, groups, S);
  __syncthreads();
  const uint16_t *b = p.b + (int64_t)ad * p.N * p.R;
  for (int n0 = c0 + 64 * wave_id(); n0 < c1; n0 += 256) {
    if (nrows <= 16) lora_b_block<RT, 1, TERMS, BF16, VEC>(p, L, nrows, b, ra, n0, S);
    else if (nrows <= 32) lora_b_block<RT, 2, TERMS, BF16, VEC>(p, L, nrows, b, ra, n0, S);
    else lora_b_block<RT, 4, TERMS, BF16, VEC>(p, L, nrows, b, ra, n0, S);
  }
}

// Tiles a window can have: u buckets in use give at most u + (w - u) / 64.
int tile_slots(const LoraParams &p) {
  const int w = p.rows < kWindow ? p.rows : kWindow;
  const int u = p.adapters + 1 < w ? p.adapters + 1 : w;
  return u + (w - u) / kTileRows;
}
int windows(const LoraParams &p) { return (p.rows + kWindow - 1) / kWindow; }

template <int RT>
void run_a(const LoraParams &p, hipStream_t s) {
  const int chunks = (p.R + RT * 16 - 1) / (RT * 16);
  const dim3 grid(tile_slots(p), lora_groups(p.K) * chunks, windows(p));
  if (p.bf16) hipLaunchKernelGGL((lora_a_kernel<RT, true>), grid, dim3(256), 0, s, p, chunks);
  else hipLaunchKernelGGL((lora_a_kernel<RT, false>), grid, dim3(256), 0, s, p, chunks);
}

template <int RT, int TERMS, bool BF16>
void run_b(const LoraParams &p, hipStream_t s) {
  const int cols = 256;
  const dim3 grid(tile_slots(p), (p.N + cols - 1) / cols, windows(p));
  const int groups = lora_groups(p.K);
  if (p.R % 8 == 0)
    hipLaunchKernelGGL((lora_b_kernel<RT, TERMS, BF16, true>), grid, dim3(256), 0, s, p, cols,
                       groups);
  else
    hipLaunchKernelGGL((lora_b_kernel<RT, TERMS, BF16, false>), grid, dim3(256), 0, s, p, cols,
                       groups);
}

template <int RT>
void run_b(const LoraParams &p, hipStream_t s) {
  if (!p.bf16) run_b<RT, 2, false>(p, s);
  else if (p.out_dtype == 3) run_b<RT, 3, true>(p, s);
  else run_b<RT, 2, true>(p, s);
}

}  // namespace

int lora_groups(int K) { return (K + kGroup - 1) / kGroup; }
int lora_padded_rank(int R) { return (R + 15) & ~15; }

hipError_t launch_lora_a(const LoraParams &p, hipStream_t s) {
  if (p.R <= 16 || p.rows <= 256) run_a<1>(p, s);
  else if (p.R <= 32) run_a<2>(p, s);
  else run_a<4>(p, s);
  return hipGetLastError();
}

hipError_t launch_lora_b(const LoraParams &p, hipStream_t s) {
  if (p.R <= 16) run_b<1>(p, s);
  else if (p.R <= 32) run_b<2>(p, s);
  else if (p.R <= 64) run_b<4>(p, s);
  else run_b<8>(p, s);
  return hipGetLastError();
}

}  // namespace exl3

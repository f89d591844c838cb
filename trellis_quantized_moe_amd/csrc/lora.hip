// Low-rank adapters of many requests beside a shared projection:
//   out_t = base_t + scale_a (x_t A_a^T) B_a^T,   a = ids[t]
// in two launches. lora_a writes s = x A^T (fp32, R values a row) to the
// workspace; lora_b multiplies s by B^T, adds the base and stores.
//
// Tiles. A tile is up to 64 rows of one adapter. Every workgroup of lora_a
// finds its tile by itself: rows are taken in windows of 2048, and the
// workgroup counts its window's IDs per adapter, scans the tile counts and
// collects its rows (plan_tile), so that no planning launch goes before it and
// rows need not be sorted. The first workgroup of a tile leaves it in the
// workspace for lora_b. Rows without an adapter are one more bucket, whose
// tiles lora_b copies.
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
  // lanes past the window read its last ID and drop it: loads without a branch
  // around them are all in flight together
  int a[kWindow / 256];
  if (p.ids_i64) {
    int64_t id[kWindow / 256];
#pragma unroll
    for (int i = 0; i < kWindow / 256; ++i)
      id[i] = ((const int64_t *)p.ids)[row0 + min(i * 256 + tid, n - 1)];
#pragma unroll
    for (int i = 0; i < kWindow / 256; ++i)
      a[i] = id[i] >= 0 && id[i] < p.adapters ? (int)id[i] : p.adapters;
  } else {
#pragma unroll
    for (int i = 0; i < kWindow / 256; ++i)
      a[i] = ((const int32_t *)p.ids)[row0 + min(i * 256 + tid, n - 1)];
#pragma unroll
    for (int i = 0; i < kWindow / 256; ++i)
      a[i] = (uint32_t)a[i] < (uint32_t)p.adapters ? a[i] : p.adapters;
  }
#pragma unroll
  for (int i = 0; i < kWindow / 256; ++i) a[i] = i * 256 + tid < n ? a[i] : -1;
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
    // kStep K steps of 32 inputs are loaded while the kStep before them go
    // through the matrix units
    constexpr int kStep = TT + RT <= 5 ? 4 : 2;
    u32x4 x[2][kStep][TT], a[2][kStep][RT];
    auto fetch = [&](int buf, int k) {
#pragma unroll
      for (int u = 0; u < kStep; ++u) {
#pragma unroll
        for (int j = 0; j < TT; ++j) x[buf][u][j] = *(gu32x4p)(uintptr_t)(px[j] + k + 32 * u);
#pragma unroll
        for (int i = 0; i < RT; ++i) a[buf][u][i] = *(gu32x4p)(uintptr_t)(pa[i] + k + 32 * u);
      }
    };
    auto multiply = [&](int buf) {
#pragma unroll
      for (int u = 0; u < kStep; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < TT; ++j)
            acc[i][j] = mfma16<BF16>(a[buf][u][i], x[buf][u][j], acc[i][j]);
    };
    int k = k0;
    if (k1 - k0 == kSlice) {
      fetch(0, k0);
#pragma unroll
      for (int n = 0; n < kSlice / (32 * kStep); ++n) {
        if (n + 1 < kSlice / (32 * kStep)) fetch((n + 1) & 1, k0 + (n + 1) * 32 * kStep);
        __builtin_amdgcn_sched_barrier(0);
        multiply(n & 1);
      }
      k = k1;
    }
    for (; k + 32 <= k1; k += 32) {  // the last slice of a K that is no multiple of kSlice
      u32x4 xs[TT], as[RT];
#pragma unroll
      for (int j = 0; j < TT; ++j) xs[j] = *(gu32x4p)(uintptr_t)(px[j] + k);
#pragma unroll
      for (int i = 0; i < RT; ++i) as[i] = *(gu32x4p)(uintptr_t)(pa[i] + k);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = mfma16<BF16>(as[i], xs[j], acc[i][j]);
    }
    if (k < k1) {  // K is a multiple of 8: a lane's eight inputs are all there or none is
      const bool ok = k + 8 * g < k1;
      const u32x4 zero = {0, 0, 0, 0};
      u32x4 xs[TT], as[RT];
#pragma unroll
      for (int j = 0; j < TT; ++j) xs[j] = ok ? *(gu32x4p)(uintptr_t)(px[j] + k) : zero;
#pragma unroll
      for (int i = 0; i < RT; ++i) as[i] = ok ? *(gu32x4p)(uintptr_t)(pa[i] + k) : zero;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = mfma16<BF16>(as[i], xs[j], acc[i][j]);
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
  if (blockIdx.y == 0) {
    LoraTile *tile = p.tiles + (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) {
      tile->adapter = ad;
      tile->nrows = nrows;
    }
    if (threadIdx.x < kTileRows) tile->rows[threadIdx.x] = L.rows[min((int)threadIdx.x, max(nrows - 1, 0))];
  }
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

// Eight consecutive columns of a row: as loaded (fp32 takes two registers of
// four, a 16-bit type one), as fp32, and stored.
struct Raw8 {
  u32x4 lo, hi;
};
__device__ __forceinline__ void load8(const void *p, int dtype, int64_t i, Raw8 &r) {
  if (dtype == 3) {
    r.lo = *(const u32x4 *)((const float *)p + i);
    r.hi = *(const u32x4 *)((const float *)p + i + 4);
  } else {
    r.lo = *(const u32x4 *)((const uint16_t *)p + i);
  }
}
__device__ __forceinline__ void widen8(const Raw8 &r, int dtype, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (dtype == 3) {
      const uint32_t w = j < 4 ? r.lo[j & 3] : r.hi[j & 3];
      v[j] = __builtin_bit_cast(float, w);
    } else {
      const uint32_t w = r.lo[j >> 1];
      v[j] = from16((uint16_t)(w >> (16 * (j & 1))), dtype == 2);
    }
  }
}
__device__ __forceinline__ void store8(void *p, int dtype, int64_t i, const float (&v)[8]) {
  if (dtype == 3) {
    *(f32x4 *)((float *)p + i) = (f32x4){v[0], v[1], v[2], v[3]};
    *(f32x4 *)((float *)p + i + 4) = (f32x4){v[4], v[5], v[6], v[7]};
  } else {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = f32x2_to_out16(v[2 * j], v[2 * j + 1], dtype == 2);
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
__device__ __forceinline__ void load_s(const LoraParams &p, const LoraTile *tile, int nrows,
                                       int ad, int ra, int groups, SLds<RT, TERMS> &S) {
  const int t = threadIdx.x >> 2, q = threadIdx.x & 3;
  if (t >= nrows) return;  // columns of the tile past its rows are not used
  const int rp = (p.R + 15) & ~15;
  const float scale = p.scale ? p.scale[ad] : 1.0f;
  const float *from = p.part + (int64_t)tile->rows[t] * rp;
  // kParts groups' sums at a time are asked for together; groups and ranks that
  // are not there repeat one that is, and are not added
  constexpr int kParts = RT <= 2 ? 4 : RT == 4 ? 2 : 1;
  f32x4 sum[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) sum[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < groups; i0 += kParts) {
    f32x4 part[kParts][RT];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int r = 4 * (q + 4 * j);
        part[i][j] = *(const f32x4 *)(from + (int64_t)min(i0 + i, groups - 1) * p.rows * rp +
                                      (r < ra ? r : 0));
      }
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j)
        if (i0 + i < groups) sum[j] = i0 + i == 0 ? part[i][j] : sum[j] + part[i][j];
  }
  float v[RT][4];
  float big = 0.0f;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int r = 4 * (q + 4 * j);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[j][u] = r + u < ra ? sum[j][u] * scale : 0.0f;
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
// last one). Ranks at or above ra give zero whatever B holds there. With R a
// multiple of 8 every load is one of 16 bytes, without a branch around it: one
// that lies past R is moved inside and its values dropped.
template <int RT>
__device__ __forceinline__ void load_b(const LoraParams &p, const uint16_t *b, int n, int rg,
                                       int ra, u32x4 (&v)[RT]) {
  const uint16_t *at = b + (int64_t)min(n, p.N - 1) * p.R;
  if (p.R % 8 == 0) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      v[rt] = *(gu32x4p)(uintptr_t)(at + min(rt * 16 + rg, p.R - 8));
  } else {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      v[rt] = (u32x4){0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = rt * 16 + rg + j;
        if (r < ra) v[rt][j >> 1] |= (uint32_t)at[r] << (16 * (j & 1));
      }
    }
  }
}
template <int RT>
__device__ __forceinline__ void mask_b(int rg, int ra, u32x4 (&v)[RT]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (rt * 16 + rg + j >= ra) v[rt][j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
}

// One wave: 64 columns from n0 of TT * 16 rows. Columns are the MFMA rows:
// row m of MFMA i is column n0 + 32 (i / 2) + 8 (m / 4) + 4 (i % 2) + m % 4,
// so that a lane's results of MFMAs 2 h and 2 h + 1 are 8 consecutive columns
// of one row, and the four lanes of a row 32: one run of 64 bytes (16-bit) or
// 128 (fp32) to each load and store. The base is asked for first and B next;
// both are on their way together.
template <int RT, int TT, int TERMS, bool BF16>
__device__ __forceinline__ void lora_b_block(const LoraParams &p, const int (&rows)[4], int nrows,
                                             const uint16_t *b, int ra, int n0,
                                             const SLds<RT, TERMS> &S) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int rg = 8 * (g & 1);
  const int nl = n0 + 8 * g;  // this lane's first column
  Raw8 base[TT][2];
  if (p.base) {
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)  // columns past N repeat the last ones
        load8(p.base, p.base_dtype, (int64_t)rows[j] * p.ldbase + min(nl + 32 * h, p.N - 8),
              base[j][h]);
  }
  f32x4 acc[4][TT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u32x4 bv[RT];
    load_b<RT>(p, b, n0 + 32 * (i >> 1) + 8 * (c >> 2) + 4 * (i & 1) + (c & 3), rg, ra, bv);
    if (ra != RT * 16) mask_b<RT>(rg, ra, bv);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const u32x4 s = *(const u32x4 *)&S.s[g >> 1][j * 16 + c][rt * 16 + rg];
        acc[i][j] = mfma16<BF16>(bv[rt], s, acc[i][j]);
        if constexpr (TERMS == 3) {
          u32x4 s3 = *(const u32x4 *)&S.s[2][j * 16 + c][rt * 16 + rg];
          if (g >> 1) s3 = (u32x4){0, 0, 0, 0};
          acc[i][j] = mfma16<BF16>(bv[rt], s3, acc[i][j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = j * 16 + c;
    if (t >= nrows) continue;
    const int e = S.e[t];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (p.base) widen8(base[j][h], p.base_dtype, v);
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] += ldexpf(acc[2 * h + (u >> 2)][j][u & 3], e);
      const int n = nl + 32 * h;
      if (n < p.N) store8(p.out, p.out_dtype, (int64_t)rows[j] * p.ldout + n, v);
    }
  }
}

// Rows without an adapter: out = base (or zeros).
__device__ __forceinline__ void copy_rows(const LoraParams &p, const LoraTile *tile, int nrows,
                                          int n0, int n1) {
  if (p.base == p.out) return;
  const int per_row = (n1 - n0) / 8;
  for (int i = threadIdx.x; i < nrows * per_row; i += 256) {
    const int t = i / per_row, n = n0 + (i - t * per_row) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (p.base) {
      Raw8 r;
      load8(p.base, p.base_dtype, (int64_t)tile->rows[t] * p.ldbase + n, r);
      widen8(r, p.base_dtype, v);
    }
    store8(p.out, p.out_dtype, (int64_t)tile->rows[t] * p.ldout + n, v);
  }
}

// Workgroup (tile, `cols` columns, window).
template <int RT, int TERMS, bool BF16>
__global__ void __launch_bounds__(256) lora_b_kernel(LoraParams p, int cols, int groups) {
  __shared__ __align__(16) SLds<RT, TERMS> S;
  const LoraTile *tile = p.tiles + (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  const int ad = uload_i32(&tile->adapter), nrows = uload_i32(&tile->nrows);
  if (ad < 0) return;
  const int c0 = blockIdx.y * cols, c1 = min(c0 + cols, p.N);
  const int ra = ad < p.adapters ? used_rank(p, ad) : 0;
  if (ra == 0) {
    copy_rows(p, tile, nrows, c0, c1);
    return;
  }
  int rows[4];  // tile row j * 16 + lane % 16; past the end the last row again
#pragma unroll
  for (int j = 0; j < 4; ++j) rows[j] = tile->rows[j * 16 + (threadIdx.x & 15)];
  load_s<RT, TERMS, BF16>(p, tile, nrows, ad, ra, groups, S);
  __syncthreads();
  const uint16_t *b = p.b + (int64_t)ad * p.N * p.R;
  for (int n0 = c0 + 64 * wave_id(); n0 < c1; n0 += 256) {
    if (nrows <= 16) lora_b_block<RT, 1, TERMS, BF16>(p, rows, nrows, b, ra, n0, S);
    else if (nrows <= 32) lora_b_block<RT, 2, TERMS, BF16>(p, rows, nrows, b, ra, n0, S);
    else lora_b_block<RT, 4, TERMS, BF16>(p, rows, nrows, b, ra, n0, S);
  }
}

int windows(int rows) { return (rows + kWindow - 1) / kWindow; }
// Tiles a window can have: u buckets in use give at most u + (w - u) / 64.
int tile_slots(int rows, int adapters) {
  const int w = rows < kWindow ? rows : kWindow;
  const int u = adapters + 1 < w ? adapters + 1 : w;
  return u + (w - u) / kTileRows;
}

template <int RT>
void run_a(const LoraParams &p, hipStream_t s) {
  const int chunks = (p.R + RT * 16 - 1) / (RT * 16);
  const dim3 grid(tile_slots(p.rows, p.adapters), lora_groups(p.K) * chunks, windows(p.rows));
  if (p.bf16) hipLaunchKernelGGL((lora_a_kernel<RT, true>), grid, dim3(256), 0, s, p, chunks);
  else hipLaunchKernelGGL((lora_a_kernel<RT, false>), grid, dim3(256), 0, s, p, chunks);
}

template <int RT, int TERMS, bool BF16>
void run_b(const LoraParams &p, hipStream_t s) {
  const int cols = 256;
  const dim3 grid(tile_slots(p.rows, p.adapters), (p.N + cols - 1) / cols, windows(p.rows));
  hipLaunchKernelGGL((lora_b_kernel<RT, TERMS, BF16>), grid, dim3(256), 0, s, p, cols,
                     lora_groups(p.K));
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
size_t lora_tiles(int rows, int adapters) {
  return (size_t)windows(rows) * tile_slots(rows, adapters);
}

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

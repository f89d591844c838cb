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
// every call (256 inputs to a wave, eight waves to a group, groups in
// ascending order), a row is one column of the MFMA tiles whichever row it
// shares them with, and the second product's scaling is per row.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace exl3 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWindow = 2048;       // rows planned together
constexpr int kTileRows = 64;       // rows of a tile
constexpr int kWavesA = 8;          // waves of a workgroup of lora_a
constexpr int kThreadsA = 64 * kWavesA;
constexpr int kSlice = 256;         // inputs a wave of lora_a sums
constexpr int kGroup = kWavesA * kSlice;  // inputs a workgroup of lora_a sums
constexpr int kMaxBuckets = 1025;  // EXL3_MAX_ADAPTERS and "none"
constexpr int kChunks = kWindow / kThreadsA;  // IDs of a thread

struct PlanLds {
  int count[kMaxBuckets];
  int hits[kChunks * kWavesA];  // rows of the bucket, by chunk and wave
  int rows[kTileRows];
};

// Inclusive sum over the lanes of a wave: shifts inside the 16-lane rows, then
// the rows' last lanes to the rows after them.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}

// Tile `tile` of window `win`: its adapter (p.adapters: rows without one; -1:
// the window has fewer tiles) and its rows in L.rows[0 .. nrows). Called by
// all kThreadsA threads.
__device__ __forceinline__ int plan_tile(const LoraParams &p, int win, int tile, PlanLds &L,
                                         int &nrows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int row0 = win * kWindow;
  const int n = min(p.rows - row0, kWindow);
  // lanes past the window read its last ID and drop it: loads without a branch
  // around them are all in flight together
  int a[kChunks];
  if (p.ids_i64) {
    int64_t id[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      id[i] = ((const int64_t *)p.ids)[row0 + min(i * kThreadsA + tid, n - 1)];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      a[i] = id[i] >= 0 && id[i] < p.adapters ? (int)id[i] : p.adapters;
  } else {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      a[i] = ((const int32_t *)p.ids)[row0 + min(i * kThreadsA + tid, n - 1)];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      a[i] = (uint32_t)a[i] < (uint32_t)p.adapters ? a[i] : p.adapters;
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) a[i] = i * kThreadsA + tid < n ? a[i] : -1;
  for (int b = tid; b <= p.adapters; b += kThreadsA) L.count[b] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    // a prompt's rows share one adapter: one addition for the wave
    const int first = __builtin_amdgcn_readfirstlane(a[i]);
    const uint64_t same = __ballot(a[i] == first), valid = __ballot(a[i] >= 0);
    if (same == valid) {
      if (lane == 0) atomicAdd(&L.count[first], __popcll(same));
    } else if (a[i] >= 0) {
      atomicAdd(&L.count[a[i]], 1);
    }
  }
  __syncthreads();
  // the bucket the tile falls into; every wave looks for itself
  int ad = -1, skip = 0, size = 0;
  for (int b0 = 0, before = 0; b0 <= p.adapters; b0 += 64) {
    const int rows = b0 + lane <= p.adapters ? L.count[b0 + lane] : 0;
    const int tiles = (rows + kTileRows - 1) / kTileRows;
    const int end = before + wave_scan(tiles);
    const uint64_t past = __ballot(end > tile);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      ad = b0 + l;
      skip = (tile - (__shfl(end, l, 64) - __shfl(tiles, l, 64))) * kTileRows;
      size = __shfl(rows, l, 64);
      break;
    }
    before = __shfl(end, 63, 64);
  }
  ad = __builtin_amdgcn_readfirstlane(ad);
  if (ad < 0) return -1;
  skip = __builtin_amdgcn_readfirstlane(skip);
  nrows = min(kTileRows, __builtin_amdgcn_readfirstlane(size) - skip);
  // the bucket's rows in order, from number `skip` on
  uint64_t hit[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    hit[i] = __ballot(a[i] == ad);
    if (lane == 0) L.hits[i * kWavesA + wave] = __popcll(hit[i]);
  }
  __syncthreads();
  // rows before this wave's of each chunk: lane i of the first kChunks *
  // kWavesA lanes sums up to entry i
  static_assert(kChunks * kWavesA <= 64, "one entry to a lane");
  const int own = lane < kChunks * kWavesA ? L.hits[lane] : 0;
  const int before = wave_scan(own) - own;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int at = __builtin_amdgcn_readlane(before, i * kWavesA + wave) +
                   __popcll(hit[i] & ((1ull << lane) - 1)) - skip;
    if (a[i] == ad && at >= 0 && at < kTileRows) L.rows[at] = row0 + i * kThreadsA + tid;
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
    // the loads of kBuf - 1 K steps of 32 inputs are on their way while one goes
    // through the matrix units: about 120 registers, two waves to a SIMD
    constexpr int kSteps = kSlice / 32;
    constexpr int kWant = 30 / (TT + RT);
    constexpr int kBuf = kWant < 3 ? 3 : kWant < kSteps ? kWant : kSteps;
    u32x4 x[kBuf][TT], a[kBuf][RT];
    auto fetch = [&](int n) {
#pragma unroll
      for (int j = 0; j < TT; ++j)
        x[n % kBuf][j] = *(gu32x4p)(uintptr_t)(px[j] + k0 + 32 * n);
#pragma unroll
      for (int i = 0; i < RT; ++i)
        a[n % kBuf][i] = *(gu32x4p)(uintptr_t)(pa[i] + k0 + 32 * n);
    };
    int k = k0;
    if (k1 - k0 == kSlice) {
#pragma unroll
      for (int n = 0; n < kBuf - 1; ++n) fetch(n);
#pragma unroll
      for (int n = 0; n < kSteps; ++n) {
        if (n + kBuf - 1 < kSteps) fetch(n + kBuf - 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < TT; ++j)
            acc[i][j] = mfma16<BF16>(a[n % kBuf][i], x[n % kBuf][j], acc[i][j]);
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
  // lane: ranks 4 g .. 4 g + 3 of row c. Waves 4 .. 7 leave theirs in LDS, waves
  // 0 .. 3 add their own; the kernel adds those four.
  const int wave = wave_id();
  float *at = red + (wave & 3) * kTileRows * kLd;
  if (wave >= 4) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j)
        *(f32x4 *)(at + (j * 16 + c) * kLd + i * 16 + 4 * g) = acc[i][j];
  }
  __syncthreads();
  if (wave < 4) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        f32x4 *to = (f32x4 *)(at + (j * 16 + c) * kLd + i * 16 + 4 * g);
        *to = acc[i][j] + *to;
      }
  }
  __syncthreads();
}

// Workgroup (tile, group and rank chunk, window).
template <int RT, bool BF16>
__global__ void __launch_bounds__(kThreadsA) lora_a_kernel(LoraParams p, int chunks) {
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
  const int rp = (p.R + 15) & ~15;
  for (int i = threadIdx.x; i < nrows * RT * 4; i += kThreadsA) {
    const int t = i / (RT * 4), r = (i - t * RT * 4) * 4;
    const float *from = red + t * kLd + r;
    constexpr int w = kTileRows * kLd;
    const f32x4 s = (*(const f32x4 *)from + *(const f32x4 *)(from + w)) +
                    (*(const f32x4 *)(from + 2 * w) + *(const f32x4 *)(from + 3 * w));
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

// Eight consecutive columns of a row: base as loaded (BASE: 0 none, 2 a 16-bit
// type, 4 fp32; the size is a template argument so that no branch stands
// between the loads), as fp32, and stored.
template <int BASE>
struct Raw8 {
  u32x4 v[BASE == 4 ? 2 : 1];
};
template <int BASE>
__device__ __forceinline__ void load8(const void *p, int64_t i, Raw8<BASE> &r) {
  if constexpr (BASE == 4) {
    r.v[0] = *(gu32x4p)(uintptr_t)((const float *)p + i);
    r.v[1] = *(gu32x4p)(uintptr_t)((const float *)p + i + 4);
  } else if constexpr (BASE == 2) {
    r.v[0] = *(gu32x4p)(uintptr_t)((const uint16_t *)p + i);
  }
}
template <int BASE>
__device__ __forceinline__ void widen8(const Raw8<BASE> &r, int dtype, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BASE == 4) {
      const uint32_t w = r.v[j >> 2][j & 3];
      v[j] = __builtin_bit_cast(float, w);
    } else if constexpr (BASE == 2) {
      const uint32_t w = r.v[0][j >> 1];
      v[j] = from16((uint16_t)(w >> (16 * (j & 1))), dtype == 2);
    } else {
      v[j] = 0.0f;
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

// Ranks go through the second product in chunks of eight. Chunk c holds ranks
// 8 c .. 8 c + 7; where R is no multiple of 8 (and at least 8), the last one
// starts at R - 8 instead, so that its load stays inside B's row, and leaves
// out the ranks that the chunk before it has. Loads of 16 bytes need no
// alignment here. First rank of a chunk:
__device__ __forceinline__ int chunk_start(int R, int c) {
  return R >= 8 ? min(8 * c, R - 8) : 8 * c;
}
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef const u32x4 __attribute__((address_space(1), aligned(2))) *gu32x4p_a2;

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
template <int RT>
struct SLds {
  static constexpr int kLd = RT * 16 + 8;  // 16-byte rows, spread over the banks
  uint16_t s[3][kTileRows][kLd];
  int e[kTileRows];
};

template <int RT, bool BF16>
__device__ __forceinline__ void load_s(const LoraParams &p, const LoraTile *tile, int nrows,
                                       int ad, int ra, int groups, SLds<RT> &S) {
  const int t = threadIdx.x >> 2, q = threadIdx.x & 3;
  if (t >= nrows) return;  // columns of the tile past its rows are not used
  const int rp = (p.R + 15) & ~15;
  const float scale = p.scale ? p.scale[ad] : 1.0f;
  const float *from = p.part + (int64_t)tile->rows[t] * rp;
  // slots 4 (q + 4 j) .. + 3 hold ranks r0[j] .. + 3, those from lo[j] on
  int r0[RT], lo[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int slot = 4 * (q + 4 * j);
    lo[j] = slot & ~7;
    r0[j] = chunk_start(p.R, slot >> 3) + (slot & 4);
  }
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
      for (int j = 0; j < RT; ++j)
        part[i][j] = *(const f32x4_a4 *)(from + (int64_t)min(i0 + i, groups - 1) * p.rows * rp +
                                         (lo[j] < ra ? r0[j] : 0));
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j)
        if (i0 + i < groups) sum[j] = i0 + i == 0 ? part[i][j] : sum[j] + part[i][j];
  }
  float v[RT][4];
  float big = 0.0f;
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0[j] + u;
      v[j][u] = r >= lo[j] && r < ra ? sum[j][u] * scale : 0.0f;
      big = fmaxf(big, fabsf(v[j][u]));
    }
  big = fmaxf(big, __shfl_xor(big, 1, 64));
  big = fmaxf(big, __shfl_xor(big, 2, 64));
  // fmaxf passes over NaN; the row's finite entries are scaled by the largest
  // (an infinity counts as exponent 255: everything finite stays below 2^14)
  const int e = (int)((__builtin_bit_cast(uint32_t, big) >> 23) & 255u) - 140;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    uint32_t w[3][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float rest = ldexpf(v[j][u], -e);
#pragma unroll
      for (int m = 0; m < (BF16 ? 3 : 2); ++m) {
        const uint16_t b = to16(rest, BF16);
        if (u & 1) w[m][u >> 1] |= (uint32_t)b << 16;
        else w[m][u >> 1] = b;
        rest = fabsf(rest) < __builtin_inff() ? rest - from16(b, BF16) : 0.0f;
      }
    }
#pragma unroll
    for (int m = 0; m < (BF16 ? 3 : 2); ++m)
      *(uint2 *)&S.s[m][t][4 * (q + 4 * j)] = make_uint2(w[m][0], w[m][1]);
  }
  if (q == 0) S.e[t] = e;
}

// What a wave loads for 32 columns of TT * 16 rows: the base and B. Columns
// are the MFMA rows: row m of MFMA i is column n0 + 8 (m / 4) + 4 i + m % 4, so
// that a lane's results of both MFMAs are 8 consecutive columns of one row, and
// the four lanes of a row 32: one run of 64 bytes (16-bit) or 128 (fp32).
template <int RT, int TT, int BASE>
struct Columns {
  Raw8<BASE> base[TT];
  u32x4 b[2][RT];
};

// WIDE: R >= 8. Below that B's rows are shorter than a load and are read one by
// one. Columns past N repeat the last ones, so no branch stands before a load.
template <int RT, int TT, int BASE, bool WIDE>
__device__ __forceinline__ void load_columns(const LoraParams &p, const int (&rows)[4],
                                             const uint16_t *b, int n0, Columns<RT, TT, BASE> &u) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
#pragma unroll
  for (int j = 0; j < TT; ++j)
    load8<BASE>(p.base, (int64_t)rows[j] * p.ldbase + min(n0 + 8 * g, p.N - 8), u.base[j]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = min(n0 + 8 * (c >> 2) + 4 * i + (c & 3), p.N - 1);
    const uint16_t *at = b + (int64_t)n * p.R;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if constexpr (WIDE) {
        u.b[i][rt] = *(gu32x4p_a2)(uintptr_t)(at + chunk_start(p.R, 2 * rt + (g & 1)));
      } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = at[min(j, p.R - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j) u.b[i][rt][j] = w[2 * j] | (w[2 * j + 1] << 16);
      }
    }
  }
}

// The rest of the work on those columns. mask: some ranks of a chunk are not
// used or not its own; their B counts as zero whatever it holds (0 * NaN).
template <int RT, int TT, bool BF16, int BASE>
__device__ __forceinline__ void use_columns(const LoraParams &p, const int (&rows)[4], int nrows,
                                            int ra, bool mask, bool three, int n0,
                                            Columns<RT, TT, BASE> &u, const SLds<RT> &S) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  if (mask) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int lo = 8 * (2 * rt + (g & 1)), r = chunk_start(p.R, 2 * rt + (g & 1));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool off = r + j < lo || r + j >= ra;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (off) u.b[i][rt][j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
      }
    }
  }
  f32x4 acc[2][TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    acc[0][j] = acc[1][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int at = rt * 16 + 8 * (g & 1);
      const u32x4 s = *(const u32x4 *)&S.s[g >> 1][j * 16 + c][at];
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][j] = mfma16<BF16>(u.b[i][rt], s, acc[i][j]);
      if (BF16 && three) {
        u32x4 s3 = *(const u32x4 *)&S.s[2][j * 16 + c][at];
        if (g >> 1) s3 = (u32x4){0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i][j] = mfma16<BF16>(u.b[i][rt], s3, acc[i][j]);
      }
    }
  }
  const int n = n0 + 8 * g;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = j * 16 + c;
    float v[8];
    widen8<BASE>(u.base[j], p.base_dtype, v);
    if (t >= nrows || n >= p.N) continue;
    const int e = S.e[t];
#pragma unroll
    for (int w = 0; w < 8; ++w) v[w] += ldexpf(acc[w >> 2][j][w & 3], e);
    store8(p.out, p.out_dtype, (int64_t)rows[j] * p.ldout + n, v);
  }
}

// A wave's columns n0 .. n1 - 1 of TT * 16 rows, 32 at a time: the next 32 are
// on their way while the present ones are multiplied and stored, and the first
// are asked for before s is.
template <int RT, int TT, bool BF16, int BASE, bool WIDE>
__device__ __forceinline__ void lora_b_tile(const LoraParams &p, const LoraTile *tile, int nrows,
                                            int ad, int ra, int groups, int n0, int n1,
                                            SLds<RT> &S) {
  int rows[4];  // tile row j * 16 + lane % 16; past the end the last row again
#pragma unroll
  for (int j = 0; j < TT; ++j) rows[j] = tile->rows[j * 16 + (threadIdx.x & 15)];
  const uint16_t *b = p.b + (int64_t)ad * p.N * p.R;
  const bool mask = ra != RT * 16, three = p.out_dtype == 3;
  Columns<RT, TT, BASE> u[2];
  load_columns<RT, TT, BASE, WIDE>(p, rows, b, n0, u[0]);
  load_s<RT, BF16>(p, tile, nrows, ad, ra, groups, S);
  __syncthreads();
  for (int n = n0; n < n1; n += 64) {
    load_columns<RT, TT, BASE, WIDE>(p, rows, b, n + 32, u[1]);
    __builtin_amdgcn_sched_barrier(0);
    use_columns<RT, TT, BF16, BASE>(p, rows, nrows, ra, mask, three, n, u[0], S);
    if (n + 32 >= n1) break;
    load_columns<RT, TT, BASE, WIDE>(p, rows, b, n + 64, u[0]);
    __builtin_amdgcn_sched_barrier(0);
    use_columns<RT, TT, BF16, BASE>(p, rows, nrows, ra, mask, three, n + 32, u[1], S);
  }
}

// Rows without an adapter: out = base (or zeros), 16 loads of a thread together.
template <int BASE>
__device__ __forceinline__ void copy_rows(const LoraParams &p, const LoraTile *tile, int nrows,
                                          int n0, int n1) {
  if (p.base == p.out || n0 >= n1) return;
  const int per_row = (n1 - n0) / 8, total = nrows * per_row;
  for (int i0 = threadIdx.x; i0 < total; i0 += 256 * 8) {
    Raw8<BASE> r[8];
    int64_t row[8];
    int n[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = min(i0 + 256 * u, total - 1), t = i / per_row;
      row[u] = tile->rows[t];
      n[u] = n0 + (i - t * per_row) * 8;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) load8<BASE>(p.base, row[u] * p.ldbase + n[u], r[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float v[8];
      widen8<BASE>(r[u], p.base_dtype, v);
      if (i0 + 256 * u < total) store8(p.out, p.out_dtype, row[u] * p.ldout + n[u], v);
    }
  }
}

// Workgroup (tile, 4 * per_wave columns, window).
template <int RT, bool BF16, int BASE, bool WIDE>
__global__ void __launch_bounds__(256) lora_b_kernel(LoraParams p, int per_wave, int groups) {
  __shared__ __align__(16) SLds<RT> S;
  const LoraTile *tile = p.tiles + (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  const int ad = uload_i32(&tile->adapter), nrows = uload_i32(&tile->nrows);
  if (ad < 0) return;
  const int c0 = blockIdx.y * 4 * per_wave;
  const int ra = ad < p.adapters ? used_rank(p, ad) : 0;
  if (ra == 0) {
    copy_rows<BASE>(p, tile, nrows, c0, min(c0 + 4 * per_wave, p.N));
    return;
  }
  const int n0 = c0 + per_wave * wave_id(), n1 = min(n0 + per_wave, p.N);
  if (nrows <= 16)
    lora_b_tile<RT, 1, BF16, BASE, WIDE>(p, tile, nrows, ad, ra, groups, n0, n1, S);
  else if (nrows <= 32)
    lora_b_tile<RT, 2, BF16, BASE, WIDE>(p, tile, nrows, ad, ra, groups, n0, n1, S);
  else
    lora_b_tile<RT, 4, BF16, BASE, WIDE>(p, tile, nrows, ad, ra, groups, n0, n1, S);
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
  if (p.bf16) hipLaunchKernelGGL((lora_a_kernel<RT, true>), grid, dim3(kThreadsA), 0, s, p, chunks);
  else hipLaunchKernelGGL((lora_a_kernel<RT, false>), grid, dim3(kThreadsA), 0, s, p, chunks);
}

template <int RT, bool BF16, int BASE, bool WIDE>
void run_b(const LoraParams &p, hipStream_t s) {
  // Columns of a wave, in units of 32. Every workgroup reads its rows' sums, 4
  // groups R bytes a row; `need` units make that at most half of the base and
  // output it moves, and are taken as far as 256 workgroups are left. Beyond
  // that, enough that no more than about 1024 are launched.
  const int64_t units = (p.N + 127) / 128 * ((p.rows + kTileRows - 1) / kTileRows);
  const int64_t row_bytes = BASE + (p.out_dtype == 3 ? 4 : 2);
  const int64_t need = 8 * lora_groups(p.K) * lora_padded_rank(p.R) / (row_bytes * 128) + 1;
  int64_t u = need < units / 256 ? need : units / 256;
  if (u < units / 1024) u = units / 1024;
  const int per_wave = 32 * (int)(u < 1 ? 1 : u > 8 ? 8 : u);
  const dim3 grid(tile_slots(p.rows, p.adapters), (p.N + 4 * per_wave - 1) / (4 * per_wave),
                  windows(p.rows));
  hipLaunchKernelGGL((lora_b_kernel<RT, BF16, BASE, WIDE>), grid, dim3(256), 0, s, p, per_wave,
                     lora_groups(p.K));
}

template <int RT, bool WIDE>
void run_b(const LoraParams &p, hipStream_t s) {
  const int base = !p.base ? 0 : p.base_dtype == 3 ? 4 : 2;
  if (p.bf16) {
    if (base == 0) run_b<RT, true, 0, WIDE>(p, s);
    else if (base == 2) run_b<RT, true, 2, WIDE>(p, s);
    else run_b<RT, true, 4, WIDE>(p, s);
  } else {
    if (base == 0) run_b<RT, false, 0, WIDE>(p, s);
    else if (base == 2) run_b<RT, false, 2, WIDE>(p, s);
    else run_b<RT, false, 4, WIDE>(p, s);
  }
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
  if (p.R < 8) run_b<1, false>(p, s);
  else if (p.R <= 16) run_b<1, true>(p, s);
  else if (p.R <= 32) run_b<2, true>(p, s);
  else if (p.R <= 64) run_b<4, true>(p, s);
  else run_b<8, true>(p, s);
  return hipGetLastError();
}

}  // namespace exl3

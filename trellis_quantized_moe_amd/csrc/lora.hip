// Low-rank adapters of many requests beside a shared projection:
//   out_t = base_t + scale_a (x_t A_a^T) B_a^T,   a = ids[t]
// Two launches: lora_a writes s = x A^T (fp32, R values a row) to the workspace;
// lora_b multiplies s by B^T, adds the base and stores. Up to 16 ranks mostly
// take one, lora_kernel, whose workgroups each form the s they need (lora_one).
// base and out are moved once; x is read by lora_kernel once for every chunk of
// columns, by lora_a once for every 64 ranks (every 16 up to 256 rows). The
// products take 3% of the matrix rate at rank 16 and 9% at rank 64 (before the
// terms of s are counted), so many rows are bound by memory: 16384 rows of
// 4096 -> 4096 at rank 16, fp32 base, 545 MB: 124 us, 4.4 TB/s (a large copy:
// 5.0). Few rows are bound by latency: one row 8.2 us, of which an empty launch
// is 2.5; beyond 16 rows finding the tile is about 3.
//
// Tiles. A tile is up to 32 rows of one adapter (16 in lora_kernel). Every
// workgroup of lora_a and lora_kernel finds its tile by itself: rows are taken
// in windows of 2048, and the workgroup counts its window's IDs per adapter,
// scans the tile counts and collects its rows (plan_tile), so that no planning
// launch goes before it and rows need not be sorted. The first workgroup of a
// tile leaves it in the workspace for lora_b. Rows without an adapter are one
// more bucket, whose tiles are copied.
//
// A row's bytes depend on that row alone: the K axis is cut the same way in
// every call (slices of 256 inputs, eight to a group, groups in ascending
// order, whichever waves take them), a row is one column of the MFMA tiles whichever row it
// shares them with, and the second product's scaling is per row.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace exl3 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWindow = 2048;       // rows planned together
constexpr int kTileRows = 32;       // rows of a tile of two launches
constexpr int kSlice = 256;         // inputs summed in one run
constexpr int kSlices = 8;          // slices of a workgroup of lora_a
constexpr int kGroup = kSlices * kSlice;
constexpr int kMaxBuckets = 1025;  // EXL3_MAX_ADAPTERS and "none"

struct PlanLds {
  int count[kMaxBuckets];
  int hits[kWindow / 64];  // rows of the bucket, by 64 rows
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
// the window has fewer tiles) and its rows, counted from the window's first,
// in L.rows[0 .. nrows). Called by all threads of a workgroup of W waves; TR:
// rows of a tile. The order of the tiles does not matter to anybody.
template <int W, int TR>
__device__ __forceinline__ int plan_tile(const LoraParams &p, int win, int tile, PlanLds &L,
                                         int &nrows) {
  constexpr int kThreads = 64 * W, kChunks = kWindow / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  if (p.rows <= 16) {
    // One row to a lane; every wave goes through the adapters as they appear,
    // with no counts in LDS to wait for (4096 -> 4096 at rank 16, 1 row 7.8 us
    // instead of 8.9, 16 rows 8.7 instead of 9.6; 61 rows of 40 adapters, rank
    // 32, would take 1.6 us more).
    const int r = min(lane, p.rows - 1);
    int a;
    if (p.ids_i64) {
      const int64_t id = ((const int64_t *)p.ids)[r];
      a = id >= 0 && id < p.adapters ? (int)id : p.adapters;
    } else {
      a = ((const int32_t *)p.ids)[r];
      a = (uint32_t)a < (uint32_t)p.adapters ? a : p.adapters;
    }
    for (uint64_t left = (1ull << p.rows) - 1; left;) {
      const int ad = __builtin_amdgcn_readlane(a, __ffsll((long long)left) - 1);
      const uint64_t same = __ballot(a == ad) & left;
      if (tile == 0) {
        static_assert(TR >= 16, "a bucket is one tile");
        nrows = __popcll(same);
        if (wave == 0 && ((same >> lane) & 1)) L.rows[__popcll(same & ((1ull << lane) - 1))] = lane;
        __syncthreads();
        return ad;
      }
      --tile;
      left &= ~same;
    }
    return -1;
  }
  const int row0 = win * kWindow;
  const int n = min(p.rows - row0, kWindow);
  // lanes past the window read its last ID and drop it: loads without a branch
  // around them are all in flight together
  int a[kChunks];
  if (p.ids_i64) {
    int64_t id[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      id[i] = ((const int64_t *)p.ids)[row0 + min(i * kThreads + tid, n - 1)];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      a[i] = id[i] >= 0 && id[i] < p.adapters ? (int)id[i] : p.adapters;
  } else {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      a[i] = ((const int32_t *)p.ids)[row0 + min(i * kThreads + tid, n - 1)];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      a[i] = (uint32_t)a[i] < (uint32_t)p.adapters ? a[i] : p.adapters;
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) a[i] = i * kThreads + tid < n ? a[i] : -1;
  for (int b = tid; b <= p.adapters; b += kThreads) L.count[b] = 0;
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
    const int tiles = (rows + TR - 1) / TR;
    const int end = before + wave_scan(tiles);
    const uint64_t past = __ballot(end > tile);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      ad = b0 + l;
      skip = (tile - (__shfl(end, l, 64) - __shfl(tiles, l, 64))) * TR;
      size = __shfl(rows, l, 64);
      break;
    }
    before = __shfl(end, 63, 64);
  }
  ad = __builtin_amdgcn_readfirstlane(ad);
  if (ad < 0) return -1;
  skip = __builtin_amdgcn_readfirstlane(skip);
  nrows = min(TR, __builtin_amdgcn_readfirstlane(size) - skip);
  // the bucket's rows in order, from number `skip` on
  uint64_t hit[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    hit[i] = __ballot(a[i] == ad);
    if (lane == 0) L.hits[i * W + wave] = __popcll(hit[i]);
  }
  __syncthreads();
  // rows before this wave's of each chunk: lane i sums up to entry i
  static_assert(kWindow / 64 <= 64, "one entry to a lane");
  const int own = lane < kWindow / 64 ? L.hits[lane] : 0;
  const int before = wave_scan(own) - own;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int at = __builtin_amdgcn_readlane(before, i * W + wave) +
                   __popcll(hit[i] & ((1ull << lane) - 1)) - skip;
    if (a[i] == ad && at >= 0 && at < TR) L.rows[at] = i * kThreads + tid;
  }
  __syncthreads();
  return ad;
}

// Ranks the adapter uses.
__device__ __forceinline__ int used_rank(const LoraParams &p, int ad) {
  return p.ranks ? max(0, min(p.R, uload_i32(p.ranks + ad))) : p.R;
}

// A load from a uniform address and a lane's byte offset: a window's rows lie
// within 2^32 bytes (row distances are at most EXL3_LORA_MAX_LD), so a row's
// address takes one register instead of two.
template <typename T>
__device__ __forceinline__ T load_at(const void *base, uint32_t off) {
  typedef const T __attribute__((address_space(1))) *gp;
  return *(gp)((uintptr_t)base + off);
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
// One wave of W: s[r][t] of RT * 16 ranks and TT * 16 rows over slices w and,
// with four waves, w + 4 of its group. Ranks are the MFMA rows, tile rows its
// columns. A lane's operand is 16 bytes of row (lane % 16), so loading operands
// as they are used puts 64 lanes on 64 cache lines, and the cache looks up one
// line a cycle: that took 58 us on 16384 x 4096 where the bytes need 27, and this
// way 43.
// Instead eight lanes take 128 bytes of a row, 64 inputs of 8 rows to a load,
// and the wave turns them round in LDS that it shares with no other: chunk k of
// row r lies at place k ^ (r % 8) of the row, so that the writes of eight lanes
// (one row) and the reads of eight (one chunk of eight rows) fall into
// different banks. lds_exchange() stands between the writes and the reads: no
// barrier. red[i], i < 4, gets the sum of slices i and i + 4.
template <int RT, int TT>
struct LdsA {
  static constexpr int kLd = RT * 16 + 4;
  static constexpr int kStage = (TT + RT) * 2048;  // bytes of a wave
};

template <int RT, int TT, int W, bool BF16>
__device__ __forceinline__ void lora_a_tile(const LoraParams &p, const int *tile_rows, int nrows,
                                            int ad, int r0, int ra, int kg, char *lds) {
  constexpr int kLd = LdsA<RT, TT>::kLd;
  constexpr int kPairs = kSlice / 64 * (kSlices / W);  // loads of 64 inputs
  constexpr int kAhead = TT + RT <= 3 ? 3 : TT + RT <= 4 ? 2 : 1;  // of them on their way
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, wave = wave_id();
  f32x4 acc[RT][TT];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  };
  // load h of a 16-row operand: row 8 h + lane / 8, inputs 8 (lane % 8) ..;
  // rows past the last row or rank repeat it, their sums are not used
  const uint16_t *x0 = p.x + (int64_t)blockIdx.z * kWindow * p.ldx;
  const uint16_t *a0 = p.a + (int64_t)ad * p.R * p.K;
  uint32_t src[TT + RT][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (lane >> 3);
#pragma unroll
    for (int j = 0; j < TT; ++j)
      src[j][h] = (uint32_t)tile_rows[min(j * 16 + r, nrows - 1)] * (uint32_t)p.ldx * 2;
#pragma unroll
    for (int i = 0; i < RT; ++i) src[TT + i][h] = min(r0 + i * 16 + r, ra - 1) * p.K * 2;
  }
  char *stage = lds + wave * LdsA<RT, TT>::kStage;
  char *put = stage + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
  const char *get[2] = {stage + c * 128 + ((g ^ (c & 7)) << 4),
                        stage + c * 128 + (((4 + g) ^ (c & 7)) << 4)};
  const int k0 = kg + wave * kSlice + 8 * (lane & 7);
  u32x4 v[kAhead][TT + RT][2];
  // K is a multiple of 8: a lane's eight inputs are all there or none is. Those
  // that are not read the row's last eight and count as zero.
  auto input = [&](int n) { return k0 + n / (kSlice / 64) * 4 * kSlice + n % (kSlice / 64) * 64; };
  auto fetch = [&](int n) {
    const int k = min(input(n), p.K - 8);
#pragma unroll
    for (int i = 0; i < TT + RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[n % kAhead][i][h] = load_at<u32x4>(i < TT ? x0 : a0, src[i][h] + 2 * k);
  };
  float *red = (float *)lds + ((wave & 3) * TT * 16 + c) * kLd + 4 * g;
  auto leave = [&](bool add) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        f32x4 *q = (f32x4 *)(red + j * 16 * kLd + i * 16);
        *q = add ? acc[i][j] + *q : acc[i][j];
      }
  };
  f32x4 first[RT][TT];  // four waves: the sums of slice w
  clear();
#pragma unroll
  for (int n = 0; n < kAhead; ++n) fetch(n);
#pragma unroll
  for (int n = 0; n < kPairs; ++n) {
    if (n == kSlice / 64) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) first[i][j] = acc[i][j];
      clear();
    }
    const bool there = input(n) < p.K;
#pragma unroll
    for (int i = 0; i < TT + RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 zero = {0, 0, 0, 0};
        *(u32x4 *)(put + i * 2048 + h * 1024) = there ? v[n % kAhead][i][h] : zero;
      }
    if (n + kAhead < kPairs) fetch(n + kAhead);
    lds_exchange();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 x[TT], a[RT];
#pragma unroll
      for (int j = 0; j < TT; ++j) x[j] = *(const u32x4 *)(get[s] + j * 2048);
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i] = *(const u32x4 *)(get[s] + (TT + i) * 2048);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = mfma16<BF16>(a[i], x[j], acc[i][j]);
    }
    lds_exchange();
  }
  __syncthreads();  // the sums take the place of the staged operands
  // lane: ranks 4 g .. 4 g + 3 of row c
  if constexpr (W == 4) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = first[i][j] + acc[i][j];
    leave(false);
  } else {
    if (wave >= 4) leave(false);
    __syncthreads();
    if (wave < 4) leave(true);
  }
  __syncthreads();
}

// Workgroup (tile, group and rank chunk, window).
template <int RT, int W, bool BF16>
__global__ void __launch_bounds__(64 * W) lora_a_kernel(LoraParams p, int chunks) {
  constexpr int kStages = W * LdsA<RT, 2>::kStage, kSums = 4 * 32 * LdsA<RT, 2>::kLd * 4;
  __shared__ PlanLds L;
  __shared__ __align__(16) char lds[kStages > kSums ? kStages : kSums];
  int nrows = 0;
  const int ad = plan_tile<W, kTileRows>(p, blockIdx.z, blockIdx.x, L, nrows);
  if (blockIdx.y == 0) {
    LoraTile *tile = p.tiles + (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) {
      tile->adapter = ad;
      tile->nrows = nrows;
    }
    if (threadIdx.x < kTileRows)
      tile->rows[threadIdx.x] = L.rows[min((int)threadIdx.x, max(nrows - 1, 0))];
  }
  if (ad < 0 || ad == p.adapters) return;
  const int group = blockIdx.y / chunks, r0 = (blockIdx.y - group * chunks) * RT * 16;
  const int ra = used_rank(p, ad);
  if (r0 >= ra) return;
  const int kg = group * kGroup;
  if (nrows <= 16) lora_a_tile<RT, 1, W, BF16>(p, L.rows, nrows, ad, r0, ra, kg, lds);
  else lora_a_tile<RT, 2, W, BF16>(p, L.rows, nrows, ad, r0, ra, kg, lds);
  const int rp = (p.R + 15) & ~15, row0 = blockIdx.z * kWindow;
  const int w = (nrows <= 16 ? 16 : 32) * LdsA<RT, 2>::kLd;
  for (int i = threadIdx.x; i < nrows * RT * 4; i += 64 * W) {
    const int t = i / (RT * 4), r = (i - t * RT * 4) * 4;
    const float *from = (const float *)lds + t * LdsA<RT, 2>::kLd + r;
    const f32x4 s = (*(const f32x4 *)from + *(const f32x4 *)(from + w)) +
                    (*(const f32x4 *)(from + 2 * w) + *(const f32x4 *)(from + 3 * w));
    if (r0 + r < rp)
      *(f32x4 *)(p.part + ((int64_t)group * p.rows + row0 + L.rows[t]) * rp + r0 + r) = s;
  }
}

// ------------------------------------------------------------------ s B^T
__device__ __forceinline__ float from16(uint16_t b, bool bf16) {
  return bf16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// Four consecutive columns of a row: base as loaded (BASE: bytes of a value, 0
// for no base; a template argument so that no branch stands between the loads),
// as fp32, and stored.
template <int BASE>
struct Raw4 {
  typedef uint32_t type __attribute__((ext_vector_type(2)));
};
template <>
struct Raw4<4> {
  typedef u32x4 type;
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <int BASE>
__device__ __forceinline__ typename Raw4<BASE>::type load4(const void *p, uint32_t i) {
  if constexpr (BASE == 0) return (u32x2){0, 0};
  else return load_at<typename Raw4<BASE>::type>(p, i * BASE);
}
template <int BASE>
__device__ __forceinline__ void widen4(const typename Raw4<BASE>::type &r, int dtype,
                                       float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BASE == 4) {
      const uint32_t w = r[j];
      v[j] = __builtin_bit_cast(float, w);
    } else if constexpr (BASE == 2) {
      const uint32_t w = r[j >> 1];
      v[j] = from16((uint16_t)(w >> (16 * (j & 1))), dtype == 2);
    } else {
      v[j] = 0.0f;
    }
  }
}
__device__ __forceinline__ void store4(void *p, int dtype, uint32_t i, const float (&v)[4]) {
  if (dtype == 3) {
    typedef f32x4 __attribute__((address_space(1))) *gp;
    *(gp)((uintptr_t)p + i * 4) = (f32x4){v[0], v[1], v[2], v[3]};
  } else {
    typedef u32x2 __attribute__((address_space(1))) *gp;
    *(gp)((uintptr_t)p + i * 2) = (u32x2){f32x2_to_out16(v[0], v[1], dtype == 2),
                                          f32x2_to_out16(v[2], v[3], dtype == 2)};
  }
}
// The window's first row of base and out.
__device__ __forceinline__ const void *window_base(const LoraParams &p, int bytes) {
  return (const char *)p.base + (int64_t)blockIdx.z * kWindow * p.ldbase * bytes;
}
__device__ __forceinline__ void *window_out(const LoraParams &p) {
  return (char *)p.out + (int64_t)blockIdx.z * kWindow * p.ldout * (p.out_dtype == 3 ? 4 : 2);
}

// s as MFMA operands. The matrix cores take 16-bit inputs, so s is written as
// a sum of 16-bit terms, each the rounded rest of the ones before: two fp16
// terms hold an entry to 2^-23, three bf16 terms to 2^-26 (two would hold 2^-17:
// enough below the last bit of a 16-bit output, but not where the ranks, or the
// sum and the base, cancel). An infinite or NaN entry is its first term alone.
//
// The row is first scaled by a power of two (exact, and undone on the fp32 sum).
// fp16: to [2^13, 2^14), so that the terms neither overflow nor lose small
// entries (those below 2^-15 of the row's largest hold 2^-38 of it); B is below
// 2^16 and the sum below 2^37. bf16 has fp32's range, in B too, so a factor
// would overflow sums that are finite, or lose small ones: there is none, but
// for rows whose largest entry is below 2^-63, whose last terms would be
// subnormal (2^48: then below 2^-15, and the sum of 128 products below 2^120),
// and for those from 2^127 on, whose first term could round to infinity (2^-8).
//
// One MFMA takes 32 inner values: the first term of 16 ranks and the second
// term of the same 16, against B given twice. The third term is a second MFMA
// with zeros in the other half.
// TR: rows of the tile, W: waves.
template <int RT, int TR, int W>
struct LdsB {
  static constexpr int kLd = RT * 16 + 8;    // entries of a row: spread over the banks
  static constexpr int kRow = RT * 32 + 16;  // bytes of a column's B
  static constexpr int kStage = W * 64 * kRow;  // every wave's 64 columns
  uint16_t s[3][TR][kLd];
  int e[TR];
};

// Row t of s, Q = 4 or 8 lanes to a row: sum[j] holds ranks 4 (q + Q j) .. + 3.
template <int RT, bool BF16, int Q, int TR, int W>
__device__ __forceinline__ void split_s(int t, int q, float scale, int ra,
                                        const f32x4 (&sum)[4 * RT / Q], LdsB<RT, TR, W> &S) {
  constexpr int J = 4 * RT / Q;
  float v[J][4];
  float big = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[j][u] = 4 * (q + Q * j) + u < ra ? sum[j][u] * scale : 0.0f;
      big = fmaxf(big, fabsf(v[j][u]));
    }
  big = fmaxf(big, __shfl_xor(big, 1, 64));
  big = fmaxf(big, __shfl_xor(big, 2, 64));
  if (Q == 8) big = fmaxf(big, __shfl_xor(big, 4, 64));
  // fmaxf passes over NaN; the row's finite entries are scaled by the largest
  // (an infinity counts as exponent 255: everything finite stays below 2^14)
  const int field = (int)((__builtin_bit_cast(uint32_t, big) >> 23) & 255u);
  const int e = !BF16 ? field - 140 : field < 64 ? -48 : field < 254 ? 0 : 8;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    uint32_t w[3][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float lo = ldexpf(v[j][2 * u], -e), hi = ldexpf(v[j][2 * u + 1], -e);
#pragma unroll
      for (int m = 0; m < (BF16 ? 3 : 2); ++m) {
        const uint32_t b = f32x2_to_out16(lo, hi, BF16);
        w[m][u] = b;
        lo = fabsf(lo) < __builtin_inff() ? lo - from16((uint16_t)b, BF16) : 0.0f;
        hi = fabsf(hi) < __builtin_inff() ? hi - from16((uint16_t)(b >> 16), BF16) : 0.0f;
      }
    }
#pragma unroll
    for (int m = 0; m < (BF16 ? 3 : 2); ++m)
      *(uint2 *)&S.s[m][t][4 * (q + Q * j)] = make_uint2(w[m][0], w[m][1]);
  }
  if (q == 0) S.e[t] = e;
}

// Eight entries of B with zeros in the place of infinities.
template <bool BF16>
__device__ __forceinline__ u32x4 without_infinities(u32x4 b) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    b[w] &= ((b[w] & 0x7fffu) == kInf ? 0u : 0xffffu) |
            ((b[w] & 0x7fff0000u) == kInf << 16 ? 0u : 0xffff0000u);
  return b;
}

// Lanes that form a row of s in lora_b.
template <int RT>
constexpr int kLanesS = RT == 1 ? 4 : 8;

// The rows' sums from the workspace. kParts groups at a time are asked for
// together; groups and ranks that are not there repeat one that is, and are
// not added.
template <int RT, bool BF16>
__device__ __forceinline__ void load_s(const LoraParams &p, int row, int nrows, float scale, int ra,
                                       int groups, LdsB<RT, kTileRows, 4> &S) {
  constexpr int Q = kLanesS<RT>, J = 4 * RT / Q;
  const int t = threadIdx.x / Q, q = threadIdx.x % Q;
  if (t >= nrows) return;  // rows of the tile past its end are not used
  const int rp = (p.R + 15) & ~15;
  const float *from = p.part + (int64_t)(blockIdx.z * kWindow + row) * rp;
  constexpr int kParts = 4;
  f32x4 sum[J];
#pragma unroll
  for (int j = 0; j < J; ++j) sum[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < groups; i0 += kParts) {
    f32x4 part[kParts][J];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int r = 4 * (q + Q * j);
        part[i][j] = *(const f32x4 *)(from + (int64_t)min(i0 + i, groups - 1) * p.rows * rp +
                                      (r < ra ? r : 0));
      }
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (i0 + i < groups) sum[j] = i0 + i == 0 ? part[i][j] : sum[j] + part[i][j];
  }
  split_s<RT, BF16, Q>(t, q, scale, ra, sum, S);
}

// One wave: columns n0 .. n1 - 1, 64 at a time, of the tile's TT * 16 rows.
// Tile rows are the MFMA rows and column n + 4 (lane % 16) + i is column
// (lane % 16) of MFMA i, so that a lane's results of four MFMAs are four
// consecutive columns of a row and 16 lanes have 64: base and output move in
// runs of 128 bytes (16-bit) or 256 (fp32) with neighbouring lanes side by side.
// (With tile rows as the MFMA columns, neighbouring lanes held different rows
// and every load and store touched 64 cache lines: 128 us instead of 105 on
// 16384 x 4096 with an fp32 base.) B's rows of 64 columns are one run of memory: they are loaded
// as such and turned round in LDS. The loads of the next 64 columns are under
// way while these are worked on.
// row_of(i): the tile's row i, past its end any of its rows; make_s, called by
// all threads, leaves s in S.
template <int RT, int TT, bool BF16, int BASE, int TR, int W, typename R, typename F>
__device__ __forceinline__ void lora_b_columns(const LoraParams &p, R row_of, int nrows, int ad,
                                               int ra, int n0, int n1, LdsB<RT, TR, W> &S,
                                               char *stages, F make_s) {
  typedef typename Raw4<BASE>::type raw_t;
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, wave = wave_id();
  constexpr int kRow = LdsB<RT, TR, W>::kRow;
  // the lane's rows 16 j + 4 g + r, as element offsets of base and out;
  // past the end the last row again
  uint32_t bo[TT][4], oo[TT][4];
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t row = row_of(16 * j + 4 * g + r);
      bo[j][r] = row * (uint32_t)p.ldbase;
      oo[j][r] = row * (uint32_t)p.ldout;
    }
  const void *base0 = window_base(p, BASE);
  void *out0 = window_out(p);
  const uint16_t *b = p.b + (int64_t)ad * p.N * p.R;
  char *stage = stages + wave * 64 * kRow;
  u32x4 bn[2 * RT];
  raw_t base[TT][4];
  // 16-byte chunk m * 64 + lane of the columns' run of B; N - n is a multiple
  // of 8, so the run is one of whole chunks. Chunks past its end repeat the last.
  auto fetch_b = [&](int n) {
    n = min(n, p.N - 8);
    const int last = min(64, p.N - n) * p.R / 8 - 1;
#pragma unroll
    for (int m = 0; m < 2 * RT; ++m)
      bn[m] = load_at<u32x4>(b, (uint32_t)(n * p.R * 2 + min(m * 64 + lane, last) * 16));
  };
  auto fetch_base = [&](int j, int r, int n) {
    base[j][r] = load4<BASE>(base0, bo[j][r] + min(n + 4 * c, p.N - 4));
  };
  // into LDS, a column's ranks kRow apart
  const int row_chunks = p.R / 8, inverse = 65536 / max(row_chunks, 1) + 1;
  auto put_b = [&] {
    if (p.R % 8 == 0) {
#pragma unroll
      for (int m = 0; m < 2 * RT; ++m) {
        const int q = m * 64 + lane, row = (q * inverse) >> 16;  // q / row_chunks: q < 1024
        if (q < 8 * p.R) *(u32x4 *)(stage + row * kRow + (q - row * row_chunks) * 16) = bn[m];
      }
    } else {  // chunks that span columns: value by value
      int l = lane;
      asm volatile("" : "+v"(l));  // the places are computed here, not kept in registers
      const int wrap = kRow - 2 * p.R;  // from behind a column's ranks to the next column
#pragma unroll
      for (int m = 0; m < 2 * RT; ++m) {
        const int first = (m * 64 + l) * 8, row = first / p.R;
        int r = first - row * p.R;
        char *to = stage + row * kRow + r * 2;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if (to < stage + 64 * kRow) *(uint16_t *)to = (uint16_t)(bn[m][w >> 1] >> (16 * (w & 1)));
          const bool end = ++r == p.R;
          to += end ? wrap + 2 : 2;
          r = end ? 0 : r;
        }
      }
    }
  };
  constexpr bool kNextB = RT <= 4;  // 128 ranks: no registers for the next B
  if (kNextB) fetch_b(n0);
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) fetch_base(j, r, n0);
  make_s();

  // Whether the columns of B on their way hold an infinity or a NaN. An infinity
  // meets the first term of s alone: with a later one, 0 or of the other sign,
  // it would give NaN. (Looking for NaN among the results instead keeps the
  // matrix instructions from running beside what follows: 51 us instead of 34 at
  // 128 ranks, 4000 rows of 1024 columns; without either 31.)
  auto odd_b = [&] {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top[4] = {};
#pragma unroll
    for (int m = 0; m < 2 * RT; ++m)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        top[w] = __builtin_elementwise_max(top[w], __builtin_bit_cast(u16x2, bn[m][w] & 0x7fff7fffu));
    const u16x2 t = __builtin_elementwise_max(__builtin_elementwise_max(top[0], top[1]),
                                              __builtin_elementwise_max(top[2], top[3]));
    constexpr uint16_t kInf = BF16 ? 0x7f80 : 0x7c00;
    return __any(t[0] >= kInf || t[1] >= kInf);
  };

  // acc += s B^T of the staged columns, ranks 16 rt ..: `count` column MFMAs from
  // `first` on
  auto multiply = [&](f32x4(&acc)[4][TT], int rt, auto first, auto count, auto clean) {
    constexpr int i0 = decltype(first)::value, i1 = i0 + decltype(count)::value;
    constexpr bool CLEAN = decltype(clean)::value;
    const int r = rt * 16 + 8 * (g & 1);
    u32x4 bv[4];
#pragma unroll
    for (int i = i0; i < i1; ++i) bv[i] = *(const u32x4 *)(stage + (4 * c + i) * kRow + r * 2);
    // ranks from ra on give zero whatever B, or LDS behind it, holds there
    if (rt * 16 + 16 > ra) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t keep = (r + 2 * w < ra ? 0xffffu : 0u) | (r + 2 * w + 1 < ra ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = i0; i < i1; ++i) bv[i][w] &= keep;
      }
    }
    if (CLEAN && g >> 1) {
#pragma unroll
      for (int i = i0; i < i1; ++i) bv[i] = without_infinities<BF16>(bv[i]);
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const u32x4 s = *(const u32x4 *)&S.s[g >> 1][j * 16 + c][r];
#pragma unroll
      for (int i = i0; i < i1; ++i) acc[i][j] = mfma16<BF16>(s, bv[i], acc[i][j]);
      if constexpr (BF16) {
        u32x4 s3 = *(const u32x4 *)&S.s[2][j * 16 + c][r];
        if (g >> 1) s3 = (u32x4){0, 0, 0, 0};
#pragma unroll
        for (int i = i0; i < i1; ++i)
          acc[i][j] = mfma16<BF16>(s3, CLEAN ? without_infinities<BF16>(bv[i]) : bv[i], acc[i][j]);
      }
    }
  };

  for (int n = n0; n < n1; n += 64) {
    if (!kNextB) fetch_b(n);
    put_b();
    const bool odd = odd_b();
    if (kNextB) fetch_b(n + 64);
    lds_exchange();
    __builtin_amdgcn_sched_barrier(0);
    f32x4 acc[4][TT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    typedef std::integral_constant<int, 0> zero;
    if (!odd) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (RT >= 4) __builtin_amdgcn_sched_barrier(0);
        multiply(acc, rt, zero(), std::integral_constant<int, 4>(), std::false_type());
      }
    } else {  // one after the other: no more registers than above
      typedef std::integral_constant<int, 1> one;
#pragma unroll 1
      for (int rt = 0; rt < RT; ++rt) {
        multiply(acc, rt, zero(), one(), std::true_type());
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc, rt, one(), one(), std::true_type());
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc, rt, std::integral_constant<int, 2>(), one(), std::true_type());
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc, rt, std::integral_constant<int, 3>(), one(), std::true_type());
      }
    }
    const int col = n + 4 * c;
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * j + 4 * g + r;
        const int e = S.e[t];
        float v[4];
        widen4<BASE>(base[j][r], p.base_dtype, v);
        fetch_base(j, r, n + 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += ldexpf(acc[i][j][r], e);
        if (t < nrows && col < p.N) store4(out0, p.out_dtype, oo[j][r] + col, v);
      }
    lds_exchange();
  }
}

// Rows without an adapter: out = base (or zeros), 8 loads of a thread together.
template <int BASE>
__device__ __forceinline__ void copy_rows(const LoraParams &p, const int *tile_rows, int nrows,
                                          int n0, int n1) {
  if (p.base == p.out || n0 >= n1) return;
  const int per_row = (n1 - n0) / 4, total = nrows * per_row, threads = blockDim.x;
  for (int i0 = threadIdx.x; i0 < total; i0 += threads * 8) {
    typename Raw4<BASE>::type raw[8];
    uint32_t row[8], n[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = min(i0 + threads * u, total - 1), t = i / per_row;
      row[u] = tile_rows[t];
      n[u] = n0 + (i - t * per_row) * 4;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      raw[u] = load4<BASE>(window_base(p, BASE), row[u] * (uint32_t)p.ldbase + n[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float v[4];
      widen4<BASE>(raw[u], p.base_dtype, v);
      if (i0 + threads * u < total)
        store4(window_out(p), p.out_dtype, row[u] * (uint32_t)p.ldout + n[u], v);
    }
  }
}

// Workgroup (tile, `cols` columns, window): each wave takes a quarter of the
// columns. 4001 rows of 2048 columns at rank 64, bf16, 34 MB: 21.8 us, a chain
// of loads (tile, sums, B, base) that two workgroups to a CU do not hide (at 19.5
// us, with two terms of s: without base 2 us less, without the sums 3, without B
// 1, without the stores 5). 16384 rows of 4096 columns, fp16, 276 MB: 91 us, 3.0
// TB/s.
// 32 ranks with a 16-bit base: three waves a SIMD (70 us instead of 80 on 16384
// rows of 4096 columns, bf16); more ranks or an fp32 base do not fit.
template <int RT, bool BF16, int BASE>
__global__ void __launch_bounds__(256, RT == 2 && BASE <= 2 ? 3 : 1)
    lora_b_kernel(LoraParams p, int cols, int groups) {
  __shared__ __align__(16) LdsB<RT, kTileRows, 4> S;
  __shared__ __align__(16) char stages[LdsB<RT, kTileRows, 4>::kStage];
  const LoraTile *tile = p.tiles + (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  // the rows are asked for together with what says whether there are any, one
  // to a lane; lanes get each other's by shuffles
  const int own_row = tile->rows[threadIdx.x & (kTileRows - 1)];
  const int ad = uload_i32(&tile->adapter), nrows = uload_i32(&tile->nrows);
  if (ad < 0) return;
  const int c0 = blockIdx.y * cols, c1 = min(c0 + cols, p.N);
  const int ra = ad < p.adapters ? used_rank(p, ad) : 0;
  if (ra == 0) {
    copy_rows<BASE>(p, tile->rows, nrows, c0, c1);
    return;
  }
  const float scale = p.scale ? uload_f32(p.scale + ad) : 1.0f;
  auto row_of = [&](int i) { return __shfl(own_row, i, 64); };
  const int s_row = row_of(threadIdx.x / kLanesS<RT>);
  auto make_s = [&] {
    load_s<RT, BF16>(p, s_row, nrows, scale, ra, groups, S);
    __syncthreads();
  };
  const int n0 = c0 + cols / 4 * wave_id(), n1 = min(n0 + cols / 4, p.N);
  if (nrows <= 16)
    lora_b_columns<RT, 1, BF16, BASE>(p, row_of, nrows, ad, ra, n0, n1, S, stages, make_s);
  else
    lora_b_columns<RT, 2, BF16, BASE>(p, row_of, nrows, ad, ra, n0, n1, S, stages, make_s);
}

// -------------------------------------------------------- both in one launch
// Up to 16 ranks. Workgroup (tile of 16 rows, `cols` columns, window), eight
// waves: s over all of K, a group of slices at a time, then the columns. The
// same sums in the same order as the two launches, so the same bytes, but s
// never leaves LDS. Workgroups that share a tile each form it.
template <bool BF16, int BASE>
__global__ void __launch_bounds__(512) lora_kernel(LoraParams p, int cols) {
  constexpr int W = kSlices, TR = 16, kLd = LdsA<1, 1>::kLd;
  // x, A and the sums, and once s is made B's columns
  constexpr int kBytesA = W * LdsA<1, 1>::kStage, kBytesB = LdsB<1, TR, W>::kStage;
  static_assert(kBytesA >= 4 * TR * kLd * 4, "the sums take the place of the operands");
  __shared__ PlanLds L;
  __shared__ __align__(16) char lds[kBytesA > kBytesB ? kBytesA : kBytesB];
  __shared__ __align__(16) LdsB<1, TR, W> S;
  int nrows = 0;
  const int ad = plan_tile<W, TR>(p, blockIdx.z, blockIdx.x, L, nrows);
  if (ad < 0) return;
  const int c0 = blockIdx.y * cols, c1 = min(c0 + cols, p.N);
  const int ra = ad < p.adapters ? used_rank(p, ad) : 0;
  if (ra == 0) {
    copy_rows<BASE>(p, L.rows, nrows, c0, c1);
    return;
  }
  const float scale = p.scale ? uload_f32(p.scale + ad) : 1.0f;
  // thread: ranks r .. r + 3 of row t
  const int t = threadIdx.x >> 2, r = (threadIdx.x & 3) * 4;
  const bool mine = t < TR;
  float *sums = (float *)lds + t * kLd + r;
  constexpr int w = TR * kLd;
  f32x4 total = {0.f, 0.f, 0.f, 0.f};
  for (int kg = 0; kg < p.K; kg += kGroup) {
    if (kg) __syncthreads();  // the sums before are taken
    lora_a_tile<1, 1, W, BF16>(p, L.rows, nrows, ad, 0, ra, kg, lds);
    if (mine) {
      const f32x4 s = (*(const f32x4 *)sums + *(const f32x4 *)(sums + w)) +
                      (*(const f32x4 *)(sums + 2 * w) + *(const f32x4 *)(sums + 3 * w));
      total = kg == 0 ? s : total + s;
    }
  }
  auto make_s = [&] {
    const f32x4 sum[1] = {total};
    if (t < nrows) split_s<1, BF16, 4>(t, threadIdx.x & 3, scale, ra, sum, S);
    __syncthreads();  // s is there, and the sums' place is free for B
  };
  const int n0 = c0 + cols / W * wave_id(), n1 = min(n0 + cols / W, p.N);
  auto row_of = [&](int i) { return L.rows[min(i, nrows - 1)]; };
  lora_b_columns<1, 1, BF16, BASE>(p, row_of, nrows, ad, ra, n0, n1, S, lds, make_s);
}

int windows(int rows) { return (rows + kWindow - 1) / kWindow; }
// Tiles a window can have: u buckets in use give at most u + (w - u) / rows.
int tile_slots(int rows, int adapters, int tile_rows = kTileRows) {
  const int w = rows < kWindow ? rows : kWindow;
  const int u = adapters + 1 < w ? adapters + 1 : w;
  return u + (w - u) / tile_rows;
}

template <int RT>
void run_a(const LoraParams &p, hipStream_t s) {
  // 64 ranks: four waves with two slices each, so that two workgroups fit on a
  // CU (6144 -> 64 ranks, 4001 rows: 18.6 us; eight waves 21.7; eight waves and
  // 64 rows 16.9, but 143 against 127 on 16384 rows of 8192 -> 128 ranks).
  // Fewer ranks: eight waves, which finish a few rows sooner (16 ranks, one row:
  // 5.6 us, four waves 6.1; 16384 rows: no difference).
  constexpr int W = RT == 4 ? 4 : 8;
  const int chunks = (p.R + RT * 16 - 1) / (RT * 16);
  const dim3 grid(tile_slots(p.rows, p.adapters), lora_groups(p.K) * chunks, windows(p.rows));
  if (p.bf16)
    hipLaunchKernelGGL((lora_a_kernel<RT, W, true>), grid, dim3(64 * W), 0, s, p, chunks);
  else
    hipLaunchKernelGGL((lora_a_kernel<RT, W, false>), grid, dim3(64 * W), 0, s, p, chunks);
}

template <int RT, bool BF16, int BASE>
void run_b(const LoraParams &p, hipStream_t s) {
  // Columns of a workgroup, in units of 256. Every workgroup reads its rows'
  // sums, 4 groups R bytes a row; `need` units make that at most half of the
  // base and output it moves, and are taken as far as 128 workgroups are left.
  // Beyond that, enough that no more than about 1024 are launched.
  const int64_t units = (p.N + 255) / 256 * (int64_t)((p.rows + kTileRows - 1) / kTileRows);
  const int64_t row_bytes = BASE + (p.out_dtype == 3 ? 4 : 2);
  const int64_t need = 8 * lora_groups(p.K) * lora_padded_rank(p.R) / (row_bytes * 256) + 1;
  int64_t u = need < units / 128 ? need : units / 128;
  if (u < units / 1024) u = units / 1024;
  const int cols = 256 * (int)(u < 1 ? 1 : u > 8 ? 8 : u);
  const dim3 grid(tile_slots(p.rows, p.adapters), (p.N + cols - 1) / cols, windows(p.rows));
  hipLaunchKernelGGL((lora_b_kernel<RT, BF16, BASE>), grid, dim3(256), 0, s, p, cols,
                     lora_groups(p.K));
}

template <bool BF16, int BASE>
void run_one(const LoraParams &p, hipStream_t s) {
  // Columns of a workgroup, in units of 512: all of them once there are 192
  // tiles or so, fewer where that leaves CUs empty (4096 -> 4096, rank 16, one
  // chunk against eight: 256 rows 17.6 and 10.5 us, 4000 rows 28 and 57)
  const int tiles = (p.rows + 15) / 16, most = (p.N + 511) / 512;
  const int chunks = tiles >= 192 ? 1 : 192 / tiles < most ? 192 / tiles : most;
  const int cols = (most + chunks - 1) / chunks * 512;
  const dim3 grid(tile_slots(p.rows, p.adapters, 16), (p.N + cols - 1) / cols, windows(p.rows));
  hipLaunchKernelGGL((lora_kernel<BF16, BASE>), grid, dim3(512), 0, s, p, cols);
}

// f(16-rank tiles, x in bf16, bytes of a base value)
template <typename F>
void by_kind(const LoraParams &p, F f) {
  auto based = [&](auto rt, auto bf16) {
    if (!p.base) f(rt, bf16, std::integral_constant<int, 0>());
    else if (p.base_dtype == 3) f(rt, bf16, std::integral_constant<int, 4>());
    else f(rt, bf16, std::integral_constant<int, 2>());
  };
  auto typed = [&](auto rt) {
    if (p.bf16) based(rt, std::true_type());
    else based(rt, std::false_type());
  };
  if (p.R <= 16) typed(std::integral_constant<int, 1>());
  else if (p.R <= 32) typed(std::integral_constant<int, 2>());
  else if (p.R <= 64) typed(std::integral_constant<int, 4>());
  else typed(std::integral_constant<int, 8>());
}

}  // namespace

int lora_groups(int K) { return (K + kGroup - 1) / kGroup; }
int lora_padded_rank(int R) { return (R + 15) & ~15; }
size_t lora_tiles(int rows, int adapters) {
  return (size_t)windows(rows) * tile_slots(rows, adapters);
}

// One launch pays for few ranks: every workgroup reads all of A for 16 rows
// (in us, one launch and two, fp16 base: 4096 -> 4096 at rank 16, 1 row 7.8 and
// 8.1, 256 rows 10.6 and 12.4, 16384 rows 100 and 107; 6144 -> 192 at rank 8, 9.2
// and 7.4, 11.3 and 11.5, 54 and 56; at rank 64, 4096 -> 4096, 18 and 14 at 256
// rows, 178 and 139 at 16384), and spares a launch on the host (2.5 us), which
// outweighs the 1.8 lost on one row of 6144 -> 192; a replayed graph does not
// pay it, and loses them. A long K and few rows leave one launch too few
// workgroups for A, which two launches split over K.
bool lora_one(const LoraParams &p) {
  return p.R <= 16 && (lora_groups(p.K) <= 4 || p.rows >= 4096);
}
hipError_t launch_lora_one(const LoraParams &p, hipStream_t s) {
  by_kind(p, [&](auto rt, auto bf16, auto base) {
    if constexpr (decltype(rt)::value == 1)
      run_one<decltype(bf16)::value, decltype(base)::value>(p, s);
  });
  return hipGetLastError();
}

hipError_t launch_lora_a(const LoraParams &p, hipStream_t s) {
  if (p.R <= 16 || p.rows <= 256) run_a<1>(p, s);
  else if (p.R <= 32) run_a<2>(p, s);
  else run_a<4>(p, s);
  return hipGetLastError();
}

hipError_t launch_lora_b(const LoraParams &p, hipStream_t s) {
  by_kind(p, [&](auto rt, auto bf16, auto base) {
    run_b<decltype(rt)::value, decltype(bf16)::value, decltype(base)::value>(p, s);
  });
  return hipGetLastError();
}

}  // namespace exl3

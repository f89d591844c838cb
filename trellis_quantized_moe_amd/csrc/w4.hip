// Products with 4-bit weights and group scales, for the sorted rows of experts
// or for all rows of one projection:
//   out[p, n] = sum over groups g of s[n, g] t_g,
//   t_g       = sum over k in g of x[p, k] (q[n, k] - z[n, g])
// q - z is a whole number of at most 15 in size, exact in fp16 and bf16, so the
// weights enter the MFMA as they are and t_g is a sum of exact products in fp32;
// the scale is applied to t_g in fp32: out = fma(s_g, t_g, out), g ascending.
// No weight is rounded. |t_g| <= 15 * 128 |x|: finite for |x| below 2^117.
//
// A row's bytes depend on that row and its expert's weights alone: every form
// sums a group by the same chain of v_mfma_f32_16x16x32 (32 inputs each,
// ascending) and adds the groups in the same order, whichever rows share a tile
// and whichever waves take which inputs.
//
// Weights lie in tiles of 16 outputs x 128 inputs, 1 KB, in the order of the
// MFMA's operand: lane l = 16 kg + n holds 16 bytes, word i of which holds
// inputs 32 i + 8 kg .. + 7 of output n. In a word, bits 4 p hold input 2 p
// (p < 4) or 2 (p - 4) + 1, so that one shift and mask gives two neighbours in
// the two halves of a dword.
#include "common.hpp"
#include "kernels.hpp"

namespace exl3 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileK = 128;

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Eight weights q - z of a word as the MFMA's operand.
// fp16, a well-known way: 0x6400 | q is 1024 + q, 0x6400 | 16 q is 1024 + 16 q: 1024 + z (64 + z
// after a sixteenth) is taken off again, exactly; nine instructions.
// bf16 has no packed subtraction: four q - z at a time as signed bytes (128 + q
// - z borrows from no neighbour), each through fp32, whose upper half is the
// value; nineteen instructions.
struct Masks {
  // in registers that the compiler does not fold back into literals: an
  // and-or takes none
  uint32_t low, high;
  __device__ __forceinline__ explicit Masks(bool bf16) {
    if (bf16) {
      asm volatile("v_mov_b32 %0, 0x0f0f0f0f" : "=v"(low));
      high = 0;
    } else {
      asm volatile("v_mov_b32 %0, 0x000f000f" : "=v"(low));
      asm volatile("v_mov_b32 %0, 0x00f000f0" : "=v"(high));
    }
  }
};
// What weights_of needs of a zero.
template <bool BF16>
struct Zero {
  uint32_t bytes;
  f16x2 one, sixteenth;
  __device__ __forceinline__ explicit Zero(int z) {
    if constexpr (BF16) {
      bytes = __builtin_amdgcn_perm(0u, (uint32_t)z, 0u);  // in all four
    } else {
      const _Float16 a = (_Float16)(float)(-1024 - z), b = (_Float16)(float)(-64 - z);
      one = (f16x2){a, a};
      sixteenth = (f16x2){b, b};
    }
  }
};
template <bool BF16>
__device__ __forceinline__ u32x4 weights_of(uint32_t w, const Zero<BF16> &z, const Masks &m) {
  u32x4 r;
  if constexpr (BF16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // bytes 0, 1, 2, 3 hold weights 2 h + 0, 4, 1, 5
      const uint32_t v =
          (((w >> (4 * h) & m.low) | 0x80808080u) - z.bytes) ^ 0x80808080u;
      uint32_t f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = __builtin_bit_cast(uint32_t, (float)(int8_t)(v >> (8 * i)));
      r[h] = __builtin_amdgcn_perm(f[2], f[0], 0x07060302u);
      r[h + 2] = __builtin_amdgcn_perm(f[3], f[1], 0x07060302u);
    }
  } else {
    const f16x2 sixteen = {(_Float16)0.0625f, (_Float16)0.0625f};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t v = w >> (4 * i);
      const f16x2 a = __builtin_bit_cast(f16x2, (v & m.low) | 0x64006400u);
      const f16x2 b = __builtin_bit_cast(f16x2, (v & m.high) | 0x64006400u);
      r[i] = __builtin_bit_cast(uint32_t, a + z.one);
      r[i + 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, sixteen, z.sixteenth));
    }
  }
  return r;
}

// + 0: see store_tile.
__device__ __forceinline__ void store_out(const W4Params &p, int64_t at, float v) {
  v += 0.f;
  if (p.out_dtype == 3) ((float *)p.out)[at] = v;
  else ((uint16_t *)p.out)[at] = f32_to_out16(v, p.out_dtype == 2);
}

// What a workgroup works on: item `item` of the tiles of `tm` rows (counted up
// through the experts, each with ceil(rows / tm) of them) times `per` blocks of
// outputs, block within tile. False past the last item. Workgroups are dealt to
// the 8 XCDs in turn; each XCD gets a run of neighbouring items, whose rows of x
// and weights its L2 then holds for several of them. Offsets are kept within
// the call's rows.
struct Item {
  int expert, row0, nrows, block;
};
__device__ __forceinline__ bool find_item(const W4Params &p, int tm, int per, Item &it) {
  const int lane = threadIdx.x & 63;
  const int C = (p.E + 63) / 64;  // experts of a lane
  constexpr int kKept = 4;        // whose ends stay in registers
  auto rows_before = [&](int e) { return (uint32_t)min(max(p.offset[e], 0), p.rows); };
  auto tiles_of = [tm](uint32_t lo, uint32_t hi) { return hi > lo ? (hi - lo + tm - 1) / tm : 0u; };
  uint32_t ends[kKept + 1];
  uint32_t mine = 0, upto = 0, total;
  if (p.offset) {
#pragma unroll
    for (int i = 0; i <= kKept; ++i) ends[i] = rows_before(min(lane * C + min(i, C), p.E));
#pragma unroll
    for (int i = 0; i < kKept; ++i) mine += tiles_of(ends[i], ends[i + 1]);
    uint32_t prev = ends[kKept];
    for (int i = kKept; i < C; ++i) {
      const uint32_t next = rows_before(min(lane * C + i + 1, p.E));
      mine += tiles_of(prev, next);
      prev = next;
    }
    upto = mine;  // tiles of the experts up to this lane's last
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t v = __shfl_up(upto, s, 64);
      upto += lane >= s ? v : 0;
    }
    total = __builtin_amdgcn_readlane(upto, 63);
  } else {
    total = (uint32_t)(p.rows + tm - 1) / tm;
  }
  const int64_t items = (int64_t)total * per, id = p.first + blockIdx.x;
  if (id >= items) return false;
  uint32_t idx;
  if (items < (1ll << 31)) {  // a division in 32 bits
    const uint32_t n = (uint32_t)items, i = (uint32_t)id;
    const uint32_t item = (i & 7) * (n >> 3) + min(i & 7, n & 7) + (i >> 3);
    idx = item / (uint32_t)per;
    it.block = (int)(item - idx * per);
  } else {
    const int64_t item = (id & 7) * (items >> 3) + min(id & 7, items & 7) + (id >> 3);
    idx = (uint32_t)(item / per);
    it.block = (int)(item % per);
  }
  if (!p.offset) {
    it.expert = 0;
    it.row0 = idx * tm;
    it.nrows = min(tm, p.rows - it.row0);
    return true;
  }
  const int l = max(__ffsll((long long)__ballot(idx < upto)) - 1, 0);
  uint32_t rel = idx - __builtin_amdgcn_readlane(upto - mine, l);  // among lane l's tiles
  // whatever the offsets are, what is returned lies within the call's rows
  auto here = [&](int e, uint32_t lo, uint32_t hi) {
    const uint32_t rows = hi > lo ? hi - lo : 0u, at = rel * tm;
    if (at < rows) {
      it.expert = e;
      it.row0 = (int)(lo + at);
      it.nrows = (int)min((uint32_t)tm, rows - at);
      return true;
    }
    rel -= tiles_of(lo, hi);
    return false;
  };
  uint32_t prev = __builtin_amdgcn_readlane(ends[0], l);
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const uint32_t next = __builtin_amdgcn_readlane(ends[i + 1], l);
    if (here(min(l * C + i, p.E - 1), prev, next)) return true;
    prev = next;
  }
  for (int e = l * C + kKept; e < min(l * C + C, p.E); ++e) {
    const uint32_t next = rows_before(e + 1);
    if (here(e, prev, next)) return true;
    prev = next;
  }
  return false;
}

// ---------------------------------------------------------------- few rows
// A lane's share of a weight tile (16 outputs x 128 inputs): its 32 weights and
// the scales and zeros of its output's groups.
template <int G>
struct Tile {
  static constexpr int NG = kTileK / G;
  u32x4 q;
  uint32_t scale[(NG + 1) / 2], zero;

  // tile: index among all weight tiles
  __device__ __forceinline__ void load(const W4Params &p, int64_t tile, int lane) {
    q = *(const u32x4 *)(p.q + (tile * 64 + lane) * 4);
    const int64_t at = (tile * 16 + (lane & 15)) * NG;
    if constexpr (NG == 1) {
      scale[0] = p.scale[at];
      zero = p.zero ? p.zero[at] : 8u;
    } else if constexpr (NG == 2) {
      scale[0] = *(const uint32_t *)(p.scale + at);
      zero = p.zero ? *(const uint16_t *)(p.zero + at) : 0x0808u;
    } else {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 v = *(const u32x2 *)(p.scale + at);
      scale[0] = v[0];
      scale[1] = v[1];
      zero = p.zero ? *(const uint32_t *)(p.zero + at) : 0x08080808u;
    }
  }
  __device__ __forceinline__ int zero_of(int g) const { return (int)(zero >> (8 * g)) & 15; }
  __device__ __forceinline__ float scale_of(const W4Params &p, int g) const {
    const uint16_t v = (uint16_t)(scale[g >> 1] >> (16 * (g & 1)));
    const float sb = bf16_bits_to_f32(v), sh = f16_bits_to_f32(v);
    return p.scale_bf16 ? sb : sh;
  }
  // t of group g, a: x of the tile's 128 inputs
  template <bool BF16>
  __device__ __forceinline__ f32x4 group(const u32x4 (&a)[4], int g, const Masks &ms) const {
    const Zero<BF16> z(zero_of(g));
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < G / 32; ++c)
      t = mfma<BF16>(a[g * (G / 32) + c], weights_of(q[g * (G / 32) + c], z, ms), t);
    return t;
  }
};

// The x operand of 128 inputs from input k on, of the row at xr (which points
// at this lane's 8 kg): pieces past K read the first one again (their groups do
// not exist).
__device__ __forceinline__ void load_x(const uint16_t *xr, int k, int K, u32x4 (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = *(const u32x4 *)(xr + k + (k + 32 * i < K ? 32 * i : 0));
}

// Few rows and few tiles: the workgroup's 8 waves share the inputs of 16 outputs
// of up to 16 rows. A wave takes every eighth tile of a window, all of whose
// weights are asked for at once, and leaves each group's t in LDS; the
// workgroup's threads add them in order, one output value each. Bound by latency
// (offsets, weights, exchange): one row, 4096 -> 4096, groups of 128, 4.8 us; 8
// experts' rows, 4096 -> 1536, 10 us.
constexpr int kSplitWaves = 8, kSlots = 32;  // groups of a window

template <int G, bool BF16>
__global__ void __launch_bounds__(64 * kSplitWaves) w4_split_kernel(W4Params p) {
  constexpr int NG = kTileK / G;
  constexpr int U = kSlots / (kSplitWaves * NG);  // tiles of a wave in a window
  __shared__ f32x4 ts[kSlots][64];
  __shared__ float ss[kSlots][16];
  const int NT = (p.N + 15) / 16, KT = (p.K + kTileK - 1) / kTileK, groups = p.K / G;
  Item it;
  if (!find_item(p, 16, NT, it)) return;
  const int nt = it.block, row0 = it.row0, nrows = it.nrows;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, kg = lane >> 4;
  const int64_t tile0 = ((int64_t)it.expert * NT + nt) * KT;
  // rows past the last one read it again and are not stored
  const uint16_t *xr = p.x + (int64_t)(row0 + min(n, nrows - 1)) * p.ldx + 8 * kg;
  Tile<G> w[U];
  const Masks ms(BF16);
  auto load = [&](int kb) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      w[u].load(p, tile0 + min(kb + u * kSplitWaves + wave, KT - 1), lane);
  };
  load(0);
  float acc = 0.f;
  for (int kb = 0; kb < KT; kb += kSplitWaves * U) {
    u32x4 a[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
      load_x(xr, min(kb + u * kSplitWaves + wave, KT - 1) * kTileK, p.K, a[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int slot = (u * kSplitWaves + wave) * NG + g;
        ts[slot][lane] = w[u].template group<BF16>(a[u], g, ms);
        if (kg == 0) ss[slot][n] = w[u].scale_of(p, g);
      }
    }
    const int next = kb + kSplitWaves * U;
    if (next < KT) load(next);
    __syncthreads();
    const int have = min(kSlots, groups - kb * NG);
    if (threadIdx.x < 256) {
      const float *t = (const float *)ts + threadIdx.x;
      const float *s = (const float *)ss + ((threadIdx.x >> 2) & 15);
      if (have == kSlots) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) acc = fmaf(s[16 * i], t[256 * i], acc);
      } else {
        for (int i = 0; i < have; ++i) acc = fmaf(s[16 * i], t[256 * i], acc);
      }
    }
    if (next < KT) __syncthreads();
  }
  // thread 4 l + r holds lane l's value r: output l % 16 of row 4 (l / 16) + r
  const int col = 16 * nt + ((threadIdx.x >> 2) & 15);
  const int r = 4 * (threadIdx.x >> 6) + (threadIdx.x & 3);
  if (threadIdx.x < 256 && col < p.N && r < nrows)
    store_out(p, (int64_t)(row0 + r) * p.ldout + col, acc);
}

// ------------------------------------------------------------- many rows
// A workgroup of four waves has 128 rows x 256 outputs, a wave all rows of 64
// outputs, so that each weight is unpacked once in a workgroup. The tile's x
// (128 x 128 a step, 32 KB) goes from global memory to LDS, where all four waves
// read it; the next step's copies run while this one is multiplied. A wave keeps
// 128 sums a lane; t of a group lives for its MFMAs. Two workgroups to a CU (70 KB
// of LDS, 256 registers): one unpacks while the other multiplies. Bound by the
// issue of vector instructions beside the MFMAs (3 an MFMA in fp16 and groups of
// 128, 5.6 in bf16, groups of 64 with zeros): 4001 rows, 6144 -> 4096, 171 us (1180
// TFLOP/s; a product of 16-bit weights by the library 161) and 231 (870).
constexpr int kWideM = 128, kWideN = 256;
constexpr int kNT = kWideN / 64;  // output tiles of a wave

// Copy of 16 bytes a lane from base + voff to LDS, lane l's at lds + 16 l. The
// wait states: the compiler does not look for the hazard of a scalar register
// written just before a vector memory instruction inside inline asm.
__device__ __forceinline__ void copy_to_lds(uint32_t voff, const void *base, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 3\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(voff), "s"(base), "s"(lds)
      : "memory");
}
// The same for the first `lanes` lanes, without a branch.
__device__ __forceinline__ void copy_to_lds(uint32_t voff, const void *base, uint32_t lds,
                                            int lanes) {
  uint64_t saved;
  asm volatile(
      "s_mov_b64 %0, exec\n\t"
      "s_and_b64 exec, exec, %4\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 1\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b64 exec, %0"
      : "=&s"(saved)
      : "v"(voff), "s"(base), "s"(lds), "s"(lanes == 64 ? ~0ull : (1ull << lanes) - 1)
      : "memory", "scc");
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ const char *uniform(const void *p) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  return (const char *)(uintptr_t)(((uint64_t)uniform((uint32_t)(b >> 32)) << 32) |
                                   uniform((uint32_t)b));
}

// Stores a wave's sums of 16 MT rows x 16 J outputs through its own piece of LDS,
// two row tiles at a time, so that a lane stores 16 bytes of a row. Stored as the
// MFMA leaves them, two or four bytes a lane, 32768 pairs x 4096 in fp32 took 564
// us in all instead of 503.
template <int MT, int J>
struct Epilogue {
  static constexpr int kRound = MT < 2 ? MT : 2;      // row tiles at a time
  static constexpr int kRow = 64 * J + 16;  // rows 4 apart start 16 banks apart
  static constexpr int kBytes = 16 * kRound * kRow;
};
template <int MT, int J>
__device__ __forceinline__ void store_tile(const W4Params &p, const Item &it, int first_tile,
                                           const f32x4 (&acc)[MT][J], char *lds) {
  using E = Epilogue<MT, J>;
  const int lane = threadIdx.x & 63, n = lane & 15, kg = lane >> 4;
  const int col0 = 16 * first_tile, rows = 16 * E::kRound;
#pragma unroll
  for (int m0 = 0; m0 < MT; m0 += E::kRound) {
    lds_exchange();
#pragma unroll
    for (int m = 0; m < E::kRound; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j)
          // + 0: a sum of only zeros that ended below the smallest subnormal is
          // +0 in every form (some add groups of zeros past K)
          *(float *)(lds + (16 * m + 4 * kg + r) * E::kRow + (16 * j + n) * 4) =
              acc[m0 + m][j][r] + 0.f;
    lds_exchange();
    if (p.out_dtype == 3) {
#pragma unroll
      for (int u = lane; u < rows * 4 * J; u += 64) {
        const int r = u / (4 * J), c = u % (4 * J) * 4, row = 16 * m0 + r;
        const f32x4 v = *(const f32x4 *)(lds + r * E::kRow + c * 4);
        if (row < it.nrows && col0 + c < p.N)
          *(f32x4 *)((float *)p.out + (int64_t)(it.row0 + row) * p.ldout + col0 + c) = v;
      }
    } else {
#pragma unroll
      for (int u = lane; u < rows * 2 * J; u += 64) {
        const int r = u / (2 * J), c = u % (2 * J) * 8, row = 16 * m0 + r;
        const f32x4 v = *(const f32x4 *)(lds + r * E::kRow + c * 4),
                    w = *(const f32x4 *)(lds + r * E::kRow + c * 4 + 16);
        u32x4 o;
        o[0] = f32x2_to_out16(v[0], v[1], p.out_dtype == 2);
        o[1] = f32x2_to_out16(v[2], v[3], p.out_dtype == 2);
        o[2] = f32x2_to_out16(w[0], w[1], p.out_dtype == 2);
        o[3] = f32x2_to_out16(w[2], w[3], p.out_dtype == 2);
        if (row < it.nrows && col0 + c < p.N)
          *(u32x4 *)((uint16_t *)p.out + (int64_t)(it.row0 + row) * p.ldout + col0 + c) = o;
      }
    }
  }
}

// Buffers of a workgroup in LDS: two steps of x, of each wave's scales (its 64
// outputs' groups) and zeros.
template <int G>
struct WideLds {
  static constexpr int NG = kTileK / G;
  static constexpr int kScales = 64 * NG * 2, kZeros = 64 * NG;
  static constexpr int kX = kWideM * kTileK * 2;
  static constexpr int kScaleOff = 2 * kX;
  static constexpr int kZeroOff = kScaleOff + 2 * 4 * kScales;
  static constexpr int kBytes = kZeroOff + 2 * 4 * kZeros;
  static_assert(kBytes <= 80 * 1024, "two workgroups per CU");
};

// A wave's part of a tile of up to 16 MT rows.
template <int G, bool BF16, int MT>
__device__ __forceinline__ void wide_tile(const W4Params &p, const Item &w, char *lds) {
  using L = WideLds<G>;
  constexpr int NG = L::NG, CH = G / 32;
  constexpr int MW = (MT + 3) / 4;  // row tiles that a wave copies
  const int NT = (p.N + 15) / 16, KT = (p.K + kTileK - 1) / kTileK;
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int first = w.block * (kWideN / 16) + wave * kNT;  // of the wave's output tiles
  const bool active = first < NT;  // a wave without outputs only copies
  const int nt0 = min(first, NT - 1), last = NT - 1 - nt0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const char *abase = uniform(p.x + (int64_t)w.row0 * p.ldx);
  const int64_t wtile = ((int64_t)w.expert * NT + nt0) * KT;
  // a tile's scales are 2 NG pieces of 16 bytes, its zeros NG
  const char *sbase = uniform(p.scale + wtile * 16 * NG);
  const char *zbase = p.zero ? uniform(p.zero + wtile * 16 * NG) : sbase;  // not used then
  // copies of step kt into buffer kt % 2
  auto copies = [&](int kt, int lane) {
    const uint32_t soff =
        (uint32_t)(min(lane / (2 * NG), last) * KT * 32 * NG + lane % (2 * NG) * 16);
    const uint32_t zoff = (uint32_t)(min(lane / NG, last) * KT * 16 * NG + lane % NG * 16);
    const int chunks = (p.K - kt * kTileK) / 32, buf = kt & 1;
    const uint32_t at = lds0 + buf * L::kX + wave * MW * 4096;
    if (MT % 4 == 0 || wave * MW < MT) {
#pragma unroll
      for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // 8 rows of 128 bytes; a row's eight pieces stand where fragment reads
          // of 16 rows meet 16 different places. Rows past the last one read it
          // again and are not stored, pieces past K the row's first of the step.
          const int row = min((wave * MW + m) * 16 + 8 * h + (lane >> 3), w.nrows - 1);
          const uint32_t piece = (lane & 7) ^ (4 * h + (lane >> 4));
          const uint32_t voff = __umul24(row, (uint32_t)(2 * p.ldx)) + 16 * piece;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t from = voff + 128 * i;
            if (NG > 1) from = (int)(8 * i + piece) < 4 * chunks ? from : voff - 16 * piece;
            copy_to_lds(from, uniform(abase + (int64_t)kt * (2 * kTileK)),
                        uniform(at + m * 4096 + i * 2048 + h * 1024));
          }
        }
    }
    if (!active) return;
    copy_to_lds(soff, uniform(sbase + (int64_t)kt * 32 * NG),
                uniform(lds0 + L::kScaleOff + (buf * 4 + wave) * L::kScales), 8 * NG);
    copy_to_lds(zoff, uniform(zbase + (int64_t)kt * 16 * NG),
                uniform(lds0 + L::kZeroOff + (buf * 4 + wave) * L::kZeros), 4 * NG);
  };
  // Zeros over the pieces of the last step past K: groups past K add nothing.
  auto clear_past_k = [&](int kt) {
    const int chunks = (p.K - kt * kTileK) / 32;
    if (NG == 1 || chunks >= 4) return;
    for (int u = threadIdx.x; u < MT * 256; u += 256) {  // 16 bytes: row tile, i, row, piece
      const int r = u >> 3 & 15, i = u >> 7 & 1, piece = (u & 7) ^ (r >> 1);
      if (8 * i + piece >= 4 * chunks)
        *(u32x4 *)(lds + (kt & 1) * L::kX + (u >> 8) * 4096 + i * 2048 + r * 128 + (u & 7) * 16) =
            (u32x4){0, 0, 0, 0};
    }
    __syncthreads();
  };
  const char *qbase = uniform(p.q + wtile * 256);
  const Masks ms(BF16);
  u32x4 raw[kNT];
  auto load_weights = [&](int kt, int lane) {  // tile j's: KT steps of 1 KB
#pragma unroll
    for (int j = 0; j < kNT; ++j)
      raw[j] = *(gu32x4p)(qbase + ((int64_t)min(j, last) * KT + kt) * 1024 + 16 * lane);
  };

  f32x4 acc[MT][kNT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < kNT; ++j) acc[m][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  copies(0, lane);
  load_weights(0, lane);

  for (int kt = 0; kt < KT; ++kt) {
    // this step's copies have landed, everybody is done with the last step's
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (kt == KT - 1) clear_past_k(kt);
    const int buf = kt & 1;
    int lane = threadIdx.x & 63;  // addresses are formed from it anew, not kept
    asm volatile("" : "+v"(lane));
    const int n = lane & 15;
    if (kt + 1 < KT) copies(kt + 1, lane);
    if (!active) continue;
    const char *ss = lds + L::kScaleOff + (buf * 4 + wave) * L::kScales;
    const char *zs = lds + L::kZeroOff + (buf * 4 + wave) * L::kZeros;
    const uint32_t xs =
        buf * L::kX + (n >> 3) * 1024 + (n & 7) * 128 + (((lane >> 4) ^ (n >> 1)) & 7) * 16;
    u32x4 now[kNT];
#pragma unroll
    for (int j = 0; j < kNT; ++j) now[j] = raw[j];
    if (NG > 1 && kt + 1 < KT) load_weights(kt + 1, lane);
    // fragment f is x of piece f % CH of row tile f / CH % MT of group f / CH / MT;
    // four are in registers, a fragment's place is filled again once its last
    // MFMAs are issued. Output tiles go in pairs: while the MFMAs of one run, the
    // t of the pair before are added. The barriers hold the compiler to this
    // order: it would load earlier and keep more than there are registers for.
    constexpr int kFrags = 4 * MT;
    auto fragment = [&](int f) {
      const int c = f % CH, m = f / CH % MT, g = f / (CH * MT);
      const int i = g * CH + c;
      return *(const u32x4 *)(lds + (i & 1 ? xs ^ 64 : xs) + m * 4096 + (i >> 1) * 2048);
    };
    u32x4 a[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) a[f] = fragment(f);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sc[kNT];
      u32x4 b[kNT][CH];
      f32x4 t[2][2];  // of two pairs of output tiles: one is formed, one added
      auto add = [&](int m, int h, int v) {  // value v of 8 of pair h of row tile m
        const int j = 2 * h + v / 4, r = v % 4;
        acc[m][j][r] = fmaf(sc[j], t[h & 1][v / 4][r], acc[m][j][r]);
      };
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        const int at = (16 * j + n) * NG + g;
        const uint16_t v = ((const uint16_t *)ss)[at];
        const float sb = bf16_bits_to_f32(v), sh = f16_bits_to_f32(v);
        sc[j] = p.scale_bf16 ? sb : sh;
        const int zv = ((const uint8_t *)zs)[at] & 15;
        const Zero<BF16> z(p.zero ? zv : 8);
#pragma unroll
        for (int c = 0; c < CH; ++c) b[j][c] = weights_of(now[j][g * CH + c], z, ms);
      }
      if (NG == 1 && kt + 1 < KT) load_weights(kt + 1, lane);  // now that `raw` is free
      // MFMAs first: the other wave's unpacking fits between them
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < kNT / 2; ++h) {
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int f = (g * MT + m) * CH + c;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              f32x4 &to = t[h & 1][i];
              const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
              __builtin_amdgcn_sched_barrier(0);
              to = mfma<BF16>(a[f % 4], b[2 * h + i][c], c == 0 ? zero : to);
              __builtin_amdgcn_sched_barrier(0);
              // a part of the sums of the pair before
              if (m > 0 || h > 0) {
                const int pm = h > 0 ? m : m - 1, ph = h > 0 ? h - 1 : kNT / 2 - 1;
#pragma unroll
                for (int v = (2 * c + i) * (4 / CH); v < (2 * c + i + 1) * (4 / CH); ++v)
                  add(pm, ph, v);
              }
            }
            if (h == kNT / 2 - 1 && f + 4 < kFrags) {
              __builtin_amdgcn_sched_barrier(0);
              a[f % 4] = fragment(f + 4);
            }
          }
        }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < 8; ++v) add(MT - 1, kNT / 2 - 1, v);
      __builtin_amdgcn_s_setprio(0);
    }
  }
  __syncthreads();  // everybody is done with x
  static_assert(4 * Epilogue<MT, kNT>::kBytes <= 2 * L::kX, "fits where x was");
  if (active) store_tile<MT, kNT>(p, w, first, acc, lds + wave * Epilogue<MT, kNT>::kBytes);
}

template <int G, bool BF16>
__global__ void __launch_bounds__(256, 2) w4_wide_kernel(W4Params p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  Item w;
  if (!find_item(p, kWideM, (p.N + kWideN - 1) / kWideN, w)) return;
  if (w.nrows <= 32) wide_tile<G, BF16, 2>(p, w, lds);
  else if (w.nrows <= 64) wide_tile<G, BF16, 4>(p, w, lds);
  else wide_tile<G, BF16, 8>(p, w, lds);
}

// ----------------------------------------------------------- in between
// Tiles of 16 MT rows x 64 J outputs, four waves of 16 J outputs: enough tiles
// for the whole card where those of the wide kernel are too few, and less left
// empty by experts of a few rows. With one or two workgroups to a CU nothing
// hides a load but distance, so everything (x, weights, scales, zeros) goes
// through LDS in a ring of S steps, S - 1 of them under way. A step's copies are
// counted and the wait leaves the later steps' in flight, so nothing else in the
// loop may load from or store to global memory. Three steps: a fourth costs
// a workgroup to a CU (bf16, groups of 32, 61 rows x top-8 of 192 experts: 349 us
// instead of 313). Few rows are bound by memory: the same in fp16 263 to 299 us (4.5
// to 5.1 TB/s). One projection of few rows is bound by the latency of a step
// (0.55 us) times their number, whatever the rows of a tile: 64 rows of 4096 -> 4096,
// where a CU has one workgroup, 15 us at a floor of 1.9.
template <int G, int MT, int J, int S, int W>
struct MidLds {
  static constexpr int NG = kTileK / G;
  static constexpr int kX = MT * 4096, kQ = J * 1024, kScales = 16 * J * NG * 2,
                       kZeros = 16 * J * NG;  // x of the workgroup, the others of a wave
  static constexpr int kQOff = kX, kScaleOff = kQOff + W * kQ, kZeroOff = kScaleOff + W * kScales,
                       kStep = kZeroOff + W * kZeros;
  static constexpr int kBytes = S * kStep;
};

template <int G, bool BF16, int MT, int J, int S, int W>
__global__ void __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 4)))
w4_mid_kernel(W4Params p) {
  using L = MidLds<G, MT, J, S, W>;
  constexpr int NG = L::NG, CH = G / 32;
  constexpr int XB = (4 * MT + W - 1) / W;   // blocks of x (1 KB) that a wave copies
  constexpr int kCopies = XB + J + 2;  // of a wave and step
  static_assert((S - 2) * kCopies < 64, "vmcnt range");
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int NT = (p.N + 15) / 16, KT = (p.K + kTileK - 1) / kTileK, groups = p.K / G;
  Item it;
  if (!find_item(p, 16 * MT, (NT + W * J - 1) / (W * J), it)) return;
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  // waves past the last output work on the last ones and do not store
  const int first = (it.block * W + wave) * J, nt0 = min(first, NT - 1), last = NT - 1 - nt0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const int64_t wtile = ((int64_t)uniform(it.expert) * NT + nt0) * KT;
  const char *abase = uniform(p.x + (int64_t)it.row0 * p.ldx);
  const char *qbase = uniform(p.q + wtile * 256);
  const char *sbase = uniform(p.scale + wtile * 16 * NG);
  const char *zbase = p.zero ? uniform(p.zero + wtile * 16 * NG) : sbase;  // not used then
  const uint32_t soff =
      (uint32_t)(min(lane / (2 * NG), last) * KT * 32 * NG + lane % (2 * NG) * 16);
  const uint32_t zoff = (uint32_t)(min(lane / NG, last) * KT * 16 * NG + lane % NG * 16);
  uint32_t avoff[XB], piece[XB];
#pragma unroll
  for (int b = 0; b < XB; ++b) {  // see the wide kernel: block b of this wave, 8 rows x 128 bytes
    const int id = (wave * XB + b) % (4 * MT), m = id >> 2, h = id & 1;
    const int row = min(m * 16 + 8 * h + (lane >> 3), it.nrows - 1);
    piece[b] = (lane & 7) ^ (4 * h + (lane >> 4));
    avoff[b] = __umul24(row, (uint32_t)(2 * p.ldx));
  }
  auto copies = [&](int kt, int slot) {
    kt = min(kt, KT - 1);  // past the end: copied and not used, to keep the count
    const int chunks = (p.K - kt * kTileK) / 32;
    const uint32_t to = lds0 + slot * L::kStep;
#pragma unroll
    for (int b = 0; b < XB; ++b) {
      const int id = (wave * XB + b) % (4 * MT), i = id >> 1 & 1;
      // pieces past K read the row's first one again; their groups are not used
      const uint32_t at = (int)(8 * i + piece[b]) < 4 * chunks ? 128 * i + 16 * piece[b] : 0;
      copy_to_lds(avoff[b] + at, uniform(abase + (int64_t)kt * (2 * kTileK)),
                  uniform(to + (id >> 2) * 4096 + i * 2048 + (id & 1) * 1024));
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      copy_to_lds(16 * lane, uniform(qbase + ((int64_t)min(j, last) * KT + kt) * 1024),
                  uniform(to + L::kQOff + wave * L::kQ + j * 1024));
    copy_to_lds(soff, uniform(sbase + (int64_t)kt * 32 * NG),
                uniform(to + L::kScaleOff + wave * L::kScales), 2 * NG * J);
    copy_to_lds(zoff, uniform(zbase + (int64_t)kt * 16 * NG),
                uniform(to + L::kZeroOff + wave * L::kZeros), NG * J);
  };
  const Masks ms(BF16);
  f32x4 acc[MT][J];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[m][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < S - 1; ++s) copies(s, s);
  const uint32_t xat = (n >> 3) * 1024 + (n & 7) * 128 + ((kg ^ (n >> 1)) & 7) * 16;
  int slot = 0;
  for (int kt = 0; kt < KT; ++kt) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 2) * kCopies) : "memory");
    __syncthreads();  // this step is there, everybody is done with the one before
    copies(kt + S - 1, slot == 0 ? S - 1 : slot - 1);
    const char *step = lds + slot * L::kStep;
    slot = slot == S - 1 ? 0 : slot + 1;
    const char *ss = step + L::kScaleOff + wave * L::kScales;
    const char *zs = step + L::kZeroOff + wave * L::kZeros;
    u32x4 q[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
      q[j] = *(const u32x4 *)(step + L::kQOff + wave * L::kQ + j * 1024 + 16 * lane);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (NG > 1 && kt * NG + g >= groups) break;
      float sc[J];
      u32x4 b[J][CH];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int at = (16 * j + n) * NG + g;
        const uint16_t v = ((const uint16_t *)ss)[at];
        const float sb = bf16_bits_to_f32(v), sh = f16_bits_to_f32(v);
        sc[j] = p.scale_bf16 ? sb : sh;
        const int zv = ((const uint8_t *)zs)[at] & 15;
        const Zero<BF16> z(p.zero ? zv : 8);
#pragma unroll
        for (int c = 0; c < CH; ++c) b[j][c] = weights_of(q[j][g * CH + c], z, ms);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 t[J];
#pragma unroll
        for (int j = 0; j < J; ++j) t[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = g * CH + c;
          const u32x4 a = *(const u32x4 *)(step + (i & 1 ? xat ^ 64 : xat) + m * 4096 +
                                           (i >> 1) * 2048);
#pragma unroll
          for (int j = 0; j < J; ++j) t[j] = mfma<BF16>(a, b[j][c], t[j]);
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][j][r] = fmaf(sc[j], t[j][r], acc[m][j][r]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no copy may land from here on
  __syncthreads();
  using E = Epilogue<MT, J>;
  static_assert(W * E::kBytes <= L::kBytes, "fits where the ring was");
  store_tile<MT, J>(p, it, first, acc, lds + wave * E::kBytes);
}

// Calls K<group, bf16, V...>.
#define EXL3_W4_KERNEL(K, threads, lds, ...)                                                     \
  do {                                                                                           \
    if (q.group == 32) {                                                                         \
      if (q.bf16) K<32, true, ##__VA_ARGS__><<<blocks, threads, lds, st>>>(q);                   \
      else K<32, false, ##__VA_ARGS__><<<blocks, threads, lds, st>>>(q);                         \
    } else if (q.group == 64) {                                                                  \
      if (q.bf16) K<64, true, ##__VA_ARGS__><<<blocks, threads, lds, st>>>(q);                   \
      else K<64, false, ##__VA_ARGS__><<<blocks, threads, lds, st>>>(q);                         \
    } else {                                                                                     \
      if (q.bf16) K<128, true, ##__VA_ARGS__><<<blocks, threads, lds, st>>>(q);                  \
      else K<128, false, ##__VA_ARGS__><<<blocks, threads, lds, st>>>(q);                        \
    }                                                                                            \
  } while (0)

// Most tiles of tm rows that the call's rows can make.
int64_t most_tiles(const W4Params &p, int tm) {
  const int64_t full = p.rows / tm, experts = p.offset ? (p.E < p.rows ? p.E : p.rows) : 1;
  const int64_t most = full + experts;
  return most < p.rows ? most : p.rows;
}

// Launches of `f` over the tiles of tm rows, with `per` workgroups each: one,
// unless a launch cannot hold them (its threads are counted in 32 bits).
template <typename F>
hipError_t over_tiles(W4Params p, int tm, int per, F f) {
  const int64_t items = most_tiles(p, tm) * per, step = 1 << 22;
  for (p.first = 0; p.first < items; p.first += step) {
    f(p, (unsigned)(items - p.first < step ? items - p.first : step));
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

template <int MT, int J, int S, int W>
hipError_t mid(const W4Params &p, hipStream_t st) {
  return over_tiles(p, 16 * MT, (p.N + 16 * W * J - 1) / (16 * W * J),
                    [&](const W4Params &q, unsigned blocks) {
                      const int lds = q.group == 32   ? MidLds<32, MT, J, S, W>::kBytes
                                      : q.group == 64 ? MidLds<64, MT, J, S, W>::kBytes
                                                      : MidLds<128, MT, J, S, W>::kBytes;
                      EXL3_W4_KERNEL(w4_mid_kernel, 64 * W, lds, MT, J, S, W);
                    });
}

}  // namespace

// The form is chosen by how many rows an expert has (its tile should not stay
// half empty) and how many tiles there are for 256 CUs. us of the forms on either
// side of a border, fp16, groups of 128:
//   4096 -> 4096, one projection:
//     rows 4096: wide 122, <4, 2, 2, 8> 154; rows 2048: 83, 78
//     rows 1024: <4, 2, 2, 8> 52, <2, 2, 3, 4> 57; rows 512: 48, 33
//     rows 512: <2, 2, 3, 4> 33, <2, 1, 3, 4> 36; rows 256: 25, 23
//     rows 128: <2, 1, 3, 4> 18, <1, 1, 3, 4> 19; rows 64: 18, 15
//     rows 64: <1, 1, 3, 4> 15, split 22; rows 32: 15, 14
//   128 experts, top-8, 4096 -> 1536:
//     tokens 2048: wide 286, <4, 2, 2, 8> 318; tokens 1024: 197, 205; tokens 512: 139, 128
//     tokens 512: <4, 2, 2, 8> 128, <2, 2, 3, 4> 123; tokens 1024: 205, 224
//     tokens 256: <2, 2, 3, 4> 89, <1, 2, 3, 4> 102; tokens 128: 88, 80
//     tokens 16: <1, 2, 3, 4> 52, <1, 1, 3, 4> 58; tokens 2: 20, 20, split 20
//   16 experts, top-4, 2048 -> 1536, tokens 256: <2, 1, 3, 4> 21.1, <2, 2, 3, 4> 19.5
// At three of these points the rule takes the slower form: 512 and 1024 tokens of
// 128 experts (<4, 2, 2, 8>, by 4% each) and the last (by 8%).
hipError_t launch_w4(const W4Params &p, hipStream_t st) {
  // what the rows make when they spread evenly over the experts
  const int64_t experts = p.offset ? (p.E < p.rows ? p.E : p.rows) : 1;
  const int64_t each = (p.rows + experts - 1) / experts;
  auto tiles = [&](int tm, int tn) {
    return experts * ((each + tm - 1) / tm) * ((p.N + tn - 1) / tn);
  };
  if (p.ldx < (1 << 23)) {  // a tile's rows of x within 32 bits
    if (each >= 96 && tiles(128, 256) >= 384)
      return over_tiles(p, kWideM, (p.N + kWideN - 1) / kWideN,
                        [&](const W4Params &q, unsigned blocks) {
                          const int lds = q.group == 32   ? WideLds<32>::kBytes
                                          : q.group == 64 ? WideLds<64>::kBytes
                                                          : WideLds<128>::kBytes;
                          EXL3_W4_KERNEL(w4_wide_kernel, 256, lds);
                        });
    if (each >= 24 && tiles(64, 256) >= 256) return mid<4, 2, 2, 8>(p, st);
    if (each >= 12 && tiles(32, 128) >= 512) return mid<2, 2, 3, 4>(p, st);
    if (each >= 12 && tiles(32, 64) >= 256) return mid<2, 1, 3, 4>(p, st);
    if (tiles(16, 128) >= 512) return mid<1, 2, 3, 4>(p, st);
    if (tiles(16, 64) >= 256) return mid<1, 1, 3, 4>(p, st);
  }
  return over_tiles(p, 16, (p.N + 15) / 16, [&](const W4Params &q, unsigned blocks) {
    EXL3_W4_KERNEL(w4_split_kernel, 64 * kSplitWaves, 0);
  });
}
#undef EXL3_W4_KERNEL

}  // namespace exl3

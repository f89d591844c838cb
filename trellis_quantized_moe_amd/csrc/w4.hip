// Products with 4-bit weights and group scales, for the sorted rows of experts
// or for all rows of one projection:
//   out[p, n] = sum over groups g of s[n, g] t_g,
//   t_g       = sum over k in g of x[p, k] (q[n, k] - z[n, g])
// q - z is a whole number of at most 15 in size, exact in fp16 and bf16, so the
// weights enter the MFMA as they are and t_g is a sum of exact products in fp32;
// the scale is applied to t_g in fp32: out = fma(s_g, t_g, out), g ascending.
// No weight is rounded.
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
// fp16: 0x6400 | q is 1024 + q, and 1024 + z is taken off again, exactly.
// bf16 has no packed subtraction: through fp32, whose upper half is the value.
template <bool BF16>
__device__ __forceinline__ u32x4 weights_of(uint32_t w, int z) {
  u32x4 r;
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = (float)((int)(w >> (4 * i) & 15u) - z);
      const float hi = (float)((int)(w >> (4 * i + 16) & 15u) - z);
      r[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi),
                                   __builtin_bit_cast(uint32_t, lo), 0x07060302u);
    }
  } else {
    const _Float16 off = (_Float16)(float)(1024 + z);
    const f16x2 o2 = {off, off};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = (w >> (4 * i) & 0x000f000fu) | 0x64006400u;
      r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, m) - o2);
    }
  }
  return r;
}

__device__ __forceinline__ float scale_of(const W4Params &p, int64_t i) {
  return p.scale_bf16 ? bf16_bits_to_f32(p.scale[i]) : f16_bits_to_f32(p.scale[i]);
}

// A sum of only zeros that ended below the smallest subnormal is +0 in every
// form (some add groups of zeros past K).
__device__ __forceinline__ void store_out(const W4Params &p, int64_t at, float v) {
  v += 0.f;
  if (p.out_dtype == 3) ((float *)p.out)[at] = v;
  else ((uint16_t *)p.out)[at] = f32_to_out16(v, p.out_dtype == 2);
}

// Rows of tile `idx` of `tm` rows: tiles count up through the experts, each
// with ceil(rows / tm) of them. False past the last tile. Offsets are kept
// within the call's rows.
__device__ __forceinline__ bool find_tile(const W4Params &p, int tm, int idx, int &expert,
                                          int &row, int &nrows) {
  if (!p.offset) {
    expert = 0;
    row = idx * tm;
    nrows = min(tm, p.rows - row);
    return row < p.rows;
  }
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, cnt = 0;
    if (e < p.E) {
      lo = min(max(p.offset[e], 0), p.rows);
      cnt = max(min(max(p.offset[e + 1], 0), p.rows) - lo, 0);
    }
    const int mine = (cnt + tm - 1) / tm;
    int upto = mine;  // tiles of this window's experts up to this lane's
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int v = __shfl_up(upto, s, 64);
      upto += lane >= s ? v : 0;
    }
    const int rel = idx - base;
    const uint64_t hit = __ballot(rel < upto);
    if (hit) {
      const int l = __ffsll((long long)hit) - 1;
      const int first = __shfl(upto - mine, l, 64);
      const int lo_l = __shfl(lo, l, 64), cnt_l = __shfl(cnt, l, 64);
      expert = __builtin_amdgcn_readfirstlane(e0 + l);
      row = __builtin_amdgcn_readfirstlane(lo_l + (rel - first) * tm);
      nrows = __builtin_amdgcn_readfirstlane(min(tm, cnt_l - (rel - first) * tm));
      return true;
    }
    base += __shfl(upto, 63, 64);
  }
  return false;
}

// Few rows: a workgroup has 16 outputs of 16 MT rows, its waves take tiles of
// 128 inputs in turn and leave each group's t in LDS, from where the
// workgroup's threads add them in order, MT values each.
constexpr int kWaves = 4;

template <int MT, int G, bool BF16>
__global__ void __launch_bounds__(64 * kWaves) w4_rows_kernel(W4Params p) {
  constexpr int NG = kTileK / G;  // groups of a tile
  constexpr int CH = G / 32;      // MFMAs of a group
  __shared__ f32x4 ts[2][kWaves * NG][MT][64];
  __shared__ float ss[2][kWaves * NG][16];
  int expert, row0, nrows;
  const int NT = (p.N + 15) / 16, KT = (p.K + kTileK - 1) / kTileK, groups = p.K / G;
  const int nt = blockIdx.x % NT;
  if (!find_tile(p, 16 * MT, p.first_tile + blockIdx.x / NT, expert, row0, nrows)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, kg = lane >> 4;
  const int64_t tile0 = ((int64_t)expert * NT + nt) * KT;
  const uint16_t *xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)  // rows past the last one read it again and are not stored
    xr[m] = p.x + (int64_t)(row0 + min(16 * m + n, nrows - 1)) * p.ldx + 8 * kg;
  float acc[MT] = {};
  int buf = 0;
  for (int kb = 0; kb < KT; kb += kWaves, buf ^= 1) {
    const int kt = kb + wave;
    if (kt < KT) {
      const u32x4 q = *(const u32x4 *)(p.q + ((tile0 + kt) * 64 + lane) * 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (kt * NG + g >= groups) break;  // K ends inside the tile
        const int64_t si = ((tile0 + kt) * 16 + n) * NG + g;
        const int z = p.zero ? p.zero[si] & 15 : 8;
        f32x4 t[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) t[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int i = g * CH + c;
          const u32x4 b = weights_of<BF16>(q[i], z);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            t[m] = mfma<BF16>(*(const u32x4 *)(xr[m] + kt * kTileK + 32 * i), b, t[m]);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) ts[buf][wave * NG + g][m][lane] = t[m];
        if (kg == 0) ss[buf][wave * NG + g][n] = scale_of(p, si);
      }
    }
    __syncthreads();
    const int have = min(kWaves * NG, groups - kb * NG);
    for (int s = 0; s < have; ++s) {
      const float sc = ss[buf][s][(threadIdx.x >> 2) & 15];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[m] = fmaf(sc, ((const float *)ts[buf][s][m])[threadIdx.x], acc[m]);
    }
  }
  // thread 4 l + r holds lane l's value r: output l % 16 of row 4 (l / 16) + r
  const int col = 16 * nt + ((threadIdx.x >> 2) & 15);
  if (col >= p.N) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = 16 * m + 4 * (threadIdx.x >> 6) + (threadIdx.x & 3);
    if (r >= nrows) break;
    store_out(p, (int64_t)(row0 + r) * p.ldout + col, acc[m]);
  }
}

// ------------------------------------------------------------- many rows
// A workgroup of four waves has 128 rows x 256 outputs, a wave all rows of 64
// outputs, so that each weight is unpacked once in a workgroup. The tile's x
// (128 x 128 a step, 32 KB) goes from global memory to LDS in the order of the
// MFMA's operand (a fragment is 1 KB, lane by lane) and is read by all four
// waves; the next step's copies run while this one is multiplied. A wave keeps
// 128 sums a lane; t of a group lives for four MFMAs.
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
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ const char *uniform(const void *p) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  return (const char *)(uintptr_t)(((uint64_t)uniform((uint32_t)(b >> 32)) << 32) |
                                   uniform((uint32_t)b));
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

// What a wave of the wide kernel is given.
struct WideArgs {
  int expert, row0, nrows, nt0;  // nt0: first of its output tiles
};

// A wave's part of a tile of up to 16 MT rows.
template <int G, bool BF16, int MT>
__device__ __forceinline__ void wide_tile(const W4Params &p, const WideArgs &w, char *lds) {
  using L = WideLds<G>;
  constexpr int NG = L::NG, CH = G / 32;
  constexpr int MW = (MT + 3) / 4;  // row tiles that a wave copies
  const int NT = (p.N + 15) / 16, KT = (p.K + kTileK - 1) / kTileK;
  const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  const bool active = w.nt0 < NT;  // a wave without outputs only copies
  const int nt0 = min(w.nt0, NT - 1), last = NT - 1 - nt0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  uint32_t avoff[MW];
#pragma unroll
  for (int m = 0; m < MW; ++m) {  // rows past the last one read it again and are not stored
    const int r = min((wave * MW + m) * 16 + n, w.nrows - 1);
    avoff[m] = (uint32_t)((r * p.ldx + 8 * kg) * 2);
  }
  const char *abase = uniform(p.x + (int64_t)w.row0 * p.ldx);
  const int64_t wtile = ((int64_t)w.expert * NT + nt0) * KT;
  // a tile's scales are 2 NG pieces of 16 bytes, its zeros NG
  const uint32_t soff = (uint32_t)(min(lane / (2 * NG), last) * KT * 32 * NG + lane % (2 * NG) * 16);
  const uint32_t zoff = (uint32_t)(min(lane / NG, last) * KT * 16 * NG + lane % NG * 16);
  const char *sbase = uniform(p.scale + wtile * 16 * NG);
  const char *zbase = uniform(p.zero ? p.zero + wtile * 16 * NG : nullptr);
  // copies of step kt into buffer kt % 2; x past K is zeros, so that groups past
  // K add nothing
  auto copies = [&](int kt) {
    const int chunks = min(4, (p.K - kt * kTileK) / 32), buf = kt & 1;
    const int at = buf * L::kX + wave * MW * 4096;
    if (MT % 4 == 0 || wave * MW < MT) {
#pragma unroll
      for (int m = 0; m < MW; ++m)
        for (int i = 0; i < 4; ++i) {
          if (i < chunks)
            copy_to_lds(avoff[m], uniform(abase + (int64_t)kt * (2 * kTileK) + 64 * i),
                        uniform(lds0 + at + m * 4096 + i * 1024));
          else
            *(u32x4 *)(lds + at + m * 4096 + i * 1024 + lane * 16) = (u32x4){0, 0, 0, 0};
        }
    }
    if (!active) return;
    if (lane < 8 * NG)
      copy_to_lds(soff, uniform(sbase + (int64_t)kt * 32 * NG),
                  uniform(lds0 + L::kScaleOff + (buf * 4 + wave) * L::kScales));
    if (zbase && lane < 4 * NG)
      copy_to_lds(zoff, uniform(zbase + (int64_t)kt * 16 * NG),
                  uniform(lds0 + L::kZeroOff + (buf * 4 + wave) * L::kZeros));
  };
  const char *qbase = uniform(p.q + wtile * 256);
  const uint32_t lane16 = 16 * lane;
  u32x4 raw[kNT];
  auto load_weights = [&](int kt) {  // tile j's: KT steps of 1 KB
#pragma unroll
    for (int j = 0; j < kNT; ++j)
      raw[j] = *(const u32x4 *)(qbase + ((int64_t)min(j, last) * KT + kt) * 1024 + lane16);
  };

  f32x4 acc[MT][kNT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < kNT; ++j) acc[m][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  copies(0);
  load_weights(0);

  for (int kt = 0; kt < KT; ++kt) {
    // this step's copies have landed, everybody is done with the last step's
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int buf = kt & 1;
    if (kt + 1 < KT) copies(kt + 1);
    if (!active) continue;
    const char *ss = lds + L::kScaleOff + (buf * 4 + wave) * L::kScales;
    const char *zs = lds + L::kZeroOff + (buf * 4 + wave) * L::kZeros;
    const char *xs = lds + buf * L::kX + lane * 16;
    u32x4 now[kNT];
#pragma unroll
    for (int j = 0; j < kNT; ++j) now[j] = raw[j];
    if (kt + 1 < KT) load_weights(kt + 1);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sc[kNT];
      u32x4 b[kNT][CH];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        const int at = (16 * j + n) * NG + g;
        const uint16_t v = ((const uint16_t *)ss)[at];
        const float sb = bf16_bits_to_f32(v), sh = f16_bits_to_f32(v);
        sc[j] = p.scale_bf16 ? sb : sh;
        const int zv = ((const uint8_t *)zs)[at] & 15;
        const int z = p.zero ? zv : 8;
#pragma unroll
        for (int c = 0; c < CH; ++c) b[j][c] = weights_of<BF16>(now[j][g * CH + c], z);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        // keeps later rows' fragments from being loaded (and held) early
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        u32x4 a[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) a[c] = *(const u32x4 *)(xs + (m * 4 + g * CH + c) * 1024);
        f32x4 t[kNT];
#pragma unroll
        for (int j = 0; j < kNT; ++j) t[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < kNT; ++j) t[j] = mfma<BF16>(a[c], b[j][c], t[j]);
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][j][r] = fmaf(sc[j], t[j][r], acc[m][j][r]);
      }
    }
  }
  if (!active) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * m + 4 * kg + r;
      if (row >= w.nrows) continue;
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        const int col = 16 * (w.nt0 + j) + n;
        if (col < p.N) store_out(p, (int64_t)(w.row0 + row) * p.ldout + col, acc[m][j][r]);
      }
    }
  }
}

template <int G, bool BF16>
__global__ void __launch_bounds__(256, 2) w4_wide_kernel(W4Params p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int NB = (p.N + kWideN - 1) / kWideN;
  WideArgs w;
  if (!find_tile(p, kWideM, p.first_tile + blockIdx.x / NB, w.expert, w.row0, w.nrows)) return;
  w.nt0 = (blockIdx.x % NB) * (kWideN / 16) + (int)uniform(threadIdx.x >> 6) * kNT;
  if (w.nrows <= 32) wide_tile<G, BF16, 2>(p, w, lds);
  else if (w.nrows <= 64) wide_tile<G, BF16, 4>(p, w, lds);
  else wide_tile<G, BF16, 8>(p, w, lds);
}

template <int G>
void wide_of(const W4Params &p, unsigned blocks, hipStream_t st) {
  if (p.bf16) w4_wide_kernel<G, true><<<blocks, 256, WideLds<G>::kBytes, st>>>(p);
  else w4_wide_kernel<G, false><<<blocks, 256, WideLds<G>::kBytes, st>>>(p);
}
void wide_kernel(const W4Params &p, unsigned blocks, hipStream_t st) {
  if (p.group == 32) wide_of<32>(p, blocks, st);
  else if (p.group == 64) wide_of<64>(p, blocks, st);
  else wide_of<128>(p, blocks, st);
}

template <int MT, int G>
void rows_of(const W4Params &p, unsigned blocks, hipStream_t st) {
  if (p.bf16) w4_rows_kernel<MT, G, true><<<blocks, 64 * kWaves, 0, st>>>(p);
  else w4_rows_kernel<MT, G, false><<<blocks, 64 * kWaves, 0, st>>>(p);
}
template <int MT>
void rows_kernel(const W4Params &p, unsigned blocks, hipStream_t st) {
  if (p.group == 32) rows_of<MT, 32>(p, blocks, st);
  else if (p.group == 64) rows_of<MT, 64>(p, blocks, st);
  else rows_of<MT, 128>(p, blocks, st);
}

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
  const int64_t tiles = most_tiles(p, tm), step = (1 << 22) / per;
  for (int64_t first = 0; first < tiles; first += step) {
    p.first_tile = (int)first;
    f(p, (unsigned)((tiles - first < step ? tiles - first : step) * per));
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_w4(const W4Params &p, hipStream_t st) {
  const int64_t each = p.rows / (p.offset ? p.E : 1);  // rows of an expert
  if (each > 64 && p.ldx < (1 << 23))
    return over_tiles(p, kWideM, (p.N + kWideN - 1) / kWideN,
                      [&](const W4Params &q, unsigned blocks) { wide_kernel(q, blocks, st); });
  return over_tiles(p, 16, (p.N + 15) / 16,
                    [&](const W4Params &q, unsigned blocks) { rows_kernel<1>(q, blocks, st); });
}

}  // namespace exl3

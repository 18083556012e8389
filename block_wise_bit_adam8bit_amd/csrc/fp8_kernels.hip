// 8-bit floating point products with a power-of-two scale per block of 128, for gfx950:
// the quantizer and the matrix products of include/qopt_fp8.h.
//
// A product sums, over blocks b of 128, 2^(sa_b + sb_b) times the dot product of two runs
// of 128 e4m3 codes.  Two ways to form it:
//   * v_mfma_scale_f32_32x32x64_f8f6f4: 8-bit operands and their scale bytes go into the
//     matrix unit as they are.  It aligns the 64 products of a step to the largest of them
//     and keeps about 18 bits (measured against binary64: 1.2e-5 to 1.8e-5 of the result's
//     size), which is far inside a bf16 result's rounding (2^-8) but not a binary32 one's.
//   * v_mfma_f32_32x32x16_bf16 on the codes widened to bf16 (exact: e4m3 has 4 significant
//     bits), with the scale put into the widening.  Binary32 products and sums (measured
//     1e-8 to 2e-7), at half the rate: used where the result is binary32.
// Sustained from registers alone the first reaches 4.4-4.5 PFLOP/s here, the second 2.15.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "qopt_fp8.h"

namespace {

constexpr int kBlock = QOPT_FP8_BLOCK;
constexpr int kWave = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ block scales

// Scale byte e + 127 of a block with the largest finite magnitude amax (its binary32
// bits): the least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), so the exponent field less 8,
// and one more where the fraction lies above .75; at least 0, and 127 for a block of zeros.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int s = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 127u : static_cast<uint32_t>(s < 0 ? 0 : s);
}
// 2^-e and 2^e of a scale byte e + 127 (0 .. 247) as binary32; 2^-127 is subnormal.
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x400000u : s << 23);  // 255 gives infinity: see widen
}

// |x| for a block maximum: infinities and NaN do not count.
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Four values scaled by a power of two (exact; what falls below binary32's range is far
// below e4m3's least step) and rounded to e4m3, ties to even: 4 code bytes.  No finite
// value of a block exceeds 448 here, so nothing saturates; infinities and NaN come out
// as NaN codes.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return static_cast<uint32_t>(w);
}

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Eight consecutive elements of a row; those from `left` on are 0.
template <typename XT>
__device__ __forceinline__ void load8(const XT* p, bool wide, int64_t left, float x[8]) {
  if (wide && left >= 8) {
    if constexpr (sizeof(XT) == 4) {
      const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = a[j];
        x[4 + j] = b[j];
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_to_f32(a[j] & 0xFFFFu);
        x[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = 0.0f;
      if (j < left) {
        if constexpr (sizeof(XT) == 4) x[j] = p[j];
        else x[j] = bf16_to_f32(p[j]);
      }
    }
  }
}

// ------------------------------------------------------------------ quantizer

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t kp, kpt;  // bytes per row of codes and codes_t
  uint32_t wide;    // rows of x allow 16-byte loads
  uint32_t tiles;   // tiles along a row
};

// One workgroup per tile of 128 x 128: thread (r, c) of 16 x 16 holds rows 8r .. 8r + 7 of
// columns 8c .. 8c + 7, so every row of the tile is read in whole 16-byte pieces, a row's
// code bytes are 8 bytes per thread, and a column's 8 rows are one 8-byte write into the
// transposed tile in LDS.
template <typename XT, bool kTiles>
__global__ void __launch_bounds__(256) quantize_kernel(QuantArgs q) {
  __shared__ __align__(16) u32x2 tile[kBlock * 16];  // [column][16 groups of 8 rows]
  __shared__ uint32_t colmax[4][kBlock];
  const int t = threadIdx.x, c = t & 15, r = t >> 4, wave = t / kWave;
  const uint32_t tr = blockIdx.x / q.tiles, tc = blockIdx.x % q.tiles;
  const int64_t row0 = static_cast<int64_t>(tr) * kBlock;
  const int64_t col0 = static_cast<int64_t>(tc) * kBlock;
  const int64_t col = col0 + 8 * c;
  const XT* x = static_cast<const XT*>(q.x);
  float v[8][8];
  uint32_t rmax[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 8 * r + i;
    load8<XT>(x + (row < q.rows ? row : 0) * q.ldx + col, q.wide != 0,
              row < q.rows ? q.cols - col : 0, v[i]);
  }
  uint32_t cmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rmax[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = finite_magnitude(v[i][j]);
      rmax[i] = umax(rmax[i], m);
      cmax[j] = umax(cmax[j], m);
    }
  }
  const int64_t kb = q.kp / kBlock, kbt = q.kpt / kBlock;
  uint32_t rs[8], cs[8];
  if constexpr (kTiles) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, rmax[i]);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) m = umax(m, __shfl_xor(m, d));
    if ((t & 63) == 0) colmax[0][wave] = m;
    __syncthreads();
    m = umax(umax(colmax[0][0], colmax[0][1]), umax(colmax[0][2], colmax[0][3]));
    const uint32_t s = scale_byte(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) rs[i] = cs[i] = s;
    if (t == 0) {
      if (q.codes) q.scales[tr * kb + tc] = static_cast<uint8_t>(s);
      if (q.codes_t) q.scales_t[tc * kbt + tr] = static_cast<uint8_t>(s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int d = 1; d < 16; d *= 2) rmax[i] = umax(rmax[i], __shfl_xor(rmax[i], d));
      rs[i] = scale_byte(rmax[i]);
      const int64_t row = row0 + 8 * r + i;
      if (q.codes && c == i && row < q.rows)
        q.scales[row * kb + tc] = static_cast<uint8_t>(rs[i]);
    }
    if (q.codes_t) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cmax[j] = umax(cmax[j], __shfl_xor(cmax[j], 16));
        cmax[j] = umax(cmax[j], __shfl_xor(cmax[j], 32));
        if ((t & 63) < 16) colmax[wave][8 * c + j] = cmax[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = 8 * c + j;
        cs[j] = scale_byte(umax(umax(colmax[0][k], colmax[1][k]), umax(colmax[2][k], colmax[3][k])));
        if (r == j && col + j < q.cols)
          q.scales_t[(col + j) * kbt + tr] = static_cast<uint8_t>(cs[j]);
      }
    }
  }
  if (q.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + 8 * r + i;
      if (row < q.rows) {
        const float inv = inverse_scale(rs[i]);
        const u32x2 w = {encode4(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                         encode4(v[i][4], v[i][5], v[i][6], v[i][7], inv)};
        *reinterpret_cast<u32x2*>(q.codes + row * q.kp + col) = w;
      }
    }
  }
  if (q.codes_t) {
    // Group r of a column lies at place r ^ (column / 8): the 16 threads of one r write
    // 16 different columns at one j, and so to 16 different places (all 32 banks).
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float inv = inverse_scale(cs[j]);
      const u32x2 w = {encode4(v[0][j], v[1][j], v[2][j], v[3][j], inv),
                       encode4(v[4][j], v[5][j], v[6][j], v[7][j], inv)};
      tile[(8 * c + j) * 16 + (r ^ c)] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = i * 32 + t / 8, g = t & 7, sw = k >> 3;  // 16 bytes: groups 2g and 2g + 1
      const u32x2 lo = tile[k * 16 + ((2 * g) ^ sw)], hi = tile[k * 16 + ((2 * g + 1) ^ sw)];
      const u32x4 w = {lo.x, lo.y, hi.x, hi.y};
      if (col0 + k < q.cols)
        *reinterpret_cast<u32x4*>(q.codes_t + (col0 + k) * q.kpt + row0 + 16 * g) = w;
    }
  }
}

// ------------------------------------------------------------------ widening to bf16

// Eight codes (two dwords) as bf16 values times 2^e.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}
template <typename OT> __device__ __forceinline__ void store1(OT* p, float x) {
  if constexpr (sizeof(OT) == 4) *p = x;
  else *p = static_cast<uint16_t>(pack_bf16(x, 0.0f) & 0xFFFFu);
}

// ------------------------------------------------------------------ few rows

struct FewArgs {
  const void* x;
  int64_t m, k, ldx;
  const uint8_t *w, *ws;
  int64_t n, kp;
  int32_t kb, w_shift;
  void* out;
  int64_t ldo;
  uint32_t wide;
};

constexpr int kFewWaves = 8;

// x w^T for at most 16 * kFrags rows of x: the time of reading the weights.  A workgroup owns
// 16 rows of w; its waves take turns at the blocks of 128 along k, and their sums are added
// in LDS in the order of the waves.  Lane (r, h) holds 32 consecutive codes of weight row r,
// and quantizes the same 32 places of row r of x in registers (a block's maximum is a
// maximum over 4 lanes), so nothing but the weights is read from memory more than once per
// workgroup and there is no launch before this one.
template <typename XT, typename OT, int kFrags>
__global__ void __launch_bounds__(kFewWaves * kWave) few_rows_kernel(FewArgs g) {
  __shared__ f32x4 sums[kFewWaves][kFrags][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int r = lane & 15, h = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t wrow = n0 + r < g.n ? n0 + r : g.n - 1;
  const uint8_t* w = g.w + wrow * g.kp + h * 32;
  const uint8_t* ws = g.ws + (wrow >> g.w_shift) * g.kb;
  f32x4 acc[kFrags];
#pragma unroll
  for (int f = 0; f < kFrags; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int b = wave; b < g.kb; b += kFewWaves) {
    const u32x4 w0 = *reinterpret_cast<const u32x4*>(w + static_cast<int64_t>(b) * kBlock);
    const u32x4 w1 = *reinterpret_cast<const u32x4*>(w + static_cast<int64_t>(b) * kBlock + 16);
    const float wscale = scale_value(ws[b]);
    bf16x8 wv[4] = {widen(w0[0], w0[1], wscale), widen(w0[2], w0[3], wscale),
                    widen(w1[0], w1[1], wscale), widen(w1[2], w1[3], wscale)};
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const int64_t row = f * 16 + r, col = static_cast<int64_t>(b) * kBlock + h * 32;
      const XT* x = static_cast<const XT*>(g.x) + (row < g.m ? row : 0) * g.ldx + col;
      const int64_t left = row < g.m ? g.k - col : 0;
      float v[4][8];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        load8<XT>(x + 8 * i, g.wide != 0, left - 8 * i, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, finite_magnitude(v[i][j]));
      }
      m = umax(m, __shfl_xor(m, 16));
      m = umax(m, __shfl_xor(m, 32));
      const uint32_t s = scale_byte(m);
      const float inv = inverse_scale(s), xscale = scale_value(s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = encode4(v[i][0], v[i][1], v[i][2], v[i][3], inv);
        const uint32_t hi = encode4(v[i][4], v[i][5], v[i][6], v[i][7], inv);
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(lo, hi, xscale), wv[i], acc[f], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < kFrags; ++f) sums[wave][f][lane] = acc[f];
  __syncthreads();
  // acc[f][i] of lane (r, h) is row 16 f + 4 h + i, column r
  for (int e = threadIdx.x; e < kFrags * kWave; e += kFewWaves * kWave) {
    const int f = e / kWave, l = e & 63;
    f32x4 a = sums[0][f][l];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) a += sums[v][f][l];
    const int64_t col = n0 + (l & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = f * 16 + 4 * (l >> 4) + i;
      if (row < g.m && col < g.n) store1(static_cast<OT*>(g.out) + row * g.ldo + col, a[i]);
    }
  }
}

// ------------------------------------------------------------------ product

struct GemmArgs {
  const uint8_t *a, *as, *b, *bs;
  int64_t m, n;
  uint32_t kp;  // bytes per row of codes
  int32_t kb;   // blocks along k
  int32_t a_shift, b_shift;
  void* out;
  int64_t ldo;
  uint32_t wide;  // rows of out allow 16-byte stores
  uint32_t tiles_m, tiles_n;
};

// 16 codes-bytes of this lane's part of rows, from memory into LDS without passing through
// registers: lane l of the wave fills bytes 16 l .. 16 l + 15 from `lds` on.  Reads past the
// buffer's end give 0.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t src, uint8_t* lds, uint32_t lane_offset,
                                            uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)lds, 16, lane_offset, offset, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const uint8_t* p, int64_t row0,
                                                              int64_t rows, int64_t most, uint32_t kp) {
  const int64_t left = rows - row0 < most ? rows - row0 : most;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + row0 * kp), 0,
                                           static_cast<int>(static_cast<uint32_t>(left * kp)), 0x00027000);
}

// One workgroup per tile of kM x kN outputs, one step per block of 128 along k: the tiles'
// code rows (128 bytes each) are loaded into one of two LDS buffers while the other one is
// multiplied.  The 16-byte piece c of a row lies at place c ^ (row % 8), so that 8
// consecutive rows' reads of one piece touch all banks once.
template <int kM, int kN, int kWavesM, int kWavesN, bool kExact, typename OT>
__global__ void __launch_bounds__(kWavesM* kWavesN* kWave) gemm_kernel(GemmArgs g) {
  constexpr int kWaves = kWavesM * kWavesN;
  constexpr int kFm = kM / kWavesM / 32, kFn = kN / kWavesN / 32;  // fragments of 32 per wave
  constexpr int kRows = kM + kN;
  constexpr int kLoads = kRows / 8 / kWaves;                       // 8 rows per wave and load
  static_assert(kM % (8 * kWaves) == 0 && kN % (8 * kWaves) == 0, "whole loads per operand");
  __shared__ __align__(16) uint8_t lds[2][kRows * kBlock];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const uint32_t tile = blockIdx.x;
  const int64_t m0 = static_cast<int64_t>(tile % g.tiles_m) * kM;
  const int64_t n0 = static_cast<int64_t>(tile / g.tiles_m) * kN;
  const __amdgpu_buffer_rsrc_t ra = rows_buffer(g.a, m0, g.m, kM, g.kp);
  const __amdgpu_buffer_rsrc_t rb = rows_buffer(g.b, n0, g.n, kN, g.kp);
  const uint32_t piece = ((lane & 7) ^ (lane >> 3)) * 16;
  auto load_step = [&](int buf, int b) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (i * kWaves + wave) * 8;  // first of the 8 rows of this load
      const bool is_a = i * kWaves * 8 < kM;
      const uint32_t src_row = static_cast<uint32_t>((is_a ? row : row - kM) + (lane >> 3));
      load_to_lds(is_a ? ra : rb, &lds[buf][row * kBlock], src_row * g.kp + piece,
                  static_cast<uint32_t>(b) * kBlock);
    }
  };
  // scale bytes of this lane's rows
  const uint8_t* sa[kFm];
  const uint8_t* sb[kFn];
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    int64_t row = m0 + (wm * kFm + i) * 32 + (lane & 31);
    row = row < g.m ? row : g.m - 1;
    sa[i] = g.as + (row >> g.a_shift) * g.kb;
  }
#pragma unroll
  for (int j = 0; j < kFn; ++j) {
    int64_t row = n0 + (wn * kFn + j) * 32 + (lane & 31);
    row = row < g.n ? row : g.n - 1;
    sb[j] = g.bs + (row >> g.b_shift) * g.kb;
  }
  f32x16 acc[kFm][kFn];
#pragma unroll
  for (int i = 0; i < kFm; ++i)
#pragma unroll
    for (int j = 0; j < kFn; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int h = lane >> 5;
  const uint32_t frag = (lane & 31) * kBlock + (((2 * h) ^ (lane & 7)) << 4);
  load_step(0, 0);
  int ca[kFm], cb[kFn];
#pragma unroll
  for (int i = 0; i < kFm; ++i) ca[i] = sa[i][0];
#pragma unroll
  for (int j = 0; j < kFn; ++j) cb[j] = sb[j][0];
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  for (int b = 0; b < g.kb; ++b) {
    const int buf = b & 1;
    int na[kFm], nb[kFn];
    const int next = b + 1 < g.kb ? b + 1 : b;
    if (b + 1 < g.kb) load_step(buf ^ 1, next);
#pragma unroll
    for (int i = 0; i < kFm; ++i) na[i] = sa[i][next];
#pragma unroll
    for (int j = 0; j < kFn; ++j) nb[j] = sb[j][next];
    const uint8_t* pa = &lds[buf][wm * kFm * 32 * kBlock];
    const uint8_t* pb = &lds[buf][(kM + wn * kFn * 32) * kBlock];
#pragma unroll
    for (int s = 0; s < 2; ++s) {  // halves of 64 along k
      i32x4 fa[kFm][2], fb[kFn][2];
#pragma unroll
      for (int i = 0; i < kFm; ++i) {
        fa[i][0] = *reinterpret_cast<const i32x4*>(pa + i * 32 * kBlock + (frag ^ (s * 64)));
        fa[i][1] = *reinterpret_cast<const i32x4*>(pa + i * 32 * kBlock + (frag ^ (s * 64) ^ 16));
      }
#pragma unroll
      for (int j = 0; j < kFn; ++j) {
        fb[j][0] = *reinterpret_cast<const i32x4*>(pb + j * 32 * kBlock + (frag ^ (s * 64)));
        fb[j][1] = *reinterpret_cast<const i32x4*>(pb + j * 32 * kBlock + (frag ^ (s * 64) ^ 16));
      }
      if constexpr (kExact) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // 8 codes each, in the same places of both operands
          bf16x8 va[kFm], vb[kFn];
#pragma unroll
          for (int i = 0; i < kFm; ++i)
            va[i] = widen(fa[i][e >> 1][2 * (e & 1)], fa[i][e >> 1][2 * (e & 1) + 1], scale_value(ca[i]));
#pragma unroll
          for (int j = 0; j < kFn; ++j)
            vb[j] = widen(fb[j][e >> 1][2 * (e & 1)], fb[j][e >> 1][2 * (e & 1) + 1], scale_value(cb[j]));
#pragma unroll
          for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vb[j], va[i], acc[i][j], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
          for (int j = 0; j < kFn; ++j) {
            const i32x8 va = __builtin_shufflevector(fa[i][0], fa[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i32x8 vb = __builtin_shufflevector(fb[j][0], fb[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, acc[i][j], 0, 0, 0,
                                                                        cb[j], 0, ca[i]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < kFm; ++i) ca[i] = na[i];
#pragma unroll
    for (int j = 0; j < kFn; ++j) cb[j] = nb[j];
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }

  // Lane (r, h) holds row r of a fragment, columns 8 q + 4 h + (0 .. 3) for q = 0 .. 3.
  OT* out = static_cast<OT*>(g.out);
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    const int64_t row = m0 + (wm * kFm + i) * 32 + (lane & 31);
    const bool in = row < g.m;
    OT* po = out + (in ? row : 0) * g.ldo;
#pragma unroll
    for (int j = 0; j < kFn; ++j) {
      const int64_t col0 = n0 + (wn * kFn + j) * 32;
      if constexpr (sizeof(OT) == 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t col = col0 + 8 * q + 4 * h;
          const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                           acc[i][j][4 * q + 3]};
          if (in && g.wide && col + 4 <= g.n) {
            *reinterpret_cast<f32x4*>(po + col) = v;
          } else if (in) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (col + e < g.n) po[col + e] = v[e];
          }
        }
      } else {
        // the halves of the wave exchange what they hold of two q, so that each lane has 8
        // consecutive columns: 8 (q + h) on
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          uint32_t x[2], y[2];
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const uint32_t p0 = pack_bf16(acc[i][j][4 * q + 2 * d], acc[i][j][4 * q + 2 * d + 1]);
            const uint32_t p1 = pack_bf16(acc[i][j][4 * q + 4 + 2 * d], acc[i][j][4 * q + 4 + 2 * d + 1]);
            const auto sw = __builtin_amdgcn_permlane32_swap(p0, p1, false, false);
            x[d] = sw[0];
            y[d] = sw[1];
          }
          const int64_t col = col0 + 8 * (q + h);
          const u32x4 v = {x[0], x[1], y[0], y[1]};
          if (in && g.wide && col + 8 <= g.n) {
            *reinterpret_cast<u32x4*>(po + col) = v;
          } else if (in) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col + e < g.n) po[col + e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
}

// out = 0, for a product over nothing.
template <typename OT> __global__ void __launch_bounds__(256) zero_kernel(OT* out, int64_t m, int64_t n, int64_t ldo) {
  for (int64_t i = blockIdx.y; i < m; i += gridDim.y)
    for (int64_t j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) out[i * ldo + j] = OT(0);
}

// ------------------------------------------------------------------ host

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status() { return hipGetLastError() == hipSuccess ? QOPT_OK : QOPT_ELAUNCH; }
bool bad_dim(int64_t d) { return d < 0 || d > QOPT_FP8_MAX_DIM; }
bool bad_dtype(int d) { return d != QOPT_F32 && d != QOPT_BF16; }
bool bad_form(int f) { return f != QOPT_FP8_ROWS && f != QOPT_FP8_TILES; }
int64_t padded(int64_t d) { return ceil_div(d, kBlock) * kBlock; }

// Workgroups of 256 threads that one launch may hold (its threads are counted in 32 bits).
constexpr int64_t kMaxGrid = int64_t{1} << 23;

template <typename XT, bool kTiles> int launch_quantize(const QuantArgs& q, hipStream_t s) {
  const int64_t tiles = q.tiles * ceil_div(q.rows, kBlock);
  if (tiles > kMaxGrid) return QOPT_EINVAL;
  hipLaunchKernelGGL((quantize_kernel<XT, kTiles>), dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, q);
  return launch_status();
}

template <typename XT, typename OT> int launch_few(const FewArgs& g, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(g.n, 16)));
  if (g.m <= 16) hipLaunchKernelGGL((few_rows_kernel<XT, OT, 1>), grid, dim3(kFewWaves * kWave), 0, s, g);
  else hipLaunchKernelGGL((few_rows_kernel<XT, OT, 2>), grid, dim3(kFewWaves * kWave), 0, s, g);
  return launch_status();
}

template <int kM, int kN, int kWavesM, int kWavesN, bool kExact, typename OT>
int launch_gemm(GemmArgs g, hipStream_t s) {
  g.tiles_m = static_cast<uint32_t>(ceil_div(g.m, kM));
  g.tiles_n = static_cast<uint32_t>(ceil_div(g.n, kN));
  const int64_t tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  if (tiles > kMaxGrid) return QOPT_EINVAL;
  hipLaunchKernelGGL((gemm_kernel<kM, kN, kWavesM, kWavesN, kExact, OT>), dim3(static_cast<unsigned>(tiles)),
                     dim3(kWavesM * kWavesN * kWave), 0, s, g);
  return launch_status();
}

int check_out(const void* out, int64_t m, int64_t n, int64_t ldo, int out_dtype) {
  if (ldo < n) return QOPT_EINVAL;
  if (m == 0 || n == 0) return QOPT_OK;
  if (!out) return QOPT_EINVAL;
  return aligned(out, out_dtype == QOPT_F32 ? 4 : 2) ? QOPT_OK : QOPT_EALIGN;
}

int zero_out(void* out, int out_dtype, int64_t m, int64_t n, int64_t ldo, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(n < 65536 ? ceil_div(n, 256) : 256),
                  static_cast<unsigned>(m < 1024 ? m : 1024));
  if (out_dtype == QOPT_F32)
    hipLaunchKernelGGL(zero_kernel<float>, grid, dim3(256), 0, s, static_cast<float*>(out), m, n, ldo);
  else
    hipLaunchKernelGGL(zero_kernel<uint16_t>, grid, dim3(256), 0, s, static_cast<uint16_t*>(out), m, n, ldo);
  return launch_status();
}

}  // namespace

// ------------------------------------------------------------------ entry points

extern "C" int qopt_fp8_quantize(const void* x_dev, int dtype, int64_t rows, int64_t cols,
                                 int64_t ldx, int form, uint8_t* codes_dev, uint8_t* scales_dev,
                                 uint8_t* codes_t_dev, uint8_t* scales_t_dev, void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || ldx < cols) return QOPT_EINVAL;
  if (bad_dtype(dtype) || bad_form(form)) return QOPT_EUNSUPPORTED;
  if (rows == 0 || cols == 0) return QOPT_OK;
  if (!x_dev || (!codes_dev) != (!scales_dev) || (!codes_t_dev) != (!scales_t_dev) ||
      (!codes_dev && !codes_t_dev))
    return QOPT_EINVAL;
  const size_t size = dtype == QOPT_F32 ? 4 : 2;
  if (!aligned(x_dev, size) || !aligned(codes_dev, 16) || !aligned(codes_t_dev, 16)) return QOPT_EALIGN;
  const QuantArgs q = {x_dev, rows, cols, ldx, codes_dev, scales_dev, codes_t_dev, scales_t_dev,
                       padded(cols), padded(rows),
                       aligned(x_dev, 16) && (ldx * size) % 16 == 0 ? 1u : 0u,
                       static_cast<uint32_t>(ceil_div(cols, kBlock))};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == QOPT_F32)
    return form == QOPT_FP8_TILES ? launch_quantize<float, true>(q, s) : launch_quantize<float, false>(q, s);
  return form == QOPT_FP8_TILES ? launch_quantize<uint16_t, true>(q, s)
                                : launch_quantize<uint16_t, false>(q, s);
}

extern "C" int qopt_fp8_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes) {
  if (!bytes || bad_dim(m) || bad_dim(n) || bad_dim(k)) return QOPT_EINVAL;
  if (bad_dtype(out_dtype)) return QOPT_EUNSUPPORTED;
  *bytes = 0;
  return QOPT_OK;
}

extern "C" int qopt_fp8_matmul(const uint8_t* a_codes_dev, const uint8_t* a_scales_dev, int a_form,
                               const uint8_t* b_codes_dev, const uint8_t* b_scales_dev, int b_form,
                               int64_t m, int64_t n, int64_t k, void* out_dev, int out_dtype,
                               int64_t ldo, void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = qopt_fp8_matmul_workspace(m, n, k, out_dtype, &need);
  if (rc != QOPT_OK) return rc;
  if (bad_form(a_form) || bad_form(b_form)) return QOPT_EUNSUPPORTED;
  rc = check_out(out_dev, m, n, ldo, out_dtype);
  if (rc != QOPT_OK || m == 0 || n == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (k == 0) return zero_out(out_dev, out_dtype, m, n, ldo, s);
  if (!a_codes_dev || !a_scales_dev || !b_codes_dev || !b_scales_dev) return QOPT_EINVAL;
  if (!aligned(a_codes_dev, 16) || !aligned(b_codes_dev, 16) || !aligned(workspace_dev, 16)) return QOPT_EALIGN;
  if (need > 0 && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  const size_t osize = out_dtype == QOPT_F32 ? 4 : 2;
  const GemmArgs g = {a_codes_dev, a_scales_dev, b_codes_dev, b_scales_dev, m, n,
                      static_cast<uint32_t>(padded(k)), static_cast<int32_t>(ceil_div(k, kBlock)),
                      a_form == QOPT_FP8_TILES ? 7 : 0, b_form == QOPT_FP8_TILES ? 7 : 0, out_dev, ldo,
                      aligned(out_dev, 16) && (ldo * osize) % 16 == 0 ? 1u : 0u, 0, 0};
  if (out_dtype == QOPT_F32) return launch_gemm<128, 128, 2, 2, true, float>(g, s);
  return launch_gemm<128, 128, 2, 2, false, uint16_t>(g, s);
}

extern "C" int qopt_fp8_linear_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes) {
  const int rc = qopt_fp8_matmul_workspace(m, n, k, out_dtype, bytes);
  if (rc != QOPT_OK) return rc;
  if (m <= QOPT_FP8_FEW_ROWS || n == 0) {
    *bytes = 0;
    return QOPT_OK;
  }
  // the codes of x, its scales (rounded up to 16 bytes), the product's own workspace
  *bytes += static_cast<size_t>(m) * padded(k) + static_cast<size_t>(ceil_div(m * (padded(k) / kBlock), 16)) * 16;
  return QOPT_OK;
}

extern "C" int qopt_fp8_linear(const void* x_dev, int dtype, int64_t m, int64_t k, int64_t ldx,
                               const uint8_t* w_codes_dev, const uint8_t* w_scales_dev, int w_form,
                               int64_t n, void* out_dev, int out_dtype, int64_t ldo,
                               void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = qopt_fp8_linear_workspace(m, n, k, out_dtype, &need);
  if (rc != QOPT_OK) return rc;
  if (ldx < k) return QOPT_EINVAL;
  if (bad_dtype(dtype) || bad_form(w_form)) return QOPT_EUNSUPPORTED;
  rc = check_out(out_dev, m, n, ldo, out_dtype);
  if (rc != QOPT_OK || m == 0 || n == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (k == 0) return zero_out(out_dev, out_dtype, m, n, ldo, s);
  if (!x_dev || !w_codes_dev || !w_scales_dev) return QOPT_EINVAL;
  const size_t size = dtype == QOPT_F32 ? 4 : 2;
  if (!aligned(x_dev, size) || !aligned(w_codes_dev, 16) || !aligned(workspace_dev, 16)) return QOPT_EALIGN;
  if (need > 0 && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  if (m > QOPT_FP8_FEW_ROWS) {
    uint8_t* codes = static_cast<uint8_t*>(workspace_dev);
    uint8_t* scales = codes + m * padded(k);
    rc = qopt_fp8_quantize(x_dev, dtype, m, k, ldx, QOPT_FP8_ROWS, codes, scales, nullptr, nullptr, stream);
    if (rc != QOPT_OK) return rc;
    const size_t used = static_cast<size_t>(m) * padded(k) +
                        static_cast<size_t>(ceil_div(m * (padded(k) / kBlock), 16)) * 16;
    return qopt_fp8_matmul(codes, scales, QOPT_FP8_ROWS, w_codes_dev, w_scales_dev, w_form, m, n, k, out_dev,
                           out_dtype, ldo, codes + used, workspace_bytes - used, stream);
  }
  const FewArgs g = {x_dev, m, k, ldx, w_codes_dev, w_scales_dev, n, padded(k),
                     static_cast<int32_t>(ceil_div(k, kBlock)), w_form == QOPT_FP8_TILES ? 7 : 0, out_dev, ldo,
                     aligned(x_dev, 16) && (ldx * size) % 16 == 0 ? 1u : 0u};
  if (dtype == QOPT_F32)
    return out_dtype == QOPT_F32 ? launch_few<float, float>(g, s) : launch_few<float, uint16_t>(g, s);
  return out_dtype == QOPT_F32 ? launch_few<uint16_t, float>(g, s) : launch_few<uint16_t, uint16_t>(g, s);
}

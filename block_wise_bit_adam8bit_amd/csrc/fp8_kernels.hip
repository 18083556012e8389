// 8-bit floating point products with a power-of-two scale per block of 128, for gfx950:
// the quantizer and the matrix products of include/qopt_fp8.h.
//
// A product sums, over blocks b of 128, 2^(sa_b + sb_b) times the dot product of two runs
// of 128 e4m3 codes.  Two ways to form it:
//   * v_mfma_scale_f32_32x32x64_f8f6f4: 8-bit operands and their scale bytes go into the
//     matrix unit as they are.  Measured, in this form and in 16x16x128: of every 8 products that
//     follow each other along the sum each is cut toward zero at 2^-13 of 2^E, E the largest sum of
//     two exponents among them (of codes under 2^-6: -6), and the eights are added in binary32.  So
//     8 places are off by less than 7 2^-13 2^E: nothing next to a bf16 result's rounding (2^-8) unless
//     products cancel (1.2e-5 to 1.8e-5 of the result's size on normal data; at most 2^-10 of the sum of
//     magnitudes, 1e-4 where positive values spread by e^2), but next to products of 256 * 256 that
//     cancel, 126 products of 1 came out as 120.
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
// 2^e of a scale byte e + 127 (0 .. 247) as binary32; 2^-127 is subnormal.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x400000u : s << 23);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t lane_xor(uint32_t x, int d) { return static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), d)); }

// Consecutive elements of a row as they are kept in registers: bf16 in pairs, binary32 by
// themselves.  `Max` is a running maximum of magnitudes over any of them: for bf16 of both halves
// of a register at once, as 16-bit integers, whose order is that of the magnitudes.  Infinities and
// NaN lie above every finite value and do not count for a block's scale; they are rare, so they
// are looked for once the maximum is known (`finite`), and only a block that holds one is gone
// over again (`finite_only`).
template <typename XT> struct Elements;

template <> struct Elements<uint16_t> {
  static constexpr int kPer = 2;  // elements per register
  typedef uint32_t Reg;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ uint32_t magnitude(uint32_t x) { return x & 0x7FFF7FFFu; }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  }
  static __device__ __forceinline__ uint32_t both(uint32_t m) { return max(m, m >> 16) & 0xFFFFu; }
  static __device__ __forceinline__ uint32_t finite_only(uint32_t x) {
    const uint32_t lo = x & 0x7FFFu, hi = x & 0x7FFF0000u;
    return (lo < 0x7F80u ? lo : 0u) | (hi < 0x7F800000u ? hi : 0u);
  }
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) { return m << 16; }
};

template <> struct Elements<float> {
  static constexpr int kPer = 1;
  typedef float Reg;
  static __device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) { return umax(a, b); }
  static __device__ __forceinline__ uint32_t both(uint32_t m) { return m; }
  static __device__ __forceinline__ uint32_t finite_only(float x) {
    const uint32_t u = magnitude(x);
    return u < kInf ? u : 0u;
  }
  static constexpr uint32_t kInf = 0x7F800000u;
  static __device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) { return m; }
};

// Four elements over a power of two, rounded to e4m3, ties to even: 4 code bytes.  One instruction
// per pair; it agrees with multiplying by 2^-e and rounding on every bf16 (checked on the hardware).
// No finite value of a block exceeds 448 2^e, so nothing saturates; infinities and NaN come out as
// NaN codes.
typedef short s16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t encode4(uint32_t ab, uint32_t cd, float scale) {
  s16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2, ab), scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2, cd), scale, true);
  return __builtin_bit_cast(uint32_t, w);
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float scale) {
  s16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

// Eight consecutive elements of a row, from an address of any element (the hardware reads 16 bytes
// at any alignment).
template <typename XT> __device__ __forceinline__ void load8(const XT* p, typename Elements<XT>::Reg (&x)[8 / Elements<XT>::kPer]) {
  __builtin_memcpy(x, p, sizeof(x));
}
// The same near a row's end, `left` elements on (any number): those from there on are 0.  No branch: the
// loads past the end read the row's last element instead.
template <typename XT>
__device__ __forceinline__ void load8_upto(const XT* p, int64_t left, typename Elements<XT>::Reg (&x)[8 / Elements<XT>::kPer]) {
  auto one = [&](int j) {
    const XT v = p[j < left ? j : left - 1];
    return j < left ? v : XT(0);
  };
#pragma unroll
  for (int j = 0; j < 8 / Elements<XT>::kPer; ++j) {
    if constexpr (sizeof(XT) == 4) x[j] = one(j);
    else x[j] = static_cast<uint32_t>(one(2 * j)) | static_cast<uint32_t>(one(2 * j + 1)) << 16;
  }
}

// ------------------------------------------------------------------ quantizer

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t kp, kpt;  // bytes per row of codes and codes_t
  int64_t sr, srt;  // bytes per block row of scales and scales_t
  uint32_t tiles;   // tiles along a row
};

// Rows r and r + 1 of one column of bf16 pairs, as a pair.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// One workgroup per tile of 128 x 128: thread (r, c) of 16 x 16 holds rows 8r .. 8r + 7 of
// columns 8c .. 8c + 7, so every row of the tile is read in whole 16-byte pieces, a row's
// code bytes are 8 bytes per thread, and a column's 8 rows are one 8-byte write into the
// transposed tile in LDS.  Reading x and writing the codes bounds it: both orientations of 8192 x 4096 in
// bf16 take 28.6 us and of 8192 x 11008 77 us (4.7 TB/s), one of 2048 x 4096 8 us, tiles of 11008 x 4096 with
// both 36 us (5.0 TB/s).  Reading x once for both is why one launch makes them; a tile kept in registers
// needs its maxima before any code, so nothing is read twice.
template <typename XT, bool kTiles>
__global__ void __launch_bounds__(256) quantize_kernel(QuantArgs q) {
  typedef Elements<XT> E;
  constexpr int kRegs = 8 / E::kPer;  // registers per 8 elements
  __shared__ __align__(16) u32x2 tile[kBlock * 16];  // [column][16 groups of 8 rows]
  __shared__ uint32_t colmax[4][kBlock];
  const int t = threadIdx.x, c = t & 15, r = t >> 4, wave = t / kWave;
  const uint32_t tr = blockIdx.x / q.tiles, tc = blockIdx.x % q.tiles;
  const int64_t row0 = static_cast<int64_t>(tr) * kBlock;
  const int64_t col0 = static_cast<int64_t>(tc) * kBlock;
  const int64_t col = col0 + 8 * c;
  const XT* x = static_cast<const XT*>(q.x);
  typename E::Reg v[8][kRegs];
  // rows past the last one: that one's values at first
  auto row_at = [&](int i) {
    const int64_t row = row0 + 8 * r + i;
    return x + (row < q.rows ? row : q.rows - 1) * q.ldx + col;
  };
  if (col0 + kBlock <= q.cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<XT>(row_at(i), v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) load8_upto<XT>(row_at(i), q.cols - col, v[i]);
  }
  if (row0 + kBlock > q.rows) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < kRegs; ++j)
        if (row0 + 8 * r + i >= q.rows) v[i][j] = typename E::Reg(0);
  }
  uint32_t rmax[8], cmax[kRegs];  // cmax: of a pair of columns for bf16
  auto maxima = [&](auto magnitude) {
#pragma unroll
    for (int j = 0; j < kRegs; ++j) cmax[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      rmax[i] = 0;
#pragma unroll
      for (int j = 0; j < kRegs; ++j) {
        const uint32_t m = magnitude(v[i][j]);
        rmax[i] = E::max(rmax[i], m);
        cmax[j] = E::max(cmax[j], m);
      }
      rmax[i] = E::both(rmax[i]);
    }
  };
  maxima([](typename E::Reg e) { return E::magnitude(e); });
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = umax(top, rmax[i]);
  if (top >= E::kInf) maxima([](typename E::Reg e) { return E::finite_only(e); });
  uint32_t rs[8], cs[8];
  if constexpr (kTiles) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = umax(top, rmax[i]);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) top = umax(top, lane_xor(top, d));
    if ((t & 63) == 0) colmax[0][wave] = top;
    __syncthreads();
    top = umax(umax(colmax[0][0], colmax[0][1]), umax(colmax[0][2], colmax[0][3]));
    const uint32_t s = scale_byte(E::as_f32_bits(top));
#pragma unroll
    for (int i = 0; i < 8; ++i) rs[i] = cs[i] = s;
    if (t == 0) {
      if (q.codes) q.scales[tr * q.sr + tc] = static_cast<uint8_t>(s);
      if (q.codes_t) q.scales_t[tc * q.srt + tr] = static_cast<uint8_t>(s);
    }
  } else {
    if (q.codes) {
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int d = 1; d < 16; d *= 2) rmax[i] = umax(rmax[i], lane_xor(rmax[i], d));
        rs[i] = scale_byte(E::as_f32_bits(rmax[i]));
        mine = c == i ? rs[i] : mine;
      }
      const int64_t row = row0 + 8 * r + c;  // thread c of a row group stores row c's
      if (c < 8 && row < q.rows) q.scales[tc * q.sr + row] = static_cast<uint8_t>(mine);
    }
    if (q.codes_t) {
#pragma unroll
      for (int j = 0; j < kRegs; ++j) {
        cmax[j] = E::max(cmax[j], lane_xor(cmax[j], 16));
        cmax[j] = E::max(cmax[j], lane_xor(cmax[j], 32));
        if ((t & 63) < 16) colmax[wave][kRegs * c + j] = cmax[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kRegs; ++j) {
        const int k = kRegs * c + j;
        const uint32_t m = E::max(E::max(colmax[0][k], colmax[1][k]), E::max(colmax[2][k], colmax[3][k]));
        if constexpr (E::kPer == 2) {
          cs[2 * j] = scale_byte(m << 16);
          cs[2 * j + 1] = scale_byte(m & 0xFFFF0000u);
        } else {
          cs[j] = scale_byte(m);
        }
      }
      uint32_t mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine = r == j ? cs[j] : mine;
      if (r < 8 && col + r < q.cols) q.scales_t[tr * q.srt + col + r] = static_cast<uint8_t>(mine);
    }
  }
  if (q.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + 8 * r + i;
      if (row < q.rows) {
        const float scale = scale_value(rs[i]);
        u32x2 w;
        if constexpr (E::kPer == 2)
          w = u32x2{encode4(v[i][0], v[i][1], scale), encode4(v[i][2], v[i][3], scale)};
        else
          w = u32x2{encode4(v[i][0], v[i][1], v[i][2], v[i][3], scale),
                    encode4(v[i][4], v[i][5], v[i][6], v[i][7], scale)};
        *reinterpret_cast<u32x2*>(q.codes + row * q.kp + col) = w;
      }
    }
  }
  if (q.codes_t) {
    // Group r of a column lies at place r ^ (column / 8): the 16 threads of one r write
    // 16 different columns at one j, and so to 16 different places (all 32 banks).
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float scale = scale_value(cs[j]);
      u32x2 w;
      if constexpr (E::kPer == 2) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[i] = j & 1 ? high_halves(v[2 * i][j / 2], v[2 * i + 1][j / 2]) : low_halves(v[2 * i][j / 2], v[2 * i + 1][j / 2]);
        w = u32x2{encode4(p[0], p[1], scale), encode4(p[2], p[3], scale)};
      } else {
        w = u32x2{encode4(v[0][j], v[1][j], v[2][j], v[3][j], scale),
                  encode4(v[4][j], v[5][j], v[6][j], v[7][j], scale)};
      }
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

// Memory by 32-bit offsets; reads past its end give 0 and go nowhere.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}

struct FewArgs {
  const void* x;
  int64_t m, k, ldx;
  const uint8_t *w, *ws;
  int64_t n;
  uint32_t kp, ws_bytes;
  uint32_t ws_row, ws_block;  // distances between the scales of rows (>> w_shift) and of blocks
  int32_t kb, w_shift;
  void* out;
  int64_t ldo;
};

// Waves per workgroup: 8, but 4 where each holds most registers (measured, 4 and 8: 32 rows of
// 50257 x 2048 34.5 and 38.8 us, 1 row of 11008 x 4096 11.6 and 9.9 us).
constexpr int few_waves(int frags, int runs) { return frags == 2 && runs == 4 ? 4 : 8; }

// x w^T for at most 16 * kFrags rows of x: the time of reading the weights.  A workgroup owns
// 16 * kRuns rows of w; its waves take turns at the blocks of 128 along k, and their sums are added
// in LDS in the order of the waves.  Lane (r, h) holds 32 consecutive codes of weight row r, and
// quantizes the same 32 places of row r of x in registers (a block's maximum is a maximum over 4
// lanes), so there is no launch before this one.
// The weights' bytes bound it at the rate of memory; what a workgroup adds to that is reading x from
// the L2 and quantizing it anew.  Measured in a graph (bf16; 2.3 us of it the launch), one weight again and
// again, which stays in the last-level cache, and 1 GiB of weights in turn: 1 row of 4096 x 4096 5.2 and
// 6.5 us, 1 of 11008 x 4096 9.1 and 11.4 us (4.9 and 4.0 TB/s), 1 of 1024 x 8192, on 64 CUs, 7.4 and 9.0 us,
// 24 of 11008 x 4096 15.0 and 16.3 us, 7 of 50257 x 2048 21.4 and 22.4 us (4.8 and 4.6 TB/s), 32 of it
// 32.6 and 34.6 us.
// Nothing around the loads branches (the compiler would wait for each before the next): weights past
// the last row are read past the end of a buffer, as 0, and a lane without a row of x takes the last
// one's values, which no result uses.  What k has beyond whole blocks comes after the loop.
// The loads of one block per wave are on their way at a time: two or four register sets in turn cost
// more waves per SIMD than they hid (1 row of 4096 x 4096 6.4 us, 6.5 with two, 7.9 with four; 16 rows
// 8.4 and 9.0; 1 row of 11008 x 4096 9.5 and 11.2).
template <typename XT, typename OT, int kFrags, int kRuns>
__global__ void __launch_bounds__(few_waves(kFrags, kRuns) * kWave) few_rows_kernel(FewArgs g) {
  typedef Elements<XT> E;
  typedef typename E::Reg Reg;
  constexpr int kFewWaves = few_waves(kFrags, kRuns);
  constexpr int kRegs = 32 / E::kPer;
  constexpr bool kExact = sizeof(OT) == 4;
  __shared__ f32x4 sums[kFewWaves][kFrags * kRuns][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, h = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * kRuns);
  const int64_t rows = g.n - n0 < 16 * kRuns ? g.n - n0 : 16 * kRuns;
  const __amdgpu_buffer_rsrc_t bs = buffer(g.ws, g.ws_bytes);
  const __amdgpu_buffer_rsrc_t bw = buffer(g.w + n0 * g.kp, static_cast<uint32_t>(rows * g.kp));
  const int whole = static_cast<int>(g.k / kBlock);  // blocks
  uint32_t ws[kRuns];
  const XT* xs[kFrags];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) ws[i] = (static_cast<uint32_t>(n0 + 16 * i + r) >> g.w_shift) * g.ws_row;
#pragma unroll
  for (int f = 0; f < kFrags; ++f)
    xs[f] = static_cast<const XT*>(g.x) + (f * 16 + r < g.m ? f * 16 + r : g.m - 1) * g.ldx + h * 32;
  f32x4 acc[kFrags][kRuns];
#pragma unroll
  for (int f = 0; f < kFrags; ++f)
#pragma unroll
    for (int i = 0; i < kRuns; ++i) acc[f][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  struct Block {
    Reg x[kFrags][kRegs];
    i32x4 c[kRuns][2];
    uint32_t s[kRuns];
  };
  auto load_weights = [&](Block& v, int b) {
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const uint32_t at = (16 * i + r) * g.kp + static_cast<uint32_t>(b) * kBlock + h * 32;
      v.c[i][0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(bw, at, 0, 0));
      v.c[i][1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(bw, at, 16, 0));
      v.s[i] = __builtin_amdgcn_raw_buffer_load_b8(bs, ws[i] + static_cast<uint32_t>(b) * g.ws_block, 0, 0);
    }
  };
  auto load = [&](Block& v, int b) {
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
      __builtin_memcpy(v.x[f], xs[f] + static_cast<int64_t>(b) * kBlock, sizeof(v.x[f]));
    load_weights(v, b);
  };
  auto multiply = [&](const Block& v) {
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const auto& x = v.x[f];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kRegs; ++i) m = E::max(m, E::magnitude(x[i]));
      m = E::both(m);
      if (m >= E::kInf) {
        m = 0;
#pragma unroll
        for (int i = 0; i < kRegs; ++i) m = E::max(m, E::finite_only(x[i]));
        m = E::both(m);
      }
      m = umax(m, lane_xor(m, 16));
      m = umax(m, lane_xor(m, 32));
      const uint32_t s = scale_byte(E::as_f32_bits(m));
      const float scale = scale_value(s);
      uint32_t code[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (E::kPer == 2) code[i] = encode4(x[2 * i], x[2 * i + 1], scale);
        else code[i] = encode4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], scale);
      }
      if constexpr (kExact) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bf16x8 xv = widen(code[2 * e], code[2 * e + 1], scale);
#pragma unroll
          for (int i = 0; i < kRuns; ++i) {
            const bf16x8 wv = widen(v.c[i][e >> 1][2 * (e & 1)], v.c[i][e >> 1][2 * (e & 1) + 1], scale_value(v.s[i]));
            acc[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv, acc[f][i], 0, 0, 0);
          }
        }
      } else {
        i32x8 xv;
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[i] = static_cast<int>(code[i]);
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
          const i32x8 wv = __builtin_shufflevector(v.c[i][0], v.c[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xv, wv, acc[f][i], 0, 0, 0, s, 0, v.s[i]);
        }
      }
    }
  };
  Block set;
  for (int b = wave; b < whole; b += kFewWaves) {
    load(set, b);
    multiply(set);
  }
  if (whole < g.kb && wave == whole % kFewWaves) {
    const int64_t col = static_cast<int64_t>(whole) * kBlock;
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Reg part[8 / E::kPer];
        load8_upto<XT>(xs[f] + col + 8 * i, g.k - col - h * 32 - 8 * i, part);
#pragma unroll
        for (int j = 0; j < 8 / E::kPer; ++j) set.x[f][8 / E::kPer * i + j] = part[j];
        __builtin_amdgcn_sched_barrier(0);  // eight at a time: all of them would cost the loop its registers
      }
    load_weights(set, whole);
    multiply(set);
  }
#pragma unroll
  for (int f = 0; f < kFrags; ++f)
#pragma unroll
    for (int i = 0; i < kRuns; ++i) sums[wave][f * kRuns + i][lane] = acc[f][i];
  __syncthreads();
  // acc[f][i][e] of lane (r, h) is row 16 f + 4 h + e, column 16 i + r
  for (int a = threadIdx.x; a < kFrags * kRuns * kWave; a += kFewWaves * kWave) {
    const int p = a / kWave, l = a & 63;
    f32x4 v = sums[0][p][l];
#pragma unroll
    for (int u = 1; u < kFewWaves; ++u) v += sums[u][p][l];
    const int64_t col = n0 + (p % kRuns) * 16 + (l & 15);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t row = (p / kRuns) * 16 + 4 * (l >> 4) + e;
      if (row < g.m && col < g.n) store1(static_cast<OT*>(g.out) + row * g.ldo + col, v[e]);
    }
  }
}

// ------------------------------------------------------------------ product

// f(i, j) for all i < kA, j < kB, with the numbers as types (for operands that are literals).
template <int kA, int kB, int kI = 0, typename F> __device__ __forceinline__ void each_pair(F&& f) {
  if constexpr (kI < kA * kB) {
    f(std::integral_constant<int, kI / kB>{}, std::integral_constant<int, kI % kB>{});
    each_pair<kA, kB, kI + 1>(f);
  }
}

struct GemmArgs {
  const uint8_t *a, *as, *b, *bs;
  int64_t m, n;
  uint32_t kp;                  // bytes per row of codes
  int32_t kb;                   // blocks along k
  uint32_t a_stride, b_stride;  // bytes between the scales of two blocks (kTilesB: of two tile rows)
  uint32_t as_bytes, bs_bytes;  // bytes of scales
  void* out;
  int64_t ldo;
  uint32_t tiles_m, tiles_n;
  uint32_t whole;               // big tiles that are taken whole; the others in halves
  uint32_t splits;
  int64_t split_stride;         // elements between the outputs of two splits
};

// Consecutive workgroups go to the 8 XCDs in turn, each with its own L2: with this order of `all`
// pieces of work every XCD takes one contiguous run of them ...
__device__ __forceinline__ uint32_t xcd_order(uint32_t wg, uint32_t all) {
  const uint32_t xcd = wg % 8, each = all / 8, more = all % 8;
  return xcd * each + (xcd < more ? xcd : more) + wg / 8;
}
// ... and the tiles are counted kGroup of them down before the next one across, so that those that an
// XCD has in work share rows of both operands.  Measured on 8192 x 11008 x 4096: against one run over
// all XCDs 6 % faster, groups of 8 against 4 another 3 %, 16 against 8 2 % slower.
constexpr uint32_t kGroup = 8;
struct TileAt {
  uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n) {
  const uint32_t group = t / (kGroup * tiles_n), left = tiles_m - group * kGroup;
  const uint32_t rows = left < kGroup ? left : kGroup, in = t % (kGroup * tiles_n);
  return {group * kGroup + in % rows, in / rows};
}

// The code rows of one tile: at most `most` of them, 2^31 bytes or less.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const uint8_t* p, int64_t row0,
                                                              int64_t rows, int64_t most, uint32_t kp) {
  const int64_t left = rows - row0 < most ? rows - row0 : most;
  return buffer(p + row0 * kp, static_cast<uint32_t>(left * kp));
}

// kCount (1, 2 or 4) consecutive scale bytes; reads past the buffer's end give 0.
template <int kCount>
__device__ __forceinline__ uint32_t load_scale_bytes(__amdgpu_buffer_rsrc_t src, uint32_t at) {
  if constexpr (kCount == 4) return __builtin_amdgcn_raw_buffer_load_b32(src, at, 0, 0);
  else if constexpr (kCount == 2) return __builtin_amdgcn_raw_buffer_load_b16(src, at, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b8(src, at, 0, 0);
}

// One tile of kM x kN outputs from row m0 and column n0 on, by one workgroup; one step per block of 128
// along k, steps `first` to `last`.
//
// A step's kM + kN rows of 128 codes are loaded from memory straight into one of kBufs LDS buffers
// (no registers), up to kBufs steps ahead; its fragments are read from LDS half a step ahead, into one of
// two register sets:
//     multiply half 0 of step t   | read half 1 of step t
//     wait: step t + 1 has landed, every wave has read all of step t (one barrier per step)
//     multiply half 1 of step t   | read half 0 of step t + 1, start loading step t + kBufs
// with the LDS reads and loads spread between the matrix instructions, which take 64 cycles each
// (reads issued ahead of them in one go kept the matrix units waiting: 4 % slower).
//
// A wave's fragment i of 32 rows holds rows kF * r + i (r = 0 .. 31), so that the scales of a lane's
// fragments are consecutive bytes: one load per operand and step, of which the matrix instruction
// picks its byte.  (A byte load per fragment from scales laid out row by row touched 32 cache lines
// each and cost a third of the time: 8192 x 4096 x 11008 at 1.7 PFLOP/s instead of 2.3.)  It also
// leaves each lane with kFn * 4 consecutive columns of the result.
// In LDS a fragment's 32 rows follow each other, and the 16-byte piece c of row r lies at place
// c ^ (r / 2 % 8): 16 lanes that read one piece of their rows touch all 64 banks once.  (Rows in the
// operand's order leave half of the banks to any one read: 1024 x 2048 x 4096 17.0 us instead of 16.4, 4096^3
// 56.3 and 54.7, 11008 x 4096 x 8192 312 and 308; but 8192 x 4096 x 11008 300 and 308, also with another
// conflict-free layout whose loads read 8 rows that follow each other.)
//
// Measured (8-bit, 256 x 256 tiles of 8 waves): 8192 x 4096 x 11008 in 293 to 308 us, 2.4 to 2.5 PFLOP/s,
// of which the matrix instructions alone take 206 us and the loads alone 280 us (193 us where the
// operands lie in the last-level cache); three and four steps of 64 in flight were no faster, and
// tiles of 4 waves of 128 x 128 6 % slower.
template <int kM, int kN, int kWavesM, int kWavesN, int kBufs, bool kExact, bool kTilesB, typename OT>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, uint8_t* lds, int64_t m0, int64_t n0, int first, int last,
                                          OT* out) {
  constexpr int kWaves = kWavesM * kWavesN;
  constexpr int kWm = kM / kWavesM, kWn = kN / kWavesN;  // a wave's part of the tile
  constexpr int kFm = kWm / 32, kFn = kWn / 32;          // fragments of 32 per wave
  constexpr int kRows = kM + kN;
  constexpr int kLoads = kRows / 8 / kWaves;             // 8 rows per wave and load
  static_assert(kM % (8 * kWaves) == 0 && kN % (8 * kWaves) == 0, "whole loads per operand");
  static_assert((kFm == 1 || kFm == 2 || kFm == 4) && (kFn == 1 || kFn == 2 || kFn == 4), "scale loads");
  static_assert(kBlock % kWn == 0 || !kTilesB, "a wave's columns lie in one tile of scales");
  static_assert(kWaves % (2 * kFm) == 0 && kWaves % (2 * kFn) == 0, "a wave's loads fill the same eight rows of 16");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const __amdgpu_buffer_rsrc_t ra = rows_buffer(g.a, m0, g.m, kM, g.kp);
  const __amdgpu_buffer_rsrc_t rb = rows_buffer(g.b, n0, g.n, kN, g.kp);
  // Lane l of a wave fills bytes 16 l .. 16 l + 15 of 8 rows in LDS, which are kF apart in the operand;
  // kF waves together read 8 kF rows that follow each other.  A row past the operand's last one lies past its buffer's
  // end and reads as 0.
  const uint32_t piece_a = ((lane & 7) ^ ((wave / kFm & 1) * 4 + (lane >> 4))) * 16;
  const uint32_t piece_b = ((lane & 7) ^ ((wave / kFn & 1) * 4 + (lane >> 4))) * 16;
  auto load_step = [&](int buf, int t) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool is_a = i * kWaves * 8 < kM;
      const int part = is_a ? kWm : kWn, frags = is_a ? kFm : kFn;
      const int at = (i * kWaves + wave) * 8 - (is_a ? 0 : kM);  // rows of the operand before this run's
      const int frag = at / 8 % frags, eight = at % part / (8 * frags);
      const int row = (is_a ? 0 : kM) + at / part * part + frag * 32 + eight * 8;  // its first row in LDS
      const uint32_t from = static_cast<uint32_t>(at / (8 * frags) * (8 * frags) + frag + frags * (lane >> 3)) * g.kp;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (lds_void*)(lds + (buf * kRows + row) * kBlock), 16,
                                               from + (is_a ? piece_a : piece_b), t * kBlock, 0, 0);
    }
  };

  const __amdgpu_buffer_rsrc_t rsa = buffer(g.as, g.as_bytes), rsb = buffer(g.bs, g.bs_bytes);
  const uint32_t sa = static_cast<uint32_t>(m0) + wm * kWm + kFm * (lane & 31);
  const uint32_t sb = kTilesB ? static_cast<uint32_t>((n0 + wn * kWn) / kBlock) * g.b_stride
                              : static_cast<uint32_t>(n0) + wn * kWn + kFn * (lane & 31);
  struct Scales {
    uint32_t a, b;  // byte i is fragment i's (kTilesB: byte 0 of b is every fragment's)
  };
  auto load_scales = [&](int t) {
    return Scales{load_scale_bytes<kFm>(rsa, sa + t * g.a_stride),
                  kTilesB ? load_scale_bytes<1>(rsb, sb + t) : load_scale_bytes<kFn>(rsb, sb + t * g.b_stride)};
  };

  const int h = lane >> 5;
  const uint32_t at = ((2 * h) ^ ((lane >> 1) & 7)) << 4;
  uint32_t oa = (wm * kWm + (lane & 31)) * kBlock + at;
  uint32_t ob = (kM + wn * kWn + (lane & 31)) * kBlock + at;
  struct Frags {
    i32x4 a[kFm][2], b[kFn][2];
  };
  auto read_half = [&](Frags& f, int buf, int half) {
    asm volatile("" : "+v"(oa), "+v"(ob));  // addresses are made anew, not kept in registers
    const uint32_t a0 = (oa ^ (half * 64)) + buf * (kRows * kBlock), b0 = (ob ^ (half * 64)) + buf * (kRows * kBlock);
#pragma unroll
    for (int j = 0; j < kFn; ++j) {
      f.b[j][0] = *reinterpret_cast<const i32x4*>(lds + b0 + j * (32 * kBlock));
      f.b[j][1] = *reinterpret_cast<const i32x4*>(lds + (b0 ^ 16) + j * (32 * kBlock));
    }
#pragma unroll
    for (int i = 0; i < kFm; ++i) {
      f.a[i][0] = *reinterpret_cast<const i32x4*>(lds + a0 + i * (32 * kBlock));
      f.a[i][1] = *reinterpret_cast<const i32x4*>(lds + (a0 ^ 16) + i * (32 * kBlock));
    }
  };

  f32x16 acc[kFm][kFn];
#pragma unroll
  for (int i = 0; i < kFm; ++i)
#pragma unroll
    for (int j = 0; j < kFn; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto multiply = [&](const Frags& f, const Scales& c) {
    if constexpr (kExact) {
      float va[kFm], vb[kFn];
#pragma unroll
      for (int i = 0; i < kFm; ++i) va[i] = scale_value((c.a >> (8 * i)) & 255);
#pragma unroll
      for (int j = 0; j < kFn; ++j) vb[j] = scale_value(kTilesB ? c.b : (c.b >> (8 * j)) & 255);
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // 8 codes each, in the same places of both operands
        bf16x8 wa[kFm], wb[kFn];
#pragma unroll
        for (int i = 0; i < kFm; ++i)
          wa[i] = widen(f.a[i][e >> 1][2 * (e & 1)], f.a[i][e >> 1][2 * (e & 1) + 1], va[i]);
#pragma unroll
        for (int j = 0; j < kFn; ++j)
          wb[j] = widen(f.b[j][e >> 1][2 * (e & 1)], f.b[j][e >> 1][2 * (e & 1) + 1], vb[j]);
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
          for (int j = 0; j < kFn; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
      }
    } else {
      each_pair<kFm, kFn>([&](auto i, auto j) {
        constexpr int I = decltype(i)::value, J = decltype(j)::value;
        const i32x8 wa = __builtin_shufflevector(f.a[I][0], f.a[I][1], 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 wb = __builtin_shufflevector(f.b[J][0], f.b[J][1], 0, 1, 2, 3, 4, 5, 6, 7);
        // formats 0: e4m3; the scale bytes are chosen by number
        acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wb, wa, acc[I][J], 0, 0, kTilesB ? 0 : J, c.b, I,
                                                                    c.a);
      });
    }
  };
  // The order of a half step's instructions: LDS reads and loads by threes between the matrix
  // instructions.
  constexpr int kMatrix = kFm * kFn * (kExact ? 4 : 1), kReads = 2 * (kFm + kFn);
  auto spread = [&](bool loads) {
#pragma unroll
    for (int i = 0; i < kMatrix; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < (kReads + 2) / 3) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
      if (loads) __builtin_amdgcn_sched_group_barrier(0x010, 3, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // All but the last kLater of this wave's loads have landed and its reads are done; then all waves'.
  constexpr int kLater = (kBufs - 2) * (kLoads + 2);
  constexpr int kFirst = kLater + kLoads;
  static_assert(kFirst < 64, "counts of loads under way");
  auto step_barrier = [&] {
    __builtin_amdgcn_s_waitcnt(0x0070 | (kLater & 15) | (kLater >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  auto upto_last = [&](int t) { return t < last ? t : last; };
  if constexpr (kBufs > 2) {
    // For tiles that have a CU to themselves and would wait for memory in every step: step t's loads are
    // issued kBufs - 1/2 steps ahead, its scales' kBufs - 1.  1024 x 2048 x 4096 (128 x 128, 128 CUs) takes
    // 17.2 us with three buffers, 23.8 with two and 17.2 with four; 4096 x 2048 x 8192 (128 x 256) 59.4 and
    // 67.8.  The exact path, which widens its operands meanwhile, gains nothing (30.0 and 30.1) and keeps
    // two.  Turns of kBufs steps, so that the registers of the scales have fixed places.
    Scales c[kBufs];
#pragma unroll
    for (int u = 0; u < kBufs; ++u) {
      if (u < kBufs - 1) c[u] = load_scales(upto_last(first + u));
      load_step(u, upto_last(first + u));
      __builtin_amdgcn_sched_barrier(0);
    }
    // of the loads behind step `first` one set of scales is not under way yet
    __builtin_amdgcn_s_waitcnt(0x0070 | (kFirst & 15) | (kFirst >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    Frags f0, f1;
    read_half(f0, 0, 0);
    for (int t = first; t <= last;) {
#pragma unroll
      for (int u = 0; u < kBufs; ++u) {
        constexpr int kLast = kBufs - 1;
        c[(u + kLast) % kBufs] = load_scales(upto_last(t + kLast));
        read_half(f1, u, 1);
        multiply(f0, c[u]);
        spread(false);
        step_barrier();
        asm volatile("" : "+v"(c[(u + 1) % kBufs].a), "+v"(c[(u + 1) % kBufs].b));
        read_half(f0, (u + 1) % kBufs, 0);
        load_step(u, upto_last(t + kBufs));
        multiply(f1, c[u]);
        spread(true);
        if (++t > last) break;
      }
    }
  } else {
    Scales c0 = load_scales(first), c1 = load_scales(upto_last(first + 1));
    load_step(0, first);
    __builtin_amdgcn_sched_barrier(0);
    step_barrier();
    load_step(1, upto_last(first + 1));
    if constexpr (kExact && kFm * kFn > 4) {
      // One register set: widened operands take the room of the second, and the other wave of the SIMD
      // works meanwhile.  8192 x 4096 x 11008 in 550 us, 1.34 PFLOP/s (594 us with tiles of 128 x 128; 570 us
      // with the widening spread between the matrix instructions).
      for (int t = first; t <= last; ++t) {
        const int buf = (t - first) & 1, ahead = upto_last(t + 2);
        Frags f;
        read_half(f, buf, 0);
        multiply(f, c0);
        __builtin_amdgcn_sched_barrier(0);
        read_half(f, buf, 1);
        multiply(f, c0);
        __builtin_amdgcn_sched_barrier(0);
        step_barrier();
        asm volatile("" : "+v"(c1.a), "+v"(c1.b));
        const Scales c2 = load_scales(ahead);
        load_step(buf, ahead);
        c0 = c1;
        c1 = c2;
      }
    } else {
      Frags f0, f1;
      read_half(f0, 0, 0);
      for (int t = first; t <= last; ++t) {
        // past the last step the last one is loaded again: no branch, which would keep the compiler from
        // spreading the loads
        const int buf = (t - first) & 1, ahead = upto_last(t + 2);
        read_half(f1, buf, 1);
        multiply(f0, c0);
        spread(false);
        step_barrier();
        asm volatile("" : "+v"(c1.a), "+v"(c1.b));  // not used before the wait that it landed with
        read_half(f0, buf ^ 1, 0);
        const Scales c2 = load_scales(ahead);
        load_step(buf, ahead);
        multiply(f1, c0);
        spread(true);
        c0 = c1;
        c1 = c2;
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // no load is on its way into LDS when the workgroup ends

  // Lane (r, h) holds row kFm r + i; its columns kFn (8 q + 4 h + e) + j for e = 0 .. 3 and all j are
  // consecutive.
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    const int64_t row = m0 + wm * kWm + kFm * (lane & 31) + i;
    if (row < g.m) {
      OT* po = out + row * g.ldo;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = n0 + wn * kWn + kFn * (8 * q + 4 * h);
        float v[4 * kFn];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < kFn; ++j) v[e * kFn + j] = acc[i][j][4 * q + e];
        if (col + 4 * kFn <= g.n) {  // 16 bytes at a time, at any alignment
          if constexpr (sizeof(OT) == 4) {
            __builtin_memcpy(po + col, v, sizeof(v));
          } else {
            uint32_t w[2 * kFn];
#pragma unroll
            for (int e = 0; e < 2 * kFn; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            __builtin_memcpy(po + col, w, sizeof(w));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4 * kFn; ++e)
            if (col + e < g.n) store1(po + col + e, v[e]);
        }
      }
    }
  }
}

// One workgroup per tile of 128 x 128 and split of k.
template <int kBufs, bool kExact, bool kTilesB, typename OT>
__global__ void __launch_bounds__(256) gemm_kernel(GemmArgs g) {
  __shared__ __align__(16) uint8_t lds[kBufs * 256 * kBlock];
  const uint32_t tiles = g.tiles_m * g.tiles_n, i = xcd_order(blockIdx.x, tiles * g.splits), split = i / tiles;
  const TileAt tile = tile_at(i % tiles, g.tiles_m, g.tiles_n);
  const int first = static_cast<int>(static_cast<int64_t>(g.kb) * split / g.splits);
  const int last = static_cast<int>(static_cast<int64_t>(g.kb) * (split + 1) / g.splits) - 1;
  gemm_tile<128, 128, 2, 2, kBufs, kExact, kTilesB, OT>(g, lds, tile.m * int64_t{128}, tile.n * int64_t{128}, first, last,
                                                 static_cast<OT*>(g.out) + split * g.split_stride);
}

// One workgroup per tile of 256 x 256, and two for each of those of the last round that would leave
// half of the CUs or more without work.
template <bool kExact, bool kTilesB, typename OT>
__global__ void __launch_bounds__(512) gemm_big_kernel(GemmArgs g) {
  constexpr int kHalfBufs = kExact ? 2 : 3;
  constexpr int kLds = 2 * 512 > kHalfBufs * 384 ? 2 * 512 : kHalfBufs * 384;
  __shared__ __align__(16) uint8_t lds[kLds * kBlock];
  OT* out = static_cast<OT*>(g.out);
  if (blockIdx.x < g.whole) {
    const TileAt tile = tile_at(xcd_order(blockIdx.x, g.whole), g.tiles_m, g.tiles_n);
    gemm_tile<256, 256, 2, 4, 2, kExact, kTilesB, OT>(g, lds, tile.m * int64_t{256}, tile.n * int64_t{256}, 0, g.kb - 1, out);
  } else {
    const uint32_t i = xcd_order(blockIdx.x - g.whole, gridDim.x - g.whole);
    const TileAt tile = tile_at(g.whole + i / 2, g.tiles_m, g.tiles_n);
    const int64_t m0 = tile.m * int64_t{256} + (i % 2) * 128;
    if (m0 < g.m)
      gemm_tile<128, 256, 2, 4, kHalfBufs, kExact, kTilesB, OT>(g, lds, m0, tile.n * int64_t{256}, 0, g.kb - 1, out);
  }
}

// out = the sum of `splits` binary32 partial results [m, ldp], in their order.
template <typename OT>
__global__ void __launch_bounds__(256) join_kernel(const float* part, int64_t m, int64_t n, int64_t ldp, int splits,
                                                   OT* out, int64_t ldo) {
  const int64_t quads = ldp / 4, all = m * quads;
  for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < all; i += gridDim.x * int64_t{256}) {
    const int64_t row = i / quads, col = (i % quads) * 4;
    const float* p = part + row * ldp + col;
    f32x4 v = *reinterpret_cast<const f32x4*>(p);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(p + s * m * ldp);
    OT* po = out + row * ldo + col;
    if (col + 4 <= n) {
      OT w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) store1(w + e, v[e]);
      __builtin_memcpy(po, w, sizeof(w));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < n) store1(po + e, v[e]);
    }
  }
}

// out = 0, for a product over nothing.
template <typename OT> __global__ void __launch_bounds__(256) zero_kernel(OT* out, int64_t m, int64_t n, int64_t ldo) {
  for (int64_t i = blockIdx.y; i < m; i += gridDim.y)
    for (int64_t j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) out[i * ldo + j] = OT(0);
}

// ------------------------------------------------------------------ host

// Workgroups that one launch may hold (its threads, at most 512 each, are counted in 32 bits).
constexpr int64_t kMaxGrid = int64_t{1} << 22;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status() { return hipGetLastError() == hipSuccess ? QOPT_OK : QOPT_ELAUNCH; }
bool bad_dim(int64_t d) { return d < 0 || d > QOPT_FP8_MAX_DIM; }
bool bad_dtype(int d) { return d != QOPT_F32 && d != QOPT_BF16; }
bool bad_form(int f) { return f != QOPT_FP8_ROWS && f != QOPT_FP8_TILES; }
int64_t padded(int64_t d) { return ceil_div(d, kBlock) * kBlock; }
// bytes between the scales of two blocks in QOPT_FP8_ROWS
int64_t scale_stride(int64_t rows) { return ceil_div(rows, 16) * 16; }
int64_t rows_scale_bytes(int64_t rows, int64_t cols) { return scale_stride(rows) * ceil_div(cols, kBlock); }
bool too_many_tiles(int64_t rows, int64_t cols) {
  return ceil_div(rows, kBlock) * ceil_div(cols, kBlock) > kMaxGrid;
}

template <typename XT, bool kTiles> int launch_quantize(const QuantArgs& q, hipStream_t s) {
  const int64_t tiles = q.tiles * ceil_div(q.rows, kBlock);
  hipLaunchKernelGGL((quantize_kernel<XT, kTiles>), dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, q);
  return launch_status();
}

template <typename XT, typename OT, int kRuns> int launch_few_runs(const FewArgs& g, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(g.n, 16 * kRuns))), block(few_waves(g.m <= 16 ? 1 : 2, kRuns) * kWave);
  if (g.m <= 16) hipLaunchKernelGGL((few_rows_kernel<XT, OT, 1, kRuns>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((few_rows_kernel<XT, OT, 2, kRuns>), grid, block, 0, s, g);
  return launch_status();
}

// More weight rows per workgroup let more of them share one reading of x, fewer fill the chip more
// evenly.  The time goes by what a CU has to read, per column of k: its rounds of workgroups times
// their rows of weights and of x.  Measured with 1 to 4 runs of 16, 1 GiB of weights in turn (us): 1 row of
// 4096 x 4096 6.4, 7.4, 9.1 and 10.7; 1 of 11008 x 4096 12.6, 14.1, 11.6 and 11.9; 24 of it 28.0, 24.7, 16.4 and
// 20.4; 7 of 50257 x 2048 29.4, 23.5, 22.4 and 23.5; 32 of it 73.2, 51.6, 44.0 and 34.5; the rule takes the
// least of each, and of the same calls with one weight again and again.
template <typename XT, typename OT> int launch_few(const FewArgs& g, hipStream_t s) {
  int runs = 1;
  int64_t least = 0;
  for (int r = 1; r <= 4; ++r) {
    const int64_t bytes = ceil_div(ceil_div(g.n, 16 * r), 256) * (16 * r + g.m * static_cast<int64_t>(sizeof(XT)));
    if (r == 1 || bytes < least) {
      least = bytes;
      runs = r;
    }
  }
  switch (runs) {
    case 1: return launch_few_runs<XT, OT, 1>(g, s);
    case 2: return launch_few_runs<XT, OT, 2>(g, s);
    case 3: return launch_few_runs<XT, OT, 3>(g, s);
    default: return launch_few_runs<XT, OT, 4>(g, s);
  }
}

// How a product is cut up: tiles of 256 x 256, `whole` of them whole and the others in halves, or (whole
// and halves 0) tiles of 128 x 128 with k in so many splits.
struct Plan {
  int64_t whole, halves;
  int splits;
};

// The plan of least time by this model, in microseconds on 256 CUs.  A step (128 along k) takes a CU
//   1.70 for one tile of 256 x 256 (2.52 PFLOP/s with all CUs busy), 0.92 for half of one,
//   1.06 for two tiles of 128 x 128 side by side (2.03), 0.70 for one, and 0.50 with three buffers, where
//   no CU has more than one; the exact path 3.2, 2.1, 1.67 and 0.96.
// Small tiles cost a quarter more per product but fill the chip at a quarter of the size: 1024 x 4096 x
// 4096 takes 18 us with them and 55 us with 64 whole tiles, 8192 x 4096 x 11008 363 us and 300 us.
// Splitting k, for products of too few tiles, adds a launch that joins the partial results (4) and
// their way to memory and back (4 TB/s).
Plan plan_for(int64_t m, int64_t n, int64_t k, bool exact) {
  const int64_t kb = ceil_div(k, kBlock);
  const int64_t small = ceil_div(m, 128) * ceil_div(n, 128), large = ceil_div(m, 256) * ceil_div(n, 256);
  const double two = exact ? 1.67 : 1.06, one = exact ? 0.96 : 0.70, alone = exact ? 0.96 : 0.50;
  Plan best = {0, 0, 1};
  double least = 0;
  for (int splits = 1; splits <= 16 && splits <= kb; splits *= 2) {
    const int64_t wgs = small * splits, steps = ceil_div(kb, splits);
    const int64_t rounds = wgs / 512, rest = wgs % 512;
    double us = static_cast<double>(steps) * (rounds * two + (rest == 0 ? 0.0 : rest > 256 ? two : rounds > 0 ? one : alone));
    if (splits > 1) us += 4.0 + static_cast<double>(splits) * m * n * 8 / 4e6;
    if (splits == 1 || us < least) {
      least = us;
      best.splits = splits;
    }
    if (wgs > 512) break;
  }
  const int64_t rest = large % 256, halved = rest <= 128 ? rest : 0;
  const double us = static_cast<double>(kb) * (ceil_div(large - halved, 256) * (exact ? 3.2 : 1.70) +
                                              (halved ? (exact ? 2.1 : 0.92) : 0.0));
  if (us <= least) best = {large - halved, 2 * halved, 1};
  return best;
}

int64_t partial_stride(int64_t n) { return ceil_div(n, 4) * 4; }

template <bool kExact, typename OT> int launch_gemm(GemmArgs g, bool b_tiles, hipStream_t s) {
  g.tiles_m = static_cast<uint32_t>(ceil_div(g.m, 128));
  g.tiles_n = static_cast<uint32_t>(ceil_div(g.n, 128));
  const int64_t wgs = static_cast<int64_t>(g.tiles_m) * g.tiles_n * g.splits;
  if (wgs > kMaxGrid) return QOPT_EINVAL;
  const dim3 grid(static_cast<unsigned>(wgs));
  if constexpr (!kExact) {
    if (wgs <= 256) {
      if (b_tiles) hipLaunchKernelGGL((gemm_kernel<3, kExact, true, OT>), grid, dim3(256), 0, s, g);
      else hipLaunchKernelGGL((gemm_kernel<3, kExact, false, OT>), grid, dim3(256), 0, s, g);
      return launch_status();
    }
  }
  if (b_tiles) hipLaunchKernelGGL((gemm_kernel<2, kExact, true, OT>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((gemm_kernel<2, kExact, false, OT>), grid, dim3(256), 0, s, g);
  return launch_status();
}

template <bool kExact, typename OT> int launch_gemm_big(GemmArgs g, const Plan& plan, bool b_tiles, hipStream_t s) {
  g.tiles_m = static_cast<uint32_t>(ceil_div(g.m, 256));
  g.tiles_n = static_cast<uint32_t>(ceil_div(g.n, 256));
  g.whole = static_cast<uint32_t>(plan.whole);
  const dim3 grid(static_cast<unsigned>(plan.whole + plan.halves));  // at most kMaxGrid tiles of 128 x 128
  if (b_tiles) hipLaunchKernelGGL((gemm_big_kernel<kExact, true, OT>), grid, dim3(512), 0, s, g);
  else hipLaunchKernelGGL((gemm_big_kernel<kExact, false, OT>), grid, dim3(512), 0, s, g);
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
  if (too_many_tiles(rows, cols)) return QOPT_EINVAL;
  if (!x_dev || (!codes_dev) != (!scales_dev) || (!codes_t_dev) != (!scales_t_dev) ||
      (!codes_dev && !codes_t_dev))
    return QOPT_EINVAL;
  const size_t size = dtype == QOPT_F32 ? 4 : 2;
  if (!aligned(x_dev, size) || !aligned(codes_dev, 16) || !aligned(codes_t_dev, 16)) return QOPT_EALIGN;
  const QuantArgs q = {x_dev, rows, cols, ldx, codes_dev, scales_dev, codes_t_dev, scales_t_dev,
                       padded(cols), padded(rows),
                       form == QOPT_FP8_TILES ? ceil_div(cols, kBlock) : scale_stride(rows),
                       form == QOPT_FP8_TILES ? ceil_div(rows, kBlock) : scale_stride(cols),
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
  if (m == 0 || n == 0 || k == 0) return QOPT_OK;
  if (too_many_tiles(m, k) || too_many_tiles(n, k) || too_many_tiles(m, n)) return QOPT_EINVAL;
  const Plan p = plan_for(m, n, k, out_dtype == QOPT_F32);
  if (p.splits > 1) *bytes = static_cast<size_t>(p.splits) * m * partial_stride(n) * sizeof(float);
  return QOPT_OK;
}

extern "C" int qopt_fp8_matmul(const uint8_t* a_codes_dev, const uint8_t* a_scales_dev,
                               const uint8_t* b_codes_dev, const uint8_t* b_scales_dev, int b_form,
                               int64_t m, int64_t n, int64_t k, void* out_dev, int out_dtype,
                               int64_t ldo, void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = qopt_fp8_matmul_workspace(m, n, k, out_dtype, &need);
  if (rc != QOPT_OK) return rc;
  if (bad_form(b_form)) return QOPT_EUNSUPPORTED;
  rc = check_out(out_dev, m, n, ldo, out_dtype);
  if (rc != QOPT_OK || m == 0 || n == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (k == 0) return zero_out(out_dev, out_dtype, m, n, ldo, s);
  if (!a_codes_dev || !a_scales_dev || !b_codes_dev || !b_scales_dev) return QOPT_EINVAL;
  if (!aligned(a_codes_dev, 16) || !aligned(b_codes_dev, 16) || !aligned(a_scales_dev, 4) ||
      !aligned(b_scales_dev, 4) || !aligned(workspace_dev, 16))
    return QOPT_EALIGN;
  if (need > 0 && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  const bool exact = out_dtype == QOPT_F32, tiles = b_form == QOPT_FP8_TILES;
  const Plan plan = plan_for(m, n, k, exact);
  const int64_t kb = ceil_div(k, kBlock);
  GemmArgs g = {};
  g.a = a_codes_dev;
  g.as = a_scales_dev;
  g.b = b_codes_dev;
  g.bs = b_scales_dev;
  g.m = m;
  g.n = n;
  g.kp = static_cast<uint32_t>(padded(k));
  g.kb = static_cast<int32_t>(kb);
  g.a_stride = static_cast<uint32_t>(scale_stride(m));
  g.b_stride = static_cast<uint32_t>(tiles ? kb : scale_stride(n));
  g.as_bytes = static_cast<uint32_t>(rows_scale_bytes(m, k));
  g.bs_bytes = static_cast<uint32_t>(tiles ? ceil_div(n, kBlock) * kb : rows_scale_bytes(n, k));
  g.splits = static_cast<uint32_t>(plan.splits);
  if (plan.splits > 1) {
    g.out = workspace_dev;
    g.ldo = partial_stride(n);
    g.split_stride = m * g.ldo;
    rc = exact ? launch_gemm<true, float>(g, tiles, s) : launch_gemm<false, float>(g, tiles, s);
    if (rc != QOPT_OK) return rc;
    const int64_t wgs = ceil_div(m * (g.ldo / 4), 256);
    const dim3 grid(static_cast<unsigned>(wgs < 4096 ? wgs : 4096));
    const float* part = static_cast<const float*>(workspace_dev);
    if (exact)
      hipLaunchKernelGGL(join_kernel<float>, grid, dim3(256), 0, s, part, m, n, g.ldo, plan.splits,
                         static_cast<float*>(out_dev), ldo);
    else
      hipLaunchKernelGGL(join_kernel<uint16_t>, grid, dim3(256), 0, s, part, m, n, g.ldo, plan.splits,
                         static_cast<uint16_t*>(out_dev), ldo);
    return launch_status();
  }
  g.out = out_dev;
  g.ldo = ldo;
  if (plan.whole + plan.halves > 0)
    return exact ? launch_gemm_big<true, float>(g, plan, tiles, s) : launch_gemm_big<false, uint16_t>(g, plan, tiles, s);
  return exact ? launch_gemm<true, float>(g, tiles, s) : launch_gemm<false, uint16_t>(g, tiles, s);
}

namespace {
// The codes of x and its scales at the start of qopt_fp8_linear's workspace, in multiples of 16 bytes.
size_t linear_codes_bytes(int64_t m, int64_t k) { return static_cast<size_t>(m) * padded(k); }
size_t linear_own_bytes(int64_t m, int64_t k) { return linear_codes_bytes(m, k) + rows_scale_bytes(m, k); }
}  // namespace

extern "C" int qopt_fp8_linear_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes) {
  const int rc = qopt_fp8_matmul_workspace(m, n, k, out_dtype, bytes);
  if (rc != QOPT_OK) return rc;
  if (m <= QOPT_FP8_FEW_ROWS || n == 0 || k == 0) *bytes = 0;
  else *bytes += linear_own_bytes(m, k);
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
  if (!aligned(x_dev, size) || !aligned(w_codes_dev, 16) || !aligned(w_scales_dev, 4) || !aligned(workspace_dev, 16))
    return QOPT_EALIGN;
  if (need > 0 && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  const bool tiles = w_form == QOPT_FP8_TILES;
  if (m > QOPT_FP8_FEW_ROWS) {
    uint8_t* codes = static_cast<uint8_t*>(workspace_dev);
    uint8_t* scales = codes + linear_codes_bytes(m, k);
    rc = qopt_fp8_quantize(x_dev, dtype, m, k, ldx, QOPT_FP8_ROWS, codes, scales, nullptr, nullptr, stream);
    if (rc != QOPT_OK) return rc;
    const size_t used = linear_own_bytes(m, k);
    return qopt_fp8_matmul(codes, scales, w_codes_dev, w_scales_dev, w_form, m, n, k, out_dev, out_dtype, ldo,
                           codes + used, workspace_bytes - used, stream);
  }
  const int64_t kb = ceil_div(k, kBlock);
  const FewArgs g = {x_dev, m, k, ldx, w_codes_dev, w_scales_dev, n, static_cast<uint32_t>(padded(k)),
                     static_cast<uint32_t>(tiles ? ceil_div(n, kBlock) * kb : rows_scale_bytes(n, k)),
                     static_cast<uint32_t>(tiles ? kb : 1), static_cast<uint32_t>(tiles ? 1 : scale_stride(n)),
                     static_cast<int32_t>(kb), tiles ? 7 : 0, out_dev, ldo};
  if (dtype == QOPT_F32)
    return out_dtype == QOPT_F32 ? launch_few<float, float>(g, s) : launch_few<float, uint16_t>(g, s);
  return out_dtype == QOPT_F32 ? launch_few<uint16_t, float>(g, s) : launch_few<uint16_t, uint16_t>(g, s);
}

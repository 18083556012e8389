// Microscaled 4-bit floating point for gfx950: the quantizer, its inverse and the matrix products
// of include/qopt_fp4.h.
//
// v_mfma_scale_f32_*_f8f6f4 takes 32 codes of a row per lane and the block's scale byte with them, so a
// block of 32 is one lane's operand.  Codes are multiples of 0.5 up to 6: the products of a block are
// multiples of 0.25 up to 36 and exact in the matrix unit, whatever the result's type.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "product_tile.h"
#include "qopt_fp4.h"

namespace {

using namespace product;

constexpr int kBlock = QOPT_FP4_BLOCK;
constexpr int kStep = 2 * kStepBytes;  // values per step of a product
static_assert(kStep == QOPT_FP4_PAD, "rows are padded to whole steps");

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ block scales

// Scale byte of a block with the largest magnitude amax (its binary32 bits): the least e with amax <=
// 6 * 2^e = 1.5 * 2^(e + 2), so the exponent field less 2, and one more where the fraction lies above .5;
// at least 0, 127 for a block of zeros, 255 where amax is an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int s = static_cast<int>(amax >> 23) - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return amax == 0 ? 127u : amax >= 0x7F800000u ? 255u : static_cast<uint32_t>(s < 0 ? 0 : s);
}
// 2^e of a scale byte e + 127 below 255 as binary32; 2^-127 is subnormal.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s == 0 ? 0x400000u : s << 23); }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t lane_xor(uint32_t x, int d) { return static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), d)); }

// Eight consecutive elements of a row as they are kept in registers: bf16 in pairs, binary32 by themselves.
template <typename XT> struct Eight {
  static constexpr int kRegs = 8 * sizeof(XT) / 4;
  uint32_t r[kRegs];
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// A running maximum of magnitudes over such registers, for bf16 of both halves at once as 16-bit integers, whose
// order is that of the magnitudes (infinities and NaN above all others); `as_f32_bits` ends it.
template <typename XT> __device__ __forceinline__ uint32_t max_of(uint32_t m, const Eight<XT>& x) {
#pragma unroll
  for (int i = 0; i < Eight<XT>::kRegs; ++i) {
    if constexpr (sizeof(XT) == 4)
      m = umax(m, x.r[i] & 0x7FFFFFFFu);
    else
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), __builtin_bit_cast(u16x2, x.r[i] & 0x7FFF7FFFu)));
  }
  return m;
}
template <typename XT> __device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) {
  return sizeof(XT) == 4 ? m : umax(m << 16, m & 0xFFFF0000u);
}

// Eight elements over a power of two, rounded to e2m1, ties to even: 4 code bytes.  No value of a block
// exceeds 6 2^e, so nothing saturates.
template <typename XT> __device__ __forceinline__ uint32_t encode8(const Eight<XT>& x, float scale) {
  uint32_t w = 0;
  if constexpr (sizeof(XT) == 4) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.r[0]), __uint_as_float(x.r[1]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.r[2]), __uint_as_float(x.r[3]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.r[4]), __uint_as_float(x.r[5]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.r[6]), __uint_as_float(x.r[7]), scale, 3);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.r[0]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.r[1]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.r[2]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, x.r[3]), scale, 3);
  }
  return w;
}

// Eight elements from p on, an address of any element (the hardware reads 16 bytes at any alignment).
template <typename XT> __device__ __forceinline__ Eight<XT> load8(const XT* p) {
  Eight<XT> x;
  __builtin_memcpy(&x, p, sizeof(x));
  return x;
}
// The same near a row's end, `left` elements on (any number): those from there on are 0, and the loads past
// the end read the row's last element instead.
template <typename XT> __device__ __forceinline__ Eight<XT> load8_upto(const XT* p, int64_t left) {
  XT one[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const XT v = p[j < left ? j : left - 1];
    one[j] = j < left ? v : XT(0);
  }
  Eight<XT> x;
  __builtin_memcpy(&x, one, sizeof(x));
  return x;
}

// ------------------------------------------------------------------ quantizer

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t* codes;
  uint32_t* scales;
  int64_t kp, rp;
  uint32_t across;  // workgroups along a row
};

// Reading x bounds it: 11008 x 4096 in bf16 take 21 us (5.5 TB/s, in part from the last-level cache), 8192 x 4096 18 us.
// A workgroup takes 16 rows of 512 columns, a wave four of the rows one after the other: a lane holds 8
// elements and four lanes a block, so a row is read in whole 1 KB pieces (bf16) and its codes written in 256
// bytes.  The scales of 16 rows and 128 columns, 64 bytes that lie together, meet in LDS.
template <typename XT> __global__ void __launch_bounds__(256) quantize_kernel(QuantArgs q) {
  __shared__ uint32_t words[4][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / q.across) * 16;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x % q.across) * 512, col = col0 + 8 * lane;
  const XT* x = static_cast<const XT*>(q.x);
  Eight<XT> v[4];
  auto row_at = [&](int i) {
    const int64_t row = row0 + 4 * wave + i;
    return x + (row < q.rows ? row : q.rows - 1) * q.ldx;
  };
  if (col0 + 512 <= q.cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load8(row_at(i) + col);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // columns behind the row's end: any element of the row, counted as 0
      const int64_t at = col < q.cols ? col : 0;
      v[i] = load8_upto(row_at(i) + at, col < q.cols ? q.cols - col : 1);
      if (col >= q.cols) v[i] = Eight<XT>{};
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * wave + i;
    uint32_t m = as_f32_bits<XT>(max_of<XT>(0, v[i]));
    m = umax(m, lane_xor(m, 1));
    m = umax(m, lane_xor(m, 2));
    const uint32_t s = row < q.rows ? scale_byte(m) : 127u;
    // the scales of a word's four blocks, each in four lanes
    uint32_t word = s << (8 * (lane >> 2 & 3));
    word |= lane_xor(word, 4);
    word |= lane_xor(word, 8);
    if ((lane & 15) == 0) words[lane >> 4][4 * wave + i] = word;
    const uint32_t w = s == 255 ? 0u : encode8<XT>(v[i], scale_value(s));
    if (row < q.rows && col < q.kp) *reinterpret_cast<uint32_t*>(q.codes + row * (q.kp / 2) + col / 2) = w;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t i = col0 / 128 + (threadIdx.x >> 4), row = row0 + (threadIdx.x & 15);
    if (i * 128 < q.kp) q.scales[i * q.rp + row] = words[threadIdx.x >> 4][threadIdx.x & 15];
  }
}

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, kp, rp;
  void* out;
  int64_t ldo;
  uint32_t across;
};

// Sixteen rows of 512 columns per workgroup, as above: a lane turns 4 code bytes into 8 values.  Writing them bounds it:
// 11008 x 4096 to bf16 take 18 us (6.4 TB/s).
template <typename OT> __global__ void __launch_bounds__(256) dequantize_kernel(DequantArgs q) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / q.across) * 16;
  const int64_t col = static_cast<int64_t>(blockIdx.x % q.across) * 512 + 8 * lane;
  if (col >= q.cols) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * wave + i;
    if (row >= q.rows) return;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q.codes + row * (q.kp / 2) + col / 2);
    const uint32_t s = q.scales[(col / 128 * q.rp + row) * 4 + (col / 32 & 3)];
    const float scale = s == 255 ? __uint_as_float(0x7FC00000u) : scale_value(s);
    float v[8];
    each<4>([&](auto j) {
      constexpr int J = decltype(j)::value;
      const auto pair = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, J);
      v[2 * J] = pair[0] * scale;
      v[2 * J + 1] = pair[1] * scale;
    });
    OT* po = static_cast<OT*>(q.out) + row * q.ldo + col;
    if (col + 8 <= q.cols) {
      OT o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) store1(o + j, v[j]);
      __builtin_memcpy(po, o, sizeof(o));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < q.cols) store1(po + j, v[j]);
    }
  }
}

// ------------------------------------------------------------------ few rows

struct FewArgs {
  const void* x;
  int64_t m, k, ldx;
  const uint8_t *w, *ws;
  int64_t n;
  uint32_t kp2, ws_bytes;  // bytes per row of codes
  uint32_t ws_group;       // bytes between the scales of two runs of 128 columns
  int32_t steps;
  void* out;
  int64_t ldo;
};

// Waves per workgroup: 8, but 4 where each holds most registers and LDS (32 rows of 50257 x 2048 30 us with 8 and 27
// with 4, at four runs of weight rows; 24 of 11008 x 4096, three runs, 12.0 and 12.5).
constexpr int few_waves(int frags, int runs) { return frags == 2 && runs >= 4 ? 4 : 8; }

// x w^T for at most 16 * kFrags rows of x: the time of reading the weights.  A workgroup owns 16 * kRuns rows
// of w; its waves take turns at the steps of 256 along k, and their sums are added in LDS in the order of the
// waves.  Of a step's two halves of 128 lane (r, h) holds the block of 32 codes h of weight row r, and
// quantizes the same 32 places of row r of x in registers: a block is one lane's, so its maximum needs no
// other lane, and there is no launch before this one.
// Nothing around the loads branches (the compiler would wait for each before the next): weights past the last
// row are read past the end of a buffer, as 0, and a lane without a row of x takes the last one's values,
// which no result uses.  What k has beyond whole steps comes after the loop.
template <typename XT, typename OT, int kFrags, int kRuns>
__global__ void __launch_bounds__(few_waves(kFrags, kRuns) * kWave) few_rows_kernel(FewArgs g) {
  constexpr int kFewWaves = few_waves(kFrags, kRuns);
  __shared__ f32x4 sums[kFewWaves][kFrags * kRuns][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, h = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * kRuns);
  const int64_t rows = g.n - n0 < 16 * kRuns ? g.n - n0 : 16 * kRuns;
  const __amdgpu_buffer_rsrc_t bs = buffer(g.ws, g.ws_bytes);
  const __amdgpu_buffer_rsrc_t bw = buffer(g.w + n0 * g.kp2, static_cast<uint32_t>(rows * g.kp2));
  const int whole = static_cast<int>(g.k / kStep);
  const uint32_t ws = static_cast<uint32_t>(n0 + r) * 4 + h;
  const XT* xs[kFrags];
#pragma unroll
  for (int f = 0; f < kFrags; ++f)
    xs[f] = static_cast<const XT*>(g.x) + (f * 16 + r < g.m ? f * 16 + r : g.m - 1) * g.ldx + h * kBlock;
  f32x4 acc[kFrags][kRuns];
#pragma unroll
  for (int f = 0; f < kFrags; ++f)
#pragma unroll
    for (int i = 0; i < kRuns; ++i) acc[f][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  struct Half {
    Eight<XT> x[kFrags][4];
    i32x4 c[kRuns];
    uint32_t s[kRuns];
  };
  auto load_weights = [&](Half& v, int b) {  // b counts halves
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      v.c[i] = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(bw, (16 * i + r) * g.kp2 + static_cast<uint32_t>(b) * 64 + h * 16, 0, 0));
      v.s[i] = __builtin_amdgcn_raw_buffer_load_b8(bs, ws + 64 * i + static_cast<uint32_t>(b) * g.ws_group, 0, 0);
    }
  };
  auto multiply = [&](const Half& v) {
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max_of<XT>(m, v.x[f][i]);
      const uint32_t s = scale_byte(as_f32_bits<XT>(m));
      const float scale = scale_value(s == 255 ? 127u : s);
      i32x8 xv = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = static_cast<int>(encode8<XT>(v.x[f][i], scale));
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const i32x8 wv = __builtin_shufflevector(v.c[i], i32x4{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
        acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xv, wv, acc[f][i], 4, 4, 0, s, 0, v.s[i]);
      }
    }
  };
  for (int t = wave; t < whole; t += kFewWaves) {
    Half v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        __builtin_memcpy(v[u].x[f], xs[f] + static_cast<int64_t>(t) * kStep + u * 128, sizeof(v[u].x[f]));
      load_weights(v[u], 2 * t + u);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) multiply(v[u]);
  }
  if (whole < g.steps && wave == whole % kFewWaves) {
    for (int u = 0; u < 2; ++u) {
      Half v;
      const int64_t col = static_cast<int64_t>(whole) * kStep + u * 128, left = g.k - col - h * kBlock;
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // from the row's end on: its last element, counted as 0
          v.x[f][i] = load8_upto(xs[f] + col + 8 * i, left - 8 * i);
          __builtin_amdgcn_sched_barrier(0);  // eight at a time: all of them would cost the loop its registers
        }
      load_weights(v, 2 * whole + u);
      multiply(v);
    }
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

struct GemmArgs {
  const uint8_t *a, *as, *b, *bs;
  int64_t m, n;
  uint32_t kp2;                 // bytes per row of codes
  int32_t steps;                // of 256 along k
  uint32_t a_group, b_group;    // bytes between the scales of two runs of 128 columns
  uint32_t as_bytes, bs_bytes;  // bytes of scales
  void* out;
  int64_t ldo;
  uint32_t tiles_m, tiles_n;
  uint32_t whole;               // big tiles that are taken whole; the others in halves
  uint32_t splits;
  int64_t split_stride;         // elements between the outputs of two splits
};

// A piece of 16 bytes is a block of 32 codes: lane (r, h) holds blocks 4 h to 4 h + 3 of a step's eight, whose
// scales are one word; the words of its fragments' rows lie side by side.  The matrix instruction picks the
// block's byte.
template <int kFm, int kFn> struct Fp4Op {
  struct Side {
    uint32_t a[kFm], b[kFn];
  };
  static constexpr int kSideLoads = 2;
  static constexpr int terms(int) { return 2; }
  __amdgpu_buffer_rsrc_t sa, sb;
  uint32_t at_a, at_b, step_a, step_b;

  template <int kCount> static __device__ __forceinline__ void words(uint32_t (&w)[kCount], __amdgpu_buffer_rsrc_t src, uint32_t at) {
    if constexpr (kCount == 4) {
      const auto v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(src, at, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = v[i];
    } else if constexpr (kCount == 2) {
      const auto v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(src, at, 0, 0));
      w[0] = v[0];
      w[1] = v[1];
    } else {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(src, at, 0, 0);
    }
  }
  __device__ __forceinline__ Side load(int t) const {
    Side s;
    words<kFm>(s.a, sa, at_a + t * step_a);
    words<kFn>(s.b, sb, at_b + t * step_b);
    return s;
  }
  static __device__ __forceinline__ void touch(Side& s) {
#pragma unroll
    for (int i = 0; i < kFm; ++i) asm volatile("" : "+v"(s.a[i]));
#pragma unroll
    for (int j = 0; j < kFn; ++j) asm volatile("" : "+v"(s.b[j]));
  }
  template <int kHalf, int kTerm, int kI, int kJ>
  static __device__ __forceinline__ void multiply(f32x16& acc, const i32x4 (&a)[2], const i32x4 (&b)[2], const Side& s) {
    constexpr i32x4 kNone = {0, 0, 0, 0};  // 4-bit operands take four registers
    const i32x8 wa = __builtin_shufflevector(a[kTerm], kNone, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 wb = __builtin_shufflevector(b[kTerm], kNone, 0, 1, 2, 3, 4, 5, 6, 7);
    // formats 4: e2m1
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wb, wa, acc, 4, 4, 2 * kHalf + kTerm, s.b[kJ], 2 * kHalf + kTerm, s.a[kI]);
  }
};

// The tiles are counted kGroup of them down before the next one across, so that those that an XCD has in
// work share rows of both operands.
constexpr uint32_t kGroup = 8;
struct TileAt {
  uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n) {
  const uint32_t group = t / (kGroup * tiles_n), left = tiles_m - group * kGroup;
  const uint32_t rows = left < kGroup ? left : kGroup, in = t % (kGroup * tiles_n);
  return {group * kGroup + in % rows, in / rows};
}

template <int kM, int kN, int kWavesM, int kWavesN, int kBufs, typename OT>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, uint8_t* lds, int64_t m0, int64_t n0, int first, int last, OT* out) {
  constexpr int kFm = kM / kWavesM / 32, kFn = kN / kWavesN / 32;
  typedef Fp4Op<kFm, kFn> Op;
  typedef Tile<kM, kN, kWavesM, kWavesN, kBufs, Op> T;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  // a step has two runs of 128 columns, run h for lane (r, h)
  const Op op = {buffer(g.as, g.as_bytes), buffer(g.bs, g.bs_bytes),
                 (static_cast<uint32_t>(m0) + wm * T::kWm + kFm * (lane & 31)) * 4 + h * g.a_group,
                 (static_cast<uint32_t>(n0) + wn * T::kWn + kFn * (lane & 31)) * 4 + h * g.b_group, 2 * g.a_group, 2 * g.b_group};
  typename T::Acc acc;
  T::sums({g.a, m0, g.m, g.kp2}, {g.b, n0, g.n, g.kp2}, op, lds, first, last, acc);
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    const int64_t row = m0 + wm * T::kWm + kFm * (lane & 31) + i;
    if (row < g.m) {
      OT* po = out + row * g.ldo;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = n0 + wn * T::kWn + kFn * (8 * q + 4 * h);
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
template <int kBufs, typename OT> __global__ void __launch_bounds__(256) gemm_kernel(GemmArgs g) {
  __shared__ __align__(16) uint8_t lds[kBufs * 256 * kStepBytes];
  const uint32_t tiles = g.tiles_m * g.tiles_n, i = xcd_order(blockIdx.x, tiles * g.splits), split = i / tiles;
  const TileAt tile = tile_at(i % tiles, g.tiles_m, g.tiles_n);
  const int first = static_cast<int>(static_cast<int64_t>(g.steps) * split / g.splits);
  const int last = static_cast<int>(static_cast<int64_t>(g.steps) * (split + 1) / g.splits) - 1;
  gemm_tile<128, 128, 2, 2, kBufs, OT>(g, lds, tile.m * int64_t{128}, tile.n * int64_t{128}, first, last,
                                       static_cast<OT*>(g.out) + split * g.split_stride);
}

// One workgroup per tile of 256 x 256, and two for each of those of the last round that would leave
// half of the CUs or more without work.
template <typename OT> __global__ void __launch_bounds__(512) gemm_big_kernel(GemmArgs g) {
  constexpr int kHalfBufs = 3;
  constexpr int kLds = 2 * 512 > kHalfBufs * 384 ? 2 * 512 : kHalfBufs * 384;
  __shared__ __align__(16) uint8_t lds[kLds * kStepBytes];
  OT* out = static_cast<OT*>(g.out);
  if (blockIdx.x < g.whole) {
    const TileAt tile = tile_at(xcd_order(blockIdx.x, g.whole), g.tiles_m, g.tiles_n);
    gemm_tile<256, 256, 2, 4, 2, OT>(g, lds, tile.m * int64_t{256}, tile.n * int64_t{256}, 0, g.steps - 1, out);
  } else {
    const uint32_t i = xcd_order(blockIdx.x - g.whole, gridDim.x - g.whole);
    const TileAt tile = tile_at(g.whole + i / 2, g.tiles_m, g.tiles_n);
    const int64_t m0 = tile.m * int64_t{256} + (i % 2) * 128;
    if (m0 < g.m) gemm_tile<128, 256, 2, 4, kHalfBufs, OT>(g, lds, m0, tile.n * int64_t{256}, 0, g.steps - 1, out);
  }
}

// out = the sum of `splits` binary32 partial results [m, ldp], in their order.
template <typename OT>
__global__ void __launch_bounds__(256) join_kernel(const float* part, int64_t m, int64_t n, int64_t ldp, int splits, OT* out, int64_t ldo) {
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
bool bad_dim(int64_t d) { return d < 0 || d > QOPT_FP4_MAX_DIM; }
bool bad_dtype(int d) { return d != QOPT_F32 && d != QOPT_BF16; }
bool bad_distance(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t{1} << 40); }
uintptr_t size_of(int d) { return d == QOPT_F32 ? 4 : 2; }
int64_t padded(int64_t d) { return ceil_div(d, kStep) * kStep; }
int64_t padded_rows(int64_t rows) { return ceil_div(rows, 16) * 16; }
int64_t code_bytes(int64_t rows, int64_t cols) { return rows * padded(cols) / 2; }
int64_t scale_bytes(int64_t rows, int64_t cols) { return padded(cols) / 128 * padded_rows(rows) * 4; }
bool too_many_tiles(int64_t rows, int64_t cols) { return ceil_div(rows, 128) * ceil_div(cols, 128) > kMaxGrid; }

template <typename XT, typename OT, int kRuns> int launch_few_runs(const FewArgs& g, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(g.n, 16 * kRuns))), block(few_waves(g.m <= 16 ? 1 : 2, kRuns) * kWave);
  if constexpr (kRuns <= 4) {
    if (g.m <= 16) {
      hipLaunchKernelGGL((few_rows_kernel<XT, OT, 1, kRuns>), grid, block, 0, s, g);
      return launch_status();
    }
  }
  hipLaunchKernelGGL((few_rows_kernel<XT, OT, 2, kRuns>), grid, block, 0, s, g);
  return launch_status();
}

// More weight rows per workgroup let more of them share one reading and quantizing of x, fewer fill the chip more
// evenly.  The time goes by what a CU has to read, per column of k: its rounds of workgroups times their rows
// of weights (half a byte) and of x.  Up to eight runs of 16 above 16 rows of x (32 rows of 50257 x 2048 27 us with
// four runs, 21 with eight), up to four below, where x weighs less.
template <typename XT, typename OT> int launch_few(const FewArgs& g, hipStream_t s) {
  int runs = 1;
  int64_t least = 0;
  for (int r : {1, 2, 3, 4, 6, 8}) {
    if (r > 4 && g.m <= 16) break;  // no such instance
    const int64_t bytes = ceil_div(ceil_div(g.n, 16 * r), 256) * (8 * r + g.m * static_cast<int64_t>(sizeof(XT)));
    if (r == 1 || bytes < least) {
      least = bytes;
      runs = r;
    }
  }
  switch (runs) {
    case 1: return launch_few_runs<XT, OT, 1>(g, s);
    case 2: return launch_few_runs<XT, OT, 2>(g, s);
    case 3: return launch_few_runs<XT, OT, 3>(g, s);
    case 4: return launch_few_runs<XT, OT, 4>(g, s);
    case 6: return launch_few_runs<XT, OT, 6>(g, s);
    default: return launch_few_runs<XT, OT, 8>(g, s);
  }
}

// How a product is cut up: tiles of 256 x 256, `whole` of them whole and the others in halves, or (whole
// and halves 0) tiles of 128 x 128 with k in so many splits.
struct Plan {
  int64_t whole, halves;
  int splits;
};

// The plan of least time by this model, in microseconds on 256 CUs.  A step (256 along k) takes a CU
//   1.70 for one tile of 256 x 256, 0.92 for half of one, 1.06 for two tiles of 128 x 128 side by
//   side, 0.70 for one, and 0.50 with three buffers, where no CU has more than one.
// (8192 x 11008 x 4096 takes 197 to 210 us, 3.5 to 3.75 PFLOP/s, of which the matrix instructions alone would take 73 at
// the full clock; the chip's power holds the clock at 1.9 GHz, and a tile's first loads and results cost it 7 us, as
// much as four steps.  8192^3 4.5 PFLOP/s.  With operands of zeros, which draw less power, 5.4 to 5.9.)
// Splitting k, for products of too few tiles, adds a launch that joins the partial results (4) and
// their way to memory and back (4 TB/s).
Plan plan_for(int64_t m, int64_t n, int64_t k) {
  const int64_t all = ceil_div(k, kStep);
  const int64_t small = ceil_div(m, 128) * ceil_div(n, 128), large = ceil_div(m, 256) * ceil_div(n, 256);
  const double two = 1.06, one = 0.70, alone = 0.50;
  Plan best = {0, 0, 1};
  double least = 0;
  for (int splits = 1; splits <= 16 && splits <= all; splits *= 2) {
    const int64_t wgs = small * splits, steps = ceil_div(all, splits);
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
  const double us = static_cast<double>(all) * (ceil_div(large - halved, 256) * 1.70 + (halved ? 0.92 : 0.0));
  if (us <= least) best = {large - halved, 2 * halved, 1};
  return best;
}

int64_t partial_stride(int64_t n) { return ceil_div(n, 4) * 4; }

template <typename OT> int launch_gemm(GemmArgs g, hipStream_t s) {
  g.tiles_m = static_cast<uint32_t>(ceil_div(g.m, 128));
  g.tiles_n = static_cast<uint32_t>(ceil_div(g.n, 128));
  const int64_t wgs = static_cast<int64_t>(g.tiles_m) * g.tiles_n * g.splits;
  if (wgs > kMaxGrid) return QOPT_EINVAL;
  const dim3 grid(static_cast<unsigned>(wgs));
  if (wgs <= 256) hipLaunchKernelGGL((gemm_kernel<3, OT>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((gemm_kernel<2, OT>), grid, dim3(256), 0, s, g);
  return launch_status();
}

template <typename OT> int launch_gemm_big(GemmArgs g, const Plan& plan, hipStream_t s) {
  g.tiles_m = static_cast<uint32_t>(ceil_div(g.m, 256));
  g.tiles_n = static_cast<uint32_t>(ceil_div(g.n, 256));
  g.whole = static_cast<uint32_t>(plan.whole);
  const dim3 grid(static_cast<unsigned>(plan.whole + plan.halves));  // at most kMaxGrid tiles of 128 x 128
  hipLaunchKernelGGL((gemm_big_kernel<OT>), grid, dim3(512), 0, s, g);
  return launch_status();
}

template <typename OT> int launch_product(GemmArgs g, const Plan& plan, OT* out, int64_t ldo, void* workspace, hipStream_t s) {
  if (plan.splits > 1) {
    g.out = workspace;
    g.ldo = partial_stride(g.n);
    g.split_stride = g.m * g.ldo;
    const int rc = launch_gemm<float>(g, s);
    if (rc != QOPT_OK) return rc;
    const int64_t wgs = ceil_div(g.m * (g.ldo / 4), 256);
    hipLaunchKernelGGL(join_kernel<OT>, dim3(static_cast<unsigned>(wgs < 4096 ? wgs : 4096)), dim3(256), 0, s,
                       static_cast<const float*>(workspace), g.m, g.n, g.ldo, plan.splits, out, ldo);
    return launch_status();
  }
  g.out = out;
  g.ldo = ldo;
  return plan.whole + plan.halves > 0 ? launch_gemm_big<OT>(g, plan, s) : launch_gemm<OT>(g, s);
}

int check_out(const void* out, int64_t m, int64_t n, int64_t ldo, int out_dtype) {
  if (bad_distance(ldo, n)) return QOPT_EINVAL;
  if (m == 0 || n == 0) return QOPT_OK;
  if (!out) return QOPT_EINVAL;
  return aligned(out, size_of(out_dtype)) ? QOPT_OK : QOPT_EALIGN;
}

int zero_out(void* out, int out_dtype, int64_t m, int64_t n, int64_t ldo, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(n < 65536 ? ceil_div(n, 256) : 256), static_cast<unsigned>(m < 1024 ? m : 1024));
  if (out_dtype == QOPT_F32)
    hipLaunchKernelGGL(zero_kernel<float>, grid, dim3(256), 0, s, static_cast<float*>(out), m, n, ldo);
  else
    hipLaunchKernelGGL(zero_kernel<uint16_t>, grid, dim3(256), 0, s, static_cast<uint16_t*>(out), m, n, ldo);
  return launch_status();
}

}  // namespace

// ------------------------------------------------------------------ entry points

extern "C" int qopt_fp4_quantize(const void* x_dev, int dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes_dev,
                                 uint8_t* scales_dev, void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || bad_distance(ldx, cols)) return QOPT_EINVAL;
  if (bad_dtype(dtype)) return QOPT_EUNSUPPORTED;
  if (rows == 0 || cols == 0) return QOPT_OK;
  if (too_many_tiles(rows, cols) || !x_dev || !codes_dev || !scales_dev) return QOPT_EINVAL;
  if (!aligned(x_dev, size_of(dtype)) || !aligned(codes_dev, 16) || !aligned(scales_dev, 4)) return QOPT_EALIGN;
  const QuantArgs q = {x_dev, rows, cols, ldx, codes_dev, reinterpret_cast<uint32_t*>(scales_dev), padded(cols), padded_rows(rows),
                       static_cast<uint32_t>(ceil_div(cols, 512))};
  const dim3 grid(static_cast<unsigned>(q.across * ceil_div(rows, 16)));  // at most twice kMaxGrid of 256 threads
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == QOPT_F32) hipLaunchKernelGGL(quantize_kernel<float>, grid, dim3(256), 0, s, q);
  else hipLaunchKernelGGL(quantize_kernel<uint16_t>, grid, dim3(256), 0, s, q);
  return launch_status();
}

extern "C" int qopt_fp4_dequantize(const uint8_t* codes_dev, const uint8_t* scales_dev, int64_t rows, int64_t cols, void* out_dev,
                                   int dtype, int64_t ldo, void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || bad_distance(ldo, cols)) return QOPT_EINVAL;
  if (bad_dtype(dtype)) return QOPT_EUNSUPPORTED;
  if (rows == 0 || cols == 0) return QOPT_OK;
  if (too_many_tiles(rows, cols) || !out_dev || !codes_dev || !scales_dev) return QOPT_EINVAL;
  if (!aligned(out_dev, size_of(dtype)) || !aligned(codes_dev, 16) || !aligned(scales_dev, 4)) return QOPT_EALIGN;
  const DequantArgs q = {codes_dev, scales_dev, rows, cols, padded(cols), padded_rows(rows), out_dev, ldo,
                         static_cast<uint32_t>(ceil_div(cols, 512))};
  const dim3 grid(static_cast<unsigned>(q.across * ceil_div(rows, 16)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == QOPT_F32) hipLaunchKernelGGL(dequantize_kernel<float>, grid, dim3(256), 0, s, q);
  else hipLaunchKernelGGL(dequantize_kernel<uint16_t>, grid, dim3(256), 0, s, q);
  return launch_status();
}

extern "C" int qopt_fp4_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes) {
  if (!bytes || bad_dim(m) || bad_dim(n) || bad_dim(k)) return QOPT_EINVAL;
  if (bad_dtype(out_dtype)) return QOPT_EUNSUPPORTED;
  *bytes = 0;
  if (m == 0 || n == 0 || k == 0) return QOPT_OK;
  if (too_many_tiles(m, k) || too_many_tiles(n, k) || too_many_tiles(m, n)) return QOPT_EINVAL;
  const Plan p = plan_for(m, n, k);
  if (p.splits > 1) *bytes = static_cast<size_t>(p.splits) * m * partial_stride(n) * sizeof(float);
  return QOPT_OK;
}

extern "C" int qopt_fp4_matmul(const uint8_t* a_codes_dev, const uint8_t* a_scales_dev, const uint8_t* b_codes_dev,
                               const uint8_t* b_scales_dev, int64_t m, int64_t n, int64_t k, void* out_dev, int out_dtype,
                               int64_t ldo, void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = qopt_fp4_matmul_workspace(m, n, k, out_dtype, &need);
  if (rc != QOPT_OK) return rc;
  rc = check_out(out_dev, m, n, ldo, out_dtype);
  if (rc != QOPT_OK || m == 0 || n == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (k == 0) return zero_out(out_dev, out_dtype, m, n, ldo, s);
  if (!a_codes_dev || !a_scales_dev || !b_codes_dev || !b_scales_dev) return QOPT_EINVAL;
  if (!aligned(a_codes_dev, 16) || !aligned(b_codes_dev, 16) || !aligned(a_scales_dev, 4) || !aligned(b_scales_dev, 4) ||
      !aligned(workspace_dev, 16))
    return QOPT_EALIGN;
  if (need > 0 && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  const Plan plan = plan_for(m, n, k);
  GemmArgs g = {};
  g.a = a_codes_dev;
  g.as = a_scales_dev;
  g.b = b_codes_dev;
  g.bs = b_scales_dev;
  g.m = m;
  g.n = n;
  g.kp2 = static_cast<uint32_t>(padded(k) / 2);
  g.steps = static_cast<int32_t>(ceil_div(k, kStep));
  g.a_group = static_cast<uint32_t>(padded_rows(m) * 4);
  g.b_group = static_cast<uint32_t>(padded_rows(n) * 4);
  g.as_bytes = static_cast<uint32_t>(scale_bytes(m, k));  // at most 2^32 - 2^9 by too_many_tiles
  g.bs_bytes = static_cast<uint32_t>(scale_bytes(n, k));
  g.splits = static_cast<uint32_t>(plan.splits);
  return out_dtype == QOPT_F32 ? launch_product(g, plan, static_cast<float*>(out_dev), ldo, workspace_dev, s)
                               : launch_product(g, plan, static_cast<uint16_t*>(out_dev), ldo, workspace_dev, s);
}

namespace {
// The codes of x and its scales at the start of qopt_fp4_linear's workspace, in multiples of 16 bytes.
size_t linear_own_bytes(int64_t m, int64_t k) { return static_cast<size_t>(code_bytes(m, k) + scale_bytes(m, k)); }
}  // namespace

extern "C" int qopt_fp4_linear_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes) {
  const int rc = qopt_fp4_matmul_workspace(m, n, k, out_dtype, bytes);
  if (rc != QOPT_OK) return rc;
  if (m <= QOPT_FP4_FEW_ROWS || n == 0 || k == 0) *bytes = 0;
  else *bytes += linear_own_bytes(m, k);
  return QOPT_OK;
}

extern "C" int qopt_fp4_linear(const void* x_dev, int dtype, int64_t m, int64_t k, int64_t ldx, const uint8_t* w_codes_dev,
                               const uint8_t* w_scales_dev, int64_t n, void* out_dev, int out_dtype, int64_t ldo,
                               void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = qopt_fp4_linear_workspace(m, n, k, out_dtype, &need);
  if (rc != QOPT_OK) return rc;
  if (bad_distance(ldx, k)) return QOPT_EINVAL;
  if (bad_dtype(dtype)) return QOPT_EUNSUPPORTED;
  rc = check_out(out_dev, m, n, ldo, out_dtype);
  if (rc != QOPT_OK || m == 0 || n == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (k == 0) return zero_out(out_dev, out_dtype, m, n, ldo, s);
  if (!x_dev || !w_codes_dev || !w_scales_dev) return QOPT_EINVAL;
  if (!aligned(x_dev, size_of(dtype)) || !aligned(w_codes_dev, 16) || !aligned(w_scales_dev, 4) || !aligned(workspace_dev, 16))
    return QOPT_EALIGN;
  if (need > 0 && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  if (m > QOPT_FP4_FEW_ROWS) {
    uint8_t* codes = static_cast<uint8_t*>(workspace_dev);
    uint8_t* scales = codes + code_bytes(m, k);
    rc = qopt_fp4_quantize(x_dev, dtype, m, k, ldx, codes, scales, stream);
    if (rc != QOPT_OK) return rc;
    const size_t used = linear_own_bytes(m, k);
    return qopt_fp4_matmul(codes, scales, w_codes_dev, w_scales_dev, m, n, k, out_dev, out_dtype, ldo,
                           static_cast<uint8_t*>(workspace_dev) + used, workspace_bytes - used, stream);
  }
  const FewArgs g = {x_dev, m, k, ldx, w_codes_dev, w_scales_dev, n, static_cast<uint32_t>(padded(k) / 2),
                     static_cast<uint32_t>(scale_bytes(n, k)), static_cast<uint32_t>(padded_rows(n) * 4),
                     static_cast<int32_t>(ceil_div(k, kStep)), out_dev, ldo};
  if (dtype == QOPT_F32)
    return out_dtype == QOPT_F32 ? launch_few<float, float>(g, s) : launch_few<float, uint16_t>(g, s);
  return out_dtype == QOPT_F32 ? launch_few<uint16_t, float>(g, s) : launch_few<uint16_t, uint16_t>(g, s);
}

// Newton-Schulz orthogonalisation and the Muon step for gfx950: the kernels of include/qopt_muon.h.
//
// With A = X X^T (m x m, m the shorter side) the iteration X = (a I + b A + c A^2) X is a polynomial of A
// times X, and so is what several iterations make: their polynomials commute and are symmetric.  A group of
// iterations is therefore carried out on m x m matrices alone,
//     P = a I + b A + c A^2,  Q = P Q,  A = P A P,
// and Q is applied to X at its end; every product but that one is symmetric, so that only the tiles on and
// below the diagonal are computed, each stored with its mirror image.  For n / m = r a group of L iterations
// takes (in products of m x m matrices) r / 2 + L / 2 + (L - 1) / 2 + (L - 1) + r, where the iterations by
// themselves take L (3 r / 2 + 1 / 2): for five iterations as 3 + 2, 3 r + 7, as 2 + 2 + 1, 4.5 r + 5.5, against
// 7.5 r + 2.5: the same for square matrices and less than half for r = 8.
// Groups are at most three long (`group_steps`), because a singular value s of X stands in A as s^2: what rounding
// adds to a small one grows by a^2 = 11.9 per iteration on A, a fresh A = X X^T brings it back.  (With rounding to 22
// bits four in one group end in infinities where eight directions are 170 times the rest.)
//
// Numbers.  A value is kept times a power of two that holds the largest possible one (|X| <= 1.203, A <= 1.45,
// P <= 3.4445, Q <= 3.4445^3) under 65504, as hi + lo, two binary16 numbers: 22 bits, or 23, down to 2^-24, under which lo
// ends: 2^-36 of X's largest possible value.  A product is hi hi + hi lo + lo hi with binary32 sums, which leaves out 2^-22
// of it.  That holds for either destination: with fewer bits a bfloat16 result would be faster (hi alone takes a third of the
// time) and off by as much as its own rounding or more, 8e-4 to 2.4e-2 of itself where that is 1.66e-3.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "blockwise_code.h"
#include "product_tile.h"
#include "qopt_muon.h"

namespace {

using namespace product;
using blockwise::BlockScale;
using blockwise::Encoder;

constexpr double kExactA = 3.4445, kExactB = -4.775, kExactC = 2.0315;
constexpr float kA = kExactA, kB = kExactB, kC = kExactC;
constexpr int kExp = 12, kExpQ = 10;  // powers of two of X, A, P and P A, and of a product Q
constexpr int kMaxJobs = 32;          // of one launch (its arguments are 4 KB at most)
// Workgroups, and partial sums of squares, per matrix at most: with codes, whose encoder's chains want more of them on a CU,
// 1024 (six matrices of 58.7 M elements 107 us; 512 of each 123), without 512 (4096 x 11008 145 us; 1024 152).
constexpr int kMaxParts = 512, kMaxCodedParts = 1024;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// A matrix as an operand: rows of a multiple of 64 values, for every 8 of them one piece of 16 bytes of hi and one of
// lo, as a product's lanes take them.
constexpr int64_t kPad = 64;
__host__ __device__ constexpr int64_t padded(int64_t d) { return ceil_div(d, kPad) * kPad; }
__host__ __device__ constexpr int64_t row_bytes(int64_t cols) { return padded(cols) * 4; }

// ------------------------------------------------------------------ momentum and norms

struct SourceJob {
  const void* g;  // gradient, or the matrix itself
  void* m;
  float* absmax;
  float* u;       // where the update goes
  double* parts;  // partial sums of squares
  int64_t n;
  uint32_t groups;
};
struct SourceArgs {
  SourceJob jobs[kMaxJobs];
  const qopt_codebook* cb;
  const float* grad_scale;
  float mu, omu;
  int nesterov;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// Elements i to i + 7 of n, 0 behind the end.
template <typename T> __device__ __forceinline__ void load8(const T* p, int64_t i, int64_t n, float (&v)[8]) {
  T w[8];
  if (i + 8 <= n) {
    __builtin_memcpy(w, p + i, sizeof(w));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = i + e < n ? to_f32(p[i + e]) : 0.0f;
  }
}

// Sum over the 4 waves of a workgroup, in a fixed order, for thread 0.
__device__ __forceinline__ double group_sum(double s, double (&slots)[4]) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x / kWave] = s;
  __syncthreads();
  return slots[0] + slots[1] + slots[2] + slots[3];
}

enum Source : int { kPlain = 0, kMomentum32 = 1, kMomentum8 = 2 };

// Blocks of 2048 of one matrix (blockIdx.y), every groups-th by a workgroup: the new momentum, the update u
// and its sum of squares (binary64: squares of any binary32 numbers neither overflow nor vanish).
// Bound by memory: 4096 x 11008 with binary32 momentum, 631 MB, 140 to 145 us, 4.4 TB/s; with codes, 58.7 M parameters in six
// matrices, 107 us for 470 MB, also 4.4 TB/s.  (Loading the next block before this one's work took 10 to 30 % longer.)
template <typename GT, int kSource> __global__ void __launch_bounds__(256) source_kernel(SourceArgs a) {
  __shared__ __align__(16) qopt_codebook cb;  // kMomentum8
  __shared__ double slots[4];
  __shared__ uint32_t maxima[2][4];
  const SourceJob& job = a.jobs[blockIdx.y];
  if (blockIdx.x >= job.groups) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  if constexpr (kSource == kMomentum8) {
    for (uint32_t i = threadIdx.x; i < sizeof(qopt_codebook) / 16; i += 256)
      reinterpret_cast<uint4*>(&cb)[i] = reinterpret_cast<const uint4*>(a.cb)[i];
    __syncthreads();
  }
  const int64_t n = job.n;
  double sum = 0.0;
  int turn = 0;
  for (int64_t b = blockIdx.x; b * QOPT_BLOCK < n; b += job.groups, turn ^= 1) {
    const int64_t i = b * QOPT_BLOCK + 8 * threadIdx.x;
    float g[8];
    load8(static_cast<const GT*>(job.g), i, n, g);
    if constexpr (kSource != kPlain) {
      float m[8];
      if constexpr (kSource == kMomentum32) {
        load8(static_cast<const float*>(job.m), i, n, m);
      } else {
        const uint8_t* codes = static_cast<const uint8_t*>(job.m);
        const float amax = job.absmax[b];
        uint8_t c[8];
        if (i + 8 <= n) {
          __builtin_memcpy(c, codes + i, 8);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) c[e] = i + e < n ? codes[i + e] : 0;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = i + e < n ? cb.decode[c[e]] * amax : 0.0f;
      }
      float most = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (a.grad_scale) g[e] = g[e] * gs;
        const float t = g[e] * a.omu;
        m[e] = m[e] * a.mu + t;
        g[e] = a.nesterov ? m[e] * a.mu + t : m[e];
        if (i + e >= n) m[e] = g[e] = 0.0f;  // behind the end a factor may be infinite
        most = __builtin_elementwise_maximum(most, fabsf(m[e]));
      }
      if constexpr (kSource == kMomentum32) {
        float* to = static_cast<float*>(job.m) + i;
        if (i + 8 <= n) {
          __builtin_memcpy(to, m, sizeof(m));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (i + e < n) to[e] = m[e];
        }
      } else {
        uint32_t bits = __float_as_uint(most);
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
          const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(bits), d));
          bits = bits > o ? bits : o;
        }
        if ((threadIdx.x & 63) == 0) maxima[turn][threadIdx.x / kWave] = bits;
        __syncthreads();
        bits = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) bits = bits > maxima[turn][w] ? bits : maxima[turn][w];
        const BlockScale s = blockwise::block_scale(__uint_as_float(bits), cb.sign_mask);
        const Encoder enc = blockwise::make_encoder(&cb);
        uint8_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = s.zero ? 0 : static_cast<uint8_t>(blockwise::encode_signed(enc, s, m[e]));
        uint8_t* to = static_cast<uint8_t*>(job.m) + i;
        if (i + 8 <= n) {
          __builtin_memcpy(to, c, 8);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (i + e < n) to[e] = c[e];
        }
        if (threadIdx.x == 0) job.absmax[b] = s.absmax;
      }
      float* u = job.u + i;
      if (i + 8 <= n) {
        __builtin_memcpy(u, g, sizeof(g));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + e < n) u[e] = g[e];
      }
    }
    double part = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) part += static_cast<double>(g[e]) * static_cast<double>(g[e]);
    sum += part;
  }
  const double s = group_sum(sum, slots);
  if (threadIdx.x == 0) job.parts[blockIdx.x] = s;
}

// ------------------------------------------------------------------ operands from the update

template <int kCount> struct HalfVec;
template <> struct HalfVec<2> { typedef f16x2 type; };
template <> struct HalfVec<4> { typedef f16x4 type; };
template <> struct HalfVec<8> { typedef f16x8 type; };

// kCount consecutive values of an operand's row, from place `at` on: a multiple of kCount.
template <int kCount> __device__ __forceinline__ void write_run(uint8_t* row, int64_t at, const float (&v)[kCount]) {
  typename HalfVec<kCount>::type hi, lo;
#pragma unroll
  for (int e = 0; e < kCount; ++e) {
    hi[e] = static_cast<_Float16>(v[e]);
    lo[e] = static_cast<_Float16>(v[e] - static_cast<float>(hi[e]));
  }
  uint8_t* to = row + (at >> 3) * 32 + (at & 7) * 2;
  __builtin_memcpy(to, &hi, sizeof(hi));
  __builtin_memcpy(to + 16, &lo, sizeof(lo));
}

// Eight values of an operand's row, from place `at` on: a multiple of 8.
__device__ __forceinline__ void read_run(const uint8_t* row, int64_t at, float (&v)[8]) {
  const f16x8 hi = *reinterpret_cast<const f16x8*>(row + at * 4), lo = *reinterpret_cast<const f16x8*>(row + at * 4 + 16);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(hi[e]) + static_cast<float>(lo[e]);
}

struct PackJob {
  const void* src;        // [rows, cols]
  uint8_t *same, *other;  // as operands: its rows, and its transpose's
  const double* parts;
  int64_t rows, cols;
  uint32_t groups, first, across;
};
struct PackArgs {
  PackJob jobs[kMaxJobs];
  int njobs;
  double eps;
};

// X = U 2^kExp / max(|U|, eps) and its transpose.  A wave takes 64 x 64 values, a lane 8 x 8 of them:
// it reads 8 runs of 8, writes them as 8 places of the operand's rows, and of the transpose's; the lanes next
// to each other make runs of 256 bytes either way.  4096 x 11008, 541 MB: 109 to 113 us, 4.9 TB/s (122 to 126 with
// a branch at every row).
template <typename ST> __global__ void __launch_bounds__(256) pack_kernel(PackArgs a) {
  __shared__ double slots[4];
  int j = 0;
  while (j + 1 < a.njobs && blockIdx.x >= a.jobs[j + 1].first) ++j;
  const PackJob& job = a.jobs[j];
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < job.groups; i += 256) s += job.parts[i];
  const double norm = sqrt(group_sum(s, slots));
  const double scale = static_cast<double>(1 << kExp) / (norm < a.eps ? a.eps : norm);  // a NaN stays one
  const uint32_t at = blockIdx.x - job.first;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int64_t r0 = static_cast<int64_t>(at / job.across) * 64 + 8 * (lane >> 3);
  const int64_t c0 = (static_cast<int64_t>(at % job.across) * 4 + wave) * 64 + 8 * (lane & 7);
  if (c0 >= padded(job.cols)) return;  // r0 lies within the padded rows always
  float v[8][8];
  const ST* src = static_cast<const ST*>(job.src);
  if (r0 - 8 * (lane >> 3) + 64 <= job.rows && c0 - 8 * (lane & 7) + 64 <= job.cols) {
    // all of the wave's values lie in the matrix: no branch between the loads
    ST w[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) __builtin_memcpy(w[i], src + (r0 + i) * job.cols + c0, sizeof(w[i]));
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = static_cast<float>(static_cast<double>(to_f32(w[i][e])) * scale);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < job.rows) {
        load8(src + (r0 + i) * job.cols, c0, job.cols, v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = c0 + e < job.cols ? static_cast<float>(static_cast<double>(v[i][e]) * scale) : 0.0f;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < job.rows) write_run<8>(job.same + (r0 + i) * row_bytes(job.cols), c0, v[i]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i][e];
    if (c0 + e < job.cols) write_run<8>(job.other + (c0 + e) * row_bytes(job.rows), r0, t);
  }
}

// ------------------------------------------------------------------ products

// One product out = l r^T, with what its epilogue needs.
struct Job {
  const uint8_t *l, *r;   // operands: rows of k_bytes
  const uint8_t* add;     // the polynomial's A
  uint8_t *out, *out_t;   // the result as an operand, and its transpose
  void* dst;              // the last product's destination, [lrows, rrows]
  int32_t lrows, rrows;
  uint32_t k_bytes, out_bytes, out_t_bytes;  // bytes per row
  uint32_t first, tiles_m, tiles_n;          // its first tile among all, and its own
  uint32_t steps, first_step;                // along the sum; of all tiles before its first
  float factor, rate;
};
struct ProductArgs {
  Job jobs[kMaxJobs];
  int njobs;
  float decay;
  // Workgroups 0 to whole - 1 take a tile each.  The steps of the others, `shared` from first_step on, are cut
  // into `workers` runs of equal length; what a run holds of a tile without all of its steps goes to `parts`.
  uint32_t whole, workers, first_step, shared, rest;
  f32x4* parts;
};
static_assert(sizeof(ProductArgs) <= 4096, "kernel arguments");

enum Epilogue : int {
  kSymmetric,   // out = factor l r^T, which is symmetric
  kPolynomial,  // out = a I + b add + c l r^T likewise
  kApply,       // out and out_t, in the layout of the group that comes next
  kResult,      // dst = factor l r^T
  kUpdate       // dst = dst * decay - factor l r^T * rate
};

// A lane's two pieces of a fragment are hi and lo of the same 8 values.
struct HalfOp {
  struct Side {};
  static constexpr int kSideLoads = 0;
  static constexpr int terms(int) { return 3; }
  __device__ __forceinline__ Side load(int) const { return {}; }
  static __device__ __forceinline__ void touch(Side&) {}
  template <int kHalf, int kTerm, int kI, int kJ>
  static __device__ __forceinline__ void multiply(f32x16& acc, const i32x4 (&a)[2], const i32x4 (&b)[2], const Side&) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b[kTerm == 1]), __builtin_bit_cast(f16x8, a[kTerm == 2]), acc,
                                                 0, 0, 0);
  }
};

template <typename OT> __device__ __forceinline__ void load_out(const OT* p, float (&v)[8]) {
  OT w[8];
  __builtin_memcpy(w, p, sizeof(w));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f32(w[e]);
}

// What a tile's sums become: quarter q of its columns.  s[i][j][e] is acc[i][j][4 q + e].
template <typename T, int kWavesN, int kEpilogue, typename OT>
__device__ __forceinline__ void finish(const Job& job, float decay, int64_t m0, int64_t n0, int q, const f32x4 (&s)[T::kFm][2]) {
  constexpr int kFm = T::kFm;
  static_assert(T::kFn == 2, "a lane's columns are eight places of an operand's row");
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row0 = m0 + wave / kWavesN * T::kWm + kFm * (lane & 31);
  const int64_t col = n0 + wave % kWavesN * T::kWn + 2 * (8 * q + 4 * h);
  const int64_t pm = padded(job.lrows), pn = padded(job.rrows);
  float v[kFm][8];
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    const int64_t row = row0 + i;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[i][2 * e] = s[i][0][e] * job.factor;
      v[i][2 * e + 1] = s[i][1][e] * job.factor;
    }
    if constexpr (kEpilogue == kPolynomial) {
      if (row < job.lrows && col < pn) {
        float x[8];
        read_run(job.add + row * job.k_bytes, col, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[i][e] = v[i][e] * kC + x[e] * kB + (row == col + e ? kA * static_cast<float>(1 << kExp) : 0.0f);
      }
    }
    if constexpr (kEpilogue == kResult || kEpilogue == kUpdate) {
      if (row < job.lrows) {
        OT* dst = static_cast<OT*>(job.dst) + row * job.rrows + col;
        if (col + 8 <= job.rrows) {  // at any alignment
          OT w[8];
          float p[8];
          if constexpr (kEpilogue == kUpdate) load_out(dst, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (kEpilogue == kUpdate) v[i][e] = p[e] * decay - v[i][e] * job.rate;
            store1(w + e, v[i][e]);
          }
          __builtin_memcpy(dst, w, sizeof(w));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < job.rrows) {
              if constexpr (kEpilogue == kUpdate) v[i][e] = to_f32(dst[e]) * decay - v[i][e] * job.rate;
              store1(dst + e, v[i][e]);
            }
        }
      }
    } else {
      if (row < job.lrows && col < pn) write_run<8>(job.out + row * job.out_bytes, col, v[i]);
    }
  }
  // the mirror image, or the transpose: rows of the result are places there, up to the padding
  if constexpr (kEpilogue == kSymmetric || kEpilogue == kPolynomial || kEpilogue == kApply) {
    uint8_t* out = kEpilogue == kApply ? job.out_t : job.out;
    const uint32_t bytes = kEpilogue == kApply ? job.out_t_bytes : job.out_bytes;
    if (row0 < pm && (kEpilogue == kApply || m0 != n0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t[kFm];
#pragma unroll
        for (int i = 0; i < kFm; ++i) t[i] = v[i][e];
        if (col + e < job.rrows) write_run<kFm>(out + (col + e) * bytes, row0, t);
      }
    }
  }
}

constexpr uint32_t kGroup = 8;  // tiles counted down before the next one across

// Tile number t of a job: its rows of l and of r, in tiles.
template <int kEpilogue> __device__ __forceinline__ void tile_at(const Job& job, uint32_t t, uint32_t& tm, uint32_t& tn) {
  if constexpr (kEpilogue == kSymmetric || kEpilogue == kPolynomial) {
    // tiles on and below the diagonal: row i begins with number i (i + 1) / 2
    tm = static_cast<uint32_t>((sqrtf(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
    while (tm * (tm + 1) / 2 > t) --tm;
    while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
    tn = t - tm * (tm + 1) / 2;
  } else {
    const uint32_t group = t / (kGroup * job.tiles_n), left = job.tiles_m - group * kGroup;
    const uint32_t rows = left < kGroup ? left : kGroup, in = t % (kGroup * job.tiles_n);
    tm = group * kGroup + in % rows;
    tn = in / rows;
  }
}

// First of the shared steps of run w.
__device__ __forceinline__ uint32_t run_start(const ProductArgs& a, uint32_t w) {
  return a.first_step + static_cast<uint32_t>(static_cast<uint64_t>(a.shared) * w / a.workers);
}

template <bool kBig> struct TileOf {
  static constexpr int kSide = kBig ? 256 : 128, kWavesN = kBig ? 4 : 2;
  typedef Tile<kSide, kSide, 2, kWavesN, kBig ? 2 : 3, HalfOp> T;
  static constexpr int kQuarter = T::kFm * 2 * T::kThreads;  // f32x4 of a quarter of the columns
};

// Whole tiles leave CUs idle in the last round: 136 tiles of 256 x 256 below the diagonal of 4096 x 4096 use
// half of the chip.  Runs of equal length over the tiles' steps use all of it; a tile that lies in several runs is
// joined by a launch of its own, which reads the runs' sums in their order and does what follows a product.
//
// Measured: Q X of 4096 x 4096 x 11008 920 to 1000 us, 1.2 PFLOP/s of single numbers (three instructions each),
// the matrix units busy 79 to 81 % of the CUs' time at 1.7 GHz, which is where the chip's power holds the clock: that is what
// bounds it.  X X^T of the same: 360 us, and 26 to join.  A symmetric product of 4096 x 4096: 170 to 183 us, and 38
// to join.  Four of 2048 x 2048: 126 to 142 us on 144 CUs, whose matrix units are busy 78 % of the time.
template <bool kBig, int kEpilogue, typename OT>
__global__ void __launch_bounds__(kBig ? 512 : 256) product_kernel(ProductArgs a) {
  typedef TileOf<kBig> O;
  typedef typename O::T T;
  __shared__ __align__(16) uint8_t lds[T::kLds];
  auto sums = [&](const Job& job, uint32_t tile, int first, int last, int64_t& m0, int64_t& n0, typename T::Acc& acc) {
    uint32_t tm, tn;
    tile_at<kEpilogue>(job, tile, tm, tn);
    m0 = static_cast<int64_t>(tm) * O::kSide;
    n0 = static_cast<int64_t>(tn) * O::kSide;
    T::sums({job.l, m0, job.lrows, job.k_bytes}, {job.r, n0, job.rrows, job.k_bytes}, HalfOp{}, lds, first, last, acc);
  };
  auto quarter = [](const typename T::Acc& acc, int q, f32x4 (&s)[T::kFm][2]) {
#pragma unroll
    for (int i = 0; i < T::kFm; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][j][e] = acc[i][j][4 * q + e];
  };
  const bool whole = blockIdx.x < a.whole;
  const uint32_t w = whole ? xcd_order(blockIdx.x, a.whole) : xcd_order(blockIdx.x - a.whole, a.workers);
  uint32_t at = 0, end = 1;
  const uint32_t start = whole ? 0 : run_start(a, w);
  if (!whole) {
    at = start;
    end = run_start(a, w + 1);
  }
  int j = 0;
  while (at < end) {
    while (j + 1 < a.njobs && (whole ? w >= a.jobs[j + 1].first : at >= a.jobs[j + 1].first_step)) ++j;
    const Job& job = a.jobs[j];
    uint32_t tile = w - job.first, first = 0, last = job.steps - 1;
    if (!whole) {
      tile = (at - job.first_step) / job.steps;
      first = at - job.first_step - tile * job.steps;
      last = job.steps - first < end - at ? job.steps - 1 : first + (end - at) - 1;
    }
    typename T::Acc acc;
    int64_t m0, n0;
    sums(job, tile, static_cast<int>(first), static_cast<int>(last), m0, n0, acc);
    if (first == 0 && last == job.steps - 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 s[T::kFm][2];
        quarter(acc, q, s);
        finish<T, O::kWavesN, kEpilogue, OT>(job, a.decay, m0, n0, q, s);
      }
    } else {
      // at most the first and the last piece of a run are not whole
      f32x4* to = a.parts + static_cast<int64_t>(2 * w + (at > start ? 1 : 0)) * 4 * O::kQuarter + threadIdx.x;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 s[T::kFm][2];
        quarter(acc, q, s);
#pragma unroll
        for (int i = 0; i < T::kFm; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) to[q * O::kQuarter + (2 * i + c) * T::kThreads] = s[i][c];
      }
    }
    if (whole) return;
    at += last - first + 1;
    __syncthreads();  // every wave has read the last step before the next piece's is loaded
  }
}

// One quarter (blockIdx.y) of the columns of each tile behind the whole ones that lies in more than one run.
template <bool kBig, int kEpilogue, typename OT>
__global__ void __launch_bounds__(kBig ? 512 : 256) join_kernel(ProductArgs a) {
  typedef TileOf<kBig> O;
  typedef typename O::T T;
  const uint32_t tile = a.whole + blockIdx.x;
  int j = 0;
  while (j + 1 < a.njobs && tile >= a.jobs[j + 1].first) ++j;
  const Job& job = a.jobs[j];
  const uint32_t begin = job.first_step + (tile - job.first) * job.steps, end = begin + job.steps;
  // the run that holds the tile's first step: the quotient, or next to it
  uint32_t w = static_cast<uint32_t>(static_cast<uint64_t>(begin - a.first_step) * a.workers / a.shared);
  while (w > 0 && run_start(a, w) > begin) --w;
  while (run_start(a, w + 1) <= begin) ++w;
  if (run_start(a, w + 1) >= end) return;  // whole in one run
  f32x4 s[T::kFm][2];
#pragma unroll
  for (int i = 0; i < T::kFm; ++i)
#pragma unroll
    for (int c = 0; c < 2; ++c) s[i][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t from = run_start(a, w); from < end; ++w, from = run_start(a, w)) {
    const f32x4* p = a.parts + static_cast<int64_t>(2 * w + (from < begin ? 1 : 0)) * 4 * O::kQuarter + blockIdx.y * O::kQuarter + threadIdx.x;
#pragma unroll
    for (int i = 0; i < T::kFm; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) s[i][c] += p[(2 * i + c) * T::kThreads];
  }
  uint32_t tm, tn;
  tile_at<kEpilogue>(job, tile - job.first, tm, tn);
  finish<T, O::kWavesN, kEpilogue, OT>(job, a.decay, static_cast<int64_t>(tm) * O::kSide, static_cast<int64_t>(tn) * O::kSide,
                                                  blockIdx.y, s);
}

// A group on matrices of at most 128 x 128: one workgroup per matrix takes it from A to Q.  A, P and Q stay in
// registers in binary32, 64 of a lane's 512 each, laid out as a product's sums; LDS holds the two operands of the
// product at hand as `Tile` would have loaded them, and since they are symmetric, as either side of it.
// One iteration takes 10 us, two 20 to 22, three 34, where each of their products in a launch of its own takes 6 to 9: in all
// of 99 x 300, 103 us against 146 (in groups of three, before their length went by the size).  What bounds it is one
// workgroup's chain of products on four matrix units, whatever the number of matrices up to one per CU.
constexpr int64_t kChainDim = 128;

struct ChainJob {
  const uint8_t* a;
  uint8_t* q;
  int32_t m;
};
struct ChainArgs {
  ChainJob jobs[kMaxJobs];
  int length;
};

__global__ void __launch_bounds__(256, 1) chain_kernel(ChainArgs args) {
  constexpr int kSteps = 4, kStep = 128 * kStepBytes;  // bytes of a step's rows
  __shared__ __align__(16) uint8_t image[2][kSteps * kStep];
  typedef f32x16 Mat[2][2];
  const ChainJob& job = args.jobs[blockIdx.x];
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wm = wave / 2, wn = wave % 2;
  const int64_t bytes = row_bytes(job.m), pn = padded(job.m);
  const uint32_t swizzle = (lane >> 1) & 7;

  // f(i, q, row, col) for the lane's runs of eight columns
  auto runs = [&](auto f) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) f(i, q, 64 * wm + 2 * r + i, 64 * wn + 16 * q + 8 * h);
  };
  auto put = [&](const Mat& x, int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f16x8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = x[i][e & 1][4 * q + e / 2];
          hi[e] = static_cast<_Float16>(v);
          lo[e] = static_cast<_Float16>(v - static_cast<float>(hi[e]));
        }
        uint8_t* row = image[b] + (2 * wn + q / 2) * kStep + (64 * wm + 32 * i + r) * kStepBytes;
        const uint32_t piece = 2 * (2 * (q & 1) + h);
        *reinterpret_cast<f16x8*>(row + ((piece ^ swizzle) << 4)) = hi;
        *reinterpret_cast<f16x8*>(row + (((piece + 1) ^ swizzle) << 4)) = lo;
      }
  };
  // x = factor times the product of images l and r
  auto multiply = [&](Mat& x, int bl, int br, float factor) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][j][e] = 0.0f;
#pragma unroll
    for (int t = 0; t < 2 * kSteps; ++t) {
      i32x4 a[2][2], b[2][2];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = t / 2 * kStep + (32 * f + r) * kStepBytes + (((4 * h + 2 * (t & 1) + e) ^ swizzle) << 4);
          a[f][e] = *reinterpret_cast<const i32x4*>(image[bl] + 64 * wm * kStepBytes + at);
          b[f][e] = *reinterpret_cast<const i32x4*>(image[br] + 64 * wn * kStepBytes + at);
        }
      // lo lo too: small matrices are where it shows
      each_pair<2, 2>([&](auto i, auto j) {
        constexpr int I = decltype(i)::value, J = decltype(j)::value;
        x[I][J] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b[J][1]), __builtin_bit_cast(f16x8, a[I][1]), x[I][J], 0, 0, 0);
      });
      each<HalfOp::terms(0)>([&](auto term) {
        each_pair<2, 2>([&](auto i, auto j) {
          constexpr int I = decltype(i)::value, J = decltype(j)::value;
          HalfOp::multiply<0, decltype(term)::value, I, J>(x[I][J], a[I], b[J], {});
        });
      });
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][j][e] *= factor;
  };

  Mat a, p, q, x;
  runs([&](int i, int c, int row, int col) {
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (row < job.m && col < pn) read_run(job.a + row * bytes, col, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[i][e & 1][4 * c + e / 2] = v[e];
  });
  put(a, 0);
  __syncthreads();
  constexpr float kDown = 1.0f / (1 << kExp);
  float q_factor = 1.0f / (1 << (2 * kExp - kExpQ));
  for (int it = 0; it < args.length; ++it) {
    const bool last = it + 1 == args.length;
    multiply(p, 0, 0, kDown);
    runs([&](int i, int c, int row, int col) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool diagonal = row == col + e && row < job.m;
        p[i][e & 1][4 * c + e / 2] = p[i][e & 1][4 * c + e / 2] * kC + a[i][e & 1][4 * c + e / 2] * kB +
                                     (diagonal ? kA * static_cast<float>(1 << kExp) : 0.0f);
      }
    });
    put(p, 1);  // nothing reads image 1 since the last barrier
    __syncthreads();
    if (!last) {
      multiply(x, 1, 0, kDown);
      __syncthreads();
      put(x, 0);
      __syncthreads();
      multiply(a, 0, 1, kDown);
    }
    if (it == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) q[i][j] = p[i][j];
    } else {
      __syncthreads();
      put(q, 0);
      __syncthreads();
      multiply(q, 1, 0, q_factor);
      q_factor = kDown;  // P has the exponent kExp, Q then stays at its own
    }
    if (!last) {
      __syncthreads();
      put(a, 0);
      __syncthreads();
    }
  }
  runs([&](int i, int c, int row, int col) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = q[i][e & 1][4 * c + e / 2];
    if (row < job.m && col < pn) write_run<8>(job.q + row * bytes, col, v);
  });
}

// ------------------------------------------------------------------ matrices of few rows or columns

// Up to kTiny on the shorter side (an adapter's rank) the products with U are short sums and what would bound the
// way above is its launches.  Here it takes three, in binary64, where up to kTinySteps iterations on A need no fresh
// start: A = U U^T, whose trace is the squared norm; the polynomial Q of A / |U|^2; and Q U / |U|.  More iterations are
// taken in groups, with X in binary64 between them.  (2^-53 of A grows by 11.9 per iteration: under 2^-24 after six,
// 1e-3 after twelve, and behind that the iteration leaves its bounds: 32 on a matrix of one direction ended in NaN.)
// 16 x 4096 takes 34 us, 32 x 4096 57, 5 x 300 21 (the way above: 99 x 300 120, 33 x 4096 182), and the results are within 2.5e-8.  The
// polynomial's products in one workgroup are most of it at 32: twice as many rows would make that chain eight times as long, and
// its four matrices, 34 KB of LDS now, four times as large.
constexpr int kTiny = 32, kTinySteps = 6;
constexpr int kGramColumns = 64, kResultColumns = 256;  // of the longer side, per workgroup and turn
constexpr int kTinyParts = 128;                         // partial A per matrix

struct TinyJob {
  const void* u;  // U, or X between groups
  double *parts, *q;
  void* dst;
  int64_t n, along, across;  // element (i, c) of U's short rows lies at i * across + c * along
  int32_t m;
  uint32_t groups, result_groups;
  float rate;
};
struct TinyArgs {
  TinyJob jobs[kMaxJobs];
  double eps;
  int steps;
  int scaled;  // X, whose norm is not divided by
  float decay;
};
static_assert(sizeof(TinyArgs) <= 4096, "kernel arguments");

// What LDS holds of an element: binary32, or X's binary64.
__device__ __forceinline__ double held(double x) { return x; }
__device__ __forceinline__ float held(float x) { return x; }
__device__ __forceinline__ float held(uint16_t x) { return to_f32(x); }
template <typename ST> using Held = decltype(held(ST{}));

// Columns c0 to c0 + kColumns - 1 of U's short rows in LDS, 0 behind the end.
template <typename ST, int kColumns> __device__ __forceinline__ void load_columns(const TinyJob& job, int64_t c0, Held<ST> (*x)[kColumns + 1]) {
  const ST* u = static_cast<const ST*>(job.u);
  const int all = job.m * kColumns;
#pragma unroll 4
  for (int i = threadIdx.x; i < all; i += 256) {
    // the index that runs along memory first
    const int row = job.along == 1 ? i / kColumns : i % job.m, c = job.along == 1 ? i % kColumns : i / job.m;
    x[row][c] = c0 + c < job.n ? held(u[row * job.across + (c0 + c) * job.along]) : Held<ST>{0};
  }
}

// A thread holds A[i][j] for i = 2 ti, 2 ti + 1 and j likewise.
template <typename ST> __global__ void __launch_bounds__(256) tiny_gram_kernel(TinyArgs a) {
  __shared__ Held<ST> x[kTiny][kGramColumns + 1];
  const TinyJob& job = a.jobs[blockIdx.y];
  if (blockIdx.x >= job.groups) return;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  double s[2][2] = {{0.0, 0.0}, {0.0, 0.0}};
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kGramColumns; c0 < job.n; c0 += static_cast<int64_t>(job.groups) * kGramColumns) {
    load_columns<ST, kGramColumns>(job, c0, x);
    __syncthreads();
    if (2 * ti < job.m && 2 * tj < job.m) {  // rows from m on hold anything, and make sums that nobody reads
#pragma unroll 8
      for (int c = 0; c < kGramColumns; ++c) {
        const double l0 = x[2 * ti][c], l1 = x[2 * ti + 1][c], r0 = x[2 * tj][c], r1 = x[2 * tj + 1][c];
        s[0][0] += l0 * r0;
        s[0][1] += l0 * r1;
        s[1][0] += l1 * r0;
        s[1][1] += l1 * r1;
      }
    }
    __syncthreads();
  }
  double* to = job.parts + static_cast<int64_t>(blockIdx.x) * job.m * job.m;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * ti + i < job.m && 2 * tj + j < job.m) to[(2 * ti + i) * job.m + 2 * tj + j] = s[i][j];
}

// Q = the product of a I + b A + c A^2 over the group's iterations, A = P A P after each, over |U| in the first group.
__global__ void __launch_bounds__(256) tiny_polynomial_kernel(TinyArgs args) {
  typedef double Mat[kTiny][kTiny + 1];
  __shared__ Mat a, p, q, h;
  const TinyJob& job = args.jobs[blockIdx.x];
  const int m = job.m, ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  auto own = [&](auto f) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) f(2 * ti + i, 2 * tj + j, 2 * i + j);
  };
  auto product = [&](const Mat& l, const Mat& r, double (&s)[4]) {  // r is symmetric
    s[0] = s[1] = s[2] = s[3] = 0.0;
    if (2 * ti >= m || 2 * tj >= m) return;
    for (int k0 = 0; k0 < m; k0 += 8)  // places from m on are 0 in the rows before it
#pragma unroll
      for (int k = k0; k < k0 + 8; ++k) {
        const double l0 = l[2 * ti][k], l1 = l[2 * ti + 1][k], r0 = r[2 * tj][k], r1 = r[2 * tj + 1][k];
        s[0] += l0 * r0;
        s[1] += l0 * r1;
        s[2] += l1 * r0;
        s[3] += l1 * r1;
      }
  };
  own([&](int i, int j, int) {
    double s = 0.0;
    if (i < m && j < m) {
#pragma unroll 16
      for (uint32_t g = 0; g < job.groups; ++g) s += job.parts[(static_cast<int64_t>(g) * m + i) * m + j];
    }
    a[i][j] = s;
  });
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < m; ++i) trace += a[i][i];
  __syncthreads();
  const double norm = sqrt(trace), size = args.scaled ? 1.0 : norm < args.eps ? args.eps : norm;
  own([&](int i, int j, int) { a[i][j] = a[i][j] / size / size; });
  __syncthreads();
  for (int it = 0; it < args.steps; ++it) {
    double s[4];
    product(a, a, s);
    own([&](int i, int j, int e) { p[i][j] = s[e] * kExactC + a[i][j] * kExactB + (i == j ? kExactA : 0.0); });
    __syncthreads();
    if (it == 0) own([&](int i, int j, int e) { s[e] = p[i][j]; });
    else product(p, q, s);
    __syncthreads();
    own([&](int i, int j, int e) { q[i][j] = s[e]; });
    if (it + 1 < args.steps) {
      product(p, a, s);
      own([&](int i, int j, int e) { h[i][j] = s[e]; });
      __syncthreads();
      product(h, p, s);
      own([&](int i, int j, int e) { a[i][j] = s[e]; });
    }
    __syncthreads();
  }
  const bool fine = trace - trace == 0.0;  // neither an infinity nor a NaN
  own([&](int i, int j, int) {
    if (i < m && j < m) job.q[i * m + j] = fine ? q[i][j] / size : __builtin_nan("");
  });
}

// dst = Q U, or dst * decay - Q U * rate: a thread per column of U's short rows, eight results of it at a time.  (X
// becomes Q X in place: a workgroup's columns are in its LDS before it writes them.)
template <typename ST, typename OT, bool kStep> __global__ void __launch_bounds__(256) tiny_result_kernel(TinyArgs a) {
  __shared__ Held<ST> x[kTiny][kResultColumns + 1];
  __shared__ __align__(16) double q[kTiny][kTiny];  // q[k][i]: Q is symmetric
  const TinyJob& job = a.jobs[blockIdx.y];
  if (blockIdx.x >= job.result_groups) return;
  for (int i = threadIdx.x; i < kTiny * kTiny; i += 256) {
    const int k = i / kTiny, c = i % kTiny;
    q[k][c] = k < job.m && c < job.m ? job.q[k * job.m + c] : 0.0;
  }
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kResultColumns; c0 < job.n; c0 += static_cast<int64_t>(job.result_groups) * kResultColumns) {
    load_columns<ST, kResultColumns>(job, c0, x);
    __syncthreads();
    const int64_t c = c0 + threadIdx.x;
    for (int i0 = 0; c < job.n && i0 < job.m; i0 += 8) {
      double s[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
      for (int k = 0; k < job.m; ++k) {
        const double v = x[k][threadIdx.x];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += q[k][i0 + i] * v;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < job.m) {
          OT* to = static_cast<OT*>(job.dst) + (i0 + i) * job.across + c * job.along;
          if constexpr (sizeof(OT) == 8) {
            *to = s[i];
          } else {
            const float o = static_cast<float>(s[i]);
            store1(to, kStep ? to_f32(*to) * a.decay - o * job.rate : o);
          }
        }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status() { return hipGetLastError() == hipSuccess ? QOPT_OK : QOPT_ELAUNCH; }
bool bad_dtype(int d) { return d != QOPT_F32 && d != QOPT_BF16; }
uintptr_t size_of(int d) { return d == QOPT_F32 ? 4 : 2; }
bool finite(float x) { return std::isfinite(x); }

// A matrix under work: its shorter side m, its longer side n, and its buffers in the workspace.
struct Matrix {
  const void* src;  // gradient, or the matrix itself
  void* moment;
  float* absmax;
  void* dst;
  int64_t rows, cols, m, n;
  float rate;
  float* u;
  double* parts;
  uint32_t groups;
  uint8_t *x, *xt[2], *g, *p, *h, *q[2];
  double *tiny_parts, *tiny_q, *tiny_x;
};

int64_t up(int64_t bytes) { return ceil_div(bytes, 256) * 256; }

// Lays a matrix's buffers out from `at` on and returns their end.  (u is read before xt[1] is first written.)
uint8_t* lay_out(Matrix& a, uint8_t* at) {
  auto take = [&](int64_t bytes) {
    uint8_t* p = at;
    at += up(bytes);
    return p;
  };
  a.parts = reinterpret_cast<double*>(take(kMaxCodedParts * 8));
  if (a.m <= kTiny) {
    a.u = reinterpret_cast<float*>(take(a.rows * a.cols * 4));
    a.tiny_parts = reinterpret_cast<double*>(take(kTinyParts * a.m * a.m * 8));
    a.tiny_q = reinterpret_cast<double*>(take(a.m * a.m * 8));
    a.tiny_x = reinterpret_cast<double*>(take(a.rows * a.cols * 8));
    return at;
  }
  a.x = take(a.m * row_bytes(a.n));
  a.xt[0] = take(a.n * row_bytes(a.m));
  a.xt[1] = take(a.n * row_bytes(a.m));
  a.u = reinterpret_cast<float*>(a.xt[1]);
  for (uint8_t** b : {&a.g, &a.p, &a.h, &a.q[0], &a.q[1]}) *b = take(a.m * row_bytes(a.m));
  return at;
}

// Iterations on A before it is made anew: fewer where rounding shows in a binary32 destination.  Groups of three, of
// two and single iterations end (1e-6 of the result; products in binary32 in brackets) 3.7, 1.2 and 0.8 off for 17 x
// 23 (0.7), 3.4, 1.5 and 0.9 for 64 x 64 (1.0), 5.9, 1.5 and 1.5 for 99 x 300 (1.4), 2.0, 1.4 and 1.1 for 300 x 1000 (1.6),
// 2.2, 1.6 and 1.9 for 1024 x 1024 (2.6).
int group_steps(int64_t m, int dst_dtype) { return dst_dtype != QOPT_F32 || m > 768 ? 3 : m > 48 ? 2 : 1; }
// Matrices that a batch may hold together.
bool alike(int64_t m, int64_t other, int dst_dtype) {
  return (m <= kTiny) == (other <= kTiny) && (m <= kTiny || group_steps(m, dst_dtype) == group_steps(other, dst_dtype));
}

int64_t tiles_of(int64_t m, int64_t side) { return ceil_div(m, side); }
int64_t triangle(int64_t t) { return t * (t + 1) / 2; }

// Matrices whose products share their launches, in the order of their m and of one length of groups: at most 32, of which 16 that take their
// products in launches of their own (two jobs each), until their symmetric products fill the chip twice.
constexpr size_t kMaxBatch = kMaxJobs, kMaxLarge = kMaxJobs / 2;
size_t batch_end(const std::vector<Matrix>& all, size_t first, int dst_dtype) {
  int64_t tiles = 0;
  size_t i = first, large = 0;
  while (i < all.size() && i - first < kMaxBatch && large < kMaxLarge && tiles < 512 &&
         alike(all[i].m, all[first].m, dst_dtype)) {
    if (all[i].m > kChainDim) ++large;
    tiles += triangle(tiles_of(all[i].m, 256));
    ++i;
  }
  return i;
}

struct Run {
  int source;  // a Source
  int src_dtype, dst_dtype;
  bool update;
  const qopt_codebook* cb;
  const float* grad_scale;
  float mu, omu, eps, decay;
  int nesterov, steps;
  hipStream_t stream;
};

template <typename GT> void launch_source(const SourceArgs& a, int source, dim3 grid, hipStream_t s) {
  if (source == kPlain) hipLaunchKernelGGL((source_kernel<GT, kPlain>), grid, dim3(256), 0, s, a);
  else if (source == kMomentum32) hipLaunchKernelGGL((source_kernel<GT, kMomentum32>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((source_kernel<GT, kMomentum8>), grid, dim3(256), 0, s, a);
}

template <bool kBig, int kEpilogue, typename OT = float>
void launch_product(const ProductArgs& a, hipStream_t s) {
  const dim3 block(kBig ? 512 : 256);
  hipLaunchKernelGGL((product_kernel<kBig, kEpilogue, OT>), dim3(a.whole + a.workers), block, 0, s, a);
  if (a.rest) hipLaunchKernelGGL((join_kernel<kBig, kEpilogue, OT>), dim3(a.rest, 4), block, 0, s, a);
}

constexpr int64_t kCus = 256;
constexpr int64_t kLeastRun = 8;  // steps

// A launch under construction: jobs, and how their tiles are cut up.
struct Launch {
  ProductArgs args = {};
  int epilogue;
  int dst_dtype = QOPT_F32;
  bool big = false;

  explicit Launch(int e) : epilogue(e) {}
  bool symmetric() const { return epilogue == kSymmetric || epilogue == kPolynomial; }
  void add(const Job& j) { args.jobs[args.njobs++] = j; }
  int64_t part_bytes() const { return big ? 256 * 256 * 4 : 128 * 128 * 4; }
  int64_t parts() const { return up(2 * static_cast<int64_t>(args.workers) * part_bytes()); }

  // Tiles of one size, whole or with the last round's steps shared; returns the time by this model, in
  // microseconds.  A step takes a CU 0.72 for a tile of 128 x 128 and 1.8 for one of 256 x 256 while half of the CUs are
  // idle, and 0.95 and 2.7 with all of them busy: the chip's power then holds its clock at 1.7 GHz (2.4), so that
  // idle CUs in the last round cost less than they seem to.
  // Sharing costs a launch (12) and the partial sums' way to memory and back (6 TB/s).
  double cut(bool large, bool share) {
    big = large;
    const int64_t side = large ? 256 : 128;
    const double fast = large ? 1.8 : 0.72, busy = large ? 2.7 : 0.95;
    int64_t tiles = 0, steps = 0, longest = 0;
    bool even = true;
    for (int i = 0; i < args.njobs; ++i) {
      Job& j = args.jobs[i];
      j.first = static_cast<uint32_t>(tiles);
      j.first_step = static_cast<uint32_t>(steps);
      j.tiles_m = static_cast<uint32_t>(ceil_div(j.lrows, side));
      j.tiles_n = static_cast<uint32_t>(ceil_div(j.rrows, side));
      j.steps = j.k_bytes / kStepBytes;
      const int64_t own = symmetric() ? triangle(j.tiles_m) : static_cast<int64_t>(j.tiles_m) * j.tiles_n;
      tiles += own;
      steps += own * j.steps;
      even = even && j.steps == args.jobs[0].steps;
      longest = std::max<int64_t>(longest, j.steps);
    }
    args.whole = static_cast<uint32_t>(tiles);
    args.workers = args.rest = 0;
    const int64_t rounds = even ? ceil_div(tiles, kCus) * longest : tiles <= kCus ? longest : steps / kCus + longest / 2;
    const double alone = std::max(rounds * fast, static_cast<double>(steps) / kCus * busy);
    if (!share) return alone;
    // whole rounds first where all tiles are equally long
    const int64_t whole = even ? tiles / kCus * kCus : 0;
    const int64_t before = even ? whole * longest : 0, shared = steps - before;
    const int64_t workers = std::min(kCus, shared / kLeastRun);
    if (workers < 2 || tiles == whole || steps >= (int64_t{1} << 31)) return alone;
    args.whole = static_cast<uint32_t>(whole);
    args.workers = static_cast<uint32_t>(workers);
    args.first_step = static_cast<uint32_t>(before);
    args.shared = static_cast<uint32_t>(shared);
    args.rest = static_cast<uint32_t>(tiles - whole);
    return static_cast<double>(whole / kCus * longest + ceil_div(shared, workers)) * (workers < kCus ? fast : busy) + 12.0 +
           static_cast<double>(workers + args.rest) * part_bytes() * 2 / 6e6;
  }
  void plan() {
    int best = 0;
    double least = 0;
    for (int i = 0; i < 4; ++i) {
      const double us = cut(i & 1, i & 2);
      if (i == 0 || us < least) {
        least = us;
        best = i;
      }
    }
    cut(best & 1, best & 2);
  }
  int run(uint8_t* parts, hipStream_t s) {
    plan();
    args.parts = reinterpret_cast<f32x4*>(parts);
    return big ? pick<true>(s) : pick<false>(s);
  }
  template <bool kBig> int pick(hipStream_t s) {
    switch (epilogue) {
      case kSymmetric:
        launch_product<kBig, kSymmetric>(args, s);
        break;
      case kPolynomial:
        launch_product<kBig, kPolynomial>(args, s);
        break;
      case kApply:
        launch_product<kBig, kApply>(args, s);
        break;
      case kResult:
        last<kBig, kResult>(s);
        break;
      default:
        last<kBig, kUpdate>(s);
    }
    return launch_status();
  }
  template <bool kBig, int kEpilogue> void last(hipStream_t s) {
    if (dst_dtype == QOPT_F32) launch_product<kBig, kEpilogue, float>(args, s);
    else launch_product<kBig, kEpilogue, uint16_t>(args, s);
  }
};

float power(int e) { return std::ldexp(1.0f, e); }

// l r^T with l [lrows, k], r [rrows, k] as operands; its result has the exponent `to`.
Job job_of(const uint8_t* l, int64_t lrows, const uint8_t* r, int64_t rrows, int64_t k, int exp_in, int to) {
  Job j = {};
  j.l = l;
  j.r = r;
  j.lrows = static_cast<int32_t>(lrows);
  j.rrows = static_cast<int32_t>(rrows);
  j.k_bytes = static_cast<uint32_t>(row_bytes(k));
  j.factor = power(to - exp_in);
  return j;
}

// Bytes that the partial sums of a batch's launches take at most: every kind of launch by its sizes.
int64_t parts_of(const Matrix* mats, int count) {
  int64_t most = 0;
  auto see = [&](int epilogue, int per, auto sizes) {  // per: jobs of a large matrix, none of the others; 0: one of each
    Launch l(epilogue);
    for (int i = 0; i < count; ++i)
      for (int k = 0; k < (per ? mats[i].m > kChainDim ? per : 0 : 1); ++k) l.add(sizes(mats[i]));
    if (l.args.njobs == 0) return;
    l.plan();
    most = std::max(most, l.parts());
  };
  auto job = [&](int64_t lrows, int64_t rrows, int64_t k) { return job_of(nullptr, lrows, nullptr, rrows, k, 0, 0); };
  see(kSymmetric, 0, [&](const Matrix& a) { return job(a.m, a.m, a.n); });
  see(kSymmetric, 1, [&](const Matrix& a) { return job(a.m, a.m, a.m); });
  see(kSymmetric, 2, [&](const Matrix& a) { return job(a.m, a.m, a.m); });
  see(kApply, 0, [&](const Matrix& a) { return job(a.m, a.n, a.m); });
  see(kResult, 0, [&](const Matrix& a) { return a.rows > a.cols ? job(a.n, a.m, a.m) : job(a.m, a.n, a.m); });
  return most;
}

int64_t workspace_of(std::vector<Matrix>& all, int dst_dtype) {
  int64_t most = 0;
  for (size_t first = 0; first < all.size();) {
    const size_t end = batch_end(all, first, dst_dtype);
    uint8_t* at = nullptr;
    for (size_t i = first; i < end; ++i) at = lay_out(all[i], at);
    const int64_t parts = all[first].m <= kTiny ? 0 : parts_of(all.data() + first, static_cast<int>(end - first));
    most = std::max<int64_t>(most, reinterpret_cast<intptr_t>(at) + parts);
    first = end;
  }
  return most;
}
// Whatever the destination's type.
int64_t workspace_of(std::vector<Matrix>& all) { return std::max(workspace_of(all, QOPT_F32), workspace_of(all, QOPT_BF16)); }

int run_source(Matrix* mats, int count, const Run& r) {
  SourceArgs a = {};
  a.cb = r.cb;
  a.grad_scale = r.grad_scale;
  a.mu = r.mu;
  a.omu = r.omu;
  a.nesterov = r.nesterov;
  uint32_t most = 0;
  for (int i = 0; i < count; ++i) {
    Matrix& m = mats[i];
    const int64_t n = m.rows * m.cols;
    m.groups = static_cast<uint32_t>(std::min<int64_t>(ceil_div(n, QOPT_BLOCK), r.source == kMomentum8 ? kMaxCodedParts : kMaxParts));
    most = std::max(most, m.groups);
    a.jobs[i] = {m.src, m.moment, m.absmax, m.u, m.parts, n, m.groups};
  }
  const dim3 grid(most, static_cast<unsigned>(count));
  if (r.src_dtype == QOPT_F32) launch_source<float>(a, r.source, grid, r.stream);
  else launch_source<uint16_t>(a, r.source, grid, r.stream);
  return launch_status();
}

template <typename ST, typename OT> void launch_tiny_result(const TinyArgs& a, bool step, dim3 grid, hipStream_t s) {
  if (step) hipLaunchKernelGGL((tiny_result_kernel<ST, OT, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((tiny_result_kernel<ST, OT, false>), grid, dim3(256), 0, s, a);
}

// One group, from matrices of type ST: to X, or the last one to the destinations.
template <typename ST> void launch_tiny(TinyArgs a, const Matrix* mats, int count, bool last, const Run& r, dim3 gram, dim3 result) {
  hipStream_t s = r.stream;
  hipLaunchKernelGGL(tiny_gram_kernel<ST>, gram, dim3(256), 0, s, a);
  hipLaunchKernelGGL(tiny_polynomial_kernel, dim3(static_cast<unsigned>(count)), dim3(256), 0, s, a);
  if (!last) {
    for (int i = 0; i < count; ++i) a.jobs[i].dst = mats[i].tiny_x;
    hipLaunchKernelGGL((tiny_result_kernel<ST, double, false>), result, dim3(256), 0, s, a);
  } else if (r.dst_dtype == QOPT_F32) {
    launch_tiny_result<ST, float>(a, r.update, result, s);
  } else {
    launch_tiny_result<ST, uint16_t>(a, r.update, result, s);
  }
}

int run_tiny(Matrix* mats, int count, const Run& r) {
  if (r.source != kPlain && run_source(mats, count, r) != QOPT_OK) return QOPT_ELAUNCH;
  TinyArgs a = {};
  a.eps = static_cast<double>(r.eps);
  a.decay = r.decay;
  uint32_t most = 0, most_results = 0;
  for (int i = 0; i < count; ++i) {
    const Matrix& m = mats[i];
    const bool tall = m.rows > m.cols;
    const uint32_t groups = static_cast<uint32_t>(std::min<int64_t>(ceil_div(m.n, kGramColumns), kTinyParts));
    const uint32_t results = static_cast<uint32_t>(ceil_div(m.n, kResultColumns));  // QOPT_MUON_MAX_DIM / 256 at most
    most = std::max(most, groups);
    most_results = std::max(most_results, results);
    a.jobs[i] = {r.source == kPlain ? m.src : m.u, m.tiny_parts, m.tiny_q, m.dst, m.n, tall ? m.cols : 1, tall ? 1 : m.cols,
                 static_cast<int32_t>(m.m), groups, results, m.rate};
  }
  const dim3 grid(most, static_cast<unsigned>(count)), wide(most_results, static_cast<unsigned>(count));
  for (int done = 0; done < r.steps; done += kTinySteps) {
    a.steps = std::min(kTinySteps, r.steps - done);
    a.scaled = done > 0;
    const bool last = done + kTinySteps >= r.steps;
    if (done > 0) {
      for (int i = 0; i < count; ++i) a.jobs[i].u = mats[i].tiny_x;
      launch_tiny<double>(a, mats, count, last, r, grid, wide);
    } else if (r.source == kPlain && r.src_dtype == QOPT_BF16) {
      launch_tiny<uint16_t>(a, mats, count, last, r, grid, wide);
    } else {
      launch_tiny<float>(a, mats, count, last, r, grid, wide);
    }
  }
  return launch_status();
}

int run_batch(Matrix* mats, int count, uint8_t* parts, const Run& r) {
  if (mats[0].m <= kTiny) return run_tiny(mats, count, r);
  hipStream_t s = r.stream;
  if (run_source(mats, count, r) != QOPT_OK) return QOPT_ELAUNCH;
  {
    PackArgs a = {};
    a.njobs = count;
    a.eps = static_cast<double>(r.eps);
    uint32_t tiles = 0;
    for (int i = 0; i < count; ++i) {
      const Matrix& m = mats[i];
      const bool tall = m.rows > m.cols;
      PackJob& j = a.jobs[i];
      j = {r.source == kPlain ? m.src : m.u, tall ? m.xt[0] : m.x, tall ? m.x : m.xt[0], m.parts, m.rows, m.cols, m.groups, tiles,
           static_cast<uint32_t>(ceil_div(padded(m.cols), 256))};
      tiles += j.across * static_cast<uint32_t>(padded(m.rows) / 64);
    }
    const dim3 grid(tiles), block(256);
    if (r.source == kPlain && r.src_dtype == QOPT_BF16) hipLaunchKernelGGL(pack_kernel<uint16_t>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(pack_kernel<float>, grid, block, 0, s, a);
    if (launch_status() != QOPT_OK) return QOPT_ELAUNCH;
  }
  int small = 0;  // matrices whose groups are one launch; they come first
  while (small < count && mats[small].m <= kChainDim) ++small;
  auto symmetric = [&](int64_t m, const uint8_t* a, const uint8_t* b, uint8_t* out, int exp_in, int to) {
    Job j = job_of(a, m, b, m, m, exp_in, to);
    j.out = out;
    j.out_bytes = j.k_bytes;
    return j;
  };
  int rc = QOPT_OK, turn = 0;  // xt[turn] is current
  for (int done = 0; done < r.steps && rc == QOPT_OK;) {
    const int length = std::min(group_steps(mats[0].m, r.dst_dtype), r.steps - done);
    const bool end = done + length == r.steps;
    {
      Launch gram(kSymmetric);
      for (int i = 0; i < count; ++i) {
        Job j = job_of(mats[i].x, mats[i].m, mats[i].x, mats[i].m, mats[i].n, 2 * kExp, kExp);
        j.out = mats[i].g;
        j.out_bytes = static_cast<uint32_t>(row_bytes(mats[i].m));
        gram.add(j);
      }
      rc = gram.run(parts, s);
    }
    if (small && rc == QOPT_OK) {
      ChainArgs a = {};
      a.length = length;
      for (int i = 0; i < small; ++i)
        a.jobs[i] = {mats[i].g, mats[i].q[(length - 1) % 2], static_cast<int32_t>(mats[i].m)};
      hipLaunchKernelGGL(chain_kernel, dim3(static_cast<unsigned>(small)), dim3(256), 0, s, a);
      rc = launch_status();
    }
    int q = 0, exp_q = kExp;  // q[q] is the product of the polynomials so far
    for (int it = 0; it < length; ++it) {
      Launch poly(kPolynomial), both(kSymmetric), next(kSymmetric);
      for (int i = small; i < count; ++i) {
        const Matrix& a = mats[i];
        uint8_t* p = it == 0 ? a.q[0] : a.p;
        Job j = symmetric(a.m, a.g, a.g, p, 2 * kExp, kExp);
        j.add = a.g;
        poly.add(j);
        if (it > 0) both.add(symmetric(a.m, p, a.q[q], a.q[1 - q], kExp + exp_q, kExpQ));
        if (it + 1 < length) {
          both.add(symmetric(a.m, p, a.g, a.h, 2 * kExp, kExp));
          next.add(symmetric(a.m, a.h, p, a.g, 2 * kExp, kExp));
        }
      }
      if (it > 0) {
        q = 1 - q;
        exp_q = kExpQ;
      }
      for (Launch* l : {&poly, &both, &next})
        if (l->args.njobs && rc == QOPT_OK) rc = l->run(parts, s);
    }
    if (rc != QOPT_OK) break;
    done += length;
    if (!end) {
      Launch apply(kApply);
      for (int i = 0; i < count; ++i) {
        const Matrix& a = mats[i];
        Job j = job_of(a.q[q], a.m, a.xt[turn], a.n, a.m, exp_q + kExp, kExp);
        j.out = a.x;
        j.out_bytes = static_cast<uint32_t>(row_bytes(a.n));
        j.out_t = a.xt[1 - turn];
        j.out_t_bytes = static_cast<uint32_t>(row_bytes(a.m));
        apply.add(j);
      }
      rc = apply.run(parts, s);
      turn = 1 - turn;
    } else {
      Launch last(r.update ? kUpdate : kResult);
      last.dst_dtype = r.dst_dtype;
      last.args.decay = r.decay;
      for (int i = 0; i < count; ++i) {
        const Matrix& a = mats[i];
        // the transpose of Q X is X^T Q: a tall matrix's rows
        Job j = a.rows > a.cols ? job_of(a.xt[turn], a.n, a.q[q], a.m, a.m, exp_q + kExp, 0)
                                : job_of(a.q[q], a.m, a.xt[turn], a.n, a.m, exp_q + kExp, 0);
        j.dst = a.dst;
        j.rate = a.rate;
        last.add(j);
      }
      rc = last.run(parts, s);
    }
  }
  return rc;
}

int run_all(std::vector<Matrix>& all, const Run& r, void* workspace) {
  for (size_t first = 0; first < all.size();) {
    const size_t end = batch_end(all, first, r.dst_dtype);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    for (size_t i = first; i < end; ++i) at = lay_out(all[i], at);
    const int rc = run_batch(all.data() + first, static_cast<int>(end - first), at, r);
    if (rc != QOPT_OK) return rc;
    first = end;
  }
  return QOPT_OK;
}

bool bad_dim(int64_t d) { return d < 0 || d > QOPT_MUON_MAX_DIM; }
bool bad_steps(int steps) { return steps < 1 || steps > QOPT_MUON_MAX_STEPS; }
bool bad_eps(float eps) { return !finite(eps) || !(eps > 0.0f); }

Matrix matrix_of(int64_t rows, int64_t cols) {
  Matrix a = {};
  a.rows = rows;
  a.cols = cols;
  a.m = std::min(rows, cols);
  a.n = std::max(rows, cols);
  return a;
}

// The step's matrices with elements, by their m, otherwise in their order.
int collect(const qopt_muon_tensor* tensors, int32_t ntensors, std::vector<Matrix>& all) {
  if (ntensors < 0 || (ntensors > 0 && !tensors)) return QOPT_EINVAL;
  for (int32_t i = 0; i < ntensors; ++i) {
    const qopt_muon_tensor& t = tensors[i];
    if (bad_dim(t.rows) || bad_dim(t.cols)) return QOPT_EINVAL;
    if (t.rows == 0 || t.cols == 0) continue;
    Matrix a = matrix_of(t.rows, t.cols);
    a.src = t.grad;
    a.moment = t.m;
    a.absmax = t.m_absmax;
    a.dst = t.param;
    all.push_back(a);
  }
  std::stable_sort(all.begin(), all.end(), [](const Matrix& a, const Matrix& b) { return a.m < b.m; });
  return QOPT_OK;
}

int muon_step(const qopt_muon_tensor* tensors, int32_t ntensors, int param_dtype, int grad_dtype, bool coded,
              const qopt_codebook* cb, const qopt_muon_hparams* hp, const float* grad_scale, void* workspace,
              size_t workspace_bytes, void* stream) {
  if (!hp) return QOPT_EINVAL;
  std::vector<Matrix> all;
  const int rc = collect(tensors, ntensors, all);
  if (rc != QOPT_OK) return rc;
  if (bad_dtype(param_dtype) || bad_dtype(grad_dtype)) return QOPT_EUNSUPPORTED;
  if (!finite(hp->lr) || hp->lr < 0.0f || !finite(hp->weight_decay) || hp->weight_decay < 0.0f || bad_eps(hp->eps) ||
      !(hp->momentum >= 0.0f && hp->momentum < 1.0f) || bad_steps(hp->steps) || (hp->nesterov != 0 && hp->nesterov != 1))
    return QOPT_EINVAL;
  if (hp->adjust != QOPT_MUON_ORIGINAL && hp->adjust != QOPT_MUON_MATCH_RMS_ADAMW) return QOPT_EUNSUPPORTED;
  for (Matrix& a : all) {
    if (!a.src || !a.moment || !a.dst || (coded && !a.absmax)) return QOPT_EINVAL;
    if (!aligned(a.src, size_of(grad_dtype)) || !aligned(a.dst, size_of(param_dtype)) || !aligned(a.moment, coded ? 1 : 4) ||
        !aligned(a.absmax, 4))
      return QOPT_EALIGN;
    const double r = static_cast<double>(a.rows), c = static_cast<double>(a.cols);
    const double shape = hp->adjust == QOPT_MUON_ORIGINAL ? std::sqrt(std::max(1.0, r / c)) : 0.2 * std::sqrt(std::max(r, c));
    a.rate = static_cast<float>(static_cast<double>(hp->lr) * shape);
  }
  if (!aligned(grad_scale, 4)) return QOPT_EALIGN;
  if (all.empty()) return QOPT_OK;
  if (coded && !cb) return QOPT_EINVAL;
  if (!aligned(cb, 16) || !aligned(workspace, 256)) return QOPT_EALIGN;
  if (!workspace || workspace_bytes < static_cast<size_t>(workspace_of(all))) return QOPT_EINVAL;
  Run r = {};
  r.source = coded ? kMomentum8 : kMomentum32;
  r.src_dtype = grad_dtype;
  r.dst_dtype = param_dtype;
  r.update = true;
  r.cb = cb;
  r.grad_scale = grad_scale;
  r.mu = hp->momentum;
  r.omu = 1.0f - hp->momentum;
  r.eps = hp->eps;
  r.decay = static_cast<float>(1.0 - static_cast<double>(hp->lr) * static_cast<double>(hp->weight_decay));
  r.nesterov = hp->nesterov;
  r.steps = hp->steps;
  r.stream = static_cast<hipStream_t>(stream);
  return run_all(all, r, workspace);
}

// Nothing thrown on the way (a list that finds no memory) leaves a C entry point.
template <typename F> int guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return QOPT_EINTERNAL;
  }
}

// A batch's matrices in lots that bound the list made for them.
constexpr int64_t kMaxMatrices = int64_t{1} << 20;

}  // namespace

// ------------------------------------------------------------------ entry points

extern "C" int qopt_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes || batch < 0 || batch > kMaxMatrices || bad_dim(rows) || bad_dim(cols)) return QOPT_EINVAL;
  *bytes = 0;
  if (batch == 0 || rows == 0 || cols == 0) return QOPT_OK;
  return guarded([&] {
    // the batches but the last are alike; the last has smaller buffers, but may share tiles' steps where they do not
    std::vector<Matrix> all(static_cast<size_t>(std::min<int64_t>(batch, kMaxBatch)), matrix_of(rows, cols));
    const size_t full = batch_end(all, 0, QOPT_F32);  // of equal matrices in either type
    if (batch > static_cast<int64_t>(full)) all.resize(full + batch % full, all[0]);
    *bytes = static_cast<size_t>(workspace_of(all));
    return static_cast<int>(QOPT_OK);
  });
}

extern "C" int qopt_orthogonalize(const void* x_dev, int dtype, int64_t batch, int64_t rows, int64_t cols, int steps, float eps,
                                  void* out_dev, int out_dtype, void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const int rc = qopt_orthogonalize_workspace(batch, rows, cols, &need);
  if (rc != QOPT_OK) return rc;
  if (bad_steps(steps) || bad_eps(eps)) return QOPT_EINVAL;
  if (bad_dtype(dtype) || bad_dtype(out_dtype)) return QOPT_EUNSUPPORTED;
  if (batch == 0 || rows == 0 || cols == 0) return QOPT_OK;
  if (!x_dev || !out_dev || !workspace_dev || workspace_bytes < need) return QOPT_EINVAL;
  if (!aligned(x_dev, size_of(dtype)) || !aligned(out_dev, size_of(out_dtype)) || !aligned(workspace_dev, 256)) return QOPT_EALIGN;
  return guarded([&] {
    std::vector<Matrix> all(static_cast<size_t>(batch), matrix_of(rows, cols));
    for (int64_t i = 0; i < batch; ++i) {
      all[i].src = static_cast<const uint8_t*>(x_dev) + i * rows * cols * static_cast<int64_t>(size_of(dtype));
      all[i].dst = static_cast<uint8_t*>(out_dev) + i * rows * cols * static_cast<int64_t>(size_of(out_dtype));
    }
    Run r = {};
    r.source = kPlain;
    r.src_dtype = dtype;
    r.dst_dtype = out_dtype;
    r.eps = eps;
    r.steps = steps;
    r.stream = static_cast<hipStream_t>(stream);
    return run_all(all, r, workspace_dev);
  });
}

extern "C" int qopt_muon_workspace(const qopt_muon_tensor* tensors, int32_t ntensors, size_t* bytes) {
  if (!bytes) return QOPT_EINVAL;
  *bytes = 0;
  return guarded([&] {
    std::vector<Matrix> all;
    const int rc = collect(tensors, ntensors, all);
    if (rc == QOPT_OK) *bytes = static_cast<size_t>(workspace_of(all));
    return rc;
  });
}

extern "C" int qopt_muon8bit_step(const qopt_muon_tensor* tensors, int32_t ntensors, int param_dtype, int grad_dtype,
                                  const qopt_codebook* cb_m_dev, const qopt_muon_hparams* hp, const float* grad_scale_dev,
                                  void* workspace_dev, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return muon_step(tensors, ntensors, param_dtype, grad_dtype, true, cb_m_dev, hp, grad_scale_dev, workspace_dev, workspace_bytes,
                     stream);
  });
}

extern "C" int qopt_muon32bit_step(const qopt_muon_tensor* tensors, int32_t ntensors, int param_dtype, int grad_dtype,
                                   const qopt_muon_hparams* hp, const float* grad_scale_dev, void* workspace_dev,
                                   size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return muon_step(tensors, ntensors, param_dtype, grad_dtype, false, nullptr, hp, grad_scale_dev, workspace_dev, workspace_bytes,
                     stream);
  });
}

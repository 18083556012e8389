// Layer normalisation of an activation's rows and its gradients, for gfx950: the kernels of
// include/qopt_norm.h.
//
// All of it is bound by memory: forward reads x and writes y, backward reads x and dy and
// writes dx.  A row is held in registers from its one reading to its writing, the next row of
// the same wave or workgroup is loaded meanwhile, and a workgroup goes through many rows, so
// that the weight and the bias are read, and the sums of their gradients written, once for all
// of them.
//
// Measured (bf16, 65536 rows of 4096; a large copy moves 4.9 TB/s): forward 217 us for its 1.07 GB, 4.95 TB/s;
// backward 309 us for 1.61 GB, 5.2 TB/s, and 5.6 us to join the groups' sums.  fp32, 1999 rows of 2048, which the
// last-level cache holds: 9.9, 12.8 and 4.7.  One row of 4096: 3.0, a launch.
//
// The mean is taken first and the squares of what differs from it are summed then: both from registers, so that
// it costs no second reading, and the variance of a row far from zero loses nothing to cancellation.  (The mean's own
// rounding stays, one to three steps of it: fp32 rows 1e4 times their spread away from zero are 4e-4 to 8e-4 off.)  Every sum is
// held in binary32 and joined in a fixed order; a result is rounded to bfloat16 once, where it is stored.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "qopt_norm.h"

namespace {

constexpr int kWave = 64;
constexpr int kChunk = 8;  // consecutive elements of a row per thread: 16 bytes of bf16

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ elements

// Eight elements as they are kept in memory.
template <typename T> struct Raw {
  uint32_t r[kChunk * sizeof(T) / 4];
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}
template <typename T> __device__ __forceinline__ void store1(T* p, float x) {
  if constexpr (sizeof(T) == 4) *p = x;
  else *p = static_cast<uint16_t>(pack_bf16(x, 0.0f) & 0xFFFFu);
}

template <typename T> __device__ __forceinline__ void widen(const Raw<T>& w, float (&v)[kChunk]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) v[e] = __uint_as_float(w.r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kChunk / 2; ++e) {
      v[2 * e] = __uint_as_float(w.r[e] << 16);
      v[2 * e + 1] = __uint_as_float(w.r[e] & 0xFFFF0000u);
    }
  }
}

// How the chunks of a row of `dim` lie.
//   kWhole   dim is a multiple of 8
//   kRagged  it is not: the row's last chunk begins at dim - 8 and shares elements with the one before, whose
//            results both write, the same bits; in sums over the row they count once
//   kShort   dim is less than 8: a single chunk
enum Width : int { kWhole, kRagged, kShort };

// The chunk that begins with element `at` if it is whole.  One behind the row's end has the row's first elements (no
// branch, which would keep the compiler from issuing the loads together), counts none of them and stores nothing.
// (16384 x 1999 in fp32 takes 49 us forward and 76 backward, as 16384 x 2000; with a branch around the loads of a chunk that
// the row's end may cut, 155 and 161.  What alignment the address has costs next to nothing, but rows of bf16 at odd
// ones a quarter: 8192 x 9001 74 us, 9000 54.)
template <Width kWidth> struct Place {
  int at, first, last;  // elements `first` to `last` - 1 of the eight count
  bool in;
  __device__ __forceinline__ Place(int i, int dim) {
    in = i < dim;
    at = !in || kWidth == kShort ? 0 : kWidth == kRagged && i > dim - kChunk ? dim - kChunk : i;
    first = in ? i - at : kChunk;
    last = kWidth == kShort ? dim : kChunk;
  }
  __device__ __forceinline__ bool counts(int e) const { return e >= first && (kWidth != kShort || e < last); }
};

template <Width kWidth, typename T> __device__ __forceinline__ Raw<T> load_chunk(const T* row, const Place<kWidth>& p) {
  Raw<T> w;
  if constexpr (kWidth == kShort) {
    T one[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) one[e] = row[e < p.last ? e : p.last - 1];
    __builtin_memcpy(&w, one, sizeof(w));
  } else {
    __builtin_memcpy(&w, row + p.at, sizeof(w));
  }
  return w;
}
template <Width kWidth, typename T>
__device__ __forceinline__ void store_chunk(T* row, const Place<kWidth>& p, const float (&v)[kChunk]) {
  if (!p.in) return;
  if constexpr (kWidth == kShort) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (e < p.last) store1(row + e, v[e]);
  } else {
    Raw<T> w;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < kChunk; ++e) w.r[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kChunk / 2; ++e) w.r[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    }
    __builtin_memcpy(row + p.at, &w, sizeof(w));
  }
}

// ------------------------------------------------------------------ sums over a row

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) x += __shfl_xor(x, d);
  return x;
}

// The sum over the kWaves waves of a row, for every thread.  `slot` is not the slot of the sum before.
template <int kWaves> __device__ __forceinline__ float row_sum(float x, float (*slots)[kWaves], int slot, int wave) {
  x = wave_sum(x);
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) slots[slot][wave] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x += slots[slot][w];
  }
  return x;
}

// ------------------------------------------------------------------ rows in registers

struct ForwardArgs {
  const void *x, *w, *b;
  void* out;
  float *mean, *rstd;
  int64_t rows, dim, ldx, ldo;
  float eps;
};

struct BackwardArgs {
  const void *x, *w, *dout;
  const float *mean, *rstd;
  void* dx;
  float* part;  // [groups][2][dim]: sums of dout h and dout; or null
  int64_t rows, dim, ldx, lddo, lddx;
};

// Rows that a workgroup holds at once: one per wave, or one.
template <int kWaves> constexpr int rows_at_once() { return kWaves == 1 ? 4 : 1; }
template <int kWaves> constexpr int threads_of() { return kWaves == 1 ? 256 : kWaves * kWave; }

// A row by kWaves waves, kChunks chunks of 8 elements per thread: dim <= kWaves * 64 * 8 * kChunks.
template <typename XT, typename WT, int kWaves, int kChunks, Width kWidth>
__global__ void __launch_bounds__(threads_of<kWaves>()) forward_kernel(ForwardArgs a) {
  __shared__ float slots[2][kWaves];
  constexpr int kLanes = kWaves * kWave, kRows = rows_at_once<kWaves>();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kLanes, dim = static_cast<int>(a.dim);
  auto place = [&](int c) { return Place<kWidth>((c * kLanes + lane) * kChunk, dim); };
  const XT* x = static_cast<const XT*>(a.x);
  const WT *pw = static_cast<const WT*>(a.w), *pb = static_cast<const WT*>(a.b);
  Raw<WT> w[kChunks], b[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    if (pw) w[c] = load_chunk(pw, place(c));
    if (pb) b[c] = load_chunk(pb, place(c));
  }
  const float n = static_cast<float>(a.dim);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (kWaves == 1 ? wave : 0);
  if (row >= a.rows) return;  // whole waves, and whole workgroups where they meet at barriers
  Raw<XT> next[kChunks];
  auto load = [&](int64_t i) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) next[c] = load_chunk(x + i * a.ldx, place(c));
  };
  load(row);
  for (; row < a.rows; row += step) {
    float v[kChunks][kChunk];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const auto p = place(c);
      widen(next[c], v[c]);
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) part += p.counts(e) ? v[c][e] : 0.0f;
      sum += part;
    }
    load(row + step < a.rows ? row + step : row);
    const float mean = row_sum<kWaves>(sum, slots, 0, wave) / n;
    float square = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const auto p = place(c);
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        v[c][e] -= mean;
        part += p.counts(e) ? v[c][e] * v[c][e] : 0.0f;
      }
      square += part;
    }
    const float rstd = 1.0f / sqrtf(row_sum<kWaves>(square, slots, 1, wave) / n + a.eps);
    XT* out = static_cast<XT*>(a.out) + row * a.ldo;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float wv[kChunk], bv[kChunk];
      widen(w[c], wv);
      widen(b[c], bv);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        v[c][e] *= rstd;
        if (pw) v[c][e] *= wv[e];
        if (pb) v[c][e] += bv[e];
      }
      store_chunk(out, place(c), v[c]);
    }
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// The same walk for the gradients: with h = (x - mean) rstd and v = dout w,
//   dx = (v - mean of v - h (mean of v h)) rstd,  dw = sum of dout h,  db = sum of dout.
// A thread's columns are the same in every row, so the sums of dout h and of dout stay in its registers; the
// workgroup's waves that hold rows of their own add theirs in LDS.
template <typename XT, typename WT, int kWaves, int kChunks, Width kWidth>
__global__ void __launch_bounds__(threads_of<kWaves>()) backward_kernel(BackwardArgs a) {
  constexpr int kLanes = kWaves * kWave, kRows = rows_at_once<kWaves>();
  constexpr bool kAhead = kWaves < 16;  // 16 waves have 128 registers each, too few for the next row
  __shared__ float slots[4][kWaves];
  __shared__ float sums[kRows > 1 ? kLanes * kChunk : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kLanes, dim = static_cast<int>(a.dim);
  auto place = [&](int c) { return Place<kWidth>((c * kLanes + lane) * kChunk, dim); };
  const XT *x = static_cast<const XT*>(a.x), *dout = static_cast<const XT*>(a.dout);
  const WT* pw = static_cast<const WT*>(a.w);
  Raw<WT> w[kChunks];
  float dw[kChunks][kChunk], db[kChunks][kChunk];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    if (pw) w[c] = load_chunk(pw, place(c));
#pragma unroll
    for (int e = 0; e < kChunk; ++e) dw[c][e] = db[c][e] = 0.0f;
  }
  const float n = static_cast<float>(a.dim);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (kWaves == 1 ? wave : 0);
  Raw<XT> next_x[kChunks], next_g[kChunks];
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto load = [&](int64_t i) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      next_x[c] = load_chunk(x + i * a.ldx, place(c));
      next_g[c] = load_chunk(dout + i * a.lddo, place(c));
    }
    next_mean = a.mean[i];
    next_rstd = a.rstd[i];
  };
  if (kAhead && row < a.rows) load(row);
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    if (!kAhead) load(row);
    const float mean = next_mean, rstd = next_rstd;
    float h[kChunks][kChunk], v[kChunks][kChunk];
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const auto p = place(c);
      float wv[kChunk];
      widen(next_x[c], h[c]);
      widen(next_g[c], v[c]);
      widen(w[c], wv);
      float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        h[c][e] = (h[c][e] - mean) * rstd;
        dw[c][e] += v[c][e] * h[c][e];
        db[c][e] += v[c][e];
        if (pw) v[c][e] *= wv[e];
        p0 += p.counts(e) ? v[c][e] : 0.0f;
        p1 += p.counts(e) ? v[c][e] * h[c][e] : 0.0f;
      }
      s0 += p0;
      s1 += p1;
    }
    if (kAhead) load(row + step < a.rows ? row + step : row);
    if (a.dx) {
      // one barrier for both sums
      s0 = wave_sum(s0);
      s1 = wave_sum(s1);
      if constexpr (kWaves > 1) {
        if ((threadIdx.x & 63) == 0) {
          slots[2 * turn][wave] = s0;
          slots[2 * turn + 1][wave] = s1;
        }
        __syncthreads();
        s0 = s1 = 0.0f;
#pragma unroll
        for (int u = 0; u < kWaves; ++u) {
          s0 += slots[2 * turn][u];
          s1 += slots[2 * turn + 1][u];
        }
      }
      s0 /= n;
      s1 /= n;
      XT* dx = static_cast<XT*>(a.dx) + row * a.lddx;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[c][e] = (v[c][e] - s0 - h[c][e] * s1) * rstd;
        store_chunk(dx, place(c), v[c]);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.dim;
  auto finish = [&](float (&s)[kChunks][kChunk], float* to) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if constexpr (kRows > 1) {
        for (int u = 0; u < kRows; ++u) {  // the waves in their order
          if (wave == u) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
              float& t = sums[lane * kChunk + e];
              t = u == 0 ? s[c][e] : t + s[c][e];
            }
          }
          __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < kChunk; ++e) s[c][e] = sums[lane * kChunk + e];
        __syncthreads();
        if (wave != 0) continue;
      }
      store_chunk(to, place(c), s[c]);
    }
  };
  finish(dw, part);
  finish(db, part + a.dim);
}

// ------------------------------------------------------------------ rows longer than the registers

constexpr int kLongThreads = 1024;

// f(place) for the thread's chunks of a row.
template <Width kWidth, typename F> __device__ __forceinline__ void chunks_of(int64_t dim, F&& f) {
  const int d = static_cast<int>(dim);
  for (int i = threadIdx.x * kChunk; i < d; i += kLongThreads * kChunk) f(Place<kWidth>(i, d));
}

// The row is read again for each of its sums (from the caches, where it still fits).  4096 x 20000 in bf16: 98 us forward
// and 208 backward, where the sums over the rows are a launch of their own.
template <typename XT, typename WT, Width kWidth> __global__ void __launch_bounds__(kLongThreads) forward_long_kernel(ForwardArgs a) {
  constexpr int kWaves = kLongThreads / kWave;
  __shared__ float slots[2][kWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const WT *pw = static_cast<const WT*>(a.w), *pb = static_cast<const WT*>(a.b);
  const float n = static_cast<float>(a.dim);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    XT* out = static_cast<XT*>(a.out) + row * a.ldo;
    float sum = 0.0f, square = 0.0f;
    chunks_of<kWidth>(a.dim, [&](const Place<kWidth>& p) {
      float v[kChunk], part = 0.0f;
      widen(load_chunk(x, p), v);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) part += p.counts(e) ? v[e] : 0.0f;
      sum += part;
    });
    const float mean = row_sum<kWaves>(sum, slots, 0, wave) / n;
    chunks_of<kWidth>(a.dim, [&](const Place<kWidth>& p) {
      float v[kChunk], part = 0.0f;
      widen(load_chunk(x, p), v);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) part += p.counts(e) ? (v[e] - mean) * (v[e] - mean) : 0.0f;
      square += part;
    });
    const float rstd = 1.0f / sqrtf(row_sum<kWaves>(square, slots, 1, wave) / n + a.eps);
    chunks_of<kWidth>(a.dim, [&](const Place<kWidth>& p) {
      float v[kChunk], wv[kChunk], bv[kChunk];
      widen(load_chunk(x, p), v);
      if (pw) widen(load_chunk(pw, p), wv);
      if (pb) widen(load_chunk(pb, p), bv);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        v[e] = (v[e] - mean) * rstd;
        if (pw) v[e] *= wv[e];
        if (pb) v[e] += bv[e];
      }
      store_chunk(out, p, v);
    });
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename XT, typename WT, Width kWidth> __global__ void __launch_bounds__(kLongThreads) dx_long_kernel(BackwardArgs a) {
  constexpr int kWaves = kLongThreads / kWave;
  __shared__ float slots[2][kWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const WT* pw = static_cast<const WT*>(a.w);
  const float n = static_cast<float>(a.dim);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XT *x = static_cast<const XT*>(a.x) + row * a.ldx, *dout = static_cast<const XT*>(a.dout) + row * a.lddo;
    XT* dx = static_cast<XT*>(a.dx) + row * a.lddx;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    auto load = [&](const Place<kWidth>& p, float (&v)[kChunk], float (&h)[kChunk]) {
      widen(load_chunk(dout, p), v);
      widen(load_chunk(x, p), h);
      float wv[kChunk];
      if (pw) widen(load_chunk(pw, p), wv);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        if (pw) v[e] *= wv[e];
        h[e] = (h[e] - mean) * rstd;
      }
    };
    chunks_of<kWidth>(a.dim, [&](const Place<kWidth>& p) {
      float v[kChunk], h[kChunk], p0 = 0.0f, p1 = 0.0f;
      load(p, v, h);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        p0 += p.counts(e) ? v[e] : 0.0f;
        p1 += p.counts(e) ? v[e] * h[e] : 0.0f;
      }
      s0 += p0;
      s1 += p1;
    });
    s0 = row_sum<kWaves>(s0, slots, 0, wave) / n;
    s1 = row_sum<kWaves>(s1, slots, 1, wave) / n;
    chunks_of<kWidth>(a.dim, [&](const Place<kWidth>& p) {
      float v[kChunk], h[kChunk];
      load(p, v, h);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[e] = (v[e] - s0 - h[e] * s1) * rstd;
      store_chunk(dx, p, v);
    });
  }
}

// Sums of dout h and dout over every gridDim.y-th row, a chunk of columns per thread.
template <typename XT, Width kWidth> __global__ void __launch_bounds__(256) columns_long_kernel(BackwardArgs a) {
  const Place<kWidth> p((blockIdx.x * 256 + threadIdx.x) * kChunk, static_cast<int>(a.dim));
  if (!p.in) return;
  float dw[kChunk], db[kChunk];
#pragma unroll
  for (int e = 0; e < kChunk; ++e) dw[e] = db[e] = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float g[kChunk], h[kChunk];
    widen(load_chunk(static_cast<const XT*>(a.dout) + row * a.lddo, p), g);
    widen(load_chunk(static_cast<const XT*>(a.x) + row * a.ldx, p), h);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      dw[e] += g[e] * ((h[e] - mean) * rstd);
      db[e] += g[e];
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.dim;
  store_chunk(part, p, dw);
  store_chunk(part + a.dim, p, db);
}

// ------------------------------------------------------------------ joining the groups' sums

// dw and db from `groups` partial sums [groups][2][dim].  A workgroup owns 64 columns; its 16 waves take turns
// at the groups, with eight of their sums' loads under way: 4.7 us for 2048 columns (one by one, 9.6), of which
// the 8 MB themselves are 2.
constexpr int kJoinWaves = 16;
template <typename WT>
__global__ void __launch_bounds__(kJoinWaves * kWave) join_kernel(const float* part, int64_t dim, int groups, WT* dw, WT* db) {
  __shared__ float sums[kJoinWaves][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int64_t j = blockIdx.x * int64_t{kWave} + lane;
  WT* to = blockIdx.y == 0 ? dw : db;
  if (!to) return;
  float s = 0.0f;
  if (j < dim)
#pragma unroll 8
    for (int g = wave; g < groups; g += kJoinWaves) s += part[(static_cast<int64_t>(g) * 2 + blockIdx.y) * dim + j];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && j < dim) {
#pragma unroll
    for (int u = 1; u < kJoinWaves; ++u) s += sums[u][lane];
    store1(to + j, s);
  }
}

// ------------------------------------------------------------------ host

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status() { return hipGetLastError() == hipSuccess ? QOPT_OK : QOPT_ELAUNCH; }
bool bad_dtype(int d) { return d != QOPT_F32 && d != QOPT_BF16; }
uintptr_t size_of(int d) { return d == QOPT_F32 ? 4 : 2; }

constexpr int64_t kLongDim = 16384;  // longest row in registers
// Workgroups: as many as are on the chip at once, since each reads the weight and the bias, and in backward
// writes sums of its own: of rows behind 8192 elements forward has two per CU (4096 x 16384 in fp32: 105 us; four
// times as many 119), and backward one behind 6144 (16384 x 8192 in bf16: 150 us; two 158, half of one 197).
// Backward of 65536 x 4096 with 256, 512 and 1024 groups: 330, 293 and 343 us.
constexpr int64_t kForwardGroups = 2048, kBackwardGroups = 512;

// f with the number of waves and chunks of a row as types: forward 32 elements per thread at most, backward,
// which keeps two sums for each of its columns, 24 (the most whose next row fits the registers too).  A shape of
// three chunks between two powers of two, so that no more than a third of the lanes is idle: 8192 x 11008 in bf16
// takes 73 us forward and 109 backward, 91 and 142 with the shapes of 16384; 8192 x 5120 30 and 50 (33 and 55).
template <int kW, int kC> struct Shape {
  static constexpr int kWaves = kW, kChunks = kC;
};
template <typename F> int forward_shape(int64_t dim, F&& f) {
  if (dim <= 512) return f(Shape<1, 1>{});
  if (dim <= 1024) return f(Shape<1, 2>{});
  if (dim <= 2048) return f(Shape<1, 4>{});
  if (dim <= 4096) return f(Shape<4, 2>{});
  if (dim <= 6144) return f(Shape<4, 3>{});
  if (dim <= 8192) return f(Shape<4, 4>{});
  if (dim <= 12288) return f(Shape<8, 3>{});
  return f(Shape<8, 4>{});
}
template <typename F> int backward_shape(int64_t dim, F&& f) {
  if (dim <= 512) return f(Shape<1, 1>{});
  if (dim <= 1024) return f(Shape<1, 2>{});
  if (dim <= 2048) return f(Shape<4, 1>{});
  if (dim <= 4096) return f(Shape<4, 2>{});
  if (dim <= 6144) return f(Shape<4, 3>{});
  if (dim <= 8192) return f(Shape<8, 2>{});
  if (dim <= 12288) return f(Shape<8, 3>{});
  return f(Shape<16, 2>{});
}
// Workgroups for so many rows.
int64_t groups_of(int64_t rows, bool one_wave, int64_t most) {
  const int64_t units = one_wave ? ceil_div(rows, rows_at_once<1>()) : rows;
  return units < most ? units : most;
}
int64_t forward_groups(int64_t rows, int64_t dim) { return groups_of(rows, dim <= 2048, dim <= 8192 ? kForwardGroups : kForwardGroups / 4); }
int64_t backward_groups(int64_t rows, int64_t dim) { return groups_of(rows, dim <= 1024, dim <= 6144 ? kBackwardGroups : kBackwardGroups / 2); }

template <typename XT, typename WT> int launch_forward(const ForwardArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(forward_groups(a.rows, a.dim)));
  if (a.dim > kLongDim) {
    if (a.dim % kChunk == 0) hipLaunchKernelGGL((forward_long_kernel<XT, WT, kWhole>), grid, dim3(kLongThreads), 0, s, a);
    else hipLaunchKernelGGL((forward_long_kernel<XT, WT, kRagged>), grid, dim3(kLongThreads), 0, s, a);
    return launch_status();
  }
  return forward_shape(a.dim, [&](auto shape) {
    constexpr int kW = decltype(shape)::kWaves, kC = decltype(shape)::kChunks;
    const dim3 block(threads_of<kW>());
    if constexpr (kW == 1 && kC == 1) {
      if (a.dim < kChunk) {
        hipLaunchKernelGGL((forward_kernel<XT, WT, kW, kC, kShort>), grid, block, 0, s, a);
        return launch_status();
      }
    }
    if (a.dim % kChunk == 0) hipLaunchKernelGGL((forward_kernel<XT, WT, kW, kC, kWhole>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((forward_kernel<XT, WT, kW, kC, kRagged>), grid, block, 0, s, a);
    return launch_status();
  });
}

template <typename XT, typename WT> int launch_backward(const BackwardArgs& a, hipStream_t s) {
  const unsigned groups = static_cast<unsigned>(backward_groups(a.rows, a.dim));
  if (a.dim > kLongDim) {
    const dim3 columns(static_cast<unsigned>(ceil_div(a.dim, 256 * kChunk)), groups), block(kLongThreads);
    if (a.dim % kChunk == 0) {
      if (a.dx) hipLaunchKernelGGL((dx_long_kernel<XT, WT, kWhole>), dim3(groups), block, 0, s, a);
      if (a.part) hipLaunchKernelGGL((columns_long_kernel<XT, kWhole>), columns, dim3(256), 0, s, a);
    } else {
      if (a.dx) hipLaunchKernelGGL((dx_long_kernel<XT, WT, kRagged>), dim3(groups), block, 0, s, a);
      if (a.part) hipLaunchKernelGGL((columns_long_kernel<XT, kRagged>), columns, dim3(256), 0, s, a);
    }
    return launch_status();
  }
  return backward_shape(a.dim, [&](auto shape) {
    constexpr int kW = decltype(shape)::kWaves, kC = decltype(shape)::kChunks;
    const dim3 block(threads_of<kW>());
    if constexpr (kW == 1 && kC == 1) {
      if (a.dim < kChunk) {
        hipLaunchKernelGGL((backward_kernel<XT, WT, kW, kC, kShort>), dim3(groups), block, 0, s, a);
        return launch_status();
      }
    }
    if (a.dim % kChunk == 0) hipLaunchKernelGGL((backward_kernel<XT, WT, kW, kC, kWhole>), dim3(groups), block, 0, s, a);
    else hipLaunchKernelGGL((backward_kernel<XT, WT, kW, kC, kRagged>), dim3(groups), block, 0, s, a);
    return launch_status();
  });
}

int check_sizes(int64_t rows, int64_t dim) {
  return rows < 0 || dim < 0 || rows > QOPT_NORM_MAX_ROWS || dim > QOPT_NORM_MAX_DIM ? QOPT_EINVAL : QOPT_OK;
}
// Row distances: rows of any length up to 2^62 bytes in all.
bool bad_distance(int64_t ld, int64_t dim) { return ld < dim || ld > (int64_t{1} << 40); }

}  // namespace

// ------------------------------------------------------------------ entry points

extern "C" int qopt_layer_norm_forward(const void* x_dev, int dtype, int64_t rows, int64_t dim, int64_t ldx,
                                       const void* w_dev, const void* b_dev, int w_dtype, float eps, void* out_dev,
                                       int64_t ldo, float* mean_dev, float* rstd_dev, void* stream) {
  const int rc = check_sizes(rows, dim);
  if (rc != QOPT_OK) return rc;
  if (bad_distance(ldx, dim) || bad_distance(ldo, dim) || !(eps >= 0.0f) || std::isinf(eps)) return QOPT_EINVAL;
  if (bad_dtype(dtype) || bad_dtype(w_dtype)) return QOPT_EUNSUPPORTED;
  if (rows == 0 || dim == 0) return QOPT_OK;
  if (!x_dev || !out_dev) return QOPT_EINVAL;
  if (!aligned(x_dev, size_of(dtype)) || !aligned(out_dev, size_of(dtype)) || !aligned(w_dev, size_of(w_dtype)) ||
      !aligned(b_dev, size_of(w_dtype)) || !aligned(mean_dev, 4) || !aligned(rstd_dev, 4))
    return QOPT_EALIGN;
  const ForwardArgs a = {x_dev, w_dev, b_dev, out_dev, mean_dev, rstd_dev, rows, dim, ldx, ldo, eps};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == QOPT_F32)
    return w_dtype == QOPT_F32 ? launch_forward<float, float>(a, s) : launch_forward<float, uint16_t>(a, s);
  return w_dtype == QOPT_F32 ? launch_forward<uint16_t, float>(a, s) : launch_forward<uint16_t, uint16_t>(a, s);
}

extern "C" int qopt_layer_norm_backward_workspace(int64_t rows, int64_t dim, size_t* bytes) {
  if (!bytes || check_sizes(rows, dim) != QOPT_OK) return QOPT_EINVAL;
  *bytes = static_cast<size_t>(backward_groups(rows, dim)) * 2 * dim * sizeof(float);
  return QOPT_OK;
}

extern "C" int qopt_layer_norm_backward(const void* x_dev, int dtype, int64_t rows, int64_t dim, int64_t ldx,
                                        const void* w_dev, int w_dtype, const float* mean_dev, const float* rstd_dev,
                                        const void* dout_dev, int64_t lddo, void* dx_dev, int64_t lddx, void* dw_dev,
                                        void* db_dev, void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const int rc = qopt_layer_norm_backward_workspace(rows, dim, &need);
  if (rc != QOPT_OK) return rc;
  if (bad_distance(ldx, dim) || bad_distance(lddo, dim) || (dx_dev && bad_distance(lddx, dim))) return QOPT_EINVAL;
  if (bad_dtype(dtype) || bad_dtype(w_dtype)) return QOPT_EUNSUPPORTED;
  if (dim == 0) return QOPT_OK;
  const bool sums = dw_dev || db_dev;
  if (rows > 0 && (!x_dev || !dout_dev || !mean_dev || !rstd_dev)) return QOPT_EINVAL;
  if (rows > 0 && sums && (!workspace_dev || workspace_bytes < need)) return QOPT_EINVAL;
  if (!aligned(x_dev, size_of(dtype)) || !aligned(dout_dev, size_of(dtype)) || !aligned(dx_dev, size_of(dtype)) ||
      !aligned(w_dev, size_of(w_dtype)) || !aligned(dw_dev, size_of(w_dtype)) || !aligned(db_dev, size_of(w_dtype)) ||
      !aligned(mean_dev, 4) || !aligned(rstd_dev, 4) || !aligned(workspace_dev, 16))
    return QOPT_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = sums ? static_cast<float*>(workspace_dev) : nullptr;
  if (rows > 0 && (dx_dev || sums)) {
    const BackwardArgs a = {x_dev, w_dev, dout_dev, mean_dev, rstd_dev, dx_dev, part, rows, dim, ldx, lddo, lddx};
    int st;
    if (dtype == QOPT_F32)
      st = w_dtype == QOPT_F32 ? launch_backward<float, float>(a, s) : launch_backward<float, uint16_t>(a, s);
    else
      st = w_dtype == QOPT_F32 ? launch_backward<uint16_t, float>(a, s) : launch_backward<uint16_t, uint16_t>(a, s);
    if (st != QOPT_OK) return st;
  }
  if (!sums) return QOPT_OK;
  const int groups = static_cast<int>(backward_groups(rows, dim));
  const dim3 grid(static_cast<unsigned>(ceil_div(dim, kWave)), 2), block(kJoinWaves * kWave);
  if (w_dtype == QOPT_F32)
    hipLaunchKernelGGL(join_kernel<float>, grid, block, 0, s, part, dim, groups, static_cast<float*>(dw_dev),
                       static_cast<float*>(db_dev));
  else
    hipLaunchKernelGGL(join_kernel<uint16_t>, grid, block, 0, s, part, dim, groups, static_cast<uint16_t*>(dw_dev),
                       static_cast<uint16_t*>(db_dev));
  return launch_status();
}

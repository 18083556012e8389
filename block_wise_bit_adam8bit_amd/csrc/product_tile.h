// One tile of a matrix product a b^T on gfx950's matrix units, for operands whose rows are runs of
// 128-byte steps along the sum: what 256 4-bit values, 64 16-bit values, or 32 values in several
// parts take.  What a step's bytes mean is the business of an `Op`.
#ifndef QOPT_PRODUCT_TILE_H
#define QOPT_PRODUCT_TILE_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace product {

constexpr int kWave = 64;
constexpr int kStepBytes = 128;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}
template <typename T> __device__ __forceinline__ void store1(T* p, float x) {
  if constexpr (sizeof(T) == 4) *p = x;
  else *p = static_cast<uint16_t>(pack_bf16(x, 0.0f) & 0xFFFFu);
}

// Memory by 32-bit offsets; reads past its end give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}

// f(i, j) for all i < kA, j < kB, with the numbers as types (for operands that are literals).
template <int kA, int kB, int kI = 0, typename F> __device__ __forceinline__ void each_pair(F&& f) {
  if constexpr (kI < kA * kB) {
    f(std::integral_constant<int, kI / kB>{}, std::integral_constant<int, kI % kB>{});
    each_pair<kA, kB, kI + 1>(f);
  }
}
template <int kN, int kI = 0, typename F> __device__ __forceinline__ void each(F&& f) {
  if constexpr (kI < kN) {
    f(std::integral_constant<int, kI>{});
    each<kN, kI + 1>(f);
  }
}

// Consecutive workgroups go to the 8 XCDs in turn, each with its own L2: with this order of `all`
// pieces of work every XCD takes one contiguous run of them.
__device__ __forceinline__ uint32_t xcd_order(uint32_t wg, uint32_t all) {
  const uint32_t xcd = wg % 8, each = all / 8, more = all % 8;
  return xcd * each + (xcd < more ? xcd : more) + wg / 8;
}

// One operand's rows from row0 on: at most 2^31 bytes of a tile's rows.
struct Rows {
  const uint8_t* p;
  int64_t row0, rows;
  uint32_t kp;  // bytes per row
};

// The sums of one tile of kM x kN results over steps `first` to `last`, by the kWavesM * kWavesN waves of a
// workgroup.  `lds` holds kBufs * (kM + kN) * 128 bytes.
//
// A step's rows are loaded from memory straight into one of kBufs LDS buffers (no registers), up to kBufs
// steps ahead; their fragments are read from LDS half a step ahead, into one of two register sets:
//     multiply half 0 of step t   | read half 1 of step t
//     wait: step t + 1 has landed, every wave has read all of step t (one barrier per step)
//     multiply half 1 of step t   | read half 0 of step t + 1, start loading step t + kBufs
// with the LDS reads and loads spread between the matrix instructions.
//
// A wave's fragment i of 32 rows holds rows kF r + i (r = 0 .. 31): what belongs to a lane's fragments
// lies side by side in memory, scales as well as results.  In LDS a fragment's 32 rows follow each other, and
// the 16-byte piece c of row r lies at place c ^ (r / 2 % 8): 16 lanes that read one piece of their
// rows touch all 64 banks once.  Of a row's 8 pieces lane (r, h) takes 4 h + 2 half + e, e = 0 and 1: the
// matrix instructions add over the places of a step in any order, as long as both operands have the same.
//
// acc[i][j][4 q + e] of lane (r, h) is row kFm r + i, column kFn (8 q + 4 h + e) + j of the wave's part.
//
// Op: `Side` (what comes with a step's codes: scales), load(t), kSideLoads (memory instructions of a load),
// touch(side), terms(half) and multiply<half, term, i, j>(acc, a, b, side), a and b the two pieces of a fragment.
template <int kM, int kN, int kWavesM, int kWavesN, int kBufs, typename Op> struct Tile {
  static constexpr int kWaves = kWavesM * kWavesN, kThreads = kWaves * kWave;
  static constexpr int kWm = kM / kWavesM, kWn = kN / kWavesN;  // a wave's part of the tile
  static constexpr int kFm = kWm / 32, kFn = kWn / 32;          // fragments of 32 per wave
  static constexpr int kRows = kM + kN;
  static constexpr int kLoads = kRows / 8 / kWaves;             // 8 rows per wave and load
  static constexpr int kLds = kBufs * kRows * kStepBytes;
  static_assert(kM % (8 * kWaves) == 0 && kN % (8 * kWaves) == 0, "whole loads per operand");
  static_assert((kFm == 1 || kFm == 2 || kFm == 4) && (kFn == 1 || kFn == 2 || kFn == 4), "fragments");
  static_assert(kWaves % (2 * kFm) == 0 && kWaves % (2 * kFn) == 0, "a wave's loads fill the same eight rows of 16");
  typedef f32x16 Acc[kFm][kFn];

  static __device__ __forceinline__ void sums(const Rows& a, const Rows& b, const Op& op, uint8_t* lds, int first, int last,
                                              Acc& acc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    auto rows_of = [](const Rows& o, int64_t most) {
      const int64_t left = o.rows - o.row0 < most ? o.rows - o.row0 : most;
      return buffer(o.p + o.row0 * o.kp, static_cast<uint32_t>(left * o.kp));
    };
    const __amdgpu_buffer_rsrc_t ra = rows_of(a, kM), rb = rows_of(b, kN);
    // Lane l of a wave fills bytes 16 l .. 16 l + 15 of 8 rows in LDS, which are kF apart in the operand; kF
    // waves together read 8 kF rows that follow each other.  A row past the operand's last one lies past its
    // buffer's end and reads as 0.
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
        const uint32_t from = static_cast<uint32_t>(at / (8 * frags) * (8 * frags) + frag + frags * (lane >> 3)) *
                              (is_a ? a.kp : b.kp);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb, (lds_void*)(lds + (buf * kRows + row) * kStepBytes), 16,
                                                 from + (is_a ? piece_a : piece_b), t * kStepBytes, 0, 0);
      }
    };

    const int h = lane >> 5;
    const uint32_t at = ((4 * h) ^ ((lane >> 1) & 7)) << 4;
    uint32_t oa = (wm * kWm + (lane & 31)) * kStepBytes + at;
    uint32_t ob = (kM + wn * kWn + (lane & 31)) * kStepBytes + at;
    struct Frags {
      i32x4 a[kFm][2], b[kFn][2];
    };
    auto read_half = [&](Frags& f, int buf, int half) {
      asm volatile("" : "+v"(oa), "+v"(ob));  // addresses are made anew, not kept in registers
      const uint32_t a0 = (oa ^ (half * 32)) + buf * (kRows * kStepBytes), b0 = (ob ^ (half * 32)) + buf * (kRows * kStepBytes);
#pragma unroll
      for (int j = 0; j < kFn; ++j) {
        f.b[j][0] = *reinterpret_cast<const i32x4*>(lds + b0 + j * (32 * kStepBytes));
        f.b[j][1] = *reinterpret_cast<const i32x4*>(lds + (b0 ^ 16) + j * (32 * kStepBytes));
      }
#pragma unroll
      for (int i = 0; i < kFm; ++i) {
        f.a[i][0] = *reinterpret_cast<const i32x4*>(lds + a0 + i * (32 * kStepBytes));
        f.a[i][1] = *reinterpret_cast<const i32x4*>(lds + (a0 ^ 16) + i * (32 * kStepBytes));
      }
    };
    auto multiply = [&](auto half, const Frags& f, const typename Op::Side& c) {
      // the terms one after the other, so that an accumulator's instructions do not follow each other at once
      each<Op::terms(decltype(half)::value)>([&](auto term) {
        each_pair<kFm, kFn>([&](auto i, auto j) {
          constexpr int I = decltype(i)::value, J = decltype(j)::value;
          Op::template multiply<decltype(half)::value, decltype(term)::value, I, J>(acc[I][J], f.a[I], f.b[J], c);
        });
      });
    };
    // The order of a half step's instructions: LDS reads between the matrix instructions of its first half,
    // loads between the ones that follow.  (The compiler keeps the reads and the loads, which write LDS, in
    // their order; a pattern that mixes them is dropped as a whole, and all of them then come before the second
    // matrix instruction: 9 % slower over 4-bit operands, 265 and 239 us for 8192^3.)
    constexpr int kReads = 2 * (kFm + kFn), kMemory = kLoads + Op::kSideLoads;
    auto spread = [&](auto half) {
      constexpr bool kLoading = decltype(half)::value == 1;
      constexpr int kMatrix = kFm * kFn * Op::terms(decltype(half)::value);
      constexpr int kReadsEach = (2 * kReads + kMatrix - 1) / kMatrix, kReadGaps = (kReads + kReadsEach - 1) / kReadsEach;
      constexpr int kLoadsEach = (kMemory + kMatrix - kReadGaps - 1) / (kMatrix - kReadGaps);
#pragma unroll
      for (int i = 0; i < kMatrix; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < kReadGaps) __builtin_amdgcn_sched_group_barrier(0x100, kReadsEach, 0);
        else if (kLoading && (i - kReadGaps) * kLoadsEach < kMemory) __builtin_amdgcn_sched_group_barrier(0x010, kLoadsEach, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // All but the last kLater of this wave's loads have landed and its reads are done; then all waves'.
    constexpr int kLater = (kBufs - 2) * kMemory;
    constexpr int kFirst = kLater + kLoads;
    static_assert(kFirst < 64, "counts of loads under way");
    auto step_barrier = [&] {
      __builtin_amdgcn_s_waitcnt(0x0070 | (kLater & 15) | (kLater >> 4) << 14);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 0> half0{};
    constexpr std::integral_constant<int, 1> half1{};

#pragma unroll
    for (int i = 0; i < kFm; ++i)
#pragma unroll
      for (int j = 0; j < kFn; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    // past the last step the last one is loaded again: no branch, which would keep the compiler from
    // spreading the loads
    auto upto_last = [&](int t) { return t < last ? t : last; };
    if constexpr (kBufs > 2) {
      // Turns of kBufs steps, so that the registers of the sides have fixed places.
      typename Op::Side c[kBufs];
#pragma unroll
      for (int u = 0; u < kBufs; ++u) {
        if (u < kBufs - 1) c[u] = op.load(upto_last(first + u));
        load_step(u, upto_last(first + u));
        __builtin_amdgcn_sched_barrier(0);
      }
      // of the loads behind step `first` one side is not under way yet
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
          c[(u + kLast) % kBufs] = op.load(upto_last(t + kLast));
          read_half(f1, u, 1);
          multiply(half0, f0, c[u]);
          spread(half0);
          step_barrier();
          Op::touch(c[(u + 1) % kBufs]);
          read_half(f0, (u + 1) % kBufs, 0);
          load_step(u, upto_last(t + kBufs));
          multiply(half1, f1, c[u]);
          spread(half1);
          if (++t > last) break;
        }
      }
    } else {
      typename Op::Side c0 = op.load(first), c1 = op.load(upto_last(first + 1));
      load_step(0, first);
      __builtin_amdgcn_sched_barrier(0);
      step_barrier();
      load_step(1, upto_last(first + 1));
      Frags f0, f1;
      read_half(f0, 0, 0);
      for (int t = first; t <= last; ++t) {
        const int buf = (t - first) & 1, ahead = upto_last(t + 2);
        read_half(f1, buf, 1);
        multiply(half0, f0, c0);
        spread(half0);
        step_barrier();
        Op::touch(c1);  // not used before the wait that it landed with
        read_half(f0, buf ^ 1, 0);
        const typename Op::Side c2 = op.load(ahead);
        load_step(buf, ahead);
        multiply(half1, f1, c0);
        spread(half1);
        c0 = c1;
        c1 = c2;
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // no load is on its way into LDS when the workgroup ends
  }
};

}  // namespace product

#endif  // QOPT_PRODUCT_TILE_H

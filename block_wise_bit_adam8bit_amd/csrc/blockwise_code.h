// The block-wise dynamic-tree code on the device: encoding of values against a codebook in LDS
// (qopt_codebook of qopt.h) and the normalisation of a block.
#ifndef QOPT_BLOCKWISE_CODE_H
#define QOPT_BLOCKWISE_CODE_H

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "qopt.h"

namespace blockwise {

// Per-codebook encoder parameters kept in registers for the whole kernel.
struct Encoder {
  const qopt_codebook* cb;  // LDS copy
  uint32_t key0;
  uint32_t last_bucket;
};

__device__ __forceinline__ Encoder make_encoder(const qopt_codebook* lds_cb) {
  Encoder e;
  e.cb = lds_cb;
  e.key0 = lds_cb->key0;
  uint32_t nb = lds_cb->nbuckets;
  nb = nb < 1u ? 1u : (nb > QOPT_MAX_BUCKETS ? QOPT_MAX_BUCKETS : nb);
  e.last_bucket = nb - 1;
  return e;
}

// Magnitude index of a >= 0: bucket start index, plus one if a reaches the single
// threshold that may lie inside the bucket.  The bucket index saturates at 0 below
// bucket 0 and is clamped to the last bucket above it, so every index stays inside
// the tables for any input and any table contents (bucket bytes <= 255, thresh has
// >= 257 entries).
__device__ __forceinline__ uint32_t encode_mag(const Encoder& e, float a) {
  uint32_t i = __builtin_elementwise_sub_sat(__float_as_uint(a) >> 15, e.key0);
  i = i < e.last_bucket ? i : e.last_bucket;
  const uint32_t b = e.cb->bucket[i];
  return b + (a >= e.cb->thresh[b + 1] ? 1u : 0u);
}

// Per-block normalisation: reciprocal, stored absmax and effective sign mask (all
// wave-uniform, held in scalar registers), and whether the block is stored as zero.
struct BlockScale {
  float r;
  float absmax;
  uint32_t sign_mask;
  uint32_t zero;
};

// Zero and subnormal blocks, and blocks whose maximum is NaN, store absmax 0 and
// every code 0.  The kernels branch on `zero` once per block (a scalar branch), so
// the encoder of ordinary blocks carries no test for it.
__device__ __forceinline__ BlockScale block_scale(float amax, uint32_t sign_mask) {
  BlockScale s;
  const bool ok = amax >= FLT_MIN;
  s.r = ok ? 1.0f / amax : 0.0f;
  s.absmax = ok ? amax : 0.0f;
  s.sign_mask = ok ? sign_mask : 0u;
  s.zero = ok ? 0u : 1u;
  return s;
}

// The sign bit is added to the bucket start before the threshold test's carry, so
// the compare feeds one add-with-carry.  This equals (magnitude index | sign bit):
// the magnitude index of a signed table is at most 127 and the sign mask is 0x80,
// or the mask is 0 (an unsigned table, or a zero block).
__device__ __forceinline__ uint32_t encode_signed(const Encoder& e, const BlockScale& s, float x) {
  const float a = fabsf(x) * s.r;
  uint32_t i = __builtin_elementwise_sub_sat(__float_as_uint(a) >> 15, e.key0);
  i = i < e.last_bucket ? i : e.last_bucket;
  const uint32_t b = e.cb->bucket[i];
  const uint32_t sign = x < 0.0f ? s.sign_mask : 0u;
  return (b + sign) + (a >= e.cb->thresh[b + 1] ? 1u : 0u);
}

// Second moments are sums of non-negative terms, so no sign bit is ever set.
__device__ __forceinline__ uint32_t encode_nonneg(const Encoder& e, const BlockScale& s, float x) {
  return encode_mag(e, x * s.r);
}

}  // namespace blockwise

#endif  // QOPT_BLOCKWISE_CODE_H

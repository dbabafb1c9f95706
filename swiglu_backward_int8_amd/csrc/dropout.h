// The mask of a dropout, made where it is used and never stored.
//
// Element (row, col) is decided by one 32-bit word of a counter-based generator:
// word col % 4 of Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with the key rng[0] and
// the counter (col / 4, row, rng[1] + offset).  The counter is the place, so the
// forward and the backward pass, and any division of the rows among lanes, give
// the same mask.  rng lies in device memory: a captured call draws another mask
// at every replay if the program has changed the numbers there.  Two calls with the
// same sum rng[1] + offset draw the same words: a program keeps the sums of its steps
// and dropouts apart (the step in the low word, the dropout in the high one).
#ifndef SILUQUANT_DROPOUT_H
#define SILUQUANT_DROPOUT_H

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rows.h"

namespace rows {

struct Dropout {
  const int64_t* rng;  // null: nothing is dropped
  int64_t offset;
  uint32_t below;  // words below this drop their element: p * 2^32, nearest
  float scale;     // of what is kept: 1 / (1 - p), rounded once
};

struct DropKey {
  uint32_t k0, k1, c2, c3;
};
// The same in every lane (scalar registers).
__device__ __forceinline__ DropKey drop_key(const Dropout& d) {
  const uint64_t seed = (uint64_t)d.rng[0], step = (uint64_t)d.rng[1] + (uint64_t)d.offset;
  auto uniform = [](uint64_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v); };
  return {uniform(seed), uniform(seed >> 32), uniform(step), uniform(step >> 32)};
}

// a ^ b ^ c in one instruction (its truth table is 0x96).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

// The words of columns 4 * block .. + 3 of a row.
__device__ __forceinline__ u32x4 philox(const DropKey& key, uint32_t block, uint32_t row) {
  uint32_t c0 = block, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = xor3((uint32_t)(b >> 32), c1, k0), c1 = (uint32_t)b;
    c2 = xor3((uint32_t)(a >> 32), c3, k1), c3 = (uint32_t)a;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return (u32x4){c0, c1, c2, c3};
}

// Eight values of a row from column col (a multiple of 8) on: one fp32 product
// for what is kept, zero for the others, whatever they were.
__device__ __forceinline__ void drop8(float (&v)[8], const Dropout& d, const DropKey& key, int64_t row, int col) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const u32x4 w = philox(key, (uint32_t)(col >> 2) + k, (uint32_t)row);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * k + i] = w[i] >= d.below ? v[4 * k + i] * d.scale : 0.0f;
  }
}

// ---- host ----
inline bool probability(float p) { return p >= 0.0f && p < 1.0f; }
inline Dropout make_dropout(float p, const int64_t* rng, int64_t offset) {
  return {p > 0.0f ? rng : nullptr, offset, (uint32_t)llrint((double)p * 4294967296.0), (float)(1.0 / (1.0 - (double)p))};
}

}  // namespace rows

#endif

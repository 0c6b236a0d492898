// Which kernel a product of 8-bit matrices takes: rows, tiles of 128 (the last of them in slices) or tiles of 256.
// Host code alone, without HIP, so that the tests ask the same rule which kernels their shapes reach.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "mx_int.h"

namespace mx {

struct Plan8 {
  bool rows, big;  // neither: tiles of 128
  int64_t whole;  // tiles of 128 in front of the sliced ones
  int slices;
  int64_t slice;
};

// What a product takes in tiles of 256 (one workgroup a compute unit) and of 128 (two), by rounds of
// workgroups over 256 compute units, in us: a round's own cost and that of 1024 values of K.  Measured,
// bf16 C: 4096^3 55 to 61 us in tiles of 256, 72 in tiles of 128; 12608x1536x384 37 and 22; 6000x3000x1024 47 and
// 36; 4093x2880x5760 68 and 85; float32 C: 4096^3 106 and 124, 5760x2880x4096 197 and 135 (125 with slices).
// The last tiles of 128, behind the full rounds, are sliced along K if that costs less: one or two workgroups a
// compute unit take step1 and step2 for 128 values of K (`few` times that where one or two rows of tiles read B
// for the first time; not for one or two columns of tiles: there A is the long operand, which the launch before has
// just written, and 14336 rows of 128x4096 take 19.0 us, 128 rows of 14336x4096 unsliced 29.2), the launch that adds
// the slices up kSum8, a slice of a tile written and read kPart8.
// Measured, unsliced and in slices of n: float32 C: 36 tiles of K 12608 86 us,
// (n 5) 27.6, (7) 27.0, (9) 34; 100 of 4096 31.6, (2) 27.2, (4) 28.1; 196 of 2048 20.0, (2) 28.5; 512 + 17 of
// 4096 135, (8) 124; bf16 C: 36 of 12608 54, (5) 20.3, (7) 21.2; 100 of 4096 18.1, (2) 19.5; 512 + 17 of 4096
// 78, (8) 76; 512 + 98 of 2048 27, (2) 29; of B read from HBM, 128 rows of 14336x4096 29.2, (2) 24.5, of
// 4096x4096 26.9, (4) 18.1, (8) 20.9; 256 of 4096x14336 84, (4) 33, (8) 36.
struct Cost8 {
  float round256, k256, round128, k128, step1, step2, few;
};
constexpr Cost8 kCost8 = {12.0f, 11.0f, 3.0f, 8.2f, 0.5f, 0.85f, 1.5f};
constexpr Cost8 kCost8Wide = {12.0f, 24.0f, 3.0f, 15.0f, 1.1f, 1.6f, 1.0f};
constexpr float kSum8 = 5.0f, kPart8 = 0.03f;

// K: the contraction rounded up to 16 values; wide: a float32 C.  Few rows take the wave-per-column kernel.  Else
// tiles by their cost.
inline Plan8 gemm8_plan(int64_t M, int64_t N, int64_t K, bool wide) {
  Plan8 p{M <= 64, false, cdiv(M, 128) * cdiv(N, 128), 1, K};
  if (p.rows) return p;
  const int64_t tiles = cdiv(M, 128) * cdiv(N, 128), tail = tiles % 512;
  const Cost8& c = wide ? kCost8Wide : kCost8;
  const float k = (float)K / 1024.0f, round = c.round128 + c.k128 * k;
  const float few = M <= 256 ? c.few : 1.0f, step1 = c.step1 * few, step2 = c.step2 * few;
  float last = tail == 0 ? 0.f : (tail <= 256 ? c.round128 + step1 * (float)cdiv(K, 128) : round);
  for (int per = 1; per <= 2 && tail > 0 && tail < 256; ++per)
    for (int64_t n = hmin(per * 256 / tail, K / 512); n >= 2; n /= 2) {
      const int64_t slice = cdiv(cdiv(K, n), 512) * 512, slices = cdiv(K, slice);
      const float cost = c.round128 + (tail * slices <= 256 ? step1 : step2) * (float)(slice / 128) + kSum8 +
                         kPart8 * (float)(tail * slices);
      if (slices > 1 && cost < last) last = cost, p.slice = slice, p.slices = (int)slices, p.whole = tiles - tail;
    }
  if (tiles > 256 && (float)cdiv(cdiv(M, 256) * cdiv(N, 256), 256) * (c.round256 + c.k256 * k) <
                         (float)(tiles / 512) * round + last)
    return Plan8{false, true, 0, 1, K};
  return p;
}

// Bytes of the slices' sums.
inline size_t plan8_bytes(const Plan8& p, int64_t M, int64_t N) {
  return p.slices > 1 ? (size_t)(cdiv(M, 128) * cdiv(N, 128) - p.whole) * p.slices * 128 * 128 * sizeof(float) : 0;
}

}  // namespace mx

// What the kernels of the paged 8-bit key/value cache share: parameter blocks,
// the search for a row's sequence, the scale of a page, conversions.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rn_device.cuh"
#include "rn_internal.h"

namespace rn {

// The scale of a page and head is 2^e, e in [kKvExpMin, kKvExpMax], stored as
// the E8M0 byte e + 127: 2^e, 2^-e and 448 2^e are normal floats (448 2^120
// would not be one), so magnitudes above 448 2^119 = 2.98e38 saturate.
constexpr int kKvExpMin = -120, kKvExpMax = 119;

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// exponent of a stored scale; a byte that no write leaves counts as the nearest one that it does
__device__ __forceinline__ int kv_exp(uint32_t byte) { return min(max((int)byte - 127, kKvExpMin), kKvExpMax); }

// smallest e with amax <= 448 2^e: 448 is 0.875 * 2^9 (exponent field 135,
// mantissa 0x600000); amax in bits, finite
__device__ __forceinline__ int kv_exp_of(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvExpMin), kKvExpMax);
}

// (d = 1: the product is n 2^31, its shift 31)
__device__ __forceinline__ int quot(int n, const FastDiv& f) {
  return f.shift < 0 ? n : (int)(__umulhi((uint32_t)n, f.mul) >> f.shift);
}

// rows [s0, s1) of sequence b, whatever the caller's array holds
struct KvRows {
  int s0, s1;
};
__device__ __forceinline__ KvRows kv_rows(const int* starts, int b, int tokens) {
  KvRows r;
  r.s0 = min(max(starts[b], 0), tokens);
  r.s1 = min(max(starts[b + 1], r.s0), tokens);
  return r;
}

// page of a block of 64 positions, -1 where the table has none that exists
__device__ __forceinline__ int kv_page(const KvSeqs& q, int64_t pages, int b, int blk) {
  if (blk < 0 || blk >= q.width) return -1;
  const int p = q.table[(int64_t)b * q.width + blk];
  return p >= 0 && p < pages ? p : -1;
}

// Called by a converged warp: the last b in [0, n) with key(b) <= u, key
// ascending and key(0) <= u; 32 keys at a time.
template <class Key>
__device__ __forceinline__ int kv_find(int n, int u, int lane, Key key) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool below = lane == 0 || (at < n && key(lo + at) <= u);
    const int j = 31 - __clz(__ballot_sync(0xFFFFFFFFu, below));
    lo += j * step;
    n = min(step, n - j * step);
  }
  return lo;
}

// two E4M3 codes -> two f16 (exact); code 0 in the low half
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)c));
  return r;
}
// four codes of a word -> two pairs
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}
// two fp32 -> f16 pair, nearest even; lo in the low half
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace rn

// Products of one or a few tokens with NVFP4 weights (E2M1 codes, an E4M3
// scale per 16 elements, a tensor scale): y = x W^T, and the gated
// feed-forward form of it.
#include <cuda_runtime.h>

#include "rn_act_math.cuh"
#include "rn_device.cuh"
#include "rn_internal.h"

namespace rn {
namespace {

__device__ __forceinline__ float e4m3_f32(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)c));
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(r));
  return f;
}

// sum_k x[k] w[r, k] over the warp (every lane gets it), without 1 / S
__device__ __forceinline__ float dot_row(const uint16_t* x, const uint8_t* codes, const uint8_t* blocks,
                                         int64_t r, int K, int lane) {
  const float lut[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
  float acc = 0.0f;
  for (int g = lane; g < K / 16; g += 32) {
    float t = 0.0f;
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = codes[r * (K / 2) + g * 8 + j];
      const float lo = lut[c & 7] * ((c & 8) ? -1.0f : 1.0f);
      const float hi = lut[(c >> 4) & 7] * ((c & 0x80) ? -1.0f : 1.0f);
      t = fmaf(lo, __uint_as_float((uint32_t)x[g * 16 + 2 * j] << 16), t);
      t = fmaf(hi, __uint_as_float((uint32_t)x[g * 16 + 2 * j + 1] << 16), t);
    }
    acc = fmaf(t, e4m3_f32(blocks[r * (K / 16) + g]), acc);
  }
  return warp_sum(acc);
}

template <int ACT>
__global__ void __launch_bounds__(1024) rn_nvfp4_mv_kernel(const MvParams p) {
  const int lane = threadIdx.x, wp = threadIdx.y;  // 32 warps: one output column each
  const int col = blockIdx.x * 32 + wp;
  const int64_t n = blockIdx.y;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + n * p.K;
  __shared__ float ys[32];
  const bool ok = col < p.H;
  float y = 0.0f;
  if (ok) {
    const float si = *p.scale_inv;
    y = dot_row(x, p.codes, p.blocks, col, p.K, lane) * si;
    if constexpr (ACT != kActNone) {
      const float b = dot_row(x, p.codes, p.blocks, (int64_t)p.H + col, p.K, lane) * si;
      y = act_value<ACT>(y, b, p.limit, p.alpha) * (p.scales ? p.scales[n] : 1.0f);
    }
  }
  if (lane == 0) ys[wp] = y;
  __syncthreads();
  if (wp != 0) return;
  const int c = blockIdx.x * 32 + lane;
  const int64_t o = n * p.H + c;
  y = ys[lane];
  if (p.mode == kFfnMx) {
    const uint32_t code = e8m0_code(warp_max_nan(fabsf(y)));
    static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * e8m0_inv_scale(code), 0.0f);
    if (lane == 0) p.row_scales[n * (p.H / 32) + blockIdx.x] = (uint8_t)code;
  } else if (p.mode == kFfnFp8) {
    const float m = warp_max_nan(fabsf(y));
    if (lane == 0) atomicMax(reinterpret_cast<unsigned*>(p.amax), abs_bits(m));
    if (c < p.H) static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * *p.scale, 0.0f);
  } else if (c < p.H) {
    if (p.mode == kFfnF32)
      static_cast<float*>(p.out)[o] = y;
    else
      static_cast<uint16_t*>(p.out)[o] = (uint16_t)pack_bf16x2(y, 0.0f);
  }
}

}  // namespace

rn_status launch_nvfp4_mv(int act, const MvParams& p, int sms, cudaStream_t s) {
  (void)sms;
  for (int64_t n0 = 0; n0 < p.N; n0 += 65535) {
    MvParams q = p;
    q.N = p.N - n0 < 65535 ? (int)(p.N - n0) : 65535;
    q.x = static_cast<const uint16_t*>(p.x) + n0 * p.K;
    q.scales = p.scales ? p.scales + n0 : nullptr;
    const int esz = p.mode == kFfnBf16 ? 2 : (p.mode == kFfnF32 ? 4 : 1);
    q.out = static_cast<uint8_t*>(p.out) + n0 * p.H * esz;
    q.row_scales = p.row_scales ? p.row_scales + n0 * (p.H / 32) : nullptr;
    const dim3 grid((unsigned)((p.H + 31) / 32), (unsigned)q.N), block(32, 32);
    if (act == kActNone)
      rn_nvfp4_mv_kernel<kActNone><<<grid, block, 0, s>>>(q);
    else if (act == kActSwiglu)
      rn_nvfp4_mv_kernel<kActSwiglu><<<grid, block, 0, s>>>(q);
    else
      rn_nvfp4_mv_kernel<kActClampedSwiglu><<<grid, block, 0, s>>>(q);
    if (cudaGetLastError() != cudaSuccess) return RN_ERR_CUDA;
  }
  return RN_OK;
}

}  // namespace rn

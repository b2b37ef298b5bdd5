// Gated feed-forward block: both projections and the activation (forward),
// and the gradients of the input and the weights (backward).
//
//   forward   p = x W^T [N, 2H] = [a | b],  y = s_i act(a, b)
//   backward  dp = s_i dy act'(pre) (rounded to bf16), dx = dp W,
//             dW = dp^T x
#include <cuda_runtime.h>

#include "rn_act_math.cuh"
#include "rn_device.cuh"
#include "rn_internal.h"

namespace rn {
namespace {

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

constexpr int kTileRows = 8;  // one warp a row

// One output per thread; a warp holds 32 columns of one row, so an MXFP8
// block is a warp.
template <int ACT>
__global__ void __launch_bounds__(32 * kTileRows) rn_ffn_fwd_kernel(const FfnParams p) {
  __shared__ float sx[kTileRows][33], sa[32][33], sb[32][33];
  const int lane = threadIdx.x, ty = threadIdx.y;
  const int64_t row = (int64_t)blockIdx.y * kTileRows + ty;
  const int col = (int)blockIdx.x * 32 + lane;
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  const uint16_t* w = static_cast<const uint16_t*>(p.w);
  float a = 0.0f, b = 0.0f;
  for (int k0 = 0; k0 < p.K; k0 += 32) {
    const int k = k0 + lane;
    sx[ty][lane] = (row < p.N && k < p.K) ? bf16_f32(x[row * p.K + k]) : 0.0f;
    for (int r = ty; r < 32; r += kTileRows) {
      const int c = (int)blockIdx.x * 32 + r;
      const bool ok = c < p.H && k < p.K;
      sa[r][lane] = ok ? bf16_f32(w[(int64_t)c * p.K + k]) : 0.0f;
      sb[r][lane] = ok ? bf16_f32(w[((int64_t)p.H + c) * p.K + k]) : 0.0f;
    }
    __syncthreads();
#pragma unroll 8
    for (int q = 0; q < 32; ++q) {
      a = fmaf(sx[ty][q], sa[lane][q], a);
      b = fmaf(sx[ty][q], sb[lane][q], b);
    }
    __syncthreads();
  }
  const bool ok = row < p.N && col < p.H;
  float y = 0.0f;
  if (ok) {
    y = act_value<ACT>(a, b, p.limit, p.alpha) * (p.scales ? p.scales[row] : 1.0f);
    if (p.pre) {
      uint16_t* pre = static_cast<uint16_t*>(p.pre) + row * 2 * p.H;
      const uint32_t v = pack_bf16x2(a, b);
      pre[col] = (uint16_t)v;
      pre[p.H + col] = (uint16_t)(v >> 16);
    }
  }
  const int64_t o = row * p.H + col;
  if (p.mode == kFfnMx) {
    const float m = warp_max_nan(fabsf(y));
    if (ok) {
      const uint32_t code = e8m0_code(m);
      static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * e8m0_inv_scale(code), 0.0f);
      if (lane == 0) p.row_scales[row * (p.H / 32) + col / 32] = (uint8_t)code;
    }
  } else if (p.mode == kFfnFp8) {
    const float m = warp_max_nan(fabsf(y));
    if (lane == 0) {
      pdl_wait();
      atomicMax(reinterpret_cast<unsigned*>(p.amax), abs_bits(m));
    }
    if (ok) static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * *p.scale, 0.0f);
  } else if (ok) {
    if (p.mode == kFfnF32)
      static_cast<float*>(p.out)[o] = y;
    else
      static_cast<uint16_t*>(p.out)[o] = (uint16_t)pack_bf16x2(y, 0.0f);
  }
}

// c[m, n] = sum_k a(m, k) b(k, n), a(m, k) = a[m * am + k * ak],
// b(k, n) = b[k * bk + n]: bf16 in, fp32 sums, bf16 out
__global__ void __launch_bounds__(32 * kTileRows)
    rn_ffn_mm_kernel(const uint16_t* a, const uint16_t* b, uint16_t* c, int64_t M, int64_t Nn,
                     int64_t Kk, int64_t am, int64_t ak, int64_t bk) {
  __shared__ float sa[kTileRows][33], sb[32][33];
  const int lane = threadIdx.x, ty = threadIdx.y;
  const int64_t m = (int64_t)blockIdx.y * kTileRows + ty, n = (int64_t)blockIdx.x * 32 + lane;
  float acc = 0.0f;
  for (int64_t k0 = 0; k0 < Kk; k0 += 32) {
    const int64_t k = k0 + lane;
    sa[ty][lane] = (m < M && k < Kk) ? bf16_f32(a[m * am + k * ak]) : 0.0f;
    for (int r = ty; r < 32; r += kTileRows)
      sb[r][lane] = (k0 + r < Kk && n < Nn) ? bf16_f32(b[(k0 + r) * bk + n]) : 0.0f;
    __syncthreads();
#pragma unroll 8
    for (int q = 0; q < 32; ++q) acc = fmaf(sa[ty][q], sb[q][lane], acc);
    __syncthreads();
  }
  if (m < M && n < Nn) c[m * Nn + n] = (uint16_t)pack_bf16x2(acc, 0.0f);
}

rn_status launch_mm(const void* a, const void* b, void* c, int64_t M, int64_t Nn, int64_t Kk,
                    int64_t am, int64_t ak, int64_t bk, cudaStream_t s) {
  const dim3 grid((unsigned)((Nn + 31) / 32), (unsigned)((M + kTileRows - 1) / kTileRows));
  rn_ffn_mm_kernel<<<grid, dim3(32, kTileRows), 0, s>>>(
      static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), static_cast<uint16_t*>(c), M,
      Nn, Kk, am, ak, bk);
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

}  // namespace

rn_status launch_ffn_fwd(int act, const FfnParams& p, int sms, cudaStream_t s) {
  (void)sms;
  const dim3 grid((unsigned)((p.H + 31) / 32), (unsigned)((p.N + kTileRows - 1) / kTileRows));
  const dim3 block(32, kTileRows);
  if (act == kActSwiglu)
    rn_ffn_fwd_kernel<kActSwiglu><<<grid, block, 0, s>>>(p);
  else
    rn_ffn_fwd_kernel<kActClampedSwiglu><<<grid, block, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

rn_status launch_ffn_bwd(const FfnBwdParams& p, int sms, cudaStream_t s) {
  (void)sms;
  const int64_t R = 2 * (int64_t)p.H;
  rn_status st;
  if (p.dx && (st = launch_mm(p.dp, p.w, p.dx, p.N, p.K, R, R, 1, p.K, s)) != RN_OK) return st;
  if (p.dw && (st = launch_mm(p.dp, p.x, p.dw, R, p.K, p.N, 1, R, p.K, s)) != RN_OK) return st;
  return RN_OK;
}

}  // namespace rn

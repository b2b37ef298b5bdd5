// Gated feed-forward block: both projections and the activation (forward),
// and the gradients of the input and the weights (backward).
//
//   forward   p = x W^T [N, 2H] = [a | b],  y = s_i act(a, b)
//   backward  dp = s_i dy act'(pre) (rounded to bf16, rn_act.cu), dx = dp W,
//             dW = dp^T x
//
// Every product runs on the tensor cores (tcgen05, bf16 operands, fp32
// accumulators in tensor memory) in one persistent kernel: a pair of CTAs
// works on tiles of 256 x 256 of the result, the reduction in slices of 64.
// Each CTA loads its 128 rows of A and its 128 columns of B of a slice by
// tensor copies (128-byte swizzle, zeros past the ends) into a ring of
// kStages slots; one warp of the pair's leader issues the products of the
// pair (M = 256, N = 256, K = 16), which read both CTAs' shared memory and
// leave 128 rows of the tile in each CTA's tensor memory.  Two accumulators of
// 256 columns alternate, so that the epilogue warps of each CTA work on one
// tile while the next is being summed.
//
// What bounds it is the tensor pipe: 93 % (forward) and 97 % (backward) of the
// active cycles.  8192 x 4096 x 8192 (N x K x H) in a burst, on two GB300s: forward
// 539 and 552 us (2039 and 1992 TFLOP/s; the library's plain product of that
// size 530 and 540 us), the backward's products 1113 and 1157 us (1976 and 1900);
// in a long loop, at the power cap, the forward that keeps the projections
// takes 645 to 666 us (1705 to 1651 TFLOP/s).  Eight epilogue warps with 32-byte
// stores: that forward at 8192 x 1024 x 4096 120 us with four and 16-byte stores,
// 85-87 us so.  Small problems split a tile's reduction: the backward over the
// workspace, the forward over the pairs of a cluster (below).
//
// Forward tiles hold 128 gate and 128 linear columns: the leader's B is 128
// gate rows of W, the other CTA's the 128 linear rows that belong to them, so
// a and b of an output stand in the same lane of tensor memory, 128 columns
// apart, and the activation needs no exchange.  A thread owns one row of the
// tile: an MXFP8 block is 32 columns of one thread.
//
// Operands are read as they lie: reduction-major ("K-major", x and W in the
// forward, dp in dx) or the other way ("MN-major", W in dx, dp and x in dW).
#include <cuda.h>
#include <cuda_runtime.h>

#include "rn_act_math.cuh"
#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_tc.cuh"

namespace rn {
namespace {

__device__ unsigned g_err_ffn;

constexpr int kStages = 6;
constexpr int kOperandBytes = 16384;              // 128 x 64 bf16
constexpr int kStageBytes = 2 * kOperandBytes;    // A and B of one CTA
constexpr int kEpiWarps = 8;                      // two for each 32 lanes of tensor memory
// and one warp each for copies and products: up to 3 warps a scheduler, so at
// most 168 registers a thread.  The forward's epilogues of bf16, FP8 and MXFP8
// spill 16 to 44 bytes: with all 64 outputs of a thread read at once, which hands
// the accumulator back before the stores (8192 x 1024 x 4096 MXFP8 76 us, 80-84
// with 32 at a time and no spills).
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + 1024;

// one product of the launch: tiles of 256 x 256 (forward: 256 x 128 outputs)
struct Job {
  int tiles_m, tiles_n;
  int slices;            // of 64 along the reduction
  int splits, per;       // the reduction in parts of `per` slices
  float* part;           // splits > 1: the parts' sums, fp32 [splits, rows, cols]
  bool a_mn, b_mn;
  void* out;             // dx / dW: bf16 [rows, cols]
  int rows, cols;
};

struct GemmParams {
  Job job[2];
  int n_jobs;
  int pairs;             // of a cluster; more than one: each sums a part of the one tile's reduction
  FfnParams f;           // forward
};

struct Maps {
  CUtensorMap a[2], b[2];
};

struct Tile {
  int job, m, n, split;
};

__host__ __device__ inline int64_t units(const Job& j) { return (int64_t)j.tiles_m * j.tiles_n * j.splits; }

// Tiles in order of their index: jobs one after another, within a job bands
// of 8 tiles of rows walked along the columns, so that the clusters that run
// together share operands in L2.
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int t) {
  Tile r;
  r.job = 0;
  const int n0 = (int)units(p.job[0]);
  if (t >= n0) {
    r.job = 1;
    t -= n0;
  }
  const Job& j = p.job[r.job];
  const int tiles = j.tiles_m * j.tiles_n;
  r.split = t / tiles;
  t -= r.split * tiles;
  const int band = t / (8 * j.tiles_n);
  const int rest = t - band * 8 * j.tiles_n;
  const int h = min(8, j.tiles_m - band * 8);
  r.n = rest / h;
  r.m = band * 8 + rest - r.n * h;
  return r;
}

// 16 columns of one row in one 32-byte store; `o` is 32-byte aligned
__device__ __forceinline__ void store16_bf16(void* o, const float* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o),
               "r"(pack_bf16x2(v[0], v[1])), "r"(pack_bf16x2(v[2], v[3])), "r"(pack_bf16x2(v[4], v[5])),
               "r"(pack_bf16x2(v[6], v[7])), "r"(pack_bf16x2(v[8], v[9])),
               "r"(pack_bf16x2(v[10], v[11])), "r"(pack_bf16x2(v[12], v[13])),
               "r"(pack_bf16x2(v[14], v[15]))
               : "memory");
}

// 8 columns of one row; `o` is 16-byte aligned
__device__ __forceinline__ void store8_bf16(void* o, const float* v) {
  *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// 32 columns of one row, of which `left` exist (a multiple of 8); wide: rows
// of whole 32 bytes, on 32 bytes
__device__ __forceinline__ void store32_bf16(uint16_t* o, const float* v, int left, bool wide) {
  if (wide) {
#pragma unroll
    for (int q = 0; q < 32; q += 16)
      if (q < left) store16_bf16(o + q, v + q);
  } else {
#pragma unroll
    for (int q = 0; q < 32; q += 8)
      if (q < left) store8_bf16(o + q, v + q);
  }
}

// 32 outputs (columns c .. c + 31, of which those below p.H exist) of a row
template <int ACT, int MODE>
__device__ __forceinline__ void epilogue32(const FfnParams& p, int64_t row, int c, const float* a,
                                           const float* b, float s, float fp8_scale, bool wide,
                                           float& amax) {
  if (p.pre != nullptr) {
    uint16_t* pre = static_cast<uint16_t*>(p.pre) + row * 2 * p.H + c;
    store32_bf16(pre, a, p.H - c, wide);
    store32_bf16(pre + p.H, b, p.H - c, wide);
  }
  float y[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) y[i] = act_value<ACT>(a[i], b[i], p.limit, p.alpha) * s;
  const int64_t o = row * p.H + c;
  if constexpr (MODE == kFfnBf16) {
    store32_bf16(static_cast<uint16_t*>(p.out) + o, y, p.H - c, wide);
  } else if constexpr (MODE == kFfnF32) {
#pragma unroll
    for (int q = 0; q < 32; q += 4)
      if (c + q < p.H)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o + q) =
            make_float4(y[q], y[q + 1], y[q + 2], y[q + 3]);
  } else {
    float scale = fp8_scale;
    if constexpr (MODE == kFfnMx) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; i += 2) m = amax_acc2(m, make_float2(y[i], y[i + 1]));
      const uint32_t code = e8m0_code(m);
      scale = e8m0_inv_scale(code);
      p.row_scales[row * (p.H / 32) + c / 32] = (uint8_t)code;
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        if (c + i < p.H) amax = amax_acc2(amax, make_float2(y[i], y[i + 1]));
    }
#pragma unroll
    for (int q = 0; q < 32; q += 8)
      if (c + q < p.H) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* v = y + q + 4 * h;
          const float2 lo = mul2(make_float2(v[0], v[1]), splat2(scale));
          const float2 hi = mul2(make_float2(v[2], v[3]), splat2(scale));
          w[h] = pack_e4m3x4(lo.x, lo.y, hi.x, hi.y);
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + o + q) = make_uint2(w[0], w[1]);
      }
  }
}

// The end of a tile whose reduction the cluster's pairs shared: pair q keeps
// the outputs [q w, q w + w) of the tile, w = 128 / pairs, and gets the other
// pairs' sums for them into the shared memory of its operands (which all
// products have left by then), [pair - 1 of them][gate, linear][w][128 rows].
// The sums are added in the order of the pairs.  Called by every thread of the
// cluster, each of which works on one tile.
template <int ACT, int MODE>
__device__ __forceinline__ void split_epilogue(const GemmParams& p, int cluster, uint32_t tmem, uint32_t ring,
                                               uint32_t done, int warp, int lane, int half, int pair, bool& ok) {
  const int w = 128 / p.pairs;
  const bool works = warp >= 2;
  const int lb = (warp & 3) * 32, side = (warp - 2) / 4;
  const uint32_t ta = tmem + ((uint32_t)lb << 16);
  if (works) ok = mbar_wait_warp(done, 0, &g_err_ffn, kErrStatsWait) && ok;
  tc_fence_after();
  cluster_sync();  // no pair's operands are needed any more
  if (works) {
    for (int q = 0; q < p.pairs; ++q) {
      if (q == pair) continue;
      const int slot = pair < q ? pair : pair - 1;
      const uint32_t to = map_to_rank(ring, 2 * q + half) + (uint32_t)(slot * 2 + side) * w * 512 + (lb + lane) * 4;
      for (int c = 0; c < w; c += 32) {
        float v[32];
        tmem_load32(ta + side * 128 + q * w + c, v);
        tmem_load_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + (c + i) * 512), "f"(v[i]) : "memory");
      }
    }
  }
  cluster_sync();
  if (works && side * 32 < w) {
    const Tile tl = tile_at(p, cluster);
    const int64_t row = (int64_t)tl.m * 256 + half * 128 + lb + lane;
    const int c = side * 32, col = tl.n * 128 + pair * w + c;
    float amax = 0.0f, fp8_scale = 1.0f;
    if constexpr (MODE == kFfnFp8) fp8_scale = *p.f.scale;
    if (col < p.f.H) {
      const bool wide = (p.f.H & 15) == 0 &&
                        ((reinterpret_cast<uintptr_t>(p.f.out) | reinterpret_cast<uintptr_t>(p.f.pre)) & 31) == 0;
      const float s = (p.f.scales != nullptr && row < p.f.N) ? __ldg(p.f.scales + row) : 1.0f;
      float v[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float own[32];
        tmem_load32(ta + h * 128 + pair * w + c, own);
        tmem_load_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[h][i] = 0.0f;
        for (int q = 0; q < p.pairs; ++q) {
          if (q == pair) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[h][i] += own[i];
          } else {
            const uint32_t from = ring + (uint32_t)((q < pair ? q : q - 1) * 2 + h) * w * 512 + (lb + lane) * 4;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float u;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u) : "r"(from + (c + i) * 512) : "memory");
              v[h][i] += u;
            }
          }
        }
      }
      if (row < p.f.N) epilogue32<ACT, MODE>(p.f, row, col, v[0], v[1], s, fp8_scale, wide, amax);
    }
    if constexpr (MODE == kFfnFp8) {
      const float m = warp_max_nan(amax);
      if (lane == 0) atomicMax(reinterpret_cast<unsigned*>(p.f.amax), abs_bits(m));
    }
  }
}

// ACT kActNone: the products of the backward, stored as they are
template <int ACT, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    rn_ffn_kernel(const GemmParams p, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full_b[kStages], empty_b[kStages], done_b[2], free_b[2];
  __shared__ uint32_t tmem_at;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  // of a cluster of `pairs` pairs: the CTA's half of its pair's tile, and its pair
  const int half = (int)rank & 1, pair = (int)rank >> 1;
  const uint32_t leader = rank & ~1u;
  const int cluster = (int)blockIdx.x / (2 * p.pairs), n_clusters = (int)gridDim.x / (2 * p.pairs);
  int total = 0;
  for (int j = 0; j < p.n_jobs; ++j) total += (int)units(p.job[j]);

  if (warp == 0 && lane == 0) {
    for (int j = 0; j < p.n_jobs; ++j) {
      prefetch_map(&maps.a[j]);
      prefetch_map(&maps.b[j]);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full_b[s]), 1);    // the leader's own arrival, with the bytes of both CTAs
      mbar_init(smem_u32(&empty_b[s]), 1);   // the products that read the slot
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&done_b[i]), 1);    // the products of a tile
      mbar_init(smem_u32(&free_b[i]), 2 * kEpiWarps);    // the epilogue warps of both CTAs
    }
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_all(smem_u32(&tmem_at));
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  // everything above overlaps the end of the kernel before; nothing of the
  // caller's memory is touched until it has completed
  pdl_launch_dependents();
  pdl_wait();

  bool ok = true;
  if (warp == 0) {
    RingPos r{0, 0};
    for (int t = cluster; t < total && ok; t += n_clusters) {
      const Tile tl = tile_at(p, t);
      const Job& j = p.job[tl.job];
      const CUtensorMap* ma = &maps.a[tl.job];
      const CUtensorMap* mb = &maps.b[tl.job];
      const int m0 = tl.m * 256 + half * 128;
      const int n0 = ACT == kActNone ? tl.n * 256 + half * 128 : tl.n * 128 + half * p.f.H;
      const int k0 = (tl.split + pair) * j.per, k1 = min(k0 + j.per, j.slices);
      for (int k = k0; k < k1; ++k) {
        if (!mbar_wait_warp(smem_u32(&empty_b[r.slot]), r.phase ^ 1u, &g_err_ffn, kErrEmptyWait)) {
          ok = false;
          break;
        }
        const uint32_t bar = map_to_rank(smem_u32(&full_b[r.slot]), leader);
        if (half == 0) mbar_expect_elected(smem_u32(&full_b[r.slot]), 2 * kStageBytes);
        const uint32_t sa = ring + r.slot * kStageBytes, sb = sa + kOperandBytes;
        if (j.a_mn) {
          tma_load_2d(sa, ma, m0, k * 64, bar);
          tma_load_2d(sa + kOperandBytes / 2, ma, m0 + 64, k * 64, bar);
        } else {
          tma_load_2d(sa, ma, k * 64, m0, bar);
        }
        if (j.b_mn) {
          tma_load_2d(sb, mb, n0, k * 64, bar);
          tma_load_2d(sb + kOperandBytes / 2, mb, n0 + 64, k * 64, bar);
        } else {
          tma_load_2d(sb, mb, k * 64, n0, bar);
        }
        r.advance(1, kStages);
      }
    }
  } else if (warp == 1) {
    if (half == 0) {
      RingPos r{0, 0};
      int it = 0;
      for (int t = cluster; t < total && ok; t += n_clusters, ++it) {
        const Tile tl = tile_at(p, t);
        const Job& j = p.job[tl.job];
        const int k0 = (tl.split + pair) * j.per, k1 = min(k0 + j.per, j.slices);
        const uint32_t acc = it & 1;
        const uint32_t idesc =
            kIdesc256 | (j.a_mn ? kIdescAMN : 0u) | (j.b_mn ? kIdescBMN : 0u);
        const uint64_t da = smem_desc_step(j.a_mn), db = smem_desc_step(j.b_mn);
        if (!mbar_wait_warp(smem_u32(&free_b[acc]), ((it >> 1) & 1) ^ 1u, &g_err_ffn, kErrReadyWait)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait_warp(smem_u32(&full_b[r.slot]), r.phase, &g_err_ffn, kErrFullWait)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = ring + r.slot * kStageBytes;
          uint64_t a = smem_desc(sa, j.a_mn), b = smem_desc(sa + kOperandBytes, j.b_mn);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mma_bf16_pair(tmem + acc * 256, a, b, idesc, k > k0 || q > 0);
            a += da;
            b += db;
          }
          mma_commit(smem_u32(&empty_b[r.slot]), 3u << leader);
          r.advance(1, kStages);
        }
        if (ok) mma_commit(smem_u32(&done_b[acc]), 3u << leader);
      }
    }
  } else if (ACT == kActNone || p.pairs == 1) {
    // epilogue warp: lanes 32 (warp % 4) .. + 31 of tensor memory, one half of the tile's columns
    const int lb = (warp & 3) * 32, side = (warp - 2) / 4;
    float amax = 0.0f, fp8_scale = 1.0f;
    if constexpr (MODE == kFfnFp8) fp8_scale = *p.f.scale;
    // 32-byte stores (whole sectors) where every row starts on 32 bytes
    bool wide = false;
    if constexpr (ACT != kActNone)
      wide = (p.f.H & 15) == 0 &&
             ((reinterpret_cast<uintptr_t>(p.f.out) | reinterpret_cast<uintptr_t>(p.f.pre)) & 31) == 0;
    int it = 0;
    for (int t = cluster; t < total && ok; t += n_clusters, ++it) {
      const Tile tl = tile_at(p, t);
      const Job& j = p.job[tl.job];
      const uint32_t acc = it & 1;
      if (!mbar_wait_warp(smem_u32(&done_b[acc]), (it >> 1) & 1, &g_err_ffn, kErrStatsWait)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int64_t row = (int64_t)tl.m * 256 + half * 128 + lb + lane;
      const uint32_t ta = tmem + acc * 256 + ((uint32_t)lb << 16);
      if constexpr (ACT == kActNone) {
        const int c0 = tl.n * 256;
        const bool wide_out = (j.cols & 15) == 0 && (reinterpret_cast<uintptr_t>(j.out) & 31) == 0;
        // all 128 columns at once: one latency of tensor memory, and the
        // accumulator is free before the stores
        float v[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + side * 128 + 32 * i < j.cols) tmem_load32(ta + side * 128 + 32 * i, v[i]);
        tmem_load_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&free_b[acc]), leader));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + side * 128 + 32 * i;
          if (row < j.rows && j.splits > 1) {
            float* o = j.part + ((int64_t)tl.split * j.rows + row) * j.cols + c;
#pragma unroll
            for (int q = 0; q < 32; q += 4)
              if (c + q < j.cols)
                *reinterpret_cast<float4*>(o + q) =
                    make_float4(v[i][q], v[i][q + 1], v[i][q + 2], v[i][q + 3]);
          } else if (row < j.rows) {
            store32_bf16(static_cast<uint16_t*>(j.out) + row * j.cols + c, v[i], j.cols - c, wide_out);
          }
        }
      } else {
        const int c0 = tl.n * 128;
        const float s = (p.f.scales != nullptr && row < p.f.N) ? __ldg(p.f.scales + row) : 1.0f;
        float a[2][32], b[2][32];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (c0 + side * 64 + 32 * i < p.f.H) {
            tmem_load32(ta + side * 64 + 32 * i, a[i]);
            tmem_load32(ta + 128 + side * 64 + 32 * i, b[i]);
          }
        tmem_load_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&free_b[acc]), leader));
        if (row < p.f.N) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = c0 + side * 64 + 32 * i;
            if (c < p.f.H) epilogue32<ACT, MODE>(p.f, row, c, a[i], b[i], s, fp8_scale, wide, amax);
          }
        }
      }
    }
    if constexpr (MODE == kFfnFp8) {
      const float m = warp_max_nan(amax);
      if (lane == 0) atomicMax(reinterpret_cast<unsigned*>(p.f.amax), abs_bits(m));
    }
  }
  if constexpr (ACT != kActNone) {
    if (p.pairs > 1) split_epilogue<ACT, MODE>(p, cluster, tmem, ring, smem_u32(&done_b[0]), warp, lane, half, pair, ok);
  }
  // A wait that ran out leaves copies and products in flight: give them a
  // millisecond to land before the memory they write is given back.
  if (!ok) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_free_all(tmem);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (no link against the driver
// library); looked up once
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// bf16 [rows, cols], boxes of 64 columns x box_rows rows, 128-byte swizzle
rn_status make_map(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int box_rows) {
  const EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return RN_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? RN_OK
             : RN_ERR_CUDA;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <int ACT, int MODE>
rn_status launch(const GemmParams& p, const Maps& maps, int sms, cudaStream_t s) {
  auto k = rn_ffn_kernel<ACT, MODE>;
  int64_t total = 0;
  for (int j = 0; j < p.n_jobs; ++j) total += units(p.job[j]);
  if (total > INT32_MAX / 2) return RN_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2u * (unsigned)p.pairs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  // pairs that run at the same time; the shared-memory limit is raised first
  static std::atomic<int> kept[kMaxDevices];
  const int resident = once_per_device(kept, [&] {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) != cudaSuccess)
      return -1;
    attr[0].val.clusterDim.x = 2;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)sms / 2 * 2);
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, k, &cfg) == cudaSuccess && n > 0 ? n : -1;
  });
  if (resident < 1) return RN_ERR_CUDA;
  attr[0].val.clusterDim.x = 2u * (unsigned)p.pairs;
  cfg.numAttrs = 2;
  // one tile a cluster where its pairs share the tile, else as many pairs as run at the same time
  cfg.gridDim = dim3(p.pairs > 1 ? 2u * (unsigned)p.pairs * (unsigned)total
                                 : 2u * (unsigned)(total < resident ? total : resident));
  if (cudaLaunchKernelEx(&cfg, k, p, maps) != cudaSuccess) return RN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

template <int ACT>
rn_status launch_mode(const GemmParams& p, const Maps& maps, int sms, cudaStream_t s) {
  switch (p.f.mode) {
    case kFfnBf16: return launch<ACT, kFfnBf16>(p, maps, sms, s);
    case kFfnF32: return launch<ACT, kFfnF32>(p, maps, sms, s);
    case kFfnFp8: return launch<ACT, kFfnFp8>(p, maps, sms, s);
    case kFfnMx: return launch<ACT, kFfnMx>(p, maps, sms, s);
    default: return RN_ERR_INVALID;
  }
}

}  // namespace

// Pairs that share a tile of the forward: 4 or 2 where the tiles are so few
// that every SM still gets at most one CTA (15 clusters of 8 CTAs, 36 of 4 run
// at the same time on a GB300) and the reduction is long (us, shared against
// not: 64 x 8192 x 512 17.0 / 37.5, 256 x 8192 x 2048 24.0 / 38.3, 512 x 4096 x
// 1024 15.4 / 21.2, 32 x 2048 x 2048 10.6 / 12.8; with 16 slices 64 x 1024 x 256
// 9.0 / 8.0, 203 x 1000 x 2056 9.9 / 10.4).
static int share_pairs(int64_t tiles, int slices) {
  if (tiles <= 15 && slices >= 40) return 4;
  if (tiles <= 36 && slices >= 20) return 2;
  return 1;
}

rn_status launch_ffn_fwd(int act, const FfnParams& f, int sms, cudaStream_t s) {
  GemmParams p{};
  p.n_jobs = 1;
  p.f = f;
  const int slices = cdiv(f.K, 64);
  const int64_t tiles = (int64_t)cdiv(f.N, 256) * cdiv(f.H, 128);
  p.pairs = share_pairs(tiles, slices);
  const int per = cdiv(slices, p.pairs);
  p.job[0] = Job{cdiv(f.N, 256), cdiv(f.H, 128), slices, 1, per, nullptr, false, false, nullptr, 0, 0};
  Maps m{};
  rn_status st;
  if ((st = make_map(&m.a[0], f.x, f.N, f.K, 128)) != RN_OK) return st;
  if ((st = make_map(&m.b[0], f.w, 2 * (int64_t)f.H, f.K, 128)) != RN_OK) return st;
  return act == kActSwiglu ? launch_mode<kActSwiglu>(p, m, sms, s)
                           : launch_mode<kActClampedSwiglu>(p, m, sms, s);
}

namespace {

// Adds the parts' sums of up to two products in their order and rounds once.
struct JoinParams {
  const float* part[2];
  void* out[2];
  int splits[2];
  int64_t size[2];  // elements of the product; 0: none
};

constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) rn_ffn_join_kernel(const JoinParams p) {
  pdl_wait();
  for (int j = 0; j < 2; ++j) {
    const int64_t n8 = p.size[j] / 8;
    for (int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; i < n8;
         i += (int64_t)gridDim.x * kJoinThreads) {
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      const float4* q = reinterpret_cast<const float4*>(p.part[j]) + i * 2;
#pragma unroll 4
      for (int s = 0; s < p.splits[j]; ++s) {
        const float4 a = q[s * (p.size[j] / 4)], b = q[s * (p.size[j] / 4) + 1];
        v[0] += a.x;
        v[1] += a.y;
        v[2] += a.z;
        v[3] += a.w;
        v[4] += b.x;
        v[5] += b.y;
        v[6] += b.z;
        v[7] += b.w;
      }
      store8_bf16(static_cast<uint16_t*>(p.out[j]) + i * 8, v);
    }
  }
}

// pairs of SMs on a GB300: what the plan spreads the work over (a constant,
// so that the workspace's size depends on the problem only)
constexpr int64_t kPairs = 76;

// A product's reduction is split where one of its tiles would take longer
// than an even share of the launch's work: into parts of that share, of 8
// slices at least (a part's sums cost about as much as 4 slices), and no more
// than two parts a pair.  203 x 1000 x 2056: dx 30.3 us unsplit.
FfnSplit split_for(int64_t tiles, int64_t slices, int64_t share) {
  int64_t n = 1;
  if (slices > share + share / 4) {
    n = (slices + share - 1) / share;
    if (n > slices / 8) n = slices / 8;
    if (n > 2 * kPairs / tiles) n = 2 * kPairs / tiles;
    if (n < 1) n = 1;
  }
  FfnSplit r;
  r.per = (int)((slices + n - 1) / n);
  r.splits = (int)((slices + r.per - 1) / r.per);
  return r;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

FfnBwdPlan ffn_bwd_plan(int64_t N, int64_t K, int64_t H) {
  FfnBwdPlan p{};
  const int64_t R = 2 * H, kc = (K + 255) / 256;
  const int64_t dx_tiles = (N + 255) / 256 * kc, dx_slices = (R + 63) / 64;
  const int64_t dw_tiles = (R + 255) / 256 * kc, dw_slices = (N + 63) / 64;
  if (N > 0) {
    // (in double: the sizes' product can pass 64 bits; exact where it matters)
    const double work = (double)dx_tiles * (double)dx_slices + (double)dw_tiles * (double)dw_slices;
    const int64_t share = work < 9e15 ? (int64_t)work / kPairs + 1 : INT64_MAX / 2;
    p.dx = split_for(dx_tiles, dx_slices, share);
    p.dw = split_for(dw_tiles, dw_slices, share);
  }
  p.dx_part = up256((size_t)N * R * 2);
  p.dw_part = p.dx_part + (p.dx.splits > 1 ? up256((size_t)p.dx.splits * N * K * 4) : 0);
  p.bytes = p.dw_part + (p.dw.splits > 1 ? up256((size_t)p.dw.splits * R * K * 4) : 0);
  return p;
}

rn_status launch_ffn_bwd(const FfnBwdParams& b, int sms, cudaStream_t s) {
  GemmParams p{};
  p.pairs = 1;
  Maps m{};
  JoinParams jp{};
  const int64_t R = 2 * (int64_t)b.H;
  const FfnBwdPlan plan = ffn_bwd_plan(b.N, b.K, b.H);
  char* ws = static_cast<char*>(b.ws);
  int64_t join = 0;
  rn_status st;
  const auto add = [&](int64_t rows, int64_t red, bool a_mn, const void* bm, int64_t b_rows, void* out,
                       const FfnSplit& sp, size_t part) -> rn_status {
    const int i = p.n_jobs++;
    p.job[i] = Job{cdiv(rows, 256), cdiv(b.K, 256), cdiv(red, 64), sp.splits, sp.per,
                   reinterpret_cast<float*>(ws + part), a_mn, true, out, (int)rows, b.K};
    if (sp.splits > 1) {
      jp.part[i] = p.job[i].part;
      jp.out[i] = out;
      jp.splits[i] = sp.splits;
      jp.size[i] = rows * b.K;
      join += jp.size[i];
    }
    if ((st = make_map(&m.a[i], ws, b.N, R, a_mn ? 64 : 128)) != RN_OK) return st;
    return make_map(&m.b[i], bm, b_rows, b.K, 64);
  };
  if (b.dx != nullptr && (st = add(b.N, R, false, b.w, R, b.dx, plan.dx, plan.dx_part)) != RN_OK) return st;
  if (b.dw != nullptr && (st = add(R, b.N, true, b.x, b.N, b.dw, plan.dw, plan.dw_part)) != RN_OK) return st;
  if (p.n_jobs == 0) return RN_OK;
  if ((st = launch<kActNone, kFfnBf16>(p, m, sms, s)) != RN_OK || join == 0) return st;
  const int64_t blocks = (join / 8 + kJoinThreads - 1) / kJoinThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 8 * sms ? blocks : 8 * sms));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, rn_ffn_join_kernel, jp) != cudaSuccess) return RN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

rn_status read_clear_error_ffn(unsigned* code) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_ffn, sizeof(v)) != cudaSuccess) return RN_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_err_ffn, &zero, sizeof(zero)) != cudaSuccess) return RN_ERR_CUDA;
  *code = v;
  return RN_OK;
}

}  // namespace rn

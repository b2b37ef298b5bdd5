// Products of one or a few tokens with a weight matrix: NVFP4 weights (E2M1
// codes, an E4M3 scale per 16 elements, a tensor scale), plain or as a gated
// feed-forward block, and the bf16 gated block for few tokens.
//
// The weights' bytes are the cost: each is read once, straight from global
// memory into the registers of the lane whose matrix fragment it is, and
// multiplied by mma.sync m16n8k16 with the weights as the 16 rows and the
// tokens as the 8 columns (few tokens leave most of a tcgen05 tile empty, and
// its operands would have to pass through shared memory, NVFP4 ones
// expanded fourfold).  Which k a lane's registers stand for is free as long as
// both operands agree, so a lane takes 16 contiguous bytes of a row (32 NVFP4
// codes, 8 bf16): four lanes read 64 contiguous bytes, an "item" is that of 32
// rows (16 gate and 16 linear rows, or 32 rows of a plain product), and each
// warp keeps kDepth items in flight.
//
// The tokens stand in shared memory in the order the fragments want them
// (16-byte conflict-free reads).  NVFP4 weights become f16 with one
// conversion and one product a pair: E2M1 value x E4M3 scale has at most 6
// significant bits and lies in [2^-10, 2688], so it is exact in f16.  The
// tokens, bf16, become f16 too, each times a power of two that puts its
// largest magnitude at 2^14: exact unless a token's magnitudes span more than
// 2^31; a CTA that finds an element that is not exact keeps its tokens in
// bf16 and expands the weights to bf16 (exact as well), which is slower.  Sums
// are fp32.
//
// Warps split the reduction KW ways and the rows 8 / KW ways, clusters of S
// CTAs split it S ways more (each holds its part of the tokens); the parts
// meet in shared memory, of the cluster's CTAs in turn, and are added in a
// fixed order.
#include <cuda_runtime.h>

#include "rn_act_math.cuh"
#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_tc.cuh"

namespace rn {
namespace {

constexpr int kMvThreads = 256;
constexpr int kMvWarps = kMvThreads / 32;
constexpr int kDepth = 2;      // items in flight per warp
constexpr int kPartStride = 36;  // floats per token of a warp's partial sums (32 rows, no bank conflicts)

enum WeightKind : int { kWBf16 = 0, kWNvfp4 = 1 };

struct MvPlan {
  int kw;       // warps along the reduction
  int split;    // CTAs of a cluster along the reduction
  int chunks;   // chunks (128 / 32 elements) of the reduction
  int part;     // chunks per CTA of the cluster
  int slab;     // chunks whose tokens are in shared memory at a time
  int steps;    // groups of 8 / kw row tiles
  int batch;    // steps whose sums are kept while the slabs change (slab < part)
};

__device__ __forceinline__ uint4 ldg_w16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_w8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// D += A B, m16n8k16, fp32 sums
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the four pairs of E2M1 codes of a word -> f16x2 (even element low)
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// two E4M3 codes -> f16x2 (exact)
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)c));
  return r;
}

__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// one item of a lane: 16 bytes of rows g and g + 8 of two 16-row tiles, and
// for NVFP4 the two scale codes of each
struct Item {
  uint4 w[2][2];
  uint32_t s[2][2];
};

// the rows a lane reads: row g of both tiles, and how far on row g + 8 is
struct Rows {
  const uint8_t* w[2];
  const uint8_t* s[2];
  int dw[2], ds[2];
};

template <int WK, int T>
struct Mv {
  static constexpr int CK = WK == kWNvfp4 ? 128 : 32;  // reduction elements of a chunk
  static constexpr int J = CK / 32;                    // 16-byte pieces of a token a lane reads per chunk

  // rows of row tile `rt`: a plain product's 32, or 16 gate and 16 linear
  // ones; rows past the end read the last row (their sums are dropped)
  template <bool GATED>
  __device__ __forceinline__ static void rows(const MvParams& p, int rt, int lane, Rows& r) {
    const int g = lane >> 2;
    const int64_t pitch = WK == kWNvfp4 ? p.K / 2 : p.K * 2ll;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int at = GATED ? rt * 16 : rt * 32 + m * 16;
      const int r0 = min(at + g, p.H - 1), r1 = min(at + g + 8, p.H - 1);
      const int64_t row = r0 + (GATED ? (int64_t)m * p.H : 0);
      r.w[m] = static_cast<const uint8_t*>(p.w) + row * pitch;
      r.dw[m] = (r1 - r0) * (int)pitch;  // 8 rows: K < 2^26 keeps it in 32 bits
      if constexpr (WK == kWNvfp4) {
        r.s[m] = p.blocks + row * (p.K / 16);
        r.ds[m] = (r1 - r0) * (p.K / 16);
      }
    }
  }

  __device__ __forceinline__ static void load(const MvParams& p, const Rows& r, int chunk, int lane,
                                              Item& it) {
    const int t = lane & 3;
    if constexpr (WK == kWBf16) {
      const int k = chunk * 32 + t * 8;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          it.w[m][h] = k < p.K ? ldg_w16(r.w[m] + (h ? r.dw[m] : 0) + k * 2) : make_uint4(0, 0, 0, 0);
    } else {
      // past the row's end the last blocks are read again: the tokens are 0 there
      const int k = chunk * 128 + t * 32;
      if ((p.K & 31) == 0) {  // rows of whole 16-byte pieces
        const int at = min(k, p.K - 32);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            it.w[m][h] = ldg_w16(r.w[m] + (h ? r.dw[m] : 0) + at / 2);
            it.s[m][h] =
                __ldg(reinterpret_cast<const unsigned short*>(r.s[m] + (h ? r.ds[m] : 0) + at / 16));
          }
      } else {  // an odd number of blocks: rows on 8 bytes
        const int at0 = min(k, p.K - 16), at1 = min(k + 16, p.K - 16);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* w = r.w[m] + (h ? r.dw[m] : 0);
            const uint8_t* sc = r.s[m] + (h ? r.ds[m] : 0);
            const uint2 lo = ldg_w8(w + at0 / 2), hi = ldg_w8(w + at1 / 2);
            it.w[m][h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            it.s[m][h] = __ldg(sc + at0 / 16) | (uint32_t)__ldg(sc + at1 / 16) << 8;
          }
      }
    }
  }

  // where this lane's fragments of each group of 8 tokens start in a chunk (in 16 bytes); columns
  // without a token read the last token's: their sums are dropped
  __device__ __forceinline__ static void lane_at(int n, int lane, int (&at)[T]) {
#pragma unroll
    for (int t = 0; t < T; ++t) at[t] = min(t * 8 + (lane >> 2), n - 1) * 4 + (lane & 3);
  }

  // acc += item x tokens; xs: the chunk's fragments
  template <bool WIDE>
  __device__ __forceinline__ static void compute(const Item& it, const uint4* xs, int n,
                                                 const int (&at)[T], float (&acc)[2][T][4]) {
    if constexpr (WK == kWBf16) {
      uint4 b[T];
#pragma unroll
      for (int t = 0; t < T; ++t) b[t] = xs[at[t]];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t a0[4] = {it.w[m][0].x, it.w[m][1].x, it.w[m][0].y, it.w[m][1].y};
        const uint32_t a1[4] = {it.w[m][0].z, it.w[m][1].z, it.w[m][0].w, it.w[m][1].w};
#pragma unroll
        for (int t = 0; t < T; ++t) {
          mma16816<false>(acc[m][t], a0, b[t].x, b[t].y);
          mma16816<false>(acc[m][t], a1, b[t].z, b[t].w);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // 8 codes of each row
        uint4 b[T];
#pragma unroll
        for (int t = 0; t < T; ++t) b[t] = xs[q * 4 * n + at[t]];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w = q == 0 ? it.w[m][h].x : q == 1 ? it.w[m][h].y : q == 2 ? it.w[m][h].z : it.w[m][h].w;
            const uint32_t s2 = e4m3x2_f16(it.s[m][h]);
            const uint32_t s = __byte_perm(s2, 0u, q < 2 ? 0x1010 : 0x3232);
            e2m1x8_f16(w, v[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[h][i] = mul_f16x2(v[h][i], s);
              if constexpr (WIDE) {
                const float2 f = f16x2_f32(v[h][i]);
                v[h][i] = pack_bf16x2(f.x, f.y);
              }
            }
          }
          const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]};
          const uint32_t a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
          for (int t = 0; t < T; ++t) {
            mma16816<!WIDE>(acc[m][t], a0, b[t].x, b[t].y);
            mma16816<!WIDE>(acc[m][t], a1, b[t].z, b[t].w);
          }
        }
      }
    }
  }
};

// y of one output column and token: stored as p.mode asks (kFfnMx: the warp
// holds the 32 columns of a block)
template <int ACT>
__device__ __forceinline__ void finish(const MvParams& p, int n, int col, float a, float b, float* amax) {
  const bool ok = col < p.H;
  float y = a;
  if constexpr (ACT != kActNone) {
    y = act_value<ACT>(a, b, p.limit, p.alpha) * (p.scales ? __ldg(p.scales + n) : 1.0f);
    if (p.pre != nullptr && ok) {
      uint16_t* pre = static_cast<uint16_t*>(p.pre) + (int64_t)n * 2 * p.H;
      const uint32_t v = pack_bf16x2(a, b);
      pre[col] = (uint16_t)v;
      pre[(int64_t)p.H + col] = (uint16_t)(v >> 16);
    }
  }
  const int64_t o = (int64_t)n * p.H + col;
  if (p.mode == kFfnMx) {
    const uint32_t code = e8m0_code(warp_max_nan(fabsf(y)));
    if (ok) {
      static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * e8m0_inv_scale(code), 0.0f);
      if ((col & 31) == 0) p.row_scales[(int64_t)n * (p.H / 32) + col / 32] = (uint8_t)code;
    }
  } else if (ok) {
    if (p.mode == kFfnBf16) {
      static_cast<uint16_t*>(p.out)[o] = (uint16_t)pack_bf16x2(y, 0.0f);
    } else if (p.mode == kFfnF32) {
      static_cast<float*>(p.out)[o] = y;
    } else {
      *amax = amax_acc(*amax, y);
      static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * __ldg(p.scale), 0.0f);
    }
  }
}

// the tokens' elements of chunks lo .. hi - 1, in fragment order (zeros past
// the row's end); returns whether they had to stay bf16 (NVFP4).  inv: what each token's sums are
// multiplied with.
template <int WK, int T>
__device__ bool stage_tokens(const MvParams& p, int lo, int hi, int n0, int n, uint4* xs, float* inv) {
  using M = Mv<WK, T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k_lo = lo * M::CK;
  const int pieces = (hi - lo) * M::CK / 8;  // per token, 8 elements each
  const auto piece = [&](int tok, int q) {
    const int k = k_lo + q * 8;
    return k < p.K
               ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                      (int64_t)(n0 + tok) * p.K + k))
               : make_uint4(0, 0, 0, 0);
  };
  const auto place = [&](int tok, int q) {
    const int chunk = q / (M::CK / 8), in = q % (M::CK / 8);
    const int t = in / M::J, j = in % M::J;
    return xs + ((chunk * M::J + j) * n + tok) * 4 + t;
  };
  bool wide = false;
  for (int tok = warp; tok < n; tok += kMvWarps) {
    if constexpr (WK == kWBf16) {
      for (int q = lane; q < pieces; q += 32) *place(tok, q) = piece(tok, q);
      if (lane == 0) inv[tok] = 1.0f;
    } else {
      uint32_t m = 0;  // largest magnitude, as bf16 bits
      for (int q = lane; q < pieces; q += 32) {
        const uint4 v = piece(tok, q);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      }
      m = warp_umax(m);
      // 2^c puts it into [2^14, 2^15); c within what fp32 holds
      const int c = m == 0u ? 0 : min(126, max(-126, 14 - ((int)(m >> 7) - 127)));
      const float up = __uint_as_float((uint32_t)(c + 127) << 23);
      const float down = __uint_as_float((uint32_t)(127 - c) << 23);
      for (int q = lane; q < pieces; q += 32) {
        const uint4 v = piece(tok, q);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_f32(w[i]);
          h[i] = pack_f16x2(f.x * up, f.y * up);
          const float2 b = f16x2_f32(h[i]);
          wide |= !(b.x * down == f.x && b.y * down == f.y);
        }
        *place(tok, q) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      if (lane == 0) inv[tok] = down;
    }
  }
  if constexpr (WK == kWNvfp4) {
    wide = __syncthreads_or(wide);
    if (wide) {
      for (int tok = warp; tok < n; tok += kMvWarps) {
        for (int q = lane; q < pieces; q += 32) *place(tok, q) = piece(tok, q);
        if (lane == 0) inv[tok] = 1.0f;
      }
    }
  }
  __syncthreads();
  return wide;
}

// one step's sums over this warp's chunks c_lo .. c_hi - 1 of the slab that
// starts at chunk `lo`.  `it` holds the first items already, and gets the
// first ones of the rows `next` (chunks n_lo .. n_hi - 1) on the way.
template <bool GATED, int WK, int T, bool WIDE>
__device__ __forceinline__ void step_sums(const MvParams& p, int tile, int next_tile, int lane, int n,
                                          const uint4* xs, int lo, int c_lo, int c_hi, int n_lo, int n_hi,
                                          const int (&at)[T], Item (&it)[kDepth], float (&acc)[2][T][4]) {
  using M = Mv<WK, T>;
  Rows r;
  if (c_lo >= c_hi) {  // nothing of this slab
    M::template rows<GATED>(p, next_tile, lane, r);
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (n_lo + d < n_hi) M::load(p, r, n_lo + d, lane, it[d]);
    return;
  }
  M::template rows<GATED>(p, tile, lane, r);
  for (int c = c_lo; c < c_hi; c += kDepth) {
    // a slot's next item: of this step, or the first ones of the next
    const bool last = c + kDepth >= c_hi;
    if (last) M::template rows<GATED>(p, next_tile, lane, r);
    const int from = last ? n_lo : c + kDepth, to = last ? n_hi : c_hi;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (c + d < c_hi) M::template compute<WIDE>(it[d], xs + (c + d - lo) * (M::J * 4 * n), n, at, acc);
      if (from + d < to) M::load(p, r, from + d, lane, it[d]);
    }
  }
}

template <int ACT, int WK, int T>
__global__ void __launch_bounds__(kMvThreads, 2) rn_matvec_kernel(const MvParams p, const MvPlan pl) {
  using M = Mv<WK, T>;
  constexpr bool GATED = ACT != kActNone;
  extern __shared__ uint4 smem[];
  __shared__ float inv[8 * T];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = pl.split > 1 ? (int)cluster_rank() : 0;
  const int group = (int)blockIdx.x / pl.split, n_groups = (int)gridDim.x / pl.split;
  const int n0 = (int)blockIdx.y * 8 * T;
  const int n = min(8 * T, p.N - n0);
  const int rw = kMvWarps / pl.kw, wr = warp / pl.kw, wk = warp % pl.kw;
  const int cols = rw * (GATED ? 16 : 32);  // outputs of a step
  // tokens; the warps' sums [8][T][8][kPartStride]; in a cluster its CTAs'
  // sums [split][rw][n][32]; with several slabs the steps' sums [batch][rw][n][32]
  const int n_max = min(8 * T, p.N);
  uint4* xs = smem;
  float* part = reinterpret_cast<float*>(xs + pl.slab * M::J * 4 * n_max);
  float* parts = part + kMvWarps * T * 8 * kPartStride;
  const int lo = rank * pl.part, hi = min(lo + pl.part, pl.chunks);
  const int slabs = max(1, (hi - lo + pl.slab - 1) / pl.slab);
  const int my_steps = (pl.steps - group + n_groups - 1) / n_groups;
  // this warp's chunks of slab i: contiguous
  const auto chunk_at = [&](int i, int w) {
    const int a = min(lo + i * pl.slab, max(lo, hi)), b = min(a + pl.slab, max(lo, hi));
    return a + (b - a) * w / pl.kw;
  };
  int at[T];
  M::lane_at(n, lane, at);
  const float si = WK == kWNvfp4 ? __ldg(p.scale_inv) : 1.0f;
  float amax = 0.0f;

  Item it[kDepth];
  {
    const int c_lo = chunk_at(0, wk), c_hi = chunk_at(0, wk + 1);
    Rows r;
    M::template rows<GATED>(p, group * rw + wr, lane, r);
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (c_lo + d < c_hi) M::load(p, r, c_lo + d, lane, it[d]);
  }
  bool wide = false;
  for (int b0 = 0; b0 < my_steps; b0 += pl.batch) {
    const int b1 = min(b0 + pl.batch, my_steps);
    for (int sl = 0; sl < slabs; ++sl) {
      if (slabs > 1 || b0 == 0) {
        const int s_lo = lo + sl * pl.slab;
        wide = stage_tokens<WK, T>(p, s_lo, max(s_lo, min(s_lo + pl.slab, hi)), n0, n, xs, inv);
      }
      const int c_lo = chunk_at(sl, wk), c_hi = chunk_at(sl, wk + 1);
      for (int j = b0; j < b1; ++j) {
        const int step = group + j * n_groups;
        // what follows: the batch's next step, its first with the next slab, the next batch's first
        const bool wrap = j + 1 == b1;
        const int sl2 = wrap ? (sl + 1) % slabs : sl;
        const int j2 = wrap ? (sl + 1 < slabs ? b0 : b1) : j + 1;
        const int n_lo = chunk_at(sl2, wk), n_hi = j2 < my_steps ? chunk_at(sl2, wk + 1) : n_lo;
        const int next = group + min(j2, my_steps - 1) * n_groups;
        float acc[2][T][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;
        if (WK == kWNvfp4 && wide)
          step_sums<GATED, WK, T, true>(p, step * rw + wr, next * rw + wr, lane, n, xs, lo + sl * pl.slab,
                                        c_lo, c_hi, n_lo, n_hi, at, it, acc);
        else
          step_sums<GATED, WK, T, false>(p, step * rw + wr, next * rw + wr, lane, n, xs, lo + sl * pl.slab,
                                         c_lo, c_hi, n_lo, n_hi, at, it, acc);
        // this warp's sums: [T][8 tokens][32 rows]
        float* mine = part + warp * T * 8 * kPartStride;
        const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mine[(t * 8 + t2 + (i & 1)) * kPartStride + m * 16 + g + (i >> 1) * 8] = acc[m][t][i];
        __syncthreads();
        // one row's sum over the CTA's warps, times what its token was scaled by
        const auto cta_sum = [&](int tile, int tok, int row) {
          const float* q = part + ((tile * pl.kw) * T * 8 + tok) * kPartStride + row;
          float v = q[0];
          for (int w = 1; w < pl.kw; ++w) v += q[w * T * 8 * kPartStride];
          return v * inv[tok];
        };
        // the outputs of the step, from what `sum` gives for a row
        const auto outputs = [&](auto sum) {
          for (int i = threadIdx.x; i < cols * n; i += kMvThreads) {
            const int tok = i / cols, col = i % cols;
            if constexpr (GATED)
              finish<ACT>(p, n0 + tok, step * cols + col, sum(col / 16, tok, col % 16) * si,
                          sum(col / 16, tok, 16 + col % 16) * si, &amax);
            else
              finish<ACT>(p, n0 + tok, step * cols + col, sum(col / 32, tok, col % 32) * si, 0.0f, &amax);
          }
        };
        const int vals = rw * n * 32;
        if (pl.split > 1) {
          // the steps' sums meet in the cluster's CTAs in turn
          const int leader = j % pl.split;
          const uint32_t to = map_to_rank(smem_u32(parts + rank * vals), leader);
          for (int i = threadIdx.x; i < vals; i += kMvThreads)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * 4),
                         "f"(cta_sum(i / (n * 32), i / 32 % n, i & 31))
                         : "memory");
          cluster_sync();
          if (rank == leader)
            outputs([&](int tile, int tok, int row) {
              const float* q = parts + (tile * n + tok) * 32 + row;
              float v = q[0];
              for (int s = 1; s < pl.split; ++s) v += q[s * vals];
              return v;
            });
        } else if (slabs > 1) {
          // slab after slab, each thread its own sums
          float* sums = parts + (j - b0) * vals;
          for (int i = threadIdx.x; i < vals; i += kMvThreads) {
            const float v = cta_sum(i / (n * 32), i / 32 % n, i & 31);
            sums[i] = sl == 0 ? v : sums[i] + v;
          }
          __syncthreads();
          if (sl + 1 == slabs)
            outputs([&](int tile, int tok, int row) { return sums[(tile * n + tok) * 32 + row]; });
        } else {
          outputs(cta_sum);
          __syncthreads();
        }
      }
    }
  }
  if (p.mode == kFfnFp8) {
    const float m = warp_max_nan(amax);
    if (lane == 0) {
      pdl_wait();  // amax was zeroed by the kernel this one depends on
      atomicMax(reinterpret_cast<unsigned*>(p.amax), abs_bits(m));
    }
  }
  if (pl.split > 1) cluster_sync();  // no CTA leaves while another writes to it
}

constexpr size_t kMvSmemHalf = 112 * 1024;  // two CTAs an SM

template <int ACT, int WK, int T>
rn_status launch_t(const MvParams& p, int sms, cudaStream_t s) {
  using M = Mv<WK, T>;
  auto k = rn_matvec_kernel<ACT, WK, T>;
  constexpr int RO = ACT == kActNone ? 32 : 16;  // outputs of a row tile
  MvPlan pl{};
  pl.chunks = (p.K + M::CK - 1) / M::CK;
  const int n = p.N < 8 * T ? p.N : 8 * T;
  const int64_t ny = ((int64_t)p.N + 8 * T - 1) / (8 * T);
  const int tiles = (p.H + RO - 1) / RO;
  const size_t chunk_bytes = (size_t)M::J * 4 * n * 16;
  const size_t warp_bytes = (size_t)kMvWarps * T * 8 * kPartStride * 4;
  // few row tiles: the reduction over a cluster, while its CTAs' warps keep
  // two chunks each
  pl.split = 1;
  while (pl.split < 8 && tiles * ny * pl.split < sms && pl.chunks >= 4 * kMvWarps * pl.split) pl.split *= 2;
  pl.part = (pl.chunks + pl.split - 1) / pl.split;
  // warps along the reduction: fewer where it is short and the rows are many
  // (an MXFP8 block needs two row tiles a step)
  pl.kw = p.mode == kFfnMx ? kMvWarps / 2 : kMvWarps;
  while (pl.kw > 1 && pl.part < kDepth * pl.kw &&
         (int64_t)tiles * ny * pl.split * pl.kw >= 2ll * sms * kMvWarps)
    pl.kw /= 2;
  const int rw = kMvWarps / pl.kw;
  pl.steps = (tiles + rw - 1) / rw;
  const size_t step_bytes = (size_t)rw * n * 32 * 4;
  int per = (2 * sms) / pl.split;  // clusters or CTAs of one token group
  if (per > pl.steps) per = pl.steps;
  if (per < 1) per = 1;
  const int my_steps = (pl.steps + per - 1) / per;
  size_t room = kMvSmemHalf - warp_bytes - (pl.split > 1 ? pl.split * step_bytes : 0);
  pl.slab = pl.part;
  pl.batch = my_steps;
  if (pl.slab * chunk_bytes > room) {
    if (pl.split > 1) {  // then the rows are few: no cluster, several slabs
      pl.split = 1;
      pl.part = pl.chunks;
      room = kMvSmemHalf - warp_bytes;
      per = 2 * sms < pl.steps ? 2 * sms : pl.steps;
    }
    pl.batch = (pl.steps + per - 1) / per;
    if (pl.slab * chunk_bytes > room || pl.part != pl.slab) {
      // a third of the room at most for the steps' sums
      const int fit = (int)(room / 3 / step_bytes);
      if (pl.batch > fit) pl.batch = fit;
      if (pl.batch < 1) return RN_ERR_UNSUPPORTED;
      pl.slab = (int)((room - pl.batch * step_bytes) / chunk_bytes);
      if (pl.slab < 1) return RN_ERR_UNSUPPORTED;
      const int slabs = (pl.part + pl.slab - 1) / pl.slab;
      pl.slab = (pl.part + slabs - 1) / slabs;
    }
  }
  size_t smem = pl.slab * chunk_bytes + warp_bytes;
  if (pl.split > 1)
    smem += pl.split * step_bytes;
  else if (pl.slab < pl.part)
    smem += pl.batch * step_bytes;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return RN_ERR_CUDA;
  if (ny > 65535) return RN_ERR_UNSUPPORTED;
  const int groups = per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * pl.split), (unsigned)ny);
  cfg.blockDim = dim3(kMvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pl.split > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = (unsigned)pl.split;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  if (p.mode == kFfnFp8) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  if (cudaLaunchKernelEx(&cfg, k, p, pl) != cudaSuccess) return RN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

// groups of 8, 16 or 32 tokens
template <int ACT, int WK>
rn_status launch_n(const MvParams& p, int sms, cudaStream_t s) {
  if (p.N <= 8) return launch_t<ACT, WK, 1>(p, sms, s);
  if (p.N <= 16) return launch_t<ACT, WK, 2>(p, sms, s);
  return launch_t<ACT, WK, 4>(p, sms, s);
}

}  // namespace

rn_status launch_nvfp4_mv(int act, const MvParams& p, int sms, cudaStream_t s) {
  switch (act) {
    case kActNone: return launch_n<kActNone, kWNvfp4>(p, sms, s);
    case kActSwiglu: return launch_n<kActSwiglu, kWNvfp4>(p, sms, s);
    default: return launch_n<kActClampedSwiglu, kWNvfp4>(p, sms, s);
  }
}

rn_status launch_bf16_mv(int act, const MvParams& p, int sms, cudaStream_t s) {
  return act == kActSwiglu ? launch_n<kActSwiglu, kWBf16>(p, sms, s)
                           : launch_n<kActClampedSwiglu, kWBf16>(p, sms, s);
}

}  // namespace rn

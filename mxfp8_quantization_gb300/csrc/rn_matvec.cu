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
constexpr int kDepth = 4;      // items in flight per warp
constexpr int kPartStride = 36;  // floats per token of a warp's partial sums (32 rows, no bank conflicts)

enum WeightKind : int { kWBf16 = 0, kWNvfp4 = 1 };

struct MvPlan {
  int kw;       // warps along the reduction
  int split;    // CTAs of a cluster along the reduction
  int chunks;   // chunks (128 / 32 elements) of the reduction
  int slab;     // chunks per CTA
  int steps;    // groups of 8 / kw row tiles
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
      const int k = chunk * 128 + t * 32;
      if ((p.K & 31) == 0) {  // rows of whole 16-byte pieces
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            it.w[m][h] = k < p.K ? ldg_w16(r.w[m] + (h ? r.dw[m] : 0) + k / 2) : make_uint4(0, 0, 0, 0);
            it.s[m][h] =
                k < p.K ? __ldg(reinterpret_cast<const unsigned short*>(r.s[m] + (h ? r.ds[m] : 0) + k / 16)) : 0u;
          }
      } else {  // an odd number of blocks: rows on 8 bytes, the last piece half
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint2 z = make_uint2(0, 0);
            const uint2 lo = k < p.K ? ldg_w8(r.w[m] + (h ? r.dw[m] : 0) + k / 2) : z;
            const uint2 hi = k + 16 < p.K ? ldg_w8(r.w[m] + (h ? r.dw[m] : 0) + k / 2 + 8) : z;
            it.w[m][h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            const uint32_t s0 = k < p.K ? __ldg(r.s[m] + (h ? r.ds[m] : 0) + k / 16) : 0u;
            const uint32_t s1 = k + 16 < p.K ? __ldg(r.s[m] + (h ? r.ds[m] : 0) + k / 16 + 1) : 0u;
            it.s[m][h] = s0 | s1 << 8;
          }
      }
    }
  }

  // acc += item x tokens; xs: the chunk's fragments of this lane
  template <bool WIDE>
  __device__ __forceinline__ static void compute(const Item& it, const uint4* xs,
                                                 float (&acc)[2][T][4]) {
    if constexpr (WK == kWBf16) {
      uint4 b[T];
#pragma unroll
      for (int t = 0; t < T; ++t) b[t] = xs[t * 32];
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
        for (int t = 0; t < T; ++t) b[t] = xs[(q * T + t) * 32];
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

template <int ACT, int WK, int T>
struct Smem {
  uint4* xs;       // [slab][J][T][32]
  float* part;     // [8 warps][T][8 tokens][kPartStride]
  float* parts;    // split > 1: [split][8 / kw row tiles][T][8][32] sums of the cluster's CTAs
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

// the tokens of this CTA's part of the reduction, in fragment order; returns
// whether they had to stay bf16 (NVFP4).  inv: what each token's sums are
// multiplied with.
template <int WK, int T>
__device__ bool stage_tokens(const MvParams& p, const MvPlan& pl, int rank, int n0, int n, uint4* xs,
                             float* inv) {
  using M = Mv<WK, T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k_lo = rank * pl.slab * M::CK;
  const int pieces = pl.slab * M::CK / 8;  // per token, 8 elements each
  const auto piece = [&](int tok, int q) {
    const int k = k_lo + q * 8;
    return tok < n && k < p.K
               ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                      (int64_t)(n0 + tok) * p.K + k))
               : make_uint4(0, 0, 0, 0);
  };
  const auto place = [&](int tok, int q) {
    const int chunk = q / (M::CK / 8), in = q % (M::CK / 8);
    const int t = in / M::J, j = in % M::J;
    return xs + ((chunk * M::J + j) * T + tok / 8) * 32 + (tok & 7) * 4 + t;
  };
  bool wide = false;
  for (int tok = warp; tok < 8 * T; tok += kMvWarps) {
    if constexpr (WK == kWBf16) {
      for (int q = lane; q < pieces; q += 32) *place(tok, q) = piece(tok, q);
      if (lane == 0) inv[tok] = 1.0f;
    } else {
      uint32_t m = 0;  // largest magnitude, as bf16 bits
      if (tok < n)
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
      for (int tok = warp; tok < 8 * T; tok += kMvWarps) {
        for (int q = lane; q < pieces; q += 32) *place(tok, q) = piece(tok, q);
        if (lane == 0) inv[tok] = 1.0f;
      }
    }
  }
  __syncthreads();
  return wide;
}

template <int ACT, int WK, int T, bool WIDE>
__device__ void run(const MvParams& p, const MvPlan& pl, int rank, int group, int n_groups, int n0, int n,
                    const uint4* xs, float* part, float* parts, const float* inv, float* amax,
                    Item (&it)[kDepth], int c_lo, int c_hi) {
  using M = Mv<WK, T>;
  constexpr bool GATED = ACT != kActNone;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rw = kMvWarps / pl.kw, wr = warp / pl.kw;
  const int cols = rw * (GATED ? 16 : 32);  // outputs of a step
  const float si = WK == kWNvfp4 ? __ldg(p.scale_inv) : 1.0f;
  for (int step = group; step < pl.steps; step += n_groups) {
    float acc[2][T][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;
    Rows r;
    M::template rows<GATED>(p, step * rw + wr, lane, r);
    const int next = step + n_groups;
    for (int c = c_lo; c < c_hi; c += kDepth) {
      // a slot's next item: of this step, or the first ones of the next step
      const bool last = c + kDepth >= c_hi;
      if (last) M::template rows<GATED>(p, next * rw + wr, lane, r);
      const int from = last ? c_lo : c + kDepth;
      const int to = last && next >= pl.steps ? from : c_hi;
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (c + d < c_hi)
          M::template compute<WIDE>(it[d], xs + (size_t)(c + d - rank * pl.slab) * M::J * T * 32 + lane, acc);
        if (from + d < to) M::load(p, r, from + d, lane, it[d]);
      }
    }
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
    if (pl.split == 1) {
      for (int i = threadIdx.x; i < cols * n; i += kMvThreads) {
        const int tok = i / cols, col = i % cols;
        if constexpr (GATED) {
          const float a = cta_sum(col / 16, tok, col % 16) * si;
          const float b = cta_sum(col / 16, tok, 16 + col % 16) * si;
          finish<ACT>(p, n0 + tok, step * cols + col, a, b, amax);
        } else {
          finish<ACT>(p, n0 + tok, step * cols + col, cta_sum(col / 32, tok, col % 32) * si, 0.0f, amax);
        }
      }
      __syncthreads();
    } else {
      // the steps' sums meet in the cluster's CTAs in turn
      const int leader = ((step - group) / n_groups) % pl.split;
      const int vals = rw * T * 8 * 32;
      const uint32_t to = map_to_rank(smem_u32(parts + rank * vals), leader);
      for (int i = threadIdx.x; i < rw * n * 32; i += kMvThreads) {
        const int tile = i / (n * 32), tok = i / 32 % n, row = i & 31;
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + ((tile * T * 8 + tok) * 32 + row) * 4),
                     "f"(cta_sum(tile, tok, row))
                     : "memory");
      }
      cluster_sync();
      if (rank == leader) {
        const auto sum = [&](int tile, int tok, int row) {
          const float* q = parts + (tile * T * 8 + tok) * 32 + row;
          float v = q[0];
          for (int s = 1; s < pl.split; ++s) v += q[s * vals];
          return v * si;
        };
        for (int i = threadIdx.x; i < cols * n; i += kMvThreads) {
          const int tok = i / cols, col = i % cols;
          if constexpr (GATED)
            finish<ACT>(p, n0 + tok, step * cols + col, sum(col / 16, tok, col % 16),
                        sum(col / 16, tok, 16 + col % 16), amax);
          else
            finish<ACT>(p, n0 + tok, step * cols + col, sum(col / 32, tok, col % 32), 0.0f, amax);
        }
      }
    }
  }
}

template <int ACT, int WK, int T>
__global__ void __launch_bounds__(kMvThreads, T == 1 ? 2 : 1)
    rn_matvec_kernel(const MvParams p, const MvPlan pl) {
  using M = Mv<WK, T>;
  extern __shared__ uint4 smem[];
  __shared__ float inv[8 * T];
  uint4* xs = smem;
  float* part = reinterpret_cast<float*>(xs + (size_t)pl.slab * M::J * T * 32);
  float* parts = part + kMvWarps * T * 8 * kPartStride;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = pl.split > 1 ? (int)cluster_rank() : 0;
  const int group = (int)blockIdx.x / pl.split, n_groups = (int)gridDim.x / pl.split;
  const int n0 = (int)blockIdx.y * 8 * T;
  const int n = min(8 * T, p.N - n0);
  const int rw = kMvWarps / pl.kw;
  // this warp's chunks, contiguous
  const int lo = rank * pl.slab, hi = min(lo + pl.slab, pl.chunks);
  const int wk = warp % pl.kw, len = max(0, hi - lo);
  const int c_lo = lo + len * wk / pl.kw, c_hi = lo + len * (wk + 1) / pl.kw;

  Item it[kDepth];
  {
    Rows r;
    M::template rows<ACT != kActNone>(p, group * rw + warp / pl.kw, lane, r);
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (c_lo + d < c_hi) M::load(p, r, c_lo + d, lane, it[d]);
  }
  const bool wide = stage_tokens<WK, T>(p, pl, rank, n0, n, xs, inv);
  float amax = 0.0f;
  if (WK == kWNvfp4 && wide)
    run<ACT, WK, T, true>(p, pl, rank, group, n_groups, n0, n, xs, part, parts, inv, &amax, it, c_lo, c_hi);
  else
    run<ACT, WK, T, false>(p, pl, rank, group, n_groups, n0, n, xs, part, parts, inv, &amax, it, c_lo, c_hi);
  if (p.mode == kFfnFp8) {
    const float m = warp_max_nan(amax);
    if (lane == 0) {
      pdl_wait();  // amax was zeroed by the kernel this one depends on
      atomicMax(reinterpret_cast<unsigned*>(p.amax), abs_bits(m));
    }
  }
  if (pl.split > 1) cluster_sync();  // no CTA leaves while another writes to it
}

constexpr size_t kMvSmemMax = 220 * 1024;

template <int WK, int T>
size_t smem_bytes(const MvPlan& pl) {
  using M = Mv<WK, T>;
  size_t b = (size_t)pl.slab * M::J * T * 32 * 16 + (size_t)kMvWarps * T * 8 * kPartStride * 4;
  if (pl.split > 1) b += (size_t)pl.split * (kMvWarps / pl.kw) * T * 8 * 32 * 4;
  return b;
}

template <int ACT, int WK, int T>
rn_status launch_t(const MvParams& p, int sms, cudaStream_t s) {
  using M = Mv<WK, T>;
  auto k = rn_matvec_kernel<ACT, WK, T>;
  constexpr int RO = ACT == kActNone ? 32 : 16;  // outputs of a row tile
  MvPlan pl{};
  pl.chunks = (p.K + M::CK - 1) / M::CK;
  const int tiles = (p.H + RO - 1) / RO;
  const int kw_max = p.mode == kFfnMx ? kMvWarps / 2 : kMvWarps;  // an MXFP8 block: two row tiles a step
  bool fits = false;
  for (pl.split = 1; pl.split <= 8; pl.split *= 2) {
    pl.slab = (pl.chunks + pl.split - 1) / pl.split;
    pl.kw = kw_max;
    if (smem_bytes<WK, T>(pl) > kMvSmemMax) continue;
    fits = true;
    if ((int64_t)tiles * pl.split >= sms || pl.slab < 2 * kMvWarps) break;
  }
  if (pl.split > 8) pl.split = 8;
  pl.slab = (pl.chunks + pl.split - 1) / pl.split;
  if (!fits) return RN_ERR_UNSUPPORTED;
  pl.kw = kw_max;
  while (pl.kw > 1 && pl.slab < 4 * pl.kw && (int64_t)tiles * pl.split * pl.kw >= 2ll * sms * kMvWarps) pl.kw /= 2;
  const int rw = kMvWarps / pl.kw;
  pl.steps = (tiles + rw - 1) / rw;
  const size_t smem = smem_bytes<WK, T>(pl);
  if (smem > kMvSmemMax) return RN_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return RN_ERR_CUDA;
  int occ = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k, kMvThreads, smem) != cudaSuccess)
    return RN_ERR_CUDA;
  if (occ < 1) return RN_ERR_UNSUPPORTED;
  int groups = sms * occ / pl.split;
  if (groups < 1) groups = 1;
  if (groups > pl.steps) groups = pl.steps;
  const int64_t ny = ((int64_t)p.N + 8 * T - 1) / (8 * T);
  if (ny > 65535) return RN_ERR_UNSUPPORTED;
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

// groups of 8, 16 or 32 tokens; long reductions, whose tokens would not fit,
// take smaller groups
template <int ACT, int WK>
rn_status launch_n(const MvParams& p, int sms, cudaStream_t s) {
  rn_status st = RN_ERR_UNSUPPORTED;
  if (p.N > 16) st = launch_t<ACT, WK, 4>(p, sms, s);
  if (p.N > 8 && st == RN_ERR_UNSUPPORTED) st = launch_t<ACT, WK, 2>(p, sms, s);
  if (st == RN_ERR_UNSUPPORTED) st = launch_t<ACT, WK, 1>(p, sms, s);
  return st;
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

// Paged 8-bit key/value cache: quantising new tokens into their pages and
// reading positions back.
//
//   write  per page of 64 positions and head: e = the smallest exponent with
//          max|x| <= 448 2^e, code = E4M3(x 2^-e)
//   read   x = value(code) 2^e
//
// A page that an earlier call began keeps the larger of its exponent and that
// of the new tokens; where it grows, the old codes are multiplied by a power
// of two and rounded again, which is exact but for codes that become
// subnormal.  Powers of two make that so, and make every cached value a bf16.
//
// A CTA owns the page of one head, keys or values; the heads of a page are
// neighbours in the grid, as their rows are in memory.  The caller's arrays say
// on the device which pages there are, so the grid holds the most there can
// be: a sequence of n rows touches at most floor(n / 64) + 2 pages, and its units
// begin at floor(starts[b] / 64) + 2 b.
//
// Keys lie [64, dim]: a thread takes 8 elements of a row.  Values lie
// transposed, [dim, 64], so that the attention's matrix product finds them
// along the positions: a thread takes 8 elements of 4 rows in a row, whose
// codes are 8 words of 4 positions; 16 lanes write (or read) the 64 bytes of a
// dim, 2 lanes the 32 bytes of a token.  No shared memory is needed.
//
// What bounds them: memory.  Reading 24 sequences of up to 16000 positions back (8
// heads of 128, 1.7 GB moved) takes 250 us, 6.8 TB/s, the measured copy rate; writing
// 16 x 4096 tokens (292 MB) 52 us, 5.6 TB/s, 0.84 of it: a page's maximum stands
// between its loads and its stores, so an SM's 8 CTAs wait for each other's loads.  One
// token of each of 32 sequences: 5.0 us, the latency of launch, arrays, rows, scale.
#include <cuda_runtime.h>

#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_kv.cuh"

namespace rn {
namespace {

// threads of a CTA: 8 chunks of 8 elements a thread, at most
template <int D>
constexpr int kNt = D <= 128 ? 128 : D;
template <int D>
constexpr int kChunks = 64 * (D / 8) / kNt<D>;

// one page's part of a call
struct Unit {
  int b, row0;      // row0 + position in the page = row (may be outside [lo, hi))
  int lo, hi;       // positions in the page that belong to the call's rows
  int page;         // -1: none
  int first;        // the unit is the sequence's first
  int s0, none;     // rows [s0, s0 + none) have no position
};

__device__ __forceinline__ bool find_unit(const KvSeqs& q, int64_t pages, int u, Unit* o) {
  const int lane = threadIdx.x & 31;
  int b, len;
  KvRows r;
  if (q.B <= 32) {
    // all sequences at once, one a lane
    const int i = min(lane, q.B - 1);
    const KvRows mine = kv_rows(q.starts, i, q.tokens);
    const int mine_len = q.lens[i];
    b = 31 - __clz(__ballot_sync(0xFFFFFFFFu, lane == 0 || (lane < q.B && mine.s0 / 64 + 2 * lane <= u)));
    r.s0 = __shfl_sync(0xFFFFFFFFu, mine.s0, b);
    r.s1 = __shfl_sync(0xFFFFFFFFu, mine.s1, b);
    len = max(__shfl_sync(0xFFFFFFFFu, mine_len, b), 0);
  } else {
    b = kv_find(q.B, u, lane, [&](int i) { return min(max(q.starts[i], 0), q.tokens) / 64 + 2 * i; });
    r = kv_rows(q.starts, b, q.tokens);
    len = max(q.lens[b], 0);
  }
  const int n = r.s1 - r.s0;
  const int k = u - (r.s0 / 64 + 2 * b);
  const int p0 = len - n, from = max(p0, 0);
  o->b = b;
  o->s0 = r.s0;
  o->first = k == 0;
  o->none = min(max(-p0, 0), n);
  const int64_t blk = (int64_t)(from >> 6) + k;
  o->lo = o->hi = 0;
  o->page = -1;
  if (n == 0 || k < 0) {
    o->none = 0;
    return false;
  }
  if (blk * 64 >= len) return o->first && o->none > 0;
  o->page = kv_page(q, pages, b, (int)blk);
  o->lo = max(from - (int)(blk * 64), 0);
  o->hi = (int)min((int64_t)64, len - blk * 64);
  o->row0 = (int)(r.s0 + (blk * 64 - p0));
  return true;
}

// 8 elements as they lie in memory
template <bool BF16>
struct Eight;
template <>
struct Eight<true> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p) { w = __ldg(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void f32(float* f) const { bf16x8_to_f32(w, f); }
  // largest magnitude as fp32 bits; NaN above infinity above all
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = max2(max2(w.x & kAbs, w.y & kAbs), max2(w.z & kAbs, w.w & kAbs));
    return max(m << 16, m & 0xFFFF0000u);
  }
  static constexpr uint32_t kAbs = 0x7FFF7FFFu;
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Eight<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldg(static_cast<const float4*>(p));
    b = __ldg(static_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void f32(float* f) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    return max(max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w))),
               max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
  }
};

// largest finite magnitude of n eights, as bits
template <bool BF16>
__device__ __forceinline__ uint32_t finite_top(const Eight<BF16>* v, int n) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) bits = max(bits, v[i].top());
  if (bits >= 0x7F800000u) {
    bits = 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float f[8];
      v[i].f32(f);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (abs_bits(f[j]) < 0x7F800000u) bits = max(bits, abs_bits(f[j]));
    }
  }
  return bits;
}

// four codes times f, rounded again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t l, h;
  e4m3x4_f16x4(w, l, h);
  const float2 a = f16x2_f32(l), b = f16x2_f32(h);
  return pack_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// the page's exponent after the call, and the old codes' factor (1: they stay)
template <int NT>
__device__ __forceinline__ int page_exp(uint32_t bits, bool begun, uint32_t old_byte, float* shrink) {
  __shared__ uint32_t part[NT / 32];
  bits = warp_umax(bits);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = bits;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) bits = max(bits, part[i]);
  int e = kv_exp_of(bits);
  *shrink = 1.0f;
  if (begun) {
    const int old = kv_exp(old_byte);
    if (e > old) *shrink = pow2i(max(old - e, -126));
    e = max(e, old);
  }
  return e;
}

template <int D, bool BF16>
__device__ __forceinline__ void write_keys(const Unit& u, const unsigned char* x, int64_t stride, const KvCache& cache,
                                           int head) {
  constexpr int NT = kNt<D>, C = kChunks<D>, ESZ = BF16 ? 2 : 4;
  Eight<BF16> v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int at = i * NT + threadIdx.x, r = at / (D / 8), c = at % (D / 8);
    if (r >= u.lo && r < u.hi)
      v[i].load(x + ((int64_t)(u.row0 + r) * stride + c * 8) * ESZ);
    else
      v[i].zero();
  }
  // (the rows do not wait for the page's number, nor for its old scale)
  if (u.page < 0) return;
  const int64_t ph = (int64_t)u.page * cache.heads + head;
  uint8_t *page = cache.k + ph * 64 * D, *scale = cache.ks + ph;
  const uint32_t old_byte = u.lo > 0 ? *scale : 0u;
  const uint32_t bits = finite_top(v, C);
  float shrink;
  const int e = page_exp<NT>(bits, u.lo > 0, old_byte, &shrink);
  const float s = pow2i(-e);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int at = i * NT + threadIdx.x, r = at / (D / 8), c = at % (D / 8);
    uint2* o = reinterpret_cast<uint2*>(page + r * D + c * 8);
    if (r >= u.lo && r < u.hi) {
      float f[8];
      v[i].f32(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
      *o = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
    } else if (r < u.lo && shrink != 1.0f) {
      const uint2 w = *o;
      *o = make_uint2(rescale4(w.x, shrink), rescale4(w.y, shrink));
    }
  }
  if (threadIdx.x == 0) *scale = (uint8_t)(e + 127);
}

template <int D, bool BF16>
__device__ __forceinline__ void write_values(const Unit& u, const unsigned char* x, int64_t stride,
                                             const KvCache& cache, int head) {
  constexpr int NT = kNt<D>, C = kChunks<D> / 4, ESZ = BF16 ? 2 : 4;
  static_assert(C * NT == 16 * (D / 8), "whole quads of rows");
  Eight<BF16> v[C][4];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int at = i * NT + threadIdx.x, r0 = at % 16 * 4, c = at / 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + q;
      if (r >= u.lo && r < u.hi)
        v[i][q].load(x + ((int64_t)(u.row0 + r) * stride + c * 8) * ESZ);
      else
        v[i][q].zero();
    }
  }
  // (the rows do not wait for the page's number, nor for its old scale)
  if (u.page < 0) return;
  const int64_t ph = (int64_t)u.page * cache.heads + head;
  uint8_t *page = cache.v + ph * 64 * D, *scale = cache.vs + ph;
  const uint32_t old_byte = u.lo > 0 ? *scale : 0u;
  const uint32_t bits = finite_top(&v[0][0], 4 * C);
  float shrink;
  const int e = page_exp<NT>(bits, u.lo > 0, old_byte, &shrink);
  const float s = pow2i(-e);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int at = i * NT + threadIdx.x, r0 = at % 16 * 4, c = at / 16;
    // which of the four positions are new (a byte of ones each), and which are old
    uint32_t fresh = 0, old = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = r0 + q;
      if (r >= u.lo && r < u.hi) fresh |= 0xFFu << (8 * q);
      if (r < u.lo && shrink != 1.0f) old |= 0xFFu << (8 * q);
    }
    if ((fresh | old) == 0) continue;
    float f[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[i][q].f32(f[q]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint8_t* o = page + (c * 8 + j) * 64 + r0;
      uint32_t w = pack_e4m3x4(f[0][j] * s, f[1][j] * s, f[2][j] * s, f[3][j] * s);
      if (fresh != 0xFFFFFFFFu) {
        const uint32_t was = *reinterpret_cast<uint32_t*>(o);
        w = (w & fresh) | (rescale4(was, shrink) & old) | (was & ~(fresh | old));
      }
      *reinterpret_cast<uint32_t*>(o) = w;
    }
  }
  if (threadIdx.x == 0) *scale = (uint8_t)(e + 127);
}

// 64 registers a thread for bf16 rows, so that an SM has 1024 threads with loads on their way
template <int D, bool BF16>
__global__ void __launch_bounds__(kNt<D>, BF16 ? 1024 / kNt<D> : 640 / kNt<D>) rn_kv_write_kernel(const KvWriteParams p) {
  pdl_launch_dependents();
  pdl_wait();
  Unit u;
  const int part = (int)(blockIdx.x % (2 * p.c.heads)), h = part >> 1, values = part & 1;
  if (!find_unit(p.q, p.c.pages, (int)(blockIdx.x / (2 * p.c.heads)), &u) || u.lo >= u.hi) return;
  constexpr int ESZ = BF16 ? 2 : 4;
  if (!values)
    write_keys<D, BF16>(u, static_cast<const unsigned char*>(p.k) + (int64_t)h * D * ESZ, p.k_stride, p.c, h);
  else
    write_values<D, BF16>(u, static_cast<const unsigned char*>(p.v) + (int64_t)h * D * ESZ, p.v_stride, p.c, h);
}

// 8 values of a row
template <bool BF16>
__device__ __forceinline__ void store8(unsigned char* o, const float* f) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
    reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// Values are exact: a code has 4 significant bits, and 2^-129, the least
// product, is a (subnormal) bf16.
template <int D, bool BF16>
__global__ void __launch_bounds__(kNt<D>) rn_kv_read_kernel(const KvReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  Unit u;
  const int split = (int)(blockIdx.x % (2 * p.c.heads)), h = split >> 1, values = split & 1;
  if (!find_unit(p.q, p.c.pages, (int)(blockIdx.x / (2 * p.c.heads)), &u)) return;
  constexpr int NT = kNt<D>, ESZ = BF16 ? 2 : 4;
  unsigned char* out = static_cast<unsigned char*>(values ? p.v : p.k) + (int64_t)h * D * ESZ;
  const int64_t stride = (int64_t)p.c.heads * D;
  const float zeros[8] = {};
  if (u.first)  // rows without a position
    for (int64_t at = threadIdx.x; at < (int64_t)u.none * (D / 8); at += NT)
      store8<BF16>(out + ((u.s0 + at / (D / 8)) * stride + at % (D / 8) * 8) * ESZ, zeros);
  if (u.lo >= u.hi) return;
  const int64_t ph = (int64_t)max(u.page, 0) * p.c.heads + h;
  const float s = u.page < 0 ? 0.0f : pow2i(kv_exp(values ? p.c.vs[ph] : p.c.ks[ph]));
  if (!values) {
    const uint8_t* page = p.c.k + ph * 64 * D;
    uint2 w[kChunks<D>];
#pragma unroll
    for (int i = 0; i < kChunks<D>; ++i) {
      const int at = i * NT + threadIdx.x, r = at / (D / 8), c = at % (D / 8);
      w[i] = make_uint2(0, 0);
      if (u.page >= 0 && r >= u.lo && r < u.hi) w[i] = *reinterpret_cast<const uint2*>(page + r * D + c * 8);
    }
#pragma unroll
    for (int i = 0; i < kChunks<D>; ++i) {
      const int at = i * NT + threadIdx.x, r = at / (D / 8), c = at % (D / 8);
      if (r < u.lo || r >= u.hi) continue;
      uint32_t h2[4];
      e4m3x4_f16x4(w[i].x, h2[0], h2[1]);
      e4m3x4_f16x4(w[i].y, h2[2], h2[3]);
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 t = f16x2_f32(h2[j]);
        f[2 * j] = t.x * s;
        f[2 * j + 1] = t.y * s;
      }
      store8<BF16>(out + ((int64_t)(u.row0 + r) * stride + c * 8) * ESZ, f);
    }
  } else {
    constexpr int C = kChunks<D> / 4;
    const uint8_t* page = p.c.v + ph * 64 * D;
    uint32_t w[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = i * NT + threadIdx.x, r0 = at % 16 * 4, c = at / 16;
      const bool any = u.page >= 0 && r0 + 4 > u.lo && r0 < u.hi;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[i][j] = any ? *reinterpret_cast<const uint32_t*>(page + (c * 8 + j) * 64 + r0) : 0u;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = i * NT + threadIdx.x, r0 = at % 16 * 4, c = at / 16;
      float f[4][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t l, hh;
        e4m3x4_f16x4(w[i][j], l, hh);
        const float2 a = f16x2_f32(l), b = f16x2_f32(hh);
        f[0][j] = a.x * s, f[1][j] = a.y * s, f[2][j] = b.x * s, f[3][j] = b.y * s;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + q;
        if (r >= u.lo && r < u.hi) store8<BF16>(out + ((int64_t)(u.row0 + r) * stride + c * 8) * ESZ, f[q]);
      }
    }
  }
}

template <class P>
rn_status launch(void (*k)(P), int threads, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.q.tokens / 64 + 2 * p.q.B) * 2 * p.c.heads));  // below 2^31: the entry points' check
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k, p) != cudaSuccess) return RN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

template <int D>
rn_status write_d(const KvWriteParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? launch(rn_kv_write_kernel<D, true>, kNt<D>, p, s) : launch(rn_kv_write_kernel<D, false>, kNt<D>, p, s);
}
template <int D>
rn_status read_d(const KvReadParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? launch(rn_kv_read_kernel<D, true>, kNt<D>, p, s) : launch(rn_kv_read_kernel<D, false>, kNt<D>, p, s);
}

}  // namespace

rn_status launch_kv_write(const KvWriteParams& p, int dim, bool bf16, cudaStream_t s) {
  switch (dim) {
    case 64: return write_d<64>(p, bf16, s);
    case 128: return write_d<128>(p, bf16, s);
    case 192: return write_d<192>(p, bf16, s);
    default: return write_d<256>(p, bf16, s);
  }
}

rn_status launch_kv_read(const KvReadParams& p, int dim, bool bf16, cudaStream_t s) {
  switch (dim) {
    case 64: return read_d<64>(p, bf16, s);
    case 128: return read_d<128>(p, bf16, s);
    case 192: return read_d<192>(p, bf16, s);
    default: return read_d<256>(p, bf16, s);
  }
}

}  // namespace rn

// Host-side plumbing shared by the translation units of the library: kernel
// parameter blocks, launch plans and the per-unit launch functions.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/rn.h"

namespace rn {

// what a kernel does before quantizing: normalize (RMSNorm / LayerNorm) or
// take its fp32 input as y already (the stand-alone quantize entry point)
enum NormKind : int { kRms = 0, kLn = 1, kIdentity = 2 };

// quantization variants of the row-wise forward kernel
enum FwdQuant : int {
  kQNone = 0,       // bf16 or fp32 output
  kQDelayed = 1,    // E4M3 with a given scale, + amax
  kQCurAmax = 2,    // current scaling, pass 1: statistics + amax, no output
  kQCurQuant = 3,   // current scaling, pass 2: quantize with 448/amax
  kQNvfp4 = 4,      // NVFP4, pass 2 (pass 1 is kQCurAmax): E2M1 codes with an
                    // E4M3 scale per 16 elements and S = 448*6/amax
  kQMxRow = 5,      // MXFP8 rowwise blocks only (1x32, E8M0 scales), one pass
};

// NVFP4 pass 2 keeps a table of the 128 element factors S / value(scale
// code) in shared memory
constexpr int kNvTableBytes = 128 * 4;

struct FwdParams {
  const void* x;
  const float* gamma;   // 16-byte aligned
  const float* beta;
  void* out;            // [N, H] (bf16/fp32 or E4M3 codes); NVFP4: [N, H/2]
  uint8_t* scales;      // NVFP4: E4M3 block-scale codes [N, H/16]; kQMxRow: E8M0 [N, H/32]
  float* mu;            // LayerNorm: written (pass 1) or read (kQCurQuant)
  float* rsigma;
  const float* scale;   // kQDelayed
  float* amax;          // kQDelayed, kQCurAmax: reduced into; kQCurQuant: read
  float* scale_inv;     // kQCurQuant, kQNvfp4 (kQDelayed: written by the init kernel)
  float* scale_out;     // kQCurQuant, kQNvfp4
  int N, H;
  float eps;
  int zcg;              // zero-centered gamma
  int out_f32;          // kQNone: 1 = fp32 output, 0 = bf16
  const void* residual; // residual add: the residual [N, H] (x's dtype), or NULL
  void* residual_out;   // residual add: h = x + residual [N, H], or NULL
  int workers;          // worker warps (a multiple of the row group size)
  int Q;                // ring slots; workers / group size <= (Q - 1) rows a slot
  int rps_log2;         // a slot holds 2^rps_log2 adjacent rows (one copy)
  int reverse;          // walk the rows from the last one
};

struct MxParams {
  const void* x;
  const float* gamma;
  const float* beta;
  uint8_t* data;        // rowwise codes [N, H] or NULL
  uint8_t* row_scales;  // [N, H/32]
  uint8_t* col_data;    // [H, N] or NULL
  uint8_t* col_scales;  // [H, N/32]
  float* mu;
  float* rsigma;
  int N, H;
  float eps;
  int zcg;
  int apply_warps;
  int stats_warps;
  int Q;
  int n_tiles;          // N / 32
  int n_tbar;           // ring kernel: tile "ready" barriers (> Q / 32 + 1)
};

struct BwdParams {
  const void* dz;
  const void* x;
  const float* mu;
  const float* rsigma;
  const float* gamma;
  void* dx;
  float* part;          // workspace partials [C][nacc][H]
  int N, H;
  int zcg;
  int chunk_rows;       // rows per dgamma/dbeta partial
  int apply_warps;
  int stats_warps;
  int Q;
  int n_chunks;
};

struct ColReduceParams {
  const float* part;    // [C][nacc][H]
  float* dgamma;
  float* dbeta;
  int H;
  int n_chunks;
  int nacc;
};

// scaled activations (forward with a quantize epilogue, backward)
enum ActKind : int { kActSrelu = 0, kActSwiglu = 1, kActClampedSwiglu = 2 };

struct ActParams {
  const void* x;          // [N, H] (SReLU) or [N, 2H] (gate half, linear half)
  const void* dy;         // backward: [N, H]
  void* out;              // forward: y (bf16 / fp32) or E4M3 codes [N, H];
                          // backward: dx, the shape of x
  uint8_t* row_scales;    // forward MXFP8 (rowwise): E8M0 [N, H/32], else NULL
  const float* scales;    // [N] row scales, or NULL (all 1)
  const float* scale;     // FP8 delayed
  float* amax;            // FP8 modes
  float* scale_inv;       // FP8 current (pass 2)
  float* scale_out;       // FP8 current (pass 2)
  float* dscales;         // backward: [N] or NULL
  int N, H;               // H: output width
  float limit, alpha;     // clamped SwiGLU
  int out_f32;            // forward NONE: fp32 output
};

// gated feed-forward block and the NVFP4 products
constexpr int kActNone = -1;  // rn_nvfp4_matvec: no activation

// The bf16 block of few tokens: up to 8 the few-token kernel, up to 32 while
// the outputs are few (us in a graph, weights in rotation, few-token kernel
// against tensor-core tiles.  K x H 2048 x 2048: 1 token 8.1 / 13.1, 8 8.6 / 11.6,
// 16 9.6 / 11.6, 32 13.6 / 11.6; 4096 x 8192: 1 25.7 / 37.4, 8 29.5 / 36.2, 16 32.6 /
// 26.7, 32 53.0 / 27.0; 8192 x 8192: 2 46.6 / 65.2, 8 51.0 / 50.5, 16 59.5 / 50.6;
// 8192 x 4096, tiles shared: 4 28.3 / 43.2, 8 30.1 / 28.8; 5120 x 13824: 8 60.0 / 64.0)
inline bool few_tokens(int64_t N, int64_t H) { return N <= 8 || (N <= 32 && N * H <= 32768); }
// few-token kernel: positions along the reduction, up to a chunk past a row's end,
// are int; groups of 32 tokens are gridDim.y
constexpr int64_t kMvMaxK = int64_t(1) << 26, kMvMaxN = int64_t(1) << 20;

// The forward's reduction: a tile's epilogue waits for all of it, and waits run
// out after about 2 s.  2^26 is 2^20 slices of 64 at 0.25 us each; 2^31, shared
// by four pairs, would be 2.1 s.
constexpr int64_t kFfnMaxK = int64_t(1) << 26;
static_assert(kFfnMaxK <= kMvMaxK, "the few-token kernel takes every K of the block");

enum FfnOut : int { kFfnBf16 = 0, kFfnF32 = 1, kFfnFp8 = 2, kFfnMx = 3 };

struct FfnParams {
  const void* x;          // bf16 [N, K]
  const void* w;          // bf16 [2H, K]: H gate rows, H linear rows
  const float* scales;    // [N] or NULL
  void* out;              // [N, H]: bf16, fp32 or E4M3 codes
  uint8_t* row_scales;    // kFfnMx: E8M0 [N, H/32]
  const float* scale;     // kFfnFp8
  float* amax;            // kFfnFp8
  void* pre;              // bf16 [N, 2H] or NULL
  int N, K, H;
  float limit, alpha;
  int mode;               // FfnOut
};

// how the backward's two products split their reductions: `splits` parts of
// `per` slices of 64 each; with more than one part their fp32 sums go to the
// workspace and a second kernel adds them
struct FfnSplit {
  int splits, per;
};
struct FfnBwdPlan {
  FfnSplit dx, dw;
  size_t dx_part, dw_part;  // byte offsets of the sums in the workspace (after dp)
  size_t bytes;             // of the workspace
};
FfnBwdPlan ffn_bwd_plan(int64_t N, int64_t K, int64_t H);

struct FfnBwdParams {
  void* ws;               // workspace: dp bf16 [N, 2H], then the parts' sums
  const void* x;          // bf16 [N, K]
  const void* w;          // bf16 [2H, K]
  void* dx;               // bf16 [N, K] or NULL
  void* dw;               // bf16 [2H, K] or NULL
  int N, K, H;
};

struct MvParams {
  const void* x;          // bf16 [N, K]
  const void* w;          // E2M1 pairs [R, K/2] or bf16 [R, K]; R = H, or 2H with an activation
  const uint8_t* blocks;  // NVFP4: E4M3 scales [R, K/16]
  const float* scale_inv; // NVFP4: 1 / S
  const float* scales;    // [N] or NULL
  void* out;              // [N, H]
  uint8_t* row_scales;    // kFfnMx
  const float* scale;     // kFfnFp8
  float* amax;            // kFfnFp8
  void* pre;              // bf16 weights: bf16 [N, 2H] or NULL
  int rows;               // how the weights' rows can be read (set at the launch)
  int N, K, H;
  float limit, alpha;
  int mode;               // FfnOut
};

// paged 8-bit key/value cache (include/rn.h: rn_kv_cache, rn_kv_seqs)
struct KvCache {
  uint8_t* k;             // E4M3 [pages, heads, 64, dim]
  uint8_t* v;             // E4M3 [pages, heads, dim, 64]
  uint8_t* ks;            // E8M0 [pages, heads]
  uint8_t* vs;
  int64_t pages;
  int heads;
};
struct KvSeqs {
  const int* table;       // [B, width]
  const int* starts;      // [B + 1]
  const int* lens;        // [B]
  int B, width, tokens;   // tokens: rows of the call's row tensors
};
struct KvWriteParams {
  KvCache c;
  KvSeqs q;
  const void* k;          // [tokens, heads, dim], rows `k_stride` elements apart
  const void* v;
  int64_t k_stride, v_stride;
};
struct KvReadParams {
  KvCache c;
  KvSeqs q;
  void* k;                // [tokens, heads, dim]
  void* v;
};
// n / d for 0 <= n < 2^31 by a product: with 2^(s-1) < d <= 2^s, mul = ceil(2^(31 + s) / d) is below 2^32 and off by
// less than 1, which makes the quotient wrong by less than n / 2^(31 + s) < 1 / d
struct FastDiv {
  uint32_t mul;
  int shift;            // of the product's upper half
  int d;
};
inline FastDiv fast_div(int d) {
  int s = 0;
  while ((int64_t(1) << s) < d) ++s;
  return FastDiv{(uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d), s - 1, d};
}
struct KvAttnParams {
  KvCache c;
  KvSeqs q;
  const void* x;          // queries, bf16 [tokens, heads * group, dim], rows `stride` elements apart
  int64_t stride;
  FastDiv group;          // query heads of a key/value head
  float scale;
  int causal;
  int window;             // 0: none
  float softcap;          // 0: none
  const float* slopes;    // [heads * group] or NULL
  void* out;              // bf16 [tokens, heads * group, dim]
  float* lse;             // [tokens, heads * group] or NULL
  void* ws;
};
rn_status launch_kv_write(const KvWriteParams& p, int dim, bool bf16, cudaStream_t s);
rn_status launch_kv_read(const KvReadParams& p, int dim, bool bf16, cudaStream_t s);
rn_status launch_kv_attn(const KvAttnParams& p, int dim, int sms, cudaStream_t s);
// bytes of the attention's workspace
size_t kv_attn_bytes(int dim);

// launch shape shared by the persistent kernels
struct Launch {
  int work;             // independent work items (tiles / chunks): grid upper bound
  int sms;              // SMs the grid may use (SMs - sm_margin)
  int per_sm;           // CTAs per SM the shared-memory plan was sized for
  int threads;          // consumer threads + one producer warp
  size_t smem;
};

// per-device limits, queried once
struct DeviceInfo {
  int sms;
  int smem_optin;       // per CTA
  int smem_per_sm;      // per SM
};
rn_status device_info(DeviceInfo* out);

// A value found out once per device and kept (0: not yet); `find` gives a
// positive value, or a negative one on failure, which is not kept.
constexpr int kMaxDevices = 64;
template <class Find>
int once_per_device(std::atomic<int> (&kept)[kMaxDevices], Find find) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  int v = kept[dev].load(std::memory_order_acquire);
  if (v <= 0) {
    v = find();
    if (v > 0) kept[dev].store(v, std::memory_order_release);
  }
  return v;
}

// Grid of a persistent kernel: min(work, sms * CTAs per SM), where CTAs per
// SM is the planned count capped by what the kernel's resources allow.
template <class Kernel>
rn_status persistent_grid(Kernel k, const Launch& l, int* grid) {
  int occ = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k, l.threads, l.smem) != cudaSuccess)
    return RN_ERR_CUDA;
  const int per = occ < 1 ? 1 : (occ < l.per_sm ? occ : l.per_sm);
  const long long g = (long long)l.sms * per;
  int n = (int)(g < l.work ? g : l.work);
  *grid = n < 1 ? 1 : n;
  return RN_OK;
}

// launch functions (one per translation unit family)
// row shape of the forward: G warps per row, NC 16-byte chunks per lane;
// one: one row a slot, compiled as such (the planner sets it when it
// groups no rows and the shape has that instantiation)
struct FwdShape {
  int g, nc;
  bool one;
};
// pdl: launch as a programmatic dependent of the previous kernel
rn_status launch_fwd(int nk, bool bf16, const FwdShape& sh, int qmode, const FwdParams& p,
                     const Launch& l, bool pdl, cudaStream_t s);
// the same with a residual add (p.residual, p.residual_out set; no pass 2 of
// current scaling, which reads the stored sum through launch_fwd)
rn_status launch_fwd_res(int nk, bool bf16, const FwdShape& sh, int qmode, const FwdParams& p,
                         const Launch& l, bool pdl, cudaStream_t s);
// one-thread kernel: amax = 0 and, when scale != NULL, scale_inv = 1/scale
rn_status launch_fwd_init(float* amax, const float* scale, float* scale_inv, cudaStream_t s);
rn_status launch_mx(int nk, bool bf16, int ng, const MxParams& p, const Launch& l,
                    cudaStream_t s);
// MXFP8 both directions from boxes of 32 rows x 4 column blocks of 128
// bytes, read twice (statistics, then quantization): 16 worker warps; H a
// multiple of 128 / element size, N of 32; Q = box slots
constexpr int kMxBoxThreads = 32 * 16;
constexpr size_t kMxBoxBytes = 16384;
rn_status launch_mx_box(int nk, bool bf16, const MxParams& p, const Launch& l, cudaStream_t s);
// backward with stats warps: bf16 rows (fp32 rows take the fused kernel);
// the wide shape (one CTA per SM) is compiled for at most 512 threads (128
// registers a thread) and for at most kBwdWideThreads (96 registers), the
// most its planner asks for (16 apply warps, 1 stats warp and the producer
// at H = 16384)
constexpr int kBwdWideThreads512 = 512;
constexpr int kBwdWideThreads = 576;
rn_status launch_bwd(bool ln, bool bf16, int ng, const BwdParams& p, const Launch& l,
                     cudaStream_t s);
// backward without stats or producer warps, fp32 rows of up to 16 warps x
// 32 threads x 16 elements (big: one CTA per SM, up to 16 warps; otherwise
// up to 8 warps, several CTAs per SM)
rn_status launch_bwd_fused(bool ln, bool big, const BwdParams& p, const Launch& l,
                           cudaStream_t s);
rn_status launch_colreduce(const ColReduceParams& p, cudaStream_t s);

// scaled activations; qmode kQNone with p.row_scales set = MXFP8 rowwise;
// sms: SMs the grid may use; pdl: programmatic dependent of the previous kernel
rn_status launch_act_fwd(int act, bool bf16, int qmode, const ActParams& p, int sms, bool pdl,
                         cudaStream_t s);
rn_status launch_act_bwd(int act, bool bf16, const ActParams& p, int sms, cudaStream_t s);

// gated feed-forward block; sms: SMs of the device
rn_status launch_ffn_fwd(int act, const FfnParams& p, int sms, cudaStream_t s);
rn_status launch_ffn_bwd(const FfnBwdParams& p, int sms, cudaStream_t s);
// products with NVFP4 weights (act kActNone: R = H rows, no activation)
rn_status launch_nvfp4_mv(int act, const MvParams& p, int sms, cudaStream_t s);
// the gated block of few tokens with bf16 weights
rn_status launch_bf16_mv(int act, const MvParams& p, int sms, cudaStream_t s);

// delayed-scaling history step (one CTA; 1 <= L <= kMaxHistory)
constexpr int kMaxHistory = 1024;
rn_status launch_amax_history(float* hist, int L, const float* amax, float* scale,
                              float* scale_inv, cudaStream_t s);

// device error words, one per translation unit
rn_status read_clear_error_fwd(unsigned* code);
rn_status read_clear_error_fwd_res(unsigned* code);
rn_status read_clear_error_mx(unsigned* code);
rn_status read_clear_error_bwd(unsigned* code);
rn_status read_clear_error_ffn(unsigned* code);
rn_status read_clear_error_mv(unsigned* code);
rn_status read_clear_error_kv(unsigned* code);
rn_status read_clear_error_kv_tile(unsigned* code);

}  // namespace rn

// C entry points of the paged 8-bit key/value cache (declared in include/rn.h):
// argument checks and dispatch, on the host, before anything is enqueued.
#include <cstdint>
#include <cuda_runtime.h>

#include "rn_internal.h"

namespace rn {
namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

rn_status check_cache(const rn_kv_cache* c, KvCache* o) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scales == nullptr || c->v_scales == nullptr ||
      c->pages < 1 || c->heads < 1 || c->dim < 1)
    return RN_ERR_INVALID;
  if ((c->dim != 64 && c->dim != 128 && c->dim != 192 && c->dim != 256) || c->heads > 65535 ||
      c->pages > INT32_MAX || !aligned(c->k, 16) || !aligned(c->v, 16))
    return RN_ERR_UNSUPPORTED;
  *o = KvCache{c->k, c->v, c->k_scales, c->v_scales, c->pages, (int)c->heads};
  return RN_OK;
}

rn_status check_seqs(const rn_kv_seqs* s, KvSeqs* o) {
  if (s == nullptr || s->sequences < 0 || s->table_width < 0 || s->tokens < 0) return RN_ERR_INVALID;
  if (s->sequences > 0 && (s->starts == nullptr || s->lens == nullptr || (s->table_width > 0 && s->table == nullptr)))
    return RN_ERR_INVALID;
  // positions and units are int: pages of 64, and the units' grid
  if (s->sequences > (1 << 24) || s->table_width > INT32_MAX / 64 || s->tokens > INT32_MAX / 2 ||
      !aligned(s->table, 4) || !aligned(s->starts, 4) || !aligned(s->lens, 4))
    return RN_ERR_UNSUPPORTED;
  *o = KvSeqs{s->table, s->starts, s->lens, (int)s->sequences, (int)s->table_width, (int)s->tokens};
  return RN_OK;
}

bool dtype_ok(rn_dtype d) { return d == RN_BF16 || d == RN_F32; }

// the grid of the write and the read: units of a page, head and side
bool grid_ok(const KvCache& c, const KvSeqs& q) {
  return ((int64_t)q.tokens / 64 + 2 * (int64_t)q.B) * 2 * c.heads <= INT32_MAX;
}

// rows of `width` elements, `stride` apart, in whole 16-byte pieces
rn_status check_rows(const void* p, rn_dtype d, int64_t stride, int64_t width) {
  if (stride < width) return RN_ERR_INVALID;
  if (!aligned(p, 16) || stride % (d == RN_BF16 ? 8 : 4) != 0 || stride > INT64_MAX / 8 / (INT32_MAX / 2))
    return RN_ERR_UNSUPPORTED;
  return RN_OK;
}

}  // namespace
}  // namespace rn

using namespace rn;

extern "C" {

rn_status rn_kv_cache_write(const void* k, const void* v, rn_dtype dtype, int64_t k_stride, int64_t v_stride,
                            const rn_kv_cache* cache, const rn_kv_seqs* seqs, void* stream) {
  KvWriteParams p{};
  rn_status st;
  if ((st = check_cache(cache, &p.c)) != RN_OK || (st = check_seqs(seqs, &p.q)) != RN_OK) return st;
  if (!dtype_ok(dtype)) return RN_ERR_INVALID;
  const bool any = p.q.tokens > 0 && p.q.B > 0;
  if (any && (k == nullptr || v == nullptr)) return RN_ERR_INVALID;
  const int64_t width = (int64_t)p.c.heads * cache->dim;
  if ((st = check_rows(k, dtype, k_stride, width)) != RN_OK || (st = check_rows(v, dtype, v_stride, width)) != RN_OK)
    return st;
  if (!grid_ok(p.c, p.q)) return RN_ERR_UNSUPPORTED;
  DeviceInfo di;
  if ((st = device_info(&di)) != RN_OK) return st;
  if (!any) return RN_OK;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return launch_kv_write(p, cache->dim, dtype == RN_BF16, static_cast<cudaStream_t>(stream));
}

rn_status rn_kv_cache_read(const rn_kv_cache* cache, const rn_kv_seqs* seqs, void* k, void* v, rn_dtype out_dtype,
                           void* stream) {
  KvReadParams p{};
  rn_status st;
  if ((st = check_cache(cache, &p.c)) != RN_OK || (st = check_seqs(seqs, &p.q)) != RN_OK) return st;
  if (!dtype_ok(out_dtype)) return RN_ERR_INVALID;
  const bool any = p.q.tokens > 0 && p.q.B > 0;
  if (any && (k == nullptr || v == nullptr)) return RN_ERR_INVALID;
  if (!aligned(k, 16) || !aligned(v, 16) || !grid_ok(p.c, p.q)) return RN_ERR_UNSUPPORTED;
  DeviceInfo di;
  if ((st = device_info(&di)) != RN_OK) return st;
  if (!any) return RN_OK;
  p.k = k;
  p.v = v;
  return launch_kv_read(p, cache->dim, out_dtype == RN_BF16, static_cast<cudaStream_t>(stream));
}

rn_status rn_kv_attention(const void* q, rn_dtype dtype, int64_t q_stride, int64_t q_heads, const rn_kv_cache* cache,
                          const rn_kv_seqs* seqs, float scale, int causal, int64_t window, float softcap,
                          const float* slopes, void* out, float* lse, void* workspace, size_t* workspace_bytes,
                          void* stream) {
  KvAttnParams p{};
  rn_status st;
  if ((st = check_cache(cache, &p.c)) != RN_OK || (st = check_seqs(seqs, &p.q)) != RN_OK) return st;
  if (!dtype_ok(dtype) || q_heads < 1 || q_heads % p.c.heads != 0 || !(scale > 0.0f) || scale > 1e30f || window < 0 ||
      !(softcap == 0.0f || softcap >= 1e-30f) || softcap > 1e30f)
    return RN_ERR_INVALID;
  const int64_t group = q_heads / p.c.heads;
  if (dtype != RN_BF16 || group > 4096 || p.q.tokens * group > INT32_MAX / 2) return RN_ERR_UNSUPPORTED;
  const size_t need = kv_attn_bytes((int)cache->dim);
  if (workspace == nullptr && out == nullptr) {
    if (workspace_bytes == nullptr) return RN_ERR_INVALID;
    *workspace_bytes = need;
    return RN_OK;
  }
  const bool any = p.q.tokens > 0 && p.q.B > 0;
  if (any && (q == nullptr || out == nullptr)) return RN_ERR_INVALID;
  if ((st = check_rows(q, dtype, q_stride, q_heads * cache->dim)) != RN_OK) return st;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(slopes, 4) || !aligned(workspace, 16))
    return RN_ERR_UNSUPPORTED;
  if (any && (workspace == nullptr || workspace_bytes == nullptr || *workspace_bytes < need))
    return RN_ERR_WORKSPACE;
  DeviceInfo di;
  if ((st = device_info(&di)) != RN_OK) return st;
  if (!any) return RN_OK;
  p.x = q;
  p.stride = q_stride;
  p.group = fast_div((int)group);
  p.scale = scale;
  p.causal = causal != 0;
  p.window = window > INT32_MAX ? 0 : (int)window;  // no position is that far away
  p.softcap = softcap;
  p.slopes = slopes;
  p.out = out;
  p.lse = lse;
  p.ws = workspace;
  return launch_kv_attn(p, cache->dim, di.sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

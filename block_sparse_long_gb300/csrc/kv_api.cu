// C ABI of libcosa_kv (declared in include/cosa_kv.h): host-side argument checks and launches.
// No allocation, no host copies.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "cosa_kv.h"
#include "kv_internal.h"

#define COSA_TRY(x)                    \
  do {                                 \
    const int rc_ = (x);               \
    if (rc_ != COSA_OK) return rc_;    \
  } while (0)

namespace {

constexpr int kMaxReqs = 65535;      // grid dimension
constexpr int kMaxHeads = 65535;
constexpr int64_t kMaxTokens = int64_t(1) << 30;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int shift_of(int page_size) {
  int s = 4;
  while ((1 << s) < page_size) ++s;
  return s;
}

// What every call asks of the parameters.
int check_common(const cosa_kv_params* p) {
  if (p == nullptr) return COSA_ERR_INVALID_ARG;
  if (p->num_reqs < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1) return COSA_ERR_INVALID_ARG;
  if (p->num_q_heads % p->num_kv_heads != 0) return COSA_ERR_INVALID_ARG;
  if ((p->flags & ~(COSA_KV_FLAG_INTERLEAVED | COSA_KV_FLAG_TEST_STALL)) != 0 || p->reserved != 0) return COSA_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return COSA_ERR_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return COSA_ERR_UNSUPPORTED;
  if (p->num_reqs > kMaxReqs || p->num_q_heads > kMaxHeads) return COSA_ERR_UNSUPPORTED;
  return COSA_OK;
}

int check_tokens(const cosa_kv_params* p) {
  if (p->total_tokens < 0) return COSA_ERR_INVALID_ARG;
  return p->total_tokens > kMaxTokens ? COSA_ERR_UNSUPPORTED : COSA_OK;
}

// Slots and page tables.
int check_slots(const cosa_kv_params* p) {
  if (p->max_seqlen < 1 || p->max_pages_per_req < 1) return COSA_ERR_INVALID_ARG;
  if (p->max_seqlen > kMaxTokens) return COSA_ERR_UNSUPPORTED;
  if (p->max_pages_per_req < ceil_div(p->max_seqlen, p->page_size)) return COSA_ERR_INVALID_ARG;
  return COSA_OK;
}

// A stride in elements: the given one, or the dense one for 0; -1 if it cannot be.
int64_t stride_of(int64_t given, int64_t dense) {
  if (given == 0) return dense;
  return given >= dense && given % 8 == 0 && given <= (int64_t(1) << 31) ? given : -1;
}

// What the attention asks of the parameters; the size of its workspace is 0 where it refuses them.
int check_attention(const cosa_kv_params* p) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_tokens(p));
  COSA_TRY(check_slots(p));
  if (p->num_kv4_pages < 1 || p->max_new_tokens < 1) return COSA_ERR_INVALID_ARG;
  if (!(p->sm_scale >= 0x1p-100 && p->sm_scale <= 0x1p60)) return COSA_ERR_INVALID_ARG;      // fp32 carries it times 2^33
  if (p->q_stride != 0 && p->q_stride != static_cast<int64_t>(p->num_q_heads) * p->head_dim) return COSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->total_tokens) * (p->num_q_heads / p->num_kv_heads) > INT32_MAX) return COSA_ERR_UNSUPPORTED;
  return COSA_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? COSA_OK : COSA_ERR_CUDA; }

}  // namespace

extern "C" {

int cosa_kv_version(void) { return (0 << 16) | 1; }

int cosa_qk_norm_rope(const cosa_kv_params* p, const void* q, const void* k, const void* v, const void* q_weight,
                      const void* k_weight, const double* inv_freq, const int32_t* positions,
                      const int32_t* cu_seqlens, const int32_t* start, void* q_out, void* k_out, void* k_cache,
                      void* v_cache, const int32_t* page_table, int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_tokens(p));
  if (p->rotary_dim < 16 || p->rotary_dim > p->head_dim || p->rotary_dim % 16 != 0) return COSA_ERR_INVALID_ARG;
  if (p->norm_eps != 0.0 && !(p->norm_eps >= 0x1p-126 && p->norm_eps <= 0x1p126)) return COSA_ERR_INVALID_ARG;
  if (p->total_tokens == 0) return COSA_OK;     // empty tensors have no address
  if (!q || !k || !inv_freq || !cu_seqlens || !q_out) return COSA_ERR_INVALID_ARG;
  const bool paged = k_cache != nullptr;
  if (paged != (v_cache != nullptr) || paged != (page_table != nullptr) || (paged && !v) || (!paged && !k_out))
    return COSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
      !aligned(inv_freq, 8) || !aligned(positions, 4) || !aligned(cu_seqlens, 4) || !aligned(start, 4) ||
      !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(page_table, 4) || !aligned(device_status, 4))
    return COSA_ERR_INVALID_ARG;
  cosa_kv::RopeLaunch L{};
  const int64_t d = p->head_dim;
  L.q_stride = stride_of(p->q_stride, p->num_q_heads * d);
  L.k_stride = stride_of(p->k_stride, p->num_kv_heads * d);
  L.v_stride = stride_of(p->v_stride, p->num_kv_heads * d);
  if (L.q_stride < 0 || L.k_stride < 0 || L.v_stride < 0) return COSA_ERR_INVALID_ARG;
  // in place only row for row
  if ((q_out == q && L.q_stride != p->num_q_heads * d) || (k_out == k && L.k_stride != p->num_kv_heads * d))
    return COSA_ERR_INVALID_ARG;
  if (paged) {
    COSA_TRY(check_slots(p));
    if (p->num_pages < 1) return COSA_ERR_INVALID_ARG;
  }
  L.q = static_cast<const uint16_t*>(q);
  L.k = static_cast<const uint16_t*>(k);
  L.v = static_cast<const uint16_t*>(v);
  L.q_weight = static_cast<const uint16_t*>(q_weight);
  L.k_weight = static_cast<const uint16_t*>(k_weight);
  L.inv_freq = inv_freq;
  L.positions = positions;
  L.cu_seqlens = cu_seqlens;
  L.start = start;
  L.page_table = page_table;
  L.q_out = static_cast<uint16_t*>(q_out);
  L.k_out = static_cast<uint16_t*>(k_out);
  L.k_cache = static_cast<uint16_t*>(k_cache);
  L.v_cache = static_cast<uint16_t*>(v_cache);
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_q_heads = p->num_q_heads;
  L.num_kv_heads = p->num_kv_heads;
  L.head_dim = p->head_dim;
  L.page_size = p->page_size;
  L.page_shift = shift_of(p->page_size);
  L.total_tokens = p->total_tokens;
  L.max_seqlen = p->max_seqlen;
  L.num_pages = p->num_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  L.rotary_dim = p->rotary_dim;
  L.interleaved = (p->flags & COSA_KV_FLAG_INTERLEAVED) != 0;
  L.eps = static_cast<float>(p->norm_eps);
  return done(cosa_kv::launch_rope(L, static_cast<cudaStream_t>(stream)));
}

int cosa_kv4_store(const cosa_kv_params* p, const void* k, const void* v, const int32_t* cu_seqlens,
                   const int32_t* src_page_table, const int32_t* start, const int32_t* kv_len, void* kv4_cache,
                   const int32_t* page_table, int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_slots(p));
  const bool pages = src_page_table != nullptr;
  if (!pages) {
    COSA_TRY(check_tokens(p));
    if (p->total_tokens == 0) return COSA_OK;
  }
  if (!k || !v || !kv4_cache || !page_table || (pages ? !kv_len : !cu_seqlens) || p->num_kv4_pages < 1)
    return COSA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4) || !aligned(src_page_table, 4) ||
      !aligned(start, 4) || !aligned(kv_len, 4) || !aligned(kv4_cache, 16) || !aligned(page_table, 4) ||
      !aligned(device_status, 4))
    return COSA_ERR_INVALID_ARG;
  cosa_kv::ConvertLaunch L{};
  const int64_t dense = static_cast<int64_t>(p->num_kv_heads) * p->head_dim;
  L.k_stride = stride_of(p->k_stride, dense);
  L.v_stride = stride_of(p->v_stride, dense);
  if (L.k_stride < 0 || L.v_stride < 0) return COSA_ERR_INVALID_ARG;
  L.k = static_cast<const uint16_t*>(k);
  L.v = static_cast<const uint16_t*>(v);
  L.cache = static_cast<uint8_t*>(kv4_cache);
  L.page_table = page_table;
  L.other_table = src_page_table;
  L.cu_seqlens = cu_seqlens;
  L.start = start;
  L.kv_len = kv_len;
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_kv_heads = p->num_kv_heads;
  L.head_dim = p->head_dim;
  L.page_size = p->page_size;
  L.max_seqlen = p->max_seqlen;
  L.num_pages = p->num_pages;
  L.page_shift = shift_of(p->page_size);
  L.num_kv4_pages = p->num_kv4_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  if (pages) {
    if (p->num_pages < 1) return COSA_ERR_INVALID_ARG;
    if (L.k_stride != dense || L.v_stride != dense) return COSA_ERR_UNSUPPORTED;   // caches are dense
    return done(cosa_kv::launch_store_pages(L, static_cast<cudaStream_t>(stream)));
  }
  L.total_tokens = p->total_tokens;
  return done(cosa_kv::launch_store_rows(L, static_cast<cudaStream_t>(stream)));
}

int cosa_kv4_load(const cosa_kv_params* p, const void* kv4_cache, const int32_t* page_table, const int32_t* start,
                  const int32_t* kv_len, void* k_cache, void* v_cache, const int32_t* dst_page_table,
                  int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_slots(p));
  if (!kv4_cache || !page_table || !kv_len || !k_cache || !v_cache || !dst_page_table) return COSA_ERR_INVALID_ARG;
  if (p->num_pages < 1 || p->num_kv4_pages < 1) return COSA_ERR_INVALID_ARG;
  if (!aligned(kv4_cache, 16) || !aligned(page_table, 4) || !aligned(start, 4) || !aligned(kv_len, 4) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(dst_page_table, 4) || !aligned(device_status, 4))
    return COSA_ERR_INVALID_ARG;
  cosa_kv::ConvertLaunch L{};
  L.k_cache = static_cast<uint16_t*>(k_cache);
  L.v_cache = static_cast<uint16_t*>(v_cache);
  L.cache = static_cast<uint8_t*>(const_cast<void*>(kv4_cache));
  L.page_table = page_table;
  L.other_table = dst_page_table;
  L.start = start;
  L.kv_len = kv_len;
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_kv_heads = p->num_kv_heads;
  L.head_dim = p->head_dim;
  L.page_size = p->page_size;
  L.max_seqlen = p->max_seqlen;
  L.num_pages = p->num_pages;
  L.page_shift = shift_of(p->page_size);
  L.num_kv4_pages = p->num_kv4_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  return done(cosa_kv::launch_load(L, static_cast<cudaStream_t>(stream)));
}

size_t cosa_kv4_attention_workspace_size(const cosa_kv_params* p, int with_weights) {
  if (check_attention(p) != COSA_OK) return 0;
  return cosa_kv::attn_workspace_bytes(p->num_q_heads, p->head_dim, p->total_tokens, p->max_seqlen, with_weights != 0);
}

int cosa_kv4_attention(const cosa_kv_params* p, const void* q, const int32_t* cu_seqlens, const void* kv4_cache,
                       const int32_t* page_table, const int32_t* kv_len, void* out, float* weights,
                       void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  COSA_TRY(check_attention(p));
  const size_t need = cosa_kv4_attention_workspace_size(p, weights != nullptr);
  if (need == 0) return COSA_ERR_UNSUPPORTED;
  if (p->total_tokens == 0) return COSA_OK;
  if (!q || !cu_seqlens || !kv4_cache || !page_table || !kv_len || !out) return COSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(cu_seqlens, 4) || !aligned(kv4_cache, 16) || !aligned(page_table, 4) ||
      !aligned(kv_len, 4) || !aligned(out, 16) || !aligned(weights, 4) || !aligned(device_status, 4))
    return COSA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return COSA_ERR_WORKSPACE;
  if (out == q) return COSA_ERR_INVALID_ARG;      // CTAs that share an item write its rows while others read theirs
  cosa_kv::AttnLaunch L{};
  L.q = static_cast<const uint16_t*>(q);
  L.cu_seqlens = cu_seqlens;
  L.page_table = page_table;
  L.kv_len = kv_len;
  L.cache = static_cast<const uint8_t*>(kv4_cache);
  L.out = static_cast<uint16_t*>(out);
  L.weights = weights;
  L.workspace = workspace;
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_q_heads = p->num_q_heads;
  L.num_kv_heads = p->num_kv_heads;
  L.head_dim = p->head_dim;
  L.page_size = p->page_size;
  L.total_tokens = p->total_tokens;
  L.max_seqlen = p->max_seqlen;
  L.num_kv4_pages = p->num_kv4_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  L.max_new_tokens = p->max_new_tokens;
  L.stall = (p->flags & COSA_KV_FLAG_TEST_STALL) != 0;
  L.scale_log2 = static_cast<float>(p->sm_scale * 1.4426950408889634074);
  return done(cosa_kv::launch_attention(L, static_cast<cudaStream_t>(stream)));
}

int cosa_kv4_evict(const cosa_kv_params* p, void* kv4_cache, const int32_t* page_table, const int32_t* kv_len,
                   const float* weights, const int32_t* dst_page_table, int32_t* new_len, int32_t* kept,
                   float* weights_out, int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_slots(p));
  if (p->num_kv4_pages < 1 || p->budget < 1 || p->sink < 0 || p->recent < 0) return COSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->sink) + p->recent > p->budget) return COSA_ERR_INVALID_ARG;
  if (p->budget > kMaxTokens) return COSA_ERR_UNSUPPORTED;
  if (p->max_dst_pages < ceil_div(p->budget, p->page_size)) return COSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->num_reqs) * p->num_kv_heads > INT32_MAX / 16) return COSA_ERR_UNSUPPORTED;
  if (!kv4_cache || !page_table || !kv_len || !weights || !dst_page_table || !new_len || !kept) return COSA_ERR_INVALID_ARG;
  if (weights_out == weights || dst_page_table == page_table) return COSA_ERR_INVALID_ARG;   // moved into other memory
  if (new_len == kv_len) return COSA_ERR_INVALID_ARG;     // the heads of a request read the one while the other is written
  if (!aligned(kv4_cache, 16) || !aligned(page_table, 4) || !aligned(kv_len, 4) || !aligned(weights, 4) ||
      !aligned(dst_page_table, 4) || !aligned(new_len, 4) || !aligned(kept, 4) || !aligned(weights_out, 4) ||
      !aligned(device_status, 4))
    return COSA_ERR_INVALID_ARG;
  cosa_kv::EvictLaunch L{};
  L.cache = static_cast<uint8_t*>(kv4_cache);
  L.page_table = page_table;
  L.kv_len = kv_len;
  L.dst_page_table = dst_page_table;
  L.weights = weights;
  L.new_len = new_len;
  L.kept = kept;
  L.weights_out = weights_out;
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_kv_heads = p->num_kv_heads;
  L.head_dim = p->head_dim;
  L.page_size = p->page_size;
  L.max_seqlen = p->max_seqlen;
  L.num_kv4_pages = p->num_kv4_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  L.max_dst_pages = p->max_dst_pages;
  L.budget = p->budget;
  L.sink = p->sink;
  L.recent = p->recent;
  L.page_shift = shift_of(p->page_size);
  return done(cosa_kv::launch_evict(L, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// C ABI of libcosa_attn (declared in include/cosa_attn.h): host-side argument checks and launches.
// No allocation, no host copies.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cosa_attn.h"

#define COSA_TRY(x)                    \
  do {                                 \
    const int rc_ = (x);               \
    if (rc_ != COSA_OK) return rc_;    \
  } while (0)

namespace {

constexpr int kMaxReqs = 65535;      // grid dimension
constexpr int kMaxHeads = 65535;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 31;
constexpr int64_t kRot = COSA_ATTN_ROPE_DIM;

template <typename... P>
bool aligned(size_t a, const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) % a == 0) && ...);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int shift_of(int page_size) {
  int s = 4;
  while ((1 << s) < page_size) ++s;
  return s;
}

// What every call asks of the parameters.
int check_common(const cosa_attn_params* p) {
  if (p == nullptr) return COSA_ERR_INVALID_ARG;
  if (p->num_reqs < 1 || p->num_q_heads < 1 || p->total_tokens < 0) return COSA_ERR_INVALID_ARG;
  if ((p->flags & ~(COSA_ATTN_FLAG_INTERLEAVED | COSA_ATTN_FLAG_TEST_STALL)) != 0 || p->reserved != 0) return COSA_ERR_INVALID_ARG;
  if (p->num_reqs > kMaxReqs || p->num_q_heads > kMaxHeads || p->total_tokens > kMaxTokens) return COSA_ERR_UNSUPPORTED;
  return COSA_OK;
}

// Slots and page tables.
int check_slots(const cosa_attn_params* p) {
  if (p->max_seqlen < 1 || p->max_pages_per_req < 1 || p->num_pages < 1) return COSA_ERR_INVALID_ARG;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return COSA_ERR_UNSUPPORTED;
  if (p->max_seqlen > kMaxTokens || static_cast<int64_t>(p->num_pages) * p->page_size > INT32_MAX) return COSA_ERR_UNSUPPORTED;
  return p->max_pages_per_req < ceil_div(p->max_seqlen, p->page_size) ? COSA_ERR_INVALID_ARG : COSA_OK;
}

int check_heads(const cosa_attn_params* p) {
  if (p->num_kv_heads < 1 || p->num_q_heads % p->num_kv_heads != 0) return COSA_ERR_INVALID_ARG;
  return p->head_dim == 64 || p->head_dim == 128 ? COSA_OK : COSA_ERR_UNSUPPORTED;
}

int check_latent(const cosa_attn_params* p) {
  return p->latent_dim == 256 || p->latent_dim == 512 ? COSA_OK : COSA_ERR_UNSUPPORTED;
}

int check_scale(const cosa_attn_params* p) {
  return p->sm_scale >= 0x1p-100 && p->sm_scale <= 0x1p60 ? COSA_OK : COSA_ERR_INVALID_ARG;
}

// A stride in elements: the given one, or the dense one for 0; -1 if it cannot be.
int64_t stride_of(int64_t given, int64_t dense) {
  if (given == 0) return dense;
  return given >= dense && given % 8 == 0 && given <= kMaxStride ? given : -1;
}

// Token and head strides of `tokens` rows of `heads` times `width` values: heads within a token, or tokens within a head.
bool strides_of(int64_t token, int64_t head, int64_t tokens, int64_t heads, int64_t width, int64_t* by_token, int64_t* by_head) {
  *by_head = head == 0 ? width : head;
  *by_token = token == 0 ? (heads - 1) * *by_head + width : token;
  for (const int64_t s : {*by_head, *by_token})
    if (s < width || s % 8 != 0 || s > kMaxStride) return false;
  return *by_token >= (heads - 1) * *by_head + width || *by_head >= (tokens - 1) * *by_token + width;
}

cosa_attn::PagedLaunch paged_of(const cosa_attn_params* p, bool latent) {
  cosa_attn::PagedLaunch L{};
  L.num_reqs = p->num_reqs;
  L.num_q_heads = p->num_q_heads;
  L.num_kv_heads = latent ? 1 : p->num_kv_heads;
  L.head_dim = latent ? 0 : p->head_dim;
  L.latent_dim = latent ? p->latent_dim : 0;
  L.page_size = p->page_size;
  L.page_shift = shift_of(p->page_size);
  L.total_tokens = p->total_tokens;
  L.max_seqlen = p->max_seqlen;
  L.num_pages = p->num_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  L.max_new_tokens = p->max_new_tokens;
  L.scale_log2 = static_cast<float>(p->sm_scale * 1.4426950408889634074);
  L.stall = (p->flags & COSA_ATTN_FLAG_TEST_STALL) != 0;
  return L;
}

bool query_strides(const cosa_attn_params* p, bool latent, cosa_attn::PagedLaunch* L) {
  const int64_t T = p->total_tokens, H = p->num_q_heads;
  return strides_of(p->q_stride, p->q_head_stride, T, H, latent ? p->latent_dim : p->head_dim, &L->q_stride, &L->q_head_stride) &&
         (!latent || strides_of(p->q_rope_stride, p->q_rope_head_stride, T, H, kRot, &L->q_rope_stride, &L->q_rope_head_stride));
}

int check_paged(const cosa_attn_params* p, bool latent) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_slots(p));
  COSA_TRY(latent ? check_latent(p) : check_heads(p));
  COSA_TRY(check_scale(p));
  if (p->max_new_tokens < 1) return COSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->total_tokens) * p->num_q_heads > INT32_MAX) return COSA_ERR_UNSUPPORTED;
  cosa_attn::PagedLaunch L = paged_of(p, latent);
  if (!query_strides(p, latent, &L)) return COSA_ERR_INVALID_ARG;
  return cosa_attn::paged_fits(L) ? COSA_OK : COSA_ERR_UNSUPPORTED;
}

int done(cudaError_t e) { return e == cudaSuccess ? COSA_OK : COSA_ERR_CUDA; }

template <typename T>
const T* as(const void* p) {
  return static_cast<const T*>(p);
}

// Both attentions over pages; q_rope of latent attention, v_cache of the other.
int run_paged(const cosa_attn_params* p, bool latent, const void* q, const void* q_rope, const int32_t* cu_seqlens,
              const void* k_cache, const void* v_cache, const int32_t* page_table, const int32_t* kv_len,
              const int64_t* tree_mask, void* out, float* lse, void* workspace, size_t workspace_bytes,
              int32_t* device_status, void* stream) {
  COSA_TRY(check_paged(p, latent));
  if (p->total_tokens == 0) return COSA_OK;      // empty tensors have no address
  if (!q || !cu_seqlens || !k_cache || !page_table || !kv_len || !out || !(latent ? q_rope : v_cache)) return COSA_ERR_INVALID_ARG;
  if (!aligned(16, q, q_rope, k_cache, v_cache, out) || !aligned(8, tree_mask) ||
      !aligned(4, cu_seqlens, page_table, kv_len, lse, device_status))
    return COSA_ERR_INVALID_ARG;
  cosa_attn::PagedLaunch L = paged_of(p, latent);
  query_strides(p, latent, &L);
  if (!workspace || !aligned(256, workspace) || workspace_bytes < cosa_attn::paged_workspace_bytes(L)) return COSA_ERR_WORKSPACE;
  if (out == q || out == q_rope) return COSA_ERR_INVALID_ARG;      // CTAs that share a row's keys write it while others read its query
  L.q = as<uint16_t>(q);
  L.q_rope = as<uint16_t>(q_rope);
  L.k_cache = as<uint16_t>(k_cache);
  L.v_cache = as<uint16_t>(v_cache);
  L.cu_seqlens = cu_seqlens;
  L.page_table = page_table;
  L.kv_len = kv_len;
  L.tree_mask = tree_mask;
  L.out = static_cast<uint16_t*>(out);
  L.lse = lse;
  L.workspace = workspace;
  L.status = device_status;
  return done(cosa_attn::launch_paged(L, static_cast<cudaStream_t>(stream)));
}

size_t workspace_of(const cosa_attn_params* p, bool latent) {
  return check_paged(p, latent) == COSA_OK ? cosa_attn::paged_workspace_bytes(paged_of(p, latent)) : 0;
}

}  // namespace

extern "C" {

int cosa_attn_version(void) { return (0 << 16) | 1; }

size_t cosa_tree_attention_workspace_size(const cosa_attn_params* p) { return workspace_of(p, false); }

int cosa_tree_attention(const cosa_attn_params* p, const void* q, const int32_t* cu_seqlens, const void* k_cache,
                        const void* v_cache, const int32_t* page_table, const int32_t* kv_len, const int64_t* tree_mask,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  return run_paged(p, false, q, nullptr, cu_seqlens, k_cache, v_cache, page_table, kv_len, tree_mask, out, lse, workspace,
                   workspace_bytes, device_status, stream);
}

size_t cosa_latent_attention_workspace_size(const cosa_attn_params* p) { return workspace_of(p, true); }

int cosa_latent_attention(const cosa_attn_params* p, const void* q_latent, const void* q_rope, const int32_t* cu_seqlens,
                          const void* latent_cache, const int32_t* page_table, const int32_t* kv_len,
                          const int64_t* tree_mask, void* out, float* lse, void* workspace, size_t workspace_bytes,
                          int32_t* device_status, void* stream) {
  return run_paged(p, true, q_latent, q_rope, cu_seqlens, latent_cache, nullptr, page_table, kv_len, tree_mask, out, lse, workspace,
                   workspace_bytes, device_status, stream);
}

int cosa_tree_commit(const cosa_attn_params* p, void* cache_a, void* cache_b, int32_t row_elems, const int32_t* cu_seqlens,
                     const int32_t* page_table, const int32_t* kv_len, const int32_t* path, const int32_t* path_len,
                     int32_t* new_len, int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_slots(p));
  if (p->max_new_tokens < 1 || row_elems < 8 || row_elems % 8 != 0) return COSA_ERR_INVALID_ARG;
  if (p->max_new_tokens > COSA_ATTN_MAX_TREE || row_elems > (1 << 22)) return COSA_ERR_UNSUPPORTED;
  if (!cache_a || !cu_seqlens || !page_table || !kv_len || !path || !path_len || !new_len) return COSA_ERR_INVALID_ARG;
  if (!aligned(16, cache_a, cache_b) || !aligned(4, cu_seqlens, page_table, kv_len, path, path_len, new_len, device_status))
    return COSA_ERR_INVALID_ARG;
  // CTAs read these while one has written new_len already; two caches in one would be moved twice
  for (const int32_t* read : {cu_seqlens, page_table, kv_len, path, path_len})
    if (new_len == read) return COSA_ERR_INVALID_ARG;
  if (cache_a == cache_b) return COSA_ERR_INVALID_ARG;
  cosa_attn::CommitLaunch L{};
  L.cache_a = static_cast<uint16_t*>(cache_a);
  L.cache_b = static_cast<uint16_t*>(cache_b);
  L.cu_seqlens = cu_seqlens;
  L.page_table = page_table;
  L.kv_len = kv_len;
  L.path = path;
  L.path_len = path_len;
  L.new_len = new_len;
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.row_elems = row_elems;
  L.page_shift = shift_of(p->page_size);
  L.max_seqlen = p->max_seqlen;
  L.num_pages = p->num_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  L.path_pitch = p->max_new_tokens;
  return done(cosa_attn::launch_commit(L, static_cast<cudaStream_t>(stream)));
}

int cosa_latent_rope(const cosa_attn_params* p, const void* kv, const void* q, const void* weight, const double* inv_freq,
                     const int32_t* positions, const int32_t* cu_seqlens, const int32_t* start, void* q_out, void* c_out,
                     void* k_out, void* latent_cache, const int32_t* page_table, int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  COSA_TRY(check_latent(p));
  if (p->norm_eps != 0.0 && !(p->norm_eps >= 0x1p-126 && p->norm_eps <= 0x1p126)) return COSA_ERR_INVALID_ARG;
  if (latent_cache != nullptr) COSA_TRY(check_slots(p));
  if (p->total_tokens == 0) return COSA_OK;
  if (!kv || !inv_freq || !cu_seqlens || (q != nullptr) != (q_out != nullptr) || (c_out != nullptr) != (k_out != nullptr) ||
      (latent_cache != nullptr) != (page_table != nullptr) || (!c_out && !latent_cache))
    return COSA_ERR_INVALID_ARG;
  if (!aligned(16, kv, q, weight, q_out, c_out, k_out, latent_cache) || !aligned(8, inv_freq) ||
      !aligned(4, positions, cu_seqlens, start, page_table, device_status))
    return COSA_ERR_INVALID_ARG;
  if (c_out == kv || k_out == kv || latent_cache == kv) return COSA_ERR_INVALID_ARG;
  cosa_attn::RopeLaunch L{};
  L.kv_stride = stride_of(p->k_stride, p->latent_dim + kRot);
  if (L.kv_stride < 0) return COSA_ERR_INVALID_ARG;
  if (q) {
    if (!strides_of(p->q_rope_stride, p->q_rope_head_stride, p->total_tokens, p->num_q_heads, kRot, &L.q_stride, &L.q_head_stride)) return COSA_ERR_INVALID_ARG;
    // in place only row for row
    if (q_out == q && (L.q_stride != p->num_q_heads * kRot || L.q_head_stride != kRot)) return COSA_ERR_INVALID_ARG;
  }
  L.kv = as<uint16_t>(kv);
  L.q = as<uint16_t>(q);
  L.weight = as<uint16_t>(weight);
  L.inv_freq = inv_freq;
  L.positions = positions;
  L.cu_seqlens = cu_seqlens;
  L.start = start;
  L.page_table = page_table;
  L.q_out = static_cast<uint16_t*>(q_out);
  L.c_out = static_cast<uint16_t*>(c_out);
  L.k_out = static_cast<uint16_t*>(k_out);
  L.cache = static_cast<uint16_t*>(latent_cache);
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_q_heads = p->num_q_heads;
  L.latent_dim = p->latent_dim;
  L.page_shift = shift_of(p->page_size);
  L.total_tokens = p->total_tokens;
  L.max_seqlen = p->max_seqlen;
  L.num_pages = p->num_pages;
  L.max_pages_per_req = p->max_pages_per_req;
  L.interleaved = (p->flags & COSA_ATTN_FLAG_INTERLEAVED) != 0;
  L.eps = static_cast<float>(p->norm_eps);
  return done(cosa_attn::launch_rope(L, static_cast<cudaStream_t>(stream)));
}

int cosa_latent_prefill(const cosa_attn_params* p, const void* q_nope, const void* q_rope, const void* k_nope,
                        const void* k_rope, const void* v, const int32_t* cu_seqlens, const int32_t* cu_kv, void* out,
                        float* lse, int32_t* device_status, void* stream) {
  COSA_TRY(check_common(p));
  if (p->head_dim != 64 && p->head_dim != 128) return COSA_ERR_UNSUPPORTED;
  COSA_TRY(check_scale(p));
  if (p->max_new_tokens < 1 || p->total_kv_tokens < 0) return COSA_ERR_INVALID_ARG;
  if (p->total_kv_tokens > kMaxTokens || static_cast<int64_t>(p->total_tokens) * p->num_q_heads > INT32_MAX) return COSA_ERR_UNSUPPORTED;
  cosa_attn::PrefillLaunch L{};
  const int64_t H = p->num_q_heads, d = p->head_dim, T = p->total_tokens, Tk = p->total_kv_tokens;
  if (!strides_of(p->q_stride, p->q_head_stride, T, H, d, &L.q_stride, &L.q_head_stride) ||
      !strides_of(p->q_rope_stride, p->q_rope_head_stride, T, H, kRot, &L.q_rope_stride, &L.q_rope_head_stride) ||
      !strides_of(p->k_stride, p->k_head_stride, Tk, H, d, &L.k_stride, &L.k_head_stride) ||
      !strides_of(p->v_stride, p->v_head_stride, Tk, H, d, &L.v_stride, &L.v_head_stride))
    return COSA_ERR_INVALID_ARG;
  L.k_rope_stride = stride_of(p->k_rope_stride, kRot);
  if (L.k_rope_stride < 0) return COSA_ERR_INVALID_ARG;
  if (!cosa_attn::prefill_fits(p->total_tokens, p->num_reqs, p->num_q_heads)) return COSA_ERR_UNSUPPORTED;
  if (p->total_tokens == 0) return COSA_OK;
  if (!q_nope || !q_rope || !cu_seqlens || !out) return COSA_ERR_INVALID_ARG;
  if (p->total_kv_tokens < 1 || !k_nope || !k_rope || !v) return COSA_ERR_INVALID_ARG;
  if (!aligned(16, q_nope, q_rope, k_nope, k_rope, v, out) || !aligned(4, cu_seqlens, cu_kv, lse, device_status))
    return COSA_ERR_INVALID_ARG;
  if (out == q_nope || out == k_nope || out == v || out == q_rope || out == k_rope) return COSA_ERR_INVALID_ARG;
  L.q = as<uint16_t>(q_nope);
  L.q_rope = as<uint16_t>(q_rope);
  L.k = as<uint16_t>(k_nope);
  L.k_rope = as<uint16_t>(k_rope);
  L.v = as<uint16_t>(v);
  L.cu_seqlens = cu_seqlens;
  L.cu_kv = cu_kv;
  L.out = static_cast<uint16_t*>(out);
  L.lse = lse;
  L.status = device_status;
  L.num_reqs = p->num_reqs;
  L.num_heads = p->num_q_heads;
  L.head_dim = p->head_dim;
  L.total_tokens = p->total_tokens;
  L.total_kv_tokens = p->total_kv_tokens;
  L.scale_log2 = static_cast<float>(p->sm_scale * 1.4426950408889634074);
  L.stall = (p->flags & COSA_ATTN_FLAG_TEST_STALL) != 0;
  return done(cosa_attn::launch_prefill(L, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

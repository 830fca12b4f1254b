// The accepted path of each request's tree moved behind its context, in place.
//
// Row i of the path goes from slot base + path[i] to slot base + i, base = kv_len - n.  The path ascends, so path[i] >= i, but a
// destination can be the source of an earlier row: a CTA has 32 neighbouring 16-byte columns of all of a request's rows (64 at
// most) and reads them all before it writes any.  Columns do not meet, so CTAs need not either.  Up to 64 rows a request: bound by
// the chain of lengths, path, pages and rows (64 requests of 40 drafted tokens, 8 heads of 128: 2.6 us).
#include <cstdint>

#include "attn_internal.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_attn {
namespace {

constexpr int kThreads = 256;
constexpr int kColumns = 32;                    // 16-byte columns of a CTA
constexpr int kGroups = kThreads / kColumns;    // rows at a time
constexpr int kRows = COSA_ATTN_MAX_TREE / kGroups;

__global__ void __launch_bounds__(kThreads) commit_kernel(const CommitLaunch L) {
  cosa_kv::wait_for_stream();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int64_t n = static_cast<int64_t>(L.cu_seqlens[b + 1]) - L.cu_seqlens[b];
  const int len = L.kv_len[b], m = L.path_len[b];
  const int32_t* path = L.path + static_cast<size_t>(b) * L.path_pitch;
  bool bad = n < 0 || len < n || len > L.max_seqlen || m < 0 || m > n || m > L.path_pitch;
  if (!bad && tid < m) bad = path[tid] < (tid ? path[tid - 1] + 1 : 0) || path[tid] >= n;
  if (__syncthreads_or(bad)) {
    if (blockIdx.y == 0 && tid == 0) {
      L.new_len[b] = len;
      cosa::report_status(L.status, cosa::kStatusBadInput);
    }
    return;
  }
  const int base = len - static_cast<int>(n);
  if (blockIdx.y == 0 && tid == 0) L.new_len[b] = base + m;
  const int columns = L.row_elems / 8, parts = (columns + kColumns - 1) / kColumns;
  uint4* cache = reinterpret_cast<uint4*>(blockIdx.y < parts ? L.cache_a : L.cache_b);
  const int column = (blockIdx.y % parts) * kColumns + tid % kColumns;
  const int mine = column < columns ? m : 0;      // rows of this thread's column
  const int32_t* table = L.page_table + static_cast<size_t>(b) * L.max_pages_per_req;
  auto place = [&](int slot) -> int64_t {         // the slot's 16 bytes of this column, or -1
    const int phys = table[slot >> L.page_shift];
    if (phys < 0 || phys >= L.num_pages) return -1;
    return ((static_cast<int64_t>(phys) << L.page_shift) + (slot & ((1 << L.page_shift) - 1))) * columns + column;
  };
  uint4 row[kRows];
  int64_t to[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = k * kGroups + tid / kColumns;
    to[k] = -1;
    if (i < mine && path[i] != i) {
      const int64_t from = place(base + path[i]);
      if (from >= 0) {
        to[k] = place(base + i);
        row[k] = cache[from];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (to[k] >= 0) cache[to[k]] = row[k];
}

}  // namespace

cudaError_t launch_commit(const CommitLaunch& L, cudaStream_t stream) {
  const int parts = (L.row_elems / 8 + kColumns - 1) / kColumns;
  const dim3 grid(static_cast<unsigned>(L.num_reqs), static_cast<unsigned>(parts * (L.cache_b ? 2 : 1)));
  return cosa_kv::launch_after(commit_kernel, grid, kThreads, 0, stream, 1, L);
}

}  // namespace cosa_attn

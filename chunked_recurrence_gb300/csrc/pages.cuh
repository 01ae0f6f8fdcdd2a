// pages.cuh -- what the calls on a cache's pages have in common: the checks of their tables and pools, the
// search for free pages, and launches that overlap the kernel before.
#pragma once

#include "block_scan.cuh"
#include "common.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace gdn {
namespace pages {

constexpr int kPlanThreads = 1024;

// Words of the workspace after the 256 bytes that hold the status.
struct PlanWords {
  int32_t ok, n_moves, live, pad;
};

struct Pools {
  void *p[GDN_MAX_POOLS];
};

// Four consecutive refs of a thread, n past the end read as `past`.
__device__ __forceinline__ int4 load_refs(const int32_t *refs, int i, int n, int past) {
  if (i + 3 < n && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) return *reinterpret_cast<const int4 *>(refs + i);
  return make_int4(i < n ? refs[i] : past, i + 1 < n ? refs[i + 1] : past, i + 2 < n ? refs[i + 2] : past,
                   i + 3 < n ? refs[i + 3] : past);
}

// The first `want` free pages into list, in rising order; returns how many there are of them.
__device__ inline int first_free(const int32_t *refs, int n_pages, int want, int32_t *list, int *sh) {
  int found = 0;
  for (int base = 0; base < n_pages && found < want; base += 4 * kPlanThreads) {
    const int i = base + 4 * threadIdx.x;
    const int4 r = load_refs(refs, i, n_pages, 1);
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    int total;
    int at = found + block_scan(f[0] + f[1] + f[2] + f[3], sh, &total) - (f[0] + f[1] + f[2] + f[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) {
        if (at < want) list[at] = i + k;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

__device__ __forceinline__ int32_t *table_row(const gdn_page_tables &t, int s) {
  return t.page_table + (int64_t)s * t.table_stride;
}

// The tables checked, strides and the status word filled in.
inline bool tables_ok(const gdn_page_tables *in, void *workspace, gdn_page_tables *t) {
  if (!in) return false;
  *t = *in;
  if (t->n_rows < 0 || t->max_pages < 0 || t->n_pages < 0 || t->page_size < 1 || !aligned(t->status, sizeof(int32_t)))
    return false;
  if (t->table_stride == 0) t->table_stride = t->max_pages;
  if (!t->status) t->status = (int32_t *)workspace;
  if (t->table_stride < t->max_pages || t->n_pages >= 1 << 21) return false;  // sums of 1024 rows' pages: 32 bits
  return (t->n_rows == 0 || (t->page_table && t->seq_lens)) && (t->n_pages == 0 || t->refs);
}

inline gdn_status pools_ok(const gdn_page_pools *in, Pools *p) {
  if (!in || in->n_pools < 0 || in->page_bytes < 0 || in->page_stride < in->page_bytes || (in->n_pools && !in->pools))
    return GDN_ERR_INVALID_ARG;
  if (in->n_pools > GDN_MAX_POOLS) return GDN_ERR_UNSUPPORTED;
  for (int i = 0; i < in->n_pools; ++i) {
    if (!in->pools[i]) return GDN_ERR_INVALID_ARG;
    p->p[i] = in->pools[i];
  }
  return GDN_OK;
}

// A launch that overlaps the end of the kernel before on the stream, whose results the kernel waits for.
template <typename... P, typename... A>
void launch_early(void (*kernel)(P...), int blocks, int threads, cudaStream_t st, size_t smem, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool ws_ok(const void *w, size_t bytes, size_t want) { return w && aligned(w, 256) && bytes >= want; }

}  // namespace pages
}  // namespace gdn

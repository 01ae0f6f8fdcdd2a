// paged_attn.cuh -- the kernels of gdn_paged_attn as its dispatch sees them.
#pragma once

#include "common.cuh"
#include "paged.cuh"

namespace gdn {

gdn_status normalise_cache_shape(const gdn_cache_shape *in, const int32_t *cu_seqlens, gdn_cache_shape *out);
PagedSeqs paged_seqs(const gdn_cache_shape &s, const int32_t *seq_lens, const int32_t *cu_seqlens);

// Whether the tensor-core kernel takes this call, and the workspace it needs (0 where it never would).
bool paged_attn_tc_supported(const void *q, const void *k, const void *v, const void *o, const gdn_cache_shape &s,
                             float scale);
size_t paged_attn_tc_workspace(const gdn_cache_shape &s, int32_t max_new);
gdn_status paged_attn_tc(const void *q, const void *k, const void *v, const int32_t *table, const PagedSeqs &seqs,
                         const gdn_cache_shape &s, int32_t max_new, float scale_log2, int32_t window, uint32_t flags,
                         void *o, float *lse, void *workspace, cudaStream_t st);

// A call as the kernels without tcgen05 take it.
struct SimtArgs {
  PagedSeqs seqs;
  const void *q, *k, *v;
  void *o;
  float *lse, *part;  // part: [splits][n_tok * Hq][2 + D] (maximum, sum, weighted sum), or null with one split
  const int32_t *table;
  int64_t table_stride, page_stride, slot_stride, head_stride, q_stride;
  int32_t Hq, Hkv, D, page_size, max_pages, n_pages, window, splits;
  float scale_log2;
  int32_t *status;
};

int paged_attn_f32_splits(const gdn_cache_shape &s, int32_t max_new, int32_t window);  // window 0: the most of any
gdn_status paged_attn_f32(const SimtArgs &a, const gdn_cache_shape &s, int32_t max_new, cudaStream_t st);

}  // namespace gdn

// paged_attn.cuh -- the kernels of gdn_paged_attn and gdn_paged_attn_shared as their dispatch sees them.
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

// The same where groups of sequences share a prefix (seqs names them).
size_t paged_shared_tc_workspace(const gdn_cache_shape &s, int32_t n_groups, int32_t max_group_new);
gdn_status paged_shared_tc(const void *q, const void *k, const void *v, const int32_t *table, const GroupedSeqs &seqs,
                           const gdn_cache_shape &s, int32_t max_group_new, float scale_log2, uint32_t flags, void *o,
                           float *lse, void *workspace, cudaStream_t st);

// A call as the kernels without tcgen05 take it.
struct SimtArgs {
  GroupedSeqs seqs;
  const void *q, *k, *v;
  void *o;
  float *lse, *part;  // part: [splits][n_tok * Hq][2 + D] (maximum, sum, weighted sum), or null with one split; with
                      // a shared prefix the splits of the prefix follow those of the own positions
  const int32_t *table;
  int64_t table_stride, page_stride, slot_stride, head_stride, q_stride;
  int32_t Hq, Hkv, D, page_size, max_pages, n_pages, window, splits;
  float scale_log2;
  int32_t *status;
};

// An item of either call, tiles of one position; the part of a block's split, and the positions that a row sees.
__device__ __forceinline__ SharedItem simt_item(const SimtArgs &a, int slot, int G, int R) {
  if (a.seqs.n_groups) return shared_item_at(a.seqs, slot, G, R, 1);
  SharedItem it;
  static_cast<Item &>(it) = item_at(a.seqs, slot, G, R, 1, a.window);
  it.g = 0, it.own = true;
  return it;
}
__device__ __forceinline__ int simt_part(const SimtArgs &a, const SharedItem &it) {
  return it.own ? blockIdx.z : a.splits + blockIdx.z;
}
__device__ __forceinline__ int simt_row_end(const SimtArgs &a, const SharedItem &it, int row, int G) {
  return it.own ? it.first + row / G + 1 : row_end(a.seqs, it, row, G);
}
__device__ __forceinline__ int simt_row_begin(const SimtArgs &a, const SharedItem &it, int row, int G) {
  const int p = it.first + row / G;
  return a.window > 0 && p >= a.window ? p - a.window + 1 : a.seqs.n_groups ? it.lo : 0;
}
inline int64_t simt_slots(const SimtArgs &a, int R) {
  const GroupedSeqs &q = a.seqs;
  return q.n_groups ? shared_slots(q.n_tok, q.n_seqs, q.n_groups, a.Hq / a.Hkv, R)
                    : item_slots(q.n_tok, q.n_seqs, a.Hq / a.Hkv, R);
}

int paged_attn_f32_splits(const gdn_cache_shape &s, int32_t max_new, int32_t window);  // window 0: the most of any
gdn_status paged_attn_f32(const SimtArgs &a, const gdn_cache_shape &s, int32_t max_new, cudaStream_t st);

}  // namespace gdn

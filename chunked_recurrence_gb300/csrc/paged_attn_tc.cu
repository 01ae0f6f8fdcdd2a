// paged_attn_tc.cu -- gdn_paged_attn on the tensor cores: which of the kernel's forms takes a call.
#include "paged_attn_tc.cuh"

namespace gdn {
namespace {

template <int D, int NQ, bool PAIR>
gdn_status launch(const void *k, const void *v, const gdn_cache_shape &s, TcArgs<false> &a, void *workspace, cudaStream_t st) {
  using C = Cfg<D, NQ, PAIR>;
  constexpr int units = kSms / C::kPair;
  char *w = (char *)workspace;
  a.meta = (int4 *)(w + 256);
  a.part_ml = (float *)(w + 256 + sizeof(int4) * 512);
  a.part = a.part_ml + (size_t)units * 2 * C::R * 2;
  return launch_two<D, NQ, PAIR, false>(k, v, s, a, st, dim3(units, C::R / 32), paged_join_kernel<D, NQ, PAIR>);
}

}  // namespace

bool paged_attn_tc_supported(const void *q, const void *k, const void *v, const void *o, const gdn_cache_shape &s,
                             float scale) {
  if (!tc_shape(s) || !(scale > 1e-20f && scale < 1e20f)) return false;
  for (const void *p : {q, k, v, o})
    if (!aligned(p, 16)) return false;
  for (int64_t x : {s.q_stride, s.slot_stride, s.Hkv > 1 ? s.head_stride : 8, s.n_pages > 1 ? s.page_stride : 8})
    if (x % 8 || x >= 1LL << 39) return false;
  return true;
}

size_t paged_attn_tc_workspace(const gdn_cache_shape &s, int32_t max_new) {
  if (!tc_shape(s)) return 0;
  const size_t rows = (size_t)kSms * 2 * (two_tiles(s, max_new) ? 256 : 128);
  return 256 + sizeof(int4) * 512 + rows * (2 + s.D) * sizeof(float);
}

gdn_status paged_attn_tc(const void *q, const void *k, const void *v, const int32_t *table, const PagedSeqs &seqs,
                         const gdn_cache_shape &s, int32_t max_new, float scale_log2, int32_t window, uint32_t flags,
                         void *o, float *lse, void *workspace, cudaStream_t st) {
  TcArgs<false> a = tc_args<false>(q, table, seqs, s, scale_log2, window, flags, o, lse, workspace);
  const bool pair = pairs(s, max_new);
  if (s.D == 256)
    return pair ? launch<256, 1, true>(k, v, s, a, workspace, st) : launch<256, 1, false>(k, v, s, a, workspace, st);
  if (pair) return launch<128, 2, true>(k, v, s, a, workspace, st);
  if (two_tiles(s, max_new))
    return s.D == 128 ? launch<128, 2, false>(k, v, s, a, workspace, st) : launch<64, 2, false>(k, v, s, a, workspace, st);
  return s.D == 128 ? launch<128, 1, false>(k, v, s, a, workspace, st) : launch<64, 1, false>(k, v, s, a, workspace, st);
}

}  // namespace gdn

// The index arithmetic of calls whose sequences share prefixes (paged.cuh) compiled for the host, so that the tests can
// check on the CPU which rows and positions the kernels take and where their pieces lie.
#include "paged.cuh"

using namespace gdn;

static GroupedSeqs seqs(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t max_tokens,
                      const int32_t *groups, const int32_t *prefix, int32_t n_groups) {
  return GroupedSeqs{{lens, cu, n_seqs, n_tok, max_tokens}, groups, prefix, n_groups};
}

extern "C" {
int64_t host_shared_slots(int64_t n_tok, int32_t n_seqs, int32_t n_groups, int32_t G, int32_t R) {
  return shared_slots(n_tok, n_seqs, n_groups, G, R);
}

// out: s, t0, first, row0, rows, lo, hi, tile0, n_tiles, ok, units, g, own; ends: the positions each row sees of a prefix
void host_shared_item(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t max_tokens,
                      const int32_t *groups, const int32_t *prefix, int32_t n_groups, int32_t slot, int32_t G, int32_t R,
                      int32_t KT, int32_t over, int32_t *out, int32_t *ends) {
  const GroupedSeqs q = seqs(lens, cu, n_seqs, n_tok, max_tokens, groups, prefix, n_groups);
  const SharedItem it = shared_item_at(q, slot, G, R, KT);
  const int32_t v[13] = {it.s, it.t0, it.first, it.row0, it.rows, it.lo, it.hi, it.tile0, it.n_tiles, it.ok,
                         shared_units(it, over), it.g, it.own};
  for (int i = 0; i < 13; ++i) out[i] = v[i];
  for (int r = 0; r < it.rows && !it.own; ++r) ends[r] = row_end(q, it, it.row0 + r, G);
}
int64_t host_share_begin(int64_t total, int32_t b, int32_t blocks) { return share_begin(total, b, blocks); }
int32_t host_share_of(int64_t total, int64_t u, int32_t blocks) { return share_of(shares_of(total, blocks), u); }
int32_t host_shares_agree(int64_t total, int32_t blocks) {
  for (int32_t b = 0; b <= blocks; ++b)
    if (share_begin(shares_of(total, blocks), b) != share_begin(total, b, blocks)) return 0;
  return 1;
}
int32_t host_unit_tile(int32_t u, int32_t over) { return unit_tile(u, over); }
}

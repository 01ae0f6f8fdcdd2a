// The paged cache's index arithmetic (paged.cuh) compiled for the host, so that the tests can
// check on the CPU what the kernels will read and write.
#include "paged.cuh"

using namespace gdn;

static PagedSeqs seqs(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t max_tokens) {
  return PagedSeqs{lens, cu, n_seqs, n_tok, max_tokens};
}

extern "C" {
int64_t host_slots(int64_t n_tok, int32_t n_seqs, int32_t G, int32_t R) { return item_slots(n_tok, n_seqs, G, R); }

// out: s, t0, first, row0, rows, lo, hi, tile0, n_tiles, ok, units
void host_item(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t max_tokens, int32_t slot,
               int32_t G, int32_t R, int32_t KT, int32_t window, int32_t *out) {
  const Item it = item_at(seqs(lens, cu, n_seqs, n_tok, max_tokens), slot, G, R, KT, window);
  const int32_t v[11] = {it.s, it.t0, it.first, it.row0, it.rows, it.lo, it.hi, it.tile0, it.n_tiles, it.ok, item_units(it, 1)};
  for (int i = 0; i < 11; ++i) out[i] = v[i];
}
int64_t host_share(int64_t total, int32_t b, int32_t blocks) { return share_begin(total, b, blocks); }
int32_t host_page(const int32_t *row, int32_t pos, int32_t page_size, int32_t max_pages, int32_t n_pages) {
  return page_of(row, pos, page_size, max_pages, n_pages);
}
}

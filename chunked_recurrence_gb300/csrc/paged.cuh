// paged.cuh -- index arithmetic of the paged cache and of the split of attention work over
// thread blocks.  Plain integer functions, compiled for the device by the kernels and for the
// host by the tests, which check on the CPU that every page read lies in the cache and that
// the blocks' shares cover every piece of work exactly once.
//
// Sequence s holds len tokens in the pages page_table[s][0 .. ceil(len / page_size)); the last
// n_new of them are this call's queries, query i at position len - n_new + i.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// What the kernels know of a call's sequences.
struct PagedSeqs {
  const int32_t *seq_lens;  // [n_seqs] cached tokens with the new ones
  const int32_t *cu;        // [n_seqs + 1] offsets of the new tokens, or null: one each
  int32_t n_seqs;
  int32_t n_tok;
  int32_t max_tokens;       // max_pages * page_size, clamped to int32: no sequence can hold more
};

struct SeqSpan {
  int32_t t0, n_new, len;  // first new token, number of them, cached tokens
  bool ok;                 // false: offsets or length outside what the call declared (clamped here)
};

GDN_HD int32_t cu_at(const PagedSeqs &q, int32_t s) {
  if (!q.cu) return s;
  const int32_t c = q.cu[s];
  return c < 0 ? 0 : c > q.n_tok ? q.n_tok : c;
}

GDN_HD SeqSpan seq_span(const PagedSeqs &q, int32_t s) {
  SeqSpan r;
  const int32_t a = cu_at(q, s), b = cu_at(q, s + 1);
  r.ok = !q.cu || (q.cu[s] == a && q.cu[s + 1] == b && a <= b);
  r.t0 = a;
  r.n_new = b > a ? b - a : 0;
  const int32_t len = q.seq_lens[s];
  r.len = len < 0 ? 0 : len > q.max_tokens ? q.max_tokens : len;
  r.ok = r.ok && r.len == len;
  return r;
}

// Query rows of a sequence and kv head: row r is new token r / G, head r % G of the group.  They
// are cut into items of R rows.  Item p of sequence s sits in slot floor(cu[s] G / R) + s + p:
// the slots of a sequence never reach the next one's first (a sequence of n rows has at most
// floor((c + n) / R) - floor(c / R) + 1 items), so a slot is found from the offsets alone, and
// item_slots bounds their number from what the host knows.  Slots without an item stay empty.
GDN_HD int32_t slot_base(const PagedSeqs &q, int32_t s, int32_t G, int32_t R) {
  return cu_at(q, s) * G / R + s;  // the call checked that n_tok * G fits 32 bits
}
GDN_HD int64_t item_slots(int64_t n_tok, int32_t n_seqs, int32_t G, int32_t R) { return n_tok * G / R + n_seqs; }

struct Item {
  int32_t s, t0, first;   // sequence, its first new token, that token's position (may be negative)
  int32_t row0, rows;     // rows [row0, row0 + rows) of the sequence and kv head; rows = 0: no item
  int32_t lo, hi;         // positions [lo, hi) that some of these rows sees
  int32_t tile0, n_tiles; // tiles of KT positions that hold them
  bool ok;
};

// The sequence whose slots hold `slot`.
GDN_HD int32_t slot_seq(const PagedSeqs &q, int32_t slot, int32_t G, int32_t R) {
  int32_t lo = 0, hi = q.n_seqs - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (slot_base(q, mid, G, R) <= slot) lo = mid; else hi = mid - 1;
  }
  return lo;
}

GDN_HD Item item_of(const PagedSeqs &q, int32_t s, int32_t slot, int32_t G, int32_t R, int32_t KT, int32_t window) {
  Item it;
  const SeqSpan sp = seq_span(q, s);
  it.s = s;
  it.t0 = sp.t0;
  it.ok = sp.ok;
  it.first = sp.len - sp.n_new;
  const int64_t row0 = (int64_t)(slot - slot_base(q, s, G, R)) * R, all = (int64_t)sp.n_new * G;
  it.row0 = (int32_t)(row0 < all ? row0 : all);
  it.rows = (int32_t)(row0 < 0 || row0 >= all ? 0 : all - row0 < R ? all - row0 : R);
  it.lo = it.hi = it.tile0 = it.n_tiles = 0;
  if (it.rows > 0) {
    const int32_t a = it.first + it.row0 / G;                    // first row's position
    const int32_t b = it.first + (it.row0 + it.rows - 1) / G;    // last row's
    it.hi = b < 0 ? 0 : b + 1;
    it.lo = window > 0 && a >= window ? a - window + 1 : 0;
    if (it.lo < it.hi) {
      it.tile0 = it.lo / KT;
      it.n_tiles = (it.hi + KT - 1) / KT - it.tile0;
    } else {
      it.lo = it.hi = 0;
    }
  }
  return it;
}
GDN_HD Item item_at(const PagedSeqs &q, int32_t slot, int32_t G, int32_t R, int32_t KT, int32_t window) {
  return item_of(q, slot_seq(q, slot, G, R), slot, G, R, KT, window);
}

// Units of work of an item and kv head: its tiles, and `over` more in front of them for what
// every item costs whatever its length (its queries in, its output out).
GDN_HD int32_t item_units(const Item &it, int32_t over) { return it.rows <= 0 ? 0 : it.n_tiles + over; }
// Tile that unit u (0 .. units) begins with, counted from the item's first.
GDN_HD int32_t unit_tile(int32_t u, int32_t over) { return u > over ? u - over : 0; }

// Block b's share [begin, end) of `total` units over `blocks` blocks.
GDN_HD int64_t share_begin(int64_t total, int32_t b, int32_t blocks) { return total / blocks * b + total % blocks * b / blocks; }

// Page of a position, or -1 where the table names none inside the cache.
GDN_HD int32_t page_of(const int32_t *row, int32_t pos, int32_t page_size, int32_t max_pages, int32_t n_pages) {
  const int32_t i = pos / page_size;
  if (pos < 0 || i >= max_pages) return -1;
  const int32_t p = row[i];
  return p >= 0 && p < n_pages ? p : -1;
}

}  // namespace gdn

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
// The same where groups of sequences share a prefix (n_groups = 0: none does).
struct GroupedSeqs : PagedSeqs {
  const int32_t *groups, *prefix;  // [n_groups + 1] offsets of the groups' sequences, [n_groups] tokens shared
  int32_t n_groups;
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

// ---- groups of sequences that share a prefix.  The rows of a group's tokens make one run of rows against the prefix (its
// pages read from the group's first row of the table), cut into items as a sequence's are; the sequences' own items then
// begin at the prefix's end.  The groups' slots come first, then the sequences'.

struct GroupSpan {
  int32_t s0, s1, prefix;  // sequences [s0, s1), tokens that they share
  bool ok;
};
GDN_HD int32_t group_at(const GroupedSeqs &q, int32_t g) {
  const int32_t s = q.groups[g];
  return s < 0 ? 0 : s > q.n_seqs ? q.n_seqs : s;
}
GDN_HD GroupSpan group_span(const GroupedSeqs &q, int32_t g) {
  GroupSpan r;
  r.s0 = group_at(q, g), r.s1 = group_at(q, g + 1);
  const int32_t p = q.prefix[g];
  r.prefix = p < 0 ? 0 : p > q.max_tokens ? q.max_tokens : p;
  r.ok = q.groups[g] == r.s0 && q.groups[g + 1] == r.s1 && r.s0 <= r.s1 && (r.prefix == p || r.s0 == r.s1) &&
         (g > 0 || r.s0 == 0) && (g + 1 < q.n_groups || r.s1 == q.n_seqs);
  return r;
}
// The group of a sequence, and the sequence of a token: the last whose offset is not past it.
GDN_HD int32_t seq_group(const GroupedSeqs &q, int32_t s) {
  int32_t lo = 0, hi = q.n_groups - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (group_at(q, mid) <= s) lo = mid; else hi = mid - 1;
  }
  return lo;
}
GDN_HD int32_t token_seq(const PagedSeqs &q, int32_t t) {
  if (!q.cu) return t;
  int32_t lo = 0, hi = q.n_seqs - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (cu_at(q, mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}
GDN_HD int32_t group_base(const GroupedSeqs &q, int32_t g, int32_t G, int32_t R) { return cu_at(q, group_at(q, g)) * G / R + g; }
GDN_HD int64_t shared_slots(int64_t n_tok, int32_t n_seqs, int32_t n_groups, int32_t G, int32_t R) {
  return item_slots(n_tok, n_groups, G, R) + item_slots(n_tok, n_seqs, G, R);
}

struct SharedItem : Item {
  int32_t g;  // the group
  bool own;   // a sequence's own positions; else the group's prefix
};

// Rows of group g against its prefix; it.s is the group's first sequence.  A row sees less than all of the prefix where
// its token lies in it (row_end).
GDN_HD SharedItem prefix_item(const GroupedSeqs &q, int32_t g, int32_t slot, int32_t G, int32_t R, int32_t KT) {
  SharedItem it;
  const GroupSpan gs = group_span(q, g);
  const int32_t a = cu_at(q, gs.s0), b = cu_at(q, gs.s1);
  it.g = g, it.own = false;
  it.s = gs.s0 < q.n_seqs ? gs.s0 : q.n_seqs - 1;
  it.t0 = a, it.first = 0;
  const int64_t row0 = (int64_t)(slot - group_base(q, g, G, R)) * R, all = b > a ? (int64_t)(b - a) * G : 0;
  it.row0 = (int32_t)(row0 < all ? row0 : all);
  it.rows = (int32_t)(row0 < 0 || row0 >= all ? 0 : all - row0 < R ? all - row0 : R);
  const int32_t len = q.seq_lens[it.s];
  it.ok = gs.ok && (it.rows == 0 || gs.prefix <= len);
  it.lo = it.tile0 = 0;
  it.hi = it.rows > 0 ? (gs.prefix < len ? gs.prefix : len < 0 ? 0 : len) : 0;
  it.n_tiles = (it.hi + KT - 1) / KT;
  return it;
}
// Rows of sequence s, of group g, against its positions behind the prefix.
GDN_HD SharedItem own_item(const GroupedSeqs &q, int32_t g, int32_t s, int32_t slot, int32_t G, int32_t R, int32_t KT) {
  SharedItem it;
  static_cast<Item &>(it) = item_of(q, s, slot, G, R, KT, 0);
  const GroupSpan gs = group_span(q, g);
  it.g = g, it.own = true;
  if (it.rows > 0) {
    it.ok = it.ok && gs.ok && gs.prefix <= q.seq_lens[s];
    it.lo = gs.prefix;
    if (it.lo < it.hi) {
      it.tile0 = it.lo / KT;
      it.n_tiles = (it.hi + KT - 1) / KT - it.tile0;
    } else {
      it.lo = it.hi = it.tile0 = it.n_tiles = 0;
    }
  }
  return it;
}
GDN_HD SharedItem shared_item_at(const GroupedSeqs &q, int32_t slot, int32_t G, int32_t R, int32_t KT) {
  const int32_t first = (int32_t)item_slots(q.n_tok, q.n_groups, G, R);
  if (slot >= first) {
    const int32_t s = slot_seq(q, slot - first, G, R);
    return own_item(q, seq_group(q, s), s, slot - first, G, R, KT);
  }
  int32_t lo = 0, hi = q.n_groups - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (group_base(q, mid, G, R) <= slot) lo = mid; else hi = mid - 1;
  }
  return prefix_item(q, lo, slot, G, R, KT);
}
// The positions [0, row_end) of its prefix that row r (of the group) of a prefix item sees.
GDN_HD int32_t row_end(const PagedSeqs &q, const SharedItem &it, int32_t r, int32_t G) {
  const int32_t t = it.t0 + r / G;
  const SeqSpan sp = seq_span(q, token_seq(q, t));
  const int32_t end = sp.len - sp.n_new + (t - sp.t0) + 1;
  return end < 0 ? 0 : end < it.hi ? end : it.hi;
}
// Units of an item as item_units, none where it has no tiles.
GDN_HD int32_t shared_units(const Item &it, int32_t over) { return it.rows <= 0 || it.n_tiles <= 0 ? 0 : it.n_tiles + over; }

// share_begin for many blocks of one line, and the block whose share holds unit u < total, with 1 <= blocks <= total: the
// 64-bit divisions (some 100 cycles each) are made once.
struct Shares {
  int64_t each;
  int32_t rest, blocks;
  float inverse;  // blocks / total
};
GDN_HD Shares shares_of(int64_t total, int32_t blocks) {
  Shares s;
  s.each = total / blocks;
  s.rest = (int32_t)(total - s.each * blocks), s.blocks = blocks;
  s.inverse = (float)blocks / (float)total;
  return s;
}
GDN_HD int64_t share_begin(const Shares &s, int32_t b) { return s.each * b + s.rest * b / s.blocks; }  // rest < blocks: a few 100
GDN_HD int32_t share_of(const Shares &s, int64_t u) {
  int32_t b = (int32_t)((float)u * s.inverse);  // off by one at most
  if (b >= s.blocks) b = s.blocks - 1;
  while (b > 0 && share_begin(s, b) > u) --b;
  while (b + 1 < s.blocks && share_begin(s, b + 1) <= u) ++b;
  return b;
}

// Page of a position, or -1 where the table names none inside the cache.
GDN_HD int32_t page_of(const int32_t *row, int32_t pos, int32_t page_size, int32_t max_pages, int32_t n_pages) {
  const int32_t i = pos / page_size;
  if (pos < 0 || i >= max_pages) return -1;
  const int32_t p = row[i];
  return p >= 0 && p < n_pages ? p : -1;
}

}  // namespace gdn

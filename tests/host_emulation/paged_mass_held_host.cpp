// The shares of gdn_paged_mass's kernel for few query rows (paged_mass.cuh), compiled for the host with the kernel's own tile
// and cost, and the query rows that a share keeps from one piece to the next.
#define int4 HostInt4
struct HostInt4 {
  int x, y, z, w;
};
#include "paged_mass.cuh"

using namespace gdn;

static constexpr int BP = 64, OVER = 1;

extern "C" {
// Over all shares: out[0] pieces, out[1] pieces with queries that a share holds already, out[2] tiles of positions seen by a row that
// is not among those held, out[3] pieces of more than one query tile that the share does not end with.
void host_mass_held(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t most, int32_t G, int32_t Hkv,
                    int32_t RQ, int32_t window, int32_t all, int32_t units, int64_t *out) {
  MassArgs a{};
  a.seqs = PagedSeqs{lens, cu, n_seqs, n_tok, most};
  a.G = G, a.Hkv = Hkv, a.RQ = RQ, a.window = window, a.all = all, a.room = most;
  int64_t total = 0;
  for (int s = 0; s < n_seqs; ++s) total += mass_units(mass_seq(a.seqs, s, BP, window, all, most), BP, window, G, RQ, OVER) * Hkv;
  const int32_t shares = (int32_t)(units < total ? units : total);
  out[0] = out[1] = out[2] = out[3] = 0;
  MassWalk w{};
  int64_t from = 0;
  w.s = -1;
  int64_t each = 0;
  for (int b = 0; b < shares; ++b) {
    const int64_t begin = share_begin(total, b, shares);
    while (w.s < 0 || begin >= from + each * Hkv) {
      from += each * Hkv;
      ++w.s;
      w.m = mass_seq(a.seqs, w.s, BP, window, all, most);
      each = mass_units(w.m, BP, window, G, RQ, OVER);
    }
    int32_t u;
    MassWalk x = w;
    x.h = (int32_t)((begin - from) / each);
    x.j = mass_find(x.m, (begin - from) % each, BP, window, G, RQ, OVER, u);
    x.left = share_begin(total, b + 1, shares) - begin;
    x.nq = -1;
    MassHeld held{-1, 0, 0, 0};
    bool more = mass_cut<BP, OVER>(a, x, u) || mass_next<BP, OVER>(a, x);
    while (more) {
      ++out[0];
      for (int t = 0; t < x.n; ++t) {
        const MassHeld want = mass_held(a, x, t);
        if (mass_holds(held, want)) ++out[1];
        else held = want;
        // rows of the tile, as the positions see them, against those held
        bool lost = false;
        const int32_t row0 = (x.q0 + t) * RQ;
        for (int p = 0; p < BP; ++p) {
          const int32_t pos = (x.m.tile0 + x.j) * BP + p;
          if (pos < x.m.seen || pos >= x.m.hi) continue;
          int32_t lo, hi;
          mass_rows(a, x, pos, lo, hi);
          hi = hi < row0 + RQ ? hi : row0 + RQ;
          lost = lost || (hi > row0 && hi > lo && x.i0 * G + hi > held.row + held.n);
        }
        out[2] += lost;
      }
      const int32_t n = x.n;
      more = mass_next<BP, OVER>(a, x);
      out[3] += n > 1 && more;
    }
  }
}
}

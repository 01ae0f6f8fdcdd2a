// The line of work of gdn_paged_mass (paged_mass.cuh) compiled for the host, so that the tests can check on the CPU which
// tiles of positions and queries the blocks take.
#define int4 HostInt4
struct HostInt4 {
  int x, y, z, w;
};
#include "paged_mass.cuh"

using namespace gdn;

static constexpr int BP = 64, OVER = 2;

static MassArgs args(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t most, int32_t G,
                     int32_t Hkv, int32_t RQ, int32_t window, int32_t all, int32_t room) {
  MassArgs a{};
  a.seqs = PagedSeqs{lens, cu, n_seqs, n_tok, most};
  a.G = G, a.Hkv = Hkv, a.RQ = RQ, a.window = window, a.all = all, a.room = room;
  return a;
}

extern "C" {
// The pieces of all shares in turn: s, h, tile (absolute), q0, n, nq, i0, i1, share, lo, hi of each.  Returns their number, or
// -1 where they do not fit; *bad: sequences that are flagged.
int32_t host_mass_pieces(const int32_t *lens, const int32_t *cu, int32_t n_seqs, int32_t n_tok, int32_t most, int32_t G,
                         int32_t Hkv, int32_t RQ, int32_t window, int32_t all, int32_t room, int32_t units, int32_t cap,
                         int32_t *out, int32_t *bad) {
  const MassArgs a = args(lens, cu, n_seqs, n_tok, most, G, Hkv, RQ, window, all, room);
  int64_t total = 0;
  *bad = 0;
  for (int s = 0; s < n_seqs; ++s) {
    const MassSeq m = mass_seq(a.seqs, s, BP, window, all, room);
    *bad += !m.ok;
    total += mass_units(m, BP, window, G, RQ, OVER) * Hkv;
  }
  const int32_t shares = (int32_t)(units < total ? units : total);
  int32_t n = 0;
  for (int b = 0; b < shares; ++b) {
    const int64_t begin = share_begin(total, b, shares), end = share_begin(total, b + 1, shares);
    int64_t from = 0;
    MassWalk w{};
    for (w.s = 0;; ++w.s) {
      w.m = mass_seq(a.seqs, w.s, BP, window, all, room);
      const int64_t each = mass_units(w.m, BP, window, G, RQ, OVER);
      if (begin < from + each * Hkv) {
        int32_t u;
        w.h = (int32_t)((begin - from) / each);
        w.j = mass_find(w.m, (begin - from) % each, BP, window, G, RQ, OVER, u);
        w.left = end - begin;
        w.nq = -1;
        bool more = mass_cut<BP, OVER>(a, w, u) || mass_next<BP, OVER>(a, w);
        for (; more; more = mass_next<BP, OVER>(a, w)) {
          if (n == cap) return -1;
          const int32_t v[11] = {w.s, w.h, w.m.tile0 + w.j, w.q0, w.n, w.nq, w.i0, w.i1, b, w.m.lo, w.m.hi};
          for (int i = 0; i < 11; ++i) out[11 * n + i] = v[i];
          ++n;
        }
        break;
      }
      from += each * Hkv;
    }
  }
  return n;
}
}

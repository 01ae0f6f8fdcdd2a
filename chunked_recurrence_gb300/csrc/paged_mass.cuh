// paged_mass.cuh -- index arithmetic of gdn_paged_mass: which queries meet which positions, and the line of work that the
// blocks share.  Plain integer functions, compiled for the device by the kernels and for the host by the tests.
//
// The positions of a sequence and kv head are cut into tiles of BP, its query rows (row = new token * group + head in the
// group) for each tile into query tiles of RQ rows from the first row that sees some position of the tile.  Work: (sequence,
// kv head, position tile, query tile) in one line; a tile costs `over` units in front of its query tiles.
#pragma once

#include "paged.cuh"

namespace gdn {

struct MassSeq {
  SeqSpan sp;
  int32_t first;          // position of the first new token (may be negative)
  int32_t lo, hi;         // positions [lo, hi) that are written
  int32_t seen;           // the first position that some query sees: none before it is read
  int32_t tile0, n_tiles; // tiles of BP that hold them
  bool ok;
};

// all: every position is written (0 where no query sees it), else those that some query sees.  room: entries of a row of masses.
GDN_HD MassSeq mass_seq(const PagedSeqs &q, int32_t s, int32_t BP, int32_t window, bool all, int32_t room) {
  MassSeq m;
  m.sp = seq_span(q, s);
  m.ok = m.sp.ok && m.sp.len <= room;
  m.first = m.sp.len - m.sp.n_new;
  m.hi = m.sp.len < room ? m.sp.len : room;
  m.lo = 0;
  m.seen = window > 0 && m.first >= window ? m.first - window + 1 : 0;
  if (!all) {
    if (m.sp.n_new == 0) m.hi = 0;
    m.lo = m.seen < m.hi ? m.seen : m.hi;
  }
  m.tile0 = m.lo / BP;
  m.n_tiles = m.lo < m.hi ? (m.hi + BP - 1) / BP - m.tile0 : 0;
  return m;
}

// New tokens [i0, i1) that see some position of the tile at `pos` (a multiple of BP).
GDN_HD void mass_tokens(const MassSeq &m, int32_t pos, int32_t BP, int32_t window, int32_t &i0, int32_t &i1) {
  i0 = pos > m.first ? pos - m.first : 0;
  i1 = m.sp.n_new;
  if (window > 0) {
    const int64_t end = (int64_t)pos + BP - 1 + window - m.first;  // the last position's last reader, and one
    if (end < i1) i1 = end < 0 ? 0 : (int32_t)end;
  }
  if (i0 > i1) i0 = i1;
}
// Query tiles of the j-th tile of the sequence.
GDN_HD int32_t mass_tiles(const MassSeq &m, int32_t j, int32_t BP, int32_t window, int32_t G, int32_t RQ) {
  int32_t i0, i1;
  mass_tokens(m, (m.tile0 + j) * BP, BP, window, i0, i1);
  return ((i1 - i0) * G + RQ - 1) / RQ;  // the call checked that n_tok * G is below 2^30
}
// How many tiles from the j-th on have as many query tiles as it (at least it): without a window all up to the first new
// token's, with one all that end before the first that some query sees.
GDN_HD int32_t mass_alike(const MassSeq &m, int32_t j, int32_t BP, int32_t window) {
  const int32_t pos = (m.tile0 + j) * BP;
  int32_t n = 1;
  if (window <= 0) {
    if (pos <= m.first) n = (m.first - pos) / BP + 1;
  } else {
    const int64_t seen = (int64_t)m.first - window + 1;  // the first position that a query sees
    if ((int64_t)pos + BP <= seen) n = (int32_t)((seen - pos) / BP);
  }
  return n < m.n_tiles - j ? n : m.n_tiles - j;
}
// Units of a kv head of the sequence.
GDN_HD int64_t mass_units(const MassSeq &m, int32_t BP, int32_t window, int32_t G, int32_t RQ, int32_t over) {
  int64_t u = 0;
  for (int32_t j = 0; j < m.n_tiles;) {
    const int32_t n = mass_alike(m, j, BP, window);
    u += (int64_t)n * (mass_tiles(m, j, BP, window, G, RQ) + over);
    j += n;
  }
  return u;
}
// The tile that holds unit u of a head, and u's place in it.
GDN_HD int32_t mass_find(const MassSeq &m, int64_t u, int32_t BP, int32_t window, int32_t G, int32_t RQ, int32_t over,
                         int32_t &into) {
  int32_t j = 0;
  for (;;) {
    const int32_t n = mass_alike(m, j, BP, window), c = mass_tiles(m, j, BP, window, G, RQ) + over;
    if (u < (int64_t)n * c) {
      into = (int32_t)(u % c);
      return j + (int32_t)(u / c);
    }
    u -= (int64_t)n * c;
    j += n;
  }
}

// What the kernels know of a call.
struct MassArgs {
  PagedSeqs seqs;
  const void *q, *k;
  const float *lse;
  float *mass;
  const int32_t *table;
  int64_t table_stride, page_stride, slot_stride, head_stride, q_stride;
  int64_t row_stride, mass_head_stride;  // of mass
  int32_t G, Hkv, D, page_size, max_pages, n_pages, window, room, all, RQ;
  int32_t tokens, page_mask;             // RQ / G, where that is whole; page_size - 1, or -1 where that is no power of two
  float c;                               // scale log2 e
  float *part;                           // [shares][2][BP]: sums of tiles that a share does not hold whole
  int4 *meta;                            // [shares][2]: how the share's first piece goes on (1: beyond it, 2: to its tile's
                                         // end), whether its last begins a tile that the next share continues, that
                                         // tile's sequence and head; its tile
  int32_t *status;
};

// A block's share, piece by piece: query tiles [q0, q0 + n) of nq of a tile.
struct MassWalk {
  MassSeq m;
  int32_t s, h, j, nq, q0, n, i0, i1;
  int64_t left;
};
GDN_HD bool mass_begins(const MassWalk &w) { return w.q0 == 0; }
GDN_HD bool mass_ends(const MassWalk &w) { return w.q0 + w.n == w.nq; }

// Rows [lo, hi) of the tile's queries, counted from its first, that see position pos.
GDN_HD void mass_rows(const MassArgs &a, const MassWalk &w, int32_t pos, int32_t &lo, int32_t &hi) {
  const int32_t i0 = pos - w.m.first > w.i0 ? pos - w.m.first : w.i0;
  int64_t i1 = w.i1;
  if (a.window > 0 && (int64_t)pos - w.m.first + a.window < i1) i1 = (int64_t)pos - w.m.first + a.window;
  lo = (i0 - w.i0) * a.G;
  hi = i1 > w.i0 ? (int32_t)(i1 - w.i0) * a.G : 0;
}

// Rows of query tile q0 + t that a kernel may keep from one piece to the next: those from row on of the new tokens of (s, h),
// n of them.  As many as the sequence has, not as many as see the tile at hand: of the first tile that a window leaves in sight
// the last tokens may see nothing, of the next one they do.
struct MassHeld {
  int32_t s, h, row, n;
};
GDN_HD MassHeld mass_held(const MassArgs &a, const MassWalk &w, int32_t t) {
  MassHeld x;
  x.s = w.s, x.h = w.h, x.row = w.i0 * a.G + (w.q0 + t) * a.RQ;
  const int32_t rest = w.m.sp.n_new * a.G - x.row;
  x.n = rest < a.RQ ? rest : a.RQ;
  return x;
}
GDN_HD bool mass_holds(const MassHeld &held, const MassHeld &want) {
  return held.s == want.s && held.h == want.h && held.row == want.row;
}

// cuts the next piece at unit u of the tile; false where it holds nothing to do
template <int BP, int OVER>
GDN_HD bool mass_cut(const MassArgs &a, MassWalk &w, int32_t u) {
  const int32_t before = w.i1 - w.i0;
  mass_tokens(w.m, (w.m.tile0 + w.j) * BP, BP, a.window, w.i0, w.i1);
  if (w.i1 - w.i0 != before || w.nq < 0) w.nq = ((w.i1 - w.i0) * a.G + a.RQ - 1) / a.RQ;  // a division saved, mostly
  const int32_t units = w.nq + OVER;
  const int32_t end = (int32_t)(u + w.left < units ? u + w.left : units);
  w.left -= end - u;
  w.q0 = unit_tile(u, OVER);
  w.n = unit_tile(end, OVER) - w.q0;
  return w.nq > 0 ? w.n > 0 : u == 0;
}
template <int BP, int OVER>
GDN_HD bool mass_next(const MassArgs &a, MassWalk &w) {
  while (w.left > 0) {
    if (++w.j >= w.m.n_tiles) {
      w.j = 0;
      if (++w.h == a.Hkv) {
        w.h = 0;
        do {
          if (++w.s >= a.seqs.n_seqs) return false;
          w.m = mass_seq(a.seqs, w.s, BP, a.window, a.all, a.room);
        } while (w.m.n_tiles == 0);
      }
    }
    if (mass_cut<BP, OVER>(a, w, 0)) return true;
  }
  return false;
}

}  // namespace gdn

#ifdef __CUDACC__
#include "common.cuh"
#include "sm100.cuh"

namespace gdn {

// Where a block's share begins, worked out by all of its threads together.
struct MassStart {
  MassSeq m;
  int32_t s, h, j, u;
  int64_t sum[20];  // a warp each
};

// The share [begin, end) of block `unit` of `units`; false where it is empty.  Each thread counts the units of a sequence,
// the inclusive sums of a round of them give the total and then the sequence that holds the share's first unit.
template <int BP, int OVER, int THREADS>
__device__ __forceinline__ bool mass_start(const MassArgs &a, int unit, int units, MassStart &st, int64_t &left) {
  static_assert(THREADS / 32 <= sizeof(st.sum) / sizeof(st.sum[0]), "a sum a warp");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t x = 0, cost = 0, each = 0, before = 0, total = 0;
  MassSeq m;
  auto round = [&](int base) {  // units of this thread's sequence, and up to it in the round; returns the round's
    const int s = base + tid;
    cost = 0;
    if (s < a.seqs.n_seqs) {
      m = mass_seq(a.seqs, s, BP, a.window, a.all, a.room);
      if (!m.ok && unit == 0) set_status(a.status, GDN_ERR_BOUNDS);
      each = mass_units(m, BP, a.window, a.G, a.RQ, OVER);
      cost = each * a.Hkv;
    }
    x = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    __syncthreads();
    if (lane == 31) st.sum[warp] = x;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) x += st.sum[i];
      all += st.sum[i];
    }
    return all;
  };
  for (int base = 0; base < a.seqs.n_seqs; base += THREADS) total += round(base);
  const int shares = (int)min((int64_t)units, total);
  const int64_t begin = share_begin(total, min(unit, shares), max(shares, 1));
  const int64_t end = share_begin(total, min(unit + 1, shares), max(shares, 1));
  left = end - begin;
  for (int base = 0; base < a.seqs.n_seqs && begin < end; base += THREADS) {
    const int64_t all = a.seqs.n_seqs <= THREADS ? total : round(base);
    const int64_t from = before + x - cost;  // units before this sequence
    if (cost > 0 && begin >= from && begin < from + cost) {
      st.m = m;
      st.s = base + tid;
      st.h = (int)((begin - from) / each);
      st.j = mass_find(m, (begin - from) % each, BP, a.window, a.G, a.RQ, OVER, st.u);
    }
    before += all;
    if (before > begin) break;
  }
  __syncthreads();
  return begin < end;
}
template <int BP, int OVER>
__device__ __forceinline__ bool mass_begin(const MassArgs &a, const MassStart &st, int64_t left, MassWalk &w) {
  w.m = st.m;
  w.s = st.s, w.h = st.h, w.j = st.j;
  w.i0 = w.i1 = 0, w.nq = -1;
  w.left = left;
  return mass_cut<BP, OVER>(a, w, st.u) || mass_next<BP, OVER>(a, w);
}
// A piece's sum of position p of its tile: into the masses, or for the join.
template <int BP>
__device__ __forceinline__ void mass_put(const MassArgs &a, const MassWalk &w, int unit, int p, float sum) {
  const int pos = (w.m.tile0 + w.j) * BP + p;
  if (mass_begins(w) && mass_ends(w)) {
    if (pos >= w.m.lo && pos < w.m.hi) {
      float *to = a.mass + w.s * a.row_stride + w.h * a.mass_head_stride + pos;
      *to = a.all ? sum : *to + sum;
    }
  } else {
    a.part[((int64_t)2 * unit + mass_begins(w)) * BP + p] = sum;
  }
}
// What the join has to know of a piece, from one thread.
__device__ __forceinline__ void mass_note(const MassArgs &a, const MassWalk &w, int unit) {
  int4 *me = a.meta + 2 * unit;
  if (!mass_begins(w)) {
    me->x = mass_ends(w) ? 2 : 1;
  } else if (!mass_ends(w)) {
    me->y = 1, me->z = w.s, me->w = w.h;
    me[1] = make_int4(w.j, 0, 0, 0);
  }
}

// Tiles that lie in several shares: share b's last piece begins one, the next share's first goes on with it, until a
// first piece ends it.  Added in that order.
template <int BP>
__global__ void __launch_bounds__(BP) mass_join_kernel(const MassArgs a, int shares) {
  sm100::grid_dependency_wait();
  const int b = blockIdx.x, p = threadIdx.x;
  const int4 me = a.meta[2 * b];
  if (!me.y) return;
  float sum = a.part[((int64_t)2 * b + 1) * BP + p];
  int how = 1;
  for (int i = b + 1; how == 1; ++i) {
    how = i < shares ? a.meta[2 * i].x : 0;
    if (how) sum += a.part[(int64_t)2 * i * BP + p];
  }
  if (how != 2) return;  // a share that gave up
  const MassSeq m = mass_seq(a.seqs, me.z, BP, a.window, a.all, a.room);
  const int pos = (m.tile0 + a.meta[2 * b + 1].x) * BP + p;
  if (pos < m.lo || pos >= m.hi) return;
  float *to = a.mass + me.z * a.row_stride + me.w * a.mass_head_stride + pos;
  *to = a.all ? sum : *to + sum;
}

// A launch that starts under the end of the kernel before on the stream, and the join behind it.
template <int BP, typename... P, typename... A>
gdn_status mass_launch(void (*kernel)(P...), const MassArgs &a, int blocks, int shares, int threads, size_t smem,
                       cudaStream_t st, A... args) {
  if (smem && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return (void)cudaGetLastError(), GDN_ERR_CUDA;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  // the join goes by what the kernel writes
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return (void)cudaGetLastError(), GDN_ERR_CUDA;
  cfg.gridDim = dim3(shares), cfg.blockDim = dim3(BP), cfg.dynamicSmemBytes = 0;
  cudaLaunchKernelEx(&cfg, mass_join_kernel<BP>, a, shares);
  return launch_status();
}

bool paged_mass_tc_supported(const gdn_cache_shape &s, const void *q, const void *k);
size_t paged_mass_tc_workspace(const gdn_cache_shape &s);
gdn_status paged_mass_tc(MassArgs &a, const gdn_cache_shape &s, uint32_t flags, void *workspace, cudaStream_t st);

// Of the calls that the one on tcgen05 takes, those of few query rows.
bool paged_mass_few(const MassArgs &a, int32_t max_new);
size_t paged_mass_few_workspace();
gdn_status paged_mass_few_run(MassArgs &a, int32_t max_new, void *workspace, cudaStream_t st);

}  // namespace gdn
#endif

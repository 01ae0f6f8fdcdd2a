// pages.cu -- the bookkeeping of a paged cache's pages, on the device: growing, freeing and
// forking sequences, bringing live pages together, copying pages.
//
// refs[page] counts the sequences that hold a page; a page at 0 is free, and free pages are taken
// in rising order.  The decisions (which pages, whether there are enough) need a sum over all
// refs or all sequences: one block makes them (plan kernels, a running block scan over refs in
// 16-byte loads) and leaves lists in the workspace.  What is proportional to the data
// (table rows, page contents) runs on the whole GPU (move_kernel), which reads the lists.
//
// Copying is bound by HBM: a moved byte is read once and written once (1.14 GB read and written to bring the pages of a
// half-empty cache together: 181 us, 94% of a copy's rate).  Small calls are launches and the plan's chain of loads:
// freeing and forking 24 of 48 sequences 14 us, some 6 of them the plan.  No page is both read and written by one call
// (compact moves pages at or past L into free ones below it; fork's new pages were free), so the copies run in any
// order.
#include <algorithm>

#include "common.cuh"
#include "paged.cuh"
#include "sm100.cuh"

using namespace gdn;
using sm100::grid_dependency_wait;
using sm100::launch_dependents;

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
// Entries of a fork's parents' rows that the plan looks through itself (1128: 8.6 us a fork, 8.9 and a launch more with a
// kernel for it; 4096: 9.9 and 8.9; unchecked 7.4 and 7.6).
constexpr int kPlanEntries = 2048;

// Words of the workspace after the 256 bytes that hold the status.
struct PlanWords {
  int32_t ok, n_moves, live, pad;
};

struct Plan {
  PlanWords *w;
  int32_t *src, *dst, *to;  // [n_pages] each: moves, and compact's new page of each moved one
  int32_t *rows;            // [n_rows] lengths saved while a list is checked
};

__device__ Plan plan_of(void *workspace, int32_t n_pages) {
  char *p = (char *)workspace;
  Plan r;
  r.w = (PlanWords *)(p + 128);
  r.src = (int32_t *)(p + 256);
  r.dst = r.src + n_pages;
  r.to = r.dst + n_pages;
  r.rows = r.to + n_pages;
  return r;
}

struct Pools {
  void *p[GDN_MAX_POOLS];
};

// Inclusive sum over the block's threads; *total gets the whole.  sh: 33 words.
__device__ __forceinline__ int block_scan(int x, int *sh, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();  // sh is free
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = lane < warps ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += u;
    }
    sh[lane] = y;
  }
  __syncthreads();
  *total = sh[warps - 1];
  return x + (warp ? sh[warp - 1] : 0);
}

// Four consecutive refs of a thread, n past the end read as `past`.
__device__ __forceinline__ int4 load_refs(const int32_t *refs, int i, int n, int past) {
  if (i + 3 < n && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) return *reinterpret_cast<const int4 *>(refs + i);
  return make_int4(i < n ? refs[i] : past, i + 1 < n ? refs[i + 1] : past, i + 2 < n ? refs[i + 2] : past,
                   i + 3 < n ? refs[i + 3] : past);
}

// The first `want` free pages into list, in rising order; returns how many there are of them.
__device__ int first_free(const int32_t *refs, int n_pages, int want, int32_t *list, int *sh) {
  int found = 0;
  for (int base = 0; base < n_pages && found < want; base += 4 * kPlanThreads) {
    const int i = base + 4 * threadIdx.x;
    const int4 r = load_refs(refs, i, n_pages, 1);
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    int total;
    int at = found + block_scan(f[0] + f[1] + f[2] + f[3], sh, &total) - (f[0] + f[1] + f[2] + f[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) {
        if (at < want) list[at] = i + k;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

__device__ __forceinline__ int32_t *table_row(const gdn_page_tables &t, int s) {
  return t.page_table + (int64_t)s * t.table_stride;
}

// ------------------------------------------------------------------- plans

// A listed row is claimed by taking its length out of seq_lens (-1 instead): a second claim of
// the same row sees it.  On an error the claims are undone and nothing has changed.
__global__ void __launch_bounds__(kPlanThreads) grow_kernel(const gdn_page_tables t, const int32_t *seqs,
                                                            const int32_t *new_lens, int n, void *workspace) {
  __shared__ int sh[33];
  const Plan pl = plan_of(workspace, t.n_pages);
  grid_dependency_wait();
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = seqs[i];
    int old = -1;
    if (s >= 0 && s < t.n_rows) old = atomicExch(&t.seq_lens[s], -1);
    pl.rows[i] = old;
    bad = bad || old < 0 || new_lens[i] < old || new_lens[i] > (int64_t)t.max_pages * t.page_size ||
          new_lens[i] / t.page_size > t.n_pages;  // keeps the sums below within 32 bits
  }
  bad = __syncthreads_or(bad);
  int total = 0;
  for (int base = 0; base < n && !bad; base += kPlanThreads) {  // pages wanted, all rows
    const int i = base + threadIdx.x;
    int part;
    block_scan(i < n ? (int)(((int64_t)new_lens[i] + t.page_size - 1) / t.page_size -
                             ((int64_t)pl.rows[i] + t.page_size - 1) / t.page_size)
                     : 0,
               sh, &part);
    total = min(total + part, t.n_pages + 1);
  }
  bad = bad || total > t.n_pages || first_free(t.refs, t.n_pages, total, pl.src, sh) < total;
  int taken = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int old = i < n ? pl.rows[i] : -1;
    if (bad) {
      if (old >= 0) t.seq_lens[seqs[i]] = old;
      continue;
    }
    const int a = i < n ? (int)(((int64_t)old + t.page_size - 1) / t.page_size) : 0;
    const int b = i < n ? (int)(((int64_t)new_lens[i] + t.page_size - 1) / t.page_size) : 0;
    int part;
    int at = taken + block_scan(b - a, sh, &part) - (b - a);
    if (i < n) {
      int32_t *row = table_row(t, seqs[i]);
      for (int k = a; k < b; ++k) {
        const int page = pl.src[at++];
        row[k] = page;
        t.refs[page] = 1;
      }
      t.seq_lens[seqs[i]] = new_lens[i];
    }
    taken += part;
  }
  if (bad && threadIdx.x == 0) set_status(t.status, GDN_ERR_PAGES);
}

__global__ void __launch_bounds__(256) free_kernel(const gdn_page_tables t, const int32_t *seqs) {
  __shared__ int s_len;
  grid_dependency_wait();
  launch_dependents();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= t.n_rows) {
    if (threadIdx.x == 0) set_status(t.status, GDN_ERR_PAGES);
    return;
  }
  if (threadIdx.x == 0) s_len = atomicExch(&t.seq_lens[s], 0);  // a row named twice is empty the second time
  __syncthreads();
  const int64_t pages = ((int64_t)max(s_len, 0) + t.page_size - 1) / t.page_size;
  if (pages > t.max_pages && threadIdx.x == 0) set_status(t.status, GDN_ERR_BOUNDS);
  int32_t *row = table_row(t, s);
  for (int i = threadIdx.x; i < min(pages, (int64_t)t.max_pages); i += blockDim.x) {
    const int page = row[i];
    row[i] = -1;
    if (page == -1) continue;
    if (page < 0 || page >= t.n_pages) {
      set_status(t.status, GDN_ERR_BOUNDS);
    } else if (atomicSub(&t.refs[page], 1) <= 0) {  // held by nobody: stays at 0
      atomicAdd(&t.refs[page], 1);
      set_status(t.status, GDN_ERR_PAGES);
    }
  }
}

// Whether a fork's parent cannot give entry k of its row: a page outside the cache, or none where it has a part-filled
// one (a full page may have been given back, -1).  Rows and lengths that cannot be are found by the plan.
__device__ __forceinline__ bool bad_entry(const gdn_page_tables &t, int parent, int k) {
  const int len = parent >= 0 && parent < t.n_rows ? __ldcg(&t.seq_lens[parent]) : -1;
  const int full = len / t.page_size, part = len % t.page_size;
  if (len < 0 || k > full || (k == full && !part)) return false;
  const int page = table_row(t, parent)[k];
  if (page < -1 || page >= t.n_pages) return set_status(t.status, GDN_ERR_BOUNDS), true;
  return page == -1 && k == full;
}

// A parent's entries, a block a parent: rows[i] says whether one is bad.
__global__ void __launch_bounds__(256) fork_check_kernel(const gdn_page_tables t, const int32_t *parents, void *workspace) {
  const Plan pl = plan_of(workspace, t.n_pages);
  grid_dependency_wait();
  launch_dependents();
  const int p = parents[blockIdx.x];
  bool bad = false;
  for (int k = threadIdx.x; k < t.max_pages; k += blockDim.x) bad = bad_entry(t, p, k) || bad;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) pl.rows[blockIdx.x] = bad;
}

// fork: checks the pairs (and the parents' entries, unless fork_check_kernel has), takes the new pages and lists the
// copies; move_kernel writes the rows.
template <bool CHECKED>
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const gdn_page_tables t, const int32_t *parents,
                                                                 const int32_t *children, int n, void *workspace) {
  __shared__ int sh[33];
  const Plan pl = plan_of(workspace, t.n_pages);
  bool bad = false;
  grid_dependency_wait();
  launch_dependents();  // the moves' blocks wait for this one's end where they read
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int c = children[i];
    int old = -1;
    if (c >= 0 && c < t.n_rows) old = atomicExch(&t.seq_lens[c], -1);
    if (CHECKED) bad = bad || pl.rows[i];
    pl.rows[i] = old;
    bad = bad || old != 0;
  }
  // no barrier before: a parent that is claimed by now is refused below
#pragma unroll 2
  for (int i = threadIdx.x; !CHECKED && i < n * t.max_pages; i += kPlanThreads)
    bad = bad_entry(t, parents[i / t.max_pages], i % t.max_pages) || bad;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int p = parents[i];  // a parent that is a child too has been claimed
    const int len = p >= 0 && p < t.n_rows ? *(volatile int32_t *)&t.seq_lens[p] : -1;
    bad = bad || len < 0 || len > (int64_t)t.max_pages * t.page_size;
  }
  bad = __syncthreads_or(bad);
  int total = 0;
  for (int base = 0; base < n && !bad; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    total += __syncthreads_count(i < n && t.seq_lens[parents[i]] % t.page_size != 0);
  }
  bad = bad || total > t.n_pages || first_free(t.refs, t.n_pages, total, pl.dst, sh) < total;
  int taken = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    if (bad) {
      if (i < n && pl.rows[i] >= 0) t.seq_lens[children[i]] = pl.rows[i];
      continue;
    }
    const int len = i < n ? t.seq_lens[parents[i]] : 0;
    const int part = len % t.page_size != 0;
    int sum;
    const int at = taken + block_scan(part, sh, &sum) - part;
    if (part) {
      pl.src[at] = table_row(t, parents[i])[len / t.page_size];
      t.refs[pl.dst[at]] = 1;
      table_row(t, children[i])[len / t.page_size] = pl.dst[at];
    }
    taken += sum;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n && !bad; i += kPlanThreads) t.seq_lens[children[i]] = t.seq_lens[parents[i]];
  if (threadIdx.x == 0) {
    pl.w->ok = !bad;
    pl.w->n_moves = bad ? 0 : total;
    if (bad) set_status(t.status, GDN_ERR_PAGES);
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const gdn_page_tables t, void *workspace) {
  __shared__ int sh[33];
  const Plan pl = plan_of(workspace, t.n_pages);
  grid_dependency_wait();
  launch_dependents();
  int live = 0;
  for (int i = 4 * threadIdx.x; i < t.n_pages; i += 4 * kPlanThreads) {
    const int4 r = load_refs(t.refs, i, t.n_pages, 0);
    live += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  int L;
  block_scan(live, sh, &L);
  // free pages below L and live ones from L on: as many of the one as of the other
  int n_dst = 0, n_src = 0;
  for (int base = 0; base < t.n_pages; base += 4 * kPlanThreads) {
    const int i = base + 4 * threadIdx.x;
    const int4 r4 = load_refs(t.refs, i, t.n_pages, 0);
    const int r[4] = {r4.x, r4.y, r4.z, r4.w};
    int d = 0, s = 0, total;
#pragma unroll
    for (int k = 0; k < 4; ++k) d += i + k < L && r[k] <= 0, s += i + k >= L && r[k] > 0;
    if (base < L) {
      int at = n_dst + block_scan(d, sh, &total) - d;
      n_dst += total;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < L && r[k] <= 0) pl.dst[at++] = i + k;
    }
    if (base + 4 * kPlanThreads > L) {
      int at = n_src + block_scan(s, sh, &total) - s;
      n_src += total;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k >= L && i + k < t.n_pages) {
          if (r[k] > 0) pl.src[at++] = i + k;
          else pl.to[i + k] = i + k;  // a table that names a free page keeps it
        }
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < n_src; k += kPlanThreads) {
    const int s = pl.src[k], d = pl.dst[k];
    pl.to[s] = d;
    t.refs[d] = t.refs[s];
    t.refs[s] = 0;
  }
  if (threadIdx.x == 0) {
    pl.w->ok = 1;
    pl.w->n_moves = n_src;
    pl.w->live = L;
  }
}

// ------------------------------------------------------------------- moves

enum MoveKind { kFork, kCompact, kCopy };

// Table rows (fork: the children's from the parents'; compact: every row by `to`), then the page copies: pieces
// of kPiece vectors, dealt out over the blocks.
template <typename V, int KIND>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const gdn_page_tables t, const int32_t *a,
                                                            const int32_t *b, int n, const Pools pools, int n_pools,
                                                            int64_t page_bytes, int64_t page_stride, void *workspace) {
  constexpr int kPer = 8;  // vectors a thread moves in one go, all loads before the first store
  grid_dependency_wait();  // for the plan
  const Plan pl = plan_of(workspace, t.n_pages);
  const int32_t *src = KIND == kCopy ? a : pl.src, *dst = KIND == kCopy ? b : pl.dst;
  int moves = n;
  if (KIND != kCopy) {
    if (!pl.w->ok) return;
    moves = pl.w->n_moves;
  }
  if (KIND == kFork) {
    const int64_t all = (int64_t)n * t.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kMoveThreads) {
      const int j = (int)(i / t.max_pages), k = (int)(i - (int64_t)j * t.max_pages);
      const int len = t.seq_lens[a[j]];
      if (k >= len / t.page_size) continue;  // the new page of a part-filled one is in place
      const int page = table_row(t, a[j])[k];
      table_row(t, b[j])[k] = page;
      if (page >= 0) atomicAdd(&t.refs[page], 1);
    }
  }
  if (KIND == kCompact) {
    const int64_t all = (int64_t)t.n_rows * t.max_pages;
    const int L = pl.w->live;
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kMoveThreads) {
      const int j = (int)(i / t.max_pages), k = (int)(i - (int64_t)j * t.max_pages);
      if ((int64_t)k * t.page_size >= t.seq_lens[j]) continue;
      int32_t *e = table_row(t, j) + k;
      const int page = *e;
      if (page < L) continue;  // stays, or -1
      if (page < t.n_pages) *e = pl.to[page];
      else set_status(t.status, GDN_ERR_BOUNDS);
    }
  }
  const int64_t vecs = page_bytes / (int64_t)sizeof(V);
  const int64_t piece = kPer * kMoveThreads, per_page = (vecs + piece - 1) / piece;
  const int64_t pieces = (int64_t)moves * n_pools * per_page;
  for (int64_t x = blockIdx.x; x < pieces; x += gridDim.x) {
    const int64_t mp = x / per_page, c = x - mp * per_page;
    const int m = (int)(mp / n_pools), pool = (int)(mp - (int64_t)m * n_pools);
    const int s = src[m], d = dst[m];
    if (KIND == kCopy && (s < 0 || d < 0 || s >= t.n_pages || d >= t.n_pages)) {
      if (threadIdx.x == 0) set_status(t.status, GDN_ERR_BOUNDS);
      continue;
    }
    const V *from = (const V *)((const char *)pools.p[pool] + s * page_stride) + c * piece + threadIdx.x;
    V *to = (V *)((char *)pools.p[pool] + d * page_stride) + c * piece + threadIdx.x;
    const int64_t left = vecs - c * piece - threadIdx.x;
    V v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kMoveThreads < left) v[i] = __ldcs(from + i * kMoveThreads);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kMoveThreads < left) __stcs(to + i * kMoveThreads, v[i]);
  }
}

// The tables checked, strides and the status word filled in.
bool tables_ok(const gdn_page_tables *in, void *workspace, gdn_page_tables *t) {
  if (!in) return false;
  *t = *in;
  if (t->n_rows < 0 || t->max_pages < 0 || t->n_pages < 0 || t->page_size < 1 || !aligned(t->status, sizeof(int32_t)))
    return false;
  if (t->table_stride == 0) t->table_stride = t->max_pages;
  if (!t->status) t->status = (int32_t *)workspace;
  if (t->table_stride < t->max_pages || t->n_pages >= 1 << 21) return false;  // sums of 1024 rows' pages: 32 bits
  return (t->n_rows == 0 || (t->page_table && t->seq_lens)) && (t->n_pages == 0 || t->refs);
}

gdn_status pools_ok(const gdn_page_pools *in, Pools *p) {
  if (!in || in->n_pools < 0 || in->page_bytes < 0 || in->page_stride < in->page_bytes || (in->n_pools && !in->pools))
    return GDN_ERR_INVALID_ARG;
  if (in->n_pools > GDN_MAX_POOLS) return GDN_ERR_UNSUPPORTED;
  for (int i = 0; i < in->n_pools; ++i) {
    if (!in->pools[i]) return GDN_ERR_INVALID_ARG;
    p->p[i] = in->pools[i];
  }
  return GDN_OK;
}

// A launch that overlaps the end of the kernel before on the stream, whose results the kernel waits for.
template <typename... P, typename... A>
void launch_early(void (*kernel)(P...), int blocks, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks), cfg.blockDim = dim3(threads), cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename V, int KIND>
void launch_move(const gdn_page_tables &t, const int32_t *a, const int32_t *b, int n, const gdn_page_pools &in,
                 const Pools &pools, void *workspace, cudaStream_t st) {
  const int blocks = 152 * 8;  // resident at once: 256 threads, eight vectors each in flight
  launch_early(move_kernel<V, KIND>, blocks, kMoveThreads, st, t, a, b, n, pools, (int)in.n_pools,
               (int64_t)in.page_bytes, (int64_t)in.page_stride, workspace);
}

template <int KIND>
gdn_status launch_moves(const gdn_page_tables &t, const int32_t *a, const int32_t *b, int n, const gdn_page_pools &in,
                        const Pools &pools, void *workspace, cudaStream_t st) {
  uintptr_t bits = (uintptr_t)in.page_bytes | (uintptr_t)in.page_stride;
  for (int i = 0; i < in.n_pools; ++i) bits |= (uintptr_t)pools.p[i];
  if (bits % 16 == 0) launch_move<uint4, KIND>(t, a, b, n, in, pools, workspace, st);
  else if (bits % 4 == 0) launch_move<uint32_t, KIND>(t, a, b, n, in, pools, workspace, st);
  else launch_move<uint8_t, KIND>(t, a, b, n, in, pools, workspace, st);
  return launch_status();
}

size_t need(int32_t n_pages, int32_t n_rows) { return 256 + sizeof(int32_t) * (3 * (size_t)n_pages + n_rows); }

bool ws_ok(const void *w, size_t bytes, size_t want) { return w && aligned(w, 256) && bytes >= want; }

}  // namespace

extern "C" size_t gdn_pages_workspace_bytes(int32_t n_pages, int32_t n_rows) {
  return n_pages < 0 || n_rows < 0 ? 0 : need(n_pages, n_rows);
}

extern "C" gdn_status gdn_pages_grow(const gdn_page_tables *tables, const int32_t *seqs, const int32_t *new_lens,
                                     int32_t n, void *workspace, size_t workspace_bytes, void *stream) {
  gdn_page_tables t;
  if (!tables_ok(tables, workspace, &t) || n < 0 || n > t.n_rows) return GDN_ERR_INVALID_ARG;  // no row twice
  if (!ws_ok(workspace, workspace_bytes, need(t.n_pages, t.n_rows))) return GDN_ERR_WORKSPACE;
  if (n == 0) return GDN_OK;
  if (!seqs || !new_lens) return GDN_ERR_INVALID_ARG;
  launch_early(grow_kernel, 1, kPlanThreads, (cudaStream_t)stream, t, seqs, new_lens, (int)n, workspace);
  return launch_status();
}

extern "C" gdn_status gdn_pages_free(const gdn_page_tables *tables, const int32_t *seqs, int32_t n, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  gdn_page_tables t;
  if (!tables_ok(tables, workspace, &t) || n < 0) return GDN_ERR_INVALID_ARG;
  if (!tables->status && !ws_ok(workspace, workspace_bytes, need(t.n_pages, t.n_rows))) return GDN_ERR_WORKSPACE;
  if (n == 0) return GDN_OK;
  if (!seqs) return GDN_ERR_INVALID_ARG;
  launch_early(free_kernel, n, 256, (cudaStream_t)stream, t, seqs);
  return launch_status();
}

extern "C" gdn_status gdn_pages_fork(const gdn_page_tables *tables, const int32_t *parents, const int32_t *children,
                                     int32_t n, const gdn_page_pools *pools, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  gdn_page_tables t;
  Pools p{};
  if (!tables_ok(tables, workspace, &t) || n < 0 || n > t.n_rows) return GDN_ERR_INVALID_ARG;
  const gdn_status ok = pools_ok(pools, &p);
  if (ok != GDN_OK) return ok;
  if (!ws_ok(workspace, workspace_bytes, need(t.n_pages, t.n_rows))) return GDN_ERR_WORKSPACE;
  if (n == 0) return GDN_OK;
  if (!parents || !children) return GDN_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if ((int64_t)n * t.max_pages <= kPlanEntries) {
    launch_early(fork_plan_kernel<false>, 1, kPlanThreads, st, t, parents, children, (int)n, workspace);
  } else {
    launch_early(fork_check_kernel, n, 256, st, t, parents, workspace);
    launch_early(fork_plan_kernel<true>, 1, kPlanThreads, st, t, parents, children, (int)n, workspace);
  }
  if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
  return launch_moves<kFork>(t, parents, children, n, *pools, p, workspace, st);
}

extern "C" gdn_status gdn_pages_compact(const gdn_page_tables *tables, const gdn_page_pools *pools, void *workspace,
                                        size_t workspace_bytes, void *stream) {
  gdn_page_tables t;
  Pools p{};
  if (!tables_ok(tables, workspace, &t)) return GDN_ERR_INVALID_ARG;
  const gdn_status ok = pools_ok(pools, &p);
  if (ok != GDN_OK) return ok;
  if (!ws_ok(workspace, workspace_bytes, need(t.n_pages, t.n_rows))) return GDN_ERR_WORKSPACE;
  if (t.n_pages == 0) return GDN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  launch_early(compact_plan_kernel, 1, kPlanThreads, st, t, workspace);
  if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
  return launch_moves<kCompact>(t, nullptr, nullptr, 0, *pools, p, workspace, st);
}

extern "C" gdn_status gdn_pages_copy(const int32_t *src, const int32_t *dst, int32_t n, int32_t n_pages,
                                     const gdn_page_pools *pools, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  Pools p{};
  if (n < 0 || n_pages < 0) return GDN_ERR_INVALID_ARG;
  const gdn_status ok = pools_ok(pools, &p);
  if (ok != GDN_OK) return ok;
  if (!ws_ok(workspace, workspace_bytes, 256)) return GDN_ERR_WORKSPACE;
  if (n == 0) return GDN_OK;
  if (!src || !dst) return GDN_ERR_INVALID_ARG;
  gdn_page_tables t{};
  t.n_pages = n_pages, t.status = (int32_t *)workspace;
  return launch_moves<kCopy>(t, src, dst, n, *pools, p, workspace, (cudaStream_t)stream);
}

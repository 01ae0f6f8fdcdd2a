// pages_evict.cu -- gdn_pages_evict: sequences of a paged cache cut to the positions that gathered the most attention
// weight, each layer and kv head its own.
//
// Of a sequence of N tokens m stay: the last r = min(recent, m), and of the N - r before them the m - r with the largest
// weight, ties to the lowest position.  In rising order they become positions 0 .. m - 1, in fresh pages of the sequence's
// own, so other sequences that share its old pages keep theirs as they are, every row is read and written once, and no
// copy waits for another.
//
// Two launches.  choose_kernel: one block checks the lists and takes the free pages, one a sequence saves and checks its row
// of the table, one a range of pages checks that none is given back more often than it is held, and one a (layer, sequence,
// head) finds the weights' order: a radix selection over the weights as whole numbers of the same order (digits of 11, 11 and
// 10 bits from the top, the counts in shared memory; after the first digit those that are left are few) ends with the
// m - r th largest T; those above T and the first of those at T are written in order to the workspace.  apply_kernel: nothing
// where a list, row or range was refused; else the rows move, 32 positions of a head a block with its place in the old and
// new pages worked out once for all pools of the layer, the weights follow, and tables, lengths and refs are written.
//
// Bounds: the second kernel moves bytes, scattered rows of 256 in and whole pages out.  24 sequences of 700 to 6000 tokens cut
// to 1900, 2 kv heads, D 256, two layers (256 MB): 50 us, 5.1 TB/s; blocks of 16 and 64 positions took as long.  The first
// takes 14 to 18 us: a block a list, passes over it from registers for the digits, each with its barriers, and the lists
// written in order (pages_choose.cuh).  48 lists are 48 of 152 SMs; a list over a cluster of blocks, counts added through
// their shared memory, is not built.
#include <algorithm>

#include "pages.cuh"
#include "pages_choose.cuh"

using namespace gdn;
using namespace gdn::pages;
using sm100::grid_dependency_wait;
using sm100::launch_dependents;

namespace {

constexpr int kApplyThreads = 128;
constexpr int kRows = 32;          // positions of a head that a block moves at a time
constexpr int kRange = sizeof(ChooseShared) / sizeof(int);  // pages whose holders a block counts

struct Evict {
  gdn_page_tables t;
  const int32_t *seqs, *keep;
  int32_t n, max_keep, recent, n_layers, heads, mass_len;
  float *mass;
  int64_t layer_stride, row_stride, head_stride;  // of mass
  int32_t *kept;
  // the workspace
  int32_t *ok;      // [1 + n + ranges] 1 where the lists, each sequence's row, and each range of pages' refs are in order
  int32_t *len;     // [n] lengths before
  int32_t *page0;   // [n] first of a sequence's fresh pages in `fresh`; -1: nothing to evict
  int32_t *mark;    // [n_rows]
  int32_t *fresh;   // [n_pages]
  int32_t *old;     // [n][max_pages] rows of the table before
  int32_t *index;   // [n_layers][n][heads][max_keep] positions that stay
  float *weight;    // the same, their weights
};

__device__ __forceinline__ int pages_for(int64_t tokens, int page_size) { return (int)((tokens + page_size - 1) / page_size); }
// Whether the list's entry i is one to evict from: its row and numbers in range, and less kept than there is.
__device__ __forceinline__ bool in_range(const Evict &e, int s, int len, int m) {
  return s >= 0 && s < e.t.n_rows && len >= 0 && len <= (int64_t)e.t.max_pages * e.t.page_size && m >= 0 && m <= e.max_keep;
}

__device__ void plan_block(const Evict &e, int *sh) {
  const gdn_page_tables &t = e.t;
  bool bad = false;
  for (int i = threadIdx.x; i < e.n; i += kChooseThreads) {
    const int s = e.seqs[i], m = e.keep[i];
    const int len = s >= 0 && s < t.n_rows ? t.seq_lens[s] : -1;
    bad = bad || !in_range(e, s, len, m);
    e.len[i] = len;
    if (s >= 0 && s < t.n_rows) e.mark[s] = i;
  }
  bad = __syncthreads_or(bad);
  // a row listed twice has one entry's mark; the fresh pages, sequence after sequence
  int64_t total = 0;
  for (int base = 0; base < e.n && !bad; base += kChooseThreads) {
    const int i = base + threadIdx.x;
    int want = 0, part;
    if (i < e.n) {
      want = e.keep[i] < e.len[i] ? pages_for(e.keep[i], t.page_size) : 0;
      bad = e.mark[e.seqs[i]] != i || want > t.n_pages;
      if (bad) want = 0;  // the sum of 1024 fits 32 bits
    }
    bad = __syncthreads_or(bad);
    const int at = (int)total + block_scan(want, sh, &part) - want;
    if (i < e.n) e.page0[i] = e.keep[i] < e.len[i] ? at : -1;
    total += part;
    if (total > t.n_pages) bad = true;  // the same for all threads
  }
  bad = bad || first_free(t.refs, t.n_pages, (int)total, e.fresh, sh) < total;
  if (threadIdx.x == 0) {
    e.ok[0] = !bad;
    if (bad) set_status(t.status, GDN_ERR_PAGES);
  }
}

__device__ void row_block(const Evict &e, int i) {
  const gdn_page_tables &t = e.t;
  const int s = e.seqs[i], m = e.keep[i];
  const int len = s >= 0 && s < t.n_rows ? t.seq_lens[s] : -1;
  bool bad = false;
  if (in_range(e, s, len, m) && m < len) {
    const int pages = pages_for(len, t.page_size);
    for (int k = threadIdx.x; k < pages; k += kChooseThreads) {
      const int page = table_row(t, s)[k];
      e.old[(int64_t)i * t.max_pages + k] = page;
      if (page < 0 || page >= t.n_pages) {
        set_status(t.status, page == -1 ? GDN_ERR_PAGES : GDN_ERR_BOUNDS);
        bad = true;
      } else if (t.refs[page] <= 0) {  // might be one of the fresh pages
        set_status(t.status, GDN_ERR_PAGES);
        bad = true;
      }
    }
    if (len > e.mass_len) {
      if (threadIdx.x == 0) set_status(t.status, GDN_ERR_BOUNDS);
      bad = true;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) e.ok[1 + i] = !bad;
}

__host__ __device__ __forceinline__ int ranges_of(const gdn_page_tables &t) { return (t.n_pages + kRange - 1) / kRange; }

// Pages [b kRange, (b + 1) kRange): no more of the sequences that give theirs back may hold one than its refs say.  A block a
// range, which reads all their rows (a warp a row, or several) and counts in shared memory: counts of all pages in memory
// would have to be cleared by a launch before.
__device__ void range_block(const Evict &e, int b, int *count) {
  const gdn_page_tables &t = e.t;
  const int first = b * kRange, pages = min(kRange, t.n_pages - first), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int p = threadIdx.x; p < pages; p += kChooseThreads) count[p] = 0;
  __syncthreads();
  const int warps = kChooseThreads / 32, parts = max(warps / e.n, 1);
  for (int w = warp; w / parts < e.n; w += warps / parts * parts) {
    if (warp >= warps / parts * parts) break;
    const int i = w / parts, s = e.seqs[i], m = e.keep[i];
    const int len = s >= 0 && s < t.n_rows ? t.seq_lens[s] : -1;
    if (!in_range(e, s, len, m) || m >= len) continue;
    const int32_t *row = table_row(t, s);
    const int held = pages_for(len, t.page_size);
#pragma unroll 4
    for (int k = w % parts * 32 + lane; k < held; k += parts * 32) {
      const uint32_t p = (uint32_t)row[k] - first;
      if (p < (uint32_t)pages) atomicAdd(&count[p], 1);
    }
  }
  __syncthreads();
  bool bad = false;
  for (int p = threadIdx.x; p < pages; p += kChooseThreads) bad = bad || (count[p] > 0 && count[p] > t.refs[first + p]);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(t.status, GDN_ERR_PAGES);
    bad = true;
  }
  if (threadIdx.x == 0) e.ok[1 + e.n + b] = !bad;
}

__global__ void __launch_bounds__(kChooseThreads) choose_kernel(const Evict e) {
  __shared__ ChooseShared sm;
  grid_dependency_wait();
  launch_dependents();
  // the lists of the largest index first: the plan and the rows are shorter
  const int lists = gridDim.x - 1 - e.n - ranges_of(e.t), other = (int)blockIdx.x - lists;
  if (other == 0) return plan_block(e, sm.sh);
  if (other > e.n) return range_block(e, other - 1 - e.n, reinterpret_cast<int *>(&sm));
  if (other > 0) return row_block(e, other - 1);
  const int64_t lih = blockIdx.x;
  const int h = (int)(lih % e.heads), i = (int)(lih / e.heads % e.n), l = (int)(lih / e.heads / e.n);
  const int s = e.seqs[i], m = e.keep[i];
  const int len = s >= 0 && s < e.t.n_rows ? e.t.seq_lens[s] : -1;
  if (!in_range(e, s, len, m) || m >= len || len > e.mass_len) return;
  const float *mass = e.mass + l * e.layer_stride + s * e.row_stride + h * e.head_stride;
  int32_t *index = e.index + lih * e.max_keep;
  float *weight = e.weight + lih * e.max_keep;
  const int recent = min(e.recent, m), N = len - recent, need = m - recent;  // need < N
  for (int j = threadIdx.x; j < recent; j += kChooseThreads) {
    index[need + j] = N + j;
    weight[need + j] = mass[N + j];
  }
  if (need > 0) choose_largest(mass, N, need, index, weight, sm);
}

template <typename V>
__global__ void __launch_bounds__(kApplyThreads) apply_kernel(const Evict e, const Pools pools, int per_layer,
                                                              int64_t page_stride, int64_t slot_stride,
                                                              int64_t slot_head_stride, int vecs) {
  constexpr int kPer = 8;  // vectors a thread moves in one go, all loads before the first store
  __shared__ int64_t from[kRows], to[kRows];
  const gdn_page_tables &t = e.t;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  bool ok = e.ok[0];
  for (int i = tid; i < e.n + ranges_of(t); i += kApplyThreads) ok = ok && e.ok[1 + i];
  bool asked = false;  // whether the lists can be carried out: after the first loads, which wait as long

  const int chunks = (e.max_keep + kRows - 1) / kRows;
  const int64_t blocks = (int64_t)e.n_layers * e.n * e.heads * chunks;
  for (int64_t x = blockIdx.x; x < blocks; x += gridDim.x) {
    // the heads of the same positions one after another: their rows lie side by side in the pages
    const int64_t li_c = x / e.heads, li = li_c / chunks;
    const int h = (int)(x - li_c * e.heads), j0 = (int)(li_c - li * chunks) * kRows, i = (int)(li % e.n);
    const int64_t lih = li * e.heads + h;
    // (of lists that cannot be carried out page0 may be anything)
    const int l = (int)(li / e.n), page0 = e.page0[i], s = e.seqs[i], len = e.len[i];
    const int m = page0 < 0 ? 0 : min(e.keep[i], e.max_keep);
    const int rows = min(kRows, m - j0);
    int src = 0;
    float weight = 0.f;
    if (tid < rows) src = e.index[lih * e.max_keep + j0 + tid], weight = e.weight[lih * e.max_keep + j0 + tid];
    if (__syncthreads_or(!asked && !ok)) return;  // and the places of the rows before are done with
    asked = true;
    float *mass = e.mass + l * e.layer_stride + s * e.row_stride + h * e.head_stride;
    if (tid < kRows) {
      const int j = j0 + tid;
      if (tid < rows) {
        from[tid] = e.old[(int64_t)i * t.max_pages + src / t.page_size] * page_stride + src % t.page_size * slot_stride +
                    h * slot_head_stride;
        to[tid] = e.fresh[page0 + j / t.page_size] * page_stride + j % t.page_size * slot_stride + h * slot_head_stride;
        mass[j] = weight;
        if (e.kept) e.kept[lih * e.max_keep + j] = src;
      } else if (e.kept && j < e.max_keep) {
        e.kept[lih * e.max_keep + j] = page0 < 0 && j < len ? j : -1;
      }
    }
    __syncthreads();
    // the rows of the layer's pools
    const int all = max(rows, 0) * vecs * per_layer;
    for (int v0 = tid; v0 < all; v0 += kPer * kApplyThreads) {
      V v[kPer];
      char *dst[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int y = v0 + k * kApplyThreads;
        if (y < all) {
          const int row = y / vecs, c = y - row * vecs, p = row / rows, r = row - p * rows;
          char *pool = (char *)pools.p[l * per_layer + p] + c * (int64_t)sizeof(V);
          v[k] = __ldcs((const V *)(pool + from[r]));
          dst[k] = pool + to[r];
        }
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (v0 + k * kApplyThreads < all) __stcs((V *)dst[k], v[k]);
    }
  }
  if (__syncthreads_or(!asked && !ok)) return;
  // weights behind what is kept
  const int64_t rows = (int64_t)e.n_layers * e.n * e.heads;
  for (int64_t lih = blockIdx.x; lih < rows; lih += gridDim.x) {
    const int h = (int)(lih % e.heads), i = (int)(lih / e.heads % e.n), l = (int)(lih / e.heads / e.n);
    if (e.page0[i] < 0) continue;
    float *mass = e.mass + l * e.layer_stride + e.seqs[i] * e.row_stride + h * e.head_stride;
    for (int j = e.keep[i] + tid; j < e.len[i]; j += kApplyThreads) mass[j] = 0.f;
  }
  // tables, lengths and refs, from the last block on: the first ones have a chunk more to move
  for (int i = gridDim.x - 1 - blockIdx.x; i < e.n; i += gridDim.x) {
    if (e.page0[i] < 0) continue;
    const int m = e.keep[i], a = pages_for(m, t.page_size), b = pages_for(e.len[i], t.page_size);
    int32_t *row = table_row(t, e.seqs[i]);
    for (int k = tid; k < b; k += kApplyThreads) {
      const int page = e.old[(int64_t)i * t.max_pages + k], now = k < a ? e.fresh[e.page0[i] + k] : -1;
      row[k] = now;
      if (now >= 0) t.refs[now] = 1;
      atomicSub(&t.refs[page], 1);
    }
    if (tid == 0) t.seq_lens[e.seqs[i]] = m;
  }
}

// The arguments checked and filled in; the workspace's places and size.
bool heads_ok(const gdn_page_heads *in, const gdn_page_tables &t, gdn_page_heads *h) {
  if (!in) return false;
  *h = *in;
  if (h->n_layers < 1 || h->heads < 1 || h->mass_len < 0 || h->row_bytes < 1) return false;
  if (h->layer_stride == 0 && h->row_stride == 0 && h->head_stride == 0) {
    h->head_stride = h->mass_len;
    h->row_stride = h->head_stride * h->heads;
    h->layer_stride = h->row_stride * t.n_rows;
  }
  if (h->slot_stride == 0 && h->slot_head_stride == 0) {
    h->slot_head_stride = h->row_bytes;
    h->slot_stride = h->row_bytes * h->heads;
  }
  return !((h->heads > 1 && (h->head_stride < h->mass_len || h->slot_head_stride < h->row_bytes)) ||
           (t.n_rows > 1 && h->row_stride < h->mass_len) || (h->n_layers > 1 && h->layer_stride < h->mass_len) ||
           (t.page_size > 1 && h->slot_stride < h->row_bytes) || h->slot_head_stride < 0 || h->slot_stride < 0 ||
           h->layer_stride < 0 || h->row_stride < 0 || h->head_stride < 0);
}

size_t lay_out(Evict &e, void *workspace) {
  const size_t lists = (size_t)e.n_layers * e.n * e.heads * e.max_keep;
  int32_t *w = (int32_t *)((char *)workspace + 256);
  e.ok = w, w += 1 + e.n + ranges_of(e.t);
  e.len = w, w += e.n;
  e.page0 = w, w += e.n;
  e.mark = w, w += e.t.n_rows;
  e.fresh = w, w += e.t.n_pages;
  e.old = w, w += (size_t)e.n * e.t.max_pages;
  e.index = w, w += lists;
  e.weight = (float *)w;
  return (char *)(w + lists) - (char *)workspace;
}

}  // namespace

extern "C" size_t gdn_pages_evict_workspace_bytes(const gdn_page_tables *tables, int32_t n, int32_t max_keep,
                                                  int32_t n_layers, int32_t heads) {
  if (!tables || tables->n_rows < 0 || tables->max_pages < 0 || tables->n_pages < 0 || n < 0 || max_keep < 0 ||
      n_layers < 1 || heads < 1)
    return 0;
  Evict e{};
  e.t = *tables;
  e.n = n, e.max_keep = max_keep, e.n_layers = n_layers, e.heads = heads;
  return lay_out(e, nullptr);
}

extern "C" gdn_status gdn_pages_evict(const gdn_page_tables *tables, const int32_t *seqs, const int32_t *keep, int32_t n,
                                      int32_t max_keep, int32_t recent, const gdn_page_heads *heads,
                                      const gdn_page_pools *pools, int32_t *kept, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  Evict e{};
  gdn_page_heads h;
  Pools p{};
  if (!tables_ok(tables, workspace, &e.t) || n < 0 || n > e.t.n_rows || max_keep < 0 || recent < 0 ||
      !heads_ok(heads, e.t, &h))
    return GDN_ERR_INVALID_ARG;
  const gdn_status ok = pools_ok(pools, &p);
  if (ok != GDN_OK) return ok;
  if (pools->n_pools % h.n_layers != 0) return GDN_ERR_INVALID_ARG;
  // a page holds its slots' heads
  const int64_t slots = e.t.page_size - 1, others = h.heads - 1, room = pools->page_bytes - h.row_bytes;
  if (pools->n_pools && (room < 0 || (slots && h.slot_stride > room / slots) || (others && h.slot_head_stride > room / others) ||
                         slots * h.slot_stride + others * h.slot_head_stride > room))
    return GDN_ERR_INVALID_ARG;
  // a thread's place in a list (up to two rounds past its end), the blocks of a launch, and the vectors of a block's rows
  // fit 32 bits
  constexpr int32_t kMost = INT32_MAX - 4 * 4 * kChooseThreads + 1;
  if (h.mass_len > kMost || max_keep > kMost) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)h.n_layers * n * h.heads > 1 << 29 || h.row_bytes > 1 << 16) return GDN_ERR_UNSUPPORTED;
  e.n = n, e.max_keep = max_keep, e.recent = recent, e.n_layers = h.n_layers, e.heads = h.heads, e.mass_len = h.mass_len;
  if (!ws_ok(workspace, workspace_bytes, lay_out(e, workspace))) return GDN_ERR_WORKSPACE;
  if (n == 0) return GDN_OK;
  if (!seqs || !keep || (!h.mass && h.mass_len > 0)) return GDN_ERR_INVALID_ARG;
  e.seqs = seqs, e.keep = keep, e.mass = h.mass, e.kept = kept;
  e.layer_stride = h.layer_stride, e.row_stride = h.row_stride, e.head_stride = h.head_stride;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t lists = (int64_t)h.n_layers * n * h.heads;
  launch_early(choose_kernel, (int)(lists + 1 + n + ranges_of(e.t)), kChooseThreads, st, 0, e);
  if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
  const int per_layer = pools->n_pools / h.n_layers;
  const int64_t work = std::max<int64_t>(lists * ((max_keep + kRows - 1) / kRows), n);
  const int blocks = (int)std::min<int64_t>(work, 1 << 16);
  uintptr_t bits = (uintptr_t)pools->page_stride | (uintptr_t)h.slot_stride | (uintptr_t)h.slot_head_stride | (uintptr_t)h.row_bytes;
  for (int i = 0; i < pools->n_pools; ++i) bits |= (uintptr_t)p.p[i];
  auto apply = [&](auto v) {
    using V = decltype(v);
    launch_early(apply_kernel<V>, blocks, kApplyThreads, st, 0, e, p, per_layer, (int64_t)pools->page_stride,
                 (int64_t)h.slot_stride, (int64_t)h.slot_head_stride, (int)(h.row_bytes / sizeof(V)));
  };
  if (bits % 16 == 0) apply(uint4{});
  else if (bits % 4 == 0) apply(uint32_t{});
  else apply(uint8_t{});
  return launch_status();
}

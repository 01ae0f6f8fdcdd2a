// paged_mass_few.cu -- gdn_paged_mass for few query rows a sequence and kv head (single tokens; bf16, D = 64, 128 or 256).
//
// HBM bounds it: the keys are read once and meet a handful of rows.  Every warp has a share of the work of its own
// (paged_mass.cuh, tiles of 64 positions) and no barrier on the way.  A lane's fragment of a product (mma.sync) of 16
// positions is four columns of a row, two pairs 8 columns apart; as the order of a sum's terms is free, the lane takes
// 16 bytes of the row that lie together, for two products, and the queries' fragments, which stay in registers, are taken
// the same way.  So a lane reads back from shared memory only what it copied there itself: a queue of its own, in which the
// rows of 16 positions are asked for three products ahead (asynchronous copies), the pages of the next tile a tile ahead.
// 64 single tokens over 500 to 16000, 32 / 8 heads, D 128: 206 us, some 10 of them the masses put back, 83% of a copy's rate
// (tcgen05 with four of a tile's 256 columns in use: 452; fragments straight from global memory, without the queue: 301).  64 x 4
// drafted tokens over 4000 to 8000: 148 us, with windows of 4096 and 1024 121 and 39 (by bytes alone 121, 83 and 21).
#include <algorithm>

#include "common.cuh"
#include "paged_attn.cuh"
#include "paged_mass.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kSms = 152, kBP = 64, kOver = 1, kDepth = 4;

// NT: tiles of 8 query rows that the registers hold
template <int D, int NT>
struct Cfg {
  static constexpr int kWarps = D == 256 ? 6 : NT == 4 ? 8 : 12;  // by their queues, and the queries in registers
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kVecs = D / 32;            // 16-byte pieces of a row a lane
  static constexpr int kEntry = 2 * kVecs * 512;  // bytes of a warp's rows of 16 positions
  static constexpr int kSmem = kWarps * kDepth * kEntry;
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {  // zeros where there is nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// The units before each thread's sequences (thread i has the i-th run of `per`), and of all.
template <int THREADS>
__device__ int64_t count_units(const MassArgs &a, int per, int64_t *before) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int64_t sums[THREADS / 32];
  int64_t mine = 0;
  for (int s = tid * per; s < min((tid + 1) * per, a.seqs.n_seqs); ++s) {
    const MassSeq m = mass_seq(a.seqs, s, kBP, a.window, a.all, a.room);
    if (!m.ok && blockIdx.x == 0) set_status(a.status, GDN_ERR_BOUNDS);
    mine += mass_units(m, kBP, a.window, a.G, a.RQ, kOver) * a.Hkv;
  }
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) x += sums[i];
    total += sums[i];
  }
  before[tid] = x - mine;
  __syncthreads();
  return total;
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) paged_mass_few_kernel(const MassArgs a) {
  using C = Cfg<D, NT>;
  constexpr int kVecs = C::kVecs;
  extern __shared__ __align__(16) uint8_t queues[];
  __shared__ int64_t before[C::kThreads];
  const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
  const int unit = blockIdx.x * C::kWarps + (threadIdx.x >> 5), units = gridDim.x * C::kWarps;
  sm100::launch_dependents();
  sm100::grid_dependency_wait();
  if (lane == 0) a.meta[2 * unit] = make_int4(0, 0, 0, 0);
  const int per = (a.seqs.n_seqs + C::kThreads - 1) / C::kThreads;
  const int64_t total = count_units<C::kThreads>(a, per, before);
  const int shares = (int)min((int64_t)units, total);
  if (unit >= shares) return;
  MassWalk w;
  {
    const int64_t begin = share_begin(total, unit, shares);
    w.left = share_begin(total, unit + 1, shares) - begin;
    int k = 0;  // the last thread with no more than `begin` units before it
    for (int base = 0; base < C::kThreads; base += 32) k += __popc(__ballot_sync(0xffffffffu, before[base + lane] <= begin));
    int64_t u = begin - before[k - 1];
    for (w.s = (k - 1) * per;; ++w.s) {
      w.m = mass_seq(a.seqs, w.s, kBP, a.window, a.all, a.room);
      const int64_t each = mass_units(w.m, kBP, a.window, a.G, a.RQ, kOver);
      if (u < each * a.Hkv) {
        w.h = (int)(u / each), u %= each;
        break;
      }
      u -= each * a.Hkv;
    }
    int into;
    w.j = mass_find(w.m, u, kBP, a.window, a.G, a.RQ, kOver, into);
    w.i0 = w.i1 = 0, w.nq = -1;
    if (!mass_cut<kBP, kOver>(a, w, into) && !mass_next<kBP, kOver>(a, w)) return;
  }
  // where the rows of positions lane and lane + 32 of a piece's tile lie, -1: not read
  auto places = [&](const MassWalk &x, bool there, int64_t (&off)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int pos = (x.m.tile0 + x.j) * kBP + lane + 32 * k;
      off[k] = -1;
      if (there && x.n > 0 && pos >= x.m.seen && pos < x.m.hi) {
        const int page = page_of(a.table + x.s * a.table_stride, pos, a.page_size, a.max_pages, a.n_pages);
        if (page < 0) set_status(a.status, GDN_ERR_BOUNDS);
        else off[k] = page * a.page_stride + (a.page_mask >= 0 ? pos & a.page_mask : pos % a.page_size) * a.slot_stride +
                      x.h * a.head_stride;
      }
    }
  };
  // rows g4 and g4 + 8 of the c-th 16 positions, this lane's pieces, into entry c of its queue and out of it
  const uint8_t *queue = queues + (threadIdx.x >> 5) * kDepth * C::kEntry + lane * 16;
  auto load = [&](const int64_t (&off)[2], int c) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t at = __shfl_sync(0xffffffffu, off[c / 2], (c & 1) * 16 + g4 + 8 * e);
      const uint4 *p = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.k + (at >= 0 ? at : 0)) + t4;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        copy16(sm100::smem_u32(queue + c * C::kEntry + (e * kVecs + j) * 512), p + 4 * j, at >= 0);
    }
    cp_async_commit();
  };
  uint4 q[NT][kVecs];
  float nl[NT][2];  // minus lse in base 2 of this lane's columns
  MassHeld held{-1, 0, 0, 0};
  auto queries = [&](int t) {  // query tile q0 + t of the piece, unless it is there
    const MassHeld want = mass_held(a, w, t);
    if (mass_holds(held, want)) return;
    held = want;
    const int row = want.row, rows = want.n;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 8 + g4, i = (row + r) / a.G, g = row + r - i * a.G;
      const uint4 *p = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.q + (w.m.sp.t0 + i) * a.q_stride +
                                                       (int64_t)(w.h * a.G + g) * D) + t4;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) q[n][j] = r < rows ? p[4 * j] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = n * 8 + 2 * t4 + e, ci = (row + c) / a.G, cg = row + c - ci * a.G;
        const float x = c < rows ? a.lse[(int64_t)(w.m.sp.t0 + ci) * (a.G * a.Hkv) + w.h * a.G + cg] : -INFINITY;
        nl[n][e] = x == -INFINITY ? x : x * -1.44269504088896340736f;  // -inf: weighs nothing
      }
    }
  };
  // adds to sum[0], sum[1] the weights of positions g4 and g4 + 8 of the c-th 16 of the tile
  auto weigh = [&](int c, int t, float (&sum)[2]) {
    const uint4 *r0 = reinterpret_cast<const uint4 *>(queue + c * C::kEntry), *r1 = r0 + kVecs * 32;
    const int row0 = (w.q0 + t) * a.RQ, pos = (w.m.tile0 + w.j) * kBP + 16 * c + g4;
    int lo[2], hi[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mass_rows(a, w, pos + 8 * e, lo[e], hi[e]);
      lo[e] -= row0, hi[e] = min(hi[e] - row0, a.RQ);
    }
    float s[NT][2][4];  // two sums, of every second product
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[n][i / 4][i % 4] = 0.f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const uint4 x = r0[j * 32], y = r1[j * 32];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma(s[n][0], x.x, y.x, x.y, y.y, q[n][j].x, q[n][j].y);
        mma(s[n][1], x.z, y.z, x.w, y.w, q[n][j].z, q[n][j].w);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = n * 8 + 2 * t4 + (i & 1);
        const float y = ex2(fmaf(s[n][0][i] + s[n][1][i], a.c, nl[n][i & 1]));
        sum[i >> 1] += col >= lo[i >> 1] && col < hi[i >> 1] ? y : 0.f;
      }
  };

  int64_t off[2], ahead[2];
  places(w, true, off);
#pragma unroll
  for (int c = 0; c < kDepth - 1; ++c) load(off, c);
  for (bool more = true; more;) {
    MassWalk next = w;
    more = mass_next<kBP, kOver>(a, next);
    places(next, more, ahead);
    // this lane's two positions in the end: of the t4-th 16 of the tile
    const int pos = (w.m.tile0 + w.j) * kBP + 16 * t4 + g4;
    const bool whole = mass_begins(w) && mass_ends(w);
    float *to = a.mass + w.s * a.row_stride + w.h * a.mass_head_stride + pos;
    float old[2], sum[4][2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      old[e] = whole && !a.all && pos + 8 * e >= w.m.lo && pos + 8 * e < w.m.hi ? to[8 * e] : 0.f;
    if (w.n > 0) queries(0);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // the entry's products came before this; it is free
      if (c == 0) load(off, 3);
      else load(ahead, c - 1);
      asm volatile("cp.async.wait_group 3;" ::: "memory");
      sum[c][0] = sum[c][1] = 0.f;
      if (w.n > 0) weigh(c, 0, sum[c]);
    }
    if (w.n > 1) {  // more rows than the call said: the tile once more for each 8 NT of them, then the next tile's first rows
      cp_async_wait_all();  // the next tile's, asked for above: copies to one place have no order
      for (int t = 1; t < w.n; ++t) {
        queries(t);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          load(off, c);
          cp_async_wait_all();
          weigh(c, t, sum[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < kDepth - 1; ++c) load(ahead, c);
    }
    float out[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = sum[c][e];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (t4 == c) out[e] = x;
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!whole) a.part[((int64_t)2 * unit + mass_begins(w)) * kBP + 16 * t4 + g4 + 8 * e] = out[e];
      else if (pos + 8 * e >= w.m.lo && pos + 8 * e < w.m.hi) to[8 * e] = old[e] + out[e];
    }
    if (lane == 0) mass_note(a, w, unit);
    w = next;
    off[0] = ahead[0], off[1] = ahead[1];
  }
  cp_async_wait_all();  // what was asked for behind the last tile
}

template <int D, int NT>
gdn_status launch(MassArgs &a, void *workspace, cudaStream_t st) {
  const int shares = kSms * Cfg<D, NT>::kWarps;
  a.meta = (int4 *)((char *)workspace + 256);
  a.part = (float *)(a.meta + 2 * shares);
  return mass_launch<kBP>(paged_mass_few_kernel<D, NT>, a, kSms, shares, Cfg<D, NT>::kThreads, Cfg<D, NT>::kSmem, st, a);
}
template <int D>
gdn_status dispatch(MassArgs &a, void *workspace, cudaStream_t st) {
  const int tiles = (a.RQ + 7) / 8;
  if (tiles <= 1) return launch<D, 1>(a, workspace, st);
  if (tiles <= 2) return launch<D, 2>(a, workspace, st);
  if constexpr (D < 256) return launch<D, 4>(a, workspace, st);
  return GDN_ERR_UNSUPPORTED;
}

}  // namespace

// Query rows that the registers hold beside the keys.
bool paged_mass_few(const MassArgs &a, int32_t max_new) {
  return (int64_t)std::max(max_new, 1) * a.G <= (a.D == 256 ? 16 : 32);
}
size_t paged_mass_few_workspace() { return 256 + (size_t)kSms * 12 * (2 * sizeof(int4) + 2 * kBP * sizeof(float)); }

gdn_status paged_mass_few_run(MassArgs &a, int32_t max_new, void *workspace, cudaStream_t st) {
  a.tokens = std::max(max_new, 1);
  a.RQ = a.tokens * a.G;
  a.page_mask = a.page_size & (a.page_size - 1) ? -1 : a.page_size - 1;
  return a.D == 64 ? dispatch<64>(a, workspace, st) : a.D == 128 ? dispatch<128>(a, workspace, st)
                                                               : dispatch<256>(a, workspace, st);
}

}  // namespace gdn

// paged_attn_tc.cuh -- the kernel of attention of new tokens over a paged cache on the tensor cores
// (tcgen05, bf16; D = 64, 128 or 256), and of the same where groups of sequences share a prefix.
//
// One pass over the keys with a running maximum m and sum l per query row,
//     S = Q K^T,  P = 2^(c S - c m),  l += sum P,  O += P V,   c = scale log2 e,
// and O, l scaled by 2^(c (m_old - m_new)) when m moves; o = O / l at the end.  m may lag
// behind the true maximum by a factor 2^8 in P (fp32 sums and bf16 weights keep their relative
// precision), so O is seldom touched after the first tiles.
//
// Query rows of a kv head (row = token * group + head in the group) are cut into items of R = 128 NQ
// rows, keys into tiles of 128 positions.  NQ = 2 (D <= 128): two 128-row tiles share each K and V
// tile and take turns, one's softmax under the other's MMAs.  NQ = 1: one row tile; S alternates between two TMEM
// slots, so the next tile's S runs under this one's softmax.  TMEM: two S slots of a tile's columns
// (P, as bf16 pairs, lies over its S), then O.
//
// Work: (item, kv head, tile) in one line, cut into equal shares, one persistent block each, so ragged lengths
// and causal shapes balance to a tile.  A share begins or ends inside an item where it must; such a piece leaves
// (m, l, O) in the workspace and join_kernel adds the pieces up.  Every block finds its share by a
// scan over the sequences' lengths: nothing is planned on the host, and the lengths stay on the
// device.
//
// Warps: softmax warpgroups (one per row tile: a thread owns a query row), a warp for K's and Q's copies and one for
// V's (pages by their table entries, 64 columns x gcd(page_size, tile) slots a box, into 128B-swizzled panels), an
// MMA thread.  K and V granules go through one ring in the order in which the MMAs read them.
//
// PAIR: two blocks of a cluster share an item of twice the rows (cta_group::2, M = 256).  Each holds its rows' Q and P
// and half of each K and V tile, so K and V come from L2 once for both and the ring holds twice the tiles.
//
// What bounds it, and what it measured (a copy 6694 GB/s, a cuBLAS product 1885 TFLOP/s in a burst, 1707 sustained).
// Single tokens, HBM: 64 x 8192 positions, 8 kv heads, D 128, pages of 16: 319 us, 101% of the copy's rate; ragged 500
// to 16000, pages of 64: 344 us, 97%; D 64: 205 us, 78% (rows of 128 bytes).  Chunks, the matrix instructions and the
// waits between them: 8192 over 16384, 32/8 heads, D 128: 1115 us, 1479 TFLOP/s; 4096 over 8192, 16/2 heads, D 256:
// 251 us, 1644.  D 64 waits on the softmax, as many weights as at D 256 for a quarter of the products: 999 us for
// the first of these.  A few short sequences: some 13 us, the chain of launch, lengths, table, copies, S, P, O, then the
// join's.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <numeric>
#include <type_traits>

#include "common.cuh"
#include "conv_tap.cuh"
#include "paged_attn.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kSms = 152;            // persistent blocks
constexpr uint32_t kSpin = 1u << 22; // polls of a wait before it gives up
constexpr int kData = 224 * 1024;    // Q and the ring
constexpr float kLag = 8.f;          // m may lag by this many powers of two

template <int D, int NQ, bool PAIR>
struct Cfg {
  static constexpr int kPair = PAIR ? 2 : 1;            // blocks (of one cluster) that share an item
  static constexpr int kTiles = NQ * kPair;             // 128-row tiles of an item
  static constexpr int R = 128 * kTiles;                // TMEM lanes of an item; it fills RT of each 128
  static constexpr int KT = D == 256 && !PAIR ? 64 : 128; // positions a tile
  // A granule is a block's part of a tile of K or V.  A pair's MMA takes its second operand in halves of N from the two
  // blocks: of K half the positions, of V half the columns.
  static constexpr int kGran = KT * D * 2 / kPair;      // bytes
  static constexpr int kRowsK = KT / kPair;
  static constexpr int kPanelK = kRowsK * 128, kPanelV = KT * 128;  // bytes of 64 columns of it
  static constexpr int kPanelsK = D / 64, kPanelsV = D / 64 / kPair;
  static constexpr int kQ = 128 * NQ * D * 2;
  static constexpr int kSlots = (kData - kQ) / kGran < 16 ? (kData - kQ) / kGran : 16;
  // softmax warpgroups, then the warps of K's copies (and Q's), the MMAs and V's copies; with two tiles a whole
  // warpgroup for those, so that the registers can be split between the warpgroups
  static constexpr int kThreads = NQ == 2 ? 384 : 224;
  static constexpr int kHalves = NQ == 1 ? 2 : 1;       // parts in which P is handed over
  static constexpr uint32_t kO = 256;                   // first TMEM column of O
  // units (tiles) an item costs beyond its tiles: its first S, the mask of its last tile, its output
  static constexpr int kOver = NQ == 1 && !PAIR ? 2 : 4;
};

// Without groups the kernel is to stay what it is without them: its schedule moves with what is beside it (8192 over 16384:
// 1147 us, 1177 with the fields of a shared call in its items).
template <bool SHARED>
using SeqsOf = std::conditional_t<SHARED, GroupedSeqs, PagedSeqs>;
template <bool SHARED>
using ItemOf = std::conditional_t<SHARED, SharedItem, Item>;

struct PlainArgs {};
struct SharedSums {
  // units before each slot [slots] and of all, and of each kind (prefix, own), kv head and row (token * G + head of the
  // group) the sums of an item that one share holds whole, with its maximum and sum: 32 rows a block, [column / 4][row] fours
  int64_t *from;
  float *full, *full_ml;
};
template <bool SHARED>
struct TcArgs : std::conditional_t<SHARED, SharedSums, PlainArgs> {
  SeqsOf<SHARED> seqs;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *o;
  float *lse;
  const int32_t *table;
  int64_t table_stride, q_stride;
  int32_t G, RT, Hkv, page_size, page_mask, box, box_log2, max_pages, n_pages, window;  // RT: rows of a 128-row tile in use, whole
                                                                // tokens; page_mask: page_size - 1, or -1 where no power of two
  float c;  // scale log2 e
  float *part, *part_ml;
  int4 *meta;  // [blocks][2]: how the share's first piece goes on (1: beyond it, 2: to its item's end), whether its last
               // one begins an item that the next share continues, that item's head and rows; its first token and row
  int32_t *status;
  int32_t no_wait;
};

__device__ __forceinline__ bool own_part(const SharedItem &it) { return it.own; }
__device__ __forceinline__ bool own_part(const Item &) { return true; }

struct SharedStart : SharedItem {
  int partial;  // some token lies in its group's prefix
};
template <bool SHARED>
struct Ctl {
  uint64_t full[16], empty[16], land[16], sfull[2], pready[2][2], odone[2], qfull[2], qfree[2], drain;
  uint32_t tmem;
  volatile int abort;
  int64_t sum[12];
  int start_slot, start_h, start_u;
  std::conditional_t<SHARED, SharedStart, Item> start;
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// The forms for a pair of blocks.  Their barriers are named by cluster addresses.
__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2,
                                                 int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Arrivals at the other block's barrier order no memory of this block at cluster scope: a release at that
// scope takes some 700 cycles, and P (tensor memory, ordered by the tcgen05 fences) and the copies (counted in
// bytes) do not need it.  Where plain stores have to be seen, the caller fences.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// The MMAs and their commits, of one block or (issued by its first block) of a pair.
template <bool PAIR>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    umma_bf16(d, a, b, idesc, accumulate);
}
// both blocks' barrier at this place (PAIR), or this block's
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    umma_commit(bar);
}

// D[tmem] (+)= A[tmem] * B[smem]
template <bool PAIR>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32u(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats to a bf16 pair (a in the low half), round to nearest even
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// a wait of all lanes, the same answer for all of them
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, kSpin, abort));
}

// A block's share of the line of work, piece by piece: `n` tiles from tile `j` of an item and
// head (n = 0 for one without tiles, whose rows get zeros).
template <bool SHARED>
struct Walk {
  ItemOf<SHARED> it;
  int slot, h, j, n, u, units;
  int64_t left;
};
// Units that an item costs beyond its tiles: where rows behind a shared prefix fill one of two row tiles, half of the two's (64
// samples of 16000: 75 us, 85 with 4; chunks of up to 300, which fill both, 348 us with 4 and 415 with 2).
template <class C, bool SHARED>
__device__ __forceinline__ int32_t over_of(const Item &it, int RT) {
  return SHARED && C::kTiles > C::kPair && it.rows <= RT * C::kPair ? C::kOver / 2 : C::kOver;
}
template <class C, bool SHARED>
__device__ __forceinline__ int32_t units_of(const Item &it, int RT) {
  return SHARED ? shared_units(it, over_of<C, SHARED>(it, RT)) : item_units(it, C::kOver);
}
// cuts the next piece at unit u of the item; false where it holds nothing to do
template <class C, bool SHARED>
__device__ __forceinline__ bool walk_cut(Walk<SHARED> &w, int RT) {
  const int end = (int)min((int64_t)w.units, w.u + w.left), over = over_of<C, SHARED>(w.it, RT);
  w.left -= end - w.u;
  w.j = unit_tile(w.u, over);
  w.n = unit_tile(end, over) - w.j;
  return w.it.n_tiles > 0 ? w.n > 0 : w.u == 0;
}
// the item of the next slot
template <class C, bool SHARED>
__device__ __forceinline__ void walk_slot(const TcArgs<SHARED> &a, Walk<SHARED> &w, int R) {
  int s = w.it.s;
  if constexpr (SHARED) {
    int g = w.it.g, slot = w.slot;
    const int first = (int)item_slots(a.seqs.n_tok, a.seqs.n_groups, a.G, R);
    if (slot < first) {
      while (g + 1 < a.seqs.n_groups && group_base(a.seqs, g + 1, a.G, R) <= slot) ++g;
      w.it = prefix_item(a.seqs, g, slot, a.G, R, C::KT);
      return;
    }
    slot -= first;
    if (!w.it.own) s = g = 0;
    while (s + 1 < a.seqs.n_seqs && slot_base(a.seqs, s + 1, a.G, R) <= slot) ++s;
    while (g + 1 < a.seqs.n_groups && group_at(a.seqs, g + 1) <= s) ++g;
    w.it = own_item(a.seqs, g, s, slot, a.G, R, C::KT);
  } else {
    while (s + 1 < a.seqs.n_seqs && slot_base(a.seqs, s + 1, a.G, R) <= w.slot) ++s;
    w.it = item_of(a.seqs, s, w.slot, a.G, R, C::KT, a.window);
  }
}
template <class C, bool SHARED>
__device__ __forceinline__ bool walk_next(const TcArgs<SHARED> &a, Walk<SHARED> &w, int R, int slots) {
  while (w.left > 0) {
    w.u = 0;
    if (++w.h == a.Hkv) {
      w.h = 0;
      do {
        if (++w.slot >= slots) return false;
        walk_slot<C, SHARED>(a, w, R);
        w.units = units_of<C, SHARED>(w.it, a.RT);
      } while (w.units == 0);
    }
    if (walk_cut<C, SHARED>(w, a.RT)) return true;
  }
  return false;
}
template <class C, bool SHARED>
__device__ __forceinline__ bool walk_begin(const TcArgs<SHARED> &a, Walk<SHARED> &w, int R, int slots, const Ctl<SHARED> &c, int64_t left) {
  w.slot = c.start_slot, w.h = c.start_h, w.u = c.start_u, w.left = left;
  w.it = c.start;
  w.units = units_of<C, SHARED>(w.it, a.RT);
  return walk_cut<C, SHARED>(w, a.RT) || walk_next<C, SHARED>(a, w, R, slots);
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// after tcgen05.wait::ld: no use of the loaded registers moves above it
template <int N>
__device__ __forceinline__ void settled(float (&v)[N], int from, int n) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i >= from && i < from + n) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// largest of n values (n a multiple of 8), four chains
template <int N>
__device__ __forceinline__ float max_of(const float (&v)[N], int from, int n, float start) {
  float m[4] = {start, start, start, start};
#pragma unroll
  for (int i = 0; i < N; i += 8)
    if (i >= from && i < from + n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = max3(m[k], v[i + 2 * k], v[i + 2 * k + 1]);
    }
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// 4 x 4 transpose of 16-byte pieces among four neighbouring lanes: lane i's piece k becomes lane k's piece i
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4]) {
  const int lane = threadIdx.x & 31;
  auto swap = [&](uint4 &a, uint4 &b, int x) {  // with lane ^ x: the lower lane gives b, the upper one a
    const bool up = lane & x;
    uint4 give = up ? a : b, got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, x);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, x);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, x);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, x);
    if (up) a = got; else b = got;
  };
  swap(v[0], v[1], 1);
  swap(v[2], v[3], 1);
  swap(v[0], v[2], 2);
  swap(v[1], v[3], 2);
}

// Granules of a piece of n tiles in ring order.  NQ = 2: K0 V0 K1 V1 ...; NQ = 1: K0 K1 V0 K2 V1 ... V(n-1).
template <int NQ>
__device__ __forceinline__ uint32_t idx_k(uint32_t base, int j) {
  return base + (NQ == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1);
}
template <int NQ>
__device__ __forceinline__ uint32_t idx_v(uint32_t base, int j, int n) {
  return base + (NQ == 2 ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1));
}

template <int D, int NQ, bool PAIR, bool SHARED>
__global__ void __launch_bounds__(Cfg<D, NQ, PAIR>::kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TcArgs<SHARED> a) {
  using C = Cfg<D, NQ, PAIR>;
  constexpr int KT = C::KT, kSlots = C::kSlots;
  static_assert(C::kRowsK / 8 * C::kPanelsK <= 32 && KT / 8 * C::kPanelsV <= 32, "a granule has at most one box a lane");
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl<SHARED> ctl;
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *ring = sm + C::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarpTma = 4 * NQ, kWarpMma = 4 * NQ + 1, kWarpTmaV = 4 * NQ + 2, kWarps = C::kThreads / 32;
  // a share belongs to a block, or to a pair of them: then rank 1 takes every second row tile and its halves of
  // K and V, and rank 0 issues the MMAs of both, waiting on its own barriers, where both blocks arrive
  const int rank = PAIR ? (int)cluster_ctarank() : 0, unit = blockIdx.x / C::kPair, units = gridDim.x / C::kPair;
  auto leader = [&](uint64_t *bar) { return PAIR ? mapa_shared(smem_u32(bar), 0) : smem_u32(bar); };
  launch_dependents();
  // The kernel before is waited for ahead of the first access to what it may write.  Where this stands in the prologue
  // moves the compiler's schedule of the loops more than its own time: with two row tiles 1131 us after it, 1153 us
  // before it (8192 over 16384, D 128); with one 144 us and 141 us (chunks over long contexts, D 256).
  auto begin_call = [&]() {
    grid_dependency_wait();
    if (!SHARED && tid == 0 && rank == 0) a.meta[2 * unit] = make_int4(0, 0, 0, 0);
  };
  if (NQ == 1) begin_call();

  if (tid == 0) {
    ctl.abort = 0;
    if constexpr (SHARED) ctl.start.partial = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ctl.full[i], C::kPair);
      mbar_init(&ctl.empty[i], 1);
      mbar_init(&ctl.land[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.sfull[i], 1);
      mbar_init(&ctl.pready[i][0], 4 * C::kPair);  // the two halves of P apart: a warp may be done with both
      mbar_init(&ctl.pready[i][1], 4 * C::kPair);  // before another is with its first
      mbar_init(&ctl.odone[i], 1);
      mbar_init(&ctl.qfull[i], C::kPair);
      mbar_init(&ctl.qfree[i], 1);
    }
    mbar_init(&ctl.drain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpTma && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpMma) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&ctl.tmem, 512);
    } else {
      tmem_alloc(&ctl.tmem, 512);
      tmem_relinquish();
    }
  }
  auto free_tmem = [&](uint32_t t) {
    if constexpr (PAIR) tmem_dealloc_pair(t, 512);
    else tmem_dealloc(t, 512);
  };
  // every thread of the block, or of the pair
  auto sync_all = [&]() {
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
  };

  if (NQ == 2) begin_call();

  // ---- this block's share: the units of all slots summed, then the slot its first unit lies in.  The lengths and
  // offsets go through shared memory (where the ring will be), so that the search in them does not wait on L2.
  const int R = a.RT * C::kTiles;
  int slots;
  if constexpr (SHARED) slots = (int)shared_slots(a.seqs.n_tok, a.seqs.n_seqs, a.seqs.n_groups, a.G, R);
  else slots = (int)item_slots(a.seqs.n_tok, a.seqs.n_seqs, a.G, R);
  SeqsOf<SHARED> sq = a.seqs;
  if (a.seqs.n_seqs < C::kSlots * C::kGran / (SHARED ? 16 : 8) - 1) {
    int32_t *len_s = reinterpret_cast<int32_t *>(ring), *cu_s = len_s + a.seqs.n_seqs;
    for (int s = tid; s <= a.seqs.n_seqs; s += C::kThreads) {
      if (s < a.seqs.n_seqs) len_s[s] = a.seqs.seq_lens[s];
      if (a.seqs.cu) cu_s[s] = a.seqs.cu[s];
    }
    sq.seq_lens = len_s;
    if (a.seqs.cu) sq.cu = cu_s;
    if constexpr (SHARED)
      if (a.seqs.n_groups <= a.seqs.n_seqs) {
        int32_t *groups_s = cu_s + a.seqs.n_seqs + 1, *prefix_s = groups_s + a.seqs.n_groups + 1;
        for (int g = tid; g <= a.seqs.n_groups; g += C::kThreads) {
          groups_s[g] = a.seqs.groups[g];
          if (g < a.seqs.n_groups) prefix_s[g] = a.seqs.prefix[g];
        }
        sq.groups = groups_s, sq.prefix = prefix_s;
      }
    __syncthreads();
  }
  // Slots in rounds of a thread each: inclusive sums of their units, the rounds before them added.  One round (the usual case)
  // gives the total and the start at once; with more, a first pass finds the total.
  int64_t x = 0, cost = 0, before = 0, total = 0;
  ItemOf<SHARED> it;
  auto round = [&](int base) {  // this thread's slot: units, and units up to it in the round; returns the round's
    const int s = base + tid;
    cost = 0;
    if (s < slots) {
      if constexpr (SHARED) {
        it = shared_item_at(sq, s, a.G, R, KT);
        // positions that the first token of the sequence sees end within the prefix
        if (it.own && it.rows > 0 && it.first + 1 < group_span(sq, it.g).prefix) ctl.start.partial = 1;
      } else {
        it = item_at(sq, s, a.G, R, KT, a.window);
      }
      if (!it.ok && blockIdx.x == 0) set_status(a.status, GDN_ERR_BOUNDS);
      cost = (int64_t)units_of<C, SHARED>(it, a.RT) * a.Hkv;
    }
    x = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    __syncthreads();
    if (lane == 31) ctl.sum[warp] = x;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) x += ctl.sum[i];
      all += ctl.sum[i];
    }
    return all;
  };
  if (SHARED) __syncthreads();  // ctl.start.partial
  for (int base = 0; base < slots; base += C::kThreads) {
    const int64_t all = round(base);
    if constexpr (SHARED)
      if (blockIdx.x == 0 && base + tid < slots) a.from[base + tid] = total + x - cost;
    total += all;
  }
  if constexpr (SHARED)
    if (blockIdx.x == 0 && tid == 0) a.from[slots] = total;
  const int shares = (int)min((int64_t)units, total);  // of at least a unit, to the first blocks
  const int64_t begin = share_begin(total, min(unit, shares), max(shares, 1));
  const int64_t end = share_begin(total, min(unit + 1, shares), max(shares, 1));
  if (begin >= end) {  // both blocks of a pair
    sync_all();
    if (warp == kWarpMma) free_tmem(ctl.tmem);
    return;
  }
  for (int base = 0; base < slots; base += C::kThreads) {
    const int64_t all = slots <= C::kThreads ? total : round(base);
    const int64_t from = before + x - cost;  // units before this slot
    if (cost > 0 && begin >= from && begin < from + cost) {
      const uint32_t its = units_of<C, SHARED>(it, a.RT), into = (uint32_t)(begin - from);  // below units * Hkv
      ctl.start_slot = base + tid;
      static_cast<ItemOf<SHARED> &>(ctl.start) = it;
      ctl.start_h = into / its;
      ctl.start_u = into % its;
    }
    before += all;
    if (before > begin) break;
  }

  tc_fence_before();
  fence_proxy_async_smem();  // the lengths' reads of the ring end before copies into it
  sync_all();
  tc_fence_after();
  const uint32_t tm = ctl.tmem;
  volatile int *abort_flag = &ctl.abort;
  auto fail = [&]() {
    *abort_flag = 1;
    if (PAIR) store_cluster(mapa_shared(smem_u32(const_cast<int *>(&ctl.abort)), rank ^ 1), 1);
    set_status(a.status, GDN_ERR_TIMEOUT);
  };
  uint32_t landed = 0;  // PAIR: phase bits of the land barriers, as this warp has used them
  uint32_t issued = 0, phase = 0;  // ring slots that this warp's copies went to, and their phases at the last of them
  uint32_t q_issued[2] = {0, 0};
  Walk<SHARED> w;
  bool more = false;

  if (warp == kWarpTma || warp == kWarpTmaV) {
    // ================================================= Q tiles and K granules, V granules: page by page.  Two warps: with
    // pages of 16 a granule is 16 copies, and one warp issuing K and V falls behind HBM
    const bool for_v = warp == kWarpTmaV;
    if (NQ == 2) set_regs_down<104>();
    more = walk_begin<C, SHARED>(a, w, R, slots, ctl, end - begin);
    uint32_t base = 0;
    bool ok = true;
    const uint32_t box_bytes = (uint32_t)a.box * 128u;
    // Pages ahead of their use: lane l holds the page of box 32 win + l, and of box 32 (win + 1) + l, where the box holds
    // a position that a row sees.  The next window's entries are asked for when this one is entered (an entry asked for
    // when it is needed costs its L2 latency, 570 cycles a granule).
    int win = 0, page[2];
    bool used[2];
    auto look_up = [&](int window, int i, const int32_t *row) {
      const int64_t pos = (int64_t)(32 * window + lane) * a.box;
      used[i] = pos < w.it.hi && pos + a.box > w.it.lo;  // then pos lies within the table's row
      page[i] = used[i] ? row[(int)pos / a.page_size] : -1;
    };
    // a granule of K or V: its boxes (rows x 64-column panels) over the lanes, all in one instruction
    auto load = [&](auto is_v, uint32_t idx, int pos0, const int32_t *row) {
      constexpr bool V = decltype(is_v)::value;
      constexpr int kPanels = V ? C::kPanelsV : C::kPanelsK, kPanel = V ? C::kPanelV : C::kPanelK;
      const CUtensorMap *map = V ? &tm_v : &tm_k;
      const uint32_t slot = idx % kSlots, ph = (idx / kSlots) & 1;
      // nb divides 32: a granule lies in one window
      const int nb = (V ? KT : C::kRowsK) >> a.box_log2, b0 = (pos0 + (V ? 0 : rank * C::kRowsK)) >> a.box_log2;
      if (b0 >> 5 > win) {
        ++win;
        page[0] = page[1], used[0] = used[1];
        look_up(win + 1, 1, row);
      }
      const int i = lane / kPanels, p = lane % kPanels, from = (b0 + i) & 31;
      int pg = page[0];
      if (used[0] && (pg < 0 || pg >= a.n_pages)) set_status(a.status, GDN_ERR_BOUNDS), pg = -1;
      pg = __shfl_sync(0xffffffffu, pg, from);
      if (i >= nb) pg = -1;
      const int at = (b0 + i) * a.box, sl = a.page_mask >= 0 ? at & a.page_mask : at % a.page_size;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, pg >= 0)) * box_bytes;
      if (!warp_wait(&ctl.empty[slot], ph ^ 1, abort_flag)) {
        ok = false;
        return;
      }
      uint8_t *to = ring + slot * C::kGran + p * kPanel + i * box_bytes;
      if constexpr (PAIR) {
        // V rows that become zeros: the copy reports to this block, whose softmax holds the product back
        const bool here = V && (pos0 < w.it.lo || pos0 + KT > w.it.hi);
        const uint32_t bar = here ? smem_u32(&ctl.land[slot]) : leader(&ctl.full[slot]);
        if (lane == 0) {
          if (here) {
            mbar_arrive_expect_tx(&ctl.land[slot], bytes);
            arrive_cluster(leader(&ctl.full[slot]));
          } else {
            arrive_expect_cluster(bar, bytes);
          }
        }
        if (here) landed = (landed ^ (landed >> (16 + slot) & 1) << slot) | 1u << (16 + slot);
        __syncwarp();
        if (pg >= 0) tma_load_4d_pair(to, map, bar, 64 * (p + (V ? rank * kPanels : 0)), sl, w.h, pg);
      } else {
        if (lane == 0) mbar_arrive_expect_tx(&ctl.full[slot], bytes);
        __syncwarp();
        if (pg >= 0) tma_load_4d(to, map, &ctl.full[slot], 64 * p, sl, w.h, pg);
      }
      issued |= 1u << slot, phase = (phase & ~(1u << slot)) | ph << slot;
    };
    while (more && ok) {
      if (w.it.n_tiles > 0) {
        const int32_t *row = a.table + (int64_t)w.it.s * a.table_stride;
        const int first = (w.it.tile0 + w.j) * KT;
        win = first >> a.box_log2 >> 5;
        look_up(win, 0, row);
        look_up(win + 1, 1, row);
        // the row tiles' queries: whole tokens with the heads of the group, a box each 64 columns; rows of other
        // sequences that come along are never used
        const int nt = NQ == 2 && w.it.rows > a.RT * C::kPair ? 2 : 1;
        for (int t = 0; t < nt && ok && !for_v; ++t) {
          if (!warp_wait(&ctl.qfree[t], (q_issued[t] & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const int tok = w.it.t0 + w.it.row0 / a.G + (t * C::kPair + rank) * (a.RT / a.G);
            if constexpr (PAIR) arrive_expect_cluster(leader(&ctl.qfull[t]), a.RT * D * 2);
            else mbar_arrive_expect_tx(&ctl.qfull[t], a.RT * D * 2);
            for (int p = 0; p < D / 64; ++p) {
              uint8_t *to = sm + t * 128 * D * 2 + p * 16384;
              if constexpr (PAIR) tma_load_3d_pair(to, &tm_q, leader(&ctl.qfull[t]), 64 * p, w.h * a.G, tok);
              else tma_load_3d(to, &tm_q, &ctl.qfull[t], 64 * p, w.h * a.G, tok);
            }
          }
          __syncwarp();
          ++q_issued[t];
        }
        for (int j = 0; j < w.n && ok; ++j) {
          if (for_v) load(std::true_type{}, idx_v<NQ>(base, j, w.n), first + j * KT, row);
          else load(std::false_type{}, idx_k<NQ>(base, j), first + j * KT, row);
        }
        base += 2 * w.n;
      }
      more = walk_next<C, SHARED>(a, w, R, slots);
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kWarpMma) {
    // ================================================= MMAs
    if (NQ == 2) set_regs_down<104>();
    if (lane == 0 && rank == 0) {
      more = walk_begin<C, SHARED>(a, w, R, slots, ctl, end - begin);
      const uint32_t id_s = idesc_bf16(128 * C::kPair, KT, false, false);
      const uint32_t id_o = idesc_bf16(128 * C::kPair, D, false, true);
      const uint64_t d_q = smem_desc(smem_u32(sm), 16, 1024, 2);
      const uint64_t d_k = smem_desc(smem_u32(ring), 16, 1024, 2);
      const uint64_t d_v = smem_desc(smem_u32(ring), C::kPanelV, 1024, 2);
      uint32_t base = 0, pieces[2] = {0, 0}, steps[2] = {0, 0};  // steps: P tiles consumed, per TMEM slot
      uint32_t total_steps = 0;                                  // NQ = 1: the S slots alternate across pieces
      bool ok = !a.no_wait;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!ok) return;
        ok = mbar_wait_spin(bar, parity, kSpin, abort_flag);
      };
      auto wait_full = [&](uint32_t idx) { wait(&ctl.full[idx % kSlots], (idx / kSlots) & 1); };
      // S[slot] = Q[t] K(j)^T
      auto issue_s = [&](int t, int slot, int j) {
        const uint32_t idx = idx_k<NQ>(base, j);
        if (t == 0) wait_full(idx);  // the second row tile reads the same K
        if (!ok) return;
        tc_fence_after();
        const uint64_t dk = d_k + (((idx % kSlots) * C::kGran) >> 4);
        const uint64_t dq = d_q + ((t * 128 * D * 2) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss<PAIR>(tm + slot * KT, dq + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                       dk + (((ks >> 2) * C::kPanelK + (ks & 3) * 32) >> 4), id_s, ks > 0);
        commit<PAIR>(&ctl.sfull[slot]);
        if (NQ == 1) commit<PAIR>(&ctl.empty[idx % kSlots]);
      };
      // O[t] (+)= P[slot] V(j).  With one row tile the first half of the positions goes as soon as their P is there; with two the
      // other tile's products cover the wait, and each wait costs this thread some 90 cycles
      auto issue_o = [&](int t, int slot, int j) {
        const uint32_t idx = idx_v<NQ>(base, j, w.n);
        const uint64_t dv = d_v + (((idx % kSlots) * C::kGran) >> 4);
#pragma unroll
        for (int half = 0; half < C::kHalves; ++half) {
          wait(&ctl.pready[slot][half], steps[slot] & 1);
          if (t == 0 && half == 0) wait_full(idx);
          if (!ok) return;
          tc_fence_after();
          constexpr int kSteps = KT / 16 / C::kHalves;
#pragma unroll
          for (int ks = half * kSteps; ks < (half + 1) * kSteps; ++ks)
            mma_ts<PAIR>(tm + C::kO + t * D, tm + slot * KT + ks * 8, dv + ((ks * 2048) >> 4), id_o, j > 0 || ks > 0);
        }
        ++steps[slot];
        if (NQ == 1) commit<PAIR>(&ctl.empty[idx % kSlots]);
      };
      while (more && ok) {
        const int n = w.it.n_tiles > 0 ? w.n : 0;
        if (n > 0) {
          const int nt = NQ == 2 && w.it.rows > a.RT * C::kPair ? 2 : 1;
          for (int t = 0; t < nt && ok; ++t) wait(&ctl.qfull[t], pieces[t]++ & 1);
          if (!ok) break;
          tc_fence_after();
          if (NQ == 2) {
            for (int t = 0; t < nt && ok; ++t) issue_s(t, t, 0);
            for (int j = 0; j < n && ok; ++j)
              for (int t = 0; t < nt && ok; ++t) {
                issue_o(t, t, j);
                if (!ok) break;
                if (j + 1 < n) issue_s(t, t, j + 1);
                else commit<PAIR>(&ctl.odone[t]);
              }
          } else {
            issue_s(0, total_steps & 1, 0);
            for (int j = 0; j < n && ok; ++j, ++total_steps) {
              if (j + 1 < n) issue_s(0, (total_steps + 1) & 1, j + 1);
              if (ok) issue_o(0, total_steps & 1, j);
            }
          }
          base += 2 * n;
        }
        more = walk_next<C, SHARED>(a, w, R, slots);
      }
      if (!ok || *abort_flag) {  // MMAs in flight end before the block's memory goes
        if (!ok) fail();
        commit<PAIR>(&ctl.drain);
        mbar_wait(&ctl.drain, 0, kSpin);
      }
    }
  } else if (warp > kWarpTmaV) {
    if (NQ == 2) set_regs_down<104>();
  } else {
    // ================================================= softmax: a thread owns a query row
    if (NQ == 2) set_regs_up<200>();
    more = walk_begin<C, SHARED>(a, w, R, slots, ctl, end - begin);
    const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lq = (uint32_t)(quarter * 32) << 16;
    auto p_ready = [&](int slot, int half) {
      if constexpr (PAIR) arrive_cluster(leader(&ctl.pready[slot][half]));
      else mbar_arrive(&ctl.pready[slot][half]);
    };
    const float lag = kLag / a.c;
    const uint64_t c2 = f2_pack(a.c, a.c);
    uint32_t base = 0, steps = 0, sphase[2] = {0, 0}, pieces = 0;
    bool ok = true;
    while (more && ok) {
      const ItemOf<SHARED> &it = w.it;
      const int tile = t * C::kPair + rank, rr = tile * a.RT + r;
      const bool valid = r < a.RT && rr < it.rows;
      // this thread's row of o, worked out where it is needed: the loop's registers are few
      auto out_row = [&]() {
        const int row = it.row0 + rr, i = row / a.G, g = row - i * a.G;
        return (int64_t)(it.t0 + i) * (a.G * a.Hkv) + w.h * a.G + g;
      };
      if (!SHARED && it.n_tiles == 0) {  // rows that see nothing
        if (valid) {
          const int64_t out = out_row();
          for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4 *>(a.o + out * D + d) = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[out] = -INFINITY;
        }
        more = walk_next<C, SHARED>(a, w, R, slots);
        continue;
      }
      const int n = w.n, nt = NQ == 2 && it.rows > a.RT * C::kPair ? 2 : 1;
      const bool begins = w.j == 0, ends = w.j + w.n == it.n_tiles;
      const int first = (it.tile0 + w.j) * KT;
      if (t < nt) {
        const bool live = tile * a.RT + quarter * 32 < it.rows && quarter * 32 < a.RT;  // this warp has a row
        const int p = it.first + (it.row0 + rr) / a.G;
        int hi = valid ? max(p + 1, 0) : 0, lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
        if constexpr (SHARED) {
          lo = it.lo;
          if (!it.own && valid) hi = ctl.start.partial ? row_end(a.seqs, it, it.row0 + rr, a.G) : it.hi;
        }
        float m = -INFINITY, l = 0.f;
        const bool releases = t == nt - 1;  // this warpgroup gives ring slots back
        for (int j = 0; j < n; ++j, ++steps) {
          const int slot = NQ == 2 ? t : steps & 1;
          if (!warp_wait(&ctl.sfull[slot], sphase[slot] & 1, abort_flag)) {
            ok = false;
            break;
          }
          ++sphase[slot];
          tc_fence_after();
          // S is there: K(j) has been read, and V(j - 1), whose product came before it (NQ = 1: the MMAs' own commits
          // give the slots back, K(j) well before this warpgroup comes to S)
          if (tid == t * 128) {
            if (NQ == 2 && releases) {
              mbar_arrive(&ctl.empty[idx_k<NQ>(base, j) % kSlots]);
              if (j > 0) mbar_arrive(&ctl.empty[idx_v<NQ>(base, j - 1, n) % kSlots]);
            }
            if (j == n - 1) mbar_arrive(&ctl.qfree[t]);
          }
          const int pos = first + j * KT;
          if (t == 0 && (pos < it.lo || pos + KT > it.hi)) {
            // positions that no row sees: their V rows become zeros (P is 0 there, and 0 * NaN is not)
            const uint32_t idx = idx_v<NQ>(base, j, n);
            uint64_t *there = PAIR ? &ctl.land[idx % kSlots] : &ctl.full[idx % kSlots];
            if (!warp_wait(there, PAIR ? landed >> (idx % kSlots) & 1 : (idx / kSlots) & 1, abort_flag)) {
              ok = false;
              break;
            }
            landed ^= 1u << (idx % kSlots);
            const int z0 = max(it.lo - pos, 0), z1 = min(it.hi - pos, KT);  // rows [0, z0) and [z1, KT)
            uint8_t *v = ring + (idx % kSlots) * C::kGran;
            for (int pn = 0; pn < C::kPanelsV; ++pn, v += C::kPanelV) {
              for (int x = r * 16; x < z0 * 128; x += 128 * 16) *reinterpret_cast<uint4 *>(v + x) = make_uint4(0, 0, 0, 0);
              for (int x = z1 * 128 + r * 16; x < KT * 128; x += 128 * 16)
                *reinterpret_cast<uint4 *>(v + x) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            if (PAIR) asm volatile("fence.acq_rel.cluster;" ::: "memory");
          }
          if (live) {
            const uint32_t ts = tm + lq + slot * KT;
            float s[KT];
#pragma unroll
            for (int x = 0; x < KT; x += 32) tmem_ld32u(ts + x, reinterpret_cast<uint32_t *>(s) + x);
            tmem_wait_ld();
            settled(s, 0, KT);
            if (valid && pos + KT > hi) {  // rows past the item's are nobody's: no care for them
              const int to = hi - pos;
#pragma unroll
              for (int x = 0; x < KT; ++x) s[x] = x < to ? s[x] : -INFINITY;
            }
            if (valid && pos < lo) {
              const int from = lo - pos;
#pragma unroll
              for (int x = 0; x < KT; ++x) s[x] = x >= from ? s[x] : -INFINITY;
            }
            const float mx = max_of(s, 0, KT, -INFINITY);
            if (j == 0) {
              m = mx;
            } else if (__any_sync(0xffffffffu, valid && mx > m + lag)) {
              // the products so far end before O is scaled
              if (NQ == 1) {
                const uint32_t idx = idx_v<NQ>(base, j - 1, n);
                ok = ok && warp_wait(&ctl.empty[idx % kSlots], (idx / kSlots) & 1, abort_flag);
                tc_fence_after();
              }
              const float top = mx > m + lag ? mx : m;
              const float f = m == top ? 1.f : m == -INFINITY ? 0.f : ex2((m - top) * a.c);
              m = top;
              l *= f;
#pragma unroll 1
              for (int x = 0; x < D; x += 32) {
                uint32_t u[32];
                tmem_ld32u(tm + lq + C::kO + t * D + x, u);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                  asm volatile("" : "+r"(u[y]));
                  u[y] = __float_as_uint(__uint_as_float(u[y]) * f);
                }
                tmem_st32u(tm + lq + C::kO + t * D + x, u);
              }
            }
            const float mc = m == -INFINITY ? 0.f : m * a.c;
            const uint64_t mc2 = f2_pack(-mc, -mc);
            uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t pk[KT / 4];
#pragma unroll
              for (int y = 0; y < KT / 2; y += 4) {
                const float *v = s + half * (KT / 2) + y;
                float p0, p1, p2, p3;
                f2_unpack(f2_fma(f2_pack(v[0], v[1]), c2, mc2), p0, p1);
                f2_unpack(f2_fma(f2_pack(v[2], v[3]), c2, mc2), p2, p3);
                p0 = ex2(p0), p1 = ex2(p1), p2 = ex2(p2), p3 = ex2(p3);
                sum0 = f2_add(sum0, f2_pack(p0, p1));
                sum1 = f2_add(sum1, f2_pack(p2, p3));
                pk[y >> 1] = bf16x2(p0, p1);
                pk[(y >> 1) + 1] = bf16x2(p2, p3);
              }
              if constexpr (KT == 128) tmem_st32u(ts + half * 32, pk);
              else tmem_st16u(ts + half * 16, pk);
              if (half + 1 < 2 && C::kHalves == 1) continue;
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) p_ready(slot, C::kHalves == 1 ? 0 : half);
            }
            float s0, s1, s2, s3;
            f2_unpack(sum0, s0, s1);
            f2_unpack(sum1, s2, s3);
            l += (s0 + s1) + (s2 + s3);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              p_ready(slot, 0);
              if (C::kHalves == 2) p_ready(slot, 1);
            }
          }
        }
        // ---- the last product done: O / l, or the piece for the join
        if (ok) {
          if (NQ == 2) {
            ok = warp_wait(&ctl.odone[t], pieces & 1, abort_flag);
            if (releases && tid == t * 128) mbar_arrive(&ctl.empty[idx_v<NQ>(base, n - 1, n) % kSlots]);
          } else {
            const uint32_t idx = idx_v<NQ>(base, n - 1, n);
            ok = warp_wait(&ctl.empty[idx % kSlots], (idx / kSlots) & 1, abort_flag);
          }
          tc_fence_after();
        }
        if (ok && live) {
          const int64_t out = out_row();
          const uint32_t to = tm + lq + C::kO + t * D;
          if (begins && ends) {
            if constexpr (SHARED) {
              const int64_t blocks = ((int64_t)a.seqs.n_tok * a.G + 31) / 32, gr = (int64_t)it.t0 * a.G + it.row0 + rr;
              const int64_t at = ((own_part(it) ? a.Hkv : 0) + w.h) * blocks + gr / 32;
              uint4 *pp = reinterpret_cast<uint4 *>(a.full) + at * (D / 4 * 32) + gr % 32;
#pragma unroll 2
              for (int x = 0; x < D; x += 32) {
                uint32_t u[32];
                tmem_ld32u(to + x, u);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) asm volatile("" : "+r"(u[y]));
                if (valid)
#pragma unroll
                  for (int y = 0; y < 32; y += 4)
                    pp[(x + y) / 4 * 32] = make_uint4(u[y], u[y + 1], u[y + 2], u[y + 3]);
              }
              if (valid) *reinterpret_cast<float2 *>(a.full_ml + (at * 32 + gr % 32) * 2) = make_float2(m * a.c, l);
            } else {
              const float inv = l == 0.f ? 0.f : 1.f / l;
              // rows of this lane's quad, -1: none
              int64_t rows4[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) rows4[k] = __shfl_sync(0xffffffffu, valid ? out : -1, (lane & ~3) + k);
#pragma unroll 2
              for (int x = 0; x < D; x += 32) {
                uint32_t u[32];
                tmem_ld32u(to + x, u);
                tmem_wait_ld();
                uint4 v[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  uint32_t *vv = reinterpret_cast<uint32_t *>(&v[y]);
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    asm volatile("" : "+r"(u[8 * y + 2 * z]), "+r"(u[8 * y + 2 * z + 1]));
                    vv[z] = bf16x2(__uint_as_float(u[8 * y + 2 * z]) * inv, __uint_as_float(u[8 * y + 2 * z + 1]) * inv);
                  }
                }
                quad_transpose(v);  // now piece k is of row k of the quad, columns 8 (lane % 4) ..
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (rows4[k] >= 0) *reinterpret_cast<uint4 *>(a.o + rows4[k] * D + x + (lane & 3) * 8) = v[k];
              }
              if (valid && a.lse) a.lse[out] = l == 0.f ? -INFINITY : fmaf(m, a.c, log2f(l)) * 0.69314718055994530942f;
            }
          } else {
            // the piece as [column / 4][row] fours, so that neighbouring rows lie side by side
            const int64_t which = 2 * unit + (begins ? 1 : 0);
            uint4 *pp = reinterpret_cast<uint4 *>(a.part) + which * (C::R * D / 4) + tile * 128 + r;
#pragma unroll 2
            for (int x = 0; x < D; x += 32) {
              uint32_t u[32];
              tmem_ld32u(to + x, u);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) asm volatile("" : "+r"(u[y]));
              if (valid)
#pragma unroll
                for (int y = 0; y < 32; y += 4)
                  pp[(x + y) / 4 * C::R] = make_uint4(u[y], u[y + 1], u[y + 2], u[y + 3]);
            }
            if (valid)
              *reinterpret_cast<float2 *>(a.part_ml + (which * C::R + tile * 128 + r) * 2) = make_float2(m * a.c, l);
          }
        }
        tc_fence_before();
        ++pieces;
      }
      base += 2 * n;
      if (!SHARED && tid == 0 && rank == 0) {
        int4 *me = a.meta + 2 * unit;
        if (!begins) {
          me->x = ends ? 2 : 1;
        } else if (!ends) {
          me->y = 1, me->z = w.h, me->w = it.rows;
          me[1] = make_int4(it.t0, it.row0, 0, 0);
        }
      }
      more = walk_next<C, SHARED>(a, w, R, slots);
    }
    if (!ok && lane == 0) fail();
  }
  __syncwarp();
  tc_fence_before();
  sync_all();
  if (*abort_flag) {  // a wait gave up: copies in flight land before the memory they go to does
    if (warp == kWarpTma || warp == kWarpTmaV) {
      for (int i = 0; i < kSlots && rank == 0; ++i)
        if (issued >> i & 1) mbar_wait(&ctl.full[i], phase >> i & 1, kSpin);
      for (int t = 0; t < NQ && rank == 0; ++t)
        if (q_issued[t] > 0) mbar_wait(&ctl.qfull[t], (q_issued[t] - 1) & 1, kSpin);
      for (int i = 0; i < kSlots && PAIR; ++i)
        if (landed >> (16 + i) & 1) mbar_wait(&ctl.land[i], landed >> i & 1, kSpin);
    }
  }
  if (PAIR || *abort_flag) sync_all();
  if (warp == kWarpMma) free_tmem(tm);
}

// Items that lie in several blocks' shares: block b's last piece begins one, b + 1's first
// continues it, until a first piece ends it.  A block takes 32 rows, a lane a row.  The pieces'
// maxima and sums are loaded at once, the warps taking turns; then a warp sums an eighth of the
// columns over the pieces, and the rows go out through shared memory, whole rows at a time.
template <int D, int NQ, bool PAIR>
__global__ void __launch_bounds__(256) paged_join_kernel(const TcArgs<false> a, int blocks) {
  constexpr int R = Cfg<D, NQ, PAIR>::R, kV = D / 32;  // fours of columns a warp
  __shared__ uint2 rows[32][D / 4 + 1];
  __shared__ float weight[kSms][32], part[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  const int4 me = a.meta[2 * blockIdx.x], me_at = a.meta[2 * blockIdx.x + 1];
  int n = 0;  // pieces after the first
  for (int base = blockIdx.x + 1;; base += 32) {
    const int b = base + lane;
    const int how = b < blocks ? a.meta[2 * b].x : 0;
    const uint32_t stop = __ballot_sync(0xffffffffu, how != 1);
    if (stop) {
      n += __ffs(stop);
      if (__shfl_sync(0xffffffffu, how, __ffs(stop) - 1) != 2) return;  // no item of this block's, or a share that gave up
      break;
    }
    n += 32;
  }
  if (!me.y) return;
  const int item_rows = me.w, lr = blockIdx.y * 32 + lane, t = lr / 128, rr = t * a.RT + lr % 128;  // lane row, row of the item
  const bool valid = lr % 128 < a.RT && rr < item_rows;
  if (!__any_sync(0xffffffffu, valid)) return;  // the same for all warps
  // piece i is slot 2 b + 1 of block b for the first, 2 (b + i) for the others
  auto at = [&](int i) { return 2 * ((int64_t)blockIdx.x + i) + (i == 0); };
  auto ml_of = [&](int i) {
    return valid && i <= n ? *reinterpret_cast<const float2 *>(a.part_ml + (at(i) * R + lr) * 2)
                           : make_float2(-INFINITY, 0.f);
  };
  constexpr int kAhead = 16 / kV;  // pieces in flight
  float4 v[kAhead][kV];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float4 *p = reinterpret_cast<const float4 *>(a.part) + at(i0 + i) * (R * D / 4) + (warp * kV) * R + lr;
#pragma unroll
      for (int e = 0; e < kV; ++e) v[i][e] = i0 + i <= n && valid ? p[e * R] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(0);
  float top = -INFINITY;
#pragma unroll 4
  for (int i = warp; i <= n; i += 8) top = fmaxf(top, ml_of(i).x);
  part[0][warp][lane] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, part[0][i][lane]);
  float sum = 0.f;
#pragma unroll 4
  for (int i = warp; i <= n; i += 8) {
    const float2 ml = ml_of(i);
    const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
    sum = fmaf(f, ml.y, sum);
    weight[i][lane] = f;
  }
  part[1][warp][lane] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += part[1][i][lane];
  float4 x[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 <= n; i0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float f = i0 + i <= n ? weight[i0 + i][lane] : 0.f;
      if (f != 0.f)
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          x[e].x = fmaf(f, v[i][e].x, x[e].x);
          x[e].y = fmaf(f, v[i][e].y, x[e].y);
          x[e].z = fmaf(f, v[i][e].z, x[e].z);
          x[e].w = fmaf(f, v[i][e].w, x[e].w);
        }
    }
    if (i0 + kAhead <= n) load(i0 + kAhead);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < kV; ++e)
    rows[lane][warp * kV + e] = make_uint2(bf16x2(x[e].x * inv, x[e].y * inv), bf16x2(x[e].z * inv, x[e].w * inv));
  const int row = me_at.y + rr, i = row / a.G, g = row - i * a.G;
  const int64_t out = valid ? (int64_t)(me_at.x + i) * (a.G * a.Hkv) + me.z * a.G + g : -1;
  if (valid && warp == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
  __syncthreads();
  for (int q = warp; q < 32; q += 8) {
    const int64_t to = __shfl_sync(0xffffffffu, out, q);
    if (to >= 0)
      for (int c = lane; c < D / 4; c += 32) *reinterpret_cast<uint2 *>(a.o + to * D + 4 * c) = rows[q][c];
  }
}

// [page][head][slot][D] of a cache, boxes of 64 columns x `box` slots
bool make_map(CUtensorMap *m, const void *base, const gdn_cache_shape &s, int box) {
  auto enc = encode_fn();
  if (!enc) return false;
  const int64_t heads = s.Hkv > 1 ? s.head_stride : s.D, pages = s.n_pages > 1 ? s.page_stride : s.slot_stride;
  cuuint64_t dims[4] = {(cuuint64_t)s.D, (cuuint64_t)s.page_size, (cuuint64_t)s.Hkv, (cuuint64_t)s.n_pages};
  cuuint64_t strides[3] = {(cuuint64_t)s.slot_stride * 2, (cuuint64_t)heads * 2, (cuuint64_t)pages * 2};
  cuuint32_t b[4] = {64, (cuuint32_t)box, 1, 1}, es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [token][head][D] of q, boxes of 64 columns x the G heads of a group x as many tokens as fill RT rows
bool make_q_map(CUtensorMap *m, const void *base, const gdn_cache_shape &s, int G, int RT) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)s.D, (cuuint64_t)s.Hq, (cuuint64_t)s.n_tok};
  cuuint64_t strides[2] = {(cuuint64_t)s.D * 2, (cuuint64_t)s.q_stride * 2};
  cuuint32_t b[3] = {64, (cuuint32_t)G, (cuuint32_t)(RT / G)}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel and the one that joins its pieces.
template <int D, int NQ, bool PAIR, bool SHARED>
gdn_status launch_two(const void *k, const void *v, const gdn_cache_shape &s, TcArgs<SHARED> &a, cudaStream_t st,
                      dim3 join_grid, void (*join)(TcArgs<SHARED>, int)) {
  using C = Cfg<D, NQ, PAIR>;
  a.box = std::gcd(s.page_size, C::kRowsK);  // a power of two
  a.box_log2 = __builtin_ctz(a.box);
  CUtensorMap mq, mk, mv;
  if (!make_q_map(&mq, a.q, s, a.G, a.RT) || !make_map(&mk, k, s, a.box) || !make_map(&mv, v, s, a.box))
    return GDN_ERR_CUDA;
  constexpr int smem = kData + 1024;
  const auto kernel = paged_attn_kernel<D, NQ, PAIR, SHARED>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return (void)cudaGetLastError(), GDN_ERR_CUDA;
  // both kernels start up under the last blocks of the one before them and wait for its end
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kSms);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, (const TcArgs<SHARED>)a) != cudaSuccess)
    return (void)cudaGetLastError(), GDN_ERR_CUDA;
  cfg.gridDim = join_grid;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join, (TcArgs<SHARED>)a, kSms / C::kPair) != cudaSuccess)
    return (void)cudaGetLastError(), GDN_ERR_CUDA;
  return launch_status();
}

// What the kernel's forms have in common of a call.
template <bool SHARED>
TcArgs<SHARED> tc_args(const void *q, const int32_t *table, const SeqsOf<SHARED> &seqs, const gdn_cache_shape &s,
                       float scale_log2, int32_t window, uint32_t flags, void *o, float *lse, void *workspace) {
  TcArgs<SHARED> a{};
  a.seqs = seqs;
  a.q = (const __nv_bfloat16 *)q, a.o = (__nv_bfloat16 *)o, a.lse = lse;
  a.table = table, a.table_stride = s.table_stride, a.q_stride = s.q_stride;
  a.G = s.Hq / s.Hkv, a.Hkv = s.Hkv;
  a.RT = 128 / a.G * a.G;
  a.page_size = s.page_size, a.page_mask = s.page_size & (s.page_size - 1) ? -1 : s.page_size - 1;
  a.max_pages = s.max_pages, a.n_pages = s.n_pages;
  a.window = window, a.c = scale_log2;
  a.status = s.status ? s.status : (int32_t *)workspace;
  a.no_wait = flags & GDN_FLAG_TEST_NO_WAIT ? 1 : 0;
  return a;
}

// Rows of the longest chunk's kv head, and the row tiles that share K and V: one, two in a block (D <= 128: their O
// and S fill the TMEM), or (D 128 and 256) twice as many in a pair of blocks, wherever a chunk's rows need more than
// one of the smaller.  8192 over 16384, D 128: 1115 us in pairs, 1162 without; 4096 over 8192, D 256: 251 us and 394;
// 16 ragged chunks of up to 509 over up to 6000, 8 heads a group, D 256: 139 us and 200.
inline int64_t chunk_rows(const gdn_cache_shape &s, int32_t max_new) { return (int64_t)max_new * (s.Hq / s.Hkv); }
inline bool two_tiles(const gdn_cache_shape &s, int32_t max_new) { return s.D <= 128 && chunk_rows(s, max_new) > 128; }
inline bool pairs(const gdn_cache_shape &s, int32_t max_new) {
  return (s.D == 128 && chunk_rows(s, max_new) > 256) || (s.D == 256 && chunk_rows(s, max_new) > 128);
}

inline bool tc_shape(const gdn_cache_shape &s) {
  return s.dtype == GDN_BF16 && (s.D == 64 || s.D == 128 || s.D == 256) && s.page_size % 8 == 0 &&
         s.page_size <= 1 << 20 && s.n_pages > 0 && s.Hq / s.Hkv <= 128;
}

}  // namespace
}  // namespace gdn

// paged_mass_tc.cu -- gdn_paged_mass on the tensor cores (tcgen05, bf16; D = 64, 128 or 256).
//
// S^T = K Q^T: a tile of 128 positions is the product's rows and stays in shared memory, a tile of up to 256 query rows its
// columns, so a thread owns a position and adds up 2^(c S - lse) over the columns, c = scale log2 e: no weight leaves
// the registers, nothing is added between threads but the warpgroups' sums.
//
// Warps: four softmax warpgroups, two for each of two TMEM slots of 256 columns, half of them each; the slots take the
// steps (a query tile of a position tile) in turn.  A warp for K's copies (pages by their table entries), one for Q's
// (whole tokens with the heads of the group), an MMA thread, and a warp that lays out beside each slot what its
// warpgroups have to know of the step, the rows' lse among it.  K and Q each have a ring of panels of 64 columns of a tile.
//
// The 8192 tokens of a prompt, 32 / 8 heads, D 128: 277 us, 993 TFLOP/s, 52% of cuBLAS.  No
// one unit bounds it (products of 16 columns, weights without the exponential, Q copied once: each less than 10%
// faster): it is the step's hand-over of a slot and two FMAs, an exponential and an add a weight, 46% of issue slots.
// Slower: part of the exponentials by a polynomial (392 -> 417), query tiles of 128 rows (457), two softmax warpgroups of more
// registers (283 to 328), 16 columns a TMEM load (280 -> 311).  Not built: pairs of blocks, each with half of a query tile (at
// D 256 the ring holds one such tile, so the next one's copy waits for this one's products).
#include <cuda.h>

#include <algorithm>
#include <numeric>

#include "common.cuh"
#include "conv_tap.cuh"
#include "paged_attn.cuh"
#include "paged_mass.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kSms = 152;            // persistent blocks
constexpr uint32_t kSpin = 1u << 22; // polls of a wait before it gives up
constexpr int kData = 218 * 1024;    // the rings
constexpr int kBP = 128, kNQ = 256, kOver = 1, kGroups = 4, kThreads = 128 * kGroups + 128;

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;                  // of a tile
  static constexpr int kPanelK = kBP * 128, kPanelQ = kNQ * 128;  // bytes
  static constexpr int kSlotsQ = 4;
  static constexpr int kSlotsK = (kData - kSlotsQ * kPanelQ) / kPanelK;
};

// A step as its warpgroups see it.
struct Step {
  int64_t mass;           // where the tile's first position lies in the masses
  int pos, lo, hi;        // that position; positions that are written
  int base, n, row0;      // position of the tile's first query token; query tokens; row (of those) of the step's first column
  int cols, flags;        // columns in use
  int swap, pad[3];       // number of the exchange of sums
};
constexpr int kFirst = 1, kLast = 2;      // of the slot's steps of its piece
constexpr int kEnds = 4, kAlone = 8;      // the piece's last step; its only one
constexpr int kWhole = 16, kBegins = 32;  // the piece has all of its tile's steps; the first of them

struct Ctl {
  uint64_t kfull[8], kempty[8], qfull[4], qempty[4], sfull[2], sempty[2], lready[2], xfull[2], xempty[2], drain;
  uint32_t tmem;
  volatile int abort;
  MassStart start;
  alignas(16) Step step[2];
  alignas(16) float lse[2][kNQ];    // minus the rows' lse in base 2
  float x[2][kGroups][128];             // the warpgroups' sums for the one that ends a piece
};

static_assert(kData + 1024 + sizeof(Ctl) <= 227 * 1024, "shared memory of a block");

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// one lane of the warp, always the same
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// a wait of all lanes, the same answer for all of them
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, kSpin, abort));
}

// A ring's next slot and the parity of its use.
template <int N>
struct Ring {
  uint32_t slot = 0, turn = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) slot = 0, turn ^= 1;
  }
};

// The weights 2^(c s + nl) of 32 columns added to the sums, with a mask those of columns [from, end).
template <bool MASK>
__device__ __forceinline__ void add_weights(const float (&s)[32], const float *nl, uint64_t c2, int from, int end,
                                            uint64_t &sum0, uint64_t &sum1) {
#pragma unroll
  for (int y = 0; y < 32; y += 4) {
    const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(nl + y);
#pragma unroll
    for (int z = 0; z < 4; z += 2) {
      const uint64_t x = f2_fma(f2_pack(s[y + z], s[y + z + 1]), c2, z ? l.y : l.x);
      uint64_t &sum = z ? sum1 : sum0;
      float e0, e1;
      f2_unpack(x, e0, e1);
      e0 = ex2(e0), e1 = ex2(e1);
      if (MASK) {
        e0 = y + z >= from && y + z < end ? e0 : 0.f;
        e1 = y + z + 1 >= from && y + z + 1 < end ? e1 : 0.f;
      }
      sum = f2_add(sum, f2_pack(e0, e1));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const MassArgs a,
                         int box_log2, int no_wait) {
  using C = Cfg<D>;
  static_assert(C::kSlotsK > C::kPanels && C::kSlotsK <= 8 && kBP / 8 <= 32, "rings; a panel has at most one box a lane");
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t *ks = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *qs = ks + C::kSlotsK * C::kPanelK;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, unit = blockIdx.x;
  constexpr int kWarpK = 4 * kGroups, kWarpQ = kWarpK + 1, kWarpMma = kWarpK + 2, kWarpLse = kWarpK + 3;
  launch_dependents();
  grid_dependency_wait();
  if (tid == 0) {
    a.meta[2 * unit] = make_int4(0, 0, 0, 0);
    ctl.abort = 0;
    for (int i = 0; i < 8; ++i) mbar_init(&ctl.kfull[i], 1), mbar_init(&ctl.kempty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&ctl.qfull[i], 1), mbar_init(&ctl.qempty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl.sfull[i], 1), mbar_init(&ctl.sempty[i], 8), mbar_init(&ctl.lready[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl.xfull[i], 4 * (kGroups - 1)), mbar_init(&ctl.xempty[i], 4);
    mbar_init(&ctl.drain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpK && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  int64_t left;
  const bool some = mass_start<kBP, kOver, kThreads>(a, unit, gridDim.x, ctl.start, left);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = ctl.tmem;
  if (!some) {
    __syncthreads();
    if (warp == kWarpMma) tmem_dealloc(tm, 512);
    return;
  }
  volatile int *abort_flag = &ctl.abort;
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(a.status, GDN_ERR_TIMEOUT);
  };
  MassWalk w;
  bool more = mass_begin<kBP, kOver>(a, ctl.start, left, w), ok = true;
  uint32_t issued = 0, phase = 0;  // ring slots that this warp's copies went to, and their parities at the last of them

  if (warp == kWarpK) {
    // ================================================= K: page by page
    Ring<C::kSlotsK> ring;
    const int box = 1 << box_log2, nb = kBP >> box_log2;
    // Pages ahead of their use: lane l holds the page of box 32 win + l of the sequence, and of box 32 (win + 1) + l, kNone
    // where no position of the box is read.  The next window's entries are asked for when this one is entered.
    constexpr int kNone = INT32_MIN;
    int win = 0, page[2] = {kNone, kNone}, of_s = -1, of_h = -1;
    auto look_up = [&](int window) {
      const int64_t pos = (int64_t)(32 * window + lane) * box;
      const bool used = pos < w.m.hi && pos + box > w.m.seen;  // then the table's row holds it
      return used ? a.table[w.s * a.table_stride + (int)pos / a.page_size] : kNone;
    };
    for (; more && ok; more = mass_next<kBP, kOver>(a, w)) {
      if (w.n == 0) continue;
      const int b0 = (w.m.tile0 + w.j) * nb;  // nb divides 32: a tile lies in one window
      if (w.s != of_s || w.h != of_h || b0 >> 5 > win + 1) {
        if (w.s != of_s || b0 >> 5 != win) page[0] = look_up(b0 >> 5), page[1] = look_up((b0 >> 5) + 1);
        of_s = w.s, of_h = w.h, win = b0 >> 5;
      } else if (b0 >> 5 > win) {
        ++win;
        page[0] = page[1], page[1] = look_up(win + 1);
      }
      const int at = (b0 + lane) * box, slot = a.page_mask >= 0 ? at & a.page_mask : at % a.page_size;
      int pg = page[0];
      if (pg != kNone && (pg < 0 || pg >= a.n_pages)) set_status(a.status, GDN_ERR_BOUNDS), pg = -1;
      pg = __shfl_sync(0xffffffffu, pg, (b0 + lane) & 31);
      if (lane >= nb) pg = -1;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, pg >= 0)) * (uint32_t)box * 128u;
      for (int p = 0; p < C::kPanels && ok; ++p, ring.step()) {
        if (!warp_wait(&ctl.kempty[ring.slot], ring.turn ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&ctl.kfull[ring.slot], bytes);
        __syncwarp();
        if (pg >= 0)
          tma_load_4d(ks + ring.slot * C::kPanelK + lane * box * 128, &tm_k, &ctl.kfull[ring.slot], 64 * p, slot, w.h, pg);
        issued |= 1u << ring.slot, phase = (phase & ~(1u << ring.slot)) | ring.turn << ring.slot;
      }
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kWarpQ) {
    // ================================================= Q: whole tokens with the heads of the group, a box each 64 columns
    if (lane == 0) {
      Ring<C::kSlotsQ> ring;
      for (; more && ok; more = mass_next<kBP, kOver>(a, w)) {
        int token = w.m.sp.t0 + w.i0 + w.q0 * a.tokens;
        for (int t = 0; t < w.n && ok; ++t, token += a.tokens)
          for (int p = 0; p < C::kPanels; ++p, ring.step()) {
            ok = mbar_wait_spin(&ctl.qempty[ring.slot], ring.turn ^ 1, kSpin, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(&ctl.qfull[ring.slot], a.RQ * 128);
            tma_load_3d(qs + ring.slot * C::kPanelQ, &tm_q, &ctl.qfull[ring.slot], 64 * p, w.h * a.G, token);
            issued |= 1u << ring.slot, phase = (phase & ~(1u << ring.slot)) | ring.turn << ring.slot;
          }
      }
      if (!ok) fail();
    }
  } else if (warp == kWarpMma) {
    // ================================================= MMAs: the warp goes together, one lane issues (its operands are then
    // known to be the warp's)
    Ring<C::kSlotsK> kr;
    Ring<C::kSlotsQ> qr;
    Ring<2> buf;
    const uint64_t d_k = smem_desc(smem_u32(ks), 16, 1024, 2), d_q = smem_desc(smem_u32(qs), 16, 1024, 2);
    ok = !no_wait;
    for (; more && ok; more = mass_next<kBP, kOver>(a, w)) {
      const Ring<C::kSlotsK> k0 = kr;
      const int n = __shfl_sync(0xffffffffu, w.n, 0);
      int left_rows = __shfl_sync(0xffffffffu, (w.i1 - w.i0) * a.G - w.q0 * a.RQ, 0);
      for (int t = 0; t < n && ok; ++t, buf.step(), left_rows -= a.RQ) {
        ok = warp_wait(&ctl.sempty[buf.slot], buf.turn ^ 1, abort_flag);
        const uint32_t id = idesc_bf16(kBP, (min(a.RQ, left_rows) + 15) & ~15, false, false);
        kr = k0;
#pragma unroll 1
        for (int p = 0; p < C::kPanels && ok; ++p, kr.step(), qr.step()) {
          if (t == 0) ok = warp_wait(&ctl.kfull[kr.slot], kr.turn, abort_flag);
          ok = ok && warp_wait(&ctl.qfull[qr.slot], qr.turn, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dk = d_k + ((kr.slot * C::kPanelK) >> 4), dq = d_q + ((qr.slot * C::kPanelQ) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              umma_bf16(tm + buf.slot * kNQ, dk + (x * 32 >> 4), dq + (x * 32 >> 4), id, p > 0 || x > 0);
            umma_commit(&ctl.qempty[qr.slot]);
            if (t + 1 == n) umma_commit(&ctl.kempty[kr.slot]);
            if (p + 1 == C::kPanels) umma_commit(&ctl.sfull[buf.slot]);
          }
          __syncwarp();
        }
      }
    }
    if (!ok || *abort_flag) {  // MMAs in flight end before the block's memory goes
      if (!ok && lane == 0) fail();
      if (elect_one()) {
        umma_commit(&ctl.drain);
        mbar_wait(&ctl.drain, 0, kSpin);
      }
      __syncwarp();
    }
  } else if (warp == kWarpLse) {
    // ================================================= what the warpgroups have to know of the steps: the rows' lse, eight
    // rows a lane, the next step's on their way, and the step itself
    Ring<2> buf;
    const int i8 = 8 * lane / a.G, g8 = 8 * lane - i8 * a.G;  // token and head of a lane's first row
    float next[8];
    int t = -1, swaps = 0;
    auto advance = [&]() {  // to the next step, whose lse is asked for; false where there is none
      for (++t; more && t >= w.n; t = 0) {
        if (w.n == 0 && a.all) {  // a tile that no query sees
          float *to = a.mass + w.s * a.row_stride + w.h * a.mass_head_stride;
          const int pos = (w.m.tile0 + w.j) * kBP;
          for (int x = max(pos, w.m.lo) + lane; x < min(pos + kBP, w.m.hi); x += 32) to[x] = 0.f;
        }
        more = mass_next<kBP, kOver>(a, w);
      }
      if (!more) return false;
      const int rows = min(a.RQ, (w.i1 - w.i0) * a.G - (w.q0 + t) * a.RQ);
      const float *at = a.lse + (int64_t)(w.m.sp.t0 + w.i0 + (w.q0 + t) * a.tokens + i8) * (a.G * a.Hkv) + w.h * a.G;
#pragma unroll
      for (int k = 0, g = g8; k < 8; ++k) {
        next[k] = 8 * lane + k < rows ? at[g] : 0.f;
        if (++g == a.G) g = 0, at += a.G * a.Hkv;
      }
      return true;
    };
    for (bool there = advance(); there && ok; buf.step()) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = next[k];
      const int row0 = (w.q0 + t) * a.RQ, n = w.i1 - w.i0;
      const bool ends = t + 1 == w.n, alone = w.n == 1;
      Step st;
      st.pos = (w.m.tile0 + w.j) * kBP, st.lo = w.m.lo, st.hi = w.m.hi;
      st.mass = w.s * a.row_stride + w.h * a.mass_head_stride + st.pos;
      st.base = w.m.first + w.i0, st.n = n, st.row0 = row0, st.cols = min(a.RQ, n * a.G - row0);
      st.flags = (t < 2 ? kFirst : 0) | (t + 2 >= w.n ? kLast : 0) | (ends ? kEnds : 0) | (alone ? kAlone : 0) |
                 (mass_begins(w) && mass_ends(w) ? kWhole : 0) | (mass_begins(w) ? kBegins : 0);
      st.swap = swaps;
      if (ends && lane == 0) mass_note(a, w, unit);
      const int slot = swaps & 1;
      const uint32_t turn = swaps >> 1 & 1;
      if (ends) ++swaps;
      there = advance();
      if (!warp_wait(&ctl.sempty[buf.slot], buf.turn ^ 1, abort_flag) ||
          (alone && !warp_wait(&ctl.xempty[slot], turn ^ 1, abort_flag))) {
        ok = false;
        break;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] == -INFINITY ? v[k] : v[k] * -1.44269504088896340736f;  // -inf: weighs nothing
      float4 *to = reinterpret_cast<float4 *>(&ctl.lse[buf.slot][8 * lane]);
      to[0] = make_float4(v[0], v[1], v[2], v[3]);
      to[1] = make_float4(v[4], v[5], v[6], v[7]);
      if (lane == 0) ctl.step[buf.slot] = st;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.lready[buf.slot]);
      // for the two warpgroups of the other slot, which have no step of this piece
      if (alone && lane < 8) mbar_arrive(&ctl.xfull[slot]);
    }
    // no step is left: the warpgroups are told so
    for (int k = 0; k < 2 && ok; ++k, buf.step()) {
      ok = warp_wait(&ctl.sempty[buf.slot], buf.turn ^ 1, abort_flag);
      if (lane == 0 && ok) {
        ctl.step[buf.slot].cols = 0;
        mbar_arrive(&ctl.lready[buf.slot]);
      }
    }
    if (!ok && lane == 0) fail();
  } else {
    // ================================================= softmax: a thread owns a position
    const int group = warp >> 2, slot = group >> 1, x0 = (group & 1) * 128, p = tid & 127;
    const uint32_t ts = tm + ((uint32_t)((warp & 3) * 32) << 16) + slot * kNQ;
    const uint64_t c2 = f2_pack(a.c, a.c);
    const float *nl = ctl.lse[slot];
    uint64_t sum0 = 0, sum1 = 0;
    float old = 0.f;
    for (uint32_t turn = 0; ok; turn ^= 1) {
      ok = warp_wait(&ctl.lready[slot], turn, abort_flag);
      if (!ok) break;
      const Step &st = ctl.step[slot];
      const int cols = st.cols, flags = st.flags, pos = st.pos + p, swap = st.swap;
      if (cols == 0) break;
      const bool mine = pos >= st.lo && pos < st.hi, writes = (flags & kEnds) && x0 == 0;
      float *to = a.mass + st.mass + p;
      if (flags & kFirst) sum0 = sum1 = f2_pack(0.f, 0.f);
      if (writes && (flags & kWhole) && mine && !a.all) old = *to;
      // columns [from, end) see the position
      const int d = pos - st.base, rows = a.window > 0 ? (int)min((int64_t)st.n, max((int64_t)d + a.window, (int64_t)0)) : st.n;
      const int from = max(d, 0) * a.G - st.row0, end = min(rows * a.G - st.row0, cols);
      ok = warp_wait(&ctl.sfull[slot], turn, abort_flag);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int x = x0; x < min(cols, x0 + 128); x += 32) {
        float v[32];
        tmem_ld32(ts + x, v);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; ++y) asm volatile("" : "+f"(v[y]));
        if (__all_sync(0xffffffffu, from <= x && end >= x + 32)) add_weights<false>(v, nl + x, c2, 0, 0, sum0, sum1);
        else add_weights<true>(v, nl + x, c2, from - x, end - x, sum0, sum1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.sempty[slot]);
      if (!(flags & kLast)) continue;
      float s0, s1, s2, s3;
      f2_unpack(sum0, s0, s1);
      f2_unpack(sum1, s2, s3);
      float sum = (s0 + s1) + (s2 + s3);
      // the four parts: three give theirs to the one that writes
      const int x = swap & 1;
      const uint32_t phase = swap >> 1 & 1;
      if (!writes) {
        ok = warp_wait(&ctl.xempty[x], phase ^ 1, abort_flag);
        ctl.x[x][group][p] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.xfull[x]);
        continue;
      }
      ok = warp_wait(&ctl.xfull[x], phase, abort_flag);
      if (!ok) break;
      sum += ctl.x[x][group ^ 1][p];
      if (!(flags & kAlone)) sum += ctl.x[x][group ^ 2][p] + ctl.x[x][group ^ 3][p];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.xempty[x]);
      if (!(flags & kWhole)) a.part[((int64_t)2 * unit + (flags & kBegins ? 1 : 0)) * kBP + p] = sum;
      else if (mine) *to = old + sum;
    }
    if (!ok && lane == 0) fail();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // a wait gave up: copies in flight land before the memory they go to does
    if (warp == kWarpK)
      for (int i = 0; i < C::kSlotsK; ++i)
        if (issued >> i & 1) mbar_wait(&ctl.kfull[i], phase >> i & 1, kSpin);
    if (warp == kWarpQ && lane == 0)
      for (int i = 0; i < C::kSlotsQ; ++i)
        if (issued >> i & 1) mbar_wait(&ctl.qfull[i], phase >> i & 1, kSpin);
    __syncthreads();
  }
  if (warp == kWarpMma) tmem_dealloc(tm, 512);
}

// [page][head][slot][D] of the cache, boxes of 64 columns x `box` slots
bool make_k_map(CUtensorMap *m, const void *base, const gdn_cache_shape &s, int box) {
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
// [token][head][D] of q, boxes of 64 columns x the G heads of a group x RQ / G tokens
bool make_q_map(CUtensorMap *m, const void *base, const gdn_cache_shape &s, int G, int RQ) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)s.D, (cuuint64_t)s.Hq, (cuuint64_t)s.n_tok};
  cuuint64_t strides[2] = {(cuuint64_t)s.D * 2, (cuuint64_t)s.q_stride * 2};
  cuuint32_t b[3] = {64, (cuuint32_t)G, (cuuint32_t)(RQ / G)}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
gdn_status launch(MassArgs &a, const gdn_cache_shape &s, uint32_t flags, void *workspace, cudaStream_t st) {
  const int box = std::gcd(s.page_size, kBP);  // a power of two
  a.tokens = kNQ / a.G;  // whole tokens
  a.RQ = a.tokens * a.G;
  CUtensorMap mq, mk;
  if (!make_q_map(&mq, a.q, s, a.G, a.RQ) || !make_k_map(&mk, a.k, s, box)) return GDN_ERR_CUDA;
  a.meta = (int4 *)((char *)workspace + 256);
  a.part = (float *)(a.meta + 2 * kSms);
  return mass_launch<kBP>(paged_mass_tc_kernel<D>, a, kSms, kSms, kThreads, kData + 1024, st, mq, mk, a,
                          __builtin_ctz(box), flags & GDN_FLAG_TEST_NO_WAIT ? 1 : 0);
}

bool tc_shape(const gdn_cache_shape &s) {
  return s.dtype == GDN_BF16 && (s.D == 64 || s.D == 128 || s.D == 256) && s.page_size % 8 == 0 &&
         s.page_size <= 1 << 20 && s.n_pages > 0 && s.Hq / s.Hkv <= 128;
}

}  // namespace

bool paged_mass_tc_supported(const gdn_cache_shape &s, const void *q, const void *k) {
  if (!tc_shape(s) || !aligned(q, 16) || !aligned(k, 16)) return false;
  for (int64_t x : {s.q_stride, s.slot_stride, s.Hkv > 1 ? s.head_stride : 8, s.n_pages > 1 ? s.page_stride : 8})
    if (x % 8 || x >= 1LL << 39) return false;
  return true;
}

size_t paged_mass_tc_workspace(const gdn_cache_shape &s) {
  return tc_shape(s) ? 256 + kSms * (2 * sizeof(int4) + 2 * kBP * sizeof(float)) : 0;
}

gdn_status paged_mass_tc(MassArgs &a, const gdn_cache_shape &s, uint32_t flags, void *workspace, cudaStream_t st) {
  a.page_mask = s.page_size & (s.page_size - 1) ? -1 : s.page_size - 1;
  if (s.D == 64) return launch<64>(a, s, flags, workspace, st);
  return s.D == 128 ? launch<128>(a, s, flags, workspace, st) : launch<256>(a, s, flags, workspace, st);
}

}  // namespace gdn

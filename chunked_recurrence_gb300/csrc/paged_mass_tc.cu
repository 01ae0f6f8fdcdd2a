// paged_mass_tc.cu -- gdn_paged_mass on the tensor cores (tcgen05, bf16; D = 64, 128 or 256).
//
// S^T = K Q^T: a tile of 128 positions is the product's rows and stays in shared memory, a tile of up to 128 query rows its
// columns, so a thread owns a position and adds up 2^(c S - lse) over the columns, c = scale log2 e: no weight leaves
// the registers, nothing is added between threads but the two warpgroups' sums.
//
// Warps: two softmax warpgroups, which take the query tiles in turn from four TMEM slots of 128 columns; a warp for K's copies
// (pages by their table entries), one for Q's (whole tokens with the heads of the group), an MMA thread, and a warp that lays
// the rows' lse out beside the slots.  K and Q each have a ring of granules of 128 columns of a tile.
//
// FEW: up to 64 query rows a sequence and head (single tokens): one query tile a position tile, so K's ring gets the room.
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
constexpr int kData = 222 * 1024;    // the rings
constexpr int kBP = 128, kOver = 1, kThreads = 384, kBufs = 4;

template <int D, bool FEW>
struct Cfg {
  static constexpr int kHalves = D == 256 ? 2 : 1;       // granules of a tile
  static constexpr int kPanels = D == 64 ? 1 : 2;        // 64 columns each, of a granule
  static constexpr int kRowsQ = FEW ? 64 : 128;
  static constexpr int kPanelK = kBP * 128, kPanelQ = kRowsQ * 128;  // bytes
  static constexpr int kGranK = kPanels * kPanelK, kGranQ = kPanels * kPanelQ;
  static constexpr int kSlotsQ = FEW ? 2 * kHalves : D == 64 ? 8 : D == 128 ? 4 : 3;
  static constexpr int kSlotsK = (kData - kSlotsQ * kGranQ) / kGranK;
};

struct Ctl {
  uint64_t kfull[16], kempty[16], qfull[8], qempty[8], sfull[kBufs], sempty[kBufs], lready[kBufs], xfull[2], xempty[2], drain;
  uint32_t tmem;
  volatile int abort;
  MassStart start;
  alignas(16) float lse[kBufs][128];  // minus the rows' lse in base 2
  float x[2][128];        // a warpgroup's sums for the other
};

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

template <int D, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
    paged_mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const MassArgs a,
                         int box_log2, int no_wait) {
  using C = Cfg<D, FEW>;
  static_assert(C::kSlotsK >= C::kHalves + 1 && C::kSlotsK <= 16 && C::kSlotsQ <= 8, "rings");
  static_assert(kBP / 8 * C::kPanels <= 32, "a granule has at most one box a lane");
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t *ks = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *qs = ks + C::kSlotsK * C::kGranK;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, unit = blockIdx.x;
  constexpr int kWarpK = 8, kWarpQ = 9, kWarpMma = 10, kWarpLse = 11;
  launch_dependents();
  grid_dependency_wait();
  if (tid == 0) {
    a.meta[2 * unit] = make_int4(0, 0, 0, 0);
    ctl.abort = 0;
    for (int i = 0; i < 16; ++i) mbar_init(&ctl.kfull[i], 1), mbar_init(&ctl.kempty[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&ctl.qfull[i], 1), mbar_init(&ctl.qempty[i], 1);
    for (int i = 0; i < kBufs; ++i) mbar_init(&ctl.sfull[i], 1), mbar_init(&ctl.sempty[i], 4), mbar_init(&ctl.lready[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl.xfull[i], 4), mbar_init(&ctl.xempty[i], 4);
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
    // pages of a tile a lane each, the next piece's asked for before this one's copies
    auto look_up = [&](const MassWalk &x, bool there) {
      const int pos = (x.m.tile0 + x.j) * kBP + lane * box;
      const bool used = there && x.n > 0 && lane < nb && pos < x.m.hi && pos + box > x.m.seen;  // then the table's row holds it
      const int page = used ? a.table[x.s * a.table_stride + pos / a.page_size] : -1;
      if (used && (page < 0 || page >= a.n_pages)) {
        set_status(a.status, GDN_ERR_BOUNDS);
        return -1;
      }
      return page;
    };
    int page = look_up(w, more);
    while (more && ok) {
      MassWalk next = w;
      const bool later = mass_next<kBP, kOver>(a, next);
      const int ahead = look_up(next, later);
      if (w.n > 0) {
        const int i = lane / C::kPanels, p = lane % C::kPanels, at = (w.m.tile0 + w.j) * kBP + i * box;
        int pg = __shfl_sync(0xffffffffu, page, i);
        if (i >= nb) pg = -1;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, pg >= 0)) * (uint32_t)box * 128u;
        for (int half = 0; half < C::kHalves && ok; ++half, ring.step()) {
          if (!warp_wait(&ctl.kempty[ring.slot], ring.turn ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&ctl.kfull[ring.slot], bytes);
          __syncwarp();
          if (pg >= 0)
            tma_load_4d(ks + ring.slot * C::kGranK + p * C::kPanelK + i * box * 128, &tm_k, &ctl.kfull[ring.slot],
                        64 * (half * C::kPanels + p), at % a.page_size, w.h, pg);
          issued |= 1u << ring.slot, phase = (phase & ~(1u << ring.slot)) | ring.turn << ring.slot;
        }
      }
      w = next, more = later, page = ahead;
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kWarpQ) {
    // ================================================= Q: whole tokens with the heads of the group, a box each 64 columns
    if (lane == 0) {
      Ring<C::kSlotsQ> ring;
      const int tokens = a.RQ / a.G;
      for (; more && ok; more = mass_next<kBP, kOver>(a, w))
        for (int t = 0; t < w.n && ok; ++t)
          for (int half = 0; half < C::kHalves && ok; ++half, ring.step()) {
            ok = mbar_wait_spin(&ctl.qempty[ring.slot], ring.turn ^ 1, kSpin, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(&ctl.qfull[ring.slot], C::kPanels * a.RQ * 128);
            for (int p = 0; p < C::kPanels; ++p)
              tma_load_3d(qs + ring.slot * C::kGranQ + p * C::kPanelQ, &tm_q, &ctl.qfull[ring.slot],
                          64 * (half * C::kPanels + p), w.h * a.G, w.m.sp.t0 + w.i0 + (w.q0 + t) * tokens);
            issued |= 1u << ring.slot, phase = (phase & ~(1u << ring.slot)) | ring.turn << ring.slot;
          }
      if (!ok) fail();
    }
  } else if (warp == kWarpMma) {
    // ================================================= MMAs
    if (lane == 0) {
      Ring<C::kSlotsK> kr;
      Ring<C::kSlotsQ> qr;
      Ring<kBufs> buf;
      const uint64_t d_k = smem_desc(smem_u32(ks), 16, 1024, 2), d_q = smem_desc(smem_u32(qs), 16, 1024, 2);
      ok = !no_wait;
      for (; more && ok; more = mass_next<kBP, kOver>(a, w)) {
        Ring<C::kSlotsK> k0 = kr;
        for (int t = 0; t < w.n && ok; ++t, buf.step()) {
          ok = mbar_wait_spin(&ctl.sempty[buf.slot], buf.turn ^ 1, kSpin, abort_flag);
          const int rows = min(a.RQ, (w.i1 - w.i0) * a.G - (w.q0 + t) * a.RQ);
          const uint32_t id = idesc_bf16(kBP, (rows + 15) & ~15, false, false);
          kr = k0;
          for (int half = 0; half < C::kHalves && ok; ++half, kr.step(), qr.step()) {
            if (t == 0) ok = mbar_wait_spin(&ctl.kfull[kr.slot], kr.turn, kSpin, abort_flag);
            ok = ok && mbar_wait_spin(&ctl.qfull[qr.slot], qr.turn, kSpin, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dk = d_k + ((kr.slot * C::kGranK) >> 4), dq = d_q + ((qr.slot * C::kGranQ) >> 4);
#pragma unroll
            for (int x = 0; x < C::kPanels * 4; ++x)
              umma_bf16(tm + buf.slot * 128, dk + (((x >> 2) * C::kPanelK + (x & 3) * 32) >> 4),
                        dq + (((x >> 2) * C::kPanelQ + (x & 3) * 32) >> 4), id, half > 0 || x > 0);
            umma_commit(&ctl.qempty[qr.slot]);
          }
          if (!ok) break;
          umma_commit(&ctl.sfull[buf.slot]);
        }
        if (w.n > 0 && ok)
          for (int half = 0; half < C::kHalves; ++half, k0.step()) umma_commit(&ctl.kempty[k0.slot]);
      }
      if (!ok || *abort_flag) {  // MMAs in flight end before the block's memory goes
        if (!ok) fail();
        umma_commit(&ctl.drain);
        mbar_wait(&ctl.drain, 0, kSpin);
      }
    }
  } else if (warp == kWarpLse) {
    // ================================================= the rows' lse, four rows a lane
    Ring<kBufs> buf;
    for (; more && ok; more = mass_next<kBP, kOver>(a, w))
      for (int t = 0; t < w.n && ok; ++t, buf.step()) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = (w.q0 + t) * a.RQ + 4 * lane + k, i = r / a.G, g = r - i * a.G;
          const bool there = 4 * lane + k < a.RQ && r < (w.i1 - w.i0) * a.G;
          const float x = there ? a.lse[(int64_t)(w.m.sp.t0 + w.i0 + i) * (a.G * a.Hkv) + w.h * a.G + g] : 0.f;
          v[k] = x == -INFINITY ? x : -x * 1.44269504088896340736f;  // such a row weighs nothing
        }
        if (!warp_wait(&ctl.sempty[buf.slot], buf.turn ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        *reinterpret_cast<float4 *>(&ctl.lse[buf.slot][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.lready[buf.slot]);
      }
    if (!ok && lane == 0) fail();
  } else {
    // ================================================= softmax: a thread owns a position, a warpgroup every second query tile
    const int group = warp >> 2, p = tid & 127;
    const uint32_t lq = (uint32_t)((warp & 3) * 32) << 16;
    const uint64_t c2 = f2_pack(a.c, a.c);
    Ring<kBufs> buf;
    uint32_t step = 0, swaps = 0;
    for (; more && ok; more = mass_next<kBP, kOver>(a, w)) {
      const int pos = (w.m.tile0 + w.j) * kBP + p;
      int lo, hi;  // rows of the tile that see the position
      mass_rows(a, w, pos, lo, hi);
      const bool last = (int)(step + w.n - 1 & 1) == group || w.n == 0;  // this warpgroup writes the sums
      const bool whole = mass_begins(w) && mass_ends(w), mine = pos >= w.m.lo && pos < w.m.hi;
      float old = 0.f;
      float *to = a.mass + w.s * a.row_stride + w.h * a.mass_head_stride + pos;
      if (last && whole && mine && !a.all) old = *to;
      uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
      for (int t = 0; t < w.n; ++t, ++step, buf.step()) {
        if ((int)(step & 1) != group) continue;
        const int row0 = (w.q0 + t) * a.RQ, cols = min(a.RQ, (w.i1 - w.i0) * a.G - row0);
        ok = ok && warp_wait(&ctl.lready[buf.slot], buf.turn, abort_flag) &&
             warp_wait(&ctl.sfull[buf.slot], buf.turn, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int from = lo - row0, end = min(hi - row0, cols);  // columns that count
#pragma unroll 1
        for (int x = 0; x < cols; x += 32) {
          float s[32];
          tmem_ld32(tm + lq + buf.slot * 128 + x, s);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; ++y) asm volatile("" : "+f"(s[y]));
          const ulonglong2 *l = reinterpret_cast<const ulonglong2 *>(&ctl.lse[buf.slot][x]);
          const bool all = __all_sync(0xffffffffu, from <= x && end >= x + 32);
#pragma unroll
          for (int y = 0; y < 32; y += 4) {
            const ulonglong2 nl = l[y / 4];
            float e0, e1, e2, e3;
            f2_unpack(f2_fma(f2_pack(s[y], s[y + 1]), c2, nl.x), e0, e1);
            f2_unpack(f2_fma(f2_pack(s[y + 2], s[y + 3]), c2, nl.y), e2, e3);
            e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
            if (!all) {
              e0 = x + y >= from && x + y < end ? e0 : 0.f;
              e1 = x + y + 1 >= from && x + y + 1 < end ? e1 : 0.f;
              e2 = x + y + 2 >= from && x + y + 2 < end ? e2 : 0.f;
              e3 = x + y + 3 >= from && x + y + 3 < end ? e3 : 0.f;
            }
            sum0 = f2_add(sum0, f2_pack(e0, e1));
            sum1 = f2_add(sum1, f2_pack(e2, e3));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.sempty[buf.slot]);
      }
      if (!ok) break;
      float s0, s1, s2, s3;
      f2_unpack(sum0, s0, s1);
      f2_unpack(sum1, s2, s3);
      float sum = (s0 + s1) + (s2 + s3);
      if (w.n >= 2) {  // both have a part: one gives it to the other
        const int x = swaps & 1;
        const uint32_t turn = swaps >> 1 & 1;
        if (!last) {
          ok = warp_wait(&ctl.xempty[x], turn ^ 1, abort_flag);
          ctl.x[x][p] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.xfull[x]);
        } else {
          ok = warp_wait(&ctl.xfull[x], turn, abort_flag);
          sum += ctl.x[x][p];
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.xempty[x]);
        }
        ++swaps;
        if (!ok) break;
      }
      if (last && (w.n > 0 || group == 0)) {
        if (!whole) a.part[((int64_t)2 * unit + mass_begins(w)) * kBP + p] = sum;
        else if (mine) *to = old + sum;
        if (p == 0) mass_note(a, w, unit);
      }
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

template <int D, bool FEW>
gdn_status launch(MassArgs &a, const gdn_cache_shape &s, uint32_t flags, void *workspace, cudaStream_t st) {
  const int box = std::gcd(s.page_size, kBP);  // a power of two
  CUtensorMap mq, mk;
  if (!make_q_map(&mq, a.q, s, a.G, a.RQ) || !make_k_map(&mk, a.k, s, box)) return GDN_ERR_CUDA;
  a.meta = (int4 *)((char *)workspace + 256);
  a.part = (float *)(a.meta + 2 * kSms);
  return mass_launch<kBP>(paged_mass_tc_kernel<D, FEW>, a, kSms, kThreads, kData + 1024, st, mq, mk, a,
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

gdn_status paged_mass_tc(MassArgs &a, const gdn_cache_shape &s, int32_t max_new, uint32_t flags, void *workspace,
                         cudaStream_t st) {
  const int64_t most = (int64_t)std::max(max_new, 1) * a.G;
  const bool few = most <= 64;
  a.RQ = few ? (int)most : 128 / a.G * a.G;  // whole tokens
  if (s.D == 64) return few ? launch<64, true>(a, s, flags, workspace, st) : launch<64, false>(a, s, flags, workspace, st);
  if (s.D == 128) return few ? launch<128, true>(a, s, flags, workspace, st) : launch<128, false>(a, s, flags, workspace, st);
  return few ? launch<256, true>(a, s, flags, workspace, st) : launch<256, false>(a, s, flags, workspace, st);
}

}  // namespace gdn

// paged_mass.cu -- gdn_paged_mass: the softmax weight that each cached position gets from new tokens, by their attention's
// log-sum-exp:
//     mass[s, h, j] (+)= sum over new tokens i of s that see j, heads g of kv head h's group, of e^(scale <q[i, g], k_j> - lse[i, g])
// Argument checks, dispatch, and the kernel for every type, width, page size, stride and alignment (bf16 of D 64, 128 and 256:
// paged_mass_tc.cu on tcgen05, paged_mass_few.cu for few query rows).
//
// A block takes equal parts of the line of work (paged_mass.cuh): 64 positions of a sequence and kv head, whose keys stay in
// shared memory as fp32 while their queries come by, 32 rows a tile, the next tile's copies under this one's
// products.  S^T = K Q^T by mma.sync with each fp32 operand in two TF32 parts, three products (one where the
// values are bf16, exact in TF32); a position is a row of the product, so its weights add up along the row in the
// registers of four lanes and nothing is added across blocks but the parts of a tile cut between two shares.  A sum that
// is not finite is worked out again in plain fp32, for an infinite operand's parts are (inf, NaN).
// Small calls are a chain of launch, lengths, copies, products and the join, 17 us at the sizes of a test; long ones the
// products' operands from shared memory, split anew for every product (paged_mass_tc.cu's prompts with this kernel: 6359 us).
#include <algorithm>

#include "chunk_bwd_mma.cuh"
#include "paged_attn.cuh"
#include "paged_mass.cuh"

namespace gdn {
namespace {

namespace tc = gdn_bwd::tc;
constexpr int kThreads = 128, kBP = 64, kRQ = 32, kOver = 1;

template <int DP>
struct Cfg {
  static constexpr int kPitch = DP + 4;  // floats a row: the fragments' loads meet no bank conflict
  static constexpr size_t kSmem = sizeof(float) * ((kBP + 2 * kRQ) * kPitch);
  static constexpr int kBlocks = DP == 256 ? 1 : DP == 128 ? 3 : 6;  // of an SM, by their shared memory
};

template <typename T>
__device__ __forceinline__ int64_t place_of(const MassArgs &a, const MassWalk &w, int pos) {
  const int page = page_of(a.table + w.s * a.table_stride, pos, a.page_size, a.max_pages, a.n_pages);
  if (page < 0) return -1;
  return page * a.page_stride + pos % a.page_size * a.slot_stride + w.h * a.head_stride;
}
template <typename T>
__device__ __forceinline__ const T *query_of(const MassArgs &a, const MassWalk &w, int r) {
  const int i = r / a.G, g = r - i * a.G;
  return (const T *)a.q + (int64_t)(w.m.sp.t0 + w.i0 + i) * a.q_stride + (int64_t)(w.h * a.G + g) * a.D;
}
__device__ __forceinline__ float lse_of(const MassArgs &a, const MassWalk &w, int r) {
  const int i = r / a.G, g = r - i * a.G;
  const float x = a.lse[(int64_t)(w.m.sp.t0 + w.i0 + i) * (a.G * a.Hkv) + w.h * a.G + g] * 1.44269504088896340736f;
  return x == -INFINITY ? INFINITY : x;  // such a row weighs nothing
}

// A piece's sums in plain fp32, a warp a position, a lane the elements lane, lane + 32, ...
template <typename T, int DP>
__device__ __noinline__ void plain_sums(const MassArgs &a, const MassWalk &w, float *sums) {
  const int lane = threadIdx.x & 31;
  for (int p = threadIdx.x >> 5; p < kBP; p += kThreads / 32) {
    const int pos = (w.m.tile0 + w.j) * kBP + p;
    int lo, hi;
    mass_rows(a, w, pos, lo, hi);
    const int64_t at = pos >= w.m.seen && pos < w.m.hi ? place_of<T>(a, w, pos) : -1;
    float sum = 0.f;
    for (int r = max(lo, w.q0 * kRQ); r < min(hi, (w.q0 + w.n) * kRQ) && at >= 0; ++r) {
      const T *q = query_of<T>(a, w, r), *k = (const T *)a.k + at;
      float x = 0.f;
#pragma unroll
      for (int d = 0; d < DP; d += 32)
        if (lane + d < a.D) x = fmaf(to_f32<T>(q[lane + d]), to_f32<T>(k[lane + d]), x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      sum += exp2f(fmaf(x, a.c, -lse_of(a, w, r)));
    }
    if (lane == 0) sums[p] = sum;
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) paged_mass_kernel(const MassArgs a, bool wide) {
  using C = Cfg<DP>;
  constexpr bool kExact = sizeof(T) == 2;
  extern __shared__ __align__(16) float smem[];
  __shared__ MassStart start;
  __shared__ float lses[2][kRQ], sums[kBP];
  float *ks = smem, *qs = ks + kBP * C::kPitch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3, unit = blockIdx.x;
  sm100::launch_dependents();
  sm100::grid_dependency_wait();
  if (tid == 0) a.meta[2 * unit] = make_int4(0, 0, 0, 0);
  int64_t left;
  if (!mass_start<kBP, kOver, kThreads>(a, unit, gridDim.x, start, left)) return;
  MassWalk w;
  bool more = mass_begin<kBP, kOver>(a, start, left, w);

  // four values of a row into shared memory (col < D)
  auto put4 = [&](float *to, const T *from, int col) {
    if (sizeof(T) == 4 && wide) {
      cp_async16(to, from + col);
    } else {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = col + i < a.D ? to_f32<T>(from[col + i]) : 0.f;
      *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
    }
  };
  auto load_q = [&](int t) {  // query tile q0 + t of the piece
    for (int i = tid; i < kRQ * (DP / 4); i += kThreads) {
      const int r = i / (DP / 4), col = (i - r * (DP / 4)) * 4, row = (w.q0 + t) * kRQ + r;
      float *to = qs + ((t & 1) * kRQ + r) * C::kPitch + col;
      if (row < (w.i1 - w.i0) * a.G && col < a.D) put4(to, query_of<T>(a, w, row), col);
      else *reinterpret_cast<float4 *>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < kRQ) {
      const int row = (w.q0 + t) * kRQ + tid;
      lses[t & 1][tid] = row < (w.i1 - w.i0) * a.G ? lse_of(a, w, row) : INFINITY;
    }
    cp_async_commit();
  };
  for (; more; more = mass_next<kBP, kOver>(a, w)) {
    const int pos0 = (w.m.tile0 + w.j) * kBP, m0 = warp * 16;
    __syncthreads();  // the piece before is done with
    if (w.n > 0) {
      for (int i = tid; i < kBP * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), col = (i - r * (DP / 4)) * 4, pos = pos0 + r;
        float *to = ks + r * C::kPitch + col;
        int64_t at = -1;
        if (pos >= w.m.seen && pos < w.m.hi && col < a.D) {
          at = place_of<T>(a, w, pos);
          if (at < 0) set_status(a.status, GDN_ERR_BOUNDS);
        }
        if (at >= 0) put4(to, (const T *)a.k + at, col);
        else *reinterpret_cast<float4 *>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      load_q(0);
    }
    int lo[2], hi[2];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) mass_rows(a, w, pos0 + m0 + g4 + 8 * e, lo[e], hi[e]);
    for (int t = 0; t < w.n; ++t) {
      cp_async_wait_all();
      __syncthreads();  // this tile is there, the one before done with
      if (t + 1 < w.n) load_q(t + 1);
      const float *q = qs + (t & 1) * kRQ * C::kPitch;
      const int row0 = (w.q0 + t) * kRQ, nb = (min((w.i1 - w.i0) * a.G - row0, kRQ) + 7) / 8;
      float s[kRQ / 8][4];
#pragma unroll
      for (int i = 0; i < kRQ / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      // the MMAs' accumulation cuts off towards zero: a sum is made of parts of four steps, added by fp32 additions
#pragma unroll 1
      for (int k0 = 0; k0 < DP; k0 += 32) {
        float x[kRQ / 8][4];
#pragma unroll
        for (int i = 0; i < kRQ / 8; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 32; kk += 8) {
          const float *k = ks + (m0 + g4) * C::kPitch + k0 + kk + t4;
          tc::FragA fa;
          if constexpr (kExact) tc::frag_a_exact(fa, k[0], k[8 * C::kPitch], k[4], k[8 * C::kPitch + 4]);
          else tc::frag_a(fa, k[0], k[8 * C::kPitch], k[4], k[8 * C::kPitch + 4]);
#pragma unroll
          for (int i = 0; i < kRQ / 8; ++i) {
            if (i >= nb) break;  // the same for the block
            const float *b = q + (i * 8 + g4) * C::kPitch + k0 + kk + t4;
            tc::FragB fb;
            if constexpr (kExact) tc::frag_b_exact(fb, b[0], b[4]);
            else tc::frag_b(fb, b[0], b[4]);
            tc::mma_x<kExact, kExact>(x[i], fa, fb);
          }
        }
#pragma unroll
        for (int i = 0; i < kRQ / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] += x[i][e];
      }
      float part[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kRQ / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = i * 8 + 2 * t4 + (e & 1), row = row0 + col;
          const float y = exp2f(fmaf(s[i][e], a.c, -lses[t & 1][col]));
          part[e >> 1] += row >= lo[e >> 1] && row < hi[e >> 1] ? y : 0.f;
        }
      sum[0] += part[0], sum[1] += part[1];
    }
    float odd = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      const int p = m0 + g4 + 8 * e;
      if (t4 == 0) sums[p] = sum[e];
      if (pos0 + p >= w.m.lo && pos0 + p < w.m.hi) odd = fmaf(sum[e], 0.f, odd);  // NaN where one is not finite
    }
    if (__syncthreads_or(isnan(odd))) {
      plain_sums<T, DP>(a, w, sums);
      __syncthreads();
    }
    if (tid < kBP) mass_put<kBP>(a, w, unit, tid, sums[tid]);
    if (tid == 0) mass_note(a, w, unit);
  }
}

template <typename T, int DP>
gdn_status launch(MassArgs &a, bool wide, void *workspace, cudaStream_t st) {
  const int shares = 152 * Cfg<DP>::kBlocks;
  a.meta = (int4 *)((char *)workspace + 256);
  a.part = (float *)(a.meta + 2 * shares);
  return mass_launch<kBP>(paged_mass_kernel<T, DP>, a, shares, shares, kThreads, Cfg<DP>::kSmem, st, a, wide);
}
size_t plain_workspace() { return 256 + 152 * 6 * (2 * sizeof(int4) + 2 * kBP * sizeof(float)); }

template <typename T>
gdn_status dispatch(MassArgs &a, bool wide, void *workspace, cudaStream_t st) {
  if (a.D <= 64) return launch<T, 64>(a, wide, workspace, st);
  if (a.D <= 128) return launch<T, 128>(a, wide, workspace, st);
  return launch<T, 256>(a, wide, workspace, st);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_paged_mass_workspace_bytes(const gdn_cache_shape *shape) {
  gdn_cache_shape s;
  static const int32_t some = 0;
  if (normalise_cache_shape(shape, &some, &s) != GDN_OK) return 0;
  return std::max({plain_workspace(), paged_mass_tc_workspace(s), paged_mass_few_workspace()});
}

extern "C" gdn_status gdn_paged_mass(const void *q, const void *k_cache, const int32_t *page_table,
                                     const int32_t *seq_lens, const int32_t *cu_seqlens, const float *lse,
                                     const gdn_cache_shape *shape, int32_t max_new, float scale, int32_t window,
                                     int32_t accumulate, uint32_t flags, float *mass, int64_t row_stride,
                                     int64_t head_stride, int32_t mass_len, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  gdn_cache_shape s;
  const gdn_status ok = normalise_cache_shape(shape, cu_seqlens, &s);
  if (ok != GDN_OK) return ok;
  if (max_new < 0 || window < 0 || mass_len < 0 || (accumulate != 0 && accumulate != 1) ||
      (flags & ~(uint32_t)(GDN_FLAG_SIMT | GDN_FLAG_TEST_NO_WAIT)))
    return GDN_ERR_INVALID_ARG;
  if (head_stride == 0 && row_stride == 0) head_stride = mass_len, row_stride = head_stride * s.Hkv;
  if ((s.Hkv > 1 && head_stride < mass_len) || (s.n_seqs > 1 && row_stride < mass_len)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < gdn_paged_mass_workspace_bytes(shape))
    return GDN_ERR_WORKSPACE;
  if (s.n_seqs == 0 || (s.n_tok == 0 && accumulate)) return GDN_OK;
  if (!page_table || !seq_lens || (!mass && mass_len > 0)) return GDN_ERR_INVALID_ARG;
  if (s.n_tok > 0 && (!q || !k_cache || !lse)) return GDN_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  MassArgs a{};
  a.seqs = paged_seqs(s, seq_lens, cu_seqlens);
  a.q = q, a.k = k_cache, a.lse = lse, a.mass = mass, a.table = page_table;
  a.table_stride = s.table_stride, a.page_stride = s.page_stride, a.slot_stride = s.slot_stride;
  a.head_stride = s.head_stride, a.q_stride = s.q_stride, a.row_stride = row_stride, a.mass_head_stride = head_stride;
  a.G = s.Hq / s.Hkv, a.Hkv = s.Hkv, a.D = s.D, a.page_size = s.page_size, a.max_pages = s.max_pages;
  a.n_pages = s.n_pages, a.room = mass_len, a.all = !accumulate;
  a.window = window >= a.seqs.max_tokens ? 0 : window;  // no window hides anything of such a cache
  a.RQ = kRQ, a.c = scale * 1.44269504088896340736f;
  a.status = s.status ? s.status : (int32_t *)workspace;
  if (!(flags & GDN_FLAG_SIMT) && s.n_tok > 0 && paged_mass_tc_supported(s, q, k_cache))
    return paged_mass_few(a, max_new) && !(flags & GDN_FLAG_TEST_NO_WAIT)  // that kernel has no waits to test
               ? paged_mass_few_run(a, max_new, workspace, st)
               : paged_mass_tc(a, s, flags, workspace, st);
  bool wide = s.D % 4 == 0 && aligned(q, 16) && aligned(k_cache, 16);
  for (int64_t x : {s.q_stride, s.page_stride, s.slot_stride, s.head_stride}) wide = wide && x % 4 == 0;
  return s.dtype == GDN_BF16 ? dispatch<__nv_bfloat16>(a, wide, workspace, st) : dispatch<float>(a, wide, workspace, st);
}

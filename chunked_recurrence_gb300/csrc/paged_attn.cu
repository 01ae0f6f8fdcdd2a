// paged_attn.cu -- attention of new tokens over a paged cache (gdn_paged_attn): argument
// checks, dispatch and the CUDA-core kernel (GDN_FLAG_SIMT).  The kernels that run by default are in
// paged_attn_tc.cu (bf16 on tcgen05) and paged_attn_f32.cu (fp32, and what the first does not take).
//
//     o[t, h] = sum_j softmax_j(scale <q[t, h], k_j>) v_j   over the positions that t sees
//
// paged_attn_simt_kernel: fp32 arithmetic for every type, width (up to 256), page size, stride
// and alignment.  A block of kWarps warps takes kRows query rows of one sequence and kv head
// (row = token * group + head in the group) and one of `splits` parts of their positions; its
// warps take the positions in turn, a lane holding the elements lane, lane + 32, ... of k, v and
// the rows.  Each warp keeps a running maximum m, sum l and weighted sum of v per row in one pass;
// at the end m, l and the sums of the warps (and, by simt_join_kernel, of the parts) join as
//     M = max m_i,   L = sum e^(m_i - M) l_i,   o = sum e^(m_i - M) acc_i / L.
// Positions that a row does not see are skipped, so nothing in them can reach it.
#include <algorithm>

#include "common.cuh"
#include "paged.cuh"
#include "paged_attn.cuh"
#include "sm100.cuh"

namespace gdn {

gdn_status normalise_cache_shape(const gdn_cache_shape *in, const int32_t *cu_seqlens, gdn_cache_shape *out) {
  if (!in) return GDN_ERR_INVALID_ARG;
  gdn_cache_shape s = *in;
  if (s.dtype != GDN_F32 && s.dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (s.n_seqs < 0 || s.n_tok < 0 || s.Hq < 1 || s.Hkv < 1 || s.Hq % s.Hkv != 0 || s.D < 1 || s.page_size < 1 ||
      s.n_pages < 0 || s.max_pages < 0)
    return GDN_ERR_INVALID_ARG;
  if (!cu_seqlens && s.n_tok != s.n_seqs) return GDN_ERR_INVALID_ARG;
  if (s.table_stride == 0) s.table_stride = s.max_pages;
  if (s.table_stride < s.max_pages) return GDN_ERR_INVALID_ARG;
  if (s.page_stride == 0 && s.slot_stride == 0 && s.head_stride == 0) {
    s.head_stride = s.D;
    s.slot_stride = (int64_t)s.Hkv * s.D;
    s.page_stride = s.slot_stride * s.page_size;
  }
  // slots, heads and pages may lie in any order but not on top of each other
  if ((s.Hkv > 1 && s.head_stride < s.D) || (s.page_size > 1 && s.slot_stride < s.D) ||
      (s.n_pages > 1 && s.page_stride < s.D))
    return GDN_ERR_INVALID_ARG;
  if (s.q_stride == 0) s.q_stride = (int64_t)s.Hq * s.D;
  if (s.k_stride == 0) s.k_stride = (int64_t)s.Hkv * s.D;
  if (s.v_stride == 0) s.v_stride = (int64_t)s.Hkv * s.D;
  if (s.q_stride < (int64_t)s.Hq * s.D || s.k_stride < (int64_t)s.Hkv * s.D || s.v_stride < (int64_t)s.Hkv * s.D)
    return GDN_ERR_INVALID_ARG;
  if (!aligned(s.status, sizeof(int32_t))) return GDN_ERR_INVALID_ARG;
  if (s.D > 256 || s.Hq > 65535) return GDN_ERR_UNSUPPORTED;
  // rows of a kv head and slots of items fit 32 bits
  if ((int64_t)s.n_tok * (s.Hq / s.Hkv) + s.n_seqs > 2147483647LL / 2) return GDN_ERR_UNSUPPORTED;
  *out = s;
  return GDN_OK;
}

PagedSeqs paged_seqs(const gdn_cache_shape &s, const int32_t *seq_lens, const int32_t *cu_seqlens) {
  const int64_t most = (int64_t)s.max_pages * s.page_size;
  return PagedSeqs{seq_lens, cu_seqlens, s.n_seqs, s.n_tok, (int32_t)std::min<int64_t>(most, 2147483647LL - 4096)};
}

namespace {

constexpr int kWarps = 4, kRows = 4, kJoin = 128;

template <typename T, int NE>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_simt_kernel(const SimtArgs a) {
  __shared__ float s_acc[kWarps][kRows][NE * 32], s_m[kWarps][kRows], s_l[kWarps][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.Hkv, h = blockIdx.y, part = blockIdx.z;
  const Item it = item_at(a.seqs, blockIdx.x, G, kRows, 1, a.window);  // tiles of one position
  if (!it.ok && threadIdx.x == 0) set_status(a.status, GDN_ERR_BOUNDS);
  if (it.rows <= 0) return;

  float q[kRows][NE], acc[kRows][NE], m[kRows], l[kRows];
  int lo[kRows], hi[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = it.row0 + min(r, it.rows - 1), i = row / G, g = row - i * G;
    const T *qp = (const T *)a.q + (int64_t)(it.t0 + i) * a.q_stride + (int64_t)(h * G + g) * a.D;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      q[r][e] = lane + 32 * e < a.D ? to_f32<T>(qp[lane + 32 * e]) : 0.f;
      acc[r][e] = 0.f;
    }
    m[r] = -INFINITY, l[r] = 0.f;
    const int p = it.first + i;
    hi[r] = r < it.rows ? p + 1 : 0;
    lo[r] = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
  }
  const int begin = it.lo + (int)share_begin(it.hi - it.lo, part, a.splits);
  const int end = it.lo + (int)share_begin(it.hi - it.lo, part + 1, a.splits);
  const int32_t *row = a.table + (int64_t)it.s * a.table_stride;
  for (int j = begin + warp; j < end; j += kWarps) {
    const int page = page_of(row, j, a.page_size, a.max_pages, a.n_pages);
    if (page < 0) {
      if (lane == 0) set_status(a.status, GDN_ERR_BOUNDS);
      continue;
    }
    const int64_t at = (int64_t)page * a.page_stride + (int64_t)(j % a.page_size) * a.slot_stride +
                       (int64_t)h * a.head_stride + lane;
    const T *kp = (const T *)a.k + at, *vp = (const T *)a.v + at;
    float kv[NE], vv[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      kv[e] = lane + 32 * e < a.D ? to_f32<T>(kp[32 * e]) : 0.f;
      vv[e] = lane + 32 * e < a.D ? to_f32<T>(vp[32 * e]) : 0.f;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < NE; ++e) s = fmaf(q[r][e], kv[e], s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (j < lo[r] || j >= hi[r]) continue;  // the same for the whole warp
      s *= a.scale_log2;
      const float top = fmaxf(m[r], s);
      // nothing but scores of -inf so far: they weigh nothing
      const float keep = m[r] == -INFINITY ? 0.f : exp2f(m[r] - top), p = s == -INFINITY ? 0.f : exp2f(s - top);
      m[r] = top;
      l[r] = l[r] * keep + p;
#pragma unroll
      for (int e = 0; e < NE; ++e) acc[r][e] = fmaf(acc[r][e], keep, p * vv[e]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int e = 0; e < NE; ++e) s_acc[warp][r][lane + 32 * e] = acc[r][e];
    if (lane == 0) s_m[warp][r] = m[r], s_l[warp][r] = l[r];
  }
  __syncthreads();
  for (int r = warp; r < it.rows; r += kWarps) {
    float top = -INFINITY, sum = 0.f, w[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_m[i][r]);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      w[i] = s_l[i][r] == 0.f ? 0.f : exp2f(s_m[i][r] - top);
      sum += w[i] * s_l[i][r];
    }
    const int rr = it.row0 + r, i = rr / G, g = rr - i * G;
    const int64_t out = (int64_t)(it.t0 + i) * a.Hq + h * G + g;
    float *pp = a.part ? a.part + ((int64_t)part * a.seqs.n_tok * a.Hq + out) * (a.D + 2) : nullptr;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int d = lane; d < a.D; d += 32) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) x += w[i] == 0.f ? 0.f : w[i] * s_acc[i][r][d];
      if (pp) pp[2 + d] = x;
      else ((T *)a.o)[out * a.D + d] = from_f32<T>(x * inv);
    }
    if (lane == 0) {
      if (pp) pp[0] = top, pp[1] = sum;
      else if (a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
    }
  }
}

// A block per row: the parts' maxima, sums and weighted sums joined.  A lane has the maximum and sum of parts lane
// and lane + 32 (there are at most 64); a warp adds up every fourth part.
template <typename T>
__global__ void __launch_bounds__(kJoin) simt_join_kernel(const float *part, int splits, int64_t rows, int D, T *o,
                                                          float *lse) {
  __shared__ float s_x[kJoin / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sm100::grid_dependency_wait();
  const int64_t r = blockIdx.x, step = rows * (D + 2);
  const float *p = part + r * (D + 2);
  float m[2], l[2], w[2], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    m[j] = i < splits ? p[i * step] : -INFINITY, l[j] = i < splits ? p[i * step + 1] : 0.f;
    top = fmaxf(top, m[j]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = l[j] == 0.f ? 0.f : exp2f(m[j] - top);
    sum += w[j] * l[j];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int d = lane; d < (D + 31) / 32 * 32; d += 32) {
    float x = 0.f;
#pragma unroll 4
    for (int i = warp; i < splits; i += kJoin / 32) {
      const float a = __shfl_sync(0xffffffffu, w[0], i & 31), b = __shfl_sync(0xffffffffu, w[1], i & 31);
      const float wi = i < 32 ? a : b, u = d < D ? p[i * step + 2 + d] : 0.f;
      if (wi != 0.f) x += wi * u;  // a part that saw nothing has no say
    }
    s_x[warp][d] = x;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kJoin) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kJoin / 32; ++i) x += s_x[i][d];
    o[r * D + d] = from_f32<T>(x * inv);
  }
  if (threadIdx.x == 0 && lse) lse[r] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

// Parts a row group's positions are cut into: enough blocks for the GPU, at most 16.
int simt_splits(const gdn_cache_shape &s) {
  const int64_t blocks = item_slots(s.n_tok, s.n_seqs, s.Hq / s.Hkv, kRows) * s.Hkv;
  const int64_t want = (152 * 8 + blocks - 1) / std::max<int64_t>(blocks, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>(16, want));
}
size_t parts_bytes(const gdn_cache_shape &s, int splits) {
  return 256 + (splits > 1 ? (size_t)splits * s.n_tok * s.Hq * (s.D + 2) * sizeof(float) : 0);
}

template <typename T, int NE>
gdn_status launch_simt(const SimtArgs &a, int64_t slots, cudaStream_t st) {
  paged_attn_simt_kernel<T, NE><<<dim3((unsigned)slots, a.Hkv, a.splits), kWarps * 32, 0, st>>>(a);
  return launch_status();
}

template <typename T>
gdn_status dispatch_simt(const SimtArgs &a, int64_t slots, cudaStream_t st) {
  switch ((a.D + 31) / 32) {
#define GDN_NE(N) \
  case N:         \
    return launch_simt<T, N>(a, slots, st);
    GDN_NE(1) GDN_NE(2) GDN_NE(3) GDN_NE(4) GDN_NE(5) GDN_NE(6) GDN_NE(7) GDN_NE(8)
#undef GDN_NE
    default: return GDN_ERR_UNSUPPORTED;
  }
}

template <typename T>
gdn_status launch_join(const SimtArgs &a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.seqs.n_tok * a.Hq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows), cfg.blockDim = dim3(kJoin), cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its launch overlaps the parts' end
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, simt_join_kernel<T>, (const float *)a.part, (int)a.splits, rows, (int)a.D, (T *)a.o, a.lse);
  return launch_status();
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_paged_attn_workspace_bytes(const gdn_cache_shape *shape, int32_t max_new) {
  gdn_cache_shape s;
  // any non-null offsets: the number of tokens is checked by the call
  static const int32_t some = 0;
  if (max_new < 0 || normalise_cache_shape(shape, &some, &s) != GDN_OK) return 0;
  return std::max({parts_bytes(s, simt_splits(s)), parts_bytes(s, paged_attn_f32_splits(s, max_new, 0)),
                   paged_attn_tc_workspace(s, max_new)});
}

extern "C" gdn_status gdn_paged_attn(const void *q, const void *k_cache, const void *v_cache,
                                     const int32_t *page_table, const int32_t *seq_lens, const int32_t *cu_seqlens,
                                     const gdn_cache_shape *shape, int32_t max_new, float scale, int32_t window,
                                     uint32_t flags, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  gdn_cache_shape s;
  const gdn_status ok = normalise_cache_shape(shape, cu_seqlens, &s);
  if (ok != GDN_OK) return ok;
  if (max_new < 0 || window < 0 || (flags & ~(uint32_t)(GDN_FLAG_SIMT | GDN_FLAG_TEST_NO_WAIT)))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < gdn_paged_attn_workspace_bytes(shape, max_new))
    return GDN_ERR_WORKSPACE;
  if (s.n_tok == 0 || s.n_seqs == 0) return GDN_OK;
  if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !o) return GDN_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const PagedSeqs seqs = paged_seqs(s, seq_lens, cu_seqlens);
  const float scale_log2 = scale * 1.44269504088896340736f;  // softmax in base 2
  if (!(flags & GDN_FLAG_SIMT) && paged_attn_tc_supported(q, k_cache, v_cache, o, s, scale))
    return paged_attn_tc(q, k_cache, v_cache, page_table, seqs, s, max_new, scale_log2, window, flags, o, lse,
                         workspace, st);
  const bool simt = flags & GDN_FLAG_SIMT;
  SimtArgs a{seqs, q, k_cache, v_cache, o, lse, nullptr, page_table, s.table_stride, s.page_stride, s.slot_stride,
             s.head_stride, s.q_stride, s.Hq, s.Hkv, s.D, s.page_size, s.max_pages, s.n_pages, window,
             simt ? simt_splits(s) : paged_attn_f32_splits(s, max_new, window), scale_log2,
             s.status ? s.status : (int32_t *)workspace};
  if (a.splits > 1) a.part = (float *)((char *)workspace + 256);
  gdn_status r;
  if (simt) {
    const int64_t slots = item_slots(s.n_tok, s.n_seqs, s.Hq / s.Hkv, kRows);
    r = s.dtype == GDN_BF16 ? dispatch_simt<__nv_bfloat16>(a, slots, st) : dispatch_simt<float>(a, slots, st);
  } else {
    r = paged_attn_f32(a, s, max_new, st);
  }
  if (r != GDN_OK || !a.part) return r;
  return s.dtype == GDN_BF16 ? launch_join<__nv_bfloat16>(a, st) : launch_join<float>(a, st);
}

// paged_attn_f32.cu -- attention over a paged cache with fp32-level products on the tensor cores
// (mma.sync m16n8k8, TF32): fp32 inputs, and bf16 ones that the tcgen05 kernel does not take
// (widths, page sizes, strides and alignments of any kind).
//
// tcgen05 would need an fp32 operand's parts staged in shared memory; here K, V and Q lie there as they
// are (fp32) and are split in registers as fragments are loaded, x = hi + lo, both TF32, a product
// taking hi*hi + hi*lo + lo*hi (the dropped term is 2^-22 of it).  bf16 values are exact in TF32 and need no lo.
// The matrix instructions, three a product, and the splitting bound chunks: 24 ragged ones of up to 200 tokens (1957 in
// all) over 1000, 64/8 heads, D 256: 4.4 ms, 27 TFLOP/s, 81 of TF32 products (the CUDA-core kernel 14.4 ms).
// Single tokens wait on their own chain of products, eight of a warp's sixteen rows unused: 24 over 1000, 32/8 heads,
// D 128: 81 us, 36% of HBM.  Small calls are a chain of latencies: 5 chunks with a window of 200: 13 us.
//
// A block of four warps takes query rows of one sequence and kv head (row = token * group + head in the
// group) and one of `splits` parts of their positions, tile by tile of BN positions, the next tile's
// copies in flight under this one's products (cp.async, 16 bytes, where rows are so aligned).  With more than 16 rows
// a warp takes 16 of 64 rows; with up to 16 the warps take a quarter of each tile's positions
// instead and join at the end.  A running maximum and sum per row, in base 2.  P's accumulator layout serves as the
// second product's operand by taking V's rows in the order 0 2 4 6 1 3 5 7 of each eight.
// Positions that no row of the block sees are zeros in shared memory; a masked weight is an exact 0.
// Infinities and NaN: an infinite operand's parts are (inf, NaN), a masked 0 times one is NaN, and a row keeps a NaN to the
// end.  A block that ends with one (or with an infinity) works its rows out again in plain fp32, position by position of
// those that a row sees.
#include <algorithm>

#include "chunk_bwd_mma.cuh"
#include "common.cuh"
#include "paged.cuh"
#include "paged_attn.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

namespace tc = gdn_bwd::tc;
constexpr int kThreads = 128;

template <typename T, int DP, bool FEW>
struct Cfg {
  static constexpr bool kExact = sizeof(T) == 2;   // values exact in TF32
  static constexpr int R = FEW ? 16 : 64;
  // positions a tile (FEW: two blocks an SM; 24 single tokens over 1000, D 128: 81 us, 109 us with 64)
  static constexpr int BN = DP == 256 || FEW ? 32 : 64;
  static constexpr int kMine = FEW ? BN / 4 : BN;  // of them a warp's
  static constexpr int kPitch = DP + 4;            // floats a row: the fragments' loads meet no bank conflict
  static constexpr int kTile = BN * kPitch;
  static constexpr size_t kSmem = sizeof(float) * (R * kPitch + 4 * kTile) + 2 * BN * sizeof(int64_t);
};

// A row's values out: o / l and lse, or the part for the join.
__device__ __forceinline__ void put_stats(const SimtArgs &a, int64_t row, float top, float sum) {
  if (a.part) {
    float *pp = a.part + ((int64_t)blockIdx.z * a.seqs.n_tok * a.Hq + row) * (a.D + 2);
    pp[0] = top, pp[1] = sum;
  } else if (a.lse) {
    a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
  }
}
template <typename T>
__device__ __forceinline__ void put(const SimtArgs &a, int64_t row, int col, float x, float inv) {
  if (col >= a.D) return;
  if (a.part) a.part[((int64_t)blockIdx.z * a.seqs.n_tok * a.Hq + row) * (a.D + 2) + 2 + col] = x;
  else ((T *)a.o)[row * a.D + col] = from_f32<T>(x * inv);
}

// A block's R rows in plain fp32 on the CUDA cores, a warp a row, a lane holding the elements lane, lane + 32, ...  Apart
// from the kernel, whose registers it would crowd (bf16 of D 96, 10 chunks of 150 over 600: 215 us, 272 in line), and
// working out its item again, which the kernel then need not keep in memory.
template <typename T, int DP>
__device__ __noinline__ void plain_rows(const SimtArgs &a, int R) {
  constexpr int kE = DP / 32;
  const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv, h = blockIdx.y;
  const Item it = item_at(a.seqs, blockIdx.x, G, R, 1, a.window);
  const int begin = it.lo + (int)share_begin(it.hi - it.lo, blockIdx.z, a.splits);
  const int end = it.lo + (int)share_begin(it.hi - it.lo, blockIdx.z + 1, a.splits);
  const int32_t *table = a.table + (int64_t)it.s * a.table_stride;
  for (int r = threadIdx.x >> 5; r < it.rows; r += kThreads / 32) {
    const int row = it.row0 + r, tok = row / G, p = it.first + tok;
    const T *qp = (const T *)a.q + (int64_t)(it.t0 + tok) * a.q_stride + (int64_t)(h * G + row - tok * G) * a.D;
    float q[kE], acc[kE], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) q[e] = lane + 32 * e < a.D ? to_f32<T>(qp[lane + 32 * e]) : 0.f, acc[e] = 0.f;
    for (int j = a.window > 0 && p >= a.window ? max(p - a.window + 1, begin) : begin; j < min(p + 1, end); ++j) {
      const int page = page_of(table, j, a.page_size, a.max_pages, a.n_pages);
      if (page < 0) continue;
      const int64_t at = (int64_t)page * a.page_stride + (int64_t)(j % a.page_size) * a.slot_stride +
                         (int64_t)h * a.head_stride + lane;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (lane + 32 * e < a.D) x = fmaf(q[e], to_f32<T>(((const T *)a.k)[at + 32 * e]), x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= a.scale_log2;
      const float up = fmaxf(top, x), keep = top == -INFINITY ? 0.f : exp2f(top - up);
      const float w = x == -INFINITY ? 0.f : exp2f(x - up);
      top = up, sum = sum * keep + w;
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (lane + 32 * e < a.D) acc[e] = fmaf(acc[e], keep, w * to_f32<T>(((const T *)a.v)[at + 32 * e]));
    }
    const int64_t out = (int64_t)(it.t0 + tok) * a.Hq + h * G + row - tok * G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (lane == 0) put_stats(a, out, top, sum);
#pragma unroll
    for (int e = 0; e < kE; ++e) put<T>(a, out, lane + 32 * e, acc[e], inv);
  }
}

template <typename T, int DP, bool FEW>
__global__ void __launch_bounds__(kThreads) paged_attn_f32_kernel(const SimtArgs a, bool wide) {
  using C = Cfg<T, DP, FEW>;
  extern __shared__ __align__(16) float smem[];
  float *qs = smem, *ks = qs + C::R * C::kPitch, *vs = ks + 2 * C::kTile;
  int64_t *off = reinterpret_cast<int64_t *>(vs + 2 * C::kTile);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
  const int G = a.Hq / a.Hkv, h = blockIdx.y, part = blockIdx.z;
  sm100::launch_dependents();
  sm100::grid_dependency_wait();
  const Item it = item_at(a.seqs, blockIdx.x, G, C::R, 1, a.window);  // tiles of one position
  if (!it.ok && tid == 0) set_status(a.status, GDN_ERR_BOUNDS);
  if (it.rows <= 0) return;
  const int begin = it.lo + (int)share_begin(it.hi - it.lo, part, a.splits);
  const int end = it.lo + (int)share_begin(it.hi - it.lo, part + 1, a.splits);
  const int n_tiles = (max(end - begin, 0) + C::BN - 1) / C::BN;
  const int32_t *table = a.table + (int64_t)it.s * a.table_stride;

  // where a position's rows lie in the caches, -1: not read
  auto places = [&](int tile) {
    if (tid < C::BN) {
      const int p = begin + tile * C::BN + tid;
      int64_t at = -1;
      if (tile < n_tiles && p < end) {
        const int page = page_of(table, p, a.page_size, a.max_pages, a.n_pages);
        if (page < 0) set_status(a.status, GDN_ERR_BOUNDS);
        else at = (int64_t)page * a.page_stride + (int64_t)(p % a.page_size) * a.slot_stride + (int64_t)h * a.head_stride;
      }
      off[(tile & 1) * C::BN + tid] = at;
    }
  };
  // four values of a row into shared memory (col < D), zeros where there are none
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
  auto load = [&](int tile) {
    const int st = tile & 1;
    for (int i = tid; i < C::BN * (DP / 4); i += kThreads) {
      const int r = i / (DP / 4), col = (i - r * (DP / 4)) * 4;
      const int64_t at = off[st * C::BN + r];
      float *k = ks + st * C::kTile + r * C::kPitch + col, *v = vs + st * C::kTile + r * C::kPitch + col;
      if (at >= 0 && col < a.D) {
        put4(k, (const T *)a.k + at, col);
        put4(v, (const T *)a.v + at, col);
      } else {
        *reinterpret_cast<float4 *>(k) = *reinterpret_cast<float4 *>(v) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    cp_async_commit();
  };
  places(0);
  for (int i = tid; i < C::R * (DP / 4); i += kThreads) {
    const int r = i / (DP / 4), col = (i - r * (DP / 4)) * 4;
    float *to = qs + r * C::kPitch + col;
    if (r < it.rows && col < a.D) {
      const int row = it.row0 + r, tok = row / G;
      put4(to, (const T *)a.q + (int64_t)(it.t0 + tok) * a.q_stride + (int64_t)(h * G + row - tok * G) * a.D, col);
    } else {
      *reinterpret_cast<float4 *>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __syncthreads();
  load(0);

  // this lane's rows (of the fragment layout): m0 + g4 and m0 + g4 + 8
  const int m0 = FEW ? 0 : warp * 16, n0 = FEW ? warp * C::kMine : 0;
  int lo[2], hi[2];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = m0 + g4 + 8 * e, p = it.first + (it.row0 + r) / G;
    hi[e] = r < it.rows ? min(p + 1, end) : 0;
    lo[e] = a.window > 0 && p >= a.window ? max(p - a.window + 1, begin) : begin;
  }
  float o[DP / 8][4];
#pragma unroll
  for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  for (int tile = 0; tile < n_tiles; ++tile) {
    places(tile + 1);
    cp_async_wait_all();
    __syncthreads();  // this tile is there, the next one's places too, and the tile before is done with
    if (tile + 1 < n_tiles) load(tile + 1);
    const float *k = ks + (tile & 1) * C::kTile + n0 * C::kPitch, *v = vs + (tile & 1) * C::kTile + n0 * C::kPitch;
    const int pos = begin + tile * C::BN + n0;

    // The MMAs' accumulation cuts off where an fp32 addition rounds, always towards zero, so a sum is made of parts of
    // four steps (with few rows, where a warp has one product at a time, of one: four that do not wait for each
    // other), added by fp32 additions: an error of 6.6e-7 for chunks of 40 over 6000, D 128, and of 3.1e-6 with one
    // chain of MMAs (fp32 products and sums in a library's order: 1.4e-6; with a window of 200 5.9e-7 to its
    // 3.5e-7).  It costs 4.4 ms for 3.95 at D 256.
    constexpr int kParts = FEW ? 4 : 1;
    float s[C::kMine / 8][4];
#pragma unroll
    for (int i = 0; i < C::kMine / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < DP; k0 += 32) {
      float x[kParts][C::kMine / 8][4];
#pragma unroll
      for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int i = 0; i < C::kMine / 8; ++i) x[c][i][0] = x[c][i][1] = x[c][i][2] = x[c][i][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 32; kk += 8) {
        const float *q = qs + (m0 + g4) * C::kPitch + k0 + kk + t4;
        tc::FragA fa;
        if constexpr (C::kExact) tc::frag_a_exact(fa, q[0], q[8 * C::kPitch], q[4], q[8 * C::kPitch + 4]);
        else tc::frag_a(fa, q[0], q[8 * C::kPitch], q[4], q[8 * C::kPitch + 4]);
#pragma unroll
        for (int i = 0; i < C::kMine / 8; ++i) {
          const float *b = k + (i * 8 + g4) * C::kPitch + k0 + kk + t4;
          tc::FragB fb;
          if constexpr (C::kExact) tc::frag_b_exact(fb, b[0], b[4]);
          else tc::frag_b(fb, b[0], b[4]);
          tc::mma_x<C::kExact, C::kExact>(x[kk / 8 % kParts][i], fa, fb);
        }
      }
#pragma unroll
      for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int i = 0; i < C::kMine / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] += x[c][i][e];
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < C::kMine / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = pos + i * 8 + 2 * t4 + (e & 1);
        s[i][e] = p >= lo[e >> 1] && p < hi[e >> 1] ? s[i][e] * a.scale_log2 : -INFINITY;
        top[e >> 1] = fmaxf(top[e >> 1], s[i][e]);
      }
    float keep[2], base[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      top[e] = fmaxf(top[e], m[e]);
      keep[e] = m[e] == -INFINITY ? 0.f : exp2f(m[e] - top[e]);
      base[e] = top[e] == -INFINITY ? 0.f : top[e];
      m[e] = top[e];
      l[e] *= keep[e];
    }
    tc::FragA pa[C::kMine / 8];  // columns 2t, 2t + 1 of P as the operand's t, t + 4
#pragma unroll
    for (int j = 0; j < C::kMine / 8; ++j) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = exp2f(s[j][e] - base[e >> 1]);
        l[e >> 1] += p[e];
      }
      tc::frag_a(pa[j], p[0], p[2], p[1], p[3]);
    }
    // four columns' products of the tile side by side, then onto the scaled sums
#pragma unroll
    for (int i0 = 0; i0 < DP / 8; i0 += 4) {
      float x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
      for (int j = 0; j < C::kMine / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float *b = v + (j * 8 + 2 * t4) * C::kPitch + (i0 + i) * 8 + g4;
          tc::FragB fb;
          if constexpr (C::kExact) tc::frag_b_exact(fb, b[0], b[C::kPitch]);
          else tc::frag_b(fb, b[0], b[C::kPitch]);
          tc::mma_x<false, C::kExact>(x[i], pa[j], fb);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i0 + i][e] = fmaf(o[i0 + i][e], keep[e >> 1], x[i][e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
  }

  auto out_row = [&](int r) {
    const int row = it.row0 + r, tok = row / G;
    return (int64_t)(it.t0 + tok) * a.Hq + h * G + row - tok * G;
  };
  float odd = 0.f;  // NaN where a row of the item's has a NaN or an infinity
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (m0 + g4 + 8 * e < it.rows) {
      odd = fmaf(l[e], 0.f, odd);
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) odd = fmaf(o[i][2 * e], 0.f, fmaf(o[i][2 * e + 1], 0.f, odd));
    }
  if (__syncthreads_or(isnan(odd))) return plain_rows<T, DP>(a, C::R);
  if constexpr (!FEW) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = m0 + g4 + 8 * e;
      if (r >= it.rows) continue;
      const int64_t row = out_row(r);
      const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
      if (t4 == 0) put_stats(a, row, m[e], l[e]);
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        put<T>(a, row, i * 8 + 2 * t4, o[i][2 * e], inv);
        put<T>(a, row, i * 8 + 2 * t4 + 1, o[i][2 * e + 1], inv);
      }
    }
  } else {
    // the warps' sums over their positions join in shared memory
    cp_async_wait_all();
    __syncthreads();
    float *acc = ks, *ml = qs;  // [4][16][kPitch], [4][16][2]
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g4 + 8 * e;
      if (t4 == 0) ml[(warp * 16 + r) * 2] = m[e], ml[(warp * 16 + r) * 2 + 1] = l[e];
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        acc[(warp * 16 + r) * C::kPitch + i * 8 + 2 * t4] = o[i][2 * e];
        acc[(warp * 16 + r) * C::kPitch + i * 8 + 2 * t4 + 1] = o[i][2 * e + 1];
      }
    }
    __syncthreads();
    for (int r = warp; r < it.rows; r += 4) {
      float top = -INFINITY, sum = 0.f, w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, ml[(i * 16 + r) * 2]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float li = ml[(i * 16 + r) * 2 + 1];
        w[i] = li == 0.f ? 0.f : exp2f(ml[(i * 16 + r) * 2] - top);
        sum += w[i] * li;
      }
      const int64_t row = out_row(r);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (lane == 0) put_stats(a, row, top, sum);
      for (int col = lane; col < a.D; col += 32) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x += w[i] == 0.f ? 0.f : w[i] * acc[(i * 16 + r) * C::kPitch + col];
        put<T>(a, row, col, x, inv);
      }
    }
  }
}

template <typename T, int DP, bool FEW>
gdn_status launch(const SimtArgs &a, bool wide, cudaStream_t st) {
  using C = Cfg<T, DP, FEW>;
  const auto kernel = paged_attn_f32_kernel<T, DP, FEW>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
    return (void)cudaGetLastError(), GDN_ERR_CUDA;
  const int64_t slots = item_slots(a.seqs.n_tok, a.seqs.n_seqs, a.Hq / a.Hkv, C::R);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)slots, a.Hkv, a.splits), cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem, cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the launch overlaps the end of the kernel before
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, a, wide);
  return launch_status();
}

template <typename T>
gdn_status dispatch(const SimtArgs &a, bool few, bool wide, cudaStream_t st) {
  if (a.D <= 64) return few ? launch<T, 64, true>(a, wide, st) : launch<T, 64, false>(a, wide, st);
  if (a.D <= 128) return few ? launch<T, 128, true>(a, wide, st) : launch<T, 128, false>(a, wide, st);
  return few ? launch<T, 256, true>(a, wide, st) : launch<T, 256, false>(a, wide, st);
}

// 16 rows a block where the longest chunk has no more, else 64
bool few_rows(const gdn_cache_shape &s, int32_t max_new) { return (int64_t)max_new * (s.Hq / s.Hkv) <= 16; }

}  // namespace

// Parts that a block's positions are cut into: two blocks an SM (three with few rows), no part below 64 positions of
// the longest span that the table and the window allow, at most 64.  Single tokens of 24 sequences over 1000, D 128:
// 81 us, 143 us with two blocks an SM (of 4 over 8000: 105 and 136); 5 chunks of up to 37 over 700 with a window of 200,
// D 64: 12.8 us, 17.6 us with parts from 128 positions on.
int paged_attn_f32_splits(const gdn_cache_shape &s, int32_t max_new, int32_t window) {
  const bool few = few_rows(s, max_new);
  const int64_t blocks = item_slots(s.n_tok, s.n_seqs, s.Hq / s.Hkv, few ? 16 : 64) * s.Hkv;
  const int64_t want = (152 * (few ? 3 : 2) + blocks - 1) / std::max<int64_t>(blocks, 1);
  int64_t span = (int64_t)s.max_pages * s.page_size;
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + std::min<int64_t>(max_new, 64));
  return (int)std::max<int64_t>(1, std::min<int64_t>({64, want, (span + 63) / 64}));
}

gdn_status paged_attn_f32(const SimtArgs &a, const gdn_cache_shape &s, int32_t max_new, cudaStream_t st) {
  bool wide = s.D % 4 == 0;
  for (const void *p : {a.q, a.k, a.v}) wide = wide && aligned(p, 16);
  for (int64_t x : {a.q_stride, a.page_stride, a.slot_stride, a.head_stride}) wide = wide && x % 4 == 0;
  const bool few = few_rows(s, max_new);
  if (s.dtype == GDN_BF16) return dispatch<__nv_bfloat16>(a, few, wide, st);
  return dispatch<float>(a, few, wide, st);
}

}  // namespace gdn

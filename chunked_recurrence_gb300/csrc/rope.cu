// rope.cu -- rotary positions of q and k (gdn_rope, forward and gradient) and the same on the
// way of new tokens into a paged cache (gdn_kv_append).
//
// A pair (x1, x2) of a head at position p turns by a = p * inv_freq:
//     y1 = s (x1 cos a - x2 sin a),   y2 = s (x2 cos a + x1 sin a);
// the gradient is the transposed rotation, the same with sin a negated.
//
// The angle is kept in turns as a 64-bit fraction: p * freq mod 2^64, one integer multiply, exact for
// every 64-bit position, of which the top 32 bits are used; freq itself is rounded, by 2^-65 turns at most
// (p * 2^-65 in the angle).  A product in fp32 would be off by p * 2^-25 rad.
//
// Bound by HBM: every element is read and written once.  A warp takes a token: it works out
// the token's cos and sin once for all heads (through its own piece of shared memory, no block
// barrier), then walks the heads.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "conv_tap.cuh"
#include "paged.cuh"
#include "sm100.cuh"

using namespace gdn;

namespace {

// Two heads a lane in flight and three blocks an SM (80 registers): 29.5 us over the rows of 8192 tokens x 40 heads x
// 128 bf16 (168 MB, 5.8 TB/s); four heads and two blocks 29.4 us, four blocks 31 us, without the rows' prefetch 31.4 us.
constexpr int kThreads = 256, kHeads = 2;

struct RopeArgs {
  const void *q, *k, *v;  // v: gdn_kv_append only
  void *qo, *ko, *vo;     // ko, vo: the caches for gdn_kv_append
  const int64_t *positions;
  const uint64_t *freqs;
  int32_t n_tok, Hq, Hk, Hv, D, rd;
  int64_t qs, ks, vs, qos, kos;  // token strides
  float scale, sign;
  int32_t copy_q, copy_k;  // elements past rd are copied (not when in place)
  // gdn_kv_append
  PagedSeqs seqs;
  const int32_t *table;
  int64_t table_stride, page_stride, slot_stride, head_stride;
  int32_t page_size, max_pages, n_pages;
  int32_t *status;
};

template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Vec {
  T v[VEC];
};

// The sequence of a new token, by a whole warp: 32 probes a round.  The largest s with cu[s] <= t.
__device__ __forceinline__ int seq_of_token_warp(const int32_t *cu, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seqs;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const uint32_t below = __ballot_sync(0xffffffffu, lane * step < n && cu[lo + lane * step] <= t);
    const int k = below ? 31 - __clz(below) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Where a new token goes: its position (where the call gives none) and the offset of its slot in
// the caches, -1 for none.  A whole warp asks for the same token.
__device__ __forceinline__ int64_t append_slot(const RopeArgs &a, int t, int64_t &pos) {
  const int s = a.seqs.cu ? seq_of_token_warp(a.seqs.cu, a.seqs.n_seqs, t) : t;
  const SeqSpan sp = seq_span(a.seqs, s);
  const int32_t at = sp.len - sp.n_new + (t - sp.t0);
  pos = at;
  if (!sp.ok || t < sp.t0 || t >= sp.t0 + sp.n_new) {
    set_status(a.status, GDN_ERR_BOUNDS);
    return -1;
  }
  if (at < 0) return -1;
  const int32_t page = page_of(a.table + (int64_t)s * a.table_stride, at, a.page_size, a.max_pages, a.n_pages);
  if (page < 0) {
    set_status(a.status, GDN_ERR_BOUNDS);
    return -1;
  }
  return (int64_t)page * a.page_stride + (int64_t)(at % a.page_size) * a.slot_stride;
}

// cos and sin of a fraction of a turn, as a signed 32-bit fraction: the eighths of the circle by
// its top bits, then the Taylor series on [-pi/4, pi/4] (the first term left out is below 2^-25).
__device__ __forceinline__ float2 cos_sin(uint32_t turn) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;  // nearest quarter of the circle
  const float y = (float)(int32_t)(turn - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), z = y * y;
  float s = fmaf(z, 1.f / 362880, -1.f / 5040), c = fmaf(z, 1.f / 40320, -1.f / 720);
  s = fmaf(z, s, 1.f / 120), c = fmaf(z, c, 1.f / 24);
  s = fmaf(z, s, -1.f / 6), c = fmaf(z, c, -0.5f);
  s = fmaf(y * z, s, y), c = fmaf(z, c, 1.f);
  const float co = (quarter & 1) ? s : c, si = (quarter & 1) ? c : s;
  return make_float2((quarter + 1) & 2 ? -co : co, quarter & 2 ? -si : si);
}

// Turns a place: pairs (x1[j], x2[j]) of two vectors.  bf16 vectors of eight go as fp32 pairs.
template <typename T, int VEC, int P>
__device__ __forceinline__ void turn_halves(Vec<T, VEC> &x1, Vec<T, VEC> &x2, const float (&cn)[P], const float (&sn)[P]) {
  if constexpr (sizeof(T) == 2 && VEC == 8) {
    uint32_t *a = reinterpret_cast<uint32_t *>(&x1), *b = reinterpret_cast<uint32_t *>(&x2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t u = f2_from_bf16x2(a[j]), z = f2_from_bf16x2(b[j]);
      const uint64_t c = f2_pack(cn[2 * j], cn[2 * j + 1]), s = f2_pack(sn[2 * j], sn[2 * j + 1]);
      const uint64_t ns = f2_pack(-sn[2 * j], -sn[2 * j + 1]);
      a[j] = bf16x2_from_f2(f2_fma(u, c, f2_mul(z, ns)));
      b[j] = bf16x2_from_f2(f2_fma(z, c, f2_mul(u, s)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float u = to_f32<T>(x1.v[j]), z = to_f32<T>(x2.v[j]);
      x1.v[j] = from_f32<T>(u * cn[j % P] - z * sn[j % P]);
      x2.v[j] = from_f32<T>(z * cn[j % P] + u * sn[j % P]);
    }
  }
}
// The same for neighbours (x[2j], x[2j + 1]) in one vector.
template <typename T, int VEC, int P>
__device__ __forceinline__ void turn_neighbours(Vec<T, VEC> &x, const float (&cn)[P], const float (&sn)[P]) {
  if constexpr (sizeof(T) == 2 && VEC == 8) {
    uint32_t *a = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u, z;
      f2_unpack(f2_from_bf16x2(a[j]), u, z);
      a[j] = bf16x2_from_f2(f2_pack(u * cn[j] - z * sn[j], z * cn[j] + u * sn[j]));
    }
  } else {
#pragma unroll
    for (int j = 0; j + 1 < VEC; j += 2) {
      const float u = to_f32<T>(x.v[j]), z = to_f32<T>(x.v[j + 1]);
      x.v[j] = from_f32<T>(u * cn[j / 2] - z * sn[j / 2]);
      x.v[j + 1] = from_f32<T>(z * cn[j / 2] + u * sn[j / 2]);
    }
  }
}

__device__ __forceinline__ void prefetch_row(const void *p, int64_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)bytes) : "memory");
}

// A warp takes a token, or one of `parts` parts of its heads and vectors, dealt out in turn (134 MB appended, 5460
// tokens in two parts: 27.1 us; 29.3 us with the parts' heads and vectors in blocks of as many as a lane has in
// flight).  In a rotary column place a lane holds VEC pairs of a head in the half layout (two vectors), VEC / 2 pairs
// interleaved (one vector; VEC = 1: one pair as two vectors of one element); 32 / rot heads go side by side over the
// lanes.
template <typename T, int VEC, bool APPEND, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeArgs a, int parts) {
  constexpr int kPairs = INTER ? (VEC + 1) / 2 : VEC;  // of a place
  __shared__ float2 s_cs[kThreads / 32][128];
  const int lane = threadIdx.x & 31, half = a.rd >> 1;
  const int64_t job = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int t = (int)(job / parts), part = (int)(job - (int64_t)t * parts);
  sm100::grid_dependency_wait();
  if (t >= a.n_tok) return;
  float2 *cs = s_cs[threadIdx.x >> 5];
  const T *q = (const T *)a.q + t * a.qs, *k = (const T *)a.k + t * a.ks;
  T *qo = (T *)a.qo + t * a.qos, *ko = (T *)a.ko + (APPEND ? 0 : t * a.kos);
  const int64_t k_head = APPEND ? a.head_stride : a.D;
  if (VEC > 1 && part == 0 && lane < 3) {  // the token's rows on their way into L2
    if (lane == 0 && a.Hq) prefetch_row(q, (int64_t)a.Hq * a.D * sizeof(T));
    if (lane == 1 && a.Hk) prefetch_row(k, (int64_t)a.Hk * a.D * sizeof(T));
    if (lane == 2 && APPEND) prefetch_row((const T *)a.v + t * a.vs, (int64_t)a.Hv * a.D * sizeof(T));
  }
  const uint64_t freq0 = lane < half ? a.freqs[lane] : 0;  // on its way while the token's place is looked up
  int64_t pos = 0, slot = 0;
  if (APPEND) {
    slot = append_slot(a, t, pos);
    ko += slot;
  }
  if (half && a.positions) pos = a.positions[t];
  for (int i = lane; i < half; i += 32) {
    const float2 f = cos_sin((uint32_t)(((uint64_t)pos * (i < 32 ? freq0 : a.freqs[i])) >> 32));
    cs[i] = make_float2(f.x * a.scale, f.y * a.scale * a.sign);
  }
  __syncwarp();

  // ---- what turns: columns [0, rd) of the heads of q, then of k
  const int heads = a.Hq + (APPEND && slot < 0 ? 0 : a.Hk);
  const int rot = half / kPairs;
  for (int c0 = 0; c0 < rot; c0 += 32) {
    const int cols = min(32, rot - c0), side = 32 / cols, c = c0 + lane % cols, hl = lane / cols;
    const int e = INTER ? 2 * kPairs * c : VEC * c, apart = INTER ? 1 : half;
    constexpr bool two = !INTER || VEC == 1;
    float cn[kPairs], sn[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const float2 f = cs[c * kPairs + j];
      cn[j] = f.x, sn[j] = f.y;
    }
    for (int h0 = part * side + hl; h0 < heads; h0 += parts * side * kHeads) {
      Vec<T, VEC> x1[kHeads], x2[kHeads];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * parts * side;
        const T *x = (h < a.Hq ? q : k - a.Hq * a.D) + h * a.D + e;
        if (h < heads && hl < side) {
          x1[i] = *reinterpret_cast<const Vec<T, VEC> *>(x);
          if (two) x2[i] = *reinterpret_cast<const Vec<T, VEC> *>(x + apart);
        }
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * parts * side;
        T *y = h < a.Hq ? qo + h * a.D + e : ko + (h - a.Hq) * k_head + e;
        if constexpr (two) turn_halves(x1[i], x2[i], cn, sn);
        else turn_neighbours(x1[i], cn, sn);
        if (h < heads && hl < side) {
          *reinterpret_cast<Vec<T, VEC> *>(y) = x1[i];
          if (two) *reinterpret_cast<Vec<T, VEC> *>(y + apart) = x2[i];
        }
      }
    }
  }

  // ---- what passes through: columns [rd, D) of q and k where they are not in place, all of v
  auto copy = [&](const T *x, T *y, int64_t y_head, int n_heads, int from) {
    const int cols = (a.D - from) / VEC, all = n_heads * cols;
    constexpr int kAhead = 4;
    // place i of a lane is (head h, column c); a step on, without a division
    const int step = 32 * parts, dh = step / cols, dc = step - dh * cols;
    for (int i0 = part * 32 + lane; i0 < all; i0 += step * kAhead) {
      Vec<T, VEC> v[kAhead];
      int h = i0 / cols, c = i0 - h * cols;
      const int h_first = h, c_first = c;
      auto next = [&]() {
        h += dh, c += dc;
        if (c >= cols) c -= cols, ++h;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i, next())
        if (h < n_heads) v[i] = *reinterpret_cast<const Vec<T, VEC> *>(x + h * a.D + from + c * VEC);
      h = h_first, c = c_first;
#pragma unroll
      for (int i = 0; i < kAhead; ++i, next())
        if (h < n_heads) *reinterpret_cast<Vec<T, VEC> *>(y + h * y_head + from + c * VEC) = v[i];
    }
  };
  if (a.rd < a.D) {
    if (a.copy_q) copy(q, qo, a.D, a.Hq, a.rd);
    if (a.copy_k && !(APPEND && slot < 0)) copy(k, ko, k_head, a.Hk, a.rd);
  }
  if (APPEND && slot >= 0) copy((const T *)a.v + t * a.vs, (T *)a.vo + slot, a.head_stride, a.Hv, 0);
}

template <typename T, int VEC, bool APPEND>
gdn_status launch_vec(const RopeArgs &a, bool inter, cudaStream_t st) {
  // a token's heads over several warps where the tokens alone would not fill the GPU some three times over
  const int parts = std::max(1, std::min((a.Hq + a.Hk + a.Hv + 7) / 8, 152 * 80 / a.n_tok));
  const int64_t blocks = ((int64_t)a.n_tok * parts * 32 + kThreads - 1) / kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks), cfg.blockDim = dim3(kThreads), cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the launch overlaps the end of the kernel before
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, inter ? rope_kernel<T, VEC, APPEND, true> : rope_kernel<T, VEC, APPEND, false>, a, parts);
  return launch_status();
}

// 16-byte vectors where every row start, stride and part of a head is a multiple of them
template <typename T, bool APPEND>
gdn_status launch_type(const RopeArgs &a, bool inter, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int unit = inter ? a.rd : a.rd / 2;
  bool wide = a.D % V == 0 && a.rd % V == 0 && unit % V == 0 && a.qs % V == 0 && a.ks % V == 0 && a.vs % V == 0 &&
              a.qos % V == 0 && a.kos % V == 0;
  for (const void *p : {a.q, a.k, a.v, (const void *)a.qo, (const void *)a.ko, (const void *)a.vo})
    wide = wide && aligned(p, 16);
  if (APPEND) wide = wide && a.page_stride % V == 0 && a.slot_stride % V == 0 && a.head_stride % V == 0;
  return wide ? launch_vec<T, V, APPEND>(a, inter, st) : launch_vec<T, 1, APPEND>(a, inter, st);
}

bool rotary_ok(int32_t D, int32_t rd) { return D >= 1 && D <= 256 && rd >= 0 && rd <= D && rd % 2 == 0; }

}  // namespace

extern "C" gdn_status gdn_rope_inv_freq(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                        double orig_len, double alpha, double beta, double *inv_freq) {
  if (!inv_freq || rotary_dim < 2 || rotary_dim % 2 || !(base > 0) || scaling < GDN_ROPE_NONE ||
      scaling > GDN_ROPE_PARTS)
    return GDN_ERR_INVALID_ARG;
  if (scaling != GDN_ROPE_NONE && !(factor > 0)) return GDN_ERR_INVALID_ARG;
  if (scaling == GDN_ROPE_BASE && rotary_dim == 2) return GDN_ERR_INVALID_ARG;
  if (scaling == GDN_ROPE_PARTS && (!(beta > alpha) || !(orig_len > 0))) return GDN_ERR_INVALID_ARG;
  if (scaling == GDN_ROPE_BASE) base *= pow(factor, (double)rotary_dim / (rotary_dim - 2));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double inv = pow(base, -2.0 * i / rotary_dim);
    if (scaling == GDN_ROPE_LINEAR) inv /= factor;
    if (scaling == GDN_ROPE_PARTS) {
      const double g = fmin(1.0, fmax(0.0, (orig_len * inv / (2 * M_PI) - alpha) / (beta - alpha)));
      inv = (1 - g) * inv / factor + g * inv;
    }
    inv_freq[i] = inv;
  }
  return GDN_OK;
}

namespace {

// 1 / 2 pi as a binary fraction, 192 bits in words from the lowest (pi by Machin's formula in whole numbers).
constexpr uint64_t kTurn[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};

// inv / 2 pi as a 64-bit fraction, rounded to nearest: inv = m 2^e with a whole m of 53 bits and e <= 0, and m / 2 pi to
// 192 bits after the point (243 in all), so that what is cut off stays below 2^-75 of the result's last bit.
uint64_t turns_word(double inv) {
  int e;
  const uint64_t m = (uint64_t)ldexp(frexp(fabs(inv), &e), 53);
  uint64_t p[5] = {};
  unsigned __int128 c = 0;
  for (int i = 0; i < 3; ++i, c >>= 64) c += (unsigned __int128)m * kTurn[i], p[i] = (uint64_t)c;
  p[3] = (uint64_t)c;
  const int at = 128 - (e - 53), i = at / 64, b = at % 64;  // the result is bits [at, at + 64) of p
  if (at > 255) return 0;
  const uint64_t half = p[(at - 1) / 64] >> ((at - 1) % 64) & 1;
  const uint64_t w = (p[i] >> b | (b ? p[i + 1] << (64 - b) : 0)) + half;
  return inv < 0 ? 0 - w : w;
}

}  // namespace

extern "C" gdn_status gdn_rope_freqs(const double *inv_freq, int32_t n, uint64_t *freqs) {
  if (n < 0 || (n > 0 && (!inv_freq || !freqs))) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (!(fabs(inv_freq[i]) < 0x1p53)) return GDN_ERR_INVALID_ARG;  // nor NaN
    freqs[i] = turns_word(inv_freq[i]);
  }
  return GDN_OK;
}

extern "C" gdn_status gdn_rope(const void *q, const void *k, const int64_t *positions, const uint64_t *freqs,
                               int32_t dtype, int32_t n_tok, int32_t Hq, int32_t Hk, int32_t D, int32_t rotary_dim,
                               int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                               float scale, uint32_t flags, void *q_out, void *k_out, void *stream) {
  if ((dtype != GDN_F32 && dtype != GDN_BF16) || n_tok < 0 || Hq < 0 || Hk < 0 || !rotary_ok(D, rotary_dim))
    return GDN_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(GDN_FLAG_ROPE_INTERLEAVED | GDN_FLAG_ROPE_BACKWARD)) return GDN_ERR_INVALID_ARG;
  if (((int64_t)Hq + Hk) * D >= 1 << 29) return GDN_ERR_UNSUPPORTED;  // places and bytes within a token: 32 bits
  RopeArgs a{};
  a.qs = q_stride ? q_stride : (int64_t)Hq * D;
  a.ks = k_stride ? k_stride : (int64_t)Hk * D;
  a.qos = q_out_stride ? q_out_stride : (int64_t)Hq * D;
  a.kos = k_out_stride ? k_out_stride : (int64_t)Hk * D;
  if (a.qs < (int64_t)Hq * D || a.ks < (int64_t)Hk * D || a.qos < (int64_t)Hq * D || a.kos < (int64_t)Hk * D)
    return GDN_ERR_INVALID_ARG;
  if (n_tok == 0 || Hq + Hk == 0) return GDN_OK;
  if ((Hq > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)) || !positions || (rotary_dim > 0 && !freqs))
    return GDN_ERR_INVALID_ARG;
  if ((Hq > 0 && q == q_out && a.qs != a.qos) || (Hk > 0 && k == k_out && a.ks != a.kos)) return GDN_ERR_INVALID_ARG;
  a.q = Hq ? q : nullptr, a.k = Hk ? k : nullptr;
  a.qo = Hq ? q_out : nullptr, a.ko = Hk ? k_out : nullptr;
  a.positions = positions, a.freqs = freqs;
  a.n_tok = n_tok, a.Hq = Hq, a.Hk = Hk, a.D = D, a.rd = rotary_dim;
  a.scale = scale, a.sign = (flags & GDN_FLAG_ROPE_BACKWARD) ? -1.f : 1.f;
  a.copy_q = q != q_out, a.copy_k = k != k_out;
  const bool inter = flags & GDN_FLAG_ROPE_INTERLEAVED;
  if (dtype == GDN_BF16) return launch_type<__nv_bfloat16, false>(a, inter, (cudaStream_t)stream);
  return launch_type<float, false>(a, inter, (cudaStream_t)stream);
}

namespace gdn {
gdn_status normalise_cache_shape(const gdn_cache_shape *in, const int32_t *cu_seqlens, gdn_cache_shape *out);
PagedSeqs paged_seqs(const gdn_cache_shape &s, const int32_t *seq_lens, const int32_t *cu_seqlens);
}  // namespace gdn

extern "C" gdn_status gdn_kv_append(const void *q, const void *k, const void *v, const int64_t *positions,
                                    const uint64_t *freqs, int32_t rotary_dim, float scale, uint32_t flags,
                                    const int32_t *page_table, const int32_t *seq_lens, const int32_t *cu_seqlens,
                                    const gdn_cache_shape *shape, void *q_out, void *k_cache, void *v_cache,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  gdn_cache_shape s;
  const gdn_status ok = normalise_cache_shape(shape, cu_seqlens, &s);
  if (ok != GDN_OK) return ok;
  if (flags & ~(uint32_t)GDN_FLAG_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
  if (!rotary_ok(s.D, rotary_dim) || (!freqs && rotary_dim != 0)) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < 256 || !aligned(workspace, 256)) return GDN_ERR_WORKSPACE;
  if (s.n_tok == 0 || s.n_seqs == 0) return GDN_OK;
  if (!k || !v || !k_cache || !v_cache || !page_table || !seq_lens || (q && !q_out)) return GDN_ERR_INVALID_ARG;
  if (q && q == q_out && s.q_stride != (int64_t)s.Hq * s.D) return GDN_ERR_INVALID_ARG;
  RopeArgs a{};
  a.q = q, a.k = k, a.v = v, a.qo = q ? q_out : nullptr, a.ko = k_cache, a.vo = v_cache;
  a.positions = positions, a.freqs = freqs;
  a.n_tok = s.n_tok, a.Hq = q ? s.Hq : 0, a.Hk = a.Hv = s.Hkv, a.D = s.D, a.rd = rotary_dim;
  a.qs = s.q_stride, a.ks = s.k_stride, a.vs = s.v_stride, a.qos = (int64_t)s.Hq * s.D;
  a.scale = scale, a.sign = 1.f;
  a.copy_q = q != q_out, a.copy_k = 1;
  a.seqs = paged_seqs(s, seq_lens, cu_seqlens);
  a.table = page_table, a.table_stride = s.table_stride;
  a.page_stride = s.page_stride, a.slot_stride = s.slot_stride, a.head_stride = s.head_stride;
  a.page_size = s.page_size, a.max_pages = s.max_pages, a.n_pages = s.n_pages;
  a.status = s.status ? s.status : (int32_t *)workspace;
  const bool inter = flags & GDN_FLAG_ROPE_INTERLEAVED;
  if (s.dtype == GDN_BF16) return launch_type<__nv_bfloat16, true>(a, inter, (cudaStream_t)stream);
  return launch_type<float, true>(a, inter, (cudaStream_t)stream);
}

// rope.cu -- rotary positions of q and k (gdn_rope, forward and gradient) and the same on the
// way of new tokens into a paged cache (gdn_kv_append).
//
// A pair (x1, x2) of a head at position p turns by a = p * inv_freq:
//     y1 = s (x1 cos a - x2 sin a),   y2 = s (x2 cos a + x1 sin a);
// the gradient is the transposed rotation, the same with sin a negated.
//
// The angle is kept in turns as a 64-bit fraction: p * freq mod 2^64, one integer multiply,
// exact for every 64-bit position; its top 32 bits (signed, so [-1/2, 1/2) turns) go to
// sincospif.  A product in fp32 would be off by p * 2^-25 rad.
//
// Bound by HBM: every element is read and written once.  A block takes up to four tokens; its
// threads put the tokens' cos and sin into shared memory (one sincospif a pair and token, shared
// by all heads), and each thread keeps one place of a token's row (a 16-byte vector of pair halves,
// or of elements that pass through).
#include <math.h>

#include "common.cuh"
#include "paged.cuh"

using namespace gdn;

namespace {

constexpr int kMaxThreads = 512;

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
    const int step = (n + 31) / 32, s = lo + lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, lane * step < n && cu[s] <= t);
    const int k = below ? 31 - __clz(below) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// One place of a token's row: element offset of the vector in its head and what happens there.
// VEC elements a vector; half layout: a rotary place holds VEC pairs (two vectors), interleaved:
// VEC / 2 pairs (one vector; VEC = 1 then holds one pair as two vectors of one element).
// A thread loads its place of all the block's tokens before the angles are worked out, so that
// those (and the look-up of the slots) run under the loads.
template <typename T, int VEC, bool APPEND, bool INTER, int TOK>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(const RopeArgs a) {
  extern __shared__ float2 cs[];  // [TOK][rd / 2]
  __shared__ int64_t s_row[TOK];  // gdn_kv_append: offset of the token's slot in the caches, -1: none
  __shared__ int64_t s_pos[TOK];
  const int t0 = blockIdx.x * TOK, nt = min(TOK, a.n_tok - t0);
  const int half = a.rd >> 1;
  const int rot = INTER && VEC > 1 ? a.rd / VEC : half / VEC;  // rotary places of a head
  const int rest = (a.D - a.rd) / VEC;
  const int nq = rot + (a.copy_q ? rest : 0), nk = rot + (a.copy_k ? rest : 0), nv = APPEND ? a.D / VEC : 0;
  const int places = a.Hq * nq + a.Hk * nk + a.Hv * nv;

  const T *in;
  T *out;
  int64_t os;
  int c, kind;  // kind 0: q, 1: k, 2: v
  bool turn, two;
  int apart;  // second vector (half layout, or VEC = 1)
  Vec<T, VEC> x1[TOK], x2[TOK];
  auto load = [&](int pl) {
    int h;
    int64_t is;
    os = 0;
    if (pl < a.Hq * nq) {
      h = pl / nq, c = pl - h * nq, kind = 0;
      in = (const T *)a.q + (int64_t)h * a.D, is = a.qs;
      out = (T *)a.qo + (int64_t)h * a.D, os = a.qos;
    } else if (pl < a.Hq * nq + a.Hk * nk) {
      const int r = pl - a.Hq * nq;
      h = r / nk, c = r - h * nk, kind = 1;
      in = (const T *)a.k + (int64_t)h * a.D, is = a.ks;
      out = (T *)a.ko + (APPEND ? (int64_t)h * a.head_stride : (int64_t)h * a.D), os = a.kos;
    } else {
      const int r = pl - a.Hq * nq - a.Hk * nk;
      h = APPEND ? r / max(nv, 1) : 0, c = r - h * nv, kind = 2;
      in = (const T *)a.v + (int64_t)h * a.D, is = a.vs;
      out = (T *)a.vo + (int64_t)h * a.head_stride;
    }
    turn = kind != 2 && c < rot;
    two = turn && (!INTER || VEC == 1);
    const int e = turn ? (INTER && VEC == 1 ? 2 * c : c * VEC) : (kind == 2 ? c * VEC : a.rd + (c - rot) * VEC);
    apart = INTER ? 1 : half;
    in += (int64_t)t0 * is + e;
    out += e;
#pragma unroll
    for (int t = 0; t < TOK; ++t)
      if (t < nt) {
        x1[t] = *reinterpret_cast<const Vec<T, VEC> *>(in + t * is);
        if (two) x2[t] = *reinterpret_cast<const Vec<T, VEC> *>(in + t * is + apart);
      }
  };
  int pl = threadIdx.x;
  if (pl < places) load(pl);

  if (APPEND) {
    for (int i = threadIdx.x >> 5; i < nt; i += blockDim.x >> 5) {  // a warp a token
      const int t = t0 + i, s = a.seqs.cu ? seq_of_token_warp(a.seqs.cu, a.seqs.n_seqs, t) : t;
      if ((threadIdx.x & 31) == 0) {
        const SeqSpan sp = seq_span(a.seqs, s);
        const int32_t at = sp.len - sp.n_new + (t - sp.t0);
        const bool mine = t >= sp.t0 && t < sp.t0 + sp.n_new;
        int64_t row = -1;
        if (!sp.ok || !mine) {
          set_status(a.status, GDN_ERR_BOUNDS);
        } else if (at >= 0) {
          const int32_t page = page_of(a.table + (int64_t)s * a.table_stride, at, a.page_size, a.max_pages, a.n_pages);
          if (page < 0) set_status(a.status, GDN_ERR_BOUNDS);
          else row = (int64_t)page * a.page_stride + (int64_t)(at % a.page_size) * a.slot_stride;
        }
        s_row[i] = row;
        s_pos[i] = a.positions ? a.positions[t] : at;
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    const uint64_t turns = (uint64_t)(APPEND ? s_pos[t] : a.positions[t0 + t]) * a.freqs[f];
    float sn, cn;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn, &cn);
    cs[i] = make_float2(cn * a.scale, sn * a.scale * a.sign);
  }
  __syncthreads();

  for (; pl < places;) {
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (t >= nt) break;
      int64_t at;
      if (APPEND && kind != 0) {
        at = s_row[t];
        if (at < 0) continue;
      } else {
        at = (int64_t)(t0 + t) * os;
      }
      if (turn) {
        const float2 *w = cs + t * half;
        if (two) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float2 f = w[c * VEC + j];
            const float u = to_f32<T>(x1[t].v[j]), z = to_f32<T>(x2[t].v[j]);
            x1[t].v[j] = from_f32<T>(u * f.x - z * f.y);
            x2[t].v[j] = from_f32<T>(z * f.x + u * f.y);
          }
        } else {
#pragma unroll
          for (int j = 0; j + 1 < VEC; j += 2) {
            const float2 f = w[(c * VEC + j) >> 1];
            const float u = to_f32<T>(x1[t].v[j]), z = to_f32<T>(x1[t].v[j + 1]);
            x1[t].v[j] = from_f32<T>(u * f.x - z * f.y);
            x1[t].v[j + 1] = from_f32<T>(z * f.x + u * f.y);
          }
        }
      }
      *reinterpret_cast<Vec<T, VEC> *>(out + at) = x1[t];
      if (two) *reinterpret_cast<Vec<T, VEC> *>(out + at + apart) = x2[t];
    }
    pl += blockDim.x;
    if (pl < places) load(pl);
  }
}

template <typename T, int VEC, bool APPEND, bool INTER, int TOK>
gdn_status launch_tok(const RopeArgs &a, int places, cudaStream_t st) {
  // threads: one round over the places where they fit, else even rounds
  const int rounds = (places + kMaxThreads - 1) / kMaxThreads;
  const int threads = max(64, ((places + rounds - 1) / rounds + 31) / 32 * 32);
  rope_kernel<T, VEC, APPEND, INTER, TOK>
      <<<(a.n_tok + TOK - 1) / TOK, threads, sizeof(float2) * TOK * (a.rd / 2), st>>>(a);
  return launch_status();
}

template <typename T, int VEC, bool APPEND>
gdn_status launch_vec(const RopeArgs &a, bool inter, cudaStream_t st) {
  const int rot = inter && VEC > 1 ? a.rd / VEC : a.rd / 2 / VEC, rest = (a.D - a.rd) / VEC;
  const int64_t places = (int64_t)a.Hq * (rot + (a.copy_q ? rest : 0)) + (int64_t)a.Hk * (rot + (a.copy_k ? rest : 0)) +
                         (APPEND ? (int64_t)a.Hv * (a.D / VEC) : 0);
  if (places > (1 << 30)) return GDN_ERR_UNSUPPORTED;
  if (places == 0) return GDN_OK;
  // four tokens a block share its set-up; with few tokens one each fills more of the GPU
  const bool many = a.n_tok >= 4 * 2 * 152;
  if (inter)
    return many ? launch_tok<T, VEC, APPEND, true, 4>(a, (int)places, st)
                : launch_tok<T, VEC, APPEND, true, 1>(a, (int)places, st);
  return many ? launch_tok<T, VEC, APPEND, false, 4>(a, (int)places, st)
              : launch_tok<T, VEC, APPEND, false, 1>(a, (int)places, st);
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

extern "C" gdn_status gdn_rope_freqs(const double *inv_freq, int32_t n, uint64_t *freqs) {
  if (n < 0 || (n > 0 && (!inv_freq || !freqs))) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (!isfinite(inv_freq[i])) return GDN_ERR_INVALID_ARG;
    // the fraction of a turn, exact in double; +1/2 is the same angle as -1/2, which fits the word
    const double turns = remainder(inv_freq[i] / (2 * M_PI), 1.0);
    freqs[i] = turns >= 0.5 ? 1ull << 63 : (uint64_t)llrint(ldexp(turns, 64));
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
  a.status = (int32_t *)workspace;
  const bool inter = flags & GDN_FLAG_ROPE_INTERLEAVED;
  if (s.dtype == GDN_BF16) return launch_type<__nv_bfloat16, true>(a, inter, (cudaStream_t)stream);
  return launch_type<float, true>(a, inter, (cudaStream_t)stream);
}

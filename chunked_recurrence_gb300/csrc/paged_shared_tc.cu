// paged_shared_tc.cu -- gdn_paged_attn_shared on the tensor cores: the kernel of paged_attn_tc.cuh over two kinds of
// items, and the join of what they leave.
//
// With the sequences of a group sharing their first P positions,
//     o = (O_p + O_s) / (l_p + l_s),   O_p = sum over j < P, O_s = over j >= P, of e^(x_j - m) v_j, l alike,
// and the first part is one product of all the group's rows with the prefix, whose K and V are read once for 128 to 512 rows
// instead of once a sequence.  A prefix item has rows of the whole group, an own item those of one sequence behind the
// prefix; both lie in one line of work with equal shares, so a long prefix and many short ends balance to a tile.  What a share
// leaves of an item it does not hold whole goes to the pieces of the plain call, a whole item's sums to a row of `full`.
// shared_join_kernel finds the pieces of both items of each row of o from the units before each slot, which the first block
// leaves, and adds them up: nothing waits between the two kinds.
//
// What bounds it, 32 query and 8 kv heads of D 128: 64 single tokens over a prompt of 16000 and up to 500 of their own, 70 us,
// because own items of a few tiles of keys are chains of copy, S, softmax and O, one at a time, in a form that the group's
// rows chose: of two row tiles, or of the two blocks of a pair, one has no row (the bytes take 20 us; the plain call 426);
// 15 chunks of up to 300 over 9001, 343 us, some 300 of them the first kernel, its tensor pipe 52% active, and 45 the join, which
// reads 94 MB of partial sums with dependent loads (the plain call 350: it reads a prefix once for 512 rows).
#include "paged_attn_tc.cuh"

namespace gdn {
namespace {

// Where the pieces of a row of o lie: in shares [from, from + n) of each kind, lane `at` of them; or, of one alone, in `full`.
struct RowPieces {
  int from[2], n[2], at[2];
};
template <class C>
__device__ __forceinline__ RowPieces find_pieces(const TcArgs<true> &a, int64_t row, int h, int blocks, int64_t &to) {
  RowPieces p = {};
  const GroupedSeqs &q = a.seqs;
  const int R = a.RT * C::kTiles, first = (int)item_slots(q.n_tok, q.n_groups, a.G, R);
  const int slots = first + (int)item_slots(q.n_tok, q.n_seqs, a.G, R);
  const int64_t total = a.from[slots];
  const Shares shares = shares_of(max(total, (int64_t)1), max((int)min((int64_t)blocks, total), 1));
  const int t = (int)(row / a.G), i = (int)(row - (int64_t)t * a.G), s = token_seq(q, t), g = seq_group(q, s);
  to = (int64_t)t * (a.G * a.Hkv) + h * a.G + i;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int64_t r = (int64_t)(t - cu_at(q, kind ? s : group_at(q, g))) * a.G + i;  // of the sequence, of the group
    if (r < 0) continue;  // offsets that fall
    const int slot = (kind ? slot_base(q, s, a.G, R) : group_base(q, g, a.G, R)) + (int)(r / R);
    if (slot >= (kind ? slots - first : first)) continue;
    const int64_t before = a.from[slot + kind * first];
    const SharedItem it = kind ? own_item(q, g, s, slot, a.G, R, C::KT) : prefix_item(q, g, slot, a.G, R, C::KT);
    const int over = over_of<C, true>(it, a.RT), its = shared_units(it, over), rr = (int)(r - it.row0);
    const int64_t u = before + (int64_t)h * its;
    if (its == 0 || rr < 0 || rr >= it.rows || u + its > total) continue;
    p.from[kind] = share_of(shares, u + over);
    p.n[kind] = share_of(shares, u + its - 1) - p.from[kind] + 1;
    p.at[kind] = rr / a.RT * 128 + rr % a.RT;
  }
  return p;
}
// Piece i of a row, those of the prefix first; of several the first lies behind its share's other one.
struct Piece {
  int64_t at;
  int kind;
  bool whole;
};
__device__ __forceinline__ Piece piece_of(const RowPieces &p, int i, int64_t in_full, int64_t of_kind) {
  Piece x;
  x.kind = i >= p.n[0];
  const int k = i - (x.kind ? p.n[0] : 0), n = x.kind ? p.n[1] : p.n[0], from = x.kind ? p.from[1] : p.from[0];
  x.whole = n == 1;
  x.at = x.whole ? in_full + x.kind * of_kind : 2 * ((int64_t)from + k) + (k == 0);
  return x;
}
__device__ __forceinline__ void add(float4 &x, float f, const float4 &y) {
  x.x = fmaf(f, y.x, x.x);
  x.y = fmaf(f, y.y, x.y);
  x.z = fmaf(f, y.z, x.z);
  x.w = fmaf(f, y.w, x.w);
}
__device__ __forceinline__ uint2 rounded(const float4 &x, float f) {
  return make_uint2(bf16x2(x.x * f, x.y * f), bf16x2(x.z * f, x.w * f));
}
__device__ __forceinline__ float lse_of(float top, float sum) {
  return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

// Many rows: 32 of a kv head a block, a lane a row, a warp an eighth of the columns; the rows go out through shared memory,
// whole.  (2250 tokens, 32/8 heads, D 128: 50 us, the other 71.)
template <int D, int NQ, bool PAIR>
__global__ void __launch_bounds__(256) shared_join_kernel(const TcArgs<true> a, int blocks) {
  using C = Cfg<D, NQ, PAIR>;
  constexpr int kV = D / 32;  // fours of columns a warp
  __shared__ uint2 out[32][D / 4 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  grid_dependency_wait();
  const int64_t row = (int64_t)blockIdx.x * 32 + lane, all = (int64_t)cu_at(a.seqs, a.seqs.n_seqs) * a.G;
  int64_t to = -1;
  RowPieces p = {};
  if (row < (int64_t)a.seqs.n_tok * a.G) p = find_pieces<C>(a, row, h, blocks, to);
  if (row >= all) to = -1;  // behind the last sequence
  const int pieces = p.n[0] + p.n[1], most = (int)__reduce_max_sync(0xffffffffu, (unsigned)pieces);
  const int64_t in_full = (int64_t)h * gridDim.x + blockIdx.x, of_kind = (int64_t)a.Hkv * gridDim.x;
  auto ml_of = [&](int i) {
    if (i >= pieces) return make_float2(-INFINITY, 0.f);
    const Piece x = piece_of(p, i, in_full, of_kind);
    return *reinterpret_cast<const float2 *>(x.whole ? a.full_ml + (x.at * 32 + lane) * 2
                                                     : a.part_ml + (x.at * C::R + (x.kind ? p.at[1] : p.at[0])) * 2);
  };
  float top = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < most; ++i) top = fmaxf(top, ml_of(i).x);
  float4 x[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < most; ++i) {
    const float2 ml = ml_of(i);
    const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
    sum = fmaf(f, ml.y, sum);
    if (f != 0.f) {
      const Piece y = piece_of(p, i, in_full, of_kind);
      const int step = y.whole ? 32 : C::R;
      const float4 *v = y.whole ? reinterpret_cast<const float4 *>(a.full) + y.at * (D / 4 * 32) + lane
                                : reinterpret_cast<const float4 *>(a.part) + y.at * (C::R * D / 4) + (y.kind ? p.at[1] : p.at[0]);
#pragma unroll
      for (int e = 0; e < kV; ++e) add(x[e], f, v[(int64_t)(warp * kV + e) * step]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < kV; ++e) out[lane][warp * kV + e] = rounded(x[e], inv);
  if (to >= 0 && warp == 0 && a.lse) a.lse[to] = lse_of(top, sum);
  __syncthreads();
  for (int r = warp; r < 32; r += 8) {
    const int64_t o = __shfl_sync(0xffffffffu, to, r);
    if (o >= 0)
      for (int c = lane; c < D / 4; c += 32) *reinterpret_cast<uint2 *>(a.o + o * D + 4 * c) = out[r][c];
  }
}

// Few rows: a warp a row, a lane its columns; a lane has the maximum and sum of one of 32 pieces.
template <int D, int NQ, bool PAIR>
__global__ void __launch_bounds__(256) shared_join_few_kernel(const TcArgs<true> a, int blocks) {
  using C = Cfg<D, NQ, PAIR>;
  constexpr int kV = (D + 127) / 128;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  grid_dependency_wait();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), rows = (int64_t)a.seqs.n_tok * a.G;
  if (row >= rows) return;
  const int64_t all = (int64_t)cu_at(a.seqs, a.seqs.n_seqs) * a.G;
  int64_t to;
  const RowPieces p = find_pieces<C>(a, row, h, blocks, to);
  if (row >= all) return;  // behind the last sequence
  const int pieces = p.n[0] + p.n[1], r = (int)(row % 32);
  const int64_t of_head = (rows + 31) / 32, in_full = (int64_t)h * of_head + row / 32, of_kind = (int64_t)a.Hkv * of_head;
  auto ml_of = [&](int i) {
    if (i >= pieces) return make_float2(-INFINITY, 0.f);
    const Piece x = piece_of(p, i, in_full, of_kind);
    return *reinterpret_cast<const float2 *>(x.whole ? a.full_ml + (x.at * 32 + r) * 2
                                                     : a.part_ml + (x.at * C::R + (x.kind ? p.at[1] : p.at[0])) * 2);
  };
  float2 ml = ml_of(lane);
  float top = ml.x, sum = 0.f;
  for (int i = 32 + lane; i < pieces; i += 32) top = fmaxf(top, ml_of(i).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float4 x[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < pieces; base += 32) {
    if (base > 0) ml = ml_of(base + lane);
    const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
    sum = fmaf(w, ml.y, sum);
    const int m = min(32, pieces - base);
#pragma unroll 4
    for (int i = 0; i < m; ++i) {
      const float f = __shfl_sync(0xffffffffu, w, i);
      const Piece y = piece_of(p, base + i, in_full, of_kind);
      const int step = y.whole ? 32 : C::R;
      const float4 *v = y.whole ? reinterpret_cast<const float4 *>(a.full) + y.at * (D / 4 * 32) + r
                                : reinterpret_cast<const float4 *>(a.part) + y.at * (C::R * D / 4) + (y.kind ? p.at[1] : p.at[0]);
#pragma unroll
      for (int e = 0; e < kV; ++e)
        if (f != 0.f && lane + 32 * e < D / 4) add(x[e], f, v[(int64_t)(lane + 32 * e) * step]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < kV; ++e)
    if (lane + 32 * e < D / 4) *reinterpret_cast<uint2 *>(a.o + to * D + 4 * (lane + 32 * e)) = rounded(x[e], inv);
  if (lane == 0 && a.lse) a.lse[to] = lse_of(top, sum);
}

// The workspace behind the status: the units before each slot, the pieces, the rows of whole items.
struct Layout {
  size_t from, part_ml, part, full_ml, full, end;
};
Layout layout(const gdn_cache_shape &s, int32_t n_groups, int row_tiles) {
  const int G = s.Hq / s.Hkv, RT = 128 / G * G;
  const size_t lanes = (size_t)kSms * 2 * 128 * row_tiles, rows = 2 * (size_t)s.Hkv * (((size_t)s.n_tok * G + 31) / 32 * 32);
  Layout l;
  l.from = 256;
  l.part_ml = (l.from + (shared_slots(s.n_tok, s.n_seqs, n_groups, G, RT) + 1) * sizeof(int64_t) + 255) & ~(size_t)255;
  l.part = l.part_ml + lanes * 2 * sizeof(float);
  l.full_ml = l.part + lanes * s.D * sizeof(float);
  l.full = (l.full_ml + rows * 2 * sizeof(float) + 255) & ~(size_t)255;
  l.end = l.full + rows * s.D * sizeof(float);
  return l;
}

template <int D, int NQ, bool PAIR>
gdn_status launch(const void *k, const void *v, const gdn_cache_shape &s, TcArgs<true> &a, void *workspace, cudaStream_t st) {
  const Layout l = layout(s, a.seqs.n_groups, NQ);  // a pair has half the shares, of twice the lanes
  char *w = (char *)workspace;
  a.from = (int64_t *)(w + l.from);
  a.part_ml = (float *)(w + l.part_ml), a.part = (float *)(w + l.part);
  a.full_ml = (float *)(w + l.full_ml), a.full = (float *)(w + l.full);
  const int64_t rows = (int64_t)s.n_tok * a.G;
  if (rows * a.Hkv >= 8 * 32 * kSms)
    return launch_two<D, NQ, PAIR, true>(k, v, s, a, st, dim3((unsigned)((rows + 31) / 32), a.Hkv),
                                         shared_join_kernel<D, NQ, PAIR>);
  return launch_two<D, NQ, PAIR, true>(k, v, s, a, st, dim3((unsigned)((rows + 7) / 8), a.Hkv),
                                       shared_join_few_kernel<D, NQ, PAIR>);
}

}  // namespace

size_t paged_shared_tc_workspace(const gdn_cache_shape &s, int32_t n_groups, int32_t max_group_new) {
  return tc_shape(s) ? layout(s, n_groups, two_tiles(s, max_group_new) ? 2 : 1).end : 0;
}

// The kernel's form goes by the rows of a group, which share the long part.
gdn_status paged_shared_tc(const void *q, const void *k, const void *v, const int32_t *table, const GroupedSeqs &seqs,
                           const gdn_cache_shape &s, int32_t max_group_new, float scale_log2, uint32_t flags, void *o,
                           float *lse, void *workspace, cudaStream_t st) {
  TcArgs<true> a = tc_args<true>(q, table, seqs, s, scale_log2, 0, flags, o, lse, workspace);
  const bool pair = pairs(s, max_group_new), two = two_tiles(s, max_group_new);
  if (s.D == 256)
    return pair ? launch<256, 1, true>(k, v, s, a, workspace, st) : launch<256, 1, false>(k, v, s, a, workspace, st);
  if (s.D == 64)
    return two ? launch<64, 2, false>(k, v, s, a, workspace, st) : launch<64, 1, false>(k, v, s, a, workspace, st);
  if (pair) return launch<128, 2, true>(k, v, s, a, workspace, st);
  return two ? launch<128, 2, false>(k, v, s, a, workspace, st) : launch<128, 1, false>(k, v, s, a, workspace, st);
}

}  // namespace gdn

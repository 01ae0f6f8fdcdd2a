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
#include "paged_attn_tc.cuh"

namespace gdn {
namespace {

// A warp takes `per` rows of o of a kv head, one at a time, a lane 4 (D = 256: 8) of a row's columns.  First each lane finds
// where the pieces of one of the block's rows lie.
template <int D, int NQ, bool PAIR>
__global__ void __launch_bounds__(256) shared_join_kernel(const TcArgs a, int blocks, int per) {
  using C = Cfg<D, NQ, PAIR>;
  constexpr int kV = (D + 127) / 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const PagedSeqs &q = a.seqs;
  const int R = a.RT * C::kTiles, first = (int)item_slots(q.n_tok, q.n_groups, a.G, R);
  const int slots = first + (int)item_slots(q.n_tok, q.n_seqs, a.G, R);
  grid_dependency_wait();
  const int64_t total = a.from[slots], rows = (int64_t)q.n_tok * a.G, all = rows * a.Hkv;
  const int shares = (int)min((int64_t)blocks, total);
  const int64_t row = (int64_t)blockIdx.x * (8 * per) + lane;
  int from[2] = {0, 0}, to[2] = {-1, -1}, at[2] = {0, 0};  // shares [from, to] that hold pieces, the row's lane in them
  int64_t out = -1;
  if (lane < 8 * per && row < rows) {
    const int t = (int)(row / a.G), i = (int)(row - (int64_t)t * a.G);
    out = (int64_t)t * (a.G * a.Hkv) + h * a.G + i;
    const int s = token_seq(q, t), g = seq_group(q, s);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int64_t r = (int64_t)(t - cu_at(q, kind ? s : group_at(q, g))) * a.G + i;  // of the sequence, of the group
      if (r < 0) continue;  // offsets that fall
      const int slot = (kind ? slot_base(q, s, a.G, R) : group_base(q, g, a.G, R)) + (int)(r / R);
      if (slot >= (kind ? slots - first : first)) continue;
      const SharedItem it = kind ? own_item(q, g, s, slot, a.G, R, C::KT) : prefix_item(q, g, slot, a.G, R, C::KT);
      const int its = shared_units(it, C::kOver), rr = (int)(r - it.row0);
      const int64_t u = a.from[slot + kind * first] + (int64_t)h * its;
      if (its == 0 || rr < 0 || rr >= it.rows || u + its > total) continue;
      from[kind] = share_of(total, u + C::kOver, shares), to[kind] = share_of(total, u + its - 1, shares);
      at[kind] = rr / a.RT * 128 + rr % a.RT;
    }
  }
  for (int j = warp * per; j < (warp + 1) * per; ++j) {
    const int64_t o = __shfl_sync(0xffffffffu, out, j);
    if (o < 0) break;
    int f[2], n[2], lr[2];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      f[kind] = __shfl_sync(0xffffffffu, from[kind], j);
      n[kind] = __shfl_sync(0xffffffffu, to[kind], j) - f[kind] + 1;
      lr[kind] = __shfl_sync(0xffffffffu, at[kind], j);
      if (n[kind] < 0) n[kind] = 0;
    }
    const int pieces = n[0] + n[1];
    // piece i: of the prefix first; of several the first lies behind its share's other one
    auto which = [&](int i, bool &whole, int &kind) {
      kind = i >= n[0];
      const int k = i - (kind ? n[0] : 0);
      whole = n[kind] == 1;
      return whole ? kind * all + o : 2 * ((int64_t)f[kind] + k) + (k == 0);
    };
    auto ml_of = [&](int i) {
      bool whole;
      int kind;
      if (i >= pieces) return make_float2(-INFINITY, 0.f);
      const int64_t w = which(i, whole, kind);
      return *reinterpret_cast<const float2 *>(whole ? a.full_ml + w * 2 : a.part_ml + (w * C::R + lr[kind]) * 2);
    };
    float2 ml = ml_of(lane);
    float top = ml.x;
    for (int i = 32 + lane; i < pieces; i += 32) top = fmaxf(top, ml_of(i).x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.f;
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
        const float wi = __shfl_sync(0xffffffffu, w, i);
        bool whole;
        int kind;
        const int64_t p = which(base + i, whole, kind);
        const float4 *v = whole ? reinterpret_cast<const float4 *>(a.full) + p * (D / 4)
                                : reinterpret_cast<const float4 *>(a.part) + p * (C::R * D / 4) + lr[kind];
#pragma unroll
        for (int e = 0; e < kV; ++e)
          if (wi != 0.f && lane + 32 * e < D / 4) {
            const float4 y = v[(int64_t)(lane + 32 * e) * (whole ? 1 : C::R)];
            x[e].x = fmaf(wi, y.x, x[e].x);
            x[e].y = fmaf(wi, y.y, x[e].y);
            x[e].z = fmaf(wi, y.z, x[e].z);
            x[e].w = fmaf(wi, y.w, x[e].w);
          }
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (lane + 32 * e < D / 4)
        *reinterpret_cast<uint2 *>(a.o + o * D + 4 * (lane + 32 * e)) =
            make_uint2(bf16x2(x[e].x * inv, x[e].y * inv), bf16x2(x[e].z * inv, x[e].w * inv));
    if (lane == 0 && a.lse) a.lse[o] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
  }
}

// The workspace behind the status: the units before each slot, the pieces, the rows of whole items.
struct Layout {
  size_t from, part_ml, part, full_ml, full, end;
};
Layout layout(const gdn_cache_shape &s, int32_t n_groups, int row_tiles) {
  const int G = s.Hq / s.Hkv, RT = 128 / G * G;
  const size_t lanes = (size_t)kSms * 2 * 128 * row_tiles, rows = 2 * (size_t)s.n_tok * s.Hq;
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
gdn_status launch(const void *k, const void *v, const gdn_cache_shape &s, TcArgs &a, void *workspace, cudaStream_t st) {
  const Layout l = layout(s, a.seqs.n_groups, NQ);  // a pair has half the shares, of twice the lanes
  char *w = (char *)workspace;
  a.from = (int64_t *)(w + l.from);
  a.part_ml = (float *)(w + l.part_ml), a.part = (float *)(w + l.part);
  a.full_ml = (float *)(w + l.full_ml), a.full = (float *)(w + l.full);
  const int64_t rows = (int64_t)s.n_tok * a.G;
  const int per = rows * a.Hkv >= 8 * 8 * kSms * 4 ? 4 : 1;  // a row a warp while the warps are few
  const dim3 grid((unsigned)((rows + 8 * per - 1) / (8 * per)), a.Hkv);
  return launch_two<D, NQ, PAIR, true>(k, v, s, a, st, grid, shared_join_kernel<D, NQ, PAIR>, per);
}

}  // namespace

size_t paged_shared_tc_workspace(const gdn_cache_shape &s, int32_t n_groups, int32_t max_group_new) {
  return tc_shape(s) ? layout(s, n_groups, two_tiles(s, max_group_new) ? 2 : 1).end : 0;
}

// The kernel's form goes by the rows of a group, which share the long part.
gdn_status paged_shared_tc(const void *q, const void *k, const void *v, const int32_t *table, const PagedSeqs &seqs,
                           const gdn_cache_shape &s, int32_t max_group_new, float scale_log2, uint32_t flags, void *o,
                           float *lse, void *workspace, cudaStream_t st) {
  TcArgs a = tc_args(q, table, seqs, s, scale_log2, 0, flags, o, lse, workspace);
  const bool pair = pairs(s, max_group_new), two = two_tiles(s, max_group_new);
  if (s.D == 256)
    return pair ? launch<256, 1, true>(k, v, s, a, workspace, st) : launch<256, 1, false>(k, v, s, a, workspace, st);
  if (s.D == 64)
    return two ? launch<64, 2, false>(k, v, s, a, workspace, st) : launch<64, 1, false>(k, v, s, a, workspace, st);
  if (pair) return launch<128, 2, true>(k, v, s, a, workspace, st);
  return two ? launch<128, 2, false>(k, v, s, a, workspace, st) : launch<128, 1, false>(k, v, s, a, workspace, st);
}

}  // namespace gdn

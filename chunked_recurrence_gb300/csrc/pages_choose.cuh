// pages_choose.cuh -- the largest of a list of weights and where they are, by one block (gdn_pages_evict): a radix selection over
// the weights as whole numbers of the same order, then their positions in rising order.  Compiled for the device by the
// kernel and for the host by the tests, which run a block's threads one after another in several orders.
#pragma once

#include "block_scan.cuh"

namespace gdn {
namespace pages {

constexpr int kChooseThreads = 1024;
constexpr int kInRegs = 8;         // fours of weights a thread keeps in registers; of longer sequences they are read again each time
constexpr int kBins = 2048;

// A weight as a whole number of the same order: NaN lowest, the two zeros alike.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

struct ChooseShared {
  int hist[kBins], sh[33], digit, left, listed;
  uint32_t list[2 * kChooseThreads];
  uint64_t sums[32];
};

// How many of the keys that each thread gives have each digit.  At once, but for keys that are alike in a warp (zeros, say),
// which would meet at one count, a lane after another.
__device__ __forceinline__ void count_digit(int *hist, uint32_t digit, bool mine) {
  const uint32_t all = __ballot_sync(0xffffffffu, mine);
  if (all == 0) return;
  if (__popc(all) > 8) {
    const uint32_t some = __shfl_sync(0xffffffffu, digit, __ffs(all) - 1);
    if (__all_sync(0xffffffffu, !mine || digit == some)) {
      if ((threadIdx.x & 31) == 0) atomicAdd(&hist[some], __popc(all));
      return;
    }
  }
  if (mine) atomicAdd(&hist[digit], 1);
}
// The digit that holds the left-th largest, and which of those with it; `many`: how many they are.
__device__ __forceinline__ uint32_t find_digit(ChooseShared &sm, int &left, int &many) {
  __syncthreads();
  // from the largest digit down: a thread has two
  const int b = kBins - 1 - 2 * threadIdx.x, x = sm.hist[b], y = sm.hist[b - 1];
  int total;
  const int upto = block_scan(x + y, sm.sh, &total), before = upto - x - y;
  if (before < left && left <= upto) {
    const bool first = left <= before + x;
    sm.digit = first ? b : b - 1;
    sm.left = left - (first ? before : before + x);
  }
  __syncthreads();
  left = sm.left;
  many = sm.hist[sm.digit];
  return sm.digit;
}
__device__ __forceinline__ void clear_counts(ChooseShared &sm) {
  __syncthreads();  // the counts before, and what was found in them, have been read
  for (int b = threadIdx.x; b < kBins; b += kChooseThreads) sm.hist[b] = 0;
  __syncthreads();
}

// Four 16-bit sums over the block's threads at once: those before this thread, and all.
__device__ __forceinline__ uint64_t sums_before(uint64_t x, ChooseShared &sm, uint64_t &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t mine = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();
  if (lane == 31) sm.sums[warp] = x;
  __syncthreads();
  uint64_t y = sm.sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += u;
  }
  all = __shfl_sync(0xffffffffu, y, 31);
  const uint64_t others = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
  return x - mine + (warp ? others : 0);
}

// The `need` largest of the N weights: their positions, in rising order, and the weights.  In round r a thread has weights
// 4096 r + 4 tid .. + 3: R rounds in registers, or with R = 0 all that there are, read again each time.
template <int R>
__device__ void choose(const float *mass, int N, int need, int32_t *index, float *weight, ChooseShared &sm) {
  const int tid = threadIdx.x;
  if (tid == 0) sm.listed = 0;  // the first count's barriers lie before its use
  const int rounds = R ? R : (N + 4 * kChooseThreads - 1) / (4 * kChooseThreads);
  const bool wide = (reinterpret_cast<uintptr_t>(mass) & 15) == 0;
  auto place = [&](int r) { return 4 * (r * kChooseThreads + tid); };
  auto read = [&](int r, uint32_t (&u)[4]) {
    const int j = place(r);
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (wide && j + 3 < N) {
      w = *reinterpret_cast<const float4 *>(mass + j);
    } else {
      if (j < N) w.x = mass[j];
      if (j + 1 < N) w.y = mass[j + 1];
      if (j + 2 < N) w.z = mass[j + 2];
      if (j + 3 < N) w.w = mass[j + 3];
    }
    u[0] = order_of(w.x), u[1] = order_of(w.y), u[2] = order_of(w.z), u[3] = order_of(w.w);
  };
  uint32_t held[R ? R : 1][4];
#pragma unroll
  for (int r = 0; r < R; ++r) read(r, held[r]);
  auto keys = [&](int r, uint32_t (&u)[4]) {
    if (R) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = held[R ? r : 0][i];
    } else {
      read(r, u);
    }
  };
  auto there = [&](int r, int i) { return place(r) + i < N; };

  // the need-th largest, digit by digit: of the numbers that begin with `top`, how many have each next digit
  int left = need, many;
  auto count = [&](int shift, uint32_t mask, uint32_t top, bool all) {
    clear_counts(sm);
#pragma unroll
    for (int r = 0; r < rounds; ++r) {
      uint32_t u[4];
      keys(r, u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        count_digit(sm.hist, u[i] >> shift & mask, there(r, i) && (all || u[i] >> shift >> (mask == 1023 ? 10 : 11) == top));
    }
  };
  count(21, 2047, 0, true);
  uint32_t top = find_digit(sm, left, many);
  if (many <= 2 * kChooseThreads) {  // those that begin so, by themselves, in any order
    clear_counts(sm);
#pragma unroll
    for (int r = 0; r < rounds; ++r) {
      uint32_t u[4];
      keys(r, u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (there(r, i) && u[i] >> 21 == top) sm.list[atomicAdd(&sm.listed, 1)] = u[i];
    }
    const int listed = many;
    uint32_t u[2];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u[i] = tid + i * kChooseThreads < listed ? sm.list[tid + i * kChooseThreads] : 0;
      count_digit(sm.hist, u[i] >> 10 & 2047, tid + i * kChooseThreads < listed);
    }
    top = top << 11 | find_digit(sm, left, many);
    clear_counts(sm);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      count_digit(sm.hist, u[i] & 1023, tid + i * kChooseThreads < listed && u[i] >> 10 == top);
    top = top << 10 | find_digit(sm, left, many);
  } else {
    count(10, 2047, top, false);
    top = top << 11 | find_digit(sm, left, many);
    count(0, 1023, top, false);
    top = top << 10 | find_digit(sm, left, many);
  }
  // above `top` all stay, of those at it the first `left`: where each round's go, four rounds' counts in a word
  int eq0 = 0, at0 = 0;  // of the rounds before
#pragma unroll
  for (int r0 = 0; r0 < rounds; r0 += 4) {
    uint64_t gt = 0, eq = 0, all;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r0 + k >= rounds) break;
      uint32_t u[4];
      keys(r0 + k, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gt += (uint64_t)(there(r0 + k, i) && u[i] > top) << 16 * k;
        eq += (uint64_t)(there(r0 + k, i) && u[i] == top) << 16 * k;
      }
    }
    const uint64_t eq_at = sums_before(eq, sm, all);
    uint64_t in = 0;  // of the thread's that are at `top`
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int before = eq0 + (int)(eq_at >> 16 * k & 0xffff);
      in += (uint64_t)min(max(left - before, 0), (int)(eq >> 16 * k & 0xffff)) << 16 * k;
      eq0 += (int)(all >> 16 * k & 0xffff);
    }
    const uint64_t at_r = sums_before(gt + in, sm, all);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r0 + k >= rounds) break;
      int at = at0 + (int)(at_r >> 16 * k & 0xffff), level = (int)(in >> 16 * k & 0xffff);
      at0 += (int)(all >> 16 * k & 0xffff);
      if ((gt + in) >> 16 * k & 0xffff) {
        uint32_t u[4];
        keys(r0 + k, u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (there(r0 + k, i) && (u[i] > top || (u[i] == top && level-- > 0))) {
            const int j = place(r0 + k) + i;
            index[at] = j;
            // the weight itself; which NaN or zero it was is not in the key
            weight[at++] = u[i] == 0 || u[i] == 0x80000000u ? mass[j]
                                                          : __uint_as_float(u[i] >> 31 ? u[i] & 0x7fffffffu : ~u[i]);
          }
      }
    }
  }
}

__device__ __forceinline__ void choose_largest(const float *mass, int N, int need, int32_t *index, float *weight,
                                               ChooseShared &sm) {
  constexpr int kRound = 4 * kChooseThreads;
  if (N <= kRound) choose<1>(mass, N, need, index, weight, sm);
  else if (N <= 4 * kRound) choose<4>(mass, N, need, index, weight, sm);
  else if (N <= kInRegs * kRound) choose<kInRegs>(mass, N, need, index, weight, sm);
  else choose<0>(mass, N, need, index, weight, sm);
}

}  // namespace pages
}  // namespace gdn

// The selection of gdn_pages_evict (pages_choose.cuh) compiled for the host: a block's 1024 threads as fibers that run one after
// another.  Between two barriers a warp may run as far ahead of the others as it likes; which goes first is the caller's
// choice, so a value that is read or written without a barrier between shows in the result.
#include <stdint.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <memory>
#include <random>
#include <vector>

namespace fibers {
constexpr int kThreads = 1024, kWarps = 32, kStack = 64 * 1024;
enum Where { kRuns, kAtWarp, kAtBlock, kDone };
struct Fiber {
  ucontext_t at;
  Where where;
};
Fiber fiber[kThreads];
ucontext_t home;
std::unique_ptr<char[]> stacks;
int tid;
uint64_t lane_value[kThreads];

void stop(Where where) {
  const int me = tid;
  fiber[me].where = where;
  swapcontext(&fiber[me].at, &home);
}
void at_block() { stop(kAtBlock); }
void at_warp() { stop(kAtWarp); }
void resume(int t) {
  tid = t;
  fiber[t].where = kRuns;
  swapcontext(&home, &fiber[t].at);
}

// A warp until all of its threads wait for the block or are done; false where they wait for different things.
bool run_warp(int w) {
  for (;;) {
    for (int t = 32 * w; t < 32 * w + 32; ++t)
      if (fiber[t].where == kRuns) resume(t);
    const Where all = fiber[32 * w].where;
    for (int t = 32 * w; t < 32 * w + 32; ++t)
      if (fiber[t].where != all) return false;
    if (all != kAtWarp) return true;
    for (int t = 32 * w; t < 32 * w + 32; ++t) fiber[t].where = kRuns;
  }
}
// order: 0 the first warp first, 1 the last first, else a seed of an order for each stretch between barriers.  False where some
// threads came to a barrier that others do not come to.
bool run_block(void (*body)(), int order) {
  if (!stacks) stacks.reset(new char[(size_t)kThreads * kStack]);
  for (int t = 0; t < kThreads; ++t) {
    getcontext(&fiber[t].at);
    fiber[t].at.uc_stack.ss_sp = stacks.get() + (size_t)t * kStack;
    fiber[t].at.uc_stack.ss_size = kStack;
    fiber[t].at.uc_link = &home;
    makecontext(&fiber[t].at, body, 0);
    fiber[t].where = kRuns;
  }
  std::mt19937 rng(order);
  std::vector<int> warps(kWarps);
  for (int w = 0; w < kWarps; ++w) warps[w] = order == 1 ? kWarps - 1 - w : w;
  for (;;) {
    if (order > 1) std::shuffle(warps.begin(), warps.end(), rng);
    for (int w : warps)
      if (!run_warp(w)) return false;
    for (int t = 0; t < kThreads; ++t)
      if (fiber[t].where != fiber[0].where) return false;
    if (fiber[0].where == kDone) return true;
    for (int t = 0; t < kThreads; ++t) fiber[t].where = kRuns;
  }
}
}  // namespace fibers

// the device's names
#define __device__
#define __forceinline__ inline
struct Index {
  struct X {
    operator int() const { return fibers::tid; }
  } x;
};
struct Size {
  int x = fibers::kThreads;
};
static const Index threadIdx;
static const Size blockDim;
struct float4 {
  float x, y, z, w;
};
static float4 make_float4(float x, float y, float z, float w) { return {x, y, z, w}; }
using std::max;
using std::min;
static void __syncthreads() { fibers::at_block(); }
template <typename T>
static T lane_of(T x, int from) {  // x of lane `from`; what the warp's threads gave is there between its two stops
  static_assert(sizeof(T) <= 8, "");
  fibers::lane_value[fibers::tid] = 0;
  memcpy(&fibers::lane_value[fibers::tid], &x, sizeof x);
  fibers::at_warp();
  T y;
  memcpy(&y, &fibers::lane_value[(fibers::tid & ~31) + (from & 31)], sizeof y);
  fibers::at_warp();
  return y;
}
template <typename T>
static T __shfl_sync(unsigned, T x, int from) { return lane_of(x, from); }
template <typename T>
static T __shfl_up_sync(unsigned, T x, int by) {
  const int lane = fibers::tid & 31;
  return lane_of(x, lane >= by ? lane - by : lane);
}
static uint32_t __ballot_sync(unsigned, bool p) {
  fibers::lane_value[fibers::tid] = p;
  fibers::at_warp();
  uint32_t all = 0;
  for (int i = 0; i < 32; ++i) all |= (uint32_t)fibers::lane_value[(fibers::tid & ~31) + i] << i;
  fibers::at_warp();
  return all;
}
static bool __all_sync(unsigned m, bool p) { return __ballot_sync(m, p) == 0xffffffffu; }
static int __popc(uint32_t x) { return __builtin_popcount(x); }
static int __ffs(uint32_t x) { return __builtin_ffs(x); }
static uint32_t __float_as_uint(float x) {
  uint32_t u;
  memcpy(&u, &x, 4);
  return u;
}
static float __uint_as_float(uint32_t u) {
  float x;
  memcpy(&x, &u, 4);
  return x;
}
static int atomicAdd(int *p, int v) {
  const int old = *p;
  *p += v;
  return old;
}

#include "pages_choose.cuh"

static struct {
  const float *mass;
  int n, need;
  int32_t *index;
  float *weight;
  gdn::pages::ChooseShared shared;
} call;

static void body() {
  gdn::pages::choose_largest(call.mass, call.n, call.need, call.index, call.weight, call.shared);
  fibers::stop(fibers::kDone);
}

// 0 < need < n.  1: done; 0: the threads parted at a barrier.
extern "C" int32_t host_choose(const float *mass, int32_t n, int32_t need, int32_t order, int32_t *index, float *weight) {
  call.mass = mass, call.n = n, call.need = need, call.index = index, call.weight = weight;
  memset(&call.shared, 0x5a, sizeof call.shared);
  return fibers::run_block(body, order);
}

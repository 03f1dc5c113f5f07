// The group plan that every expert operator derives on the device from the
// offsets of its launch: checked offsets in shared memory and the exclusive
// prefix of a per-group work count.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxGroups = 257;   // 256 routed experts and the shared one

// One try of a wait whose barrier other CTAs of the cluster arrive on: what
// they did before their arrivals is visible behind it.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait for the expert operators' stages: looks at the abort flag and the
// clock only every 32nd poll. Same limit, abort flag and status. CLUSTER: the
// barrier's arrivals come from both CTAs of a pair.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_stage(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status,
                                                unsigned long long limit_ns) {
  const uint32_t a = smem_u32(bar);
  unsigned long long t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (CLUSTER ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity)) return true;
    if ((i & 31u) == 0) {
      if (*abort) return false;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > limit_ns) {
        set_status(status, STATUS_WAIT_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
}

struct GroupPlan {
  int off[kMaxGroups + 1];     // row offsets, [ngroups + 1]
  int prefix[kMaxGroups + 1];  // exclusive prefix of the work counts
  int wsum[32];
};

// Fills `s` from offsets[0..ngroups] with count(rows of the group) units of
// work per group; returns the total, or -1 when the offsets start below 0,
// decrease, end beyond `rows`, or give rows to a group without weights
// (index >= nweights): the launch then does no work and has set
// STATUS_BAD_PLAN. Called by all THREADS threads of the block, which take
// the groups in rounds; ends with a block barrier.
template <int THREADS, typename F>
__device__ __forceinline__ int build_plan(GroupPlan& s, const int32_t* __restrict__ offsets, int ngroups, int nweights,
                                          int rows, uint32_t* status, F count) {
  constexpr int ROUNDS = (kMaxGroups + THREADS - 1) / THREADS;
  int o0[ROUNDS], o1[ROUNDS];   // all loads first: one trip to memory
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int g = r * THREADS + int(threadIdx.x);
    o0[r] = g < ngroups ? offsets[g] : 0;
    o1[r] = g < ngroups ? offsets[g + 1] : 0;
  }
  int base = 0;
  int bad_any = 0;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    if (r * THREADS >= ngroups) break;
    const int g = r * THREADS + int(threadIdx.x);
    int v = 0, bad = 0;
    if (g < ngroups) {
      bad = o0[r] < 0 || o1[r] < o0[r] || o1[r] > rows || (g >= nweights && o1[r] != o0[r]);
      s.off[g] = o0[r];
      if (g == ngroups - 1) s.off[ngroups] = o1[r];
      if (!bad && g < nweights) v = count(o1[r] - o0[r]);
    }
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if ((threadIdx.x & 31) >= d) incl += o;
    }
    if ((threadIdx.x & 31) == 31) s.wsum[threadIdx.x >> 5] = incl;
    bad_any |= __syncthreads_or(bad);
    int before = base, all = base;
    for (int j = 0; j < THREADS / 32; ++j) {
      const int w = s.wsum[j];
      if (j < int(threadIdx.x >> 5)) before += w;
      all += w;
    }
    if (g < ngroups) s.prefix[g] = before + incl - v;
    if (g == ngroups - 1) s.prefix[ngroups] = before + incl;
    base = all;
    __syncthreads();   // wsum is rewritten in the next round; prefix and off are complete
  }
  if (bad_any) {
    if (threadIdx.x == 0) set_status(status, STATUS_BAD_PLAN);
    return -1;
  }
  return base;
}

// The group that holds unit i of the work list (groups without units are
// passed over): the last one whose prefix is <= i.
__device__ __forceinline__ int find_group(const int* prefix, int ngroups, int i) {
  int lo = 0, hi = ngroups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace moe

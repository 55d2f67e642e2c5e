// Page hand-out, shared by the calls that give pages of a cache to requests:
// who is served, and with which pages, is a scan over the requests and a scan
// over the pages' states, done by ONE CTA.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace sa {
namespace handout {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = kKv4MaxRequests / kPlanThreads;  // requests per thread
constexpr int kScanPages = 16;                            // counts per thread and step
constexpr int kListPages = 4096;
constexpr int kBloomBits = 32768;
constexpr int kSaturated = 0x7fffffff;

struct PlanShared {
  int slot[kKv4MaxRequests];
  int upto[kKv4MaxRequests];  // pages asked for by the requests up to and including this one, saturating
  uint32_t seen[kBloomBits / 32], again[kBloomBits / 32];
  int page[kListPages];  // free pages found, by rank
  int warp[32];
  int total;
};

SA_DEV int sat_add(int a, int b) { return a > kSaturated - b ? kSaturated : a + b; }  // a, b >= 0

// Inclusive saturating scan over the CTA; the total goes to *total.
SA_DEV int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = sat_add(x, y);
  }
  __syncthreads();  // the previous use of warp_sums and total is over
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int y = lane < (blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y = sat_add(y, z);
    }
    warp_sums[lane] = y;
    if (lane == 31) *total = y;
  }
  __syncthreads();
  return w > 0 ? sat_add(x, warp_sums[w - 1]) : x;
}

// Marks in `dup` (bit c: request tid + 1024 c) the requests whose slot an
// earlier request names too.  A table of slot numbers modulo 32768 finds the
// few that can be repeated; those alone are compared with all before them.
SA_DEV uint32_t find_repeats(PlanShared& sh, int n) {
  for (int i = threadIdx.x; i < kBloomBits / 32; i += kPlanThreads) sh.seen[i] = sh.again[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const uint32_t h = static_cast<uint32_t>(sh.slot[i]) % kBloomBits, bit = 1u << (h & 31);
    if (atomicOr(&sh.seen[h >> 5], bit) & bit) atomicOr(&sh.again[h >> 5], bit);
  }
  __syncthreads();
  uint32_t dup = 0;
  for (int c = 0, i = threadIdx.x; i < n; ++c, i += kPlanThreads) {
    const uint32_t h = static_cast<uint32_t>(sh.slot[i]) % kBloomBits;
    if (!(sh.again[h >> 5] >> (h & 31) & 1u)) continue;
    for (int j = 0; j < i; ++j)
      if (sh.slot[j] == sh.slot[i]) {
        dup |= 1u << c;
        break;
      }
  }
  return dup;
}

// Turns sh.upto from each request's own need into the running total.
SA_DEV int scan_needs(PlanShared& sh, int n) {
  int carry = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int x = block_scan(i < n ? sh.upto[i] : 0, sh.warp, &sh.total);
    if (i < n) sh.upto[i] = sat_add(carry, x);
    carry = sat_add(carry, sh.total);
  }
  __syncthreads();
  return carry;
}

// The request that the rank-th page goes to: the first with upto > rank.
SA_DEV int request_of(const PlanShared& sh, int n, int rank) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sh.upto[mid] > rank)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Calls give(rank, page) for the lowest free pages (those whose entry in
// `held`, 16-byte aligned, is kFree), rank = 0 .. need - 1, and returns how
// many there are, at most `need`.  Free pages come in runs, which one thread
// finds: they go through a list, so that all threads hand out.
template <int kFree, class F>
SA_DEV int hand_out(PlanShared& sh, const int32_t* held, int num_pages, int need, F give) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < need; base += kPlanThreads * kScanPages) {
    const int64_t p0 = base + threadIdx.x * kScanPages;
    uint32_t free_bits = 0;
    if (p0 + kScanPages <= num_pages) {
      int4 v[kScanPages / 4];
#pragma unroll
      for (int k = 0; k < kScanPages / 4; ++k) v[k] = reinterpret_cast<const int4*>(held + p0)[k];
#pragma unroll
      for (int k = 0; k < kScanPages / 4; ++k)
        free_bits |= static_cast<uint32_t>((v[k].x == kFree) | (v[k].y == kFree) << 1 | (v[k].z == kFree) << 2 | (v[k].w == kFree) << 3)
                     << (4 * k);
    } else {
      for (int k = 0; p0 + k < num_pages; ++k) free_bits |= static_cast<uint32_t>(held[p0 + k] == kFree) << k;
    }
    const int mine = __popc(free_bits);
    int rank = found + block_scan(mine, sh.warp, &sh.total) - mine;
    const int end = min(found + sh.total, need);
    for (int first = found; first < end; first += kListPages) {
      const int last = min(first + kListPages, end);
      while (free_bits != 0 && rank < last) {  // the ranks below `first` are through
        sh.page[rank++ - first] = static_cast<int>(p0) + __ffs(free_bits) - 1;
        free_bits &= free_bits - 1;
      }
      __syncthreads();
      for (int r = first + threadIdx.x; r < last; r += kPlanThreads) give(r, sh.page[r - first]);
      __syncthreads();
    }
    found += sh.total;
  }
  return min(found, need);
}

}  // namespace handout
}  // namespace sa

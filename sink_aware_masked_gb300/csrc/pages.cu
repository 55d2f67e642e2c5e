// Pages of bf16 keys and values: the plan of a step (which pages a slot gives
// back and gets, where each new row goes) and the write of the new rows.
//
// All state is on the device, as for the 4-bit cache: a page is free when its
// owner is -1, requests take the lowest-numbered free pages in the order in
// which they stand, and every result is the same from run to run.
#include "handout.cuh"

#include <algorithm>

namespace sa {
namespace {

using namespace handout;

// ---------------------------------------------------------------- plan
// left = max(len - drop, 0), then len = left + new: pages beyond left go back
// first, all of them, then the requests are served.  One CTA, and for long
// calls a second launch that writes the rows' places on all SMs.  What bounds it
// is the chain of scans, searches and dependent loads (GB300: 1 slot 5.0 us with
// its launch, 256 slots with 1 to 5 rows each 9.8, 512 slots of which 64 are
// refilled with 220 k rows 18.0, of these 5 for the rows' places).
constexpr int kRowsInPlan = 4096;  // rows whose places the plan's own CTA writes
constexpr int kMapThreads = 256;
constexpr int kMapPer = 4;  // rows per thread of the second launch

struct StepShared {
  PlanShared p;
  int base[kKv4MaxRequests];  // pages that a request keeps, then its tokens kept, -1 where it is not served
};

SA_DEV int pages_for(const KvPages& c, int tokens) {
  return static_cast<int>((static_cast<int64_t>(tokens) + c.page_size - 1) >> c.page_log2);
}

// Where row `row` goes: position `pos` of `slot`.
SA_DEV void put_place(const KvPages& c, int row, int slot, int pos, int32_t* slot_map, int32_t* positions) {
  int place = -1;
  if (slot >= 0) {
    const int p = c.block_table[static_cast<int64_t>(slot) * c.max_pages + (pos >> c.page_log2)];
    if (p >= 0 && p < c.num_pages) place = (p << c.page_log2) + (pos & (c.page_size - 1));
  }
  slot_map[row] = place;
  positions[row] = slot >= 0 ? pos : -1;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPages c, const KvPlanArgs a) {
  extern __shared__ uint8_t smem[];
  StepShared& st = *reinterpret_cast<StepShared*>(smem);
  PlanShared& sh = st.p;
  const int n = a.n, tid = threadIdx.x;
  for (int i = tid; i < n; i += kPlanThreads) sh.slot[i] = a.slots[i];
  __syncthreads();
  const uint32_t dup = find_repeats(sh, n);
  int left[kPlanPer], add[kPlanPer], held[kPlanPer];
  uint32_t valid = 0, fits = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = tid + k * kPlanThreads;
    if (i >= n) break;
    const int slot = sh.slot[i];
    add[k] = a.new_tokens[i];
    left[k] = held[k] = 0;
    const bool ok = slot >= 0 && slot < c.num_slots && !(dup >> k & 1u) && add[k] >= 0;
    if (ok) {
      const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_log2;
      const int len = static_cast<int>(min(static_cast<int64_t>(max(c.seqlens[slot], 0)), most));
      const int drop = a.drop != nullptr ? max(a.drop[i], 0) : 0;
      left[k] = max(len - drop, 0);
      held[k] = pages_for(c, len);
      valid |= 1u << k;
      if (static_cast<int64_t>(left[k]) + add[k] <= most) fits |= 1u << k;
    }
    sh.upto[i] = held[k] - pages_for(c, left[k]);
    st.base[i] = pages_for(c, left[k]);
  }
  __syncthreads();
  // where the rank-th page given back, or handed out, stands in the table; it is request i's
  const auto entry_of = [&](int i, int rank) -> int32_t* {
    return c.block_table + static_cast<int64_t>(sh.slot[i]) * c.max_pages + st.base[i] + rank -
           (i > 0 ? sh.upto[i - 1] : 0);
  };
  const int back = scan_needs(sh, n);
  constexpr int kAtOnce = 4;  // pages whose table entries, and then owners, a thread waits for together
  for (int r0 = tid; r0 < back; r0 += kAtOnce * kPlanThreads) {
    int32_t* e[kAtOnce];
    int page[kAtOnce], slot[kAtOnce], owner[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int r = r0 + k * kPlanThreads;
      slot[k] = -1;
      if (r >= back) continue;
      const int i = request_of(sh, n, r);
      slot[k] = sh.slot[i];
      e[k] = entry_of(i, r);
      page[k] = *e[k];
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) owner[k] = slot[k] >= 0 && page[k] >= 0 && page[k] < c.num_pages ? c.owner[page[k]] : -1;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (slot[k] < 0) continue;
      if (owner[k] == slot[k]) c.owner[page[k]] = -1;
      *e[k] = -1;
    }
  }
  __syncthreads();
  uint32_t needs = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = tid + k * kPlanThreads;
    if (i >= n) break;
    const int need = (fits >> k & 1u) ? pages_for(c, left[k] + add[k]) - pages_for(c, left[k]) : 0;
    if (need > 0) needs |= 1u << k;
    sh.upto[i] = need;
  }
  __syncthreads();
  const int need = scan_needs(sh, n);
  const int found = hand_out<-1>(sh, c.owner, c.num_pages, need, [&](int rank, int page) {
    const int i = request_of(sh, n, rank);
    *entry_of(i, rank) = page;
    c.owner[page] = sh.slot[i];
  });
  __syncthreads();
  if (found < need) {  // the request in which the pages ran out, if it had begun
    const int i = request_of(sh, n, found);
    for (int r = (i > 0 ? sh.upto[i - 1] : 0) + tid; r < found; r += kPlanThreads) {
      int32_t* e = entry_of(i, r);
      c.owner[*e] = -1;
      *e = -1;
    }
    __syncthreads();
  }
  uint32_t served = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = tid + k * kPlanThreads;
    if (i >= n) break;
    const bool ok = (fits >> k & 1u) && (!(needs >> k & 1u) || sh.upto[i] <= found);
    if (ok) served |= 1u << k;
    if (valid >> k & 1u) c.seqlens[sh.slot[i]] = left[k] + (ok ? add[k] : 0);
    a.live[i] = ok ? sh.slot[i] : -1;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = tid + k * kPlanThreads;
    if (i >= n) break;
    st.base[i] = (served >> k & 1u) ? left[k] : -1;
    sh.upto[i] = max(add[k], 0);
  }
  __syncthreads();
  const int rows = scan_needs(sh, n);
  for (int i = tid; i <= n; i += kPlanThreads) a.cu[i] = i > 0 ? sh.upto[i - 1] : 0;
  if (a.total > kRowsInPlan) return;
  for (int row = tid; row < a.total; row += kPlanThreads) {
    int slot = -1, pos = 0;
    if (row < rows) {
      const int i = request_of(sh, n, row);
      if (st.base[i] >= 0) {
        slot = sh.slot[i];
        pos = st.base[i] + row - (i > 0 ? sh.upto[i - 1] : 0);
      }
    }
    put_place(c, row, slot, pos, a.slot_map, a.positions);
  }
}

// The rows' places from what the plan left: a served slot's length counts its
// new tokens.  Two warps look for the entries of the CTA's first and last row,
// the threads between those.
__global__ void __launch_bounds__(kMapThreads) kv_map_kernel(const KvPages c, const KvPlanArgs a) {
  __shared__ int range[2];
  const int first = blockIdx.x * (kMapThreads * kMapPer), tid = threadIdx.x, lane = tid & 31;
  cudaGridDependencySynchronize();
  const int rows = a.cu[a.n];
  if (tid < 64) {  // the number of entries that end at or before the row: 32 probes at a time
    const int row = tid < 32 ? first : min(first + kMapThreads * kMapPer, a.total) - 1;
    int lo = 0, hi = a.n;  // the answer lies in [lo, hi]
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const uint32_t done = __ballot_sync(0xffffffffu, at < hi && a.cu[min(at, a.n - 1) + 1] <= row);
      const int k = __popc(done);  // probes 0 .. k - 1 end before it
      if (k < 32) hi = min(hi, lo + k * step);
      if (k > 0) lo += (k - 1) * step + 1;
    }
    if (lane == 0) range[tid >> 5] = lo;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMapPer; ++k) {
    const int row = first + k * kMapThreads + tid;
    if (row >= a.total) break;
    int slot = -1, pos = 0;
    if (row < rows) {
      int lo = range[0], hi = min(range[1], a.n - 1);  // the first with cu[i + 1] > row
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > row)
          hi = mid;
        else
          lo = mid + 1;
      }
      slot = a.live[lo];
      if (slot >= 0) pos = c.seqlens[slot] - (a.cu[lo + 1] - row);
    }
    put_place(c, row, slot, pos, a.slot_map, a.positions);
  }
}

// ---------------------------------------------------------------- write
// A copy: `lanes` lanes take a row (the power of two that covers its 16-byte
// units, 32 at most), several rows in flight each.  70001 tokens x 8 heads out
// of wider rows 44.3 us, 97 % of the copy rate.
constexpr int kWriteThreads = 256;
constexpr int kWriteRows = 4;

__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const KvPages c, const KvWriteArgs a, int lanes_log2) {
  const int lanes = 1 << lanes_log2, in_row = threadIdx.x & (lanes - 1);
  const int units = c.num_heads_kv * (kHeadDim / 8);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kWriteThreads >> lanes_log2);
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (kWriteThreads >> lanes_log2) + (threadIdx.x >> lanes_log2);
  const int64_t places = static_cast<int64_t>(c.num_pages) << c.page_log2;
  for (int64_t row0 = group * kWriteRows; row0 < a.rows; row0 += groups * kWriteRows) {
    int64_t to[kWriteRows];
#pragma unroll
    for (int r = 0; r < kWriteRows; ++r) {
      const int64_t place = row0 + r < a.rows ? a.slot_map[row0 + r] : -1;
      to[r] = place >= 0 && place < places ? place * units : -1;
    }
    for (int u = in_row; u < units; u += lanes) {
      uint4 kv[kWriteRows][2];
#pragma unroll
      for (int r = 0; r < kWriteRows; ++r) {
        if (to[r] < 0) continue;
        kv[r][0] = __ldcs(reinterpret_cast<const uint4*>(a.k + (row0 + r) * a.k_stride) + u);
        kv[r][1] = __ldcs(reinterpret_cast<const uint4*>(a.v + (row0 + r) * a.v_stride) + u);
      }
#pragma unroll
      for (int r = 0; r < kWriteRows; ++r) {
        if (to[r] < 0) continue;
        reinterpret_cast<uint4*>(c.k)[to[r] + u] = kv[r][0];
        reinterpret_cast<uint4*>(c.v)[to[r] + u] = kv[r][1];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPages& c, const KvPlanArgs& a, cudaStream_t s) {
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(kv_plan_kernel, sizeof(StepShared));
  if (e != cudaSuccess) return e;
  kv_plan_kernel<<<1, kPlanThreads, sizeof(StepShared), s>>>(c, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.total <= kRowsInPlan) return e;
  // waits for the plan on the device, so that its launch does not come on top
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(a.total, kMapThreads * kMapPer));
  cfg.blockDim = dim3(kMapThreads);
  cfg.stream = s;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_map_kernel, c, a);
}

cudaError_t launch_kv_write(const KvPages& c, const KvWriteArgs& a, cudaStream_t s) {
  int lanes_log2 = 3;
  while (lanes_log2 < 5 && (1 << lanes_log2) < c.num_heads_kv * (kHeadDim / 8)) ++lanes_log2;
  const int per_cta = (kWriteThreads >> lanes_log2) * kWriteRows;
  const int ctas = std::min(ceil_div(a.rows, per_cta), device_sms() * 32);
  kv_write_kernel<<<ctas, kWriteThreads, 0, s>>>(c, a, lanes_log2);
  return cudaGetLastError();
}

}  // namespace sa

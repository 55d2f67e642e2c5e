// The 4-bit paged cache: handing out, sharing, freeing and packing its pages,
// and writing and reading its tokens.
//
// Page state is two arrays and a table on the device, so a rollout loop never
// waits for the host: a page is free when its count is zero, requests take
// the lowest-numbered free pages in the order in which they stand, and every
// result is the same from run to run.
#include "kv4.cuh"

#include <algorithm>

namespace sa {
namespace {

using namespace kv4;

// ------------------------------------------------------------ page hand-out
// reserve and fork run as ONE CTA: what they decide (who is served, and with
// which pages) is a scan over the requests and a scan over the counts.
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

// Calls give(rank, page) for the lowest free pages, rank = 0 .. need - 1, and
// returns how many there are, at most `need`.  Free pages come in runs, which
// one thread finds: they go through a list, so that all threads hand out.
template <class F>
SA_DEV int hand_out(PlanShared& sh, const Kv4Cache& c, int need, F give) {
  int found = 0;
  for (int64_t base = 0; base < c.num_pages && found < need; base += kPlanThreads * kScanPages) {
    const int64_t p0 = base + threadIdx.x * kScanPages;
    uint32_t free_bits = 0;
    if (p0 + kScanPages <= c.num_pages) {
      int4 v[kScanPages / 4];
#pragma unroll
      for (int k = 0; k < kScanPages / 4; ++k) v[k] = reinterpret_cast<const int4*>(c.refcount + p0)[k];
#pragma unroll
      for (int k = 0; k < kScanPages / 4; ++k)
        free_bits |= static_cast<uint32_t>((v[k].x == 0) | (v[k].y == 0) << 1 | (v[k].z == 0) << 2 | (v[k].w == 0) << 3)
                     << (4 * k);
    } else {
      for (int k = 0; p0 + k < c.num_pages; ++k) free_bits |= static_cast<uint32_t>(c.refcount[p0 + k] == 0) << k;
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

// reserve: slot i grows by add[i] tokens.  Its table entries and the pages'
// counts are written as the pages are found; where the pages run out inside a
// request, what that request was given is taken back.
__global__ void __launch_bounds__(kPlanThreads) kv4_reserve_kernel(const Kv4Cache c, const int32_t* __restrict__ slots,
                                                                   const int32_t* __restrict__ add, int n,
                                                                   int32_t* __restrict__ done) {
  extern __shared__ uint8_t smem[];
  PlanShared& sh = *reinterpret_cast<PlanShared*>(smem);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) sh.slot[i] = slots[i];
  __syncthreads();
  const uint32_t dup = find_repeats(sh, n);
  int len[kPlanPer], grow[kPlanPer];
  uint32_t valid = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = threadIdx.x + k * kPlanThreads;
    if (i >= n) break;
    const int slot = sh.slot[i];
    grow[k] = add[i];
    len[k] = slot_len(c, slot);
    const int64_t size = static_cast<int64_t>(len[k]) + grow[k];
    const bool ok = slot >= 0 && slot < c.num_slots && !(dup >> k & 1u) && grow[k] >= 0 &&
                    size <= (static_cast<int64_t>(c.max_pages) << c.page_log2);
    if (ok) valid |= 1u << k;
    const int up = c.page_size - 1;
    sh.upto[i] = ok ? static_cast<int>((size + up) >> c.page_log2) - ((len[k] + up) >> c.page_log2) : 0;
  }
  __syncthreads();
  uint32_t needs = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = threadIdx.x + k * kPlanThreads;
    if (i < n && sh.upto[i] > 0) needs |= 1u << k;
  }
  const int need = scan_needs(sh, n);
  const auto entry = [&](int rank) -> int32_t* {
    const int i = request_of(sh, n, rank), slot = sh.slot[i];
    const int col = (slot_len(c, slot) + c.page_size - 1 >> c.page_log2) + rank - (i > 0 ? sh.upto[i - 1] : 0);
    return c.page_table + static_cast<int64_t>(slot) * c.max_pages + col;
  };
  const int found = hand_out(sh, c, need, [&](int rank, int page) {
    *entry(rank) = page;
    c.refcount[page] = 1;
  });
  __syncthreads();
  if (found < need) {  // the request in which the pages ran out, if it had begun
    const int i = request_of(sh, n, found);
    for (int r = (i > 0 ? sh.upto[i - 1] : 0) + threadIdx.x; r < found; r += kPlanThreads) {
      int32_t* e = entry(r);
      c.refcount[*e] = 0;
      *e = -1;
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = threadIdx.x + k * kPlanThreads;
    if (i >= n) break;
    const bool ok = (valid >> k & 1u) && (!(needs >> k & 1u) || sh.upto[i] <= found);
    if (ok) c.seqlens[sh.slot[i]] = len[k] + grow[k];
    done[i] = ok;
  }
}

// fork, first part (512 forks from a pool of 2 k pages: 9 us, one CTA's scans
// and their barriers; the second part, 20 MB of open pages, 7.5 us): who is served, the new pages, lengths.  The second part
// shares the full pages and copies the open one.
__global__ void __launch_bounds__(kPlanThreads) kv4_fork_plan_kernel(const Kv4Cache c, const int32_t* __restrict__ src,
                                                                     const int32_t* __restrict__ dst, int n,
                                                                     int32_t* __restrict__ done) {
  extern __shared__ uint8_t smem[];
  PlanShared& sh = *reinterpret_cast<PlanShared*>(smem);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) sh.slot[i] = dst[i];
  __syncthreads();
  const uint32_t dup = find_repeats(sh, n);
  int len[kPlanPer];
  uint32_t valid = 0, needs = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = threadIdx.x + k * kPlanThreads;
    if (i >= n) break;
    const int from = src[i], to = sh.slot[i];
    len[k] = slot_len(c, from);
    const bool ok = from >= 0 && from < c.num_slots && to >= 0 && to < c.num_slots && !(dup >> k & 1u) &&
                    slot_len(c, to) == 0 && len[k] <= (static_cast<int64_t>(c.max_pages) << c.page_log2);
    const bool open = ok && (len[k] & (c.page_size - 1)) != 0;
    if (ok) valid |= 1u << k;
    if (open) needs |= 1u << k;
    sh.upto[i] = open;
  }
  __syncthreads();  // every length has been read
  const int need = scan_needs(sh, n);
  const int found = hand_out(sh, c, need, [&](int rank, int page) {
    const int i = request_of(sh, n, rank);
    // the source's length again: a source with an open page is no destination, so nobody writes it here
    const int col = slot_len(c, src[i]) >> c.page_log2;
    c.page_table[static_cast<int64_t>(sh.slot[i]) * c.max_pages + col] = page;
    c.refcount[page] = 1;
  });
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int i = threadIdx.x + k * kPlanThreads;
    if (i >= n) break;
    const bool ok = (valid >> k & 1u) && (!(needs >> k & 1u) || sh.upto[i] <= found);
    if (ok) c.seqlens[sh.slot[i]] = len[k];
    done[i] = ok;
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// Copies `units` 16-byte units, the CTA's share `part` of `parts`: `unit(i)` gives the offset of unit i on both sides.
template <class F>
SA_DEV void copy_units(const uint8_t* from, uint8_t* to, int units, int part, int parts, F unit) {
  for (int i0 = part * kCopyThreads * kCopyUnroll; i0 < units; i0 += parts * kCopyThreads * kCopyUnroll) {
    uint4 v[kCopyUnroll];
    int64_t at[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
      const int i = i0 + k * kCopyThreads + threadIdx.x;
      at[k] = i < units ? unit(i) : -1;
      if (at[k] >= 0) v[k] = *reinterpret_cast<const uint4*>(from + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
      if (at[k] >= 0) *reinterpret_cast<uint4*>(to + at[k]) = v[k];
  }
}

__global__ void __launch_bounds__(kCopyThreads) kv4_fork_copy_kernel(const Kv4Cache c, const int32_t* __restrict__ src,
                                                                     const int32_t* __restrict__ dst,
                                                                     const int32_t* __restrict__ done) {
  const int i = blockIdx.x;
  if (!done[i]) return;
  const int from = src[i], to = dst[i], len = slot_len(c, to);
  const int full = len >> c.page_log2;
  const int32_t* row = c.page_table + static_cast<int64_t>(from) * c.max_pages;
  int32_t* out = c.page_table + static_cast<int64_t>(to) * c.max_pages;
  if (blockIdx.y == 0)
    for (int j = threadIdx.x; j < full; j += kCopyThreads) {
      const int p = row[j];
      out[j] = p;
      if (p >= 0 && p < c.num_pages) atomicAdd(c.refcount + p, 1);
    }
  const int open = len & (c.page_size - 1);
  if (open == 0) return;
  const int old_page = row[full], new_page = out[full];
  if (old_page < 0 || old_page >= c.num_pages) {  // nothing to copy: these tokens read as NaN from the copy too
    if (blockIdx.y == 0 && threadIdx.x == 0) {
      out[full] = -1;
      c.refcount[new_page] = 0;
    }
    return;
  }
  const int per_head = ((open + kBlockTokens - 1) / kBlockTokens) * (kBlockBytes / 16);
  const int64_t head = static_cast<int64_t>(kBlockBytes) << c.blocks_log2;
  copy_units(c.pages + old_page * head * c.num_heads_kv, c.pages + new_page * head * c.num_heads_kv,
             per_head * c.num_heads_kv, blockIdx.y, gridDim.y,
             [&](int u) { return (u / per_head) * head + static_cast<int64_t>(u % per_head) * 16; });
}

// free: the exchange of the length lets exactly one of several entries that
// name a slot act.
__global__ void __launch_bounds__(128) kv4_free_kernel(const Kv4Cache c, const int32_t* __restrict__ slots) {
  __shared__ int held_sh;
  const int slot = slots[blockIdx.x];
  if (slot < 0 || slot >= c.num_slots) return;
  if (threadIdx.x == 0) {
    const int len = max(atomicExch(c.seqlens + slot, 0), 0);
    held_sh = min(static_cast<int>((static_cast<int64_t>(len) + c.page_size - 1) >> c.page_log2), c.max_pages);
  }
  __syncthreads();
  int32_t* row = c.page_table + static_cast<int64_t>(slot) * c.max_pages;
  for (int j = threadIdx.x; j < held_sh; j += 128) {
    const int p = row[j];
    if (p >= 0 && p < c.num_pages) atomicSub(c.refcount + p, 1);
    row[j] = -1;
  }
}

// ------------------------------------------------------------ compaction
// Each live page gets its new number (a chunk of counts sums the chunks
// before it) and a place in the list of live pages; then come the copies,
// shared evenly over the CTAs by the list, with tables and counts.  In pools
// of more than kDirectPages a launch before those counts the chunks; in
// smaller ones a chunk reads all counts before its own, which costs less (12.6 k
// pages: 5.1 us instead of 7.1 + 3.5).  The copies run at 7.1 TB/s, read and
// written (100 MB live in 28 us).
constexpr int kChunkThreads = 256;
constexpr int kChunkPer = 4;
constexpr int kChunk = kChunkThreads * kChunkPer;

struct CompactWs {
  int32_t* per_chunk;  // [chunks]
  int32_t* place;      // [num_pages] new number or -1
  int32_t* list;       // [live] old numbers
};

constexpr int kDirectPages = 32768;

SA_DEV uint32_t live_bits(const Kv4Cache& c, int64_t p0) {
  if (p0 + kChunkPer <= c.num_pages) {
    const int4 v = *reinterpret_cast<const int4*>(c.refcount + p0);
    return (v.x > 0) | (v.y > 0) << 1 | (v.z > 0) << 2 | (v.w > 0) << 3;
  }
  uint32_t bits = 0;
  for (int k = 0; p0 + k < c.num_pages; ++k) bits |= static_cast<uint32_t>(c.refcount[p0 + k] > 0) << k;
  return bits;
}

__global__ void __launch_bounds__(kChunkThreads) kv4_live_kernel(const Kv4Cache c, const CompactWs w) {
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * kChunkPer;
  __shared__ int warp[32], total;
  block_scan(__popc(live_bits(c, p0)), warp, &total);
  if (threadIdx.x == 0) w.per_chunk[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kChunkThreads) kv4_place_kernel(const Kv4Cache c, const CompactWs w, bool direct,
                                                                  int32_t* __restrict__ count) {
  __shared__ int warp[32], total;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * kChunkPer;
  const uint32_t bits = live_bits(c, p0);
  int before = 0;
  if (direct) {
#pragma unroll 8
    for (int i = 0; i < static_cast<int>(blockIdx.x); ++i)
      before += __popc(live_bits(c, static_cast<int64_t>(i) * kChunk + threadIdx.x * kChunkPer));
  } else {
    for (int i = threadIdx.x; i < static_cast<int>(blockIdx.x); i += kChunkThreads) before += w.per_chunk[i];
  }
  block_scan(before, warp, &total);
  const int base = total;
  const int mine = __popc(bits);
  int at = base + block_scan(mine, warp, &total) - mine;
#pragma unroll
  for (int k = 0; k < kChunkPer; ++k) {
    if (p0 + k >= c.num_pages) break;
    const bool live = bits >> k & 1u;
    w.place[p0 + k] = live ? at : -1;
    if (live) w.list[at++] = static_cast<int32_t>(p0 + k);
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *count = base + total;
}

__global__ void __launch_bounds__(kCopyThreads) kv4_compact_kernel(const Kv4Cache from, const Kv4Cache to,
                                                                   const CompactWs w,
                                                                   const int32_t* __restrict__ count) {
  const int live = *count;
  if (live > to.num_pages) return;  // it does not fit: `to` stays as it was
  const int64_t page_bytes = (static_cast<int64_t>(kBlockBytes) << from.blocks_log2) * from.num_heads_kv;
  const int units = static_cast<int>(page_bytes / 16);
  for (int r = blockIdx.x; r < live; r += gridDim.x)
    copy_units(from.pages + w.list[r] * page_bytes, to.pages + r * page_bytes, units, 0, 1,
               [](int u) { return static_cast<int64_t>(u) * 16; });
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  for (int64_t r = first; r < to.num_pages; r += stride) to.refcount[r] = r < live ? from.refcount[w.list[r]] : 0;
  const int64_t entries = static_cast<int64_t>(from.num_slots) * from.max_pages;
  for (int64_t e = first; e < entries; e += stride) {
    const int slot = static_cast<int>(e / from.max_pages), col = static_cast<int>(e % from.max_pages);
    const int len = slot_len(from, slot);
    if (col == 0) to.seqlens[slot] = len;
    const int p = from.page_table[e];
    const bool held = (static_cast<int64_t>(col) << from.page_log2) < len && p >= 0 && p < from.num_pages;
    to.page_table[e] = held ? w.place[p] : -1;
  }
}

// ------------------------------------------------------------ tokens
// One warp per (block of 16 tokens, head).  Entry b's rows [cu[b], cu[b+1])
// are the last positions of its slot; its blocks take the numbers from
// cu[b] / 16 + 2 b on (an entry of n rows touches at most n / 16 + 2 blocks),
// so that a block finds its entry by a search in cu alone.
struct TokenArgs {
  const int32_t* slots;
  const int32_t* cu;  // or nullptr: total / n rows per entry
  int n, total, per;
};

struct BlockPlace {
  int slot, blk, first_row, row0, lo, hi;  // positions [lo, hi) of the slot belong to rows row0 + position - lo
};

SA_DEV int cu_at(const TokenArgs& a, int b) {
  return a.cu == nullptr ? b * a.per : min(max(a.cu[b], 0), a.total);
}

// All lanes of a warp ask for one block.
SA_DEV bool find_block(const Kv4Cache& c, const TokenArgs& a, int id, BlockPlace& out) {
  int lo = 0, left = a.n;  // the last entry whose first number is <= id lies in [lo, lo + left)
  while (left > 1) {       // 32 of them looked at at once
    const int step = (left + 31) / 32, at = static_cast<int>(threadIdx.x & 31) * step;
    const bool le = at == 0 || (at < left && (cu_at(a, lo + at) >> 4) + 2 * (lo + at) <= id);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));
    lo += last * step;
    left = min(step, left - last * step);
  }
  const int r0 = cu_at(a, lo), r1 = max(cu_at(a, lo + 1), r0);
  const int slot = a.slots[lo], len = slot_len(c, slot);
  out.slot = slot;
  out.row0 = r0;
  out.lo = len - (r1 - r0);
  out.hi = len;
  out.blk = (out.lo >> 4) + id - (r0 >> 4) - 2 * lo;
  return id >= (r0 >> 4) + 2 * lo && out.blk * kBlockTokens < len;
}

// x / d for one divisor and many x (in pairs), correctly rounded, with r = 1 / d
// rounded to nearest: one residual and one correction (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34 (1), 1990).  Quotients so small that the residual underflows are
// far below the smallest scale and round to the code 0 either way.
struct Divisor {
  float2 neg, r;  // -d and 1 / d, twice
  SA_DEV explicit Divisor(float d) {
    const float inv = __fdiv_rn(1.f, d);
    neg = make_float2(-d, -d);
    r = make_float2(inv, inv);
  }
  SA_DEV Divisor(float d, float inv) : neg(make_float2(-d, -d)), r(make_float2(inv, inv)) {}
  SA_DEV float2 operator()(float2 x) const {
    const float2 q = fmul2(x, r);
    return ffma2(ffma2(q, neg, x), r, q);
  }
};

// |a| and |b|, the larger one; NaN if one of them is.
SA_DEV float max_abs_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

// The e4m3 scale of 16 dims whose largest |y| is `top` (NaN or infinite: not
// all of them are finite).
struct GroupScale {
  uint32_t byte;
  float s, r;  // the scale's value and its reciprocal; r = 0 makes all codes 0
};

SA_DEV GroupScale group_scale(float top) {
  GroupScale g;
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(two) : "f"(0.f), "f"(fminf(__fdiv_rn(top, 6.f), 448.f)));
  g.byte = two & 0xffu;
  if (!(top < INFINITY)) g.byte = kNaNScale;
  g.s = f16x2_to_f32(e4m3x2(g.byte)).x;
  g.r = g.s > 0.f ? __fdiv_rn(1.f, g.s) : 0.f;
  return g;
}

SA_DEV uint32_t e2m1_codes(const float2 (&y)[4], const GroupScale& g) {  // 8 values -> 8 nibbles
  const Divisor by(g.s, g.r);
  const float2 a = by(y[0]), b = by(y[1]), c = by(y[2]), d = by(y[3]);
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}

// y = x / factor of 8 dims; returns the largest |y| (NaN if one is).
SA_DEV float scaled8(uint4 v, const Divisor& factor, float2 (&y)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = factor(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)));
    top = max_abs_nan(top, max_abs_nan(y[i].x, y[i].y));
  }
  return top;
}

// Measured: 83 k tokens x 8 heads in 46.8 us (220 MB, 32.5 us at the copy
// rate), bound by the loads' latency: a third of the warps, 56 % of the issue
// slots, most stalls on the rows' loads, which a warp with one block has nothing
// to overlap with (one dim per instruction: 63 us).  64 x 1 tokens in about 4 us,
// a chain of loads (offset, slot, length, page).
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4Cache c, const TokenArgs a,
                                                         const __nv_bfloat16* __restrict__ k,
                                                         const __nv_bfloat16* __restrict__ v, int64_t warps) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (w >= warps) return;
  const int head = static_cast<int>(w % c.num_heads_kv);
  BlockPlace pl;
  if (!find_block(c, a, static_cast<int>(w / c.num_heads_kv), pl)) return;
  if (pl.blk < 0) return;
  const int page = page_of(c, pl.slot, pl.blk);
  if (page < 0) return;
  uint8_t* block = block_ptr(c, page, head, pl.blk);
  const int lane = threadIdx.x & 31, g = lane_g(), t = lane_t();
  const int pos0 = pl.blk * kBlockTokens;
  const auto mine = [&](int token) { return pos0 + token >= pl.lo && pos0 + token < pl.hi; };
  const auto row = [&](int token) {
    return (static_cast<int64_t>(pl.row0 + pos0 + token - pl.lo) * c.num_heads_kv + head) * kHeadDim;
  };
  // all loads first
  uint4 kv[2][2], vv[4];
  bool in[2];
  uint32_t v_in = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    in[h] = mine(g + 8 * h);
    kv[h][0] = kv[h][1] = make_uint4(0, 0, 0, 0);
    if (in[h]) {
      const uint4* x = reinterpret_cast<const uint4*>(k + row(g + 8 * h) + 16 * t);
      kv[h][0] = __ldcs(x);
      kv[h][1] = __ldcs(x + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int token = 2 * t + (i & 1) + 8 * (i >> 1);
    vv[i] = make_uint4(0, 0, 0, 0);
    if (mine(token)) {
      vv[i] = __ldcs(reinterpret_cast<const uint4*>(v + row(token) + 8 * g));
      v_in |= 1u << i;
    }
  }
  {  // keys: tokens g and g + 8, the 16 dims of scale t
    const Divisor factor(c.k_scale[head]);
    uint32_t codes[2][2], scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 y[2][4];
      const float top = scaled8(kv[h][0], factor, y[0]);
      const GroupScale gs = group_scale(max_abs_nan(top, scaled8(kv[h][1], factor, y[1])));
      codes[h][0] = e2m1_codes(y[0], gs);
      codes[h][1] = e2m1_codes(y[1], gs);
      scale[h] = gs.byte;
    }
    if (in[0] && in[1]) {
      *reinterpret_cast<uint4*>(block + 16 * lane) = make_uint4(codes[0][0], codes[0][1], codes[1][0], codes[1][1]);
      *reinterpret_cast<uint16_t*>(block + kKScales + 2 * lane) = static_cast<uint16_t>(scale[0] | scale[1] << 8);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (in[h]) {
          *reinterpret_cast<uint2*>(block + 16 * lane + 8 * h) = make_uint2(codes[h][0], codes[h][1]);
          block[kKScales + 2 * lane + h] = static_cast<uint8_t>(scale[h]);
        }
    }
  }
  {  // values: tokens 2t, 2t+1, 2t+8, 2t+9, 8 dims; the other 8 of their scale are lane ^ 4's
    const Divisor factor(c.v_scale[head]);
    uint32_t codes[4], scales = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 y[4];
      float top = scaled8(vv[i], factor, y);
      top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, 4));
      const GroupScale gs = group_scale(top);
      codes[i] = e2m1_codes(y, gs);
      scales |= gs.byte << (8 * i);
    }
    if (v_in == 15u) {
      *reinterpret_cast<uint4*>(block + kVCodes + 16 * lane) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
      if ((g & 1) == 0) *reinterpret_cast<uint32_t*>(block + kVScales + 4 * (4 * (g >> 1) + t)) = scales;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v_in >> i & 1u) {
          *reinterpret_cast<uint32_t*>(block + kVCodes + 16 * lane + 4 * i) = codes[i];
          if ((g & 1) == 0) block[kVScales + 4 * (4 * (g >> 1) + t) + i] = static_cast<uint8_t>(scales >> (8 * i));
        }
    }
  }
}

// One f16 pair of exact values -> bf16 pair under the head's factor, rounded once from fp32.
SA_DEV uint32_t out_pair(uint32_t v, float factor) {
  const float2 f = f16x2_to_f32(v);
  return pack_bf16(f.x * factor, f.y * factor);
}

// Measured: 83 k tokens x 8 heads in 31 us, the copy rate (the pages come from L2).
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4Cache c, const TokenArgs a,
                                                       __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v,
                                                       int64_t warps) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (w >= warps) return;
  const int head = static_cast<int>(w % c.num_heads_kv);
  BlockPlace pl;
  if (!find_block(c, a, static_cast<int>(w / c.num_heads_kv), pl)) return;
  const int lane = threadIdx.x & 31, g = lane_g(), t = lane_t();
  // A block before the sequence's begin reads as zeros, one without a page as NaN.
  uint4 kc = make_uint4(0, 0, 0, 0), vc = kc;
  uint32_t ks = 0, vs = 0;
  if (pl.blk >= 0) {
    const int page = page_of(c, pl.slot, pl.blk);
    ks = kNaNScale * 0x0101u;
    vs = kNaNScale * 0x01010101u;
    if (page >= 0) {
      const uint8_t* block = block_ptr(c, page, head, pl.blk);
      kc = *reinterpret_cast<const uint4*>(block + 16 * lane);
      vc = *reinterpret_cast<const uint4*>(block + kVCodes + 16 * lane);
      ks = *reinterpret_cast<const uint16_t*>(block + kKScales + 2 * lane);
      vs = *reinterpret_cast<const uint32_t*>(block + kVScales + 4 * (4 * (g >> 1) + t));
    }
  }
  const int pos0 = pl.blk * kBlockTokens;
  const auto mine = [&](int token) { return pos0 + token >= pl.lo && pos0 + token < pl.hi; };
  const auto row = [&](int token) {
    return (static_cast<int64_t>(pl.row0 + pos0 + token - pl.lo) * c.num_heads_kv + head) * kHeadDim;
  };
  const auto put = [&](__nv_bfloat16* to, uint32_t codes, uint32_t scale2, float factor) {
    uint32_t d[4];
    e2m1x8(codes, d);
    *reinterpret_cast<uint4*>(to) =
        make_uint4(out_pair(hmul2(d[0], scale2), factor), out_pair(hmul2(d[1], scale2), factor),
                   out_pair(hmul2(d[2], scale2), factor), out_pair(hmul2(d[3], scale2), factor));
  };
  const uint32_t k2 = e4m3x2(ks), v01 = e4m3x2(vs), v23 = e4m3x2(vs >> 16);
  const float kf = c.k_scale[head], vf = c.v_scale[head];
  if (mine(g)) {
    const uint32_t s = __byte_perm(k2, 0, 0x1010);
    put(k + row(g) + 16 * t, kc.x, s, kf);
    put(k + row(g) + 16 * t + 8, kc.y, s, kf);
  }
  if (mine(g + 8)) {
    const uint32_t s = __byte_perm(k2, 0, 0x3232);
    put(k + row(g + 8) + 16 * t, kc.z, s, kf);
    put(k + row(g + 8) + 16 * t + 8, kc.w, s, kf);
  }
  if (mine(2 * t)) put(v + row(2 * t) + 8 * g, vc.x, __byte_perm(v01, 0, 0x1010), vf);
  if (mine(2 * t + 1)) put(v + row(2 * t + 1) + 8 * g, vc.y, __byte_perm(v01, 0, 0x3232), vf);
  if (mine(2 * t + 8)) put(v + row(2 * t + 8) + 8 * g, vc.z, __byte_perm(v23, 0, 0x1010), vf);
  if (mine(2 * t + 9)) put(v + row(2 * t + 9) + 8 * g, vc.w, __byte_perm(v23, 0, 0x3232), vf);
}

int64_t token_warps(const Kv4Cache& c, const TokenArgs& a) {
  return (static_cast<int64_t>(a.total) / kBlockTokens + 2 * static_cast<int64_t>(a.n)) * c.num_heads_kv;
}

}  // namespace

cudaError_t launch_kv4_reserve(const Kv4Cache& c, const int32_t* slots, const int32_t* add, int n, int32_t* done,
                               cudaStream_t s) {
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(kv4_reserve_kernel, sizeof(PlanShared));
  if (e != cudaSuccess) return e;
  kv4_reserve_kernel<<<1, kPlanThreads, sizeof(PlanShared), s>>>(c, slots, add, n, done);
  return cudaGetLastError();
}

cudaError_t launch_kv4_fork(const Kv4Cache& c, const int32_t* src, const int32_t* dst, int n, int32_t* done,
                            cudaStream_t s) {
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(kv4_fork_plan_kernel, sizeof(PlanShared));
  if (e != cudaSuccess) return e;
  kv4_fork_plan_kernel<<<1, kPlanThreads, sizeof(PlanShared), s>>>(c, src, dst, n, done);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long units = (static_cast<long long>(kBlockBytes) << c.blocks_log2) * c.num_heads_kv / 16;
  const int parts = static_cast<int>(std::min<long long>(ceil_div(units, kCopyThreads * kCopyUnroll), 64));
  kv4_fork_copy_kernel<<<dim3(n, parts), kCopyThreads, 0, s>>>(c, src, dst, done);
  return cudaGetLastError();
}

cudaError_t launch_kv4_free(const Kv4Cache& c, const int32_t* slots, int n, cudaStream_t s) {
  kv4_free_kernel<<<n, 128, 0, s>>>(c, slots);
  return cudaGetLastError();
}

size_t kv4_compact_workspace_bytes(int num_pages) {
  return (static_cast<size_t>(ceil_div(num_pages, kChunk)) + 2 * static_cast<size_t>(num_pages)) * 4;
}

cudaError_t launch_kv4_compact(const Kv4Cache& from, const Kv4Cache& to, int32_t* count, void* workspace,
                               cudaStream_t s) {
  const int chunks = ceil_div(from.num_pages, kChunk);
  CompactWs w;
  w.per_chunk = static_cast<int32_t*>(workspace);
  w.place = w.per_chunk + chunks;
  w.list = w.place + from.num_pages;
  const bool direct = from.num_pages <= kDirectPages;
  cudaError_t e;
  if (!direct) {
    kv4_live_kernel<<<chunks, kChunkThreads, 0, s>>>(from, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  kv4_place_kernel<<<chunks, kChunkThreads, 0, s>>>(from, w, direct, count);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  kv4_compact_kernel<<<device_sms() * 8, kCopyThreads, 0, s>>>(from, to, w, count);
  return cudaGetLastError();
}

cudaError_t launch_kv4_append(const Kv4Cache& c, const int32_t* slots, int n, const int32_t* cu, int total,
                              const void* k, const void* v, cudaStream_t s) {
  const TokenArgs a{slots, cu, n, total, total / n};
  const int64_t warps = token_warps(c, a);
  kv4_append_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(
      c, a, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), warps);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Cache& c, const int32_t* slots, int n, const int32_t* cu, int total, void* k,
                            void* v, cudaStream_t s) {
  const TokenArgs a{slots, cu, n, total, total / n};
  const int64_t warps = token_warps(c, a);
  kv4_read_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(
      c, a, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), warps);
  return cudaGetLastError();
}

}  // namespace sa

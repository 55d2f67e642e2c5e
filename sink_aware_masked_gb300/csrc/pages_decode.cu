// Decode forward over pages of bf16 keys and values: the new rows of each
// sequence against its whole history, with the mask, sink and lse of the
// contiguous decode forward; 1 row a sequence in an ordinary step, several
// where drafted tokens are attended to, and not the same number everywhere.
//
//   s = scale <q, K_k>,  l = log sum_{visible} e^s,  o = sigmoid(l - sink) softmax(s) V
//
// 256 bytes per key and kv head, and 4 x 64 x rows operations on them: a
// stream over the pages, bound by HBM up to some 64 rows.  Keys and values
// come as TMA boxes of 32 tokens (two of 16 where a page has 16), each warp
// through a ring of its own, and are multiplied by warp-level matrix
// instructions with keys and dims on the 16-wide side, so that 8 query rows
// fill the 8-wide side:
//   S^T [16 keys x 8 rows] = K [16 x 64] Q^T,   O^T [64 dims x 8 rows] += V^T [64 x 16] P^T
//
// The softmax keeps a reference score m per row that need not be the maximum:
// it moves (and O and the sums are rescaled) only when a score exceeds it by
// more than 8 log2 units.  A key at the reference has P = 2^-8, so P is at
// most 1.  P is rounded to bf16 for the product (off by 2^-9 of itself at
// most), and O is divided by the sum of the rounded P, so that one key alone
// gives its value exactly; lse takes the fp32 sum of the unrounded ones.
//
// Work: the visible turns (32 tokens) of all (sequence, kv head) pairs in one
// line, each as long as it costs, cut into equal shares, one per worker.  A worker is a CTA, whose warps
// take a pair's turns in turn and merge in shared memory; or, where there are
// many pairs with few turns each, a single warp, which takes whole pairs.  A
// pair cut between CTAs leaves partial results in the workspace, and the last
// CTA of the pair to arrive merges them in order.  Above 48 rows two or four
// warps share a ring and split the rows.
//
// Measured (GB300): 32 x 8192 keys, 64/8 heads, 88.2 us (537 MB: 91 % of the
// copy rate); 8 x 32768 keys x 1 to 5 rows 121 us (514 MB, 63 %: dependent
// instructions, 8 warps an SM at 255 registers); 200 windowed sequences 17.9 us
// (3000 instructions of one pair per warp); one sequence of 37 keys 6.1 us.
#include "shares.cuh"
#include "tc.cuh"
#include "tmap.h"

#include <algorithm>
#include <type_traits>

#include "internal.h"

namespace sa {
namespace {

constexpr int kTurn = 32;                          // tokens of a turn
constexpr int kTurnHalf = kTurn * kHeadDim * 2;    // bytes of its keys (or values)
constexpr int kTurnBytes = 2 * kTurnHalf;
constexpr int kBoxBytes = kTurnHalf / 2;           // 16 tokens
constexpr int kRowPad = 68;                        // floats per row in shared memory
constexpr float kSlack = 8.f;                      // log2 units a score may exceed its row's reference
constexpr int kPartPad = 4;                        // floats of statistics per row of a partial result
// Partial rows that the CTAs of one SM can leave in the workspace: two cut pairs each.
constexpr int kPartRowsPerSm = 256;

// What a turn costs a CTA, in places of the line that is shared out, and a tile
// of 8 rows on top; what beginning a pair costs.  (8 x 32768 keys x 1 to 5 rows:
// 123.5 us with 7 and 2, 134 with 7 and 1, 133 with 4 and 2, 141 with 2 and 2,
// 152 without the tiles; the pairs' cost shows little between 20 and 60.)
constexpr int kTurnCost = 7, kTileCost = 2, kPairCost = 60;
// Turns of the longest pair up to which warps work alone, each on whole pairs
// (200 sequences of 6 visible turns: 17.9 us; the 4-bit cache's decode, of the
// same build, takes 10.6 this way and 40.9 by CTAs and shares).
constexpr int kAloneTurns = 24;

struct PageDecK {
  CUtensorMap tm_k, tm_v;
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* slots;
  const int32_t* cu;
  const __nv_bfloat16* q;
  const float* sink;
  __nv_bfloat16* o;
  float* lse;
  float* part;
  int* counters;  // [pairs]
  int* status;
  int num_pages, page_log2, num_slots, max_pages, num_heads_kv;
  int num_seqs, total_rows, n, hq, group, window, prefix;
  int row_groups;        // of a pair, where warps are alone: a warp has every row_groups-th tile
  uint32_t group_magic;  // ceil(2^16 / group)
  float coef;            // scale * log2 e
  // row / group, exact while row * group <= 2^16 (rows and groups are up to 128)
  SA_DEV int row_of_seq(int row) const { return static_cast<int>(row * group_magic >> 16); }
};

// D = A B, A 16 x 16 (keys), B 16 x 8.
SA_DEV void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// D += A B; nothing keeps the compiler from moving it among the loads.
SA_DEV void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 16-bit transpose across the warp.
SA_DEV uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(v));
  return d;
}

SA_DEV float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

SA_DEV float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
SA_DEV float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// Bits 15 and 31 are set where a half has an exponent of ones (an infinity or a NaN).
SA_DEV uint32_t ones_exponent(uint32_t v) { return (v & 0x7fff7fffu) + 0x00800080u; }

// A sequence of the call: its slot, length, and rows row0 .. row0 + n - 1 of q;
// `rows` of a pair (query heads times rows of q) are computed.
struct Seq {
  int slot, len, row0, n, rows;
};

SA_DEV Seq sequence(const PageDecK& p, int b) {
  Seq s;
  s.slot = p.slots[b];
  s.len = 0;
  if (s.slot >= 0 && s.slot < p.num_slots)
    s.len = min(static_cast<long long>(max(p.seqlens[s.slot], 0)), static_cast<long long>(p.max_pages) << p.page_log2);
  if (p.cu == nullptr) {
    s.row0 = b * p.n;
    s.n = p.n;
  } else {
    s.row0 = min(max(p.cu[b], 0), p.total_rows);
    s.n = min(max(p.cu[b + 1], s.row0), p.total_rows) - s.row0;
  }
  s.rows = p.group * min(s.n, p.n);
  return s;
}

// What a turn of a sequence costs.
SA_DEV int turn_cost(const Seq& q) { return kTurnCost + kTileCost * ((q.rows + 7) / 8); }

// The turns of a sequence that its last n positions can see: [0, pre) and [lo, end).
struct Span {
  int pre, lo, end;
  // at least 1: an empty sequence's rows are written too
  SA_DEV int count() const { return max(pre + end - lo, 1); }
  SA_DEV int turn(int i) const { return i < pre ? i : i - pre + lo; }
};

SA_DEV Span visible_span(const PageDecK& p, const Seq& q) {
  Span s;
  s.end = q.n > 0 ? q.len / kTurn + (q.len % kTurn != 0) : 0;
  const int first = max(q.len - q.n, 0);  // the earliest of the positions
  s.lo = min(p.window < 0 ? 0 : max(first - p.window, 0) / kTurn, s.end);
  const int pre = min(p.prefix, q.len);
  s.pre = min(pre / kTurn + (pre % kTurn != 0), s.lo);
  return s;
}

// The part of a pair that a worker takes: turns [t0, t1) of `turns`.
struct Segment {
  long long x;  // where its pair begins in the line that is shared out
  int b, head, row_group, t0, t1, turns, cost;
  Seq seq;
  Span span;
};

// A turn as a warp sees it.
struct Turn {
  int key0;      // position of its first key
  int loaded;    // halves of it that are in the ring, a bit each
  int missing;   // halves with tokens whose page is not in the pool
  bool masked;   // some (row, key) is not visible, or a half is not in the ring
};

// A warp's way through its turns of a segment (part, part + parts, ...): page
// numbers are loaded a batch of 32 turns ahead; the boxes come through the
// ring, kStages turns in flight.  Of the kShare warps that use one ring the
// first starts the copies, once all have read what a stage held.
template <int kShare, int kStages>
class Stream {
 public:
  SA_DEV Stream(const PageDecK& p, uint32_t ring, uint32_t bars, const tc::Abort& abort, int part, int parts, bool leads)
      : p_(p), ring_(ring), bars_(bars), abort_(abort), part_(part), parts_(parts), leads_(leads) {}

  // Starts a segment's first copies; none of an earlier one is in flight.
  SA_DEV void begin(const Segment& s) {
    seg_ = s;
    const int all = s.t1 - s.t0;
    turns_ = s.seq.n > 0 && s.seq.len > 0 && all > part_ && !dead_ ? (all - part_ + parts_ - 1) / parts_ : 0;
    if (turns_ == 0) return;
    load_places(0);
    cur0_ = to_row(next0_, 0, 0);
    cur1_ = to_row(next1_, 0, 1);
    if (turns_ > 32) load_places(32);
    __syncwarp();  // every lane is done with the ring
    const int now = min(turns_, kStages);
    for (int d = 0; d < now; ++d) fetch(d, used_ + d, cur0_, cur1_);
  }

  // Calls step(address of the turn's keys, turn) for every turn.
  template <class F>
  SA_DEV void run(F step) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = 0; i < turns_; ++i) {
      const int stage = used_ % kStages;
      if ((i & 31) == 16 && turns_ > i + 16) {  // the next batch's places are here by now
        next0_ = to_row(next0_, i + 16, 0);
        next1_ = to_row(next1_, i + 16, 1);
      }
      if (!tc::mbar_wait_warp(full(stage), used_ / kStages & 1, abort_)) {
        // Out of time, which the status word says: nothing more is started,
        // and what is in flight has as long again to land.
        dead_ = true;
        const long long t0 = clock64();
        for (int use = used_, last = used_ + min(kStages, turns_ - i); use < last;)
          if (tc::mbar_try_wait(full(use % kStages), use / kStages & 1) || clock64() - t0 > tc::kTimeoutCycles) ++use;
        break;
      }
      Turn t;
      const int r0 = __shfl_sync(0xffffffffu, cur0_, i & 31), r1 = __shfl_sync(0xffffffffu, cur1_, i & 31);
      t.key0 = seg_.span.turn(place(i)) * kTurn;
      t.loaded = (r0 >= 0) | (r1 >= 0) << 1;
      t.missing = ~t.loaded & (t.key0 + 16 < seg_.seq.len ? 3 : 1);
      const int key1 = t.key0 + kTurn - 1;
      // seen by all rows: the earliest position causally, the last one's window
      t.masked = t.loaded != 3 || key1 > seg_.seq.len - seg_.seq.n ||
                 !(p_.window < 0 || t.key0 >= seg_.seq.len - 1 - p_.window || key1 < p_.prefix);
      step(ring_ + stage * kTurnBytes, t);
      __syncwarp();  // every lane is done with the stage
      if (kShare > 1 && lane == 0) tc::mbar_arrive(empty(stage));
      if (i + kStages < turns_) {
        const bool same = (i & 31) + kStages < 32;
        fetch((i + kStages) & 31, used_ + kStages, same ? cur0_ : next0_, same ? cur1_ : next1_);
      }
      ++used_;
      if ((i & 31) == 31) {
        cur0_ = next0_;
        cur1_ = next1_;
        if (turns_ > i + 33) load_places(i + 33);
      }
    }
  }

 private:
  SA_DEV uint32_t full(int stage) const { return bars_ + 8 * stage; }
  SA_DEV uint32_t empty(int stage) const { return bars_ + 8 * (kStages + stage); }
  SA_DEV int place(int i) const { return seg_.t0 + part_ + parts_ * i; }  // the i-th turn as a number in the pair
  // The pages of the lane's turn of the batch from the j0-th on: of its first token, and of its 17th.
  SA_DEV void load_places(int j0) {
    const int i = j0 + (threadIdx.x & 31);
    next0_ = next1_ = -1;
    if (i >= turns_) return;
    const int pos = seg_.span.turn(place(i)) * kTurn, col = pos >> p_.page_log2, col1 = (pos + 16) >> p_.page_log2;
    const int32_t* row = p_.block_table + static_cast<int64_t>(seg_.seq.slot) * p_.max_pages;
    next0_ = row[col];  // a visible turn's first token is below the length, and that is inside the table
    if (pos + 16 < seg_.seq.len) next1_ = col1 == col ? next0_ : row[col1];
  }
  // The pool's row of a half's first token, -1 where it has none.
  SA_DEV int to_row(int page, int j0, int half) const {
    const int i = j0 + (threadIdx.x & 31);
    if (i >= turns_ || page < 0 || page >= p_.num_pages) return -1;
    const int pos = seg_.span.turn(place(i)) * kTurn + 16 * half;
    return (page << p_.page_log2) + (pos & ((1 << p_.page_log2) - 1));
  }
  // Starts the copies of a turn of the batch, the ring's use-th.
  SA_DEV void fetch(int in_batch, int use, int rows0, int rows1) {
    const int r0 = __shfl_sync(0xffffffffu, rows0, in_batch), r1 = __shfl_sync(0xffffffffu, rows1, in_batch);
    if (kShare > 1) {
      if (!leads_) return;
      if (use >= kStages && !tc::mbar_wait_warp(empty(use % kStages), (use / kStages - 1) & 1, abort_)) {
        // the wait for this turn's bytes finds the abort word set
        return;
      }
    }
    if ((threadIdx.x & 31) != 0) return;
    const uint32_t bar = full(use % kStages), to = ring_ + use % kStages * kTurnBytes;
    const int c = seg_.head * kHeadDim;
    if (p_.page_log2 > 4) {  // one page, one box of 32 rows (what lies behind the length is read and masked)
      tc::mbar_expect_tx(bar, r0 >= 0 ? kTurnBytes : 0);
      if (r0 >= 0) {
        tc::tma_load_2d(to, &p_.tm_k, c, r0, bar);
        tc::tma_load_2d(to + kTurnHalf, &p_.tm_v, c, r0, bar);
      }
    } else {
      tc::mbar_expect_tx(bar, ((r0 >= 0) + (r1 >= 0)) * 2 * kBoxBytes);
      if (r0 >= 0) {
        tc::tma_load_2d(to, &p_.tm_k, c, r0, bar);
        tc::tma_load_2d(to + kTurnHalf, &p_.tm_v, c, r0, bar);
      }
      if (r1 >= 0) {
        tc::tma_load_2d(to + kBoxBytes, &p_.tm_k, c, r1, bar);
        tc::tma_load_2d(to + kTurnHalf + kBoxBytes, &p_.tm_v, c, r1, bar);
      }
    }
  }

  const PageDecK& p_;
  uint32_t ring_, bars_;
  tc::Abort abort_;
  int part_, parts_, used_ = 0, turns_ = 0;
  bool leads_, dead_ = false;
  int cur0_ = -1, cur1_ = -1, next0_ = -1, next1_ = -1;
  Segment seg_;
};

constexpr float kUnseen = -3.402823466e38f;

// What a warp keeps of its rows.  Rows 2 t and 2 t + 1 of its tile nt of 8 rows
// are lane (g, t)'s entry [nt], .x and .y (the same in all g) except the sums,
// which are over the lane's own keys until they are reduced.
template <int NT>
struct Rows {
  float o[NT][4][4];  // O^T: [i][e] dim 16 i + g, [i][2 + e] dim 16 i + g + 8
  float2 sum[NT];     // of P
  float2 sum_o[NT];   // of P rounded to bf16
  float2 ref[NT];     // reference score (before the coefficient), kUnseen while the row has seen no key
};

template <int NT>
SA_DEV void rows_clear(Rows<NT>& r) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) r.o[nt][i][e] = 0.f;
    r.sum[nt] = r.sum_o[nt] = make_float2(0.f, 0.f);
    r.ref[nt] = make_float2(kUnseen, kUnseen);
  }
}

// Bits below n set, n >= 0.
SA_DEV uint32_t low_bits(int n) {
  uint32_t d;
  asm("bmsk.clamp.b32 %0, 0, %1;\n" : "=r"(d) : "r"(n));
  return d;
}
// The keys of a turn that row position `at` sees (-1: none), as bits; of the
// prefix: low_bits(prefix - key0), all without a window.
SA_DEV uint32_t seen_bits(int at, int key0, int window, uint32_t of_prefix) {
  return low_bits(max(at - key0 + 1, 0)) & (~low_bits(max(at - window - key0, 0)) | of_prefix);
}
// 0 or a NaN added to acc for each half: a NaN where v is an infinity or a NaN.
SA_DEV uint32_t not_finite(uint32_t v, uint32_t acc) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;\n" : "=r"(d) : "r"(v), "r"(0u), "r"(acc));
  return d;
}

// Moves a row's reference: all that was summed relative to the old one.
template <int NT>
SA_DEV void move_reference(Rows<NT>& r, int nt, int e, float top, float coef, float slack) {
  float m = top;
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
  float& ref = e ? r.ref[nt].y : r.ref[nt].x;
  if (m > ref + slack || (ref == kUnseen && m > kUnseen)) {
    // a row that has seen nothing holds zeros (or a NaN, which stays)
    const float f = ref == kUnseen ? 0.f : ex2((ref - m) * coef);
    ref = m;
    (e ? r.sum[nt].y : r.sum[nt].x) *= f;
    (e ? r.sum_o[nt].y : r.sum_o[nt].x) *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.o[nt][i][e] *= f;
      r.o[nt][i][2 + e] *= f;
    }
  }
}

// One turn and tiles [kFirst, kFirst + HT) of the warp's: two blocks of 16
// keys, whose chains of products run side by side.  kMasked: some (row, key) of
// them is not visible, or a half is not there; pos(nt, e): the rows' positions.
template <int NT, int kFirst, int HT, bool kMasked, class Pos>
SA_DEV void turn_step(Rows<NT>& r, uint32_t keys, const uint32_t (&qf)[HT][4][2], int tiles, float coef, float slack,
                      const Pos& pos, const Turn& turn, int window, int prefix) {
  constexpr int U = kTurn / 16, kEnd = kFirst + HT;
  constexpr bool kSkip = NT > 1;  // tiles without rows are left out
  const int lane = threadIdx.x & 31, g = lane >> 2;
  // Rows of 128 bytes, 16-byte chunks XORed with the row's low three bits.
  const uint32_t row_k = (lane & 7) + (lane & 8), chunk_k = lane >> 4;
  const uint32_t row_v = (lane & 7) + (lane >> 4) * 8, chunk_v = lane >> 3 & 1;
  // scores before the coefficient: s[u][nt - kFirst][e] key g of block u, s[u][nt - kFirst][2 + e] key g + 8, row 2 t + e
  float s[U][HT][4];
  constexpr int kAhead = NT <= 2 ? 4 : 1;  // chunks of 16 dims that are loaded before their products
#pragma unroll
  for (int j0 = 0; j0 < 4; j0 += kAhead) {
    uint32_t ka[U][kAhead][4];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u)
        ldsm_x4(keys + (16 * u + row_k) * 128 + (((2 * (j0 + j) + chunk_k) ^ (lane & 7)) << 4), ka[u][j][0], ka[u][j][1],
                ka[u][j][2], ka[u][j][3]);
#pragma unroll
    for (int i = 0; i < kAhead * U; ++i) {
      const int j = j0 + i / U, u = i % U;
      const uint32_t(&a)[4] = ka[u][j - j0];
#pragma unroll
      for (int nt = kFirst; nt < kEnd; ++nt) {
        if (kSkip && nt >= tiles) continue;
        if (j == 0)
          mma_first(s[u][nt - kFirst], a, qf[nt - kFirst][j][0], qf[nt - kFirst][j][1]);
        else
          mma_add(s[u][nt - kFirst], a, qf[nt - kFirst][j][0], qf[nt - kFirst][j][1]);
      }
    }
  }
  const uint32_t of_prefix = window < 0 ? 0xffffffffu : low_bits(max(prefix - turn.key0, 0));
  bool move = false;
  float top[HT][2];
#pragma unroll
  for (int nt = kFirst; nt < kEnd; ++nt) {
    if (kSkip && nt >= tiles) continue;
    if (kMasked) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t bits = seen_bits(pos(nt, e), turn.key0, window, of_prefix) >> (g);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& x = s[u][nt - kFirst][2 * h + e];
            if (turn.missing != 0 && (turn.missing >> u & 1)) x = __int_as_float(0x7fffffff);  // it reads as NaN
            if (!(bits >> (16 * u + 8 * h) & 1u)) x = -INFINITY;
          }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[nt - kFirst][e] = fmaxf(s[0][nt - kFirst][e], s[0][nt - kFirst][2 + e]);
#pragma unroll
      for (int u = 1; u < U; ++u) top[nt - kFirst][e] = fmax3(top[nt - kFirst][e], s[u][nt - kFirst][e], s[u][nt - kFirst][2 + e]);
      const float ref = e ? r.ref[nt].y : r.ref[nt].x;
      move |= top[nt - kFirst][e] > ref + slack || (ref == kUnseen && top[nt - kFirst][e] > kUnseen);
    }
  }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = kFirst; nt < kEnd; ++nt) {
      if (kSkip && nt >= tiles) continue;
      move_reference(r, nt, 0, top[nt - kFirst][0], coef, slack);
      move_reference(r, nt, 1, top[nt - kFirst][1], coef, slack);
    }
  }
  uint32_t pf[U][HT][2];
#pragma unroll
  for (int nt = kFirst; nt < kEnd; ++nt) {
    if (kSkip && nt >= tiles) continue;
    const float2 minus = make_float2(-r.ref[nt].x, -r.ref[nt].y), c2 = make_float2(coef, coef);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // subtracted first: the largest of huge scores has to give exactly 2^-8
        const float2 d = fadd2(make_float2(s[u][nt - kFirst][2 * h], s[u][nt - kFirst][2 * h + 1]), minus);
        const float2 x = ffma2(d, c2, make_float2(-kSlack, -kSlack));
        const float2 p = make_float2(ex2(x.x), ex2(x.y));
        r.sum[nt] = fadd2(r.sum[nt], p);
        const uint32_t two = pack_bf16(p.x, p.y);
        r.sum_o[nt] = fadd2(r.sum_o[nt], make_float2(bf16_lo(two), bf16_hi(two)));
        pf[u][nt - kFirst][h] = transpose8(two);
      }
    }
  }
  // What a masked key holds must not reach a row that does not see it, and 0
  // times an infinity or a NaN would: they are taken out of the product, and
  // added to the rows that do see them.
  bool odd = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ldsm_x4_t(keys + kTurnHalf + (16 * u + row_v) * 128 + (((2 * i + chunk_v) ^ (lane & 7)) << 4), a[i][0], a[i][1],
                a[i][2], a[i][3]);
    if (kMasked) {
      if (!(turn.loaded >> u & 1)) {  // nothing to add
#pragma unroll
        for (int nt = kFirst; nt < kEnd; ++nt) {
          // its keys count 0, or NaN for the rows that would see them
          if (kSkip && nt >= tiles) continue;
          pf[u][nt - kFirst][0] = pf[u][nt - kFirst][1] = 0u;
        }
      }
      uint32_t nan = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) nan = not_finite(a[i][m], nan);
      if (__any_sync(0xffffffffu, (nan & 0x7fff7fffu) != 0u)) {
        odd = true;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) a[i][m] &= ~((ones_exponent(a[i][m]) >> 15 & 0x00010001u) * 0xffffu);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int nt = kFirst; nt < kEnd; ++nt) {
        if (kSkip && nt >= tiles) continue;
        mma_add(r.o[nt][i], a[i], pf[u][nt - kFirst][0], pf[u][nt - kFirst][1]);
      }
  }
  if (kMasked && odd) {
#pragma unroll 1
    for (int key = 0; key < 16 * U; ++key) {
      if (!(turn.loaded >> (key >> 4) & 1)) continue;  // its rows are NaN by their scores
      uint32_t sees = 0;
#pragma unroll
      for (int nt = kFirst; nt < kEnd; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sees |= (seen_bits(pos(nt, e), turn.key0, window, of_prefix) >> (key) & 1u) << (2 * nt + e);
      const uint32_t row = keys + kTurnHalf + key * 128;
#pragma unroll
      for (int d = 0; d < 8; ++d) {  // dims 8 d + g: [d / 2][2 (d % 2) + e]
        uint32_t two;
        asm volatile("ld.shared.u16 %0, [%1];\n" : "=r"(two) : "r"(row + ((d ^ (key & 7)) << 4) + 2 * g));
        const float v = (two & 0x7f80u) == 0x7f80u ? bf16_lo(two) : 0.f;
#pragma unroll
        for (int nt = kFirst; nt < kEnd; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) r.o[nt][d >> 1][2 * (d & 1) + e] += sees >> (2 * nt + e) & 1u ? v : 0.f;
      }
    }
  }
}

// A row's running softmax over some of its keys: kD of the accumulator's dims.
// ref is in log2 units, -inf where none of the keys was seen; a key at ref
// counts as 2^-kSlack in the sums and acc.
template <int kD>
struct Piece {
  float acc[kD], sum, sum_o, ref;
};

// A reference score in log2 units, -inf where the row has seen no key.
SA_DEV float log2_ref(float ref, float coef) { return ref == kUnseen ? -INFINITY : ref * coef; }

// What finishes a row from its sums: o is acc times first, then times last; and lse.
struct Finish {
  float first, last, lse;
};

SA_DEV Finish finish_of(float ref, float sum, float sum_o, float sink) {
  Finish f;
  f.lse = sum == 0.f ? -INFINITY : (ref + kSlack + lg2(sum)) * kLn2;
  // sigmoid(lse - sink) = a^2 / (1 + h^2) with h = e^(-|sink - lse| / 2) and a = h where the sink is the larger one,
  // else 1.  What a sink far above leaves, e^(lse - sink), need not be in fp32's range where the mean is large: one a
  // goes with the sum, the other comes last.
  const float x = sink - f.lse, h = __expf(-0.5f * fabsf(x)), a = x > 0.f ? h : 1.f;
  f.first = sum == 0.f ? 0.f : __fdividef(a, sum_o * (1.f + h * h));
  f.last = sum == 0.f ? 0.f : a;
  return f;
}

// Writes dims d0 .. d0 + kD - 1 of a finished row: o = sigmoid(lse - sink) * acc / sum_o, and lse.
template <int kD>
SA_DEV void finish_row(const PageDecK& p, const Seq& q, int head, int row, int d0, const Piece<kD>& f) {
  const int i = p.row_of_seq(row), h_q = head * p.group + row - i * p.group;
  const int64_t at = static_cast<int64_t>(q.row0) + i;
  const Finish w = finish_of(f.ref, f.sum, f.sum_o, __ldg(p.sink + h_q));
  uint32_t v[kD / 2];
#pragma unroll
  for (int e = 0; e < kD / 2; ++e)
    v[e] = pack_bf16(f.acc[2 * e] * w.first * w.last, f.acc[2 * e + 1] * w.first * w.last);
  __nv_bfloat16* o = p.o + (at * p.hq + h_q) * kHeadDim + d0;
  if constexpr (kD == 4) {
    *reinterpret_cast<uint2*>(o) = make_uint2(v[0], v[1]);
  } else {
    static_assert(kD % 8 == 0, "16-byte stores");
#pragma unroll
    for (int e = 0; e < kD / 8; ++e)
      reinterpret_cast<uint4*>(o)[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
  }
  if (d0 == 0) p.lse[static_cast<int64_t>(h_q) * p.total_rows + at] = w.lse;
}

// Writes the rows of a warp that had all keys of a pair, tiles first, first + step, ...: 8x8 transposes bring a row's
// dims together.
template <int NT>
SA_DEV void finish_tiles(const PageDecK& p, const Seq& q, int head, int rows, int first, int step, const Rows<NT>& r) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row0 = 8 * (nt * step + first);
    if (row0 >= rows) break;
    Finish w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = row0 + 2 * t + e, i = p.row_of_seq(row), h_q = head * p.group + row - i * p.group;
      w[e] = finish_of(log2_ref(e ? r.ref[nt].y : r.ref[nt].x, p.coef), e ? r.sum[nt].y : r.sum[nt].x, e ? r.sum_o[nt].y : r.sum_o[nt].x,
                       row < rows ? __ldg(p.sink + h_q) : 0.f);
      if (g == 0 && row < rows) p.lse[static_cast<int64_t>(h_q) * p.total_rows + q.row0 + i] = w[e].lse;
    }
    const int row = row0 + g, i = p.row_of_seq(row), h_q = head * p.group + row - i * p.group;
    uint32_t* o = reinterpret_cast<uint32_t*>(p.o + ((static_cast<int64_t>(q.row0) + i) * p.hq + h_q) * kHeadDim);
#pragma unroll
    for (int c = 0; c < 8; ++c) {  // dims 8 c + g of rows 2 t, 2 t + 1 -> dims 8 c + 2 t, + 1 of row g
      const float x = r.o[nt][c >> 1][2 * (c & 1)] * w[0].first * w[0].last;
      const float y = r.o[nt][c >> 1][2 * (c & 1) + 1] * w[1].first * w[1].last;
      const uint32_t two = transpose8(pack_bf16(x, y));
      if (row < rows) o[4 * c + t] = two;
    }
  }
}

// Partial results in the workspace: kRows x 64 accumulators, then (ref, sum, sum_o, 0) per row.
template <int kRows, int kD>
SA_DEV void put_piece(float* part, int row, int d0, const Piece<kD>& f) {
#pragma unroll
  for (int d = 0; d < kD; d += 4)
    __stcg(reinterpret_cast<float4*>(part + row * kHeadDim + d0 + d),
           make_float4(f.acc[d], f.acc[d + 1], f.acc[d + 2], f.acc[d + 3]));
  if (d0 == 0)
    __stcg(reinterpret_cast<float4*>(part + kRows * kHeadDim + kPartPad * row), make_float4(f.ref, f.sum, f.sum_o, 0.f));
}

// What a piece with reference `ref` and sum `sum` counts beside one with reference `top`: a piece that saw nothing
// holds zeros, or a NaN that must come through.
SA_DEV float weight_of(float ref, float sum, float top) {
  return ref == -INFINITY ? (sum == 0.f ? 0.f : 1.f) : ex2(ref - top);
}

// The pieces of workers c0 .. c1, in order.
template <int kRows, int kD, class F>
SA_DEV Piece<kD> merge_pieces(F part_of, int c0, int c1, int row, int d0) {
  Piece<kD> all;
  all.sum = all.sum_o = 0.f;
  all.ref = -INFINITY;
#pragma unroll
  for (int d = 0; d < kD; ++d) all.acc[d] = 0.f;
  constexpr int kAtOnce = kD >= 16 ? 2 : 32 / kD;  // pieces in flight: their number, not their size, is what a merge waits for
#pragma unroll 1
  for (int first = c0; first <= c1; first += kAtOnce) {
    float4 st[kAtOnce], v[kAtOnce][kD / 4];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float* from = part_of(min(first + i, c1));
      st[i] = __ldcg(reinterpret_cast<const float4*>(from + kRows * kHeadDim + kPartPad * row));
#pragma unroll
      for (int d = 0; d < kD / 4; ++d)
        v[i][d] = __ldcg(reinterpret_cast<const float4*>(from + row * kHeadDim + d0 + 4 * d));
    }
    float top = all.ref;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, st[i].x);
    const float old = all.ref == -INFINITY ? 1.f : ex2(all.ref - top);
    all.ref = top;
    all.sum *= old;
    all.sum_o *= old;
#pragma unroll
    for (int d = 0; d < kD; ++d) all.acc[d] *= old;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (first + i > c1) break;
      const float f = weight_of(st[i].x, st[i].y, top);
      all.sum += f * st[i].y;
      all.sum_o += f * st[i].z;
#pragma unroll
      for (int d = 0; d < kD / 4; ++d) {
        all.acc[4 * d] += f * v[i][d].x;
        all.acc[4 * d + 1] += f * v[i][d].y;
        all.acc[4 * d + 2] += f * v[i][d].z;
        all.acc[4 * d + 3] += f * v[i][d].w;
      }
    }
  }
  return all;
}

struct Cut {  // a pair that other workers have parts of
  long long p0;  // its place in its head's line
  int c0, c1, b, head;
};

constexpr int kUptoStep = 4;  // every fourth sequence's place in the line is kept

// How a CTA is made up.  NT: tiles of 8 rows a warp has (above four it takes a
// turn in two halves of them, and a half's queries from shared memory); kShare: warps that share a
// ring and split the tiles; kTeams: rings of a CTA.
template <int NT_, int kShare_, int kTeams_, int kStages_, int kPerSm_>
struct Shape {
  static constexpr int NT = NT_, kShare = kShare_, kTeams = kTeams_, kStages = kStages_, kPerSm = kPerSm_;
  static constexpr int HT = NT > 4 ? NT / 2 : NT;
  static constexpr int kWarps = kShare * kTeams, kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT * kShare;
  // Teams that merge by rows in shared memory; where there are twice as many, the others' results are added to
  // theirs before.
  static constexpr int kSlots = kTeams > 4 || kShare > 1 ? kTeams / 2 : kTeams;
  static constexpr int kPerRow = kThreads / kRows >= 16 ? 16 : kThreads / kRows >= 8 ? 8 : kThreads / kRows >= 4 ? 4 : 2;
  static constexpr int kDims = kHeadDim / kPerRow;  // dims per thread when a CTA merges
  static_assert(kThreads >= 2 * kRows, "a row's threads");
  static constexpr int kPartFloats = kRows * (kHeadDim + kPartPad);
  static constexpr size_t kRing = static_cast<size_t>(kTeams) * kStages * kTurnBytes;
  static constexpr size_t kMerge = static_cast<size_t>(kSlots) * kRows * (kRowPad * 4 + 16);
  static constexpr size_t kQueries = HT < NT ? kRows * kHeadDim * 2 : 0;
  static_assert(2 * kPerSm * kRows <= kPartRowsPerSm, "the workspace has no room for every CTA's cut pairs");
};

// The warp's query rows in registers: lane (g, t) has dims 16 j + 2 t, + 1 and
// + 8, + 9 of row g of each tile (tile nt is number nt * step + first of the pair's).
template <int NT>
SA_DEV void load_queries(const PageDecK& p, const Seq& q, int head, int rows, int first, int step,
                         uint32_t (&qf)[NT][4][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = 8 * (nt * step + first) + g;
#pragma unroll
    for (int j = 0; j < 4; ++j) qf[nt][j][0] = qf[nt][j][1] = 0u;
    if (row < rows) {
      const int i = p.row_of_seq(row), h = head * p.group + row - i * p.group;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + ((static_cast<int64_t>(q.row0) + i) * p.hq + h) * kHeadDim + 2 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qf[nt][j][0] = __ldg(src + 8 * j);
        qf[nt][j][1] = __ldg(src + 8 * j + 4);
      }
    }
  }
}

// The same from shared memory, where row 8 tile + i of the pair lies at 128 bytes a row, swizzled.
template <int HT>
SA_DEV void fetch_queries(uint32_t queries, int first, int step, uint32_t (&qf)[HT][4][2]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int nt = 0; nt < HT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const uint32_t row = 8 * (nt * step + first) + (lane & 7);
      ldsm_x4(queries + row * 128 + (((2 * j + (lane >> 3)) ^ (lane & 7)) << 4), qf[nt][j][0], qf[nt][j][1],
              qf[nt][j + 1][0], qf[nt][j + 1][1]);
    }
}

// kAlone: every warp takes whole pairs, by the host's word that all are short.
template <class S, bool kAlone>
__global__ void __launch_bounds__(S::kThreads, S::kPerSm) kv_decode_kernel(const __grid_constant__ PageDecK p) {
  constexpr int NT = S::NT, kShare = S::kShare, kTeams = S::kTeams, kStages = S::kStages;
  constexpr int kQueryBytes = S::kRows * kHeadDim * 2;
  constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kRows = S::kRows, kSlots = S::kSlots, kDims = S::kDims;
  constexpr bool kMayAlone = kAlone || (kShare == 1 && NT <= 2);
  static_assert(!kAlone || kShare == 1, "a warp alone shares its ring with no other");
  extern __shared__ uint8_t smem_raw[];
  // the rings (boxes are swizzled by their address: 1024-byte aligned), queries [rows][64], merge area
  // [slots][rows][kRowPad] and statistics [slots][rows][4], then the places of the sequences in the line
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* queries = smem + S::kRing;
  float* acc_sh = reinterpret_cast<float*>(queries + S::kQueries);
  float4* stat_sh = reinterpret_cast<float4*>(acc_sh + kSlots * kRows * kRowPad);
  long long* upto = reinterpret_cast<long long*>(stat_sh + kSlots * kRows);  // turns of the sequences before
  __shared__ long long warp_sum[kWarps];
  __shared__ __align__(8) uint64_t bars[kTeams * 2 * kStages];
  __shared__ Cut cuts[2];
  __shared__ Segment segments[2][kWarps];  // a warp's segment and its next one: registers are short while turns are taken
  __shared__ int last_sh[2], abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int team = warp / kShare, share = warp % kShare;
  const int heads = p.num_heads_kv;

  if (tid == 0) {
    for (int i = 0; i < kTeams; ++i)
      for (int s = 0; s < kStages; ++s) {
        tc::mbar_init(smem_u32(&bars[i * 2 * kStages + s]), 1);
        tc::mbar_init(smem_u32(&bars[i * 2 * kStages + kStages + s]), kShare);
      }
    tc::fence_mbar_init();
    abort_flag = 0;
    tc::tma_prefetch_map(&p.tm_k);
    tc::tma_prefetch_map(&p.tm_v);
  }
  // what the sequences' turns cost, and its running total
  long long cost_all = 0;
  bool alone = kAlone;
  if (!kAlone) {
    int longest = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
      const int b = base + tid;
      long long x = 0;
      if (b < p.num_seqs) {
        const Seq q = sequence(p, b);
        const int count = visible_span(p, q).count();
        longest = max(longest, count);
        x = static_cast<long long>(count) * turn_cost(q);
      }
      const long long mine = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      long long before = cost_all;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        cost_all += warp_sum[w];
      }
      if (b < p.num_seqs && b % kUptoStep == 0) upto[b / kUptoStep] = before + x - mine;
      __syncthreads();
    }
    // many pairs, all of them short
    const bool few = __syncthreads_and(longest <= kAloneTurns) != 0;
    alone = kMayAlone && few && static_cast<long long>(p.num_seqs) * heads >= gridDim.x;
  } else {
    __syncthreads();
  }

  const float slack = __fdividef(kSlack, p.coef);
  Stream<kShare, kStages> stream(p, smem_u32(smem) + team * kStages * kTurnBytes, smem_u32(&bars[team * 2 * kStages]),
                                 tc::Abort{&abort_flag, p.status}, alone ? 0 : team, alone ? 1 : kTeams, share == 0);
  Rows<NT> r;
  // All turns of a segment that are the warp's, summed up in r.
  const auto process = [&](const Segment& seg) {
    const int rows = seg.seq.rows;
    // tiles nt step + first of the pair's are the warp's
    const int first_tile = kAlone ? seg.row_group : share, step_tile = kAlone ? p.row_groups : kShare;
    const int tiles = min(max(((rows + 7) / 8 - first_tile + step_tile - 1) / step_tile, 0), NT);
    uint32_t qf[S::HT][4][2];
    if (S::HT == NT) load_queries<S::HT>(p, seg.seq, seg.head, rows, first_tile, step_tile, qf);
    const int first = seg.seq.len - seg.seq.n;
    const auto pos = [&](int nt, int e) {
      const int row = 8 * (nt * step_tile + first_tile) + 2 * t + e;
      return row < rows ? first + p.row_of_seq(row) : -1;
    };
    rows_clear(r);
    stream.run([&](uint32_t keys, const Turn& turn) {
      if (tiles == 0) return;
      const auto step = [&](auto first) {
        constexpr int kFirst = decltype(first)::value;
        if (S::HT < NT)
          fetch_queries<S::HT>(smem_u32(queries) + (kAlone ? warp * kQueryBytes : 0), kFirst * kShare + share, kShare, qf);
        if (turn.masked)
          turn_step<NT, kFirst, S::HT, true>(r, keys, qf, tiles, p.coef, slack, pos, turn, p.window, p.prefix);
        else
          turn_step<NT, kFirst, S::HT, false>(r, keys, qf, tiles, p.coef, slack, pos, turn, p.window, p.prefix);
      };
      step(std::integral_constant<int, 0>());
      if constexpr (S::HT < NT) {
        if (tiles > S::HT) step(std::integral_constant<int, S::HT>());
      }
    });
    // sums over the keys
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        r.sum[nt].x += __shfl_xor_sync(0xffffffffu, r.sum[nt].x, o);
        r.sum[nt].y += __shfl_xor_sync(0xffffffffu, r.sum[nt].y, o);
        r.sum_o[nt].x += __shfl_xor_sync(0xffffffffu, r.sum_o[nt].x, o);
        r.sum_o[nt].y += __shfl_xor_sync(0xffffffffu, r.sum_o[nt].y, o);
      }
  };
  // Alone, a warp takes pairs gridDim.x * kWarps apart, and meets no other warp
  // from here on.  Else every head's turns make one line, in which the turns of
  // each sequence stand behind `pad` places for what beginning a pair costs a
  // CTA.  All heads' lines are cut alike, into equal shares, and neighbouring
  // CTAs take the same share of neighbouring heads, which lie side by side in
  // memory.  (More heads than CTAs: a line is not cut, and a CTA takes several.)
  const int ctas = static_cast<int>(gridDim.x), heads_at_once = min(heads, ctas);
  const int group = static_cast<int>(blockIdx.x) / heads_at_once;
  int b_first = 0, head_first = static_cast<int>(blockIdx.x) - group * heads_at_once, pad = 0;
  long long x_first = 0, x_begin = 0, x_end = 0;  // places in the line: of the first pair, and of the share
  int pair = warp * ctas + static_cast<int>(blockIdx.x);  // of 4096 entries with 256 heads and 3 groups of rows at most
  const int per_seq = heads * (kAlone ? p.row_groups : 1);
  Shares shares(1, 1);
  if (alone) {
    if (pair >= p.num_seqs * per_seq) return;
    b_first = pair / per_seq;
    head_first = pair - b_first * per_seq;
  } else if constexpr (!kAlone) {
    // a turn at least for every team, unless that leaves pairs without a worker of their own; no less than the most
    // that a turn costs, so that every share between a cut pair's first and last has a turn of it
    constexpr int kMostCost = kTurnCost + kTileCost * NT * kShare;
    const long long want = max(cost_all / (kTeams * (kTurnCost + kTileCost)), static_cast<long long>(p.num_seqs));
    const int n_workers = heads > ctas ? 1 : static_cast<int>(max(min(min(static_cast<long long>(ctas / heads_at_once), want),
                                                                      cost_all / kMostCost), 1LL));
    pad = cost_all >= 4LL * kPairCost * n_workers ? kPairCost : 0;
    shares = Shares(cost_all + static_cast<long long>(p.num_seqs) * pad, n_workers);
    if (group >= n_workers) return;
    x_begin = shares.start(group);
    x_end = shares.start(group + 1);
    int lo = 0, hi = (p.num_seqs - 1) / kUptoStep;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (upto[mid] + static_cast<long long>(mid) * kUptoStep * pad <= x_begin)
        lo = mid;
      else
        hi = mid - 1;
    }
    // the first pair that the share holds a turn of
    b_first = lo * kUptoStep;
    x_first = upto[lo] + static_cast<long long>(b_first) * pad;
#pragma unroll 1
    while (true) {
      const Seq q = sequence(p, b_first);
      const int count = visible_span(p, q).count(), cost = turn_cost(q);
      if (x_first + pad + static_cast<long long>(count - 1) * cost >= x_begin) break;
      x_first += pad + static_cast<long long>(count) * cost;
      ++b_first;
      if (b_first >= p.num_seqs || x_first + pad >= x_end) return;  // it lies in one turn, or in what beginning a pair costs
    }
  }
  // The worker's part of a pair that begins at x of the line (alone: of head / row_groups, and that group of rows).
  const auto segment_at = [&](int b, int head, long long x) {
    Segment s;
    s.x = x;
    s.b = b;
    s.head = kAlone ? head / p.row_groups : head;
    s.row_group = kAlone ? head - s.head * p.row_groups : 0;
    s.seq = sequence(p, b);
    s.span = visible_span(p, s.seq);
    s.turns = s.t1 = s.span.count();
    s.t0 = 0;
    s.cost = turn_cost(s.seq);
    if (!alone) {  // turn t is the share's that holds place x + pad + t cost
      s.t0 = static_cast<int>((max(x_begin - x - pad, 0LL) + s.cost - 1) / s.cost);
      s.t1 = static_cast<int>(min(static_cast<long long>(s.turns), (x_end - x - pad + s.cost - 1) / s.cost));
    }
    return s;
  };

  const int merge_row = min(tid / S::kPerRow, kRows), merge_dim = tid % S::kPerRow * kDims;  // kRows: none
  int n_cuts = 0, cur = 0;
  // Lane 0's word for the warp's next segment.
  const auto set_next = [&](const Segment& s) {
    if (lane == 0) segments[cur ^ 1][warp] = s;
    __syncwarp();
  };
  set_next(segment_at(b_first, head_first, x_first));
  bool first = true, more = true;
  while (true) {
    if (more) stream.begin(segments[cur ^ 1][warp]);  // on its way while the one before is finished
    const Segment& done = segments[cur][warp];
    if (!first) {
      const int rows = done.seq.rows;
      if (kMayAlone && alone) {
        finish_tiles<NT>(p, done.seq, done.head, rows, kAlone ? done.row_group : 0, kAlone ? p.row_groups : 1, r);
      } else if constexpr (!kAlone) {
        // A pair that is cut is published when the worker is through, with one
        // fence and no copies in flight for it to wait for.
        const bool whole = done.t0 == 0 && done.t1 == done.turns;
        float* mine = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (done.x > x_begin ? 1 : 0)) * S::kPartFloats;
        if (!whole) {
          if (tid == 0) {
            Cut c;
            c.p0 = done.x;
            c.c0 = shares.owner(done.x + pad);
            c.c1 = shares.owner(done.x + pad + static_cast<long long>(done.turns - 1) * done.cost);
            c.b = done.b;
            c.head = done.head;
            cuts[n_cuts] = c;
          }
          ++n_cuts;
        }
        if constexpr (kSlots < kTeams) {
          // the upper teams' results, lane for lane, to the lower ones
          float* slot = acc_sh + ((team % kSlots) * kShare + share) * (NT * 16 * 32) + 4 * lane;
          float4* stat = stat_sh + ((team % kSlots) * kShare + share) * (NT * 8);
          if (team >= kSlots) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(slot + (nt * 4 + i) * 128) =
                    make_float4(r.o[nt][i][0], r.o[nt][i][1], r.o[nt][i][2], r.o[nt][i][3]);
              if (g == 0) {
                stat[nt * 8 + 2 * t] = make_float4(r.ref[nt].x, r.sum[nt].x, r.sum_o[nt].x, 0.f);
                stat[nt * 8 + 2 * t + 1] = make_float4(r.ref[nt].y, r.sum[nt].y, r.sum_o[nt].y, 0.f);
              }
            }
          }
          __syncthreads();
          if (team < kSlots) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float own[2], other[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float4 st = stat[nt * 8 + 2 * t + e];
                float& ref = e ? r.ref[nt].y : r.ref[nt].x;
                float& sum = e ? r.sum[nt].y : r.sum[nt].x;
                float& sum_o = e ? r.sum_o[nt].y : r.sum_o[nt].x;
                const float top = fmaxf(ref, st.x), unit = log2_ref(top, p.coef);
                own[e] = weight_of(log2_ref(ref, p.coef), sum, unit);
                other[e] = weight_of(log2_ref(st.x, p.coef), st.y, unit);
                sum = own[e] * sum + other[e] * st.y;
                sum_o = own[e] * sum_o + other[e] * st.z;
                ref = top;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(slot + (nt * 4 + i) * 128);
                r.o[nt][i][0] = own[0] * r.o[nt][i][0] + other[0] * v.x;
                r.o[nt][i][1] = own[1] * r.o[nt][i][1] + other[1] * v.y;
                r.o[nt][i][2] = own[0] * r.o[nt][i][2] + other[0] * v.z;
                r.o[nt][i][3] = own[1] * r.o[nt][i][3] + other[1] * v.w;
              }
            }
          }
          __syncthreads();
        }
        if (team < kSlots) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = team * kRows + 8 * (nt * kShare + share) + 2 * t + e;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                acc_sh[at * kRowPad + 16 * i + g] = r.o[nt][i][e];
                acc_sh[at * kRowPad + 16 * i + g + 8] = r.o[nt][i][2 + e];
              }
              if (g == 0) {
                stat_sh[at] = make_float4(log2_ref(e ? r.ref[nt].y : r.ref[nt].x, p.coef),
                                          e ? r.sum[nt].y : r.sum[nt].x, e ? r.sum_o[nt].y : r.sum_o[nt].x, 0.f);
              }
            }
        }
        __syncthreads();
        // thread: one row, kDims of its dims
        Piece<kDims> f;
        f.sum = f.sum_o = 0.f;
        f.ref = -INFINITY;
#pragma unroll
        for (int d = 0; d < kDims; ++d) f.acc[d] = 0.f;
        const int row_sh = min(merge_row, kRows - 1);
#pragma unroll
        for (int w = 0; w < kSlots; ++w) f.ref = fmaxf(f.ref, stat_sh[w * kRows + row_sh].x);
#pragma unroll
        for (int w = 0; w < kSlots; ++w) {
          const float4 st = stat_sh[w * kRows + row_sh];
          const float m = weight_of(st.x, st.y, f.ref);
          f.sum += m * st.y;
          f.sum_o += m * st.z;
#pragma unroll
          for (int d = 0; d < kDims; d += 4) {
            const float4 v = *reinterpret_cast<const float4*>(acc_sh + (w * kRows + row_sh) * kRowPad + merge_dim + d);
            f.acc[d] += m * v.x;
            f.acc[d + 1] += m * v.y;
            f.acc[d + 2] += m * v.z;
            f.acc[d + 3] += m * v.w;
          }
        }
        if (merge_row < rows) {
          if (whole)
            finish_row<kDims>(p, done.seq, done.head, merge_row, merge_dim, f);
          else
            put_piece<kRows, kDims>(mine, merge_row, merge_dim, f);
        }
        if (more) __syncthreads();  // the merge area is free again, and the queries
      }
      if (!more) break;
    }
    cur ^= 1;
    first = false;
    if (S::HT < NT) {
      // the pair's queries into shared memory, zeros behind the last row (alone: the warp's tiles)
      const Segment& now = segments[cur][warp];
      uint8_t* to = queries + (kAlone ? warp * kQueryBytes : 0);
      for (int u = kAlone ? lane : tid; u < kRows * 8; u += kAlone ? 32 : kThreads) {
        const int at = u >> 3, c = u & 7;
        const int row = kAlone ? 8 * ((at >> 3) * p.row_groups + now.row_group) + (at & 7) : at;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < now.seq.rows) {
          const int i = p.row_of_seq(row), h = now.head * p.group + row - i * p.group;
          v = __ldg(reinterpret_cast<const uint4*>(p.q + ((static_cast<int64_t>(now.seq.row0) + i) * p.hq + h) * kHeadDim) + c);
        }
        *reinterpret_cast<uint4*>(to + swz(at, c)) = v;
      }
      if (kAlone)
        __syncwarp();
      else
        __syncthreads();
    }
    process(segments[cur][warp]);
    if (alone) {
      pair += ctas * kWarps;
      more = pair < p.num_seqs * per_seq;
      const int b = pair / per_seq;
      if (more) set_next(segment_at(b, pair - b * per_seq, 0));
    } else {
      const Segment& done = segments[cur][warp];
      const long long x = done.x + static_cast<long long>(done.turns) * done.cost + pad;
      const bool on = done.t1 == done.turns && done.b + 1 < p.num_seqs && x + pad < x_end;
      more = on || done.head + ctas < heads;  // more heads than CTAs
      if (more) set_next(segment_at(on ? done.b + 1 : b_first, on ? done.head : done.head + ctas, on ? x : x_first));
    }
  }

  if constexpr (!kAlone) {
    if (n_cuts == 0) return;
    const auto arrive = [&](const Cut& c) {  // by one thread, after a barrier: is this worker the pair's last?
      int* counter = p.counters + static_cast<int64_t>(c.b) * heads + c.head;
      __threadfence();  // the worker's piece, ordered before by the barrier, is there for whoever sees the count
      const bool last = atomicAdd(counter, 1) == c.c1 - c.c0;
      __threadfence();
      if (last) *counter = 0;
      return last;
    };
    // a worker's first pair left its piece in the first of its two places, a later one in the second
    const auto part_of = [&](const Cut& c) {
      return [&p, &shares, heads, p0 = c.p0, head = c.head](int w) {
        return p.part + (2 * (static_cast<int64_t>(w) * heads + head) + (p0 > shares.start(w) ? 1 : 0)) * S::kPartFloats;
      };
    };
    __syncthreads();
    if (tid < n_cuts) last_sh[tid] = arrive(cuts[tid]);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < n_cuts; ++i) {
      if (!last_sh[i]) continue;
      const Cut c = cuts[i];
      const Seq q = sequence(p, c.b);
      if (merge_row < q.rows)
        finish_row<kDims>(p, q, c.head, merge_row, merge_dim,
                          merge_pieces<kRows, kDims>(part_of(c), c.c0, c.c1, merge_row, merge_dim));
    }
  }
}

template <class S, bool kAlone>
cudaError_t launch_kernel(const PageDecK& p, cudaStream_t s) {
  constexpr size_t kFixed = 1024 + S::kRing + (kAlone ? S::kWarps * S::kQueries : S::kQueries + S::kMerge);
  static_assert(kFixed + kKv4MaxRequests / kUptoStep * sizeof(long long) <= 227 * 1024, "shared memory");
  const auto kernel = kv_decode_kernel<S, kAlone>;
  const auto bytes = [](int seqs) { return kFixed + (kAlone ? 0 : ceil_div(seqs, kUptoStep) * sizeof(long long)); };
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(kernel, bytes(kKv4MaxRequests));
  if (e != cudaSuccess) return e;
  kernel<<<device_sms() * S::kPerSm, S::kThreads, bytes(p.num_seqs), s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Partial results first, in a place that depends on the GPU alone, then the
// counters (zero between calls, one per pair): a workspace zeroed once serves
// every call with as many kv heads or fewer.
static size_t part_bytes() {
  return static_cast<size_t>(device_sms()) * kPartRowsPerSm * (kHeadDim + kPartPad) * 4;
}

size_t kv_decode_workspace_bytes(int hkv) { return part_bytes() + static_cast<size_t>(kKv4MaxRequests) * hkv * 4; }

cudaError_t launch_kv_decode(const KvPages& c, const KvDecodeArgs& a, int* status, cudaStream_t s) {
  PageDecK p;
  const long long places = static_cast<long long>(c.num_pages) << c.page_log2;
  const int box = std::min(c.page_size, kTurn);
  if (!make_rows_map(&p.tm_k, c.k, places, c.num_heads_kv, box) ||
      !make_rows_map(&p.tm_v, c.v, places, c.num_heads_kv, box))
    return cudaErrorInvalidValue;
  p.block_table = c.block_table;
  p.seqlens = c.seqlens;
  p.slots = a.slots;
  p.cu = a.cu;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.sink = a.sink;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.part = static_cast<float*>(a.workspace);
  p.counters = reinterpret_cast<int*>(static_cast<uint8_t*>(a.workspace) + part_bytes());
  p.status = status;
  p.num_pages = c.num_pages;
  p.page_log2 = c.page_log2;
  p.num_slots = c.num_slots;
  p.max_pages = c.max_pages;
  p.num_heads_kv = c.num_heads_kv;
  p.num_seqs = a.num_seqs;
  p.total_rows = a.rows;
  p.n = a.n;
  p.hq = a.hq;
  p.group = a.hq / c.num_heads_kv;
  p.window = a.window;
  p.prefix = a.prefix;
  // Not below the least normal number: such scores are nothing beside 1 either way, and 0 times a masked key's -inf
  // would be a NaN.
  p.coef = std::max(a.scale * kLog2e, 1.17549435e-38f);
  p.group_magic = static_cast<uint32_t>(ceil_div(1 << 16, p.group));
  const int rows = p.group * a.n;
  // what a sequence's rows can see at most, in turns
  const long long table = static_cast<long long>(c.max_pages) << c.page_log2;
  const long long most = a.window < 0 ? ceil_div(table, kTurn)
                                      : ceil_div(std::min<long long>(a.prefix, table), kTurn) +
                                            ceil_div(static_cast<long long>(a.window) + a.n, kTurn) + 1;
  const bool alone = most <= kAloneTurns && static_cast<long long>(a.num_seqs) * c.num_heads_kv >= device_sms();
  // One tile of rows: two turns in flight for each of 8 warps an SM (32 x 8192 keys 88.5 us; three turns 92.3, two for
  // 12 warps 91.1, four for 4 warps 92.5).  Up to 48 rows a warp has them all, in halves above 32 (8 x 32768 keys x 1 to
  // 5 rows 121 us; thirds 126, three tiles by each of two warps 180, two turns ahead for 6 warps 154).  Alone: 12 warps an
  // SM (200 windowed sequences 17.9 us; 8 warps 25.4), 8 above 16 rows (with 4 rows each 39.8 us, by shares 64.9), and
  // above 48 rows groups of them go to a warp each (with 8 rows, 40 a kv head, 84.9 us, by shares 150).
  p.row_groups = 1;
  if (alone) {
    if (rows <= 8) return launch_kernel<Shape<1, 1, 4, 2, 3>, true>(p, s);
    if (rows <= 16) return launch_kernel<Shape<2, 1, 4, 2, 3>, true>(p, s);
    if (rows <= 32) return launch_kernel<Shape<4, 1, 4, 2, 2>, true>(p, s);
    p.row_groups = ceil_div(rows, 48);
    return launch_kernel<Shape<6, 1, 8, 2, 1>, true>(p, s);
  }
  if (rows <= 8) return launch_kernel<Shape<1, 1, 4, 2, 2>, false>(p, s);
  if (rows <= 16) return launch_kernel<Shape<2, 1, 4, 2, 2>, false>(p, s);
  if (rows <= 32) return launch_kernel<Shape<4, 1, 4, 2, 2>, false>(p, s);
  if (rows <= 48) return launch_kernel<Shape<6, 1, 8, 2, 1>, false>(p, s);
  if (rows <= 64) return launch_kernel<Shape<4, 2, 4, 3, 1>, false>(p, s);
  return launch_kernel<Shape<4, 4, 2, 6, 1>, false>(p, s);
}

}  // namespace sa

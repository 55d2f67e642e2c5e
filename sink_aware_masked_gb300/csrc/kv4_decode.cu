// Decode forward over the 4-bit paged cache: the last n query positions of
// each sequence against its whole history, with the mask, sink and lse of the
// bf16 decode forward.
//
//   s = scale <q, K_k>,  l = log sum_{visible} e^s,  o = sigmoid(l - sink) softmax(s) V
//
// The cache is 72 bytes per token and kv head, so the step is a stream over
// it; per byte it needs the conversion of two codes and, with 8 query heads
// on a kv head, 28 multiply-adds.  A warp takes a block of 16 tokens with two
// 16-byte loads a lane and multiplies it without any reordering, because the
// cache keeps the codes in fragment order:
//   S^T [16 keys x 8 rows] = K [16 x 64] Q^T,   O^T [64 dims x 8 rows] += V^T [64 x 16] P^T
// Keys and dims are the 16-wide side, so 8 query rows fill the matrix
// instruction's 8-wide side and none of it is padding.  code * scale has at
// most 6 significant bits and is exact in f16; q is brought into f16's range
// by a power of two per row (its 8 bits fit); P is rounded to f16; S, O and the
// statistics are fp32.
//
// The softmax keeps a reference score m per row that need not be the
// maximum: it moves (and O and l are rescaled) only when a score exceeds it by
// more than 8 log2 units, which leaves one compare and one vote per two blocks
// in the ordinary case.  A key at the reference has P = 2^7, so P stays below
// 2^15, inside f16's range, and has most of that range below it: P is off by
// 2^-11 of itself, or, where it is weaker than 2^-21 of the largest and f16
// is subnormal, by 2^-32 of the largest (one strong key over a million weak
// ones leaves these their share in O as in l).
//
// Work: the visible blocks of all (sequence, kv head, row group) pairs in one
// line, cut into equal shares, one per worker.  A worker is a CTA, whose warps
// take a pair's blocks in turn and merge in shared memory; or, where there are
// many pairs with few blocks each, a single warp, which takes whole pairs and
// merges nothing.  A pair cut between CTAs leaves partial results in the
// workspace, and the last CTA of the pair to arrive merges them in order.
//
// Measured (GB300): 32 x 8192 keys, 64/8 heads, 42.2 us (151 MB, 22.4 us at the
// copy rate): 53 of an SM's cycles per block, 147 instructions, of them 69
// conversions and scalings and 8 products; without conversions and products a
// block takes 41, the memory's rate.  It is bound by dependent instructions: 2.1
// of 4 a clock, most stalls the wait for a warp's own last one, 12 warps an SM.
// 8 x 32768 keys x 4 rows 84.4 us, 200 windowed sequences 10.6 us, one sequence
// of 37 keys 6.5 us.
#include "kv4.cuh"
#include "shares.cuh"
#include "tc.cuh"

#include <algorithm>

namespace sa {
namespace {

using namespace kv4;

constexpr int kRowPad = 68;       // floats per row in shared memory
constexpr float kSlack = 8.f;     // log2 units a score may exceed its row's reference
constexpr float kRefLog2 = 7.f;   // log2 of the probability that stands for the reference,
constexpr float kRefScale = 1.f / 128.f;  // 2^-kRefLog2
// CTAs that an SM holds of the variants with 8, 16 and 32 rows, and the partial
// rows that they can leave in the workspace: two cut pairs each.
constexpr int kPerSm8 = 3, kPerSm16 = 2, kPerSm32 = 1;
constexpr int kPartRowsPerSm = 2 * std::max({8 * kPerSm8, 16 * kPerSm16, 32 * kPerSm32});

// What beginning a pair costs a CTA, in blocks.  A CTA whose share holds the
// end of one pair and the begin of the next gets that many blocks less
// (32 x 8192 keys: 43.0 us without, 42.4 with 24, 42.0 with 40, 42.1 with 64).
constexpr int kPairCost = 40;

// Blocks of the longest pair up to which warps work alone, each on whole pairs
// (200 sequences of 10 visible blocks: 10.6 us, by CTAs and shares 40.9).
constexpr int kAloneBlocks = 48;

struct DecK {
  Kv4Cache c;
  const int32_t* slots;
  const __nv_bfloat16* q;
  const float* sink;
  __nv_bfloat16* o;
  float* lse;
  float* part;    // [2 * workers][rows][64 + 2]
  int* counters;  // [pairs]
  int* status;    // the library's status word (bounded waits)
  int num_seqs, n, hq, group, rows, row_groups, window, prefix;
  float scale;
};

SA_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
SA_DEV void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8x8 f16 transpose across the warp.
SA_DEV uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(v));
  return d;
}

SA_DEV uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

SA_DEV float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The blocks of a sequence that its last n positions can see: [0, pre) and [lo, end).
struct Span {
  int len, pre, lo, end;
  SA_DEV int count() const { return pre + end - lo; }
  SA_DEV int block(int i) const { return i < pre ? i : i - pre + lo; }
};

SA_DEV Span visible_span(const DecK& p, int len) {
  Span s;
  s.len = len;
  s.end = (len >> 4) + ((len & 15) != 0);
  const int first = max(len - p.n, 0);  // the earliest of the positions
  s.lo = p.window < 0 ? 0 : max(first - p.window, 0) >> 4;
  const int pre = min(p.prefix, len);
  s.pre = min((pre >> 4) + ((pre & 15) != 0), s.lo);
  return s;
}

struct Tile {  // one block's bytes as this lane needs them
  uint4 k, v;
  uint32_t ks, vs;
};

// A warp's ring in shared memory: a turn is four blocks.
constexpr int kTurnBlocks = 4;
constexpr int kTurnBytes = kTurnBlocks * kBlockBytes;
constexpr int kStages = 2;
constexpr int kBatchTurns = 32 / kTurnBlocks;

SA_DEV void read_tile(const uint8_t* stage, Tile& t) {
  const int lane = threadIdx.x & 31;
  t.k = *reinterpret_cast<const uint4*>(stage + 16 * lane);
  t.v = *reinterpret_cast<const uint4*>(stage + kVCodes + 16 * lane);
  t.ks = *reinterpret_cast<const uint16_t*>(stage + kKScales + 2 * lane);
  t.vs = *reinterpret_cast<const uint32_t*>(stage + kVScales + 4 * (4 * (lane >> 3) + (lane & 3)));
}

// What a warp keeps of its rows.  Row 8 nt + 2 t + e of the tile is lane t's
// entry [nt][e] (the same in all g) except the sum, which is over the lane's
// own keys until it is reduced.
template <int NT>
struct Rows {
  float o[NT][4][4];     // O^T: [dim pair 8 g + 2 i, + 1][row e]: c0 c1 dim 8g+2i, c2 c3 dim 8g+2i+1
  float sum[NT][2];
  float ref[NT][2];      // reference score (before the coefficient), 0 while the row has seen no key
  float limit[NT][2];    // score beyond which ref moves, -inf while the row has seen no key
};

template <int NT>
SA_DEV void rows_clear(Rows<NT>& r) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) r.o[nt][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      r.sum[nt][e] = 0.f;
      r.ref[nt][e] = 0.f;
      r.limit[nt][e] = -INFINITY;
    }
  }
}

template <int U>
struct MaskArgs {
  int key0[U];      // positions of the blocks' first keys; kVoid for a block that is not there
  bool missing[U];  // its page is not in the pool: it reads as NaN
  int window, prefix;
  SA_DEV bool sees(int at, int key) const {
    return key <= at && (window < 0 || key >= at - window || key < prefix);
  }
};
constexpr int kVoid = 0x7fffff00;  // beyond every position

// U blocks of 16 keys.  kMasked: some (row, key) of them is not visible, or a page is missing.
// pos[nt][e]: the rows' positions (-1 for rows that are not there).
template <int NT, int U, bool kMasked>
SA_DEV void block_step(Rows<NT>& r, const Tile (&tile)[U], const uint32_t (&qf)[NT][4][2], const float (&coef)[NT][2],
                       const int (&pos)[NT][2], const MaskArgs<U>& mk) {
  const int g = lane_g();
  // scores before their row's coefficient: s[u][nt][e] key g of block u, s[u][nt][2 + e] key g + 8, row e
  float s[U][NT][4];
  uint32_t x[U][4], y[U][4], z[U][4], w[U][4], sa[U], sb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t ks = tile[u].ks;
    if (kMasked && mk.missing[u]) ks = kNaNScale * 0x0101u;
    const uint32_t two = e4m3x2(ks);
    sa[u] = __byte_perm(two, 0, 0x1010);
    sb[u] = __byte_perm(two, 0, 0x3232);
    e2m1x8(tile[u].k.x, x[u]);
    e2m1x8(tile[u].k.z, z[u]);
    e2m1x8(tile[u].k.y, y[u]);
    e2m1x8(tile[u].k.w, w[u]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int u = 0; u < U; ++u) {  // the blocks' chains of products run side by side
      const uint32_t a0 = hmul2(x[u][j], sa[u]), a1 = hmul2(z[u][j], sb[u]);
      const uint32_t a2 = hmul2(y[u][j], sa[u]), a3 = hmul2(w[u][j], sb[u]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (j == 0)
          mma_f16_first(s[u][nt], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
        else
          mma_f16(s[u][nt], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
      }
    }
  bool move = false;
  float top[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kMasked) {
          if (!mk.sees(pos[nt][e], mk.key0[u] + g)) s[u][nt][e] = -INFINITY;
          if (!mk.sees(pos[nt][e], mk.key0[u] + g + 8)) s[u][nt][2 + e] = -INFINITY;
        }
      }
      top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
      for (int u = 1; u < U; ++u) top[nt][e] = fmaxf(top[nt][e], fmaxf(s[u][nt][e], s[u][nt][2 + e]));
      move |= top[nt][e] > r.limit[nt][e];
    }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = top[nt][e];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (m > r.limit[nt][e]) {
          // a row that has seen nothing holds zeros (or a NaN, which stays)
          const float f = r.limit[nt][e] == -INFINITY ? 0.f : ex2((r.ref[nt][e] - m) * coef[nt][e]);
          r.ref[nt][e] = m;
          r.limit[nt][e] = m + __fdividef(kSlack, coef[nt][e]);
          r.sum[nt][e] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            r.o[nt][i][e] *= f;
            r.o[nt][i][2 + e] *= f;
          }
        }
      }
  }
  uint32_t pf[U][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // subtracted first: the largest of huge scores has to give exactly 2^7
        s[u][nt][e] = ex2(fmaf(s[u][nt][e] - r.ref[nt][e], coef[nt][e], kRefLog2));
        s[u][nt][2 + e] = ex2(fmaf(s[u][nt][2 + e] - r.ref[nt][e], coef[nt][e], kRefLog2));
        r.sum[nt][e] += s[u][nt][e] + s[u][nt][2 + e];
      }
      pf[u][nt][0] = transpose8(pack_f16(s[u][nt][0], s[u][nt][1]));
      pf[u][nt][1] = transpose8(pack_f16(s[u][nt][2], s[u][nt][3]));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t vs = tile[u].vs;
    if (kMasked) {
      // What a masked key holds must not reach a row that does not see it, and
      // 0 * NaN would: NaN scales are taken out of the product, and the rows
      // that do see such a key get a NaN in the dims it stands for.
      if (mk.missing[u]) vs = kNaNScale * 0x01010101u;
      if (__any_sync(0xffffffffu, any_nan_scale(vs))) {
#pragma unroll 1
        for (int key = 0; key < 16; ++key) {
          const int i = (key & 1) + 2 * (key >> 3);
          const uint32_t byte = __shfl_sync(0xffffffffu, vs, 4 * g + ((key & 7) >> 1)) >> (8 * i) & 0x7fu;
          if (byte != kNaNScale) continue;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (mk.sees(pos[nt][e], mk.key0[u] + key)) {
#pragma unroll
                for (int d = 0; d < 4; ++d) r.o[nt][d][e] = r.o[nt][d][2 + e] = __int_as_float(0x7fffffff);
              }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((vs >> (8 * i) & 0x7fu) == kNaNScale) vs &= ~(0xffu << (8 * i));
      }
    }
    const uint32_t s01 = e4m3x2(vs), s23 = e4m3x2(vs >> 16);
    uint32_t e01, o01, e23, o23, a[4], b[4], c[4], d[4];
    pair_tokens(tile[u].v.x, tile[u].v.y, e01, o01);
    pair_tokens(tile[u].v.z, tile[u].v.w, e23, o23);
    e2m1x8(e01, a);
    e2m1x8(o01, b);
    e2m1x8(e23, c);
    e2m1x8(o23, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a0 = hmul2(a[i], s01), a1 = hmul2(b[i], s01), a2 = hmul2(c[i], s23), a3 = hmul2(d[i], s23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_f16(r.o[nt][i], a0, a1, a2, a3, pf[u][nt][0], pf[u][nt][1]);
    }
  }
}

// What a warp will do next: 32 of its blocks, one per lane.
struct Batch {
  const uint8_t* src;  // the lane's block
  int key0;            // position of its first key
  // bit per block, the same in all lanes; missing: its page is not in the pool; next: it follows the one before it
  // in memory
  uint32_t valid, masked, missing, next;
};

// The part of a pair that a worker takes: blocks [blk0, blk1) of `blocks`.
struct Segment {
  long long x;  // where its pair begins in the line that is shared out
  int b, in_seq, blk0, blk1, blocks, slot, head, row0;
  Span span;
};

// A warp's way through its blocks of a segment (turns part, part + parts, ...,
// each the part of four aligned blocks that the segment has): page numbers are
// loaded two batches ahead; the blocks come through the ring by bulk copies,
// two turns in flight.
class Stream {
 public:
  SA_DEV Stream(const DecK& p, const uint8_t* ring, uint32_t bars, const tc::Abort& abort, int part, int parts)
      : p_(p), ring_(ring), bars_(bars), abort_(abort), part_(part), parts_(parts) {}

  // Starts a segment's first copies; none of an earlier one is in flight.
  SA_DEV void begin(const Segment& s) {
    seg_ = s;
    const int all = (s.blk1 - 1) / kTurnBlocks - s.blk0 / kTurnBlocks + 1;
    turns_ = s.span.len > 0 && all > part_ && !dead_ ? (all - part_ + parts_ - 1) / parts_ : 0;
    if (turns_ == 0) return;
    const int page0 = load_page(0);
    page_ = turns_ > kBatchTurns ? load_page(32) : -1;
    cur_ = to_batch(page0, 0);
    __syncwarp();  // every lane is done with the ring
    const int now = min(turns_, kStages);
#pragma unroll
    for (int d = 0; d < kStages; ++d)
      if (d < now) fetch(cur_, d, used_ + d);
  }

  // Calls step(the turn's bytes, its batch, its first bit) for every turn.
  template <class F>
  SA_DEV void run(F step) {
#pragma unroll 1
    for (int turn = 0; turn < turns_; ++turn) {
      const int in_batch = turn % kBatchTurns, stage = used_ % kStages;
      if (in_batch == kBatchTurns / 2 && turns_ > turn + kBatchTurns / 2)
        next_ = to_batch(page_, (turn + kBatchTurns / 2) * kTurnBlocks);
      if (!tc::mbar_wait_warp(bars_ + 8 * stage, used_ / kStages & 1, abort_)) {
        // Out of time, which the status word says: nothing more is started,
        // and what is in flight has as long again to land.
        dead_ = true;
        const long long t0 = clock64();
        for (int use = used_, last = used_ + min(kStages, turns_ - turn); use < last;)
          if (tc::mbar_try_wait(bars_ + 8 * (use % kStages), use / kStages & 1) ||
              clock64() - t0 > tc::kTimeoutCycles)
            ++use;
        break;
      }
      step(ring_ + stage * kTurnBytes, cur_, in_batch * kTurnBlocks);
      __syncwarp();  // every lane is done with the stage
      if (turn + kStages < turns_)
        fetch(in_batch + kStages < kBatchTurns ? cur_ : next_, (in_batch + kStages) % kBatchTurns, used_ + kStages);
      ++used_;
      if (in_batch == kBatchTurns - 1) {
        cur_ = next_;
        if (turns_ > turn + 1 + kBatchTurns) page_ = load_page((turn + 1 + kBatchTurns) * kTurnBlocks);
      }
    }
  }

 private:
  SA_DEV int place(int j0) const {  // the lane's block j0 + lane, as a number in the pair
    const int j = j0 + (threadIdx.x & 31);
    return (seg_.blk0 & ~(kTurnBlocks - 1)) + kTurnBlocks * part_ + parts_ * (j & ~(kTurnBlocks - 1)) +
           (j & (kTurnBlocks - 1));
  }
  SA_DEV int load_page(int j0) const {
    const int i = place(j0);
    return i >= seg_.blk0 && i < seg_.blk1 ? page_of(p_.c, seg_.slot, seg_.span.block(i)) : -1;
  }
  SA_DEV Batch to_batch(int page, int j0) const {
    Batch b;
    b.src = p_.c.pages;
    b.key0 = kVoid;
    bool masked = true;
    const int i = place(j0);
    const bool valid = i >= seg_.blk0 && i < seg_.blk1, missing = valid && page < 0;
    if (valid) {
      const int blk = seg_.span.block(i);
      if (!missing) b.src = block_ptr(p_.c, page, seg_.head, blk);
      b.key0 = blk * kBlockTokens;
      const int key1 = b.key0 + kBlockTokens - 1, len = seg_.span.len;
      // seen by all rows: the earliest position causally, the last one's window
      masked = missing || key1 > len - p_.n ||
               !(p_.window < 0 || b.key0 >= len - 1 - p_.window || key1 < p_.prefix);
    }
    b.valid = __ballot_sync(0xffffffffu, valid);
    b.masked = __ballot_sync(0xffffffffu, masked);
    b.missing = __ballot_sync(0xffffffffu, missing);
    const uint64_t at = reinterpret_cast<uint64_t>(b.src), before = __shfl_up_sync(0xffffffffu, at, 1);
    b.next = __ballot_sync(0xffffffffu, before + kBlockBytes == at);
    return b;
  }
  // Starts the copies of a batch's turn, the warp's use-th.
  SA_DEV void fetch(const Batch& b, int in_batch, int use) {
    const int lane = threadIdx.x & 31, stage = use % kStages;
    constexpr uint32_t kAll = (1u << kTurnBlocks) - 1;
    const int bit0 = in_batch * kTurnBlocks;
    const uint32_t there = (b.valid & ~b.missing) >> bit0 & kAll;
    const uint32_t bar = bars_ + 8 * stage, to = smem_u32(ring_) + stage * kTurnBytes;
    if (there == kAll && (b.next >> bit0 & kAll & ~1u) == (kAll & ~1u)) {  // the ordinary case: one run in one page
      if (lane == bit0) {
        tc::mbar_expect_tx(bar, kTurnBytes);
        tc::bulk_load(to, b.src, kTurnBytes, bar);
      }
      return;
    }
    if (lane == 0) tc::mbar_expect_tx(bar, __popc(there) * kBlockBytes);
    __syncwarp();
    const int mine = lane & (kTurnBlocks - 1);
    if (lane / kTurnBlocks == in_batch && (there >> mine & 1u))
      tc::bulk_load(to + mine * kBlockBytes, b.src, kBlockBytes, bar);
  }

  const DecK& p_;
  const uint8_t* ring_;
  uint32_t bars_;
  tc::Abort abort_;
  int part_, parts_, used_ = 0, turns_ = 0, page_ = -1;
  bool dead_ = false;
  Segment seg_;
  Batch cur_, next_;
};

// A row's running softmax over some of its keys: kD of the accumulator's
// dims.  ref is -inf where none of the keys was seen; a key at ref counts as
// 2^kRefLog2 in sum and acc.
template <int kD>
struct Piece {
  float acc[kD], sum, ref;
};

// Writes dims d0 .. d0 + kD - 1 of a finished row: o = factor * sigmoid(lse - sink) * acc / sum, and lse.
template <int kD>
SA_DEV void finish_row(const DecK& p, int b, int head, int row, int d0, const Piece<kD>& f, float sink, float factor) {
  const int i = row / p.group, h_q = head * p.group + row % p.group;
  const int64_t at = static_cast<int64_t>(b) * p.n + i;
  const float lse = f.sum == 0.f ? -INFINITY : (f.ref + lg2(f.sum * kRefScale)) * kLn2;
  // sigmoid(lse - sink) = a^2 / (1 + h^2) with h = e^(-|sink - lse| / 2) and a = h where the sink is the larger one,
  // else 1.  Neither what a sink far above leaves, e^(lse - sink), nor factor / sum need be in fp32's range: one a
  // goes with the sum, which brings the accumulators to the values' size, the other with the factor.
  const float x = sink - lse, h = __expf(-0.5f * fabsf(x)), a = x > 0.f ? h : 1.f;
  const float mean = __fdividef(a, f.sum * (1.f + h * h)), w = factor * a;
  __nv_bfloat16* o = p.o + (at * p.hq + h_q) * kHeadDim + d0;
  uint32_t v[kD / 2];
#pragma unroll
  for (int e = 0; e < kD / 2; ++e)
    v[e] = f.sum == 0.f ? 0u : pack_bf16(f.acc[2 * e] * mean * w, f.acc[2 * e + 1] * mean * w);
  static_assert(kD == 4 || kD == 8, "one store");
  if constexpr (kD == 4) *reinterpret_cast<uint2*>(o) = make_uint2(v[0], v[1]);
  if constexpr (kD == 8) *reinterpret_cast<uint4*>(o) = make_uint4(v[0], v[1], v[2], v[3]);
  if (d0 == 0) p.lse[static_cast<int64_t>(h_q) * p.num_seqs * p.n + at] = lse;
}

// Partial results in the workspace: kRows x 64 accumulators, then (ref, sum) per row.
template <int kRows, int kD>
SA_DEV void put_piece(float* part, int row, int d0, const Piece<kD>& f) {
#pragma unroll
  for (int d = 0; d < kD; d += 2)
    __stcg(reinterpret_cast<float2*>(part + row * kHeadDim + d0 + d), make_float2(f.acc[d], f.acc[d + 1]));
  if (d0 == 0) __stcg(reinterpret_cast<float2*>(part + kRows * kHeadDim + 2 * row), make_float2(f.ref, f.sum));
}

// The pieces of workers c0 .. c1, in order.
template <int kRows, int kD, class F>
SA_DEV Piece<kD> merge_pieces(F part_of, int c0, int c1, int row, int d0) {
  Piece<kD> all;
  all.sum = 0.f;
  all.ref = -INFINITY;
#pragma unroll
  for (int d = 0; d < kD; ++d) all.acc[d] = 0.f;
  constexpr int kAtOnce = 64 / kD;  // pieces in flight: their number, not their size, is what a merge waits for
#pragma unroll 1
  for (int first = c0; first <= c1; first += kAtOnce) {
    float2 st[kAtOnce], v[kAtOnce][kD / 2];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float* from = part_of(min(first + i, c1));
      st[i] = __ldcg(reinterpret_cast<const float2*>(from + kRows * kHeadDim + 2 * row));
#pragma unroll
      for (int d = 0; d < kD / 2; ++d)
        v[i][d] = __ldcg(reinterpret_cast<const float2*>(from + row * kHeadDim + d0 + 2 * d));
    }
    float top = all.ref;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, st[i].x);
    const float old = all.ref == -INFINITY ? 1.f : ex2(all.ref - top);
    all.ref = top;
    all.sum *= old;
#pragma unroll
    for (int d = 0; d < kD; ++d) all.acc[d] *= old;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      // a piece that saw nothing holds zeros, or a NaN that must come through
      float f = st[i].x == -INFINITY ? (st[i].y == 0.f ? 0.f : 1.f) : ex2(st[i].x - top);
      if (first + i > c1) f = 0.f, st[i].y = 0.f;
      all.sum += f * st[i].y;
#pragma unroll
      for (int d = 0; d < kD / 2; ++d) {
        if (first + i <= c1) {
          all.acc[2 * d] += f * v[i][d].x;
          all.acc[2 * d + 1] += f * v[i][d].y;
        }
      }
    }
  }
  return all;
}

struct SeqInfo {  // a sequence of the call, in shared memory
  long long upto;  // blocks of the sequences before it
  int len, slot;
};

struct Cut {  // a pair that other workers have parts of
  long long pair, p0;  // its number and its place in the line
  int c0, c1, b, head, row0;
};

template <int NT, int kWarps, int kPerSm>
__global__ void __launch_bounds__(kWarps * 32, kPerSm) kv4_decode_kernel(const DecK p) {
  constexpr int kThreads = kWarps * 32;
  constexpr int kRows = 8 * NT;
  constexpr int kAloneRows = NT <= 2 ? 2 * NT : 1;  // rows a lane finishes when its warp works alone
  constexpr int kPartFloats = kRows * (kHeadDim + 2);
  constexpr int kDims = kRows * kHeadDim / kThreads;  // dims per thread when a CTA merges: 4 or 8
  extern __shared__ __align__(16) uint8_t smem[];
  // the warps' rings, merge area [warps][rows][kRowPad], statistics [warps][rows][2], then the sequences
  float* acc_sh = reinterpret_cast<float*>(smem + kWarps * kStages * kTurnBytes);
  float* stat_sh = acc_sh + kWarps * kRows * kRowPad;
  SeqInfo* seqs = reinterpret_cast<SeqInfo*>(stat_sh + kWarps * kRows * 2);
  __shared__ long long warp_sum[kWarps];
  __shared__ __align__(8) uint64_t bars[kWarps * kStages];
  __shared__ Cut cuts[2];
  __shared__ int last_sh[2], abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane_g(), t = lane_t();

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) tc::mbar_init(smem_u32(&bars[warp * kStages + i]), 1);
    tc::fence_mbar_init();
    if (warp == 0) abort_flag = 0;
  }
  // blocks per sequence (an empty one counts as one: its rows are written too) and their running total
  long long blocks_all = 0;
  int longest = 0;
  for (int base = 0; base < p.num_seqs; base += kThreads) {
    const int b = base + tid;
    long long x = 0;
    SeqInfo info;
    if (b < p.num_seqs) {
      info.slot = p.slots[b];
      info.len = slot_len(p.c, info.slot);
      x = max(visible_span(p, info.len).count(), 1);
    }
    const long long own = x;
    longest = max(longest, static_cast<int>(min(x, 1LL << 30)));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long before = blocks_all;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      blocks_all += warp_sum[w];
    }
    if (b < p.num_seqs) {
      info.upto = before + x - own;
      seqs[b] = info;
    }
    __syncthreads();
  }

  const bool few = __syncthreads_and(longest <= kAloneBlocks) != 0;
  const int per_seq = p.c.num_heads_kv * p.row_groups;  // pairs per sequence
  const long long work = blocks_all * per_seq, pairs = static_cast<long long>(p.num_seqs) * per_seq;
  // many pairs, all of them short
  const bool alone = NT <= 2 && few && pairs >= gridDim.x;
  // a turn at least for every warp, unless that leaves pairs without a worker of their own
  const long long want = alone ? pairs : max((work + kTurnBlocks * kWarps - 1) / (kTurnBlocks * kWarps), pairs);
  const int most = static_cast<int>(gridDim.x) * (alone ? kWarps : 1);
  const int n_workers = static_cast<int>(min(static_cast<long long>(most), want));
  // The line that is shared out: all pairs, or all blocks, where the blocks of
  // each pair stand behind `pad` places for what beginning a pair costs a CTA.
  const int pad = !alone && work >= 4LL * kPairCost * n_workers ? kPairCost : 0;
  const Shares shares(alone ? pairs : work + pairs * pad, n_workers);
  const int worker = alone ? warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x) : blockIdx.x;
  if (worker >= shares.workers) return;  // a whole CTA, or a warp of one that never meets the others again
  const long long x_end = shares.start(worker + 1);

  // The worker's part of pair in_seq of sequence b, which begins at x of the line, from blk0 on.
  const auto segment_at = [&](long long x, int b, int in_seq, int blk0) {
    Segment s;
    const SeqInfo info = seqs[b];
    s.x = x;
    s.b = b;
    s.in_seq = in_seq;
    s.blk0 = blk0;
    s.slot = info.slot;
    s.span = visible_span(p, info.len);
    s.blocks = max(s.span.count(), 1);
    s.blk1 = alone ? s.blocks : static_cast<int>(min(static_cast<long long>(s.blocks), x_end - x - pad));
    s.head = p.row_groups == 1 ? in_seq : in_seq / p.row_groups;
    s.row0 = (in_seq - s.head * p.row_groups) * kRows;
    return s;
  };
  Segment seg;
  {  // the pair that holds the share's first place
    const long long x = shares.start(worker);
    int lo = 0, hi = p.num_seqs - 1;
    while (!alone && lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((seqs[mid].upto + static_cast<long long>(mid) * pad) * per_seq <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    if (alone) {
      lo = static_cast<int>(x / per_seq);
      seg = segment_at(x, lo, static_cast<int>(x - static_cast<long long>(lo) * per_seq), 0);
    } else {
      const long long off = x - (seqs[lo].upto + static_cast<long long>(lo) * pad) * per_seq;
      const long long places = max(visible_span(p, seqs[lo].len).count(), 1) + pad;
      int in_seq = min(static_cast<int>(__fdividef(static_cast<float>(off), static_cast<float>(places))), per_seq - 1);
      while (in_seq * places > off) --in_seq;
      while ((in_seq + 1) * places <= off) ++in_seq;
      const long long in_pair = off - in_seq * places;
      seg = segment_at(x - in_pair, lo, in_seq, static_cast<int>(max(in_pair - pad, 0LL)));
    }
  }

  // What a segment needs besides its blocks, loaded ahead: query rows (lane
  // (g, t): row g's dims 16 t .. 16 t + 15), factors, and the sinks of the
  // rows that this thread will finish.
  uint32_t qw[NT][8];
  float k_factor, v_factor, sink[kAloneRows];
  const int merge_row = tid / (kThreads / kRows), merge_dim = tid % (kThreads / kRows) * kDims;
  const auto load_ahead = [&](const Segment& s) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = s.row0 + 8 * nt + g;
#pragma unroll
      for (int i = 0; i < 8; ++i) qw[nt][i] = 0;
      if (row < p.rows) {
        const int64_t at = static_cast<int64_t>(s.b) * p.n + row / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (at * p.hq + s.head * p.group + row % p.group) * kHeadDim + 16 * t);
        const uint4 u = __ldg(src), v = __ldg(src + 1);
        qw[nt][0] = u.x, qw[nt][1] = u.y, qw[nt][2] = u.z, qw[nt][3] = u.w;
        qw[nt][4] = v.x, qw[nt][5] = v.y, qw[nt][6] = v.z, qw[nt][7] = v.w;
      }
    }
    k_factor = __ldg(p.c.k_scale + s.head);
    v_factor = __ldg(p.c.v_scale + s.head);
    const auto sink_of = [&](int row) { return row < p.rows ? __ldg(p.sink + s.head * p.group + row % p.group) : 0.f; };
    if (NT <= 2 && alone) {
#pragma unroll
      for (int i = 0; i < kAloneRows; ++i) sink[i] = sink_of(s.row0 + 8 * (i >> 1) + 2 * t + (i & 1));
    } else {
      sink[0] = sink_of(s.row0 + merge_row);
    }
  };

  Stream stream(p, smem + warp * kStages * kTurnBytes, smem_u32(&bars[warp * kStages]), tc::Abort{&abort_flag, p.status},
                alone ? 0 : warp, alone ? 1 : kWarps);
  int n_cuts = 0;
  load_ahead(seg);
  stream.begin(seg);
  while (true) {
    uint32_t qf[NT][4][2];
    float coef[NT][2];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t(&w)[8] = qw[nt];
      uint32_t top = 0;  // the row's largest exponent field
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, max(w[i] >> 7 & 0xffu, w[i] >> 23 & 0xffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // q * 2^(8 - e) has its largest entry in [2^8, 2^9); rows with an infinity or NaN stay as they are
      const int e = top == 255 ? 8 : min(max(static_cast<int>(top) - 127, -110), 126);
      const float up = __int_as_float((127 + 8 - e) << 23);
      const float down = __int_as_float((127 - 8 + e) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[nt][i][0] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
        qf[nt][i][1] = pack_f16(__uint_as_float(w[4 + i] << 16) * up, __uint_as_float(w[4 + i] & 0xffff0000u) * up);
      }
      // Not below the least normal number: such scores are nothing beside 1 either way, and 0 times a masked key's
      // -inf would be a NaN.
      const float mine = fmaxf(down * (p.scale * kLog2e) * k_factor, 1.17549435e-38f);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        coef[nt][r] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + r));
        const int rr = seg.row0 + 8 * nt + 2 * t + r;
        pos[nt][r] = rr < p.rows ? seg.span.len - p.n + rr / p.group : -1;
      }
    }
    const float v_scale = v_factor;
    float row_sink[kAloneRows];
#pragma unroll
    for (int i = 0; i < kAloneRows; ++i) row_sink[i] = sink[i];

    Rows<NT> r;
    rows_clear(r);
    stream.run([&](const uint8_t* at, const Batch& batch, int bit0) {
      constexpr int U = 2;  // blocks per step: two independent chains of products
      constexpr uint32_t kAny = (1u << U) - 1;
#pragma unroll 1
      for (int u0 = 0; u0 < kTurnBlocks; u0 += U) {
        const int bit = bit0 + u0;
        if ((batch.valid >> bit & kAny) == 0) continue;
        Tile tile[U];
#pragma unroll
        for (int u = 0; u < U; ++u) read_tile(at + (u0 + u) * kBlockBytes, tile[u]);
        MaskArgs<U> mk;
        mk.window = p.window;
        mk.prefix = p.prefix;
        if ((batch.masked >> bit & kAny) == 0) {
          block_step<NT, U, false>(r, tile, qf, coef, pos, mk);
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            mk.key0[u] = __shfl_sync(0xffffffffu, batch.key0, bit + u);
            mk.missing[u] = batch.missing >> (bit + u) & 1u;
          }
          block_step<NT, U, true>(r, tile, qf, coef, pos, mk);
        }
      }
    });

    // the next segment is on its way while this one is finished
    const Segment done = seg;
    const long long x_next = done.x + (alone ? 1 : done.blocks + pad);
    const bool more = done.blk1 == done.blocks && x_next + pad < x_end;
    if (more) {
      const bool same = done.in_seq + 1 < per_seq;
      seg = segment_at(x_next, same ? done.b : done.b + 1, same ? done.in_seq + 1 : 0, 0);
      load_ahead(seg);
      stream.begin(seg);
    }

    // A pair that is cut is published when the worker is through, with one
    // fence and no copies in flight for it to wait for.
    const bool whole = done.blk0 == 0 && done.blk1 == done.blocks;
    float* mine = p.part + (2 * static_cast<int64_t>(worker) + (done.x > shares.start(worker) ? 1 : 0)) * kPartFloats;
    if (!whole) {
      if (tid == 0) {
        Cut c;
        c.pair = static_cast<long long>(done.b) * per_seq + done.in_seq;
        c.p0 = done.x;
        c.c0 = shares.owner(done.x + pad);
        c.c1 = shares.owner(done.x + pad + done.blocks - 1);
        c.b = done.b;
        c.head = done.head;
        c.row0 = done.row0;
        cuts[n_cuts] = c;
      }
      ++n_cuts;
    }

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = r.sum[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        r.sum[nt][e] = sum + __shfl_xor_sync(0xffffffffu, sum, 16);
        r.ref[nt][e] = r.limit[nt][e] == -INFINITY ? -INFINITY : r.ref[nt][e] * coef[nt][e];  // log2 units from here
      }
    const auto piece_of = [&](int nt, int e) {
      Piece<8> f;
#pragma unroll
      for (int i = 0; i < 4; ++i) f.acc[2 * i] = r.o[nt][i][e], f.acc[2 * i + 1] = r.o[nt][i][2 + e];
      f.sum = r.sum[nt][e];
      f.ref = r.ref[nt][e];
      return f;
    };
    if (NT <= 2 && alone) {
      const auto each_row = [&](auto f) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (done.row0 + 8 * nt + 2 * t + e < p.rows) f(nt, e, 8 * nt + 2 * t + e);
      };
      each_row([&](int nt, int e, int row) {
        finish_row<8>(p, done.b, done.head, done.row0 + row, 8 * g, piece_of(nt, e), row_sink[(2 * nt + e) % kAloneRows],
                      v_scale);
      });
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Piece<8> f = piece_of(nt, e);
          const int at = warp * kRows + 8 * nt + 2 * t + e;
          float4* to = reinterpret_cast<float4*>(acc_sh + at * kRowPad + 8 * g);
          to[0] = make_float4(f.acc[0], f.acc[1], f.acc[2], f.acc[3]);
          to[1] = make_float4(f.acc[4], f.acc[5], f.acc[6], f.acc[7]);
          if (g == 0) *reinterpret_cast<float2*>(stat_sh + 2 * at) = make_float2(f.ref, f.sum);
        }
      __syncthreads();
      // thread: one row, kDims of its dims
      Piece<kDims> f;
      f.sum = 0.f;
      f.ref = -INFINITY;
#pragma unroll
      for (int d = 0; d < kDims; ++d) f.acc[d] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) f.ref = fmaxf(f.ref, stat_sh[(w * kRows + merge_row) * 2]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 st = *reinterpret_cast<const float2*>(stat_sh + (w * kRows + merge_row) * 2);
        const float m = st.x == -INFINITY ? (st.y == 0.f ? 0.f : 1.f) : ex2(st.x - f.ref);
        f.sum += m * st.y;
#pragma unroll
        for (int d = 0; d < kDims; ++d) f.acc[d] += m * acc_sh[(w * kRows + merge_row) * kRowPad + merge_dim + d];
      }
      const bool there = done.row0 + merge_row < p.rows;
      if (there) {
        if (whole)
          finish_row<kDims>(p, done.b, done.head, done.row0 + merge_row, merge_dim, f, row_sink[0], v_scale);
        else
          put_piece<kRows, kDims>(mine, merge_row, merge_dim, f);
      }
      if (more) __syncthreads();  // the merge area is free again
    }
    if (!more) break;
  }

  if (n_cuts == 0) return;
  const auto arrive = [&](const Cut& c) {  // by one thread, after a barrier: is this worker the pair's last?
    __threadfence();  // the worker's piece, ordered before by the barrier, is there for whoever sees the count
    const bool last = atomicAdd(p.counters + c.pair, 1) == c.c1 - c.c0;
    __threadfence();
    if (last) p.counters[c.pair] = 0;
    return last;
  };
  // a worker's first pair left its piece in the first of its two places, a later one in the second
  const auto part_of = [&](const Cut& c) {
    return [&p, &shares, p0 = c.p0](int w) {
      return p.part + (2 * static_cast<int64_t>(w) + (p0 > shares.start(w) ? 1 : 0)) * kPartFloats;
    };
  };
  const auto sink_at = [&](const Cut& c, int row) { return __ldg(p.sink + c.head * p.group + row % p.group); };
  __syncthreads();
  if (tid < n_cuts) last_sh[tid] = arrive(cuts[tid]);
  __syncthreads();
  for (int i = 0; i < n_cuts; ++i) {
    if (!last_sh[i]) continue;
    const Cut c = cuts[i];
    if (c.row0 + merge_row < p.rows)
      finish_row<kDims>(p, c.b, c.head, c.row0 + merge_row, merge_dim,
                        merge_pieces<kRows, kDims>(part_of(c), c.c0, c.c1, merge_row, merge_dim),
                        sink_at(c, c.row0 + merge_row), __ldg(p.c.v_scale + c.head));
  }
}

template <int NT, int kWarps, int kPerSm>
cudaError_t launch_variant(const DecK& p, cudaStream_t s) {
  constexpr size_t kFixed = static_cast<size_t>(kWarps) * (kStages * kTurnBytes + 8 * NT * (kRowPad + 2) * 4);
  const auto kernel = kv4_decode_kernel<NT, kWarps, kPerSm>;
  static_assert(2 * kPerSm * 8 * NT <= kPartRowsPerSm, "the workspace has no room for every CTA's cut pairs");
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(kernel, kFixed + kKv4MaxRequests * sizeof(SeqInfo));
  if (e != cudaSuccess) return e;
  kernel<<<device_sms() * kPerSm, kWarps * 32, kFixed + p.num_seqs * sizeof(SeqInfo), s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Partial results first, in a place that depends on the GPU alone, then the
// counters (zero between calls, at most one per query row and head): a
// workspace zeroed once serves calls of any shape it is large enough for.
static size_t part_bytes() {
  return (static_cast<size_t>(device_sms()) * kPartRowsPerSm * (kHeadDim + 2) * 4 + 255) / 256 * 256;
}

size_t kv4_decode_workspace_bytes(long long rows, int hq) { return part_bytes() + static_cast<size_t>(rows) * hq * 4; }

cudaError_t launch_kv4_decode(const Kv4Cache& c, const Kv4DecodeArgs& a, int* status, cudaStream_t s) {
  DecK p;
  p.status = status;
  p.c = c;
  p.slots = a.slots;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.sink = a.sink;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.part = static_cast<float*>(a.workspace);
  p.counters = reinterpret_cast<int*>(static_cast<uint8_t*>(a.workspace) + part_bytes());
  p.num_seqs = a.num_seqs;
  p.n = a.n;
  p.hq = a.hq;
  p.group = a.hq / c.num_heads_kv;
  p.rows = p.group * a.n;
  p.window = a.window;
  p.prefix = a.prefix;
  p.scale = a.scale;
  // Tiles of 8, 16 or 32 rows; wider ones come as row groups.  An SM holds 12
  // warps at 8 rows (42.0 us; 16 warps at 128 registers 45.4), 8 at 16 rows
  // (2 CTAs of 4: 57.2 us at 32 x 8192 x 2 rows, 1 of 8: 62.1) and 8 at 32
  // (1 CTA of 8: 85.5 us at 8 x 32768 x 4 rows, 2 of 4: 91.7).
  const int nt = p.rows <= 8 ? 1 : p.rows <= 16 ? 2 : 4;
  p.row_groups = ceil_div(p.rows, 8 * nt);
  if (nt == 1) return launch_variant<1, 4, kPerSm8>(p, s);
  if (nt == 2) return launch_variant<2, 4, kPerSm16>(p, s);
  return launch_variant<4, 8, kPerSm32>(p, s);
}

}  // namespace sa

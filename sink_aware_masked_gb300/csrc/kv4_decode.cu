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
// by a power of two per row (its 8 bits fit); P is rounded to f16 (2^-11);
// S, O and the statistics are fp32.
//
// The softmax keeps a reference exponent m per row that need not be the
// maximum: it moves (and O and l are rescaled) only when a score exceeds it
// by 2^8, which keeps P below f16's range and leaves one compare and one vote
// per block in the ordinary case.
//
// Work: the visible blocks of all (sequence, kv head, row group) pairs in one
// line, cut into equal shares, one per CTA; a share's blocks of one pair are
// taken by the CTA's warps in turn and merged in shared memory.  A pair cut
// between CTAs leaves partial results in the workspace, and the last CTA of
// the pair to arrive merges them in CTA order.
#include "kv4.cuh"

namespace sa {
namespace {

using namespace kv4;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRowPad = 68;       // floats per row in shared memory
constexpr float kSlack = 8.f;     // log2 units a score may exceed its row's reference
// Partial rows that the CTAs of one SM can leave: two pairs cut per CTA, and
// CTAs x rows per SM is 2 x 8, 1 x 16 or 1 x 32 by variant.
constexpr int kPartRowsPerSm = 64;

struct DecK {
  Kv4Cache c;
  const int32_t* slots;
  const __nv_bfloat16* q;
  const float* sink;
  __nv_bfloat16* o;
  float* lse;
  float* part;    // [2 * grid][rows][64 + 2]
  int* counters;  // [pairs]
  int num_seqs, n, hq, group, rows, row_groups, window, prefix;
  float scale;
};

SA_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

SA_DEV Span visible_span(const DecK& p, int b) {
  Span s;
  s.len = slot_len(p.c, p.slots[b]);
  s.end = (s.len >> 4) + ((s.len & 15) != 0);
  const int first = max(s.len - p.n, 0);  // the earliest of the positions
  s.lo = p.window < 0 ? 0 : max(first - p.window, 0) >> 4;
  const int pre = min(p.prefix, s.len);
  s.pre = min((pre >> 4) + ((pre & 15) != 0), s.lo);
  return s;
}

struct Tile {  // one block's bytes as this lane needs them
  uint4 k, v;
  uint32_t ks, vs;
};

SA_DEV void load_tile(const Kv4Cache& c, int page, int head, int blk, Tile& t) {
  const uint8_t* b = block_ptr(c, max(page, 0), head, blk);
  const int lane = threadIdx.x & 31;
  t.k = __ldg(reinterpret_cast<const uint4*>(b) + lane);
  t.v = __ldg(reinterpret_cast<const uint4*>(b + kVCodes) + lane);
  t.ks = __ldg(reinterpret_cast<const uint16_t*>(b + kKScales) + lane);
  t.vs = __ldg(reinterpret_cast<const uint32_t*>(b + kVScales) + 4 * (lane >> 3) + (lane & 3));
  if (page < 0) {  // a missing page reads as NaN
    t.ks = kNaNScale * 0x0101u;
    t.vs = kNaNScale * 0x01010101u;
  }
}

// What a warp keeps of its rows.  Row 8 nt + 2 t + e of the tile is lane t's
// entry [nt][e] (the same in all g) except the sum, which is over the lane's
// own keys until it is reduced.
template <int NT>
struct Rows {
  float o[NT][4][4];     // O^T: [dim pair 8 g + 2 i, + 1][row e]: c0 c1 dim 8g+2i, c2 c3 dim 8g+2i+1
  float sum[NT][2];
  float ref[NT][2];      // reference exponent, 0 while the row has seen no key
  float limit[NT][2];    // ref + kSlack, -inf while the row has seen no key
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

struct MaskArgs {
  int key0;  // position of the block's first key
  int window, prefix;
};

// One block of 16 keys.  kMasked: some (row, key) of it is not visible.
// pos[nt][e]: the rows' positions (-1 for rows that are not there).
template <int NT, bool kMasked>
SA_DEV void block_step(Rows<NT>& r, const Tile& tile, const uint32_t (&qf)[NT][4][2], const float (&coef)[NT][2],
                       const int (&pos)[NT][2], const MaskArgs& mk) {
  const int g = lane_g(), t = lane_t();
  float s[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
  {
    const uint32_t two = e4m3x2(tile.ks);
    const uint32_t sa = __byte_perm(two, 0, 0x1010), sb = __byte_perm(two, 0, 0x3232);
    uint32_t x[4], y[4], z[4], w[4];
    e2m1x8(tile.k.x, x);
    e2m1x8(tile.k.z, z);
    e2m1x8(tile.k.y, y);
    e2m1x8(tile.k.w, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a0 = hmul2(x[j], sa), a1 = hmul2(z[j], sb), a2 = hmul2(y[j], sa), a3 = hmul2(w[j], sb);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
    }
  }
  // scores in log2 units: s[nt][e] key g, s[nt][2 + e] key g + 8, row e
  bool move = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[nt][e] *= coef[nt][e];
      s[nt][2 + e] *= coef[nt][e];
      if (kMasked) {
        const int at = pos[nt][e], lo = mk.window < 0 ? 0 : at - mk.window;
        const int k0 = mk.key0 + g, k1 = k0 + 8;
        if (!(k0 <= at && (k0 >= lo || k0 < mk.prefix))) s[nt][e] = -INFINITY;
        if (!(k1 <= at && (k1 >= lo || k1 < mk.prefix))) s[nt][2 + e] = -INFINITY;
      }
      move |= fmaxf(s[nt][e], s[nt][2 + e]) > r.limit[nt][e];
    }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = fmaxf(s[nt][e], s[nt][2 + e]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        // rows that have seen nothing hold zeros: their factor may be anything finite
        if (m > r.limit[nt][e]) {
          const float f = r.limit[nt][e] == -INFINITY ? 0.f : ex2(r.ref[nt][e] - m);
          r.ref[nt][e] = m;
          r.limit[nt][e] = m + kSlack;
          r.sum[nt][e] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            r.o[nt][i][e] *= f;
            r.o[nt][i][2 + e] *= f;
          }
        }
      }
  }
  uint32_t pf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[nt][e] = ex2(s[nt][e] - r.ref[nt][e]);
      s[nt][2 + e] = ex2(s[nt][2 + e] - r.ref[nt][e]);
      r.sum[nt][e] += s[nt][e] + s[nt][2 + e];
    }
    pf[nt][0] = transpose8(pack_f16(s[nt][0], s[nt][1]));
    pf[nt][1] = transpose8(pack_f16(s[nt][2], s[nt][3]));
  }
  uint32_t vs = tile.vs;
  if (kMasked) {
    // What a masked key holds must not reach a row that does not see it, and
    // 0 * NaN would: NaN scales are taken out of the product, and the rows
    // that do see such a key get a NaN in the dims it stands for.
    const bool nan = any_nan_scale(vs);
    if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
      for (int key = 0; key < 16; ++key) {
        const int i = (key & 1) + 2 * (key >> 3);
        const uint32_t byte = __shfl_sync(0xffffffffu, vs, 4 * g + ((key & 7) >> 1)) >> (8 * i) & 0x7fu;
        if (byte != kNaNScale) continue;
        const int kp = mk.key0 + key;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = pos[nt][e];
            if (kp <= at && (mk.window < 0 || kp >= at - mk.window || kp < mk.prefix)) {
#pragma unroll
              for (int d = 0; d < 4; ++d) r.o[nt][d][e] = r.o[nt][d][2 + e] = __int_as_float(0x7fffffff);
            }
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((vs >> (8 * i) & 0x7fu) == kNaNScale) vs &= ~(0xffu << (8 * i));
    }
  }
  const uint32_t s01 = e4m3x2(vs), s23 = e4m3x2(vs >> 16);
  uint32_t e01, o01, e23, o23, a[4], b[4], c[4], d[4];
  pair_tokens(tile.v.x, tile.v.y, e01, o01);
  pair_tokens(tile.v.z, tile.v.w, e23, o23);
  e2m1x8(e01, a);
  e2m1x8(o01, b);
  e2m1x8(e23, c);
  e2m1x8(o23, d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a0 = hmul2(a[i], s01), a1 = hmul2(b[i], s01), a2 = hmul2(c[i], s23), a3 = hmul2(d[i], s23);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma_f16(r.o[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
  }
}

// Writes one finished row pair of dims: o = alpha * acc / sum, lse.
SA_DEV void finish_row(const DecK& p, int b, int head, int row, int d0, int nd, const float* acc, float sum, float ref,
                       float factor) {
  const int i = row / p.group, h = head * p.group + row % p.group;
  const int64_t at = static_cast<int64_t>(b) * p.n + i;
  const float lse = sum == 0.f ? -INFINITY : (ref + lg2(sum)) * kLn2;
  const float w = sum == 0.f ? 0.f : factor / (sum * (1.f + __expf(p.sink[h] - lse)));
  __nv_bfloat16* o = p.o + (at * p.hq + h) * kHeadDim + d0;
  for (int e = 0; e < nd; e += 2)
    *reinterpret_cast<uint32_t*>(o + e) = sum == 0.f ? 0u : pack_bf16(acc[e] * w, acc[e + 1] * w);
  if (d0 == 0) p.lse[static_cast<int64_t>(h) * p.num_seqs * p.n + at] = lse;
}

template <int NT, int kDepth>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) kv4_decode_kernel(const DecK p) {
  constexpr int kRows = 8 * NT;
  constexpr int kPartFloats = kRows * (kHeadDim + 2);
  constexpr int kDims = kRows * kHeadDim / kThreads;  // output dims per thread when merging: 2, 4 or 8
  extern __shared__ __align__(16) uint8_t smem[];
  // merge area [warps][rows][kRowPad], statistics [warps][rows][2], then the running block counts [num_seqs + 1]
  float* acc_sh = reinterpret_cast<float*>(smem);
  float* stat_sh = acc_sh + kWarps * kRows * kRowPad;
  long long* upto = reinterpret_cast<long long*>(stat_sh + kWarps * kRows * 2);
  __shared__ long long warp_sum[kWarps];
  __shared__ int last_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane_g(), t = lane_t();

  // blocks per sequence (an empty one counts as one: its rows are written too) and their running total
  long long carry = 0;
  for (int base = 0; base < p.num_seqs; base += kThreads) {
    const int b = base + tid;
    long long x = b < p.num_seqs ? max(visible_span(p, b).count(), 1) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long before = carry, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (b < p.num_seqs) upto[b + 1] = before + x;
    carry += all;
    __syncthreads();
  }
  if (tid == 0) upto[0] = 0;
  __syncthreads();

  const int per_seq = p.c.num_heads_kv * p.row_groups;  // pairs per sequence
  const long long work = carry * per_seq, pairs = static_cast<long long>(p.num_seqs) * per_seq;
  // at least a block for every warp of a CTA, unless that leaves pairs without a CTA of their own
  const long long want = max((work + kWarps - 1) / kWarps, pairs);
  const long long ctas = min(static_cast<long long>(gridDim.x), want);
  const long long cta = blockIdx.x;
  if (cta >= ctas) return;
  long long x = cta * work / ctas;
  const long long x_end = (cta + 1) * work / ctas;

  while (x < x_end) {
    int b;
    {  // the sequence that holds x
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (upto[mid] * per_seq <= x)
          lo = mid;
        else
          hi = mid - 1;
      }
      b = lo;
    }
    const Span span = visible_span(p, b);
    const int blocks = max(span.count(), 1);
    const long long off = x - upto[b] * per_seq;
    const int in_seq = static_cast<int>(off / blocks), blk0 = static_cast<int>(off % blocks);
    const int blk1 = static_cast<int>(min(static_cast<long long>(blocks), blk0 + (x_end - x)));
    const int head = in_seq / p.row_groups, row0 = in_seq % p.row_groups * kRows;
    const int slot = p.slots[b];

    // query rows: lane (g, t) holds row g's dims 16 t .. 16 t + 15 as B fragments
    uint32_t qf[NT][4][2];
    float coef[NT][2];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + 8 * nt + g;
      uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (row < p.rows) {
        const int64_t at = static_cast<int64_t>(b) * p.n + row / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (at * p.hq + head * p.group + row % p.group) * kHeadDim + 16 * t);
        const uint4 u = __ldg(src), v = __ldg(src + 1);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
      }
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
      const float mine = down * (p.scale * kLog2e * p.c.k_scale[head]);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        coef[nt][r] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + r));
        const int rr = row0 + 8 * nt + 2 * t + r;
        pos[nt][r] = rr < p.rows ? span.len - p.n + rr / p.group : -1;
      }
    }

    Rows<NT> r;
    rows_clear(r);
    if (span.len > 0) {
      const int first = span.len - p.n;  // every block wholly at or before `first` is seen by all rows causally
      const int last_lo = p.window < 0 ? 0 : span.len - 1 - p.window;
      Tile tile[kDepth];
      int page[kDepth];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int i = blk0 + warp + d * kWarps;
        page[d] = i < blk1 ? page_of(p.c, slot, span.block(i)) : -1;
      }
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int i = blk0 + warp + d * kWarps;
        if (i < blk1) load_tile(p.c, page[d], head, span.block(i), tile[d]);
        const int ahead = i + kDepth * kWarps;
        page[d] = ahead < blk1 ? page_of(p.c, slot, span.block(ahead)) : -1;
      }
      for (int i0 = blk0 + warp; i0 < blk1; i0 += kDepth * kWarps) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int i = i0 + d * kWarps;
          if (i >= blk1) break;
          const int key0 = span.block(i) * kBlockTokens, key1 = key0 + kBlockTokens - 1;
          const MaskArgs mk{key0, p.window, p.prefix};
          if (key1 <= first && (key0 >= last_lo || key1 < p.prefix))
            block_step<NT, false>(r, tile[d], qf, coef, pos, mk);
          else
            block_step<NT, true>(r, tile[d], qf, coef, pos, mk);
          const int ahead = i + kDepth * kWarps;
          if (ahead < blk1) load_tile(p.c, page[d], head, span.block(ahead), tile[d]);
          const int further = ahead + kDepth * kWarps;
          page[d] = further < blk1 ? page_of(p.c, slot, span.block(further)) : -1;
        }
      }
    }

    // the warps' results into shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = r.sum[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * nt + 2 * t + e;
        float4* to = reinterpret_cast<float4*>(acc_sh + (warp * kRows + row) * kRowPad + 8 * g);
        to[0] = make_float4(r.o[nt][0][e], r.o[nt][0][2 + e], r.o[nt][1][e], r.o[nt][1][2 + e]);
        to[1] = make_float4(r.o[nt][2][e], r.o[nt][2][2 + e], r.o[nt][3][e], r.o[nt][3][2 + e]);
        if (g == 0) {
          stat_sh[(warp * kRows + row) * 2] = r.limit[nt][e] == -INFINITY ? -INFINITY : r.ref[nt][e];
          stat_sh[(warp * kRows + row) * 2 + 1] = sum;
        }
      }
    __syncthreads();

    // thread: one row, kDims of its dims
    const int row = tid / (kThreads / kRows), d0 = tid % (kThreads / kRows) * kDims;
    float acc[kDims], sum = 0.f, ref = -INFINITY;
#pragma unroll
    for (int d = 0; d < kDims; ++d) acc[d] = 0.f;
    for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, stat_sh[(w * kRows + row) * 2]);
    for (int w = 0; w < kWarps; ++w) {
      const float m = stat_sh[(w * kRows + row) * 2];
      if (m == -INFINITY) {  // nothing of it was seen; what it holds is zero, or NaN where a score was
        sum += stat_sh[(w * kRows + row) * 2 + 1];
        continue;
      }
      const float f = ex2(m - ref);
      sum += f * stat_sh[(w * kRows + row) * 2 + 1];
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] += f * acc_sh[(w * kRows + row) * kRowPad + d0 + d];
    }

    const float factor = p.c.v_scale[head];
    const bool there = row0 + row < p.rows;
    if (blk0 == 0 && blk1 == blocks) {
      if (there) finish_row(p, b, head, row0 + row, d0, kDims, acc, sum, ref, factor);
    } else {
      const long long pair = static_cast<long long>(b) * per_seq + in_seq;
      const long long p0 = x - blk0, p1 = p0 + blocks;  // the pair's place in the line
      const long long c0 = ((p0 + 1) * ctas - 1) / work, c1 = (p1 * ctas - 1) / work;
      const auto slot_of = [&](long long c) { return p.part + (2 * c + (p0 > c * work / ctas ? 1 : 0)) * kPartFloats; };
      float* mine = slot_of(cta);
      if (there) {
#pragma unroll
        for (int d = 0; d < kDims; ++d) __stcg(mine + row * kHeadDim + d0 + d, acc[d]);
        if (d0 == 0) {
          __stcg(mine + kRows * kHeadDim + 2 * row, ref);
          __stcg(mine + kRows * kHeadDim + 2 * row + 1, sum);
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) last_sh = atomicAdd(p.counters + pair, 1) == static_cast<int>(c1 - c0);
      __syncthreads();
      if (last_sh) {
        __threadfence();
        if (tid == 0) p.counters[pair] = 0;
        if (there) {
          float all[kDims], total = 0.f, top = -INFINITY;
#pragma unroll
          for (int d = 0; d < kDims; ++d) all[d] = 0.f;
          for (long long c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(slot_of(c) + kRows * kHeadDim + 2 * row));
          for (long long c = c0; c <= c1; ++c) {
            const float* from = slot_of(c);
            const float m = __ldcg(from + kRows * kHeadDim + 2 * row), l = __ldcg(from + kRows * kHeadDim + 2 * row + 1);
            const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - top);
            total += f * l;
#pragma unroll
            for (int d = 0; d < kDims; ++d) all[d] += f * __ldcg(from + row * kHeadDim + d0 + d);
          }
          finish_row(p, b, head, row0 + row, d0, kDims, all, total, top, factor);
        }
      }
    }
    __syncthreads();  // the merge area is free again
    x += blk1 - blk0;
  }
}

template <int NT, int kDepth>
cudaError_t launch_variant(const DecK& p, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kWarps) * 8 * NT * (kRowPad + 2) * 4 + (p.num_seqs + 1) * 8;
  const auto kernel = kv4_decode_kernel<NT, kDepth>;
  if (smem > 48 * 1024) {  // more than a kernel has without asking
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int grid = device_sms() * (NT == 1 ? 2 : 1);
  kernel<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Partial results first, in a place that depends on the GPU alone, then the
// counters (zero between calls, at most one per query row and head): a
// workspace zeroed once serves calls of any shape it is large enough for.
static size_t part_bytes() { return static_cast<size_t>(device_sms()) * kPartRowsPerSm * (kHeadDim + 2) * 4; }

size_t kv4_decode_workspace_bytes(long long rows, int hq) {
  return (part_bytes() + 255) / 256 * 256 + static_cast<size_t>(rows) * hq * 4;
}

cudaError_t launch_kv4_decode(const Kv4Cache& c, const Kv4DecodeArgs& a, cudaStream_t s) {
  DecK p;
  p.c = c;
  p.slots = a.slots;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.sink = a.sink;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.part = static_cast<float*>(a.workspace);
  p.counters = reinterpret_cast<int*>(static_cast<uint8_t*>(a.workspace) + (part_bytes() + 255) / 256 * 256);
  p.num_seqs = a.num_seqs;
  p.n = a.n;
  p.hq = a.hq;
  p.group = a.hq / c.num_heads_kv;
  p.rows = p.group * a.n;
  p.window = a.window;
  p.prefix = a.prefix;
  p.scale = a.scale;
  const int nt = p.rows <= 8 ? 1 : p.rows <= 16 ? 2 : 4;
  p.row_groups = ceil_div(p.rows, 8 * nt);
  if (nt == 1) return launch_variant<1, 4>(p, s);
  if (nt == 2) return launch_variant<2, 3>(p, s);
  return launch_variant<4, 2>(p, s);
}

}  // namespace sa

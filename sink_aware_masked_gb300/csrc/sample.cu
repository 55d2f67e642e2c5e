// Token sampling with temperature, top-k, top-p and min-p from given random
// numbers, with the token's log-probability (what the GRPO loss takes as
// logp_old).
//
//   e_i = exp((x_i - max x) / T),  Z = sum e
//   order: larger x first, of equal ones the lower index
//   top-k keeps the first k; top-p of those the shortest run whose mass is at
//   least p times theirs; min-p of those the ones with e_i >= min_p
//   token = the first index, in index order, whose kept mass up to and
//   including it exceeds u times the kept mass
//
// A cluster of CTAs takes one row: every CTA keeps its slice of the logits in
// shared memory, so HBM is read once, and what follows is passes over shared
// memory with a few numbers exchanged between the CTAs.
//
// Selection without sorting: a histogram (count and mass) of the candidates
// over equal steps of x finds the step in which the cut lies; its members, if
// few, are ranked by one CTA, else they are split again by their exact key
// (x's bits and the index, so all keys differ) until they are few.
//
// Masses are 43-bit fixed point, e / Z * 2^43: integer sums are the same in
// every order, so histogram atomics leave the result reproducible, and 2^18
// of them lose at most 2^-25 of the whole.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kIndexBits = 18;            // vocabularies up to 2^18
constexpr int kBins = 1024;
constexpr int kList = 4096;               // candidates a CTA keeps a list of
constexpr int kGather = kThreads;         // members the last step ranks, one per thread
constexpr double kMassOne = 8796093022208.0;  // 2^43
constexpr int kLowBits = 13;

typedef unsigned long long u64;

struct Pick {  // what a histogram step found
  int bin;
  u64 members;     // candidates in the bin
  u64 count, mass; // of all bins before it
};

struct Shared {
  u64 exchange[2][kMaxCluster];
  double warp_d[kWarps];
  u64 warp_u[kWarps], warp_v[kWarps];
  float warp_f[kWarps];
  u64 lo, hi, cut, cut_mass;
  Pick pick;
  int list_n, gathered, found;
  uint32_t count[kBins], mass_hi[kBins], mass_lo[kBins];  // this CTA's histogram
  uint32_t all_count[kBins];                              // CTA 0: the row's
  u64 all_mass[kBins];
  u64 key[kGather], key_mass[kGather], sorted[kGather], sorted_mass[kGather];
  uint16_t list[kList];
};

template <int kType>
struct Elem;
template <>
struct Elem<0> {
  typedef float T;
  static constexpr int kVec = 4;
  static SA_DEV void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static SA_DEV float one(T v) { return v; }
  static SA_DEV T lowest() { return -INFINITY; }
};
template <>
struct Elem<1> {
  typedef uint16_t T;
  static constexpr int kVec = 8;
  static SA_DEV void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  static SA_DEV float one(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static SA_DEV T lowest() { return 0xff80u; }
};
template <>
struct Elem<2> {
  typedef uint16_t T;
  static constexpr int kVec = 8;
  static SA_DEV void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static SA_DEV float one(T v) { return __half2float(*reinterpret_cast<const __half*>(&v)); }
  static SA_DEV T lowest() { return 0xfc00u; }
};

// Larger x, larger key; -0 and +0 are one value.
SA_DEV uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
SA_DEV u64 full_key(float x, int index) {
  return static_cast<u64>(order_key(x)) << kIndexBits | ((1u << kIndexBits) - 1 - index);
}

SA_DEV float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <class T>
SA_DEV T warp_sum(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <class T>
SA_DEV T warp_scan(T x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

template <int kType>
class Row {
 public:
  typedef Elem<kType> E;
  typedef typename E::T T;

  SA_DEV Row(Shared& sh, T* raw) : sh_(sh), raw_(raw), cluster_(cg::this_cluster()) {
    rank_ = cluster_.block_rank();
    ctas_ = cluster_.num_blocks();
  }

  SA_DEV void run(const SampleArgs& a, int row, int slice) {
    const int tid = threadIdx.x;
    vocab_ = a.vocab;
    first_ = min(static_cast<int>(rank_) * slice, a.vocab);
    const int last = min(first_ + slice, a.vocab);
    const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.stride;
    cluster_.barrier_arrive();
    float mine = load(x, last);
    const float thread_max = mine;
    mine = warp_max(mine);
    if ((tid & 31) == 0) sh_.warp_f[tid >> 5] = mine;
    __syncthreads();
    mine = sh_.warp_f[0];
    for (int w = 1; w < kWarps; ++w) mine = fmaxf(mine, sh_.warp_f[w]);
    max_ = -INFINITY;
    cluster_.barrier_wait();  // every CTA of the cluster runs: its shared memory may be written
    exchange(__float_as_uint(mine), [&](u64 v) { max_ = fmaxf(max_, __uint_as_float(static_cast<uint32_t>(v))); });

    const float temperature = a.temperature[row], top_p = a.top_p[row], min_p = a.min_p[row], u = a.u[row];
    int k = a.top_k[row];
    const bool greedy = temperature == 0.f;
    const double inv_t = greedy ? 1.0 : 1.0 / static_cast<double>(temperature);
    scale_ = static_cast<float>(fmin(1.4426950408889634 * inv_t, 1e38));
    if (!(temperature >= 0.f && temperature < INFINITY) || top_p != top_p || min_p != min_p || u != u) {
      if (rank_ == 0 && tid == 0) put(a, row, -1, NAN, NAN);
      return;
    }
    if (max_ == -INFINITY) {  // nothing is allowed, or all there is is NaN
      const float v = any_nan() ? NAN : -INFINITY;
      if (rank_ == 0 && tid == 0) put(a, row, -1, v, v);
      return;
    }
    // Z; a NaN among the logits makes it NaN, an infinite one too
    float part = 0.f;
    each_vector([&](const float* v, int) {
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) part += mass(v[e]);
    });
    const double slice_z = block_sum_d(static_cast<double>(part));
    z_ = 0.0;
    exchange(__double_as_longlong(slice_z), [&](u64 v) { z_ += __longlong_as_double(static_cast<long long>(v)); });
    if (max_ == INFINITY || z_ != z_) {
      if (rank_ == 0 && tid == 0) put(a, row, -1, NAN, NAN);
      return;
    }
    to_fixed_ = static_cast<float>(kMassOne / z_);

    if (greedy || top_p <= 0.f) k = 1;
    if (k == 1) {  // the largest, of equal ones the lowest index
      int at = vocab_;
      each_vector([&](const float* v, int base) {
#pragma unroll
        for (int e = E::kVec - 1; e >= 0; --e)
          if (v[e] == max_) at = min(at, base + e);
      });
      at = block_min(at);
      int best = vocab_;
      exchange(static_cast<u64>(at), [&](u64 v) { best = min(best, static_cast<int>(v)); });
      if (rank_ == 0 && tid == 0) put(a, row, best, static_cast<float>(-log(z_)), 0.f);
      return;
    }

    cut_ = 0;
    min_mass_ = fminf(min_p, 1.f);
    const bool by_count = k > 0 && k < vocab_, by_mass = top_p < 1.f;
    if (by_count || by_mass) {
      float floor = -INFINITY;
      if (by_count) {
        floor = count_floor(thread_max, k);
      } else {
        // what lies below (1 - p) Z / vocab holds less than (1 - p) Z together; 1 % to spare for rounding
        const double least = (1.0 - static_cast<double>(top_p)) * 0.99 * z_ / vocab_;
        floor = static_cast<float>(max_ + log(least) / inv_t * 1.0001);
        floor -= fabsf(floor) * 2.4e-7f;
      }
      make_list(floor);
      // steps for the first histogram: the candidates' range, or what holds all mass that counts
      const float range = floor > -INFINITY ? max_ - floor : static_cast<float>(30.0 / inv_t);
      per_step_ = range > 0.f ? fminf((kBins - 1) / range, 1e30f) : 0.f;
      double kept = z_ * static_cast<double>(to_fixed_);
      if (by_count) kept = static_cast<double>(search(true, static_cast<double>(k)));
      if (by_mass) search(false, static_cast<double>(top_p) * kept);
    }
    sample(a, row, u, inv_t);
  }

 private:
  // Every CTA of the cluster gives a number and takes all of them in rank order.
  template <class F>
  SA_DEV void exchange(u64 v, F take) {
    u64* buf = sh_.exchange[parity_];
    parity_ ^= 1;  // the other half may still be read by a slower CTA
    if (threadIdx.x < ctas_) cluster_.map_shared_rank(buf, threadIdx.x)[rank_] = v;
    cluster_.sync();
    for (unsigned r = 0; r < ctas_; ++r) take(buf[r]);
  }

  // Copies the slice into shared memory at the alignment it has in global
  // memory, -inf around it, and returns the thread's largest logit.
  SA_DEV float load(const T* x, int last) {
    const int tid = threadIdx.x;
    shift_ = static_cast<int>((reinterpret_cast<uintptr_t>(x + first_) / sizeof(T)) % E::kVec);
    const int n = last - first_, end = shift_ + n;
    vectors_ = n > 0 ? (end + E::kVec - 1) / E::kVec : 0;
    float top = -INFINITY;
    const T* base = x + first_ - shift_;
    const auto keep = [&](int v, uint4 w) {
      reinterpret_cast<uint4*>(raw_)[v] = w;
      float f[E::kVec];
      E::unpack(w, f);
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) top = fmaxf(top, f[e]);
    };
    const auto edge = [&](int v) {
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) {
        const int i = v * E::kVec + e;
        const T w = i >= shift_ && i < end ? base[i] : E::lowest();
        raw_[i] = w;
        top = fmaxf(top, E::one(w));
      }
    };
    const int v0 = shift_ > 0 ? 1 : 0, v1 = end / E::kVec;  // [v0, v1): whole vectors
    constexpr int kUnroll = 4;
    int v = v0 + tid;
    for (; v + (kUnroll - 1) * kThreads < v1; v += kUnroll * kThreads) {
      uint4 w[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(base) + v + i * kThreads);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) keep(v + i * kThreads, w[i]);
    }
    for (; v < v1; v += kThreads) keep(v, __ldcs(reinterpret_cast<const uint4*>(base) + v));
    if (vectors_ > 0) {
      if (tid == 0 && v0 == 1) edge(0);
      if (tid == 32 && vectors_ - 1 >= v1 && (vectors_ > 1 || v0 == 0)) edge(vectors_ - 1);
    }
    __syncthreads();
    return top;
  }

  // f(values, index of the first) for every vector; the indices of padding lie outside [first, last) but are -inf.
  template <class F>
  SA_DEV void each_vector(F f) {
    for (int v = threadIdx.x; v < vectors_; v += kThreads) {
      float x[E::kVec];
      E::unpack(reinterpret_cast<const uint4*>(raw_)[v], x);
      f(x, first_ + v * E::kVec - shift_);
    }
  }

  SA_DEV float mass(float x) const { return ex2((x - max_) * scale_); }
  SA_DEV u64 fixed(float x) const { return static_cast<u64>(mass(x) * to_fixed_); }

  SA_DEV bool any_nan() {  // in the whole row; every CTA of the cluster asks
    int bad = 0;
    each_vector([&](const float* v, int) {
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) bad |= v[e] != v[e];
    });
    bad = __syncthreads_or(bad);
    bool any = false;
    exchange(static_cast<u64>(bad), [&](u64 v) { any |= v != 0; });
    return any;
  }

  SA_DEV double block_sum_d(double x) {
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) sh_.warp_d[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kWarps; ++w) s += sh_.warp_d[w];
    return s;
  }
  SA_DEV int block_min(int x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
    if ((threadIdx.x & 31) == 0) sh_.warp_u[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) x = min(x, static_cast<int>(sh_.warp_u[w]));
    return x;
  }

  // A value that at least k logits reach: in each CTA the k / ctas-th largest
  // of the threads' maxima, and the least of those over the CTAs.
  SA_DEV float count_floor(float thread_max, int k) {
    const int quota = (k + ctas_ - 1) / ctas_;
    if (quota > kThreads) return -INFINITY;
    const uint32_t key = order_key(thread_max);
    uint32_t lo = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t mid = lo | 1u << bit;
      if (__syncthreads_count(key >= mid) >= quota) lo = mid;
    }
    uint32_t least = 0xffffffffu;
    exchange(lo, [&](u64 v) { least = min(least, static_cast<uint32_t>(v)); });
    const uint32_t bits = (least >> 31) ? least ^ 0x80000000u : ~least;
    const float f = __uint_as_float(bits);
    return f == f ? f : -INFINITY;  // fewer threads than the quota hold anything: key 0
  }

  // The slice's candidates (x >= floor); scan_all_ where they are too many for a list.
  SA_DEV void make_list(float floor) {
    floor_ = floor;
    if (threadIdx.x == 0) sh_.list_n = 0;
    __syncthreads();
    each_vector([&](const float* x, int base) {
#pragma unroll
      for (int e = 0; e < E::kVec; ++e)
        if (x[e] >= floor && x[e] > -INFINITY) {
          const int at = atomicAdd(&sh_.list_n, 1);
          if (at < kList) sh_.list[at] = static_cast<uint16_t>(base + e - first_);
        }
    });
    __syncthreads();
    list_n_ = sh_.list_n;
  }

  // f(x, index) for the slice's candidates.
  template <class F>
  SA_DEV void each_candidate(F f) {
    if (list_n_ <= kList) {
      for (int i = threadIdx.x; i < list_n_; i += kThreads) {
        const int at = sh_.list[i];
        f(E::one(raw_[at + shift_]), first_ + at);
      }
    } else {
      each_vector([&](const float* x, int base) {
#pragma unroll
        for (int e = 0; e < E::kVec; ++e)
          if (x[e] >= floor_ && x[e] > -INFINITY) f(x[e], base + e);
      });
    }
  }

  SA_DEV int step_of(float x) const { return static_cast<int>(fminf((max_ - x) * per_step_, kBins - 1.f)); }

  // Histogram of what bin_of gives a bin (>= 0), summed over the cluster; the
  // first bin at which count or mass reaches the target, starting from before.
  template <class F>
  SA_DEV Pick histogram(bool by_count, double target, u64 count0, u64 mass0, F bin_of) {
    const int tid = threadIdx.x;
    for (int i = tid; i < kBins; i += kThreads) sh_.count[i] = sh_.mass_hi[i] = sh_.mass_lo[i] = 0;
    __syncthreads();
    each_candidate([&](float x, int index) {
      const int bin = bin_of(x, index);
      if (bin < 0) return;
      const u64 m = fixed(x);
      atomicAdd(&sh_.count[bin], 1u);
      atomicAdd(&sh_.mass_hi[bin], static_cast<uint32_t>(m >> kLowBits));
      atomicAdd(&sh_.mass_lo[bin], static_cast<uint32_t>(m & ((1u << kLowBits) - 1)));
    });
    cluster_.sync();
    const int share = kBins / ctas_;
    for (int i = rank_ * share + tid; i < static_cast<int>(rank_ + 1) * share; i += kThreads) {
      uint32_t n = 0;
      u64 m = 0;
      for (unsigned r = 0; r < ctas_; ++r) {
        n += cluster_.map_shared_rank(sh_.count, r)[i];
        m += (static_cast<u64>(cluster_.map_shared_rank(sh_.mass_hi, r)[i]) << kLowBits) +
             cluster_.map_shared_rank(sh_.mass_lo, r)[i];
      }
      cluster_.map_shared_rank(sh_.all_count, 0)[i] = n;
      cluster_.map_shared_rank(sh_.all_mass, 0)[i] = m;
    }
    cluster_.sync();
    if (rank_ == 0) {
      constexpr int kPer = kBins / kThreads;
      u64 n = 0, m = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) n += sh_.all_count[tid * kPer + j], m += sh_.all_mass[tid * kPer + j];
      const u64 n_in = block_scan(n, sh_.warp_u), m_in = block_scan(m, sh_.warp_v);
      if (tid == 0) sh_.found = kBins;
      __syncthreads();
      u64 nb = count0 + n_in - n, mb = mass0 + m_in - m;
      Pick p;
      p.bin = kBins;
      int last = -1;  // the thread's last bin with members
      Pick lastp;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int bin = tid * kPer + j;
        const u64 c = sh_.all_count[bin], ms = sh_.all_mass[bin];
        const bool reached = by_count ? static_cast<double>(nb + c) >= target : static_cast<double>(mb + ms) >= target;
        if (c > 0) last = bin, lastp.bin = bin, lastp.members = c, lastp.count = nb, lastp.mass = mb;
        if (reached && c > 0 && p.bin == kBins) p.bin = bin, p.members = c, p.count = nb, p.mass = mb;
        nb += c;
        mb += ms;
      }
      if (p.bin < kBins) atomicMin(&sh_.found, p.bin);
      __syncthreads();
      const int hit = sh_.found;
      __syncthreads();
      if (hit == kBins) {  // rounding kept the sum below the target: the last bin that has members
        if (tid == 0) sh_.found = -1;
        __syncthreads();
        if (last >= 0) atomicMax(&sh_.found, last);
        __syncthreads();
        if (last >= 0 && sh_.found == last) sh_.pick = lastp;
        if (sh_.found < 0 && tid == 0) sh_.pick = Pick{-1, 0, count0, mass0};
      } else if (p.bin == hit) {
        sh_.pick = p;
      }
      __syncthreads();
      if (tid > 0 && tid < ctas_) *cluster_.map_shared_rank(&sh_.pick, tid) = sh_.pick;
    }
    cluster_.sync();
    return sh_.pick;
  }

  SA_DEV u64 block_scan(u64 x, u64* sums) {
    x = warp_scan(x);
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 31) sums[w] = x;
    __syncthreads();
    for (int i = 0; i < w; ++i) x += sums[i];
    return x;
  }

  // Moves cut_ to the key of the last candidate that is kept and returns the
  // mass of the kept ones.  Candidates below the present cut do not count.
  SA_DEV u64 search(bool by_count, double target) {
    const int tid = threadIdx.x;
    const u64 cut = cut_;
    Pick p = histogram(by_count, target, 0, 0, [&](float x, int index) {
      return full_key(x, index) >= cut ? step_of(x) : -1;
    });
    const int step = p.bin;
    u64 lo = 0, hi = ~0ull;
    if (p.members > kGather) {  // the members' range of keys
      u64 least = ~0ull, most = 0;
      each_candidate([&](float x, int index) {
        const u64 key = full_key(x, index);
        if (key >= cut && step_of(x) == step) least = least < key ? least : key, most = most > key ? most : key;
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const u64 a = __shfl_xor_sync(0xffffffffu, least, o), b = __shfl_xor_sync(0xffffffffu, most, o);
        least = least < a ? least : a;
        most = most > b ? most : b;
      }
      if ((tid & 31) == 0) sh_.warp_u[tid >> 5] = least, sh_.warp_v[tid >> 5] = most;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) {
        least = least < sh_.warp_u[w] ? least : sh_.warp_u[w];
        most = most > sh_.warp_v[w] ? most : sh_.warp_v[w];
      }
      exchange(least, [&](u64 v) { least = least < v ? least : v; });
      exchange(most, [&](u64 v) { most = most > v ? most : v; });
      lo = least;
      hi = most;
    }
    while (p.members > kGather) {  // keys differ, so each turn leaves fewer
      int shift = 0;
      while (((hi - lo) >> shift) >= kBins) ++shift;
      p = histogram(by_count, target, p.count, p.mass, [&](float x, int index) {
        const u64 key = full_key(x, index);
        return key >= cut && key >= lo && key <= hi && step_of(x) == step ? static_cast<int>((hi - key) >> shift) : -1;
      });
      const u64 top = hi - (static_cast<u64>(p.bin) << shift);
      const u64 width = (1ull << shift) - 1;
      lo = top - lo > width ? top - width : lo;
      hi = top;
    }
    // the members to CTA 0, which ranks them
    if (tid == 0) sh_.gathered = 0;
    cluster_.sync();
    {
      int* n = cluster_.map_shared_rank(&sh_.gathered, 0);
      u64* keys = cluster_.map_shared_rank(sh_.key, 0);
      u64* masses = cluster_.map_shared_rank(sh_.key_mass, 0);
      each_candidate([&](float x, int index) {
        const u64 key = full_key(x, index);
        if (key >= cut && key >= lo && key <= hi && step_of(x) == step) {
          const int at = atomicAdd(n, 1);
          if (at < kGather) keys[at] = key, masses[at] = fixed(x);
        }
      });
    }
    cluster_.sync();
    if (rank_ == 0) {
      const int n = min(sh_.gathered, kGather);
      u64 key = 0;
      if (tid < n) {
        key = sh_.key[tid];
        int r = 0;
        for (int j = 0; j < n; ++j) r += sh_.key[j] > key;
        sh_.sorted[r] = key;
        sh_.sorted_mass[r] = sh_.key_mass[tid];
      }
      if (tid == 0) sh_.found = n - 1;
      __syncthreads();
      const u64 m = p.mass + block_scan(tid < n ? sh_.sorted_mass[tid] : 0, sh_.warp_u);
      const bool reached = by_count ? static_cast<double>(p.count + tid + 1) >= target : static_cast<double>(m) >= target;
      if (tid < n && reached) atomicMin(&sh_.found, tid);
      __syncthreads();
      if (tid == max(sh_.found, 0)) {
        sh_.cut = n > 0 ? sh_.sorted[tid] : cut;
        sh_.cut_mass = m;
      }
      __syncthreads();
      if (tid > 0 && tid < ctas_) {
        *cluster_.map_shared_rank(&sh_.cut, tid) = sh_.cut;
        *cluster_.map_shared_rank(&sh_.cut_mass, tid) = sh_.cut_mass;
      }
    }
    cluster_.sync();
    cut_ = sh_.cut;
    return sh_.cut_mass;
  }

  SA_DEV u64 kept_mass(float x, int index) const {
    if (static_cast<u64>(order_key(x)) < (cut_ >> kIndexBits) || full_key(x, index) < cut_) return 0;
    const float e = mass(x);
    return e >= min_mass_ ? static_cast<u64>(e * to_fixed_) : 0;
  }

  // Index order: a CTA's slice, in it the warps' runs of vectors, in those the turns, lanes and elements.
  SA_DEV void sample(const SampleArgs& a, int row, float u, double inv_t) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (vectors_ + kWarps - 1) / kWarps;
    const int v0 = min(warp * per, vectors_), v1 = min(v0 + per, vectors_);
    const auto vector_mass = [&](int v, u64* each) {
      u64 s = 0;
      float f[E::kVec];
      E::unpack(reinterpret_cast<const uint4*>(raw_)[v], f);
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) {
        const u64 m = kept_mass(f[e], first_ + v * E::kVec + e - shift_);
        if (each != nullptr) each[e] = m;
        s += m;
      }
      return s;
    };
    u64 mine = 0;
    for (int v = v0 + lane; v < v1; v += 32) mine += vector_mass(v, nullptr);
    mine = warp_sum(mine);
    __syncthreads();
    if (lane == 0) sh_.warp_u[warp] = mine;
    __syncthreads();
    u64 before = 0, slice = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh_.warp_u[w];
      slice += sh_.warp_u[w];
    }
    u64 total = 0, earlier = 0;
    unsigned r = 0;
    exchange(slice, [&](u64 v) {
      if (r++ < rank_) earlier += v;
      total += v;
    });
    // below 1, so that the sum over all exceeds the target
    const double target = static_cast<double>(fminf(fmaxf(u, 0.f), 0.99999994f)) * static_cast<double>(total);
    before += earlier;
    if (!(static_cast<double>(before) <= target && static_cast<double>(before + mine) > target)) return;
    for (int v = v0; v < v1; v += 32) {
      u64 each[E::kVec];
      const u64 m = v + lane < v1 ? vector_mass(v + lane, each) : 0;
      const u64 upto = before + warp_scan(m);
      const unsigned hit = __ballot_sync(0xffffffffu, static_cast<double>(upto) > target);
      if (hit == 0) {
        before = __shfl_sync(0xffffffffu, upto, 31);
        continue;
      }
      if (lane == __ffs(hit) - 1) {
        u64 run = upto - m;
#pragma unroll
        for (int e = 0; e < E::kVec; ++e) {
          run += each[e];
          if (static_cast<double>(run) > target) {
            const int at = (v + lane) * E::kVec + e;
            const double d = (static_cast<double>(E::one(raw_[at])) - static_cast<double>(max_)) * inv_t;
            const double kept = static_cast<double>(total) / static_cast<double>(to_fixed_);
            put(a, row, first_ + at - shift_, static_cast<float>(d - log(z_)), static_cast<float>(d - log(kept)));
            break;
          }
        }
      }
      return;
    }
  }

  static SA_DEV void put(const SampleArgs& a, int row, int token, float logp, float logq) {
    a.tokens[row] = token;
    a.logp[row] = logp;
    a.logq[row] = logq;
  }

  Shared& sh_;
  T* raw_;
  cg::cluster_group cluster_;
  unsigned rank_, ctas_;
  int parity_ = 0;
  int vocab_, first_, shift_, vectors_, list_n_;
  float max_, scale_, to_fixed_, min_mass_, floor_, per_step_;
  double z_;
  u64 cut_;
};

template <int kType>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a, int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  Row<kType> row(sh, reinterpret_cast<typename Elem<kType>::T*>(smem + (sizeof(Shared) + 15) / 16 * 16));
  row.run(a, blockIdx.x / cg::this_cluster().num_blocks(), slice);
}

template <int kType>
cudaError_t launch_type(const SampleArgs& a, cudaStream_t s) {
  int ctas = 1;
  while (ctas < kMaxCluster && ceil_div(a.vocab, ctas) > 4096) ctas *= 2;
  const int vec = Elem<kType>::kVec;
  const int slice = ceil_div(ceil_div(a.vocab, ctas), vec) * vec;
  const size_t smem =
      (sizeof(Shared) + 15) / 16 * 16 + (static_cast<size_t>(slice) + 2 * vec) * sizeof(typename Elem<kType>::T);
  const auto kernel = sample_kernel<kType>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, slice);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_type<0>(a, s);
  if (a.dtype == 1) return launch_type<1>(a, s);
  return launch_type<2>(a, s);
}

}  // namespace sa

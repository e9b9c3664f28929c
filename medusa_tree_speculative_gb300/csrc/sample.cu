// A token per row of logits: temperature, top-k, top-p and min-p, from a given
// number.
//
// In the order of falling logits (equal ones by index) each of the three rules
// keeps a first part of the row, so together they keep what comes up to one "cut".
// The token is where the running sum of the kept weights e^((z - max) / T), in
// vocabulary order, passes u times their sum.  Both the cut and the token are
// decided by sums over up to the whole row, in which one token's share may be
// 1e-6, so float32 weights (off by 1e-7, and their sums by more) would decide
// otherwise than the formula does now and then.  Here
//   * a weight is 2^(-k/32) (1 + q), k a whole number: k and the rest a / 32 of the
//     exponent come from a float32 product and what its rounding left, q from four
//     terms of the series.  |a| <= 1/2, and 1/8 more where the logits' product with
//     1/T's low part is that large (|max c| near 2^21 below), so |q| < 0.0137; its
//     roundings, of numbers below 2^-6, are together less than 2^-27 of the weight
//     (2^-28 where |a| is at most 0.51), as likely up as down;
//   * sums are of whole numbers: of q in units of 2^-31, with the count, per k (a
//     bin), or of weights in units of 2^-44, to which each is rounded: one below 2^-45
//     is kept, but adds nothing.  They do not depend on the order.  u = 0, the first
//     kept token whatever it weighs, is no matter of sums.
//
// A cluster of CTAs takes a row and keeps it in shared memory: one read, a bulk copy
// per warp.  The cut is found by narrowing: a histogram over k, the bin in which the
// count (top-k) or the sum (top-p) reaches its mark, then histograms over (logit,
// index) inside that bin until one token is left: two or three rounds, each a pass
// over shared memory and three cluster barriers.  A last pass sums the kept weights
// per warp, in vocabulary order, and the warp whose sum passes the mark finds the
// token.  (top-k with top-p ends in one CTA: `shorten`.)
// Bound for few rows by the chain: a cluster barrier takes 1100 cycles, a round 4500
// by counts and 5800 by sums, a pass over 16384 logits 2500 (counts) to 8000
// (weights).  Bound for many rows by the weights' instructions, about 30 a logit and
// pass; atomics are not it (three in place of one per logit: 322 and 312 us).
// Measured: one row of 32000 4.2 us greedy, 9.6 without cuts, 14 with top-k, 18 with
// top-p, 20 with both; 320 rows of 128257 (164 MB) 60, 159, 182, 333 and 187 us, 186
// with all kinds of settings among the rows.
// What did not go: sums in 64-bit floats (16 cycles a warp's instruction; 480 us in
// place of 342), 64-bit atomics (loops; 342 in place of 225), 1024 threads to a CTA
// and half the CTAs (201 in place of 192).
#include <math.h>

#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;          // of a histogram; k = 2047: weights below 2^-63, nothing in any unit
constexpr int kTail = kBins - 1;
constexpr int kIndexBits = 18;       // V <= 2^18
constexpr int kMaxV = 1 << kIndexBits;
constexpr int kShort = 1024;         // tokens that one CTA sorts
constexpr int kUnit = 44;            // weights are summed in units of 2^-44: 2^18 of them are below 2^63
// |q| 2^31 < 2^25: q 2^31 + 2^25 is summed as kLowBits low bits and what is above
// them, 13 bits each, in 32 bits (a CTA has at most 2^15 tokens)
constexpr int kQBias = 1 << 25, kLowBits = 13;

// 2^(31 - j/32), rounded
__device__ const uint32_t kPowers[32] = {
    2147483648u, 2101467502u, 2056437387u, 2012372174u, 1969251188u, 1927054196u, 1885761398u, 1845353420u,
    1805811301u, 1767116489u, 1729250827u, 1692196547u, 1655936265u, 1620452965u, 1585730000u, 1551751076u,
    1518500250u, 1485961921u, 1454120821u, 1422962010u, 1392470869u, 1362633090u, 1333434672u, 1304861917u,
    1276901417u, 1249540052u, 1222764986u, 1196563654u, 1170923762u, 1145833280u, 1121280436u, 1097253708u};

struct SampleArgs {
  const float* logits;
  const int32_t* node;
  int T, R, V, slice;  // slice: elements per CTA
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniforms;
  int32_t* token;
  float* logp;
  int32_t* kept;
  int32_t* err;
};

// Order of a token: the larger logit first (-0 and 0 are equal), then the lower index.
MDEV uint32_t falling(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return ~(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u));
}
MDEV uint64_t order_of(float z, int index) { return (uint64_t)falling(z) << kIndexBits | (uint32_t)index; }
MDEV float logit_of(uint64_t order) {
  const uint32_t f = ~(uint32_t)(order >> kIndexBits);
  return __uint_as_float(f ^ ((f >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint64_t kNone = ~0ull;    // after any order
constexpr float kLowest = -3.402823466e38f;

MDEV void st_cluster_u64(void* p, int rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(cluster_map(smem_u32(p), (uint32_t)rank)), "l"(v) : "memory");
}

// What weights of a row need.  `top` is whole, so that a bin's number is a whole
// number less rint(z c): weights are relative to 2^(-top/32) and not to the row's
// maximum, which changes none of their shares.
struct Scale {
  float max, c, c_low;  // 32 / (T ln 2) in two parts
  float top;            // max c, rounded, and 1: no bin is below 0
};
// k and q of a logit; q is nothing for the last k.  NEAR: max c is below 2^21, and
// one rounding of z c does; otherwise from the difference max - z, rounded, and what
// that left.
template <bool NEAR>
MDEV int weight_of(const Scale& s, float z, float& q) {
  constexpr float kRound = 12582912.f;  // 1.5 2^23: added, it leaves a whole number
  float y, a;
  if (NEAR) {
    y = fmaf(-z, s.c, kRound + s.top);
    a = fmaf(-z, s.c, kRound + s.top - y);
    a = fmaf(-z, s.c_low, a);
  } else {
    const float d = s.max - z, b = d - s.max, e = (s.max - (d - b)) + (-z - b);  // d + e = max - z
    y = fmaf(d, s.c, kRound);
    a = fmaf(d, s.c, kRound - y);
    a = fmaf(d, s.c_low, a);
    a = fmaf(e, s.c, a);
  }
  // 2^(-a/32) - 1
  constexpr float x = 0.0216608493924982909f;  // ln 2 / 32
  q = a * (-x + a * (x * x / 2 + a * (-x * x * x / 6 + a * (x * x * x * x / 24))));
  return y < kRound + kTail ? __float_as_int(y) - 0x4b400000 : kTail;
}
// A number below 1 as a part of 2^64 (below 2^-32 its last bits go).
MDEV uint64_t share_of(float x) { return (uint64_t)(x * 16777216.f * 4294967296.f) << 8; }
// Adds the weight, rounded, to a sum in units of 2^-kUnit.  Whole warps call it; lane
// j holds 2^(31 - j/32).
MDEV void add_weight(uint64_t& sum, uint32_t power, bool on, int k, float q) {
  const uint32_t p = __shfl_sync(0xffffffffu, power, k & 31);
  const float pf = __uint_as_float(((p + 64) >> 7) + (0x4e800000u - (1u << 23)));  // 2^30 < p <= 2^31
  const uint32_t w = p + (uint32_t)__float2int_rn(q * pf);                  // units of 2^-31
  const int down = (k >> 5) - (kUnit - 31);
  uint32_t half;  // 2^(down - 1), 0 where nothing is cut off: shifts past 31 give 0
  asm("shl.b32 %0, 1, %1;" : "=r"(half) : "r"(down - 1));
  const uint32_t m = on ? __funnelshift_rc(w + half, 0u, (uint32_t)max(down, 0)) : 0u;
  sum += (uint64_t)m * (1u << max(-down, 0));
}

// Where the mark lies: the bin, the tokens and the sum of weights before and in it.
struct Found {
  uint64_t bin, count, before, mark;  // tokens in the bin; count or sum before it
};

template <int CL>
struct alignas(16) Smem {
  uint32_t hist[3][kBins];  // count, and the sums of the low and high bits of q
  uint32_t powers[32];
  uint64_t warp[kWarps];
  uint64_t loaded[kWarps];  // barriers: a warp's logits are there
  uint64_t row_best[CL], slice[CL], kept_m[CL];  // a word of each CTA of the cluster, which writes it
  uint32_t row_count[CL], kept_n[CL], listed_by[CL], first_by[CL], warp_n[kWarps], warp_first[kWarps];
  uint32_t listed;
  Found found;
  float c, c_low;
  double min_gap;  // T log min_p
  uint64_t start, mark;
  int owner, chosen, last;
};

template <int CL>
MDEV void sync_all() {
  if constexpr (CL == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    cluster_sync();
  }
}
template <int CL>
MDEV uint32_t peer(const uint32_t* p, int r) {
  if constexpr (CL == 1) {
    return *p;
  } else {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(cluster_map(smem_u32(p), (uint32_t)r)) : "memory");
    return v;
  }
}
MDEV uint64_t ld_cluster_u64(const uint64_t* p, int r) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];\n" : "=l"(v) : "r"(cluster_map(smem_u32(p), (uint32_t)r)) : "memory");
  return v;
}
// This CTA's word into every CTA's array (lanes 0 .. CL-1 of a warp call it); seen
// after the next sync_all.
template <int CL>
MDEV void tell(uint64_t* words, int lane, int rank, uint64_t v) {
  if constexpr (CL == 1) words[0] = v;
  else st_cluster_u64(words + rank, lane, v);
}
template <int CL>
MDEV void tell(uint32_t* words, int lane, int rank, uint32_t v) {
  if constexpr (CL == 1) words[0] = v;
  else asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(cluster_map(smem_u32(words + rank), (uint32_t)lane)), "r"(v)
                    : "memory");
}

// The sum of n weights of bin k, whose q + bias come to lo + 2^kLowBits hi, in units
// of 2^-kUnit.
MDEV uint64_t bin_mass(const uint32_t* powers, int k, uint64_t n, uint64_t lo, uint64_t hi) {
  if (n == 0 || k == kTail) return 0;
  const int64_t q = (int64_t)(lo + (hi << kLowBits)) - (int64_t)n * kQBias;
  const uint64_t p = powers[k & 31];
  const uint64_t w = p * n + (uint64_t)__mul64hi((int64_t)(p << 31), q * 4);  // units of 2^-31
  return ((w << (kUnit - 31 + 1) >> (k >> 5)) + 1) >> 1;
}

// The bin in which the count of tokens (COUNT) or the sum of their weights, from
// `before` on, reaches the mark.  share > 0: the mark is share / 2^64 of the
// histogram's own sum, rounded up as sums are whole.  hist is this CTA's part of a
// histogram, over k (in < 0) or inside bin `in`, and zeros again after the call.
template <int CL, bool COUNT>
MDEV Found find_bin(Smem<CL>& s, int rank, uint64_t mark, uint64_t share, int in, uint64_t before) {
  constexpr int kOwn = kBins / CL, kPer = kOwn > kThreads ? kOwn / kThreads : 1;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint32_t n[kPer];
  uint64_t m[kPer], mine = 0;  // count or sum of this thread's bins
  sync_all<CL>();
  // this CTA's bins, summed over the cluster
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int bin = rank * kOwn + t * kPer + i;
    n[i] = 0;
    m[i] = 0;
    if (t * kPer >= kOwn) continue;
    uint64_t lo = 0, hi = 0;
    uint32_t v[COUNT ? 1 : 3][CL];  // all loads before the first sum
#pragma unroll
    for (int e = 0; e < (COUNT ? 1 : 3); ++e)
#pragma unroll
      for (int r = 0; r < CL; ++r) v[e][r] = peer<CL>(&s.hist[e][bin], r);
#pragma unroll
    for (int r = 0; r < CL; ++r) {
      n[i] += v[0][r];
      if (!COUNT) {
        lo += v[1][r];
        hi += v[2][r];
      }
    }
    m[i] = COUNT ? n[i] : bin_mass(s.powers, in < 0 ? bin : in, n[i], lo, hi);
    mine += m[i];
  }
  // a scan over the threads
  uint64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t a = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += a;
  }
  const bool some = __any_sync(0xffffffffu, [&] {
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) all |= n[i];
    return all != 0;
  }());
  if (lane == 31) s.warp[warp] = scan << 1 | (some ? 1 : 0);
  __syncthreads();
  if (warp == 0) {
    const uint64_t a0 = lane < kWarps ? s.warp[lane] : 0;
    uint64_t a = a0 >> 1;
    const bool any = __any_sync(0xffffffffu, a0 & 1);
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, a, o);
      if (lane >= o) a += x;
    }
    if (lane < kWarps) s.warp[lane] = a - (a0 >> 1);  // before each warp
    const uint64_t all = __shfl_sync(0xffffffffu, a, kWarps - 1) << 1 | (any ? 1 : 0);
    if (lane < CL) tell<CL>(s.slice, lane, rank, all);
  }
  sync_all<CL>();
  for (int i = t; i < (COUNT ? 1 : 3) * kBins; i += kThreads) s.hist[0][i] = 0;  // everyone has read it
  // the CTA that has the bin: the first whose bins reach the mark, or the last with tokens
  if (warp == 0) {
    const uint64_t a0 = lane < CL ? s.slice[lane] : 0;
    uint64_t a = a0 >> 1;
#pragma unroll
    for (int o = 1; o < CL; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, a, o);
      if (lane >= o) a += x;
    }
    if (share) {
      const uint64_t all = __shfl_sync(0xffffffffu, a, CL - 1);
      mark = __umul64hi(share, all) + (share * all != 0);
    }
    a += before;
    const uint32_t with = __ballot_sync(0xffffffffu, (a0 & 1) != 0);
    const uint32_t hit = __ballot_sync(0xffffffffu, (a0 & 1) && a >= mark);
    if (lane == 0) {
      s.owner = hit ? __ffs(hit) - 1 : 31 - __clz(with);
      s.chosen = 0x7fffffff;
      s.last = -1;
      s.mark = mark;
    }
    if (lane == rank) s.start = a - (a0 >> 1);
  }
  __syncthreads();
  if (rank == s.owner) {
    const uint64_t a0 = s.start + s.warp[warp] + scan - mine;
    mark = s.mark;
    uint64_t a = a0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      a += m[i];
      if (n[i]) {
        atomicMax(&s.last, t * kPer + i);
        if (a >= mark) atomicMin(&s.chosen, t * kPer + i);
      }
    }
    __syncthreads();
    const int pick = s.chosen != 0x7fffffff ? s.chosen : s.last;
    a = a0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (t * kPer + i == pick) {
        const uint64_t out[4] = {(uint64_t)(rank * kOwn + pick), n[i], a, mark};
        uint64_t* dst = &s.found.bin;
#pragma unroll
        for (int r = 0; r < CL; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (CL == 1) dst[e] = out[e];
            else st_cluster_u64(dst + e, r, out[e]);
          }
      }
      a += m[i];
    }
  }
  sync_all<CL>();
  return s.found;
}

// v[0 .. n-1] in rising order, n a power of two, 64 to kShort: a bitonic network, a
// pair per thread.  A warp's pairs at distances up to 32 lie in 64 words of its own.
MDEV void sort(uint64_t* v, int n) {
  const int t = threadIdx.x;
  for (int size = 2; size <= n; size *= 2)
    for (int d = size / 2; d > 0; d /= 2) {
      if (d >= 32) __syncthreads();
      else __syncwarp();
      if (t < n / 2) {
        const int i = t / d * 2 * d + t % d;
        const uint64_t a = v[i], b = v[i + d];
        if ((a > b) == ((i & size) == 0)) {
          v[i] = b;
          v[i + d] = a;
        }
      }
    }
  __syncthreads();
}

// A row's token, from its logits in shared memory.
struct Draw {
  int row, node, rank, t, i0, np, w0, w1;  // places up to np hold tokens i0 + place; this warp's: w0 .. w1
  uint32_t k;                        // top_k, 0: all
  float p, low, u, T;                // low: min_p's least logit
};
template <int CL, bool NEAR>
__device__ __noinline__ void draw(const SampleArgs& a, Smem<CL>& s, float* zs, const Scale sc, const Draw d) {
  const int row = d.row, rank = d.rank, t = d.t, i0 = d.i0, np = d.np, w0 = d.w0, w1 = d.w1;
  const int lane = t & 31, warp = t >> 5;
  const float low = d.low, u = d.u, T0 = d.T, p0 = d.p;
  // log of the share of `total` that a logit with weight w has; near 1 from the rest
  auto log_share = [&](float z, uint64_t w, uint64_t total) {
    if (w >= total - w) return (float)-log1p((double)(total - w) / (double)w);
    const double y = NEAR ? (double)z / (double)T0 - (double)sc.top * (0.69314718055994530942 / 32)
                          : ((double)z - (double)sc.max) / (double)T0;
    return (float)(y - log((double)total * (1.0 / 17592186044416.0)));
  };
  // ---- the cut of top-k, then of top-p: kept are the tokens up to (z_cut, i_cut) in
  // order whose k is at most k_cut
  const uint32_t power = s.powers[lane];
  float z_cut = kLowest;
  int i_cut = kMaxV, k_cut = kTail;
  // top-k and top-p in one CTA, where the tokens of the bins up to `last` (no logit
  // below `down`) are at most kShort: sorted there, cut, sorted by index, and drawn
  // from, with no more barriers of the cluster, whose other CTAs end.  (320 rows of
  // 128257, 200 tokens kept, then 0.8 of them: 291 to 190 us; one row 31 to 23, of
  // 32000 22 to 20.  With one of the two rules, or one CTA to a row, the two sorts
  // take longer than what they save: top-k alone, one row of 32000, 17 us for 14.)
  auto shorten = [&](int last, float down, uint32_t k) {
    uint64_t* mine = reinterpret_cast<uint64_t*>(s.hist[1]);  // zeros, and not in use
#pragma unroll 2
    for (int i = t * 4; i < np; i += kThreads * 4) {
      const float4 v = *reinterpret_cast<const float4*>(zs + i);
      if (!(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= down)) continue;
      const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float q;
        if (!(z[e] >= down) || weight_of<NEAR>(sc, z[e], q) > last) continue;
        mine[min(atomicAdd(&s.listed, 1u), (uint32_t)kShort - 1)] = order_of(z[e], i0 + i + e);
      }
    }
    __syncthreads();
    if (t < CL) tell<CL>(s.listed_by, t, rank, s.listed);
    sync_all<CL>();
    uint32_t n = 0;
#pragma unroll
    for (int r = 0; r < CL; ++r) n += s.listed_by[r];
    uint64_t* list = reinterpret_cast<uint64_t*>(s.hist[0]);
    int size = 64;
    while (size < (int)n) size *= 2;
    if (rank == 0) {
      uint32_t at = 0;
#pragma unroll
      for (int r = 0; r < CL; ++r) {
        for (uint32_t i = t; i < s.listed_by[r]; i += kThreads) list[at + i] = ld_cluster_u64(mine + i, r);
        at += s.listed_by[r];
      }
      for (int i = (int)n + t; i < size; i += kThreads) list[i] = kNone;
    }
    sync_all<CL>();  // the lists have been read
    if (rank != 0) return;
    sort(list, size);
    // two neighbours per thread: their weights, and the sums up to each
    uint64_t* weight = mine;
    uint32_t kept_n = min(k, n);
    auto sums = [&](uint64_t w0, uint64_t w1, uint64_t& up_to0, uint64_t& up_to1) {
      uint64_t x = w0 + w1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s.warp[warp] = x;
      __syncthreads();
      uint64_t v = lane < kWarps ? s.warp[lane] : 0;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      const uint64_t all = __shfl_sync(0xffffffffu, v, kWarps - 1);
      if (warp > 0) x += __shfl_sync(0xffffffffu, v, warp - 1);
      up_to1 = x;
      up_to0 = x - w1;
      return all;
    };
    uint64_t w[2], up_to[2];
    float z[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t i = 2 * t + e;
      const bool on = i < kept_n;
      z[e] = on ? logit_of(list[i]) : -INFINITY;
      float q;
      const int b = weight_of<NEAR>(sc, z[e], q);
      w[e] = 0;
      add_weight(w[e], power, on, b, q);
    }
    if (t == 0) s.listed = kept_n;
    const uint64_t all = sums(w[0], w[1], up_to[0], up_to[1]);
    const uint64_t mark = __umul64hi(share_of(p0), all) + (share_of(p0) * all != 0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t i = 2 * t + e;
      if (i >= kept_n) continue;
      if (up_to[e] >= mark) atomicMin(&s.listed, i + 1);  // the first that reaches it is the last kept
      if (z[e] < low) atomicMin(&s.listed, i);
      weight[i] = w[e];
    }
    __syncthreads();
    kept_n = s.listed;
    // by index
    size = 64;
    while (size < (int)kept_n) size *= 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t i = 2 * t + e;
      if ((int)i < size) list[i] = i < kept_n ? (list[i] & (kMaxV - 1)) << 32 | i : kNone;
    }
    sort(list, size);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t i = 2 * t + e;
      w[e] = i < kept_n ? weight[(uint32_t)list[i]] : 0;
    }
    const uint64_t total = sums(w[0], w[1], up_to[0], up_to[1]);
    const uint64_t at = __umul64hi(share_of(u), total);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t i = 2 * t + e;
      if (i < kept_n && up_to[e] > at && up_to[e] - w[e] <= at) {
        const int token = (int)(list[i] >> 32);
        a.token[row] = token;
        if (a.kept) a.kept[row] = (int)kept_n;
        if (a.logp) a.logp[row] = log_share(a.logits[((int64_t)row * a.T + d.node) * a.V + token], w[e], total);
      }
    }
  };
  // Cuts behind the token in which the mark is reached; `among`: only kept ones count.
  // True: the token is drawn.
  auto narrow = [&](auto by_count, uint64_t mark, uint64_t share, bool among) {
    constexpr bool COUNT = decltype(by_count)::value;
    auto put = [&](int bin, float q) {
      atomicAdd(&s.hist[0][bin], 1u);
      if (!COUNT) {
        const uint32_t w = (uint32_t)(__float2int_rn(q * 2147483648.f) + kQBias);
        atomicAdd(&s.hist[1][bin], w & ((1u << kLowBits) - 1));
        atomicAdd(&s.hist[2][bin], w >> kLowBits);
      }
    };
    auto counts = [&](float z, int i) { return !among || z > z_cut || (z == z_cut && i0 + i <= i_cut); };
#pragma unroll 2
    for (int i = t * 4; i < np; i += kThreads * 4) {
      const float4 v = *reinterpret_cast<const float4*>(zs + i);
      const float z[4] = {v.x, v.y, v.z, v.w};
      if (among && fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < z_cut) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float q;
        const int k = weight_of<NEAR>(sc, z[e], q);
        if (z[e] > -INFINITY && k <= k_cut && counts(z[e], i + e)) put(k, k == kTail ? 0.f : q);
      }
    }
    Found f = find_bin<CL, COUNT>(s, rank, mark, share, -1, 0);
    const int k = (int)f.bin;
    mark = f.mark;
    // every order in the bin: logits further off than any in it
    uint64_t lo, hi;
    {
      const float step = 1.f / sc.c;
      // (NEAR counts bins from a whole number 0.3 to 1.7 above max c)
      const float up = k < 3 ? sc.max : sc.max - ((float)k - 2.5f) * step;
      const float down = k == kTail ? kLowest : sc.max - ((float)k + 1.25f) * step;
      lo = order_of(fminf(up, sc.max), 0);
      hi = order_of(fmaxf(down, kLowest), kMaxV - 1);
      if constexpr (COUNT && CL > 1)
        if (p0 < 1.f && f.before + f.count <= kShort) {
          shorten(k, fmaxf(down, kLowest), d.k);
          return true;
        }
    }
    while (f.count > 1) {
      const int bits = 64 - __clzll((long long)(hi - lo)), shift = max(0, bits - 11);
      const float z_top = logit_of(lo), z_low = logit_of(hi);
      for (int i = t * 4; i < np; i += kThreads * 4) {
        const float4 v = *reinterpret_cast<const float4*>(zs + i);
        const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (z[e] > z_top || z[e] < z_low) continue;
          const uint64_t c = order_of(z[e], i0 + i + e);
          if (c < lo || c > hi || !counts(z[e], i + e)) continue;
          float q;
          if (weight_of<NEAR>(sc, z[e], q) == k) put((int)((c - lo) >> shift), k == kTail ? 0.f : q);
        }
      }
      f = find_bin<CL, COUNT>(s, rank, mark, 0, k, f.before);
      lo += f.bin << shift;
      hi = min(hi, lo + (((uint64_t)1 << shift) - 1));
      if (shift == 0) break;
    }
    // lo .. hi holds one token of bin k, and perhaps some of the bins beside it:
    // those of lower bins come before it, those of higher ones are past k_cut.  (The
    // cut of an earlier call is not undone: a bin of its last token is no further on.)
    const float z = logit_of(hi);
    const int i = (int)(hi & (kMaxV - 1));
    if (z > z_cut || (z == z_cut && i < i_cut)) {
      z_cut = z;
      i_cut = i;
    }
    k_cut = min(k_cut, k);
    return false;
  };
  const bool by_k = d.k > 0;
  if (by_k && narrow(std::true_type(), d.k, 0, false)) return;
  // at p = 0 the sum of no token is enough, and the first one is kept
  if (p0 < 1.f && narrow(std::false_type(), 0, share_of(p0), by_k)) return;
  // ---- the token
  uint64_t sum = 0;
  uint32_t kept = 0;
  auto is_kept = [&](float z, int i) { return z >= low && (z > z_cut || (z == z_cut && i0 + i <= i_cut)); };
  auto add = [&](uint64_t& to, float z, int i) {
    float q;
    const int k = weight_of<NEAR>(sc, z, q);
    const bool on = is_kept(z, i) && k <= k_cut;
    add_weight(to, power, on, k, q);
    return on;
  };
#pragma unroll 2
  for (int i = w0 + lane * 4; i < w1; i += 128) {
    const float4 v = *reinterpret_cast<const float4*>(zs + i);
    if (!__any_sync(0xffffffffu, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= fmaxf(low, z_cut))) continue;
    kept += add(sum, v.x, i);
    kept += add(sum, v.y, i + 1);
    kept += add(sum, v.z, i + 2);
    kept += add(sum, v.w, i + 3);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  kept = __reduce_add_sync(0xffffffffu, kept);
  // u = 0: the first kept token, also where its weight is nothing in the sums' units.
  // (With top-p none weighs so little: up to 2^18 tokens share more than 2^-24 from the
  // last kept one on, and those before it weigh more.)
  if (u == 0.f) {
    const double least = (double)sc.max - (double)T0 * 745.13321910194122;  // the weight is 2^-1075: 0 in 64 bits
    uint32_t first = ~0u;
    for (int i = w0 + lane; i < w1 && first == ~0u; i += 32) {
      float q;
      const uint32_t on = __ballot_sync(
          0xffffffffu, is_kept(zs[i], i) && (zs[i] == sc.max || (double)zs[i] > least) && weight_of<NEAR>(sc, zs[i], q) <= k_cut);
      if (on) first = (uint32_t)(i0 + i - lane + __ffs(on) - 1);
    }
    if (lane == 0) s.warp_first[warp] = first;
  }
  if (lane == 0) {
    s.warp[warp] = sum;
    s.warp_n[warp] = kept;
  }
  __syncthreads();
  uint64_t total = 0, before = lane < kWarps ? s.warp[lane] : 0;  // a lane for each warp's sum
  kept = lane < kWarps ? s.warp_n[lane] : 0;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  const uint64_t own = __shfl_sync(0xffffffffu, before, kWarps - 1);
  before = __shfl_sync(0xffffffffu, before, warp) - sum;
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (t < CL) {
    tell<CL>(s.kept_m, t, rank, own);
    tell<CL>(s.kept_n, t, rank, kept);
  }
  if (u == 0.f && warp == 0) {
    const uint32_t least = __reduce_min_sync(0xffffffffu, lane < kWarps ? s.warp_first[lane] : ~0u);
    if (lane < CL) tell<CL>(s.first_by, lane, rank, least);
  }
  sync_all<CL>();  // the last words that CTAs exchange
  kept = 0;
#pragma unroll
  for (int r = 0; r < CL; ++r) {
    if (r < rank) before += s.kept_m[r];
    total += s.kept_m[r];
    kept += s.kept_n[r];
  }
  if (u == 0.f) {
    uint32_t least = ~0u;
#pragma unroll
    for (int r = 0; r < CL; ++r) least = min(least, s.first_by[r]);
    if (s.warp_first[warp] != least) return;  // the token is not this warp's
    const int i = (int)least - i0;
    uint64_t w = 0;
    add(w, zs[i], i);
    if (lane == 0) {
      a.token[row] = (int)least;
      if (a.kept) a.kept[row] = (int)kept;
      if (a.logp) a.logp[row] = log_share(zs[i], w, total);
    }
    return;
  }
  const uint64_t mark = __umul64hi(share_of(u), total);
  if (sum == 0 || before > mark || before + sum <= mark) return;
  for (int i = w0 + lane * 4; i < w1; i += 128) {  // this warp's tokens pass the mark
    uint64_t x[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      add(x[e], zs[i + e], i + e);
      if (e > 0) x[e] += x[e - 1];
    }
    uint64_t scan = x[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + scan > mark);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        before += scan - x[3];
        const int e = before + x[0] > mark ? 0 : before + x[1] > mark ? 1 : before + x[2] > mark ? 2 : 3;
        a.token[row] = i0 + i + e;
        if (a.kept) a.kept[row] = (int)kept;
        if (a.logp)
          a.logp[row] = log_share(zs[i + e], x[e] - (e > 0 ? x[e - 1] : 0), total);
      }
      return;
    }
    before += __shfl_sync(0xffffffffu, scan, 31);
  }
}

template <int CL>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<CL>& s = *reinterpret_cast<Smem<CL>*>(smem_raw);
  float* zs = reinterpret_cast<float*>(smem_raw + sizeof(Smem<CL>));  // this CTA's logits
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int row = blockIdx.x / CL, rank = CL == 1 ? 0 : (int)cluster_rank();
  if constexpr (CL > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  const float T0 = a.temperature ? a.temperature[row] : 1.f;
  const int k0 = a.top_k ? a.top_k[row] : 0;
  const float p0 = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.uniforms[row];
  const int node = a.node ? a.node[row] : 0;
  int bad = 0;
  if (!(T0 >= 0.f && T0 < INFINITY) || !(p0 >= 0.f && p0 <= 1.f) || !(mp >= 0.f && mp <= 1.f) || !(u >= 0.f && u < 1.f))
    bad = MEDUSA_DEVERR_TOKEN;
  if ((unsigned)node >= (unsigned)a.T) bad |= MEDUSA_DEVERR_NODE;
  // ---- the row into shared memory; its first token in order, and how many it has.
  // A warp copies and looks through the places of its own.  Places begin at the
  // 16-byte boundary at or before this CTA's first logit; those without one hold
  // minus infinity.
  const float* src = a.logits + ((int64_t)row * a.T + (bad ? 0 : node)) * a.V + rank * a.slice;
  const int lead = (int)(reinterpret_cast<uintptr_t>(src) / 4 & 3), i0 = rank * a.slice - lead;
  const int n = lead + max(0, min(a.V - rank * a.slice, a.slice)), np = (n + 127) & ~127;
  const int per = (((n + kWarps - 1) / kWarps) + 127) & ~127;
  const int w0 = min(np, warp * per), w1 = min(np, w0 + per);
  uint64_t best = kNone;
  uint32_t count = 0;
  if (!bad) {
    const int c0 = max(w0, lead > 0 ? 4 : 0), c1 = min(w1, n) & ~3;  // in whole 16 bytes
    if (lane == 0 && c0 < c1) {
      sm100::mbar_init(&s.loaded[warp], 1);
      sm100::fence_barrier_init();
      sm100::mbar_expect_tx(&s.loaded[warp], (c1 - c0) * 4);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                       smem_u32(zs + c0)),
                   "l"(src + (c0 - lead)), "r"((c1 - c0) * 4), "r"(smem_u32(&s.loaded[warp]))
                   : "memory");
    }
    for (int i = w0 + lane; i < w1; i += 32)
      if (i < c0 || i >= c1) zs[i] = i >= lead && i < n ? __ldg(src + (i - lead)) : -INFINITY;
  }
  for (int i = t; i < 3 * kBins; i += kThreads) s.hist[0][i] = 0;
  if (t == 0) s.listed = 0;
  if (t < 32) s.powers[t] = kPowers[t];
  // 64-bit arithmetic is slow: two threads', while the logits come
  if (t == kThreads - 33 && mp > 0.f) s.min_gap = (double)T0 * log((double)mp);
  if (t == kThreads - 1 && T0 > 0.f) {
    const double c = fmin(32.0 / ((double)T0 * 0.693147180559945309417), 1e38);
    s.c = (float)c;
    s.c_low = (float)(c - (double)s.c);
  }
  __syncwarp();
  if (!bad) {
    if ((min(w1, n) & ~3) > max(w0, lead > 0 ? 4 : 0) && !sm100::mbar_wait(&s.loaded[warp], 0)) {
      set_err(a.err, MEDUSA_DEVERR_TIMEOUT);
      best = 0;
      sm100::mbar_wait(&s.loaded[warp], 0);  // the copy lands before the CTA ends
    }
    bool wrong = best == 0;
    int at_top = 0;
    float top = -INFINITY;
#pragma unroll 2
    for (int i = w0 + lane * 4; i < w1; i += 128) {
      const float4 v = *reinterpret_cast<const float4*>(zs + i);
      const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wrong |= !(z[e] < INFINITY);
        count += z[e] > -INFINITY;
        if (z[e] > top) {
          top = z[e];
          at_top = i + e;
        }
      }
    }
    if (top > -INFINITY) best = order_of(top, i0 + at_top);
    if (wrong) best = 0;  // before any order of a number
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) {
    s.warp[warp] = best;
    s.warp_n[warp] = count;
  }
  __syncwarp();
  // the others have begun: their shared memory may be written
  if constexpr (CL > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  __syncthreads();
  if (warp == 0) {
    best = lane < kWarps ? s.warp[lane] : kNone;
    count = lane < kWarps ? s.warp_n[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane < CL) {
      tell<CL>(s.row_best, lane, rank, best);
      tell<CL>(s.row_count, lane, rank, count);
    }
  }
  sync_all<CL>();
  best = kNone;
  count = 0;
#pragma unroll
  for (int r = 0; r < CL; ++r) {
    best = min(best, s.row_best[r]);
    count += s.row_count[r];
  }
  if (!bad && (best == 0 || best == kNone)) bad = MEDUSA_DEVERR_TOKEN;
  const uint32_t k_mark = k0 > 0 && (uint32_t)k0 < count ? (uint32_t)k0 : count;
  if (bad || T0 == 0.f || k_mark == 1) {
    if (rank == 0 && t == 0) {
      a.token[row] = bad ? -1 : (int)(best & (kMaxV - 1));
      if (a.logp) a.logp[row] = bad ? -INFINITY : 0.f;
      if (a.kept) a.kept[row] = bad ? 0 : 1;
      if (bad) set_err(a.err, bad);
    }
    return;  // the whole cluster
  }
  const float row_max = logit_of(best), top = row_max * s.c;
  const bool near = fabsf(top) < 2097152.f;
  const Scale sc{row_max, s.c, s.c_low, near ? rintf(top) + 1.f : 0.f};
  float low = kLowest;  // min_p's least logit: the least float at or above max + T log min_p
  if (mp > 0.f) {
    const double z = (double)sc.max + s.min_gap;
    low = fmaxf((float)z, kLowest);
    if ((double)low < z) low = nextafterf(low, INFINITY);
  }
  const Draw d{row, node, rank, t, i0, np, w0, w1, k_mark < count ? k_mark : 0u, p0, low, u, T0};
  if (near) draw<CL, true>(a, s, zs, sc, d);
  else draw<CL, false>(a, s, zs, sc, d);
}

template <int CL>
int run(const SampleArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const size_t most = 227 * 1024, smem = sizeof(Smem<CL>) + (size_t)((a.slice + 3 + 127) & ~127) * 4;
  auto* fn = sample_kernel<CL>;
  if (int rc = prepare_kernel(reinterpret_cast<const void*>(fn), most, 0, 0, &done, "medusa_sample")) return rc;
  if (CL == 1) launch_kernel(fn, dim3(a.R), dim3(kThreads), smem, stream, a);
  else launch_cluster(fn, CL, dim3(a.R * CL), dim3(kThreads), smem, stream, a);
  return check_launch("medusa_sample");
}

// CTAs for a row: few, as each adds barriers to wait at, but enough that the row
// fits them (kMost logits each, so that an SM has two CTAs), and that the CTAs of a
// call with few rows have at least kLeast each to share the SMs with.
constexpr int kMost = 16384, kLeast = 4096;
int cluster_for(int R, int V, int sms) {
  int cl = 1;
  while (cl < 8 && (V > cl * kMost || (V > cl * kLeast && (int64_t)R * cl * 2 <= sms))) cl *= 2;
  return cl;
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" int medusa_sample(const float* logits, int T, const int32_t* node, int R, int V, const float* temperature,
                             const int32_t* top_k, const float* top_p, const float* min_p, const float* uniforms,
                             int32_t* token, float* logp, int32_t* kept, int32_t* err, void* stream) {
  const char* fn = "medusa_sample";
  if (T < 1 || R < 0 || V < 1) return fail(MEDUSA_ERR_INVALID, "%s: T=%d R=%d V=%d", fn, T, R, V);
  if (V > kMaxV || R > (1 << 24)) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: V=%d (at most %d) R=%d", fn, V, kMaxV, R);
  if (R == 0) return MEDUSA_OK;
  if (!logits || !uniforms || !token) return fail(MEDUSA_ERR_INVALID, "%s: NULL tensor", fn);
  if (reinterpret_cast<uintptr_t>(logits) % 4) return fail(MEDUSA_ERR_INVALID, "%s: logits not 4-byte aligned", fn);
  SampleArgs a{logits, node, T, R, V, 0, temperature, top_k, top_p, min_p, uniforms, token, logp, kept, err};
  const int cl = cluster_for(R, V, sm_count());
  a.slice = (V + cl - 1) / cl;
  cudaStream_t st = as_stream(stream);
  return cl == 1 ? run<1>(a, st) : cl == 2 ? run<2>(a, st) : cl == 4 ? run<4>(a, st) : run<8>(a, st);
}

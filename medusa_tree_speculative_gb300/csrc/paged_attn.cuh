// Chunk attention over the paged cache: what its kernels share.
//
// Work is cut into units (sequence, key head, block of query rows).  The g =
// H / Hkv query heads of a key head are rows of one matrix: row r of a
// sequence's key head is token r / g, head r % g, and a block holds whole
// tokens (RB / g of them), so that one pass over the keys serves all g heads.
// A unit reads the key tiles its last token sees.  All units' tiles, in the
// order (sequence, key head, block, tile), form one list, in which each unit
// also has `EC` empty places before its first tile, for the time that
// beginning and ending a unit takes.  The grid's CTAs share the list's N
// places out evenly: CTA c of G takes [c N / G, (c + 1) N / G).  So ragged
// batches, one long sequence and a causal triangle are balanced alike, and
// nothing about the lengths is needed on the host.  (Without the empty places
// the CTAs with a causal triangle's short units ran a third longer than the
// mean.)  A unit that several
// CTAs share is joined by the last of them to finish (an arrival counter);
// every partial goes through the workspace and is added in CTA order, whoever
// adds it, so the result does not depend on timing.
#pragma once

#include <stdint.h>

#include <cuda.h>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "sm100.cuh"

namespace medusa {

constexpr int kPagedMaxGroup = 64;     // query heads per key head
constexpr int kFewRows = 16;           // rows (tokens x heads of a key head) of the kernels for few rows
constexpr int kPagedCounters = 1024;   // arrival counters of one kernel
constexpr float kPagedLog2e = 1.4426950408889634f;

struct PagedAttnArgs {
  const void* q;
  const void* k_new;
  const void* v_new;
  int64_t q_stride, k_stride, v_stride;
  void* k_pages;
  void* v_pages;
  PagesDev p;
  const int32_t* rows;
  const int32_t* q_start;
  int B, total_q, max_new;
  int T, W, K;  // tree rows (0: causal), mask words per row, depth
  const int32_t* depth;
  const uint32_t* anc;
  int H, Hkv, g;
  uint64_t turns[64];  // theta^(-2j/Dh) / (2 pi) as a fraction of 2^64
  float qscale;        // scale * log2(e)
  void* out;
  void* q_rot;         // [Hkv][total_q * g][Dh]: rotated queries times qscale
  int64_t q_low;       // bf16: elements from q_rot to what its rounding left, rounded
  int* counters;
  float* part;         // two partials per CTA: RB rows of Dh sums, then RB (max, sum) pairs
  int32_t* err;
};

// Sequence b: its row, tokens and prefix; false (and an error code, 0 where it
// merely has no tokens) if it is skipped.
// Where q_start decreases at any sequence, the tokens of the others are no longer
// their own either, and the whole call is refused: `starts_decrease`.
struct SeqInfo {
  int row, q0, n, L;
};
MDEV bool starts_decrease(const PagedAttnArgs& a, int b) { return a.q_start[b + 1] < a.q_start[b]; }
MDEV bool seq_info(const PagedAttnArgs& a, int b, SeqInfo& s, int& code) {
  code = 0;
  s.q0 = a.q_start[b];
  const int q1 = a.q_start[b + 1];
  s.row = a.rows ? a.rows[b] : b;
  s.n = 0;
  s.L = 0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > a.total_q || q1 - s.q0 > a.max_new || (a.T && q1 != s.q0 && q1 - s.q0 != a.T)) {
    code = MEDUSA_DEVERR_LENGTH;
    return false;
  }
  if ((unsigned)s.row >= (unsigned)a.p.rows) {
    code = MEDUSA_DEVERR_ROW;
    return false;
  }
  s.n = q1 - s.q0;
  s.L = a.p.length[s.row];
  const int held = a.p.held[s.row];
  if (!row_state_ok(a.p, s.L, held)) code = MEDUSA_DEVERR_PAGE;
  else if ((int64_t)s.L + s.n > (int64_t)held * a.p.page_size) code = MEDUSA_DEVERR_CAPACITY;
  return code == 0 && s.n > 0;
}

// Key tiles of block u (tb tokens per block) of a sequence.
template <int KT>
MDEV int unit_tiles(const PagedAttnArgs& a, const SeqInfo& s, int tb, int u) {
  const int seen = a.T ? s.n : min(s.n, (u + 1) * tb);
  return (s.L + seen + KT - 1) / KT;
}
// Places of blocks 0 .. u-1, all of them full: u EC and the sum over i of
// floor((L + (i + 1) tb + KT - 1) / KT), by Euclid's reduction of the sum of
// floor((A i + C) / M) (lattice points below a line).
template <int KT, int EC>
MDEV int64_t places_before(const PagedAttnArgs& a, const SeqInfo& s, int tb, int u) {
  if (u <= 0) return 0;
  if (a.T) return (int64_t)u * ((s.L + s.n + KT - 1) / KT + EC);
  uint64_t n = (uint64_t)u, m = KT, x = (uint64_t)tb, c = (uint64_t)s.L + tb + KT - 1;
  int64_t sum = (int64_t)u * EC;
  while (true) {
    sum += (int64_t)((n - 1) * n / 2 * (x / m));
    x %= m;
    sum += (int64_t)(n * (c / m));
    c %= m;
    const uint64_t y = x * n + c;
    if (y < m) break;
    n = y / m;
    c = y % m;
    const uint64_t t = m;
    m = x;
    x = t;
  }
  return sum;
}
// Places of one key head of a sequence.
template <int KT, int EC>
MDEV int64_t seq_places(const PagedAttnArgs& a, const SeqInfo& s, int tb) {
  const int m = (s.n + tb - 1) / tb;
  return places_before<KT, EC>(a, s, tb, m - 1) + EC + unit_tiles<KT>(a, s, tb, m - 1);
}

// Shared memory for the plan: scratch, used only while it is made, and what
// stays.
struct PlanScratch {
  int owner[MEDUSA_MAX_ROWS];        // cache row -> the first entry that names it
  int64_t pre[MEDUSA_MAX_ROWS + 1];  // places before each sequence
  int64_t warp_sum[32];
};
struct Plan {
  uint32_t valid[MEDUSA_MAX_ROWS / 32];  // the sequences that are not skipped
  int64_t total;                         // places in all (negative: refused)
};

// Where in the list a CTA stands: a unit and the tiles of it that are its own.
struct Segment {
  SeqInfo s;
  int b, head, u, m, tiles;  // m blocks; tiles of this unit
  int t0, t1;                // t0 < t1: there are no segments without tiles
  int64_t unit_x;            // the unit's first place in the list
};

// Build the plan (all NT threads of the CTA); x0, x1: this CTA's places.
template <int NT, int RB, int KT, int EC>
MDEV void make_plan(const PagedAttnArgs& a, PlanScratch& sc, Plan& pl, int64_t& x0, int64_t& x1) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int tb = RB / a.g;
  if (a.rows) {
    for (int r = t; r < a.p.rows; r += NT) sc.owner[r] = 0x7fffffff;
  }
  for (int w = t; w < MEDUSA_MAX_ROWS / 32; w += NT) pl.valid[w] = 0u;
  __syncthreads();
  if (a.rows) {
    for (int b = t; b < a.B; b += NT) {
      const int r = a.rows[b];
      if ((unsigned)r < (unsigned)a.p.rows && a.q_start[b + 1] > a.q_start[b]) atomicMin(&sc.owner[r], b);
    }
    __syncthreads();
  }
  const int per = (a.B + NT - 1) / NT;
  int64_t mine = 0;
  for (int k = 0; k < per; ++k) {
    const int b = t * per + k;
    if (b >= a.B) break;
    SeqInfo s;
    int code;
    bool ok = seq_info(a, b, s, code);
    if (ok && a.rows && sc.owner[s.row] != b) {
      ok = false;
      code = MEDUSA_DEVERR_ROW;
    }
    if (code && blockIdx.x == 0) set_err(a.err, code);
    sc.pre[b] = mine;
    if (ok) {
      atomicOr(&pl.valid[b >> 5], 1u << (b & 31));
      mine += (int64_t)a.Hkv * seq_places<KT, EC>(a, s, tb);
    }
    if (starts_decrease(a, b)) mine -= 1ll << 52;  // the call is refused: no places are as many, the sum is negative
  }
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sc.warp_sum[warp] = x;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    const int64_t v = sc.warp_sum[w];
    if (w < warp) before += v;
    total += v;
  }
  before += x - mine;
  for (int k = 0; k < per; ++k) {
    const int b = t * per + k;
    if (b < a.B) sc.pre[b] += before;
  }
  if (t == 0) {
    sc.pre[a.B] = total;
    pl.total = total;
  }
  __syncthreads();
  const int64_t G = min((int64_t)gridDim.x, total);
  if ((int64_t)blockIdx.x < G) {
    x0 = (int64_t)blockIdx.x * total / G;
    x1 = ((int64_t)blockIdx.x + 1) * total / G;
  } else {
    x0 = x1 = 0;
  }
}

// The tiles of unit g in places [x, x1) of the list; false if there are none.
template <int EC>
MDEV bool set_tiles(Segment& g, int64_t x, int64_t x1) {
  const int64_t tile0 = g.unit_x + EC;
  g.t0 = (int)max((int64_t)0, x - tile0);
  g.t1 = (int)min((int64_t)g.tiles, x1 - tile0);
  return g.t0 < g.t1;
}

// The segment that place x of the list is in (x < x1); false if [x, x1) has no
// tiles.  Whole warps call it: a lane per block tried (a search by halves, each
// step an Euclid of 64-bit divisions, took 8 us for 128 blocks).
template <int RB, int KT, int EC>
MDEV bool seek_segment(const PagedAttnArgs& a, const PlanScratch& sc, int64_t x, int64_t x1, Segment& g) {
  const int tb = RB / a.g, lane = threadIdx.x & 31;
  int lo = 0, hi = a.B - 1;  // the last sequence that starts at or before x: it has places, or total would be x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sc.pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  g.b = lo;
  int code;
  seq_info(a, lo, g.s, code);
  g.m = (g.s.n + tb - 1) / tb;
  const int64_t each = (sc.pre[lo + 1] - sc.pre[lo]) / a.Hkv;
  int64_t rest = x - sc.pre[lo], before = 0;
  g.head = (int)(rest / each);
  rest -= (int64_t)g.head * each;
  int u = 0, last = g.m - 1;  // the last block that starts at or before `rest`
  while (u < last) {
    const int step = (last - u + 31) >> 5, v = u + (lane + 1) * step;
    int64_t at = 0;
    if (v <= last) at = places_before<KT, EC>(a, g.s, tb, v);
    const int k = __popc(__ballot_sync(0xffffffffu, v <= last && at <= rest));
    if (k > 0) before = __shfl_sync(0xffffffffu, at, k - 1);
    u += k * step;
    last = min(last, u + step - 1);
  }
  g.u = u;
  rest -= before;
  g.tiles = unit_tiles<KT>(a, g.s, tb, u);
  g.unit_x = x - rest;
  return set_tiles<EC>(g, x, x1);
}

// The segment after g; false if this CTA's places before x1 have none.
template <int RB, int KT, int EC>
MDEV bool next_segment(const PagedAttnArgs& a, const Plan& pl, int64_t x1, Segment& g) {
  const int tb = RB / a.g;
  g.unit_x += g.tiles + EC;
  if (g.unit_x >= x1) return false;
  if (++g.u == g.m) {
    g.u = 0;
    if (++g.head == a.Hkv) {
      g.head = 0;
      do ++g.b; while (g.b < a.B && !(pl.valid[g.b >> 5] >> (g.b & 31) & 1u));
      if (g.b >= a.B) return false;  // not reached: unit_x < x1 <= total
      int code;
      seq_info(a, g.b, g.s, code);
      g.m = (g.s.n + tb - 1) / tb;
    }
  }
  g.tiles = unit_tiles<KT>(a, g.s, tb, g.u);
  return set_tiles<EC>(g, g.unit_x, x1);
}

// CTA that holds place x of the list.
MDEV int cta_of(int64_t x, int64_t total, int64_t G) { return (int)(((x + 1) * G - 1) / total); }

// Who shares the unit of g: its first and last CTA.
template <int EC>
MDEV void unit_shares(const Segment& g, int64_t total, int64_t G, int& first, int& last) {
  first = cta_of(g.unit_x + EC, total, G);
  last = cta_of(g.unit_x + EC + g.tiles - 1, total, G);
}
// Slot (of two) of CTA c's partial of the unit that starts at unit_x: 0 if it
// is the CTA's first segment, else 1 (a CTA that starts in an earlier unit has
// that one's last tile).
MDEV int part_slot(int64_t unit_x, int c, int64_t total, int64_t G) {
  const int64_t x0 = (int64_t)c * total / G;
  return 2 * c + (x0 >= unit_x ? 0 : 1);
}

// Whether token i of the sequence sees key x.
MDEV bool key_seen(const PagedAttnArgs& a, const SeqInfo& s, int i, int x) {
  if (a.T == 0) return x <= s.L + i;
  const int node = x - s.L;
  if (node < 0) return true;
  return node < a.T && (__ldg(a.anc + (int64_t)i * a.W + (node >> 5)) >> (node & 31) & 1u);
}

// The page of key x of a row, or -1 (and MEDUSA_DEVERR_PAGE) where the table
// names none.  x must lie in a held page.
MDEV int page_of(const PagedAttnArgs& a, const SeqInfo& s, int x) {
  const int page = a.p.table[(int64_t)s.row * a.p.max_pages + (x >> a.p.shift)];
  if (page_ok(a.p, page)) return page;
  set_err(a.err, MEDUSA_DEVERR_PAGE);
  return -1;
}

// Wait for a barrier's phase.  After kSpinLimit polls, or once another thread
// of the CTA has given up, it returns all the same: the caller goes on, through
// every barrier as ever, on whatever data there are, and the kernel's end
// reports MEDUSA_DEVERR_TIMEOUT.
MDEV void paged_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  for (uint32_t i = 0; i < sm100::kSpinLimit; ++i) {
    if (sm100::mbar_try_wait(bar, parity)) return;
    if ((i & 63) == 63 && *abort_flag) return;
  }
  *abort_flag = 1;
}

// Host side: launches of the kernels (paged_attn.cu picks).
struct PagedKernels {
  cudaStream_t stream;
  int sms;
};
int launch_paged_prep(const PagedAttnArgs& a, int Dh, medusa_dtype dtype, const PagedKernels& k);
// Rows of Dh bf16 (a pool's lines) in boxes of `box` rows x 64 values, 128-byte
// swizzle; rows past the last read zeros.
bool make_rows_map(CUtensorMap* m, const void* base, int64_t rows, int Dh, int box);
inline bool make_pool_map(CUtensorMap* m, const void* pool, const PagedAttnArgs& a, int Dh, int box) {
  return make_rows_map(m, pool, (int64_t)a.p.num_pages * a.Hkv * a.p.page_size, Dh, box);
}
// The same in boxes of all halves: [Dh / 64][box rows][64 values].
bool make_lines_map(CUtensorMap* m, const void* base, int64_t rows, int Dh, int box);
size_t paged_decode_part_bytes(int Dh, int sms);
int launch_paged_decode(const PagedAttnArgs& a, int Dh, const PagedKernels& k);
size_t paged_chunk_part_bytes(int Dh, int sms);
int launch_paged_chunk(const PagedAttnArgs& a, int Dh, const PagedKernels& k);
int launch_paged_generic(const PagedAttnArgs& a, int Dh, bool few_rows, const PagedKernels& k);

}  // namespace medusa

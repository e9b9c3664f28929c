// Pages of a paged key/value cache: reserve, fork, free, commit, compact and
// copy.
//
// A free page has no references; free_bits holds the same fact as one bit per
// page, so that finding the lowest free pages reads 1/32 of a word per page.
// Every call is deterministic: reference counts and bits change by commutative
// atomics only, pages are handed out lowest first, and lists are in row or
// page order.
//
// reserve and compact need one prefix sum over the whole bit map, which one CTA
// of 1024 threads takes (65536 pages are 2048 words, two per thread): what
// bounds it is the latency of a few dependent loads and block barriers, not
// bytes (compact's plan 5 us).  reserve hands out its few pages there as well
// (15 us for 420 rows); compact leaves table, counts and list to all SMs (7 us).
// fork and free run a CTA per row (7 to 8 us for 256 and 420 rows).  copy moves 16
// bytes per thread, eight loads in flight, and is bound by memory: 16384 pages
// of 64 KB in 321 us, 6.7 TB/s.
#include "internal.h"
#include "paged.cuh"

namespace medusa {
namespace {

constexpr int kBlock = 1024;
constexpr int kNone = 0x7fffffff;

// Exclusive sum over the block (kBlock threads) and the block's total.
MDEV uint64_t block_exclusive_sum(uint64_t v, uint64_t* warp_sums, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous call's readers are done with warp_sums
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const uint64_t w = warp_sums[lane];
    uint64_t z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    warp_sums[lane] = z - w;
    if (lane == 31) warp_sums[32] = z;
  }
  __syncthreads();
  total = warp_sums[32];
  return warp_sums[warp] + x - v;
}

// Bits of word w that stand for pages below num_pages.
MDEV uint32_t live_word_mask(int w, int num_pages) {
  const int left = num_pages - w * 32;
  return left >= 32 ? 0xffffffffu : (1u << left) - 1u;
}

__global__ void __launch_bounds__(256) pages_init_kernel(PagesDev p) {
  const int64_t n = (int64_t)gridDim.x * blockDim.x, i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int words = (p.num_pages + 31) / 32;
  for (int64_t i = i0; i < p.num_pages; i += n) p.refs[i] = 0;
  for (int64_t i = i0; i < words; i += n) p.free_bits[i] = live_word_mask((int)i, p.num_pages);
  for (int64_t i = i0; i < p.rows; i += n) p.length[i] = p.held[i] = 0;
  for (int64_t i = i0; i < (int64_t)p.rows * p.max_pages; i += n) p.table[i] = -1;
}

// One CTA per row.
__global__ void __launch_bounds__(128) pages_free_kernel(PagesDev p, const int32_t* keep_len, int32_t* err) {
  const int r = blockIdx.x, keep = keep_len[r];
  if (keep < 0) return;
  const int len = p.length[r], held = p.held[r];
  if (!row_state_ok(p, len, held)) {
    if (threadIdx.x == 0) set_err(err, MEDUSA_DEVERR_PAGE);
    return;
  }
  __syncthreads();  // every thread has read the row's state
  const int len1 = min(len, keep), held1 = (len1 + p.page_size - 1) >> p.shift;
  int32_t* row = p.table + (int64_t)r * p.max_pages;
  for (int c = held1 + threadIdx.x; c < held; c += blockDim.x) {
    const int page = row[c];
    row[c] = -1;
    if (!page_ok(p, page)) {
      set_err(err, MEDUSA_DEVERR_PAGE);
      continue;
    }
    const int old = atomicSub(p.refs + page, 1);
    if (old == 1) {
      atomicOr(p.free_bits + (page >> 5), 1u << (page & 31));
    } else if (old < 1) {  // not a held page: put the count back
      atomicAdd(p.refs + page, 1);
      set_err(err, MEDUSA_DEVERR_PAGE);
    }
  }
  if (threadIdx.x == 0) {
    p.length[r] = len1;
    p.held[r] = held1;
  }
}

// One CTA per (source, destination) pair.
__global__ void __launch_bounds__(128) pages_fork_kernel(PagesDev p, const int32_t* src, const int32_t* dst, int n,
                                                         int32_t* err) {
  const int i = blockIdx.x, s = src[i], d = dst[i];
  bool bad = (unsigned)s >= (unsigned)p.rows || (unsigned)d >= (unsigned)p.rows;
  // a destination named before, or a row that is source and destination
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int dj = dst[j];
    bad |= (j < i && dj == d) || dj == s || src[j] == d;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_err(err, MEDUSA_DEVERR_ROW);
    return;
  }
  const int len = p.length[s], held = p.held[s], np = (len + p.page_size - 1) >> p.shift;
  const bool taken = p.length[d] != 0 || p.held[d] != 0;
  if (taken || !row_state_ok(p, len, held)) {
    if (threadIdx.x == 0) set_err(err, taken ? MEDUSA_DEVERR_ROW : MEDUSA_DEVERR_PAGE);
    return;
  }
  __syncthreads();  // every thread has read the rows' state
  const int32_t* from = p.table + (int64_t)s * p.max_pages;
  int32_t* to = p.table + (int64_t)d * p.max_pages;
  for (int c = threadIdx.x; c < np; c += blockDim.x) {
    int page = from[c];
    if (page_ok(p, page) && atomicAdd(p.refs + page, 1) < 1) {  // not a held page: put the count back
      atomicSub(p.refs + page, 1);
      page = -1;
    }
    if (!page_ok(p, page)) {
      set_err(err, MEDUSA_DEVERR_PAGE);
      page = -1;
    }
    to[c] = page;
  }
  if (threadIdx.x == 0) {
    p.length[d] = len;
    p.held[d] = np;
  }
}

// One CTA; thread r is row r.
//   1. each row's need (new pages, plus one where its partly filled tail page
//      is shared and it is not the last of the call's sharers to write it),
//      and its place in the row order by one prefix sum;
//   2. the free pages are counted, 32 per word, and numbered from the lowest;
//   3. warps walk the words, a lane per page: the k-th free page goes to the
//      row whose range of places holds k.
__global__ void __launch_bounds__(kBlock) pages_reserve_kernel(PagesDev p, const int32_t* n_new, int32_t* copies,
                                                               int32_t* n_copies, int32_t* granted, int32_t* err) {
  __shared__ uint64_t sums[33];
  __shared__ int tails[kBlock];   // the rows with a shared, partly filled tail page: that page, in row order
  __shared__ int tail_of[kBlock]; // row -> its tail page where it takes a copy, else -1
  __shared__ int lead[kBlock];    // row -> its places among the handed-out pages: [lead, last)
  __shared__ int last[kBlock];
  __shared__ int slot[kBlock];    // row -> its line in `copies`
  __shared__ int base[kBlock];    // word chunk -> free pages before it
  const int t = threadIdx.x;
  const int words = (p.num_pages + 31) / 32, per = (words + kBlock - 1) / kBlock;
  // the free pages of this thread's words
  uint64_t free_here = 0;
  for (int k = 0; k < per; ++k) {
    const int w = t * per + k;
    if (w < words) free_here += __popc(p.free_bits[w] & live_word_mask(w, p.num_pages));
  }
  int n = 0, len = 0, held = 0, more = 0, tail = -1, refs = 0;
  bool bad = false;
  if (t < p.rows) {
    n = n_new[t];
    if (n != 0) {
      len = p.length[t];
      held = p.held[t];
      const int64_t end = (int64_t)len + n;
      int code = 0;
      if (n < 0) code = MEDUSA_DEVERR_LENGTH;
      else if (!row_state_ok(p, len, held)) code = MEDUSA_DEVERR_PAGE;
      else if (end > (int64_t)p.max_pages * p.page_size) code = MEDUSA_DEVERR_CAPACITY;
      else {
        more = max(0, (int)((end + p.page_size - 1) >> p.shift) - held);
        if (len & (p.page_size - 1)) {
          tail = p.table[(int64_t)t * p.max_pages + (len >> p.shift)];
          if (page_ok(p, tail)) refs = p.refs[tail];
          if (refs < 1) code = MEDUSA_DEVERR_PAGE;  // not a held page: it may be handed out
        }
      }
      if (code) {
        set_err(err, code);
        bad = true;
        more = 0;
      }
    }
  }
  const bool shared_tail = !bad && tail >= 0 && refs > 1;
  uint64_t total;
  const uint64_t both = block_exclusive_sum((uint64_t)shared_tail << 32 | free_here, sums, total);
  const int n_free = (int)(uint32_t)total, my = (int)(both >> 32);
  base[t] = (int)(uint32_t)both;
  if (shared_tail) tails[my] = tail;
  __syncthreads();
  // earlier rows of the call with the same tail page: each of them takes a
  // copy until one reference is left
  bool cow = false;
  if (shared_tail) {
    int earlier = 0;
    for (int j = 0; j < my; ++j) earlier += tails[j] == tail;
    cow = refs - earlier > 1;
  }
  const uint64_t need = (uint64_t)(more + (cow ? 1 : 0));
  const uint64_t place = block_exclusive_sum((uint64_t)cow << 48 | need, sums, total);
  const uint64_t first = place & 0xffffffffffffull, upto = first + need;
  const bool fits = upto <= (uint64_t)n_free;
  const bool ok = fits && !bad;
  if (t < p.rows) {
    if (granted) granted[t] = ok;
    if (!fits && n > 0 && !bad) set_err(err, MEDUSA_DEVERR_CAPACITY);
  }
  const int handed = (int)(ok ? need : 0);
  lead[t] = (int)min(first, (uint64_t)kNone);
  last[t] = (int)min(upto, (uint64_t)kNone);
  tail_of[t] = ok && cow ? tail : -1;
  slot[t] = (int)(place >> 48);
  uint64_t counts;
  block_exclusive_sum((uint64_t)(ok && cow) << 32 | (uint64_t)handed, sums, counts);
  const int hand_out = (int)(uint32_t)counts;
  if (t == 0) *n_copies = (int)(counts >> 32);
  if (ok && cow) atomicSub(p.refs + tail, 1);
  if (ok && more > 0) p.held[t] = held + more;
  // hand out: chunk c of `per` words to warp c % 32
  const int lane = t & 31;
  for (int c = t >> 5; c < kBlock && c * per < words; c += 32) {
    int k0 = base[c];
    if (k0 >= hand_out) break;
    for (int k = 0; k < per && c * per + k < words && k0 < hand_out; ++k) {
      const int w = c * per + k;
      const uint32_t bits = p.free_bits[w] & live_word_mask(w, p.num_pages);
      const int place_k = k0 + __popc(bits & ((1u << lane) - 1u));
      const bool mine = (bits >> lane & 1u) && place_k < hand_out;
      if (mine) {
        int lo = 0, hi = p.rows - 1;  // the first row whose range ends past place_k
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (last[mid] > place_k) hi = mid; else lo = mid + 1;
        }
        const int page = w * 32 + lane, src = tail_of[lo], copied = src >= 0 ? 1 : 0;
        const int nth = place_k - lead[lo] - copied;
        const int rlen = p.length[lo];
        int32_t* row = p.table + (int64_t)lo * p.max_pages;
        p.refs[page] = 1;
        if (nth < 0) {  // the tail page's copy
          row[rlen >> p.shift] = page;
          *reinterpret_cast<int4*>(copies + 4 * (int64_t)slot[lo]) =
              make_int4(src, page, rlen & (p.page_size - 1), lo);
        } else {  // the last of the row's range is the last page of its new length
          const int end = (int)(((int64_t)rlen + n_new[lo] + p.page_size - 1) >> p.shift);
          row[end - (last[lo] - lead[lo] - copied) + nth] = page;
        }
      }
      const uint32_t taken = __ballot_sync(0xffffffffu, mine);
      if (lane == 0 && taken) p.free_bits[w] = p.free_bits[w] & ~taken;
      k0 += __popc(bits);
    }
  }
}

__global__ void __launch_bounds__(kBlock) pages_served_kernel(PagesDev p, const int32_t* rows, const int32_t* granted,
                                                              int B, int32_t* served) {
  const int b = threadIdx.x;
  if (b >= B) return;
  const int r = rows ? rows[b] : b;
  served[b] = (unsigned)r < (unsigned)p.rows && granted[r] != 0 ? r : -1;
}

// Thread b is entry b of the batch; a row named twice counts once.
__global__ void __launch_bounds__(kBlock) pages_commit_kernel(PagesDev p, const int32_t* rows, const int32_t* n_new,
                                                              int bias, int B, int32_t* err) {
  __shared__ int owner[MEDUSA_MAX_ROWS];
  const int b = threadIdx.x;
  owner[b] = kNone;
  __syncthreads();
  int r = -1;
  if (b < B) {
    r = rows ? rows[b] : b;
    if ((unsigned)r >= (unsigned)p.rows) {
      set_err(err, MEDUSA_DEVERR_ROW);
      r = -1;
    } else {
      atomicMin(&owner[r], b);
    }
  }
  __syncthreads();
  if (r < 0) return;
  if (owner[r] != b) {
    set_err(err, MEDUSA_DEVERR_ROW);
    return;
  }
  const int n = n_new[b], len = p.length[r], held = p.held[r];
  const int64_t end = (int64_t)len + n + bias;
  if (n < 0) set_err(err, MEDUSA_DEVERR_LENGTH);
  else if (!row_state_ok(p, len, held)) set_err(err, MEDUSA_DEVERR_PAGE);
  else if (end > (int64_t)held * p.page_size) set_err(err, MEDUSA_DEVERR_CAPACITY);
  else p.length[r] = (int)end;
}

// The plan of a compaction, one CTA: with n live pages, the i-th live page at
// or past n goes to the i-th free page below n.  It leaves n (or -1 where
// nothing moves) in work[0], and a PlanWord per word of the bit map at work + 16.
struct alignas(16) PlanWord {
  uint32_t out, hole;            // live pages past n, free pages below n
  int32_t outs_before, holes_before;
};

__global__ void __launch_bounds__(kBlock) pages_plan_kernel(PagesDev p, int max_copies, int32_t* n_copies,
                                                            int32_t* work, int32_t* err) {
  __shared__ uint64_t sums[33];
  const int t = threadIdx.x;
  const int words = (p.num_pages + 31) / 32, per = (words + kBlock - 1) / kBlock;
  uint64_t live = 0, total;
  for (int k = 0; k < per; ++k) {
    const int w = t * per + k;
    if (w < words) live += __popc(~p.free_bits[w] & live_word_mask(w, p.num_pages));
  }
  block_exclusive_sum(live, sums, total);
  const int n = (int)total;
  auto low_mask = [&](int w) {  // bits of word w below page n
    const int left = n - w * 32;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
  };
  auto split = [&](int w, uint32_t& out, uint32_t& hole) {  // live pages >= n, free pages < n
    const uint32_t in = live_word_mask(w, p.num_pages), f = p.free_bits[w], low = low_mask(w);
    out = ~f & in & ~low;
    hole = f & in & low;
  };
  uint64_t mine = 0;
  for (int k = 0; k < per; ++k) {
    const int w = t * per + k;
    if (w >= words) break;
    uint32_t out, hole;
    split(w, out, hole);
    mine += (uint64_t)__popc(out) << 32 | (uint64_t)__popc(hole);
  }
  uint64_t at = block_exclusive_sum(mine, sums, total);
  const int moves = (int)(total >> 32);
  if (moves > max_copies) {  // nothing changes
    if (t == 0) {
      *n_copies = 0;
      work[0] = -1;
      set_err(err, MEDUSA_DEVERR_CAPACITY);
    }
    return;
  }
  PlanWord* plan = reinterpret_cast<PlanWord*>(work + 16);
  for (int k = 0; k < per; ++k) {
    const int w = t * per + k;
    if (w >= words) break;
    PlanWord x;
    split(w, x.out, x.hole);
    x.outs_before = (int)(at >> 32);
    x.holes_before = (int)(uint32_t)at;
    plan[w] = x;
    at += (uint64_t)__popc(x.out) << 32 | (uint64_t)__popc(x.hole);
    p.free_bits[w] = live_word_mask(w, p.num_pages) & ~low_mask(w);
  }
  if (t == 0) {
    *n_copies = moves;
    work[0] = moves > 0 ? n : -1;
  }
}

// The i-th free page below n, from the last word with at most i such pages
// before it.
MDEV int nth_hole(const PlanWord* plan, int words, int i) {
  int lo = 0, hi = words - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (plan[mid].holes_before <= i) lo = mid; else hi = mid - 1;
  }
  uint32_t bits = plan[lo].hole;
  int nth = i - plan[lo].holes_before, at = 0;
#pragma unroll
  for (int half = 16; half > 0; half >>= 1) {  // the nth set bit, by halves
    const int below = __popc(bits & ((1u << half) - 1u));
    if (nth >= below) {
      nth -= below;
      bits >>= half;
      at += half;
    }
  }
  return lo * 32 + at;
}

// The rest of it: a CTA per row brings the table in line with the plan, and the
// CTAs behind those write the list and move the reference counts, a thread per
// page.  (One CTA that writes the list too takes 35 us for 16384 moves of 65536
// pages, bound by its own issue and scattered stores.)
__global__ void __launch_bounds__(256) pages_move_kernel(PagesDev p, const int32_t* work, int32_t* copies,
                                                         int32_t* err) {
  const int n = work[0], words = (p.num_pages + 31) / 32;
  if (n < 0) return;
  const PlanWord* plan = reinterpret_cast<const PlanWord*>(work + 16);
  auto moves_to = [&](int page, int& i) {  // where a page goes (-1: it is free); i = its line in the list
    const PlanWord x = plan[page >> 5];
    if (!(x.out >> (page & 31) & 1u)) return -1;
    i = x.outs_before + __popc(x.out & ((1u << (page & 31)) - 1u));
    return nth_hole(plan, words, i);
  };
  int i;
  if ((int)blockIdx.x < p.rows) {
    const int r = blockIdx.x, held = min(max(p.held[r], 0), p.max_pages);
    int32_t* row = p.table + (int64_t)r * p.max_pages;
    for (int c = threadIdx.x; c < held; c += blockDim.x) {
      const int page = row[c], to = page_ok(p, page) && page >= n ? moves_to(page, i) : page;
      if (!page_ok(p, to)) set_err(err, MEDUSA_DEVERR_PAGE);
      else if (to != page) row[c] = to;
    }
    return;
  }
  const int step = (gridDim.x - p.rows) * blockDim.x;
  for (int page = n + (blockIdx.x - p.rows) * blockDim.x + threadIdx.x; page < p.num_pages; page += step) {
    const int to = moves_to(page, i);
    if (to < 0) continue;
    *reinterpret_cast<int4*>(copies + 4 * (int64_t)i) = make_int4(page, to, p.page_size, -1);
    p.refs[to] = p.refs[page];
    p.refs[page] = 0;
  }
}

// A warp per (copy, pool, head): `tokens` lines of line_bytes bytes lie side
// by side in a head of a page.
__global__ void __launch_bounds__(256) pages_copy_kernel(uint8_t* k_pages, uint8_t* v_pages, int num_pages,
                                                         int page_size, int Hkv, int line_bytes,
                                                         const int32_t* copies, const int32_t* n_copies,
                                                         int max_copies, int32_t* err) {
  int n = *n_copies;
  if (n < 0 || n > max_copies) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_err(err, MEDUSA_DEVERR_CAPACITY);
    n = n < 0 ? 0 : max_copies;
  }
  const int lane = threadIdx.x & 31;
  const int64_t items = (int64_t)n * 2 * Hkv, step = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t head_bytes = (int64_t)page_size * line_bytes;
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += step) {
    const int i = (int)(it / (2 * Hkv)), ph = (int)(it % (2 * Hkv));
    const int4 e = __ldg(reinterpret_cast<const int4*>(copies) + i);
    if ((unsigned)e.x >= (unsigned)num_pages || (unsigned)e.y >= (unsigned)num_pages || e.z < 0 || e.z > page_size) {
      if (lane == 0) set_err(err, MEDUSA_DEVERR_PAGE);
      continue;
    }
    uint8_t* pool = ph < Hkv ? k_pages : v_pages;
    const int h = ph < Hkv ? ph : ph - Hkv;
    const uint4* from = reinterpret_cast<const uint4*>(pool + ((int64_t)e.x * Hkv + h) * head_bytes);
    uint4* to = reinterpret_cast<uint4*>(pool + ((int64_t)e.y * Hkv + h) * head_bytes);
    const int vecs = e.z * (line_bytes / 16);
    for (int v0 = lane; v0 < vecs; v0 += 32 * 8) {
      uint4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (v0 + u * 32 < vecs) x[u] = from[v0 + u * 32];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (v0 + u * 32 < vecs) to[v0 + u * 32] = x[u];
    }
  }
}

// The accepted path inside a row's pages: slot L + j <- slot L + nodes[j].
// blockIdx.y is the batch entry; a thread owns one 16-byte column of the
// token's lines in one pool and reads all its sources before it writes.
__global__ void __launch_bounds__(256) paged_compact_kernel(uint8_t* k_pages, uint8_t* v_pages, PagesDev p,
                                                            const int32_t* rows, const int32_t* nodes,
                                                            const int32_t* accept_len, int Hkv, int line_vecs,
                                                            int Kmax, int T, int32_t* err) {
  __shared__ int64_t from[MEDUSA_MAX_K + 1], to[MEDUSA_MAX_K + 1];  // lines of head 0
  __shared__ int moves;
  const int b = blockIdx.y, r = rows ? rows[b] : b;
  bool twice = false;
  if (rows)
    for (int j = threadIdx.x; j < b; j += blockDim.x) twice |= rows[j] == r;
  twice = __syncthreads_or(twice);
  if (threadIdx.x == 0) {
    int code = 0, n = 0;
    const int A = accept_len[b];
    if (twice || (unsigned)r >= (unsigned)p.rows) {
      code = MEDUSA_DEVERR_ROW;
    } else if (A < 0 || A > Kmax) {
      code = MEDUSA_DEVERR_LENGTH;
    } else {
      const int L = p.length[r], held = p.held[r];
      const int32_t* tab = p.table + (int64_t)r * p.max_pages;
      if (!row_state_ok(p, L, held)) code = MEDUSA_DEVERR_PAGE;
      for (int j = 0; j <= A && !code; ++j) {
        const int a = nodes[(int64_t)b * (Kmax + 1) + j];
        if (a < j || a >= T) {
          code = MEDUSA_DEVERR_NODE;
        } else if (((int64_t)L + a) >> p.shift >= held) {
          code = MEDUSA_DEVERR_CAPACITY;
        } else if (a != j) {
          const int ps = tab[(L + a) >> p.shift], pd = tab[(L + j) >> p.shift];
          if (!page_ok(p, ps) || !page_ok(p, pd)) code = MEDUSA_DEVERR_PAGE;
          else {
            from[n] = page_line(p, ps, Hkv, 0, (L + a) & (p.page_size - 1));
            to[n] = page_line(p, pd, Hkv, 0, (L + j) & (p.page_size - 1));
            ++n;
          }
        }
      }
    }
    moves = code ? 0 : n;
    if (code && blockIdx.x == 0) set_err(err, code);
  }
  __syncthreads();
  const int n = moves, col = blockIdx.x * blockDim.x + threadIdx.x;
  if (n == 0 || col >= 2 * Hkv * line_vecs) return;
  const int v = col % line_vecs, ph = col / line_vecs;
  uint4* pool = reinterpret_cast<uint4*>(ph < Hkv ? k_pages : v_pages);
  const int64_t head = (int64_t)(ph < Hkv ? ph : ph - Hkv) << p.shift;
  uint4 x[MEDUSA_MAX_K + 1];
#pragma unroll
  for (int j = 0; j <= MEDUSA_MAX_K; ++j)
    if (j < n) x[j] = pool[(from[j] + head) * line_vecs + v];
#pragma unroll
  for (int j = 0; j <= MEDUSA_MAX_K; ++j)
    if (j < n) pool[(to[j] + head) * line_vecs + v] = x[j];
}

}  // namespace

int check_pages(const medusa_pages_t* p, const char* fn) {
  if (!p) return fail(MEDUSA_ERR_INVALID, "%s: pages is NULL", fn);
  if (!p->refs || !p->free_bits || !p->length || !p->held || !p->table)
    return fail(MEDUSA_ERR_INVALID, "%s: pages has a NULL device array", fn);
  const int ps = p->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256)
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: page_size=%d not in {16,32,64,128,256}", fn, ps);
  if (p->rows < 1 || p->rows > MEDUSA_MAX_ROWS)
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: rows=%d outside [1, %d]", fn, p->rows, MEDUSA_MAX_ROWS);
  if (p->num_pages < 1 || p->num_pages > (1 << 26))
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: num_pages=%d outside [1, 2^26]", fn, p->num_pages);
  if (p->max_pages < 1 || (int64_t)p->max_pages * ps > (1 << 28))
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: max_pages=%d (a row may hold up to 2^28 tokens)", fn, p->max_pages);
  return MEDUSA_OK;
}

int check_pool(const void* k_pages, const void* v_pages, int num_pages, int page_size, int Hkv, int Dh,
               medusa_dtype dtype, const char* fn) {
  if (!k_pages || !v_pages) return fail(MEDUSA_ERR_INVALID, "%s: NULL pool", fn);
  if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: dtype", fn);
  if (Dh != 64 && Dh != 128) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: Dh=%d not in {64,128}", fn, Dh);
  if (Hkv < 1 || Hkv > 1024) return fail(MEDUSA_ERR_INVALID, "%s: Hkv=%d", fn, Hkv);
  if ((int64_t)num_pages * page_size * Hkv >= (1ll << 31))
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: a pool holds fewer than 2^31 lines (pages x heads x page_size)", fn);
  if ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) % 16)
    return fail(MEDUSA_ERR_INVALID, "%s: pools not 16-byte aligned", fn);
  return MEDUSA_OK;
}

}  // namespace medusa

using namespace medusa;

extern "C" int medusa_pages_init(const medusa_pages_t* pages, void* stream) {
  const char* fn = "medusa_pages_init";
  if (int rc = check_pages(pages, fn)) return rc;
  launch_kernel(pages_init_kernel, dim3(sm_count()), dim3(256), 0, as_stream(stream), pages_dev(pages));
  return check_launch(fn);
}

extern "C" int medusa_pages_free(const medusa_pages_t* pages, const int32_t* keep_len, int32_t* err, void* stream) {
  const char* fn = "medusa_pages_free";
  if (int rc = check_pages(pages, fn)) return rc;
  if (!keep_len) return fail(MEDUSA_ERR_INVALID, "%s: NULL keep_len", fn);
  launch_kernel(pages_free_kernel, dim3(pages->rows), dim3(128), 0, as_stream(stream), pages_dev(pages), keep_len, err);
  return check_launch(fn);
}

extern "C" int medusa_pages_fork(const medusa_pages_t* pages, const int32_t* src, const int32_t* dst, int n,
                                 int32_t* err, void* stream) {
  const char* fn = "medusa_pages_fork";
  if (int rc = check_pages(pages, fn)) return rc;
  if (n < 0 || n > MEDUSA_MAX_ROWS) return fail(MEDUSA_ERR_INVALID, "%s: n=%d outside [0, %d]", fn, n, MEDUSA_MAX_ROWS);
  if (n == 0) return MEDUSA_OK;
  if (!src || !dst) return fail(MEDUSA_ERR_INVALID, "%s: NULL src or dst", fn);
  launch_kernel(pages_fork_kernel, dim3(n), dim3(128), 0, as_stream(stream), pages_dev(pages), src, dst, n, err);
  return check_launch(fn);
}

extern "C" int medusa_pages_reserve(const medusa_pages_t* pages, const int32_t* n_new, int32_t* copies,
                                    int max_copies, int32_t* n_copies, int32_t* granted, int32_t* err,
                                    void* stream) {
  const char* fn = "medusa_pages_reserve";
  if (int rc = check_pages(pages, fn)) return rc;
  if (!n_new || !copies || !n_copies) return fail(MEDUSA_ERR_INVALID, "%s: NULL n_new, copies or n_copies", fn);
  if (reinterpret_cast<uintptr_t>(copies) % 16) return fail(MEDUSA_ERR_INVALID, "%s: copies not 16-byte aligned", fn);
  if (max_copies < pages->rows)
    return fail(MEDUSA_ERR_CAPACITY, "%s: copies has %d lines, a call may need one per row (%d)", fn, max_copies,
                pages->rows);
  launch_kernel(pages_reserve_kernel, dim3(1), dim3(kBlock), 0, as_stream(stream), pages_dev(pages), n_new, copies,
                n_copies, granted, err);
  return check_launch(fn);
}

extern "C" int medusa_pages_served(const medusa_pages_t* pages, const int32_t* rows, const int32_t* granted, int B,
                                   int32_t* served, void* stream) {
  const char* fn = "medusa_pages_served";
  if (int rc = check_pages(pages, fn)) return rc;
  if (B < 0 || B > MEDUSA_MAX_ROWS || (!rows && B > pages->rows))
    return fail(MEDUSA_ERR_INVALID, "%s: B=%d for %d rows", fn, B, pages->rows);
  if (B == 0) return MEDUSA_OK;
  if (!granted || !served) return fail(MEDUSA_ERR_INVALID, "%s: NULL granted or served", fn);
  launch_kernel(pages_served_kernel, dim3(1), dim3(kBlock), 0, as_stream(stream), pages_dev(pages), rows, granted, B,
                served);
  return check_launch(fn);
}

extern "C" int medusa_pages_commit(const medusa_pages_t* pages, const int32_t* rows, const int32_t* n_new, int bias,
                                   int B, int32_t* err, void* stream) {
  const char* fn = "medusa_pages_commit";
  if (int rc = check_pages(pages, fn)) return rc;
  if (B < 0 || B > MEDUSA_MAX_ROWS || (!rows && B > pages->rows))
    return fail(MEDUSA_ERR_INVALID, "%s: B=%d for %d rows", fn, B, pages->rows);
  if (bias < 0 || bias > MEDUSA_MAX_T) return fail(MEDUSA_ERR_INVALID, "%s: bias=%d", fn, bias);
  if (B == 0) return MEDUSA_OK;
  if (!n_new) return fail(MEDUSA_ERR_INVALID, "%s: NULL n_new", fn);
  launch_kernel(pages_commit_kernel, dim3(1), dim3(kBlock), 0, as_stream(stream), pages_dev(pages), rows, n_new, bias,
                B, err);
  return check_launch(fn);
}

extern "C" size_t medusa_pages_compact_workspace_size(int num_pages) {
  return num_pages < 1 ? 0 : align_up(64 + (((size_t)num_pages + 31) / 32) * sizeof(PlanWord), 256);
}

extern "C" int medusa_pages_compact(const medusa_pages_t* pages, int32_t* copies, int max_copies, int32_t* n_copies,
                                    void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  const char* fn = "medusa_pages_compact";
  if (int rc = check_pages(pages, fn)) return rc;
  if (!copies || !n_copies) return fail(MEDUSA_ERR_INVALID, "%s: NULL copies or n_copies", fn);
  if (max_copies < 0) return fail(MEDUSA_ERR_INVALID, "%s: max_copies=%d", fn, max_copies);
  if (reinterpret_cast<uintptr_t>(copies) % 16) return fail(MEDUSA_ERR_INVALID, "%s: copies not 16-byte aligned", fn);
  if (reinterpret_cast<uintptr_t>(workspace) % 16)
    return fail(MEDUSA_ERR_INVALID, "%s: workspace not 16-byte aligned", fn);
  if (!workspace || workspace_bytes < medusa_pages_compact_workspace_size(pages->num_pages))
    return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace of %zu bytes is too small", fn, workspace_bytes);
  const PagesDev p = pages_dev(pages);
  auto* work = static_cast<int32_t*>(workspace);
  launch_kernel(pages_plan_kernel, dim3(1), dim3(kBlock), 0, as_stream(stream), p, max_copies, n_copies, work, err);
  if (int rc = check_launch(fn)) return rc;
  const int blocks = (pages->num_pages + 255) / 256, movers = blocks < 2 * sm_count() ? blocks : 2 * sm_count();
  launch_kernel(pages_move_kernel, dim3(pages->rows + movers), dim3(256), 0, as_stream(stream), p, work, copies, err);
  return check_launch(fn);
}

extern "C" int medusa_pages_copy(void* k_pages, void* v_pages, int num_pages, int page_size, int Hkv, int Dh,
                                 medusa_dtype dtype, const int32_t* copies, const int32_t* n_copies, int max_copies,
                                 int32_t* err, void* stream) {
  const char* fn = "medusa_pages_copy";
  if (num_pages < 1 || page_size < 1)
    return fail(MEDUSA_ERR_INVALID, "%s: num_pages=%d page_size=%d", fn, num_pages, page_size);
  if (int rc = check_pool(k_pages, v_pages, num_pages, page_size, Hkv, Dh, dtype, fn)) return rc;
  if (!copies || !n_copies) return fail(MEDUSA_ERR_INVALID, "%s: NULL copies or n_copies", fn);
  if (max_copies < 0) return fail(MEDUSA_ERR_INVALID, "%s: max_copies=%d", fn, max_copies);
  if (reinterpret_cast<uintptr_t>(copies) % 16) return fail(MEDUSA_ERR_INVALID, "%s: copies not 16-byte aligned", fn);
  if (max_copies == 0) return MEDUSA_OK;
  const int64_t warps = (int64_t)max_copies * 2 * Hkv, ctas = (warps + 7) / 8;
  const int grid = (int)(ctas < (int64_t)sm_count() * 6 ? ctas : (int64_t)sm_count() * 6);
  launch_kernel(pages_copy_kernel, dim3(grid), dim3(256), 0, as_stream(stream), static_cast<uint8_t*>(k_pages),
                static_cast<uint8_t*>(v_pages), num_pages, page_size, Hkv, Dh * (dtype == MEDUSA_BF16 ? 2 : 4),
                copies, n_copies, max_copies, err);
  return check_launch(fn);
}

extern "C" int medusa_paged_compact(void* k_pages, void* v_pages, const medusa_pages_t* pages, const int32_t* rows,
                                    const int32_t* accepted_nodes, const int32_t* accept_len, int B, int Hkv, int Dh,
                                    int Kmax, int T, medusa_dtype dtype, int32_t* err, void* stream) {
  const char* fn = "medusa_paged_compact";
  if (int rc = check_pages(pages, fn)) return rc;
  if (int rc = check_pool(k_pages, v_pages, pages->num_pages, pages->page_size, Hkv, Dh, dtype, fn)) return rc;
  if (B < 0 || B > MEDUSA_MAX_ROWS || (!rows && B > pages->rows))
    return fail(MEDUSA_ERR_INVALID, "%s: B=%d for %d rows", fn, B, pages->rows);
  if (Kmax < 0 || Kmax > MEDUSA_MAX_K)
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: Kmax=%d outside [0, %d]", fn, Kmax, MEDUSA_MAX_K);
  if (T < 1 || T > MEDUSA_MAX_T) return fail(MEDUSA_ERR_INVALID, "%s: T=%d outside [1, %d]", fn, T, MEDUSA_MAX_T);
  if (B == 0) return MEDUSA_OK;
  if (!accepted_nodes || !accept_len) return fail(MEDUSA_ERR_INVALID, "%s: NULL accepted_nodes or accept_len", fn);
  const int line_vecs = Dh * (dtype == MEDUSA_BF16 ? 2 : 4) / 16;
  const dim3 grid((2 * Hkv * line_vecs + 255) / 256, B);
  launch_kernel(paged_compact_kernel, grid, dim3(256), 0, as_stream(stream), static_cast<uint8_t*>(k_pages),
                static_cast<uint8_t*>(v_pages), pages_dev(pages), rows, accepted_nodes, accept_len, Hkv, line_vecs,
                Kmax, T, err);
  return check_launch(fn);
}

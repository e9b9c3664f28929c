// Chunk attention over the paged cache for many query rows, bf16, on the
// tensor cores (tcgen05, accumulators in tensor memory).
//
// A block of up to 256 query rows is two MMA tiles of 128 rows ("lanes" 0 and
// 1), and a tile of KT keys (96, or 128 where heads have 64 columns) costs each
// lane
//   S = Q K^T  (128 x KT x Dh, twice)   and   O += P V  (128 x Dh x KT),
// 1152 cycles of the SM's tensor core together at Dh = 128.  While one lane's
// scores are exponentiated, the tensor core works for the other: the issuing
// thread's order is PV0(j), QK0(j+1), PV1(j), QK1(j+1), ..., so a lane's
// softmax has the other lane's products, 1152 cycles, to hide behind.  The
// kernel is bound by the tensor core where that holds.
//   * warps 0-3 and 4-7 are the lanes' softmax: a thread per query row (its
//     tensor-memory lane) reads KT scores and writes P = 2^(S - m) in bf16
//     over them in tensor memory, with no exchange between threads.  (Two
//     threads per row, which agree on the maximum through shared memory, take
//     less time from scores to P, but issue 1.7 times the instructions, and the
//     MMA warp shares the issue slots: 4% longer for 8192 tokens, with queries
//     in one part.)
//   * O stays in tensor memory.  The base m of a row only moves when the
//     row's maximum passes it by more than 8 (P is at most 2^8, its sum is
//     kept in 32 bits), so O is rescaled a few times per row and not per tile.
//   * a warp loads keys and values by TMA, page by page, into a ring of
//     slots; a thread issues the MMAs and the query tiles' loads.
// A block of at most 128 rows has one query tile: the lanes then take the key
// tiles in turn, with the same queries, and their results are joined at the
// segment's end.
// Queries come rotated and scaled from the launch before this one, which also
// appends the chunk, as two bf16 parts, high and low, 2^-16 relative together:
// an error of a query is one of every score, and grows with the scores.  Each
// part has a product of its own.  (One part alone takes 363 us in place of 488
// for 8192 tokens of 32 heads of 128, and its error, at scores of deviation 1, is
// as large as the result's own rounding.)  The low parts take the room that
// tiles of 128 keys would need at Dh = 128.
// P is rounded once to bf16 where a call has two query tiles: a relative 2^-8 a
// weight at most, independent from key to key, so no larger in the result than
// its own rounding, whatever the scores.  (In two parts, with queries in one: 104
// us in place of 79 for the mixed batch below, 579 in place of 412 for the
// prompt, and as far from 64 bits as this way round.)  A call with one query
// tile, bound by memory, has time for two parts of P as well (4 of its 110 us).
// Behind a shared prefix the rows of a group are those of many sequences: where each
// has at most 128, kCommon holds P in two parts however many there are (FINE), so
// that a token's weights are as exact as without sharing, whoever shares with it
// (104 tokens behind up to 16384, 32 heads of 128 on 8: error against 64 bits 0.0023
// to 0.0017, its own rounding, for 167 to 174 us; 120 tokens behind up to 12000, 64
// heads of 64, 111 to 128 us).
// MMAs that one thread issues run in issue order on the CTA's tensor core:
// QK(j+1) may overwrite the columns from which PV(j), issued before it, reads
// P.
// Measured, with the launch before it: 8192 tokens of 32 heads of 128 (8 key
// heads) 564 to 573 us, the kernel itself 488 us or 1.69 PFLOP/s with both parts'
// products, 97% of what a library product sustains, at the power limit (SM clock
// 1950 MHz; 2070 for the others); trees of 65 rows on four prefixes up to 8192, 52
// heads of 128, 111 us (bound by memory in the loop over tiles; plan, first loads
// and joins around it); eleven sequences of 1 .. 700 tokens, 40 heads of 64 (8 key
// heads), prefixes up to 5000, 88 us (bound by the way from one tile's scores to
// the next one's).
// Other kinds of keys (kWindow, kCommon, kOwn) change which tiles a unit has, the mask
// of the first and last ones, whose unseen values become zeros, and the results'
// place.  With a window of 2048: 8192 tokens behind 4096, 32 heads of 128, 311 us and
// 60 for the launch before it, the same 3200 cycles a tile of two lanes as without
// one (queries in two parts, at the power limit).  Trees of 65 rows on eight prefixes
// up to 16384, 32 heads of 128, with a window of 2048: 90 us with the launch before it.
// Groups of 64, 20 and 12 single tokens behind 6000 .. 8192, 32 heads of 128 on 8: 41 us
// (37 with P in one part), and 8 for the launch that adds the partials.
#pragma once

#include <utility>

#include "paged_attn.cuh"
#include "sm100.cuh"

namespace medusa {
namespace {
namespace chunk {

using namespace sm100;

constexpr int RB = 256;
// places that beginning and ending a unit is worth
constexpr int kCost = 2;  // 8192 tokens: 585, 565, 565 us at 1, 2, 3; the mixed batch 89, 88, 90; trees 111, 110, 111
constexpr int kThreads = 384;  // two softmax groups of 128; the load warp, the MMA warp and two segment warps
constexpr int kSoft = 256, kLoadWarp = 8, kMmaWarp = 9;
// Registers: the block starts with 168 a thread (384 x 168 = 64512); the softmax
// threads, which hold up to 128 scores, then take what the other warps give up:
// 256 x 208 + 128 x 88.
constexpr int kLaunchRegs = 168, kSoftRegs = 208, kOtherRegs = 88;
static_assert(kSoft * kSoftRegs + (kThreads - kSoft) * kOtherRegs <= kThreads * kLaunchRegs, "registers");
constexpr uint32_t kTmemCols = 512;
// Where dynamic shared memory begins in a kernel without static: behind what the
// system keeps of a block's.  prepare_kernel asks the device, the kernel checks.
constexpr uint32_t kSmemBase = 1024;

// Keys that one copy may bring: a tile is a whole number of copies, and they
// begin where a page's lines may (a page ends inside none of them).
MDEV __host__ constexpr int key_box(int kt) { return kt & -kt; }

template <uint32_t B>
struct Half {
  static constexpr uint32_t value = B;
};

// NARROW: a call whose chunks all have one query tile (at most 128 rows per key
// head), bound by memory: the second tile's place goes to the ring (the trees
// above, 2% less time than without).
template <int DH, bool NARROW, Keys KEYS>
struct ChunkCfg {
  static constexpr int kHalves = DH / 64;
  // keys per tile: as many as leave room for both parts of the queries
  static constexpr int KT = DH == 64 ? 128 : 96;
  static constexpr uint32_t kQHalf = 128 * 128;           // 128 rows of one swizzle span
  static constexpr uint32_t kQTile = kQHalf * kHalves;    // 128 rows x DH bf16
  static constexpr int kQTiles = NARROW ? 1 : 2;          // their high parts, then their low parts
  static constexpr uint32_t kHalf = KT * 128, kTile = kHalf * kHalves;  // KT keys, or values
  // a stage: the values of a tile and the keys of the next, one wait for both
  static constexpr int kStages = !NARROW ? 2 : DH == 128 ? 3 : 6;
  static constexpr uint32_t kRingOff = 2 * kQTiles * kQTile;
  static constexpr uint32_t kBarOff = kRingOff + kStages * 2 * kTile;
  static constexpr int kBars = 2 * kStages + 2 + 2 + 2 + 1 + 1 + 1;
  static constexpr uint32_t kSegOff = (kBarOff + kBars * 8 + 16 + 15) & ~15u;    // [2 lanes][2] segments
  static constexpr uint32_t kPlanOff = (kSegOff + 4 * sizeof(Segment<KEYS>) + 15) & ~15u;
  static constexpr uint32_t kRowOff = (kPlanOff + sizeof(Plan) + 15) & ~15u;  // [2 lanes][128 rows] 8 bytes
  static constexpr size_t smem = kRowOff + 2 * 128 * 8;
  static_assert(smem <= 232448, "shared memory");
  static constexpr int part_floats = 128 * DH + 2 * 128;  // one lane's partial
  static_assert(sizeof(PlanScratch) <= kStages * 2 * kTile, "the plan's scratch lies in the ring");
};

// One thread of a converged warp, the same one every time.  The MMA's operands
// are warp-wide registers: behind an `elect` the compiler knows that one thread
// issues, behind a comparison of the lane it goes through the lanes one by one.
MDEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}
MDEV void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
// Barriers of a lane's threads and the warp that writes its segments, of a
// lane's 128 threads, of all 256.
MDEV void bar_segment(int i) { asm volatile("bar.sync %0, 160;\n" ::"r"(1 + i) : "memory"); }
MDEV void bar_lane(int i) { asm volatile("bar.sync %0, 128;\n" ::"r"(3 + i) : "memory"); }
MDEV void bar_all() { asm volatile("bar.sync 5, 256;\n" ::: "memory"); }
MDEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
MDEV void add2(float& a, float& b, float x, float y) {
  asm("{\n .reg .b64 A, X;\n mov.b64 A, {%0, %1};\n mov.b64 X, {%2, %3};\n add.rn.f32x2 A, A, X;\n"
      " mov.b64 {%0, %1}, A;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// 32 consecutive columns of this thread's tensor-memory lane.
MDEV void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// MMAs whose operands are all constants.  An MMA takes its descriptors and
// addresses from warp-wide registers; anything that comes from a thread's
// register is moved there first, six moves an MMA, which the issuing warp had
// no time for beside the softmax.  Tensor memory starts at column 0: a block
// that allocates all 512 columns gets them there.
template <uint32_t D, uint64_t A, uint64_t B, uint32_t IDESC, bool ADD>
MDEV void umma_const() {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 A, B;\n\t.reg .b32 D, I;\n\t"
      "mov.b32 D, %0;\n\tmov.b64 A, %1;\n\tmov.b64 B, %2;\n\tmov.b32 I, %3;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [D], A, B, I, p;\n\t}\n" ::"n"(D),
      "n"(A), "n"(B), "n"(IDESC), "n"((int)ADD)
      : "memory");
}
template <uint32_t D, uint32_t A, uint64_t B, uint32_t IDESC>
MDEV void umma_ts_const(uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 B;\n\t.reg .b32 A, D, I;\n\t"
      "mov.b32 D, %0;\n\tmov.b32 A, %1;\n\tmov.b64 B, %2;\n\tmov.b32 I, %3;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [D], [A], B, I, p;\n\t}\n" ::"n"(D),
      "n"(A), "n"(B), "n"(IDESC), "r"(add)
      : "memory");
}
// The same from words known at run time (both descriptors' high words are the
// same).
MDEV void umma_words(uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 A, B;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 A, {%1, %3};\n\tmov.b64 B, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], A, B, %4, p;\n\t}\n" ::"r"(d),
      "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(add)
      : "memory");
}
MDEV void umma_ts_words(uint32_t d, uint32_t a, uint32_t blo, uint32_t hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 B;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 B, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], B, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(blo), "r"(hi), "r"(idesc), "r"(add)
      : "memory");
}
// The products of lane I with the keys or values in stage B (QT: the query
// tile).  Matrix descriptors: 128-byte swizzle, 1024 bytes between 8-row
// groups; low word address / 16 and, for V, the bytes / 16 between its halves.
template <int DH, bool FINE>
struct Products {
  using G = ChunkCfg<DH, false, kAll>;  // tiles and stages do not depend on the keys
  static constexpr uint64_t kHi = (uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32;
  static constexpr int KT = G::KT;
  static constexpr uint32_t kQHalf16 = G::kQHalf >> 4, kQTile16 = G::kQTile >> 4;
  static constexpr uint32_t kHalf16 = G::kHalf >> 4, kTile16 = G::kTile >> 4;
  static constexpr uint32_t kQ = kSmemBase >> 4 | 1u << 16, kK = (kSmemBase + G::kRingOff) >> 4 | 1u << 16;
  static constexpr uint32_t kV = ((kSmemBase + G::kRingOff) >> 4) + kTile16 | kHalf16 << 16;
  static __host__ __device__ constexpr uint32_t step(int kk, uint32_t half) { return (kk >> 2) * half + (kk & 3) * 2; }
  // step KK of the high parts (PART 0) or the low parts (1) of query tile QT
  template <uint32_t I, uint32_t QT, uint32_t B, int PART, int... KK>
  static MDEV void qk_steps(std::integer_sequence<int, KK...>) {
    (umma_const<I * 128, kHi | (kQ + (PART * G::kQTiles + QT) * kQTile16 + step(KK, kQHalf16)),
                kHi | (kK + B * 2 * kTile16 + step(KK, kHalf16)), idesc_bf16_f32(128, KT), PART != 0 || KK != 0>(),
     ...);
  }
  // (steps past KT / 16: P's low parts)
  template <uint32_t I, uint32_t B, int... J>
  static MDEV void pv_steps(uint32_t add, std::integer_sequence<int, J...>) {
    // V as stored, keys x values, is MN-major
    (umma_ts_const<256 + I * 128, I * 128 + J * 8, kHi | (kV + B * 2 * kTile16 + J % (KT / 16) * (2048 >> 4)),
                   idesc_bf16_f32(128, DH) | 1u << 16>(J == 0 ? add : 1u),
     ...);
  }
  template <uint32_t I, uint32_t QT, uint32_t B>
  static MDEV void qk() {
    qk_steps<I, QT, B, 0>(std::make_integer_sequence<int, DH / 16>());
    qk_steps<I, QT, B, 1>(std::make_integer_sequence<int, DH / 16>());
  }
  template <uint32_t I, uint32_t B>
  static MDEV void pv(uint32_t add) {
    pv_steps<I, B>(add, std::make_integer_sequence<int, (FINE ? 2 : 1) * KT / 16>());
  }
};

MDEV void commit_at(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
MDEV bool try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// paged_wait by shared-memory address.
MDEV void wait_at(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (try_wait_at(bar, parity)) return;
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (try_wait_at(bar, parity)) return;
    if ((i & 63) == 63 && *abort_flag) return;
  }
  *abort_flag = 1;
}

// FINE: P in two parts.
template <int DH, bool NARROW, bool FINE, Keys KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQl,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ PagedAttnArgs a) {
  using G = ChunkCfg<DH, NARROW, KEYS>;
  static_assert(FINE || !NARROW, "a call with one query tile has time for both parts");
  constexpr int KT = G::KT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase != kSmemBase) {  // the host has asked the device, too
    if (threadIdx.x == 0) set_err(a.err, MEDUSA_DEVERR_LAYOUT);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kBarOff);  // [stages] TMA -> MMA
  uint64_t* empty = full + G::kStages;                              // [stages] MMA -> TMA
  uint64_t* s_full = empty + G::kStages;                             // [2] MMA -> softmax: scores
  uint64_t* p_full = s_full + 2;                                    // [2] softmax -> MMA: P written, O rescaled
  uint64_t* pv_done = p_full + 2;                                   // [2] MMA -> softmax: the segment's O is complete
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_empty = q_full + 1;                                   // MMA -> TMA: every product of these queries is done
  uint64_t* all_done = q_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + 1);
  int* s_abort = reinterpret_cast<int*>(tmem_slot + 1);
  int* s_flag = s_abort + 1;  // [2]
  Plan& pl = *reinterpret_cast<Plan*>(smem + G::kPlanOff);
  PlanScratch& sc = *reinterpret_cast<PlanScratch*>(smem + G::kRingOff);
  Segment<KEYS>* segs = reinterpret_cast<Segment<KEYS>*>(smem + G::kSegOff);
  volatile int* abort_flag = s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);  // its values are used, its keys are used
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(all_done, 1);
    fence_barrier_init();
    *s_abort = 0;
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmQl);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // kCommon needs the groups for its plan.  kOwn starts when it has ended: what the
  // first launch wrote is there, and it waits for the common parts only where it
  // joins them.
  if constexpr (KEYS == kCommon) asm volatile("griddepcontrol.wait;\n" ::: "memory");
  int64_t x0, x1;
  make_plan<kThreads, RB, KT, kCost, KEYS>(a, sc, pl, x0, x1);
  const int64_t total = pl.total, grid = min((int64_t)gridDim.x, total);
  Segment<KEYS> sg;
  const bool any = x0 < x1 && seek_segment<RB, KT, kCost>(a, sc, x0, x1, sg);
  fence_smem_async();  // the scratch was read and written; the ring's copies follow
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // 0: all of it
  const int tb = RB / a.g;
  // A CTA without work waits here for the launch before this one: the grid must
  // not end before that one's reads, which the next call on the stream may
  // change.  With work, its loading warps wait.
  if (!any) asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (warp >= kSoft / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp && any) {
      // ------------------------------------------------ keys and values
      // the appended tokens, written by the launch before
      if constexpr (KEYS != kOwn) asm volatile("griddepcontrol.wait;\n" ::: "memory");
      asm volatile("fence.proxy.async.global;\n" ::: "memory");
      const int box = min(a.p.page_size, key_box(KT)), runs = KT / box;
      const int op_run = lane / G::kHalves, op_half = lane % G::kHalves;
      const bool mine = op_run < runs;
      const int nowhere = (a.p.num_pages * a.Hkv) << a.p.shift;  // past the pool: reads zeros
      // fill n of the ring: the values of the CTA's tile n - 1, the keys of tile n
      int n = 0, yv = 0, st = 0;
      uint32_t ph = 1;
      bool more = true;
      int t = sg.t0;
      while (true) {
        int y = nowhere;
        if (more) {
          const SeqInfo<KEYS>& s = sg.s;
          const int key = sg.real_tile(t) * KT + op_run * box;
          if (mine && key < s.keys()) {
            const int page = a.p.table[(int64_t)s.row * a.p.max_pages + (key >> a.p.shift)];
            if (page_ok(a.p, page)) y = (int)page_line(a.p, page, a.Hkv, sg.head, key & (a.p.page_size - 1));
            else set_err(a.err, MEDUSA_DEVERR_PAGE);
          }
        }
        paged_wait(&empty[st], ph, abort_flag);
        if (lane == 0) mbar_expect_tx(&full[st], (more ? G::kTile : 0u) + (n > 0 ? G::kTile : 0u));
        __syncwarp();
        uint8_t* dst = smem + G::kRingOff + st * 2 * G::kTile + op_half * G::kHalf + op_run * box * 128;
        if (mine && n > 0) tma_load_2d(dst + G::kTile, &tmV, &full[st], op_half * 64, yv);
        if (mine && more) tma_load_2d(dst, &tmK, &full[st], op_half * 64, y);
        yv = y;
        ++n;
        if (++st == G::kStages) {
          st = 0;
          ph ^= 1u;
        }
        if (!more) break;
        if (++t == sg.t1) {
          more = next_segment<RB, KT, kCost>(a, pl, x1, sg);
          t = sg.t0;
        }
      }
      // the copies in flight land before the CTA can end, whatever happened
      for (int j = max(0, n - G::kStages); j < n; ++j)
        if (!mbar_wait(&full[j % G::kStages], (uint32_t)(j / G::kStages) & 1u)) *abort_flag = 1;
    } else if (warp == kMmaWarp && any) {
      // ------------------------------------------------ MMAs
      // One thread issues 44 products' instructions per tile of 2304 cycles.
      // Issuing does not run ahead of the tensor core by more than an
      // instruction or two, and beside the softmax warps a wait costs 150
      // cycles even where it is over: so addresses are constants, and there are
      // as few waits and commits as will do (QK(j+1)'s commit also says that
      // PV(j), issued before it, is done).
      constexpr uint32_t bars = kSmemBase + G::kBarOff;
      constexpr uint32_t kEmpty = bars + G::kStages * 8, kS = kEmpty + G::kStages * 8, kP = kS + 2 * 8, kPV = kP + 2 * 8,
                         kQ = kPV + 2 * 8, kQE = kQ + 8, kDone = kQE + 8;
      if (NARROW) {
        // Bound by memory: addresses at run time, a ring of more stages.  Lane
        // j & 1 has tile j; QK runs two tiles ahead of PV, of the segment only.
        if (elect_one()) {
          constexpr uint32_t kStage16 = 2 * G::kTile >> 4, kHalf16 = G::kHalf >> 4, kTile16 = G::kTile >> 4;
          constexpr uint32_t kQHalf16 = G::kQHalf >> 4, kQTile16 = G::kQTile >> 4;
          constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
          constexpr uint32_t q16 = kSmemBase >> 4 | 1u << 16, k16 = (kSmemBase + G::kRingOff) >> 4 | 1u << 16;
          constexpr uint32_t v16 = ((kSmemBase + G::kRingOff) >> 4) + kTile16 | kHalf16 << 16;
          auto next_stage = [](uint32_t& st, uint32_t& ph) {
            if (++st == G::kStages) {
              st = 0;
              ph ^= 1u;
            }
          };
          uint32_t kst = 0, kph = 0;     // the stage with the next QK's keys
          uint32_t vst = 0, vph = 0;     // ... with the next PV's values: the one after its keys'
          next_stage(vst, vph);
          uint32_t pph[2] = {0, 0}, qph = 0;
          bool first = true, more = true;
          auto scores = [&](uint32_t i) {
            wait_at(bars + kst * 8, kph, abort_flag);
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 2 * DH / 16; ++e) {  // the queries' high parts, then their low parts
              const int kk = e % (DH / 16), part = e / (DH / 16);
              umma_words(i * 128, q16 + part * kQTile16 + (kk >> 2) * kQHalf16 + (kk & 3) * 2,
                         k16 + kst * kStage16 + (kk >> 2) * kHalf16 + (kk & 3) * 2, kDescHi, idesc_bf16_f32(128, KT),
                         e != 0);
            }
            commit_at(kS + i * 8);
            commit_at(kEmpty + kst * 8);
            if (first) commit_at(kEmpty + kst * 8);  // the first stage has no values
            first = false;
            next_stage(kst, kph);
          };
          do {
            const uint32_t n = sg.t1 - sg.t0;
            wait_at(kQ, qph, abort_flag);
            qph ^= 1u;
            scores(0);
            if (n > 1) scores(1);
            if (n <= 2) commit_at(kQE);
            for (uint32_t j = 0; j < n; ++j) {
              const uint32_t i = j & 1u;
              wait_at(bars + vst * 8, vph, abort_flag);
              wait_at(kP + i * 8, pph[i], abort_flag);
              pph[i] ^= 1u;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 2 * KT / 16; ++k)  // P's high parts, then its low parts
                umma_ts_words(256 + i * 128, i * 128 + k * 8, v16 + vst * kStage16 + k % (KT / 16) * (2048 >> 4),
                              kDescHi, idesc_bf16_f32(128, DH) | 1u << 16, k == 0 ? (uint32_t)(j > 1) : 1u);
              commit_at(kEmpty + vst * 8);
              next_stage(vst, vph);
              if (j + 2 < n) {
                scores(i);
                if (j + 3 == n) commit_at(kQE);
              } else {
                commit_at(kPV + i * 8);
              }
            }
            more = next_segment<RB, KT, kCost>(a, pl, x1, sg);
          } while (more);
          commit_at(kDone);
          wait_at(kDone, 0, abort_flag);
        }
      } else if (elect_one()) {
        using P = Products<DH, FINE>;
        uint32_t t = 0, ph0 = 0, ph1 = 0, qph = 0;  // the CTA's tiles so far; phases of p_full and q_full
        uint32_t nt = sg.t1 - sg.t0, wide = min(tb, sg.s.n - sg.u * tb) * a.g > 128;
        bool ready = false;  // the segment's first scores are on their way
        while (true) {
          const uint32_t n = nt, w = wide;
          const bool more = next_segment<RB, KT, kCost>(a, pl, x1, sg);
          if (more) {
            nt = sg.t1 - sg.t0;
            wide = min(tb, sg.s.n - sg.u * tb) * a.g > 128;
          }
          const bool chain = more && w && wide;  // the next segment's first scores follow this one's last
          // QK of lane 0 (or, narrow, of lane i) with the keys of tile u
          auto one = [&](uint32_t i, uint32_t u) {
            if (i == 0) {
              if (u & 1u) P::template qk<0, 0, 1>(); else P::template qk<0, 0, 0>();
            } else {
              if (u & 1u) P::template qk<1, 0, 1>(); else P::template qk<1, 0, 0>();
            }
            commit_at(kS + i * 8);
          };
          if (!ready) {
            wait_at(kQ, qph, abort_flag);
            qph ^= 1u;
            for (uint32_t i = 0; i < 2 && (w ? i < 1 : i < n); ++i) {
              const uint32_t u = t + i;
              wait_at(bars + (u & 1u) * 8, u >> 1 & 1u, abort_flag);
              tc_fence_after();
              one(i, u);
              if (w) {
                if (u & 1u) P::template qk<1, 1, 1>(); else P::template qk<1, 1, 0>();
                commit_at(kS + 8);
              }
              commit_at(kEmpty + (u & 1u) * 8);
              if (u == 0) commit_at(kEmpty);  // the first stage has no values
              if (w ? n == 1 : i + 1 == n) commit_at(kQE);
            }
          }
          if (w) {
            // tile t with its keys in stage B and its values in the other one:
            // PV0(t), QK0(t + 1), PV1(t), QK1(t + 1)
            auto tile = [&](auto stage, uint32_t j) {
              constexpr uint32_t B = decltype(stage)::value, O = B ^ 1;
              const bool end = j + 1 == n, go = !end || chain;
              wait_at(bars + O * 8, (t + 1) >> 1 & 1u, abort_flag);  // V(t) and K(t + 1)
              wait_at(kP, ph0, abort_flag);
              tc_fence_after();
              P::template pv<0, O>(j > 0);
              if (go) {
                if (end) {
                  commit_at(kPV);
                  wait_at(kQ, qph, abort_flag);
                  qph ^= 1u;
                }
                P::template qk<0, 0, O>();
                commit_at(kS);
              } else {
                commit_at(kPV);
              }
              wait_at(kP + 8, ph1, abort_flag);
              tc_fence_after();
              P::template pv<1, O>(j > 0);
              commit_at(kEmpty + O * 8);
              if (end) commit_at(kPV + 8);
              if (go) {
                P::template qk<1, 1, O>();
                commit_at(kS + 8);
                commit_at(kEmpty + O * 8);
                if (j + 2 == n || (end && nt == 1)) commit_at(kQE);
              }
              ph0 ^= 1u;
              ph1 ^= 1u;
              ++t;
            };
            for (uint32_t j = 0; j < n; ++j) {
              if (t & 1u) tile(Half<1>(), j);
              else tile(Half<0>(), j);
            }
            ready = chain;
          } else {
            for (uint32_t j = 0; j < n; ++j) {
              const uint32_t i = j & 1u, o = (t + 1) & 1u;
              wait_at(bars + o * 8, (t + 1) >> 1 & 1u, abort_flag);
              wait_at(kP + i * 8, i ? ph1 : ph0, abort_flag);
              if (i) ph1 ^= 1u; else ph0 ^= 1u;
              tc_fence_after();
              if (i == 0) {
                if (o) P::template pv<0, 1>(j > 1); else P::template pv<0, 0>(j > 1);
              } else {
                if (o) P::template pv<1, 1>(j > 1); else P::template pv<1, 0>(j > 1);
              }
              commit_at(kEmpty + o * 8);
              if (j + 2 < n) {
                wait_at(bars + (t & 1u) * 8, (t + 2) >> 1 & 1u, abort_flag);
                tc_fence_after();
                one(i, t + 2);
                commit_at(kEmpty + (t & 1u) * 8);
                if (j + 3 == n) commit_at(kQE);
              } else {
                commit_at(kPV + i * 8);
              }
              ++t;
            }
            ready = false;
          }
          if (!more) break;
        }
        commit_at(kDone);
        wait_at(kDone, 0, abort_flag);
      }
      __syncwarp();
    } else if (warp > kMmaWarp && any) {
      // ------------------------------------------------ a lane's segments
      // one ahead of its softmax, which keeps its registers for scores; lane
      // 0's warp also loads the segment's queries
      const int i = warp - kMmaWarp - 1;
      if constexpr (KEYS != kOwn) asm volatile("griddepcontrol.wait;\n" ::: "memory");
      asm volatile("fence.proxy.async.global;\n" ::: "memory");
      int ns = 0;
      for (;; ++ns) {
        if (lane == 0) segs[i * 2 + (ns & 1)] = sg;
        if (i == 0) {
          if (ns > 0) paged_wait(q_empty, (uint32_t)(ns - 1) & 1u, abort_flag);
          if (lane == 0) {
            const int tiles = min(tb, sg.s.n - sg.u * tb) * a.g > 128 ? 2 : 1;
            const int y = (sg.head * a.total_q + sg.s.q0 + sg.u * tb) * a.g;
            mbar_expect_tx(q_full, 2 * tiles * G::kQTile);
            for (int k = 0; k < tiles; ++k)
              for (int h = 0; h < G::kHalves; ++h) {
                tma_load_2d(smem + k * G::kQTile + h * G::kQHalf, &tmQ, q_full, h * 64, y + k * 128);
                tma_load_2d(smem + (G::kQTiles + k) * G::kQTile + h * G::kQHalf, &tmQl, q_full, h * 64, y + k * 128);
              }
          }
        }
        __syncwarp();
        bar_segment(i);
        if (!next_segment<RB, KT, kCost>(a, pl, x1, sg)) break;
      }
      if (i == 0 && !mbar_wait(q_full, (uint32_t)ns & 1u)) *abort_flag = 1;  // landed, whatever happened
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    if (any) {
      // ------------------------------------------------ softmax of lane `i`
      const int i = warp >> 2, q = warp & 3, r = 32 * q + lane;
      const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16);
      const uint32_t tS = trow + i * 128, tO = trow + 256 + i * 128;
      float2* row_ml = reinterpret_cast<float2*>(smem + G::kRowOff);  // [2 lanes][128 rows] (max, sum)
      uint32_t cnt = 0, nend = 0;  // this lane's tiles, and segments with tiles, so far
      int it = 0, ns = 0;
      for (;; ++ns) {
        bar_segment(i);
        const Segment<KEYS>& g = segs[i * 2 + (ns & 1)];
        const int nt = g.t1 - g.t0, L = g.s.L, nkeys = g.s.keys(), tok0 = g.u * tb;
        const int live = min(tb, g.s.n - tok0) * a.g;
        const bool wide = !NARROW && live > 128;
        const int row = wide ? i * 128 + r : r;
        const bool on = row < live;
        const int tok = min(tok0 + row / a.g, g.s.n - 1);
        const int t0 = g.t0;
        // keys low0 .. low1 - 1 are seen by no token of the block, those to low2 not
        // by all; low: the first one past low0 that this thread's token sees
        int low0 = 0, low1 = 0, low2 = 0, low = 0;
        if constexpr (kSkips<KEYS>) {
          unseen_keys(a, g.s, tok0, min(g.s.n, tok0 + tb) - 1, low0, low1, low2);
          low = KEYS == kOwn ? common_keys(g.s) : a.T ? min(L, window_low(a, L, node_depth(a, tok))) : window_low(a, L, tok);
        }
        float m = -INFINITY, l = 0.f;
        int done = 0;  // this lane's tiles of the segment
        for (int j = wide ? 0 : i; j < nt; j += wide ? 1 : 2, ++done) {
          const int key0 = g.real_tile(t0 + j) * KT;
          paged_wait(&s_full[i], cnt & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
          uint32_t v[KT];
#pragma unroll
          for (int c = 0; c < KT; c += 32) tmem_ld32(tS + c, v + c);
          tmem_ld_wait();
          constexpr int kPiece = KT % 64 ? KT : 64;
          auto mask = [&](int c0) {  // keys c0 .. c0 + kPiece - 1 of the tile
            if constexpr (kSkips<KEYS>) {
              if (key0 + c0 < low2 && key0 + c0 + kPiece > low0) {
                const int from = low0 - key0, to = low - key0;  // keys from .. to - 1 are not seen
#pragma unroll
                for (int e = 0; e < kPiece; ++e)
                  v[c0 + e] = c0 + e >= from && c0 + e < to ? 0xff800000u : v[c0 + e];
              }
            }
            if (a.T == 0 || KEYS == kCommon) {
              const int d = KEYS == kCommon ? L - key0 : L + tok + 1 - key0;  // keys below this are seen
              if (__any_sync(0xffffffffu, d < c0 + kPiece)) {
#pragma unroll
                for (int e = 0; e < kPiece; ++e) v[c0 + e] = c0 + e < d ? v[c0 + e] : 0xff800000u;
              }
            } else if (key0 + c0 + kPiece > L) {
              const uint32_t* anc = a.anc + (int64_t)tok * a.W;
#pragma unroll
              for (int w = 0; w < kPiece / 32; ++w) {
                const int j0 = key0 + c0 + 32 * w, n0 = j0 - L;  // tree node of bit 0 (negative: prefix keys first)
                uint32_t bits = 0xffffffffu;
                if (n0 >= 0) {
                  const int k = n0 >> 5, sh = n0 & 31;
                  const uint32_t lo = k < a.W ? __ldg(anc + k) : 0u, hi = k + 1 < a.W ? __ldg(anc + k + 1) : 0u;
                  bits = sh ? (lo >> sh) | (hi << (32 - sh)) : lo;
                } else if (n0 > -32) {
                  bits = (0xffffffffu >> (32 + n0)) | (__ldg(anc) << (-n0));
                }
                const int past = nkeys - j0;  // nothing past the sequence
                if (past < 32) bits &= past > 0 ? (1u << past) - 1u : 0u;
#pragma unroll
                for (int e = 0; e < 32; ++e) v[c0 + 32 * w + e] = (bits >> e & 1u) ? v[c0 + 32 * w + e] : 0xff800000u;
              }
            }
          };
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto maxima = [&](int c0) {
#pragma unroll
            for (int e = 0; e < kPiece; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(v[c0 + e + 2 * k])), __uint_as_float(v[c0 + e + 2 * k + 1]));
          };
#pragma unroll
          for (int c = 0; c < KT; c += kPiece) {
            mask(c);
            maxima(c);
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool far = mt > m + 8.f;
          if (__any_sync(0xffffffffu, far)) {  // a segment's first tile, and seldom after
            const float mn = far ? mt : m;
            // O so far holds what the old base gave.  This tile's scores say that
            // the product before is done.
            if (done > 0) {
              const float al = m == -INFINITY ? 0.f : ex2(m - mn);
              l *= al;
#pragma unroll 1
              for (int c = 0; c < DH / 16; ++c) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(tO + c * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st_32x32b_x16(tO + c * 16, o);
              }
            }
            m = mn;
          }
          const float base = m == -INFINITY ? 0.f : m;
          float sa[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
#pragma unroll
          for (int h = 0; h < KT / 32; ++h) {
            uint32_t p[16], low[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float u = __uint_as_float(v[32 * h + 2 * e]), w = __uint_as_float(v[32 * h + 2 * e + 1]);
              add2(u, w, -base, -base);
              u = ex2(u);
              w = ex2(w);
              add2(sa[e & 1], sb[e & 1], u, w);
              p[e] = pack2_bf16(u, w);
              if (FINE) low[e] = pack2_bf16(u - __uint_as_float(p[e] << 16), w - __uint_as_float(p[e] & 0xffff0000u));
            }
            tmem_st_32x32b_x16(tS + h * 16, p);
            if (FINE) tmem_st_32x32b_x16(tS + KT / 2 + h * 16, low);
          }
          l += (sa[0] + sb[0]) + (sa[1] + sb[1]);
          tmem_st_wait();
          // value rows past the sequence, and those that no token sees, hold
          // whatever the page does: zeros (lane 0's P is waited for before either lane's product)
          const bool unseen = kSkips<KEYS> && key0 < low1 && key0 + KT > low0;
          if ((key0 + KT > nkeys || unseen) && (i == 0 || !wide)) {
            const int n = it + j + 1, st = n % G::kStages;  // the values' fill and stage
            paged_wait(&full[st], (uint32_t)(n / G::kStages) & 1u, abort_flag);
            if (r < KT && (key0 + r >= nkeys || (unseen && key0 + r >= low0 && key0 + r < low1))) {
#pragma unroll
              for (int c = 0; c < G::kHalves * 8; ++c)
                *reinterpret_cast<uint4*>(smem + G::kRingOff + st * 2 * G::kTile + G::kTile + (c >> 3) * G::kHalf +
                                          r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_smem_async();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[i]);
          ++cnt;
        }
        if (done > 0) {
          paged_wait(&pv_done[i], nend & 1u, abort_flag);
          ++nend;
          __syncwarp();
          tc_fence_after();
        }
        if (l != l) m = INFINITY;  // so that no join drops a part whose scores are all NaN
        if constexpr (KEYS == kOwn) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        // Two query tiles: a thread ends with its row.  One: the lanes' results
        // are joined, and it has half of the columns (both threads read the
        // same tensor-memory lane).
        int c0 = 0, c1 = DH;
        float wa = 1.f, wb = 0.f;
        uint32_t ta = tO;
        const uint32_t tB = trow + 256 + 128;
        const bool two = !wide && nt > 1;
        if (!wide) {
          row_ml[i * 128 + r] = make_float2(m, l);
          tc_fence_before();
          bar_all();
          tc_fence_after();
          const float2 e0 = row_ml[r], e1 = row_ml[128 + r];
          m = fmaxf(e0.x, e1.x);
          wa = e0.x == -INFINITY ? 0.f : ex2(e0.x - m);
          wb = e1.x == -INFINITY ? 0.f : ex2(e1.x - m);
          l = wa * e0.y + wb * e1.y;
          ta = trow + 256;
          c0 = i * (DH / 2);
          c1 = c0 + DH / 2;
        }
        auto columns = [&](int c, float* o) {  // columns c .. c+15 of the row
          tmem_ld_32x32b_x16(ta + c, reinterpret_cast<uint32_t*>(o));
          tmem_ld_wait();
          if (two) {
            uint32_t u[16];
            tmem_ld_32x32b_x16(tB + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = o[e] * wa + __uint_as_float(u[e]) * wb;
          }
        };
        uint16_t* dst = static_cast<uint16_t*>(a.out) +
                        ((int64_t)(g.s.q0 + tok) * a.H + (int64_t)g.head * a.g + row % a.g) * DH;
        // kCommon: the row's sums as they are; kOwn: joined with those
        const int64_t qrow = ((int64_t)g.head * a.total_q + g.s.q0 + tok0) * a.g + row;
        const bool joins = on && common_keys(g.s) > 0;
        auto finish = [&](float max, float sum) {  // what `put` multiplies with: own sums, and common ones
          if constexpr (KEYS == kCommon) {
            if (on && c0 == 0) a.common_ml[qrow] = make_float2(max, sum);
            return make_float2(1.f, 0.f);
          }
          if (joins) {
            const CommonPart p(__ldcg(a.common_ml + qrow), max, sum);
            const float inv = p.sum == 0.f ? 0.f : 1.f / p.sum;
            return make_float2(p.own * inv, p.theirs * inv);
          }
          return make_float2(sum == 0.f ? 0.f : 1.f / sum, 0.f);
        };
        auto put = [&](int c, float* o, float2 w) {
          if constexpr (KEYS == kCommon) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(a.common_o + qrow * DH + c + e * 4) =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            return;
          }
          const float inv = w.x;
          if constexpr (KEYS == kOwn) {
            if (joins) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(a.common_o + qrow * DH + c + e * 4));
                o[4 * e] = o[4 * e] * inv + f.x * w.y;
                o[4 * e + 1] = o[4 * e + 1] * inv + f.y * w.y;
                o[4 * e + 2] = o[4 * e + 2] * inv + f.z * w.y;
                o[4 * e + 3] = o[4 * e + 3] * inv + f.w * w.y;
              }
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<uint4*>(dst + c + e * 8) =
                    make_uint4(pack2_bf16(o[8 * e], o[8 * e + 1]), pack2_bf16(o[8 * e + 2], o[8 * e + 3]),
                               pack2_bf16(o[8 * e + 4], o[8 * e + 5]), pack2_bf16(o[8 * e + 6], o[8 * e + 7]));
              return;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<uint4*>(dst + c + e * 8) =
                make_uint4(pack2_bf16(o[8 * e] * inv, o[8 * e + 1] * inv), pack2_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                           pack2_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                           pack2_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        };
        if (nt == g.tiles) {
          if constexpr (KEYS == kCommon)
            if (on && c0 == 0) a.parts[qrow] = kNoJoin;
          const float2 inv = finish(m, l);
#pragma unroll 1
          for (int c = c0; c < c1; c += 16) {
            float o[16];
            columns(c, o);
            if (on) put(c, o, inv);
          }
          tc_fence_before();
        } else {
          // a partial: four columns of a row in 16 bytes, rows side by side; then (m, l)
          int first, last;
          unit_shares<kCost>(g, total, grid, first, last);
          const int pi = wide ? i : 0;
          const int64_t unit_x = g.unit_x;
          auto part = [&](int c) {
            return a.part + ((int64_t)part_slot(unit_x, c, total, grid) * 2 + pi) * G::part_floats;
          };
          float* mine = part(blockIdx.x);
#pragma unroll 1
          for (int c = c0; c < c1; c += 16) {
            float o[16];
            columns(c, o);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (on)
                *reinterpret_cast<float4*>(mine + ((c / 4 + e) * 128 + r) * 4) =
                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          tc_fence_before();
          if (pi == i) *reinterpret_cast<float2*>(mine + 128 * DH + 2 * r) = make_float2(m, l);
          if constexpr (KEYS == kCommon) {  // the next launch adds them
            if (on && pi == i && g.t0 == 0)
              a.parts[qrow] = parts_word(r, pi, part_slot(unit_x, first, total, grid) & 1, first, last - first + 1);
          } else {
            if (wide) bar_lane(i); else bar_all();
            if (r == 0 && pi == i) {
              const int before = arrive_acq_rel(a.counters + first * 2 + i);
              s_flag[i] = before == last - first;
              if (before == last - first) a.counters[first * 2 + i] = 0;  // ready for the next call
            }
            if (wide) bar_lane(i); else bar_all();
          }
          if (KEYS != kCommon && s_flag[pi] && on) {
            float M = -INFINITY, sum = 0.f;
            for (int c = first; c <= last; ++c) {
              const float2 e = __ldcg(reinterpret_cast<const float2*>(part(c) + 128 * DH + 2 * r));
              const float N = fmaxf(M, e.x);
              if (N != -INFINITY) sum = sum * ex2(M - N) + e.y * ex2(e.x - N);
              M = N;
            }
            const float2 inv = finish(M, sum);
            constexpr int kCols = DH == 128 ? 64 : 32;  // a partial's columns in flight
#pragma unroll 1
            for (int c = c0; c < c1; c += kCols) {
              float acc[kCols];
#pragma unroll
              for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
              for (int k = first; k <= last; ++k) {
                const float* pt = part(k);
                const float pm = __ldcg(pt + 128 * DH + 2 * r);
                float4 f[kCols / 4];
#pragma unroll
                for (int e = 0; e < kCols / 4; ++e)
                  f[e] = __ldcg(reinterpret_cast<const float4*>(pt + ((c / 4 + e) * 128 + r) * 4));
                if (pm == -INFINITY) continue;
                const float w = ex2(pm - M);
#pragma unroll
                for (int e = 0; e < kCols / 4; ++e) {
                  acc[4 * e] += w * f[e].x;
                  acc[4 * e + 1] += w * f[e].y;
                  acc[4 * e + 2] += w * f[e].z;
                  acc[4 * e + 3] += w * f[e].w;
                }
              }
#pragma unroll
              for (int e = 0; e < kCols; e += 16) put(c + e, acc + e, inv);
            }
          }
          __syncwarp();
        }
        if (!wide) bar_all();  // everyone has read both lanes and the rows' words
        it += nt;
        // another unit with a tile before x1?
        if (g.unit_x + g.tiles + 2 * kCost >= x1) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort_flag) set_err(a.err, MEDUSA_DEVERR_TIMEOUT);
}

template <int DH, bool NARROW, bool FINE, Keys KEYS>
int run_chunk(const PagedAttnArgs& a, const PagedKernels& k) {
  CUtensorMap tmQ, tmQl, tmK, tmV;
  const int most = key_box(ChunkCfg<DH, NARROW, KEYS>::KT), box = a.p.page_size < most ? a.p.page_size : most;
  const int64_t rows = (int64_t)a.total_q * a.H;
  if (!make_rows_map(&tmQ, a.q_rot, rows, DH, 128) ||
      !make_rows_map(&tmQl, static_cast<uint16_t*>(a.q_rot) + a.q_low, rows, DH, 128) || !make_pool_map(&tmK, a.k_pages, a, DH, box) || !make_pool_map(&tmV, a.v_pages, a, DH, box))
    return fail(MEDUSA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", k.name);
  auto* fn = paged_chunk_kernel<DH, NARROW, FINE, KEYS>;
  static std::atomic<uint64_t> done{0};
  // the registers' redistribution would wait for ever if the block had fewer to give
  if (int rc = prepare_kernel(reinterpret_cast<const void*>(fn), ChunkCfg<DH, NARROW, KEYS>::smem, kLaunchRegs, kSmemBase, &done,
                              k.name))
    return rc;
  launch_after(fn, dim3(k.sms), dim3(kThreads), ChunkCfg<DH, NARROW, KEYS>::smem, k.stream, tmQ, tmQl, tmK, tmV, a);
  return check_launch(k.name);
}

}  // namespace chunk
}  // namespace

template <Keys KEYS>
int launch_paged_chunk(const PagedAttnArgs& a, int Dh, const PagedKernels& k) {
  // a group's rows are those of all its sequences
  if ((int64_t)(KEYS == kCommon ? a.total_q : a.max_new) * a.g <= 128)
    return Dh == 64 ? chunk::run_chunk<64, true, true, KEYS>(a, k) : chunk::run_chunk<128, true, true, KEYS>(a, k);
  // the others of a group do not make a sequence's weights less exact
  if constexpr (KEYS == kCommon)
    if ((int64_t)a.max_new * a.g <= 128)
      return Dh == 64 ? chunk::run_chunk<64, false, true, KEYS>(a, k) : chunk::run_chunk<128, false, true, KEYS>(a, k);
  return Dh == 64 ? chunk::run_chunk<64, false, false, KEYS>(a, k) : chunk::run_chunk<128, false, false, KEYS>(a, k);
}

}  // namespace medusa

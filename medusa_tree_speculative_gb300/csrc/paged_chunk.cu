// Chunk attention over the paged cache for many query rows, bf16, on the
// tensor cores (tcgen05, accumulators in tensor memory).
//
// A block of up to 256 query rows is two MMA tiles of 128 rows ("lanes" 0 and
// 1), and a tile of 128 keys costs each lane two products,
//   S = Q K^T  (128 x 128 x Dh)   and   O += P V  (128 x Dh x 128),
// 1024 cycles of the SM's tensor core together at Dh = 128.  While one lane's
// scores are exponentiated, the tensor core works for the other: the issuing
// thread's order is PV0(j), QK0(j+1), PV1(j), QK1(j+1), ..., so a lane's
// softmax has the other lane's two products, 1024 cycles, to hide behind.  The
// kernel is bound by the tensor core where that holds.
//   * warps 0-3 and 4-7 are the lanes' softmax: a thread per query row (its
//     tensor-memory lane) reads 128 scores, and writes P = 2^(S - m) in bf16
//     over them in tensor memory; no exchange between threads.
//   * O stays in tensor memory.  The base m of a row only moves when the
//     row's maximum passes it by more than 8 (P is at most 2^8, its sum is
//     kept in 32 bits), so O is rescaled a few times per row and not per tile.
//   * a warp loads keys and values by TMA, page by page, into a ring of
//     slots; a thread issues the MMAs and the query tiles' loads.
// A block of at most 128 rows has one query tile: the lanes then take the key
// tiles in turn, with the same queries, and their results are joined at the
// segment's end.
// Queries come rotated and scaled from the launch before this one, which also
// appends the chunk; P is rounded to bf16, as the queries are (2^-8 relative
// each, independent from element to element): the MMA takes both factors in
// one type, and the values are bf16.
// MMAs that one thread issues run in issue order on the CTA's tensor core:
// QK(j+1) may overwrite the columns from which PV(j), issued before it, reads
// P.
#include "paged_attn.cuh"
#include "sm100.cuh"

namespace medusa {
namespace {

using namespace sm100;

constexpr int RB = 256, KT = 128;
constexpr int kThreads = 384;  // two softmax groups; the load warp, the MMA warp and two idle ones
// Registers: the block starts with 168 a thread (384 x 168 = 64512); the
// softmax threads, which hold 128 scores each, then take what the third group
// gives up: 256 x 208 + 128 x 88 = 64512.
constexpr int kLaunchRegs = 168, kSoftRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "registers");
constexpr uint32_t kTmemCols = 512;

template <int DH>
struct Cfg {
  static constexpr int kHalves = DH / 64;
  static constexpr uint32_t kHalf = 128 * 128;          // 128 rows of one swizzle span
  static constexpr uint32_t kTile = kHalf * kHalves;    // 128 rows x DH bf16
  static constexpr int kSlots = DH == 128 ? 5 : 10;
  static constexpr uint32_t kRingOff = 2 * kTile;
  static constexpr uint32_t kBarOff = kRingOff + kSlots * kTile;
  static constexpr int kBars = 2 * kSlots + 2 + 2 + 2 + 1 + 1;
  static constexpr uint32_t kPlanOff = (kBarOff + kBars * 8 + 16 + 15) & ~15u;
  static constexpr uint32_t kMlOff = (kPlanOff + sizeof(Plan) + 15) & ~15u;  // [2 lanes][128 rows] (max, sum)
  static constexpr size_t smem = kMlOff + 2 * 128 * 8;
  static_assert(smem <= 232448, "shared memory");
  static constexpr int part_floats = 128 * DH + 2 * 128;  // one lane's partial
  static_assert(sizeof(PlanScratch) <= kSlots * kTile, "the plan's scratch lies in the ring");
};

MDEV uint64_t desc_mnmajor(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
MDEV void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
MDEV void bar_group(int lane_id) {
  if (lane_id == 0) asm volatile("bar.sync 1, 128;\n" ::: "memory");
  else asm volatile("bar.sync 2, 128;\n" ::: "memory");
}
MDEV void bar_both() { asm volatile("bar.sync 3, 256;\n" ::: "memory"); }
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
MDEV void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedAttnArgs a) {
  using G = Cfg<DH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {  // the swizzle's atoms: there is no room to round the address up
    if (threadIdx.x == 0) set_err(a.err, MEDUSA_DEVERR_TIMEOUT);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kBarOff);  // [slots] TMA -> MMA
  uint64_t* empty = full + G::kSlots;                               // [slots] MMA -> TMA
  uint64_t* s_full = empty + G::kSlots;                             // [2] MMA -> softmax: scores
  uint64_t* p_full = s_full + 2;                                    // [2] softmax -> MMA: P written, O rescaled
  uint64_t* pv_done = p_full + 2;                                   // [2] MMA -> softmax: O up to date
  uint64_t* q_full = pv_done + 2;
  uint64_t* all_done = q_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + 1);
  int* s_abort = reinterpret_cast<int*>(tmem_slot + 1);
  int* s_flag = s_abort + 1;  // [2]
  Plan& pl = *reinterpret_cast<Plan*>(smem + G::kPlanOff);
  PlanScratch& sc = *reinterpret_cast<PlanScratch*>(smem + G::kRingOff);
  float2* xml = reinterpret_cast<float2*>(smem + G::kMlOff);
  volatile int* abort_flag = s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(all_done, 1);
    fence_barrier_init();
    *s_abort = 0;
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  int64_t x0, x1;
  make_plan<kThreads, RB, KT>(a, sc, pl, x0, x1);
  const int64_t total = pl.total, grid = min((int64_t)gridDim.x, total);
  Segment sg;
  if (x0 < x1) seek_segment<RB, KT>(a, sc, x0, x1, sg);
  fence_smem_async();  // the scratch was read and written; the ring's copies follow
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tb = RB / a.g;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == 8 && x0 < x1) {
      // ------------------------------------------------ keys and values
      asm volatile("fence.proxy.async.global;\n" ::: "memory");  // the appended tokens, written by the launch before
      const int box = min(a.p.page_size, KT), runs = KT / box;
      const int op_run = lane / G::kHalves, op_half = lane % G::kHalves;
      const bool mine = op_run < runs;
      const int nowhere = (a.p.num_pages * a.Hkv) << a.p.shift;  // past the pool: reads zeros
      int n = 0;
      for (int64_t x = x0;;) {
        const SeqInfo& s = sg.s;
        const int nkeys = s.L + s.n;
        for (int t = sg.t0; t < sg.t1; ++t) {
          const int key = t * KT + op_run * box;
          int y = nowhere;
          if (mine && key < nkeys) {
            const int page = a.p.table[(int64_t)s.row * a.p.max_pages + (key >> a.p.shift)];
            if (page_ok(a.p, page)) y = (int)page_line(a.p, page, a.Hkv, sg.head, key & (a.p.page_size - 1));
            else set_err(a.err, MEDUSA_DEVERR_PAGE);
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int sl = n % G::kSlots;
            paged_wait(&empty[sl], ((uint32_t)(n / G::kSlots) & 1u) ^ 1u, abort_flag);
            if (lane == 0) mbar_expect_tx(&full[sl], G::kTile);
            __syncwarp();
            if (mine)
              tma_load_2d(smem + G::kRingOff + sl * G::kTile + op_half * G::kHalf + op_run * box * 128,
                          kv ? &tmV : &tmK, &full[sl], op_half * 64, y);
          }
        }
        x += sg.t1 - sg.t0;
        if (x >= x1) break;
        next_segment<RB, KT>(a, pl, x, x1, sg);
      }
      // the copies in flight land before the CTA can end, whatever happened
      for (int j = max(0, n - G::kSlots); j < n; ++j)
        if (!mbar_wait(&full[j % G::kSlots], (uint32_t)(j / G::kSlots) & 1u)) *abort_flag = 1;
    } else if (warp == 9 && x0 < x1) {
      // ------------------------------------------------ MMAs and query tiles
      if (lane == 0) {
        const uint32_t idS = idesc_bf16_f32(128, KT);
        const uint32_t idPV = idesc_bf16_f32(128, DH) | (1u << 16);  // V as stored, keys x values: MN-major
        int nq = 0, it = 0;
        uint32_t cnt[2] = {0, 0};  // this lane's tiles so far
        auto live_of = [&](const Segment& g) { return min(tb, g.s.n - g.u * tb) * a.g; };
        auto load_q = [&](const Segment& g) {
          const int tiles = live_of(g) > 128 ? 2 : 1;
          const int y = (g.head * a.total_q + g.s.q0 + g.u * tb) * a.g;
          mbar_expect_tx(q_full, tiles * G::kTile);
          for (int i = 0; i < tiles; ++i)
            for (int h = 0; h < G::kHalves; ++h)
              tma_load_2d(smem + i * G::kTile + h * G::kHalf, &tmQ, q_full, h * 64, y + i * 128);
        };
        auto wait_kv = [&](int n) { paged_wait(&full[n % G::kSlots], (uint32_t)(n / G::kSlots) & 1u, abort_flag); };
        auto free_kv = [&](int n) { umma_commit(&empty[n % G::kSlots]); };
        auto qk = [&](int i, int qt, int t) {  // lane i's scores of tile t (of the CTA's count) from query tile qt
          const uint32_t k = sbase + G::kRingOff + (uint32_t)((2 * t) % G::kSlots) * G::kTile;
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint64_t da = desc_kmajor_sw128(sbase + qt * G::kTile + (kk >> 2) * G::kHalf) + (uint64_t)((kk & 3) * 2);
            const uint64_t db = desc_kmajor_sw128(k + (kk >> 2) * G::kHalf) + (uint64_t)((kk & 3) * 2);
            umma_bf16(tmem + i * 128, da, db, idS, kk != 0);
          }
          umma_commit(&s_full[i]);
        };
        auto pv = [&](int i, int t, bool add) {
          const uint32_t v = sbase + G::kRingOff + (uint32_t)((2 * t + 1) % G::kSlots) * G::kTile;
#pragma unroll
          for (int j = 0; j < KT / 16; ++j)
            umma_bf16_ts(tmem + 256 + i * 128, tmem + i * 128 + j * 8, desc_mnmajor(v + j * 2048, G::kHalf, 1024), idPV,
                         add || j != 0);
          umma_commit(&pv_done[i]);
        };
        auto wait_p = [&](int i) {
          paged_wait(&p_full[i], cnt[i] & 1u, abort_flag);
          ++cnt[i];
          tc_fence_after();
        };
        load_q(sg);
        for (int64_t x = x0;; ++nq) {
          const int nt = sg.t1 - sg.t0;
          const bool wide = live_of(sg) > 128;
          paged_wait(q_full, (uint32_t)nq & 1u, abort_flag);
          if (wide) {
            wait_kv(2 * it);
            tc_fence_after();
            qk(0, 0, it);
            qk(1, 1, it);
            free_kv(2 * it);
            for (int j = 0; j < nt; ++j) {
              const bool more = j + 1 < nt;
              wait_p(0);
              wait_kv(2 * (it + j) + 1);
              pv(0, it + j, j > 0);
              if (more) {
                wait_kv(2 * (it + j + 1));
                tc_fence_after();
                qk(0, 0, it + j + 1);
              }
              wait_p(1);
              pv(1, it + j, j > 0);
              free_kv(2 * (it + j) + 1);
              if (more) {
                qk(1, 1, it + j + 1);
                free_kv(2 * (it + j + 1));
              }
            }
          } else {
            for (int i = 0; i < 2 && i < nt; ++i) {
              wait_kv(2 * (it + i));
              tc_fence_after();
              qk(i, 0, it + i);
              free_kv(2 * (it + i));
            }
            for (int j = 0; j < nt; ++j) {
              const int i = j & 1;
              wait_p(i);
              wait_kv(2 * (it + j) + 1);
              pv(i, it + j, j > 1);
              free_kv(2 * (it + j) + 1);
              if (j + 2 < nt) {
                wait_kv(2 * (it + j + 2));
                tc_fence_after();
                qk(i, 0, it + j + 2);
                free_kv(2 * (it + j + 2));
              }
            }
          }
          it += nt;
          x += nt;
          if (x >= x1) break;
          next_segment<RB, KT>(a, pl, x, x1, sg);
          load_q(sg);  // the last waits for P say that every product of the old queries is done
        }
        umma_commit(all_done);
        if (!mbar_wait(all_done, 0)) *abort_flag = 1;
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    if (x0 < x1) {
      // ------------------------------------------------ softmax of lane `i`
      const int i = warp >> 2, r = tid & 127;
      const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      const uint32_t tS = trow + i * 128, tO = trow + 256 + i * 128;
      uint32_t cnt = 0;
      int it = 0;
      for (int64_t x = x0;;) {
        const SeqInfo s = sg.s;
        const int nt = sg.t1 - sg.t0, tok0 = sg.u * tb, live = min(tb, s.n - tok0) * a.g, nkeys = s.L + s.n;
        const bool wide = live > 128;
        const int row = wide ? i * 128 + r : r;
        const bool on = row < live;
        const int tok = min(tok0 + row / a.g, s.n - 1);
        const int lim = a.T ? nkeys : s.L + tok + 1;  // causal: keys below this
        const uint32_t* anc = a.anc + (int64_t)tok * a.W;
        float m = -INFINITY, l = 0.f;
        int done = 0;  // this lane's tiles of the segment
        for (int j = wide ? 0 : i; j < nt; j += wide ? 1 : 2, ++done) {
          const int t = sg.t0 + j, key0 = t * KT;
          paged_wait(&s_full[i], cnt & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
          uint32_t v[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, v + c * 32);
          tmem_ld_wait();
          if (a.T == 0) {
            if (__any_sync(0xffffffffu, lim < key0 + KT)) {
              const int d = lim - key0;
#pragma unroll
              for (int e = 0; e < 128; ++e) v[e] = e < d ? v[e] : 0xff800000u;
            }
          } else if (key0 + KT > s.L) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int j0 = key0 + 32 * w, n0 = j0 - s.L;  // tree node of bit 0 (negative: prefix keys first)
              uint32_t bits = 0xffffffffu;
              if (n0 >= 0) {
                const int q = n0 >> 5, sh = n0 & 31;
                const uint32_t lo = q < a.W ? __ldg(anc + q) : 0u, hi = q + 1 < a.W ? __ldg(anc + q + 1) : 0u;
                bits = sh ? (lo >> sh) | (hi << (32 - sh)) : lo;
              } else if (n0 > -32) {
                bits = (0xffffffffu >> (32 + n0)) | (__ldg(anc) << (-n0));
              }
              const int past = nkeys - j0;  // nothing past the sequence
              if (past < 32) bits &= past > 0 ? (1u << past) - 1u : 0u;
#pragma unroll
              for (int e = 0; e < 32; ++e) v[32 * w + e] = (bits >> e & 1u) ? v[32 * w + e] : 0xff800000u;
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(v[e + 2 * k])), __uint_as_float(v[e + 2 * k + 1]));
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool far = mt > m + 8.f;
          if (__any_sync(0xffffffffu, far)) {
            const float mn = far ? mt : m;
            const float al = m == -INFINITY ? 0.f : ex2(m - mn);
            if (done > 0) {  // O so far holds what the old base gave
              l *= al;
              paged_wait(&pv_done[i], (cnt - 1) & 1u, abort_flag);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st32(tO + c * 32, o);
              }
            }
            m = mn;
          }
          const float base = m == -INFINITY ? 0.f : m;
          float sa[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float u = __uint_as_float(v[64 * h + 2 * e]), w = __uint_as_float(v[64 * h + 2 * e + 1]);
              add2(u, w, -base, -base);
              u = ex2(u);
              w = ex2(w);
              add2(sa[e & 1], sb[e & 1], u, w);
              p[e] = pack2_bf16(u, w);
            }
            tmem_st32(tS + h * 32, p);
          }
          tmem_st_wait();
          l += (sa[0] + sb[0]) + (sa[1] + sb[1]);
          // value rows past the sequence hold whatever the page does: zeros
          // (lane 0's P is waited for before either lane's product)
          if (key0 + KT > nkeys && (i == 0 || !wide)) {
            const int n = 2 * (it + j) + 1;
            paged_wait(&full[n % G::kSlots], (uint32_t)(n / G::kSlots) & 1u, abort_flag);
            if (key0 + r >= nkeys) {
#pragma unroll
              for (int c = 0; c < G::kHalves * 8; ++c)
                *reinterpret_cast<uint4*>(smem + G::kRingOff + (n % G::kSlots) * G::kTile + (c >> 3) * G::kHalf +
                                          r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_smem_async();
          }
          tc_fence_before();
          mbar_arrive(&p_full[i]);
          ++cnt;
        }
        if (done > 0) {
          paged_wait(&pv_done[i], (cnt - 1) & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
        }
        // One query tile: the lanes' results are joined, half of the columns
        // by each group (both read the same tensor-memory lanes).
        int c0 = 0, c1 = DH / 32;
        float wa = 1.f, wb = 0.f;
        uint32_t ta = tO;
        const uint32_t tB = trow + 256 + 128;
        const bool two = !wide && nt > 1;
        if (!wide) {
          xml[i * 128 + r] = make_float2(m, l);
          tc_fence_before();
          bar_both();
          tc_fence_after();
          const float2 e0 = xml[r], e1 = xml[128 + r];
          m = fmaxf(e0.x, e1.x);
          wa = e0.x == -INFINITY ? 0.f : ex2(e0.x - m);
          wb = e1.x == -INFINITY ? 0.f : ex2(e1.x - m);
          l = wa * e0.y + wb * e1.y;
          ta = trow + 256;
          c0 = i * (DH / 64);
          c1 = c0 + DH / 64;
        }
        auto columns = [&](int c, float* o) {  // columns 32c .. 32c+31 of the row
          tmem_ld32(ta + c * 32, reinterpret_cast<uint32_t*>(o));
          tmem_ld_wait();
          if (two) {
            uint32_t u[32];
            tmem_ld32(tB + c * 32, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * wa + __uint_as_float(u[e]) * wb;
          }
        };
        auto put = [&](int c, const float* o, float inv) {
          uint16_t* dst = static_cast<uint16_t*>(a.out) +
                          ((int64_t)(s.q0 + tok) * a.H + (int64_t)sg.head * a.g + row % a.g) * DH + c * 32;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(dst + e * 8) =
                make_uint4(pack2_bf16(o[8 * e] * inv, o[8 * e + 1] * inv), pack2_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                           pack2_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                           pack2_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        };
        if (nt == sg.tiles) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float o[32];
            columns(c, o);
            if (on) put(c, o, inv);
          }
          tc_fence_before();
          if (!wide) bar_both();  // both groups have read both lanes
        } else {
          // a partial: four columns of a row in 16 bytes, rows side by side; then (m, l)
          int first, last;
          unit_shares(sg, total, grid, first, last);
          const int pi = wide ? i : 0;
          auto part = [&](int c) {
            return a.part + ((int64_t)part_slot(sg.unit_x, c, total, grid) * 2 + pi) * G::part_floats;
          };
          float* mine = part(blockIdx.x);
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float o[32];
            columns(c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (on)
                *reinterpret_cast<float4*>(mine + ((c * 8 + e) * 128 + r) * 4) =
                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          tc_fence_before();
          if (wide || i == 0) *reinterpret_cast<float2*>(mine + 128 * DH + 2 * r) = make_float2(m, l);
          if (wide) bar_group(i); else bar_both();
          if (r == 0 && pi == i) {
            const int before = arrive_acq_rel(a.counters + first * 2 + i);
            s_flag[i] = before == last - first;
            if (before == last - first) a.counters[first * 2 + i] = 0;  // ready for the next call
          }
          if (wide) bar_group(i); else bar_both();
          if (s_flag[pi] && on) {
            float M = -INFINITY, sum = 0.f;
            for (int c = first; c <= last; ++c) {
              const float2 e = __ldcg(reinterpret_cast<const float2*>(part(c) + 128 * DH + 2 * r));
              const float N = fmaxf(M, e.x);
              if (N != -INFINITY) sum = sum * ex2(M - N) + e.y * ex2(e.x - N);
              M = N;
            }
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
              float acc[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) acc[e] = 0.f;
              for (int k = first; k <= last; ++k) {
                const float* pt = part(k);
                const float pm = __ldcg(pt + 128 * DH + 2 * r);
                if (pm == -INFINITY) continue;
                const float w = ex2(pm - M);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 f = __ldcg(reinterpret_cast<const float4*>(pt + ((c * 8 + e) * 128 + r) * 4));
                  acc[4 * e] += w * f.x;
                  acc[4 * e + 1] += w * f.y;
                  acc[4 * e + 2] += w * f.z;
                  acc[4 * e + 3] += w * f.w;
                }
              }
              put(c, acc, inv);
            }
          }
          __syncwarp();
        }
        it += nt;
        x += nt;
        if (x >= x1) break;
        next_segment<RB, KT>(a, pl, x, x1, sg);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort_flag) set_err(a.err, MEDUSA_DEVERR_TIMEOUT);
}

template <int DH>
int run(const PagedAttnArgs& a, const PagedKernels& k) {
  CUtensorMap tmQ, tmK, tmV;
  const int box = a.p.page_size < KT ? a.p.page_size : KT;
  if (!make_rows_map(&tmQ, a.q_rot, (int64_t)a.total_q * a.H, DH, 128) ||
      !make_pool_map(&tmK, a.k_pages, a, DH, box) || !make_pool_map(&tmV, a.v_pages, a, DH, box))
    return fail(MEDUSA_ERR_CUDA, "medusa_paged_attn: cuTensorMapEncodeTiled failed");
  auto* fn = paged_chunk_kernel<DH>;
  static std::atomic<uint64_t> done{0};
  // the registers' redistribution would wait for ever if the block had fewer to give
  if (int rc = prepare_kernel(reinterpret_cast<const void*>(fn), Cfg<DH>::smem, kLaunchRegs, &done, "medusa_paged_attn"))
    return rc;
  launch_kernel(fn, dim3(k.sms), dim3(kThreads), Cfg<DH>::smem, k.stream, tmQ, tmK, tmV, a);
  return check_launch("medusa_paged_attn");
}

}  // namespace

size_t paged_chunk_part_bytes(int Dh, int sms) { return (size_t)sms * 4 * (128 * Dh + 2 * 128) * 4; }
int launch_paged_chunk(const PagedAttnArgs& a, int Dh, const PagedKernels& k) {
  return Dh == 64 ? run<64>(a, k) : run<128>(a, k);
}

}  // namespace medusa

// Chunk attention over the paged cache for few query rows, bf16: a sequence's
// new tokens times the query heads of a key head fill at most one 16-row MMA
// tile (single tokens, with up to 16 heads per key head, and short drafts).
//
// Every key and value is read once for up to 16 rows, 16 operations per byte:
// the kernel is bound by memory, and what matters is that loads never pause.
// One CTA per SM holds six warps:
//   * the load warp brings tiles of 64 keys and values into a ring of stages
//     (160 KB, about 3.5 us of the SM's share of the memory's rate) by TMA, a
//     lane per (page, pool), both 64-column halves of a line in one copy, and
//     runs on over the segments of the CTA's list;
//   * the query warp rotates the next segment's query rows while the present
//     one runs (two buffers).  Queries and the weights P are kept as two bf16
//     parts, high and low (2^-16 relative together), and multiplied in two
//     MMAs: the tensor cores have time to spare here, and the result is off by
//     its own rounding only;
//   * warps 0-3 take 16 keys of each tile each: S = Q K^T and O += P V by
//     mma.sync (M = 16), the running maximum and sum per warp, no barrier among
//     them until the segment ends and their four results are joined.
// Before the loads of a tile that holds new tokens, the CTA itself (the only
// one with that tile of that key head) rotates and appends them: no separate
// launch.
// Small calls are bound by latency.  Where every row's pages hold few tiles and
// there are SMs to spare, a cluster of CL CTAs takes a unit instead: no list to
// plan, and the join goes through distributed shared memory in place of the
// workspace and its counters (one token at a prefix of 1024, 32 heads: 11.9 us
// against 16.4).
// Measured (SM clock 2070 MHz): 64 tokens with prefixes of 500 .. 8192, 32 heads
// of 128 on 8 key heads, 181 to 185 us, 6.0 TB/s (174 to 177 with pages of 32
// tokens or more: half as many copies).
#include "cluster.cuh"
#include "paged_attn.cuh"
#include "sm100.cuh"

namespace medusa {
namespace {

using namespace sm100;

constexpr int RB = 16, KT = 64, kCost = 2;  // kCost: the tiles that beginning and ending a unit costs
constexpr int kThreads = 192;
constexpr int kConsumers = 128;

template <int DH>
struct Cfg {
  static constexpr int kStages = DH == 128 ? 5 : 10;
  static constexpr uint32_t kTile = KT * DH * 2;                  // one pool's tile
  static constexpr uint32_t kRing = kStages * 2 * kTile;
  static constexpr int kQStride = DH * 2 + 16;                    // bytes of a query row (padded: no bank conflicts)
  static constexpr uint32_t kQOff = kRing;                        // [2 buffers][high, low][16 rows]
  static constexpr uint32_t kQBytes = 4 * RB * kQStride;
  static constexpr int kOStride = DH + 4;
  static constexpr uint32_t kOOff = kQOff + kQBytes;              // [4 warps][16 rows][kOStride] floats
  static constexpr uint32_t kOBytes = 4 * RB * kOStride * 4;
  static constexpr uint32_t kScratch = kOBytes > sizeof(PlanScratch) ? kOBytes : (uint32_t)sizeof(PlanScratch);
  static constexpr uint32_t kMlOff = kOOff + ((kScratch + 15) & ~15u);  // [4 warps][16 rows] (max, sum)
  static constexpr uint32_t kPlanOff = kMlOff + 4 * RB * 8;
  static constexpr uint32_t kSegOff = (kPlanOff + sizeof(Plan) + 15) & ~15u;  // [2] segments
  static constexpr uint32_t kBarOff = (kSegOff + 2 * sizeof(Segment) + 15) & ~15u;
  static constexpr uint32_t kBytes = kBarOff + (2 * kStages + 5) * 8 + 16;
  static constexpr size_t smem = 1024 + kBytes;
  static constexpr int part_floats = RB * DH + 2 * RB;
};

MDEV void bar_consumers() { asm volatile("bar.sync 1, 128;\n" ::: "memory"); }

// Lines y .. of a pool, both halves: a box of [halves][lines][64 values].
MDEV void tma_load_lines(void* dst, const CUtensorMap* map, uint64_t* bar, int y) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %3}], [%2];\n" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(y)
      : "memory");
}

// The new tokens of a segment that lie in its tiles, rotated and written to
// their pages by one warp.
template <int DH>
MDEV void append_tokens(const PagedAttnArgs& a, const Segment& g, int lane) {
  const SeqInfo& s = g.s;
  const int lo = max(0, g.t0 * KT - s.L), hi = min(s.n, g.t1 * KT - s.L);
  for (int i = lo; i < hi; ++i) {
    const int slot = s.L + i, page = page_of(a, s, slot);
    if (page < 0) continue;
    const int pos = s.L + (a.T ? min(max(__ldg(a.depth + i), 0), a.K) : i);
    const int64_t line = page_line(a.p, page, a.Hkv, g.head, slot & (a.p.page_size - 1)) * DH;
    const uint16_t* k = static_cast<const uint16_t*>(a.k_new) + (int64_t)(s.q0 + i) * a.k_stride + g.head * DH;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v_new) +
                                                          (int64_t)(s.q0 + i) * a.v_stride + g.head * DH);
    uint16_t* kd = static_cast<uint16_t*>(a.k_pages) + line;
    uint32_t* vd = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.v_pages) + line);
#pragma unroll
    for (int j = lane; j < DH / 2; j += 32) {
      const float x = bf16_bits_to_f32(k[j]), y = bf16_bits_to_f32(k[j + DH / 2]);
      const uint32_t w = v[j];
      float c, t;
      rope_cos_sin(pos, a.turns[j], c, t);
      kd[j] = f32_to_bf16_bits(x * c - y * t);
      kd[j + DH / 2] = f32_to_bf16_bits(y * c + x * t);
      vd[j] = w;
    }
  }
}

template <int DH, int CL>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ PagedAttnArgs a) {
  using G = Cfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  PlanScratch& sc = *reinterpret_cast<PlanScratch*>(smem + G::kOOff);
  Plan& pl = *reinterpret_cast<Plan*>(smem + G::kPlanOff);
  Segment* segs = reinterpret_cast<Segment*>(smem + G::kSegOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kBarOff);
  uint64_t* empty = full + G::kStages;
  uint64_t* q_full = empty + G::kStages;   // [2]
  uint64_t* q_empty = q_full + 2;          // [2]
  uint64_t* appended = q_empty + 2;
  int* s_abort = reinterpret_cast<int*>(appended + 1);
  int* s_flag = s_abort + 1;
  volatile int* abort_flag = s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 4);
    }
    mbar_init(appended, kConsumers);
    fence_barrier_init();
    *s_abort = 0;
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // rows past a segment's own keep whatever was here before: finite numbers
  for (uint32_t e = tid; e < G::kQBytes / 4; e += kThreads) reinterpret_cast<uint32_t*>(smem + G::kQOff)[e] = 0u;
  int64_t x1 = 0, total = 0, grid = 0;
  Segment sg;
  bool any;
  if constexpr (CL == 1) {
    int64_t x0;
    make_plan<kThreads, RB, KT, kCost>(a, sc, pl, x0, x1);
    total = pl.total;
    grid = min((int64_t)gridDim.x, total);
    any = x0 < x1 && seek_segment<RB, KT, kCost>(a, sc, x0, x1, sg);
    __syncthreads();  // the scratch becomes the warps' results
  } else {
    // a cluster per unit, which is all of a sequence's rows of a key head
    const int unit = blockIdx.x / CL, rank = (int)cluster_rank();
    sg.b = unit / a.Hkv;
    sg.head = unit - sg.b * a.Hkv;
    sg.u = 0;
    sg.m = 1;
    sg.unit_x = 0;
    int code, start0 = 0, start1 = 0;  // thread b looks at sequence b: at most a unit per two SMs
    if (tid < a.B) {
      start0 = a.q_start[tid];
      start1 = a.q_start[tid + 1];
    }
    bool ok = seq_info(a, sg.b, sg.s, code), twice = false;
    if (a.rows && ok)
      for (int j = tid; j < sg.b; j += kThreads) twice |= a.rows[j] == sg.s.row && a.q_start[j + 1] > a.q_start[j];
    if (__syncthreads_or(twice)) {
      ok = false;
      code = MEDUSA_DEVERR_ROW;
    }
    if (__syncthreads_or(start1 < start0)) ok = false;  // the sequence where they decrease reports it
    if (code && sg.head == 0 && rank == 0 && tid == 0) set_err(a.err, code);
    if (!ok) return;  // the whole cluster
    sg.tiles = (sg.s.L + sg.s.n + KT - 1) / KT;
    sg.t0 = (int)((int64_t)rank * sg.tiles / CL);
    sg.t1 = (int)((int64_t)(rank + 1) * sg.tiles / CL);
    any = sg.t0 < sg.t1;
  }
  auto next = [&](Segment& g) {
    if constexpr (CL == 1) return next_segment<RB, KT, kCost>(a, pl, x1, g);
    else return false;
  };
  // a cluster's join: every CTA's (max, sum) and sums of its tiles, at these
  // places (the queries are in registers by then)
  float* join = reinterpret_cast<float*>(smem + G::kQOff);
  float2* join_ml = reinterpret_cast<float2*>(smem + G::kQOff + RB * G::kOStride * 4);
  if constexpr (CL > 1) {
    static_assert(RB * G::kOStride * 4 + RB * 8 <= G::kQBytes, "the join's place");
    if (!any && tid < RB) join_ml[tid] = make_float2(-INFINITY, 0.f);
  }
  if (any) {
    if (warp == 4) {
      // ------------------------------------------------ loads
      const int box = min(a.p.page_size, KT), runs = KT / box;  // runs of keys in one page each
      const int op_run = lane >> 1, op_v = lane & 1;
      const bool mine = op_run < runs;
      const int nowhere = a.p.num_pages * a.Hkv << a.p.shift;  // past the pool: reads zeros
      const CUtensorMap* map = op_v ? &tmV : &tmK;
      bool told = false;
      int it = 0;
      while (true) {
        const SeqInfo& s = sg.s;
        const int nkeys = s.L + s.n;
        for (int t = sg.t0; t < sg.t1; ++t, ++it) {
          const int st = it % G::kStages;
          if (!told && (t + 1) * KT > s.L) {  // this tile holds new tokens
            paged_wait(appended, 0, abort_flag);
            told = true;
          }
          const int key = t * KT + op_run * box;
          int y = nowhere;
          if (mine && key < nkeys) {
            const int page = a.p.table[(int64_t)s.row * a.p.max_pages + (key >> a.p.shift)];
            if (page_ok(a.p, page)) y = (int)page_line(a.p, page, a.Hkv, sg.head, key & (a.p.page_size - 1));
            else set_err(a.err, MEDUSA_DEVERR_PAGE);
          }
          paged_wait(&empty[st], ((uint32_t)(it / G::kStages) & 1u) ^ 1u, abort_flag);
          if (lane == 0) mbar_expect_tx(&full[st], 2 * G::kTile);
          __syncwarp();
          if (mine)
            tma_load_lines(smem + st * 2 * G::kTile + op_v * G::kTile + op_run * box * DH * 2, map, &full[st], y);
        }
        if (!next(sg)) break;
      }
      // the copies in flight land before the CTA can end, whatever happened
      for (int j = max(0, it - G::kStages); j < it; ++j)
        if (!mbar_wait(&full[j % G::kStages], (uint32_t)(j / G::kStages) & 1u)) *abort_flag = 1;
    } else if (warp == 5) {
      // ------------------------------------------------ queries
      int n = 0;
      for (;; ++n) {
        const int bf = n & 1;
        const int live = sg.s.n * a.g;
        paged_wait(&q_empty[bf], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort_flag);
        uint8_t* qb = smem + G::kQOff + bf * 2 * RB * G::kQStride;
        for (int j = lane; j < DH / 2; j += 32) {
          int tok = -1;
          float c = 0.f, t = 0.f;
          for (int r = 0; r < live; ++r) {
            const int i = r / a.g;
            const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(sg.s.q0 + i) * a.q_stride +
                                (int64_t)(sg.head * a.g + r - i * a.g) * DH;
            const float u = bf16_bits_to_f32(q[j]), v = bf16_bits_to_f32(q[j + DH / 2]);
            if (i != tok) {
              tok = i;
              rope_cos_sin(sg.s.L + (a.T ? min(max(__ldg(a.depth + i), 0), a.K) : i), a.turns[j], c, t);
            }
            const float p0 = (u * c - v * t) * a.qscale, p1 = (v * c + u * t) * a.qscale;
            uint16_t* hi = reinterpret_cast<uint16_t*>(qb + r * G::kQStride);
            uint16_t* lo = reinterpret_cast<uint16_t*>(qb + (RB + r) * G::kQStride);
            hi[j] = f32_to_bf16_bits(p0);
            hi[j + DH / 2] = f32_to_bf16_bits(p1);
            lo[j] = f32_to_bf16_bits(p0 - bf16_bits_to_f32(hi[j]));
            lo[j + DH / 2] = f32_to_bf16_bits(p1 - bf16_bits_to_f32(hi[j + DH / 2]));
          }
        }
        if (lane == 0) segs[bf] = sg;
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[bf]);
        if (!next(sg)) break;
      }
    } else {
      // ------------------------------------------------ append, then attend
      int segments;
      {
        int n = 0;
        Segment g = sg;
        do {  // segments in turn to the four warps
          if ((n++ & 3) == warp && g.t1 * KT > g.s.L) append_tokens<DH>(a, g, lane);
        } while (next(g));
        segments = n;
        asm volatile("fence.proxy.async.global;\n" ::: "memory");  // the tiles' loads read them back
        mbar_arrive(appended);
      }
      // a tile in shared memory: runs of `box` keys, each [halves][box][128 bytes]
      const int box = min(a.p.page_size, KT);
      const uint32_t half = box * 128, first = (warp * 16 / box) * box * DH * 2 + (warp * 16 % box) * 128;
      const int r0 = lane >> 2, r1 = r0 + 8, kc = (lane & 3) * 2;  // this thread's rows and key columns
      int it = 0;
      for (int n = 0; n < segments; ++n) {
        const int bf = n & 1;
        paged_wait(&q_full[bf], (uint32_t)(n >> 1) & 1u, abort_flag);
        const Segment g = segs[bf];
        const SeqInfo& s = g.s;
        uint32_t qh[DH / 16][4], ql[DH / 16][4];
        {
          const uint32_t row = sbase + G::kQOff + bf * 2 * RB * G::kQStride + (lane & 15) * G::kQStride + (lane >> 4) * 16;
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            ldmatrix_x4(qh[kk], row + kk * 32);
            ldmatrix_x4(ql[kk], row + RB * G::kQStride + kk * 32);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[bf]);
        const int nkeys = s.L + s.n, live = s.n * a.g;
        const int i0 = r0 / a.g, i1 = r1 / a.g;  // tokens of the two rows
        float o[DH / 8][4];
#pragma unroll
        for (int j = 0; j < DH / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        for (int t = g.t0; t < g.t1; ++t, ++it) {
          const int st = it % G::kStages;
          paged_wait(&full[st], (uint32_t)(it / G::kStages) & 1u, abort_flag);
          const uint32_t kb = sbase + st * 2 * G::kTile + first, vb = kb + G::kTile;
          float z[2][4] = {};
          {
            const int row = (lane & 7) + (lane >> 4) * 8, ch = lane >> 3 & 1;
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              const int c = kk * 2 + ch;
              uint32_t b[4];
              ldmatrix_x4(b, kb + (c >> 3) * half + row * 128 + (((c & 7) ^ (row & 7)) << 4));
              mma_bf16_16816(z[0], qh[kk], b[0], b[1]);
              mma_bf16_16816(z[1], qh[kk], b[2], b[3]);
              mma_bf16_16816(z[0], ql[kk], b[0], b[1]);
              mma_bf16_16816(z[1], ql[kk], b[2], b[3]);
            }
          }
          const int key0 = t * KT + warp * 16;
          const bool edge = key0 + 16 > s.L;  // keys past the prefix: the mask decides
          if (edge) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int key = key0 + (e >> 2) * 8 + kc + (e & 1), i = (e & 2) ? i1 : i0;
              if (key >= nkeys || i >= s.n || !key_seen(a, s, i, key)) z[e >> 2][e & 3] = -INFINITY;
            }
          }
          float t0 = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
          float t1 = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
#pragma unroll
          for (int w = 1; w < 4; w <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, w));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, w));
          }
          if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {  // a row's maximum moves
            const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
            const float a0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), a1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int j = 0; j < DH / 8; ++j) {
              o[j][0] *= a0;
              o[j][1] *= a0;
              o[j][2] *= a1;
              o[j][3] *= a1;
            }
          }
          const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            z[j][0] = exp2f(z[j][0] - b0);
            z[j][1] = exp2f(z[j][1] - b0);
            z[j][2] = exp2f(z[j][2] - b1);
            z[j][3] = exp2f(z[j][3] - b1);
          }
          l0 += (z[0][0] + z[0][1]) + (z[1][0] + z[1][1]);
          l1 += (z[0][2] + z[0][3]) + (z[1][2] + z[1][3]);
          uint32_t ph[4], pl[4];  // the weights' two parts
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = z[e >> 1][(e & 1) * 2], w = z[e >> 1][(e & 1) * 2 + 1];
            ph[e] = pack2_bf16(u, w);
            pl[e] = pack2_bf16(u - __uint_as_float(ph[e] << 16), w - __uint_as_float(ph[e] & 0xffff0000u));
          }
          // value rows past the sequence hold whatever the page does: zeros
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (edge) {
            const int left = nkeys - key0;
            keep0 = (kc < left ? 0xffffu : 0u) | (kc + 1 < left ? 0xffff0000u : 0u);
            keep1 = (kc + 8 < left ? 0xffffu : 0u) | (kc + 9 < left ? 0xffff0000u : 0u);
          }
          const int row = (lane & 7) + (lane >> 3 & 1) * 8, ch = lane >> 4;
#pragma unroll
          for (int j = 0; j < DH / 16; ++j) {
            const int c = j * 2 + ch;
            uint32_t b[4];
            ldmatrix_x4_trans(b, vb + (c >> 3) * half + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            if (edge) {
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
            mma_bf16_16816(o[2 * j], ph, b[0], b[1]);
            mma_bf16_16816(o[2 * j + 1], ph, b[2], b[3]);
            mma_bf16_16816(o[2 * j], pl, b[0], b[1]);
            mma_bf16_16816(o[2 * j + 1], pl, b[2], b[3]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
#pragma unroll
        for (int w = 1; w < 4; w <<= 1) {
          l0 += __shfl_xor_sync(0xffffffffu, l0, w);
          l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }
        if (l0 != l0) m0 = INFINITY;  // so that no join drops a part whose scores are all NaN
        if (l1 != l1) m1 = INFINITY;
        // the four warps' results joined: eight threads per row
        bar_consumers();  // the previous segment's are read
        float* ob = reinterpret_cast<float*>(smem + G::kOOff) + warp * RB * G::kOStride;
        float2* ml = reinterpret_cast<float2*>(smem + G::kMlOff);
#pragma unroll
        for (int j = 0; j < DH / 8; ++j) {
          *reinterpret_cast<float2*>(ob + r0 * G::kOStride + j * 8 + kc) = make_float2(o[j][0], o[j][1]);
          *reinterpret_cast<float2*>(ob + r1 * G::kOStride + j * 8 + kc) = make_float2(o[j][2], o[j][3]);
        }
        if ((lane & 3) == 0) {
          ml[warp * RB + r0] = make_float2(m0, l0);
          ml[warp * RB + r1] = make_float2(m1, l1);
        }
        bar_consumers();
        const int r = tid >> 3, c0 = (tid & 7) * 4;  // columns c0 + 32 k
        float M = -INFINITY, sum = 0.f, acc[DH / 32][4] = {};
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[w * RB + r].x);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 e = ml[w * RB + r];
          const float f = e.x == -INFINITY ? 0.f : exp2f(e.x - M);
          sum += f * e.y;
          const float* src = reinterpret_cast<const float*>(smem + G::kOOff) + (w * RB + r) * G::kOStride + c0;
#pragma unroll
          for (int k = 0; k < DH / 32; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(src + 32 * k);
            acc[k][0] += f * v.x;
            acc[k][1] += f * v.y;
            acc[k][2] += f * v.z;
            acc[k][3] += f * v.w;
          }
        }
        auto put = [&]() {
          if (r >= live) return;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int i = r / a.g;
          uint16_t* dst = static_cast<uint16_t*>(a.out) +
                          ((int64_t)(s.q0 + i) * a.H + (int64_t)g.head * a.g + r - i * a.g) * DH + c0;
#pragma unroll
          for (int k = 0; k < DH / 32; ++k)
            *reinterpret_cast<uint2*>(dst + 32 * k) = make_uint2(pack2_bf16(acc[k][0] * inv, acc[k][1] * inv),
                                                                 pack2_bf16(acc[k][2] * inv, acc[k][3] * inv));
        };
        if constexpr (CL > 1) {
#pragma unroll
          for (int k = 0; k < DH / 32; ++k)
            *reinterpret_cast<float4*>(join + r * G::kOStride + c0 + 32 * k) =
                make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
          if ((tid & 7) == 0) join_ml[r] = make_float2(M, sum);
        } else if (g.t0 == 0 && g.t1 == g.tiles) {
          put();
        } else {
          int c_first, c_last;
          unit_shares<kCost>(g, total, grid, c_first, c_last);
          float* mine = a.part + (int64_t)part_slot(g.unit_x, blockIdx.x, total, grid) * G::part_floats;
          if (r < live) {
#pragma unroll
            for (int k = 0; k < DH / 32; ++k)
              *reinterpret_cast<float4*>(mine + r * DH + c0 + 32 * k) =
                  make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
            if ((tid & 7) == 0) *reinterpret_cast<float2*>(mine + RB * DH + 2 * r) = make_float2(M, sum);
          }
          bar_consumers();
          if (tid == 0) {
            const int before = arrive_acq_rel(a.counters + c_first);
            *s_flag = before == c_last - c_first;
            if (before == c_last - c_first) a.counters[c_first] = 0;  // ready for the next call
          }
          bar_consumers();
          if (*s_flag && r < live) {
            M = -INFINITY;
            sum = 0.f;
#pragma unroll
            for (int k = 0; k < DH / 32; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
            for (int c = c_first; c <= c_last; ++c) {
              const float* pt = a.part + (int64_t)part_slot(g.unit_x, c, total, grid) * G::part_floats;
              const float2 e = __ldcg(reinterpret_cast<const float2*>(pt + RB * DH + 2 * r));
              float4 v[DH / 32];
#pragma unroll
              for (int k = 0; k < DH / 32; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(pt + r * DH + c0 + 32 * k));
              const float N = fmaxf(M, e.x);
              const float f0 = M == -INFINITY ? 0.f : exp2f(M - N), f1 = e.x == -INFINITY ? 0.f : exp2f(e.x - N);
              M = N;
              sum = sum * f0 + e.y * f1;
#pragma unroll
              for (int k = 0; k < DH / 32; ++k) {
                acc[k][0] = acc[k][0] * f0 + v[k].x * f1;
                acc[k][1] = acc[k][1] * f0 + v[k].y * f1;
                acc[k][2] = acc[k][2] * f0 + v[k].z * f1;
                acc[k][3] = acc[k][3] * f0 + v[k].w * f1;
              }
            }
            put();
          }
        }
      }
    }
  }
  if constexpr (CL > 1) {
    __syncwarp();
    cluster_sync();  // every CTA's part is in place
    constexpr int CW = DH / CL, kPer = CW / 4;  // this CTA's columns, four per thread
    const int live = sg.s.n * a.g, rank = (int)cluster_rank();
    for (int e = tid; e < live * kPer; e += kThreads) {
      const int r = e / kPer, col = rank * CW + e % kPer * 4;
      float2 ml[CL];
      float4 v[CL];
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        ml[c] = ld_cluster_f2(cluster_map(smem_u32(join_ml + r), (uint32_t)c));
        v[c] = ld_cluster_f4(cluster_map(smem_u32(join + r * G::kOStride + col), (uint32_t)c));
      }
      float M = -INFINITY, sum = 0.f, acc[4] = {};
#pragma unroll
      for (int c = 0; c < CL; ++c) M = fmaxf(M, ml[c].x);
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        if (ml[c].x == -INFINITY) continue;  // no tiles: nothing was written
        const float f = exp2f(ml[c].x - M);
        sum += f * ml[c].y;
        acc[0] += f * v[c].x;
        acc[1] += f * v[c].y;
        acc[2] += f * v[c].z;
        acc[3] += f * v[c].w;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int i = r / a.g;
      uint16_t* dst = static_cast<uint16_t*>(a.out) +
                      ((int64_t)(sg.s.q0 + i) * a.H + (int64_t)sg.head * a.g + r - i * a.g) * DH + col;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack2_bf16(acc[0] * inv, acc[1] * inv), pack2_bf16(acc[2] * inv, acc[3] * inv));
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its part may still be read
  } else {
    __syncthreads();
  }
  if (tid == 0 && *abort_flag) set_err(a.err, MEDUSA_DEVERR_TIMEOUT);
}

template <int DH, int CL>
int run(const PagedAttnArgs& a, const PagedKernels& k) {
  CUtensorMap tmK, tmV;
  const int box = a.p.page_size < KT ? a.p.page_size : KT;
  const int64_t lines = (int64_t)a.p.num_pages * a.Hkv * a.p.page_size;
  if (!make_lines_map(&tmK, a.k_pages, lines, DH, box) || !make_lines_map(&tmV, a.v_pages, lines, DH, box))
    return fail(MEDUSA_ERR_CUDA, "medusa_paged_attn: cuTensorMapEncodeTiled failed");
  auto* fn = paged_decode_kernel<DH, CL>;
  static std::atomic<uint64_t> done{0};
  if (int rc = prepare_kernel(reinterpret_cast<const void*>(fn), Cfg<DH>::smem, 0, 0, &done, "medusa_paged_attn")) return rc;
  if (CL == 1) launch_kernel(fn, dim3(k.sms), dim3(kThreads), Cfg<DH>::smem, k.stream, tmK, tmV, a);
  else launch_cluster(fn, CL, dim3(a.B * a.Hkv * CL), dim3(kThreads), Cfg<DH>::smem, k.stream, tmK, tmV, a);
  return check_launch("medusa_paged_attn");
}

// The cluster that takes a unit (1: the shared list): as large as the SMs
// allow, where the longest row that the cache can hold leaves a CTA at most
// kClusterTiles tiles.
constexpr int kClusterTiles = 16;
template <int DH>
int run_any(const PagedAttnArgs& a, const PagedKernels& k) {
  const int64_t units = (int64_t)a.B * a.Hkv, tiles = ((int64_t)a.p.max_pages * a.p.page_size + KT - 1) / KT;
  const int cl = a.B > kThreads ? 1 : units * 8 <= k.sms ? 8 : units * 4 <= k.sms ? 4 : units * 2 <= k.sms ? 2 : 1;
  if (cl > 1 && tiles <= (int64_t)kClusterTiles * cl) {
    if (cl == 8) return run<DH, 8>(a, k);
    return cl == 4 ? run<DH, 4>(a, k) : run<DH, 2>(a, k);
  }
  return run<DH, 1>(a, k);
}

}  // namespace

size_t paged_decode_part_bytes(int Dh, int sms) { return (size_t)sms * 2 * (RB * Dh + 2 * RB) * 4; }
int launch_paged_decode(const PagedAttnArgs& a, int Dh, const PagedKernels& k) {
  return Dh == 64 ? run_any<64>(a, k) : run_any<128>(a, k);
}

}  // namespace medusa

// Chunk attention over the paged cache: the call, the rotation and append of a
// chunk, and the float32 kernels.
#include <cmath>
#include <mutex>
#include <type_traits>

#include "paged_attn.cuh"

namespace medusa {
namespace {

// ------------------------------------------------ rotate, scale, append --
// A CTA per TOK tokens and group of heads: cos and sin of a token's position
// once per pair, in shared memory, then eight pairs per thread and step, the
// loads of kPrepSteps steps in flight.  Queries go to q_rot with the softmax
// scale in them (bf16: rounded, and in a second plane what the rounding left,
// rounded), keys and values to their pages.  Every element is read and
// written once: bound by memory for long chunks (16 tokens per CTA, all heads:
// 8192 tokens of 48 heads, 268 MB, in 58 us on cold caches), by the latency of a
// thread's few steps for short ones (4 tokens, as many groups of heads as give a
// thread kPrepSteps).  16 against 4 tokens per CTA, with the attention: 999 and
// 1030 us for 32768 tokens of 4 heads, 572 and 571 for 8192 of 32 heads; 51 and
// 40 us for 260 of 32.
constexpr int kPrepThreads = 256;
constexpr int kPrepSteps = 4;

template <typename T>
MDEV void load8(const T* p, float* f);
template <>
MDEV void load8<float>(const float* p, float* f) {
  const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
  f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
  f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
}
template <>
MDEV void load8<uint16_t>(const uint16_t* p, float* f) {
  unpack8_bf16(*reinterpret_cast<const uint4*>(p), f);
}
template <typename T>
MDEV void store8(T* p, const float* f);
template <>
MDEV void store8<float>(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
MDEV void store8<uint16_t>(uint16_t* p, const float* f) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
}

template <typename T, int DH, int TOK>
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(const __grid_constant__ PagedAttnArgs a) {
  __shared__ __align__(16) float cs[TOK][DH / 2], sn[TOK][DH / 2];
  __shared__ int64_t line0[TOK];  // head 0's line of the token's slot, -1: no page
  __shared__ int use[TOK], pos[TOK], seq[TOK], twice[TOK];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // they wait for this grid's end
  const int t = threadIdx.x, tok0 = blockIdx.x * TOK, nt = min(TOK, a.total_q - tok0);
  if (t < TOK) {
    seq[t] = -1;
    use[t] = 0;
    twice[t] = 0;
    pos[t] = 0;
    line0[t] = -1;
    if (t < nt) {
      const int tok = tok0 + t;
      int lo = 0, hi = a.B - 1;  // the last sequence that starts at or before the token
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.q_start[mid] <= tok) lo = mid; else hi = mid - 1;
      }
      SeqInfo s;
      int code;
      if (seq_info(a, lo, s, code) && tok >= s.q0 && tok < s.q0 + s.n) {
        const int i = tok - s.q0;
        seq[t] = lo;
        use[t] = 1;
        pos[t] = s.L + (a.T ? min(max(a.depth[i], 0), a.K) : i);
        const int page = page_of(a, s, s.L + i);
        if (page >= 0) line0[t] = page_line(a.p, page, a.Hkv, 0, (s.L + i) & (a.p.page_size - 1));
      }
    }
  }
  bool down = false;  // looked up beside the first warp's search
  for (int b = t - 32; t >= 32 && b < a.B; b += kPrepThreads - 32) down |= starts_decrease(a, b);
  if (__syncthreads_or(down)) return;
  if (a.rows) {  // an entry whose row an earlier one names is skipped
    for (int k = 0; k < nt; ++k) {
      const int b = seq[k];
      if (b > 0 && (k == 0 || seq[k - 1] != b))
        for (int j = t; j < b; j += kPrepThreads)
          if (a.rows[j] == a.rows[b] && a.q_start[j + 1] > a.q_start[j]) twice[k] = 1;
    }
  }
  for (int e = t; e < nt * (DH / 2); e += kPrepThreads)
    rope_cos_sin(pos[e / (DH / 2)], a.turns[e % (DH / 2)], cs[e / (DH / 2)][e % (DH / 2)],
                 sn[e / (DH / 2)][e % (DH / 2)]);
  __syncthreads();
  if (a.rows && t == 0)
    for (int k = 0; k < nt; ++k) {
      if (k > 0 && seq[k - 1] == seq[k]) twice[k] = twice[k - 1];
      if (twice[k]) use[k] = 0;
    }
  if (a.rows) __syncthreads();
  constexpr int kChunks = DH / 16;  // runs of eight pairs in a head
  constexpr int kRows = kPrepThreads / kChunks;
  const int all = a.H + 2 * a.Hkv, per = (all + gridDim.y - 1) / gridDim.y;
  const int head0 = blockIdx.y * per, heads = min(per, all - head0), rows = nt * heads;
  const int c = t % kChunks;
  const float inv = 1.f / (float)heads;
  using V = uint4;
  constexpr int kVecs = 8 * sizeof(T) / 16;  // 16-byte loads of eight elements
  for (int r0 = t / kChunks; r0 < rows; r0 += kPrepSteps * kRows) {
    V lo[kPrepSteps][kVecs], hi[kPrepSteps][kVecs];
    T* dst[kPrepSteps];
    int tk[kPrepSteps];  // token, or -1 - token where nothing turns; kNone: nothing to do
    constexpr int kNone = 1 << 20;
#pragma unroll
    for (int u = 0; u < kPrepSteps; ++u) {
      const int r = r0 + u * kRows;
      tk[u] = kNone;
      if (r >= rows) continue;
      const int k = (int)(((float)r + 0.5f) * inv), h = head0 + r - k * heads;  // exact: rows and heads are small
      if (!use[k]) continue;
      const int64_t tok = tok0 + k;
      const T* src;
      if (h < a.H) {
        src = static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)h * DH;
        const int hk = h / a.g;
        dst[u] = static_cast<T*>(a.q_rot) + (((int64_t)hk * a.total_q + tok) * a.g + h - hk * a.g) * DH;
        tk[u] = k;
      } else {
        if (line0[k] < 0) continue;
        const bool key = h < a.H + a.Hkv;
        const int hk = key ? h - a.H : h - a.H - a.Hkv;
        src = key ? static_cast<const T*>(a.k_new) + tok * a.k_stride + (int64_t)hk * DH
                  : static_cast<const T*>(a.v_new) + tok * a.v_stride + (int64_t)hk * DH;
        dst[u] = static_cast<T*>(key ? a.k_pages : a.v_pages) + (line0[k] + ((int64_t)hk << a.p.shift)) * DH;
        tk[u] = key ? k : -1 - k;
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        lo[u][v] = __ldg(reinterpret_cast<const V*>(src + c * 8) + v);
        hi[u][v] = __ldg(reinterpret_cast<const V*>(src + DH / 2 + c * 8) + v);
      }
    }
#pragma unroll
    for (int u = 0; u < kPrepSteps; ++u) {
      if (tk[u] == kNone) continue;
      if (tk[u] >= 0) {
        const int h = head0 + (r0 + u * kRows) - tk[u] * heads;
        const float mul = h < a.H ? a.qscale : 1.f;
        float x[8], y[8];
        load8(reinterpret_cast<const T*>(lo[u]), x);
        load8(reinterpret_cast<const T*>(hi[u]), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float co = cs[tk[u]][c * 8 + j], si = sn[tk[u]][c * 8 + j], p = x[j], q = y[j];
          x[j] = (p * co - q * si) * mul;
          y[j] = (q * co + p * si) * mul;
        }
        store8(reinterpret_cast<T*>(lo[u]), x);
        store8(reinterpret_cast<T*>(hi[u]), y);
        if (sizeof(T) == 2 && h < a.H) {  // what the rounding left
          float rx[8], ry[8];
          load8(reinterpret_cast<const T*>(lo[u]), rx);
          load8(reinterpret_cast<const T*>(hi[u]), ry);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            rx[j] = x[j] - rx[j];
            ry[j] = y[j] - ry[j];
          }
          store8(dst[u] + a.q_low + c * 8, rx);
          store8(dst[u] + a.q_low + DH / 2 + c * 8, ry);
        }
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        *(reinterpret_cast<V*>(dst[u] + c * 8) + v) = lo[u][v];
        *(reinterpret_cast<V*>(dst[u] + DH / 2 + c * 8) + v) = hi[u][v];
      }
    }
  }
}

// ------------------------------------------------------ float32 kernel --
// S = Q K^T and O += P V on the CUDA cores: 256 threads as 16 x 16, thread
// (ty, tx) with rows ty + 16 a of the block, keys tx + 16 b of the tile and,
// for O, columns tx * 4 + 64 c.  A row's sixteen threads are half a warp, so
// its maximum and sum are four shuffles.  Key rows are padded by 16 bytes
// (eight threads' 16-byte loads of eight rows then hit different banks).  The
// value tile loads while S is computed and the next key tile while O is.
// A tile's sums are added to the row's once (error against 64 bits at 60000 keys:
// 4.2e-7, 2-norm; 2.7e-6 with one running sum over the keys).
// Bound by shared memory and by the barriers between a tile's four phases: the
// FMA pipe is 43% busy (4 x 8 and 8 x 8 products per thread need fewer loads but
// leave fewer warps, and gain nothing; nor do two FMAs per instruction).  345
// tokens in five sequences, 16 heads of 64 (four per key head), prefixes up to
// 2000: 75 us with the rotation's launch.  Blocks of at most 16 rows have a form
// of their own where the call has no others: one token at a prefix of 1024, 32
// heads of 128, 24.8 us against 30.8 in the form for 64 rows; 64 tokens, 16
// heads of 128 (four per key head), prefixes up to 4000, 144 against 161.
// CTAs per SM (the 345 and the 64 tokens): 75 and 144 us; with 1, 85 and 198; with 3, 83 and 190.
constexpr int kGenThreads = 256, kGenCtas = 2;

template <int DH, int RB, int KT>
struct Gen {
  static constexpr int TM = RB / 16, TN = KT / 16, CC = DH / 64;
  static constexpr int kQ = RB * (DH + 4), kK = KT * (DH + 4), kV = KT * DH, kP = RB * (KT + 4);
  // the plan's scratch lies where the tiles come later
  static constexpr size_t smem = (size_t)(kQ + kK + kV + kP) * 4 + sizeof(Plan) + 64;
  static_assert(sizeof(PlanScratch) <= (size_t)(kQ + kK) * 4, "the plan's scratch");
  static constexpr int part_floats = RB * DH + 2 * RB;
};

template <int DH, int RB, int KT>
__global__ void __launch_bounds__(kGenThreads, kGenCtas) paged_generic_kernel(const __grid_constant__ PagedAttnArgs a) {
  using G = Gen<DH, RB, KT>;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;                  // [RB][DH + 4]
  float* Ks = Qs + G::kQ;          // [KT][DH + 4]
  float* Vs = Ks + G::kK;          // [KT][DH]
  float* Ps = Vs + G::kV;          // [RB][KT + 4]
  PlanScratch& sc = *reinterpret_cast<PlanScratch*>(sm);
  Plan& pl = *reinterpret_cast<Plan*>(Ps + G::kP);
  int* flag = reinterpret_cast<int*>(&pl + 1);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  int64_t x, x1;
  make_plan<kGenThreads, RB, KT, 1>(a, sc, pl, x, x1);
  const int64_t total = pl.total, grid = min((int64_t)gridDim.x, total);
  const int tb = RB / a.g;
  Segment sg;
  const bool any = x < x1 && seek_segment<RB, KT, 1>(a, sc, x, x1, sg);
  // the rotated queries and the appended tokens; and no grid ends before the
  // launch that it follows, whose reads the next call on the stream may change
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (!any) return;
  while (true) {
    const SeqInfo& s = sg.s;
    const int nkeys = s.L + s.n, tok0 = sg.u * tb, live = min(tb, s.n - tok0) * a.g;
    // The lines this thread copies of a tile (-1: none, zeros), looked up a
    // tile ahead: a copy waits for no page number.
    constexpr int kRow = DH / 4, kCopies = KT * kRow / kGenThreads;
    int line[kCopies];
    auto find = [&](int t) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int key = t * KT + (tid + i * kGenThreads) / kRow;
        line[i] = -1;
        if (t < sg.t1 && key < nkeys) {
          const int page = page_of(a, s, key);
          if (page >= 0) line[i] = (int)page_line(a.p, page, a.Hkv, sg.head, key & (a.p.page_size - 1));
        }
      }
    };
    auto load = [&](const void* pool, float* dst, int stride) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int e = tid + i * kGenThreads, c = e % kRow;
        cp_async16(smem_u32(dst + (e / kRow) * stride + c * 4),
                   static_cast<const float*>(pool) + (int64_t)max(line[i], 0) * DH + c * 4, line[i] >= 0 ? 16 : 0);
      }
      cp_async_commit();
    };
    find(sg.t0);
    __syncthreads();  // the previous segment's tiles are read
    {
      const float* qr = static_cast<const float*>(a.q_rot) +
                    ((int64_t)sg.head * a.total_q + s.q0 + tok0) * a.g * (int64_t)DH;
      for (int e = tid; e < RB * (DH / 8); e += kGenThreads) {
        const int r = e / (DH / 8), c = e % (DH / 8);
        float f[8] = {};
        if (r < live) load8(qr + (int64_t)r * DH + c * 8, f);
        store8(Qs + r * (DH + 4) + c * 8, f);
      }
    }
    load(a.k_pages, Ks, DH + 4);
    load(a.v_pages, Vs, DH);
    find(sg.t0 + 1);
    float o[G::TM][G::CC * 4], m[G::TM], l[G::TM];
#pragma unroll
    for (int i = 0; i < G::TM; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < G::CC * 4; ++c) o[i][c] = 0.f;
    }
    // A block with at most 16 rows (a single token, alone or beside longer
    // chunks) has them all in i = 0; the warps past its rows only copy, since
    // every row costs shared memory's bandwidth, live or not.
    const bool on = (tid >> 5) * 2 < live;
    auto tiles = [&](auto active) {
      constexpr int N = decltype(active)::value;
      for (int t = sg.t0; t < sg.t1; ++t) {
        cp_async_wait<1>();  // this tile's keys
        __syncthreads();
        float z[N][G::TN] = {};
#pragma unroll 4
        for (int d = 0; d < (on ? DH : 0); d += 4) {
          float4 qv[N], kv[G::TN];
#pragma unroll
          for (int i = 0; i < N; ++i) qv[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * (DH + 4) + d);
#pragma unroll
          for (int j = 0; j < G::TN; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * (DH + 4) + d);
#pragma unroll
          for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < G::TN; ++j)
              z[i][j] += qv[i].x * kv[j].x + qv[i].y * kv[j].y + qv[i].z * kv[j].z + qv[i].w * kv[j].w;
        }
        __syncthreads();  // the keys are read
        if (t + 1 < sg.t1) load(a.k_pages, Ks, DH + 4);
        else cp_async_commit();
        const bool masked = (t + 1) * KT > s.L;  // keys past the prefix: the mask decides
        float alpha[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (!on) break;
          const int r = ty + 16 * i, tok = tok0 + r / a.g;
          if (masked) {
#pragma unroll
            for (int j = 0; j < G::TN; ++j) {
              const int key = t * KT + tx + 16 * j;
              if (r >= live || key >= nkeys || !key_seen(a, s, tok, key)) z[i][j] = -INFINITY;
            }
          }
          float mt = z[i][0];
#pragma unroll
          for (int j = 1; j < G::TN; ++j) mt = fmaxf(mt, z[i][j]);
#pragma unroll
          for (int w = 8; w > 0; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));
          const float mn = fmaxf(m[i], mt), base = mn == -INFINITY ? 0.f : mn;
          alpha[i] = exp2f(m[i] - base);
          m[i] = mn;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < G::TN; ++j) {
            const float pj = exp2f(z[i][j] - base);
            sum += pj;
            Ps[r * (KT + 4) + tx + 16 * j] = pj;
          }
          l[i] = l[i] * alpha[i] + sum;  // this thread's keys; the sixteen parts are added at the end
        }
        cp_async_wait<1>();  // this tile's values
        __syncthreads();
        // The tile's products are summed for themselves and added to the rest
        // once: a running sum over the keys loses a rounding of its whole size
        // with each of them.
        float w[N][G::CC * 4] = {};
#pragma unroll 2
        for (int k = 0; k < (on ? KT : 0); k += 4) {
          float4 pv[N];
#pragma unroll
          for (int i = 0; i < N; ++i) pv[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * (KT + 4) + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            float4 vv[G::CC];
#pragma unroll
            for (int c = 0; c < G::CC; ++c)
              vv[c] = *reinterpret_cast<const float4*>(Vs + (k + kk) * DH + tx * 4 + 64 * c);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float pj = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
#pragma unroll
              for (int c = 0; c < G::CC; ++c) {
                w[i][c * 4] += pj * vv[c].x;
                w[i][c * 4 + 1] += pj * vv[c].y;
                w[i][c * 4 + 2] += pj * vv[c].z;
                w[i][c * 4 + 3] += pj * vv[c].w;
              }
            }
          }
        }
        if (on) {
#pragma unroll
          for (int i = 0; i < N; ++i)
#pragma unroll
            for (int c = 0; c < G::CC * 4; ++c) o[i][c] = o[i][c] * alpha[i] + w[i][c];
        }
        __syncthreads();  // the values are read
        if (t + 1 < sg.t1) load(a.v_pages, Vs, DH);
        else cp_async_commit();
        find(t + 2);
      }
    };
    if (live <= 16) tiles(std::integral_constant<int, 1>());
    else tiles(std::integral_constant<int, G::TM>());
#pragma unroll
    for (int i = 0; i < G::TM; ++i) {
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
      if (l[i] != l[i]) m[i] = INFINITY;  // so that no join drops a part whose scores are all NaN
    }
    auto put = [&](int i, const float* v, float sum) {  // row ty + 16 i of the block
      const int r = ty + 16 * i;
      if (r >= live) return;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      float* dst = static_cast<float*>(a.out) +
               ((int64_t)(s.q0 + tok0 + r / a.g) * a.H + (int64_t)sg.head * a.g + r % a.g) * DH;
#pragma unroll
      for (int c = 0; c < G::CC; ++c)
        *reinterpret_cast<float4*>(dst + tx * 4 + 64 * c) =
            make_float4(v[c * 4] * inv, v[c * 4 + 1] * inv, v[c * 4 + 2] * inv, v[c * 4 + 3] * inv);
    };
    if (sg.t0 == 0 && sg.t1 == sg.tiles) {
#pragma unroll
      for (int i = 0; i < G::TM; ++i) put(i, o[i], l[i]);
    } else {
      int first, last;
      unit_shares<1>(sg, total, grid, first, last);
      float* mine = a.part + (int64_t)part_slot(sg.unit_x, blockIdx.x, total, grid) * G::part_floats;
#pragma unroll
      for (int i = 0; i < G::TM; ++i) {
        const int r = ty + 16 * i;
#pragma unroll
        for (int c = 0; c < G::CC; ++c)
          *reinterpret_cast<float4*>(mine + r * DH + tx * 4 + 64 * c) =
              make_float4(o[i][c * 4], o[i][c * 4 + 1], o[i][c * 4 + 2], o[i][c * 4 + 3]);
        if (tx == 0) *reinterpret_cast<float2*>(mine + RB * DH + 2 * r) = make_float2(m[i], l[i]);
      }
      __syncthreads();
      if (tid == 0) {
        const int before = arrive_acq_rel(a.counters + first);
        *flag = before == last - first;
        if (before == last - first) a.counters[first] = 0;  // ready for the next call
      }
      __syncthreads();
      if (*flag) {  // one partial at a time, all its rows' loads in flight
#pragma unroll
        for (int i = 0; i < G::TM; ++i) {
          m[i] = -INFINITY;
          l[i] = 0.f;
#pragma unroll
          for (int c = 0; c < G::CC * 4; ++c) o[i][c] = 0.f;
        }
        for (int c = first; c <= last; ++c) {
          const float* pt = a.part + (int64_t)part_slot(sg.unit_x, c, total, grid) * G::part_floats;
          float2 ml[G::TM];
          float4 v[G::TM][G::CC];
#pragma unroll
          for (int i = 0; i < G::TM; ++i) {
            const int r = ty + 16 * i;
            ml[i] = __ldcg(reinterpret_cast<const float2*>(pt + RB * DH + 2 * r));
#pragma unroll
            for (int cc = 0; cc < G::CC; ++cc)
              v[i][cc] = __ldcg(reinterpret_cast<const float4*>(pt + r * DH + tx * 4 + 64 * cc));
          }
#pragma unroll
          for (int i = 0; i < G::TM; ++i) {
            const float N = fmaxf(m[i], ml[i].x);
            const float f0 = m[i] == -INFINITY ? 0.f : exp2f(m[i] - N), f1 = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - N);
            m[i] = N;
            l[i] = l[i] * f0 + ml[i].y * f1;
#pragma unroll
            for (int cc = 0; cc < G::CC; ++cc) {
              o[i][cc * 4] = o[i][cc * 4] * f0 + v[i][cc].x * f1;
              o[i][cc * 4 + 1] = o[i][cc * 4 + 1] * f0 + v[i][cc].y * f1;
              o[i][cc * 4 + 2] = o[i][cc * 4 + 2] * f0 + v[i][cc].z * f1;
              o[i][cc * 4 + 3] = o[i][cc * 4 + 3] * f0 + v[i][cc].w * f1;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < G::TM; ++i) put(i, o[i], l[i]);
      }
    }
    if (!next_segment<RB, KT, 1>(a, pl, x1, sg)) break;
  }
}

template <int DH, int RB, int KT>
int run_generic(const PagedAttnArgs& a, const PagedKernels& k) {
  using G = Gen<DH, RB, KT>;
  auto* fn = paged_generic_kernel<DH, RB, KT>;
  static std::atomic<uint64_t> done{0};
  if (int rc = prepare_kernel(reinterpret_cast<const void*>(fn), G::smem, 0, 0, &done, "medusa_paged_attn")) return rc;
  launch_after(fn, dim3(k.sms * kGenCtas), dim3(kGenThreads), G::smem, k.stream, a);
  return check_launch("medusa_paged_attn");
}

size_t generic_part_bytes(int RB, int Dh, int sms) { return (size_t)(sms * kGenCtas) * 2 * (RB * Dh + 2 * RB) * 4; }

// The workspace: both kernels' counters first, at the same place for every
// size, then the rotated queries, then the partials.
struct PagedWorkspace {
  size_t q_rot, part, total;
};
constexpr size_t kCounterBytes = 2 * kPagedCounters * 4;

PagedWorkspace workspace_of(int total_q, int H, int Dh, medusa_dtype dtype, int sms) {
  PagedWorkspace w;
  const bool bf16 = dtype == MEDUSA_BF16;
  w.q_rot = kCounterBytes;
  w.part = align_up(w.q_rot + (size_t)total_q * H * Dh * 4, 256);  // float32, or two bf16 parts
  const size_t few = bf16 ? paged_decode_part_bytes(Dh, sms) : generic_part_bytes(16, Dh, sms);
  const size_t many = bf16 ? paged_chunk_part_bytes(Dh, sms) : generic_part_bytes(64, Dh, sms);
  w.total = align_up(w.part + (few > many ? few : many), 256);
  return w;
}

// The fractions of a turn per position (theta < 1 may turn more than once),
// kept for the thread's next call: 64 powers take as long as a launch.
void fill_turns(uint64_t* turns, float theta, int Dh) {
  static thread_local float last_theta = 0.f;
  static thread_local int last_dh = 0;
  static thread_local uint64_t last[64];
  if (theta != last_theta || Dh != last_dh) {
    for (int j = 0; j < Dh / 2; ++j) {
      double f = std::pow((double)theta, -2.0 * j / (double)Dh) / 6.283185307179586476925;
      f -= std::floor(f);
      last[j] = (uint64_t)std::ldexp(f, 64);
    }
    last_theta = theta;
    last_dh = Dh;
  }
  for (int j = 0; j < Dh / 2; ++j) turns[j] = last[j];
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) ==
            cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

}  // namespace

bool make_rows_map(CUtensorMap* m, const void* base, int64_t rows, int Dh, int box) {
  EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)Dh, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)Dh * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_lines_map(CUtensorMap* m, const void* base, int64_t rows, int Dh, int box) {
  EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(Dh / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)Dh * 2, 128};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)box, (cuuint32_t)(Dh / 64)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {
template <typename T, int DH>
int run_prep(const PagedAttnArgs& a, const PagedKernels& k) {
  if (a.total_q >= 16 * 2 * k.sms) {  // two CTAs of 16 tokens for every SM
    launch_kernel(paged_prep_kernel<T, DH, 16>, dim3((a.total_q + 15) / 16), dim3(kPrepThreads), 0, k.stream, a);
  } else {
    const int per = kPrepThreads * kPrepSteps, items = 4 * (a.H + 2 * a.Hkv) * (DH / 16);
    launch_kernel(paged_prep_kernel<T, DH, 4>, dim3((a.total_q + 3) / 4, (items + per - 1) / per), dim3(kPrepThreads),
                  0, k.stream, a);
  }
  return check_launch("medusa_paged_attn");
}
}  // namespace

int launch_paged_prep(const PagedAttnArgs& a, int Dh, medusa_dtype dtype, const PagedKernels& k) {
  if (dtype == MEDUSA_BF16) return Dh == 64 ? run_prep<uint16_t, 64>(a, k) : run_prep<uint16_t, 128>(a, k);
  return Dh == 64 ? run_prep<float, 64>(a, k) : run_prep<float, 128>(a, k);
}

int launch_paged_generic(const PagedAttnArgs& a, int Dh, bool few_rows, const PagedKernels& k) {
  if (few_rows) return Dh == 64 ? run_generic<64, 16, 64>(a, k) : run_generic<128, 16, 64>(a, k);
  return Dh == 64 ? run_generic<64, 64, 64>(a, k) : run_generic<128, 64, 32>(a, k);
}

}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_paged_attn_workspace_size(int B, int total_q, int max_new, int H, int Hkv, int Dh,
                                                   medusa_dtype dtype) {
  if (B < 0 || total_q < 0 || max_new < 0 || H < 1 || Hkv < 1 || Dh < 1) return 0;
  return workspace_of(total_q, H, Dh, dtype, sm_count()).total;
}

extern "C" int medusa_paged_attn(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                 const void* v_new, int64_t v_stride, void* k_pages, void* v_pages,
                                 const medusa_pages_t* pages, const int32_t* rows, const int32_t* q_start, int B,
                                 int total_q, int max_new, const medusa_tree_t* tree, int H, int Hkv, int Dh,
                                 float rope_theta, float scale, medusa_dtype dtype, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* err, void* stream) {
  const char* fn = "medusa_paged_attn";
  if (int rc = check_pages(pages, fn)) return rc;
  if (int rc = check_pool(k_pages, v_pages, pages->num_pages, pages->page_size, Hkv, Dh, dtype, fn)) return rc;
  if (tree)
    if (int rc = check_tree(tree, fn)) return rc;
  if (B < 0 || B > MEDUSA_MAX_ROWS || (!rows && B > pages->rows) || total_q < 0 || max_new < 0 || max_new > (1 << 24))
    return fail(MEDUSA_ERR_INVALID, "%s: B=%d total_q=%d max_new=%d", fn, B, total_q, max_new);
  if (H < Hkv || H % Hkv || H / Hkv > kPagedMaxGroup)
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: H=%d Hkv=%d (H a multiple of Hkv, H / Hkv at most %d)", fn, H, Hkv,
                kPagedMaxGroup);
  if ((int64_t)total_q * H >= (1ll << 31))
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: total_q * H must be below 2^31", fn);
  if (!(rope_theta > 0.f) || !(scale > 0.f)) return fail(MEDUSA_ERR_INVALID, "%s: rope_theta/scale", fn);
  if (B == 0 || total_q == 0 || max_new == 0) return MEDUSA_OK;
  if (!q || !k_new || !v_new || !out || !q_start) return fail(MEDUSA_ERR_INVALID, "%s: NULL tensor", fn);
  const int es = dtype == MEDUSA_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
       reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) % 16 ||
      ((q_stride | k_stride | v_stride) * es) % 16)
    return fail(MEDUSA_ERR_INVALID, "%s: tensors or strides not 16-byte aligned", fn);
  if (total_q > 1 && (q_stride < (int64_t)H * Dh || k_stride < (int64_t)Hkv * Dh || v_stride < (int64_t)Hkv * Dh))
    return fail(MEDUSA_ERR_INVALID, "%s: a token stride is shorter than a token's heads", fn);
  const int sms = sm_count();
  const PagedWorkspace w = workspace_of(total_q, H, Dh, dtype, sms);
  if (!workspace || workspace_bytes < w.total)
    return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, w.total);
  auto* ws = static_cast<uint8_t*>(workspace);
  PagedAttnArgs a{};
  a.q = q; a.k_new = k_new; a.v_new = v_new;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.k_pages = k_pages; a.v_pages = v_pages;
  a.p = pages_dev(pages);
  a.rows = rows; a.q_start = q_start; a.B = B; a.total_q = total_q; a.max_new = max_new;
  if (tree) {
    a.T = tree->T; a.W = tree->W; a.K = tree->K; a.depth = tree->depth; a.anc = tree->anc_mask;
  }
  a.H = H; a.Hkv = Hkv; a.g = H / Hkv;
  fill_turns(a.turns, rope_theta, Dh);
  a.qscale = scale * kPagedLog2e;
  a.out = out;
  a.q_rot = ws + w.q_rot;
  a.q_low = (int64_t)total_q * H * Dh;
  a.err = err;
  const PagedKernels k{as_stream(stream), sms};
  // One attention launch for the whole call, by its longest chunk.  A batch
  // with both kinds of sequences goes through the kernels for many rows: two
  // launches, one per kind, took 14% longer for eleven sequences of 1 .. 700
  // tokens (40 heads of 64, prefixes up to 5000).  Up to kFewRows rows per key
  // head the kernels for few rows are ahead: 64 single tokens with four heads
  // per key head and prefixes up to 8192 take 185 us, 246 us in the other one;
  // one token at a prefix of 1024, 12 and 24 us.
  const bool few = (int64_t)max_new * a.g <= kFewRows;
  a.counters = reinterpret_cast<int*>(ws) + (few ? 0 : kPagedCounters);
  a.part = reinterpret_cast<float*>(ws + w.part);
  if (dtype == MEDUSA_BF16 && few) return launch_paged_decode(a, Dh, k);
  if (int rc = launch_paged_prep(a, Dh, dtype, k)) return rc;
  return dtype == MEDUSA_BF16 ? launch_paged_chunk(a, Dh, k) : launch_paged_generic(a, Dh, few, k);
}

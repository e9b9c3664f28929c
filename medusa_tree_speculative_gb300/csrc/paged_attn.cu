// Chunk attention over the paged cache: the calls, and the rotation and append of
// a chunk.
#include <cmath>
#include <mutex>

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
// Sharing takes three launches more than one call's one or two, 10 to 20 us, writes
// the rows' common parts and reads them, and pays where it saves as much reading.
// Single tokens, us shared and in one launch: 4 behind 1024, 32 heads of 128 (50 MB
// saved) 33 and 25; 8 (117 MB) 35 and 35; 16 behind 2048, 8 key heads (126 MB) 33 and
// 35; 64 behind 512 (132 MB) 40 and 41; 4 behind 4096 (201 MB) 41 and 52.  Chunks: 16
// of 16 tokens behind 4096, 8 key heads (252 MB) 68 and 72; of 65 tokens, 32 heads of
// 128, 16 behind 1024 (252 MB) 128 and 88, behind 2048 (503 MB) 152 and 139, behind
// 4096 (1007 MB) 194 and 231; 8 behind 4096 (470 MB) 129 and 127, behind 6000 (688 MB)
// 153 and 171: 64 bytes more for each of the outputs' elements.  (Where the products
// of a group's many rows bind, that is too little: 4 trees of 65 behind 8192, 403 MB,
// 143 and 124.)  Float32 chunks, where the arithmetic counts and blocks fill up: 16
// times 9 tokens behind 1024 (31 MB) 56 and 52, 8 behind 4096 (59 MB) 75 and 85, 4
// times 30 behind 1024 (50 MB) 75 and 91; single tokens (126 MB) 51 and 49.  The host
// knows how long the rows may be, not how long they are: a call whose rows' capacity
// saves less does not look at its groups, and in a table with room for long rows short
// ones share at that price.  A group whose common tokens fill no two tiles shares
// nothing.
int64_t worth_sharing(int total_q, int H, int Dh, bool f32, bool few) {
  return f32 && !few ? 32ll << 20 : (128ll << 20) + (few ? 0 : 64ll * total_q * H * Dh);
}
constexpr int kMinCommon = 128;
constexpr int kPrepSteps = 4;

// The groups of a call with common tokens, by one CTA: which of a group's rows is
// read for all of them, and how many tokens.  Sharing changes nothing but what is
// read, so whatever is wrong with a group is reported and turns it off.
struct GroupScratch {
  int start[MEDUSA_MAX_ROWS + 1], live[MEDUSA_MAX_ROWS], shortest[MEDUSA_MAX_ROWS], lead[MEDUSA_MAX_ROWS];
};
MDEV void find_groups(const PagedAttnArgs& a, GroupScratch& g) {
  const int t = threadIdx.x;
  bool down = false, bad = false;
  for (int b = t; b < a.B; b += kPrepThreads) down |= starts_decrease(a, b);
  for (int i = t; i <= a.n_groups; i += kPrepThreads) {
    const int at = a.group_start[i];
    g.start[i] = at;
    bad |= at < 0 || at > a.B || (i > 0 && at < a.group_start[i - 1]);
    if (i < a.n_groups) {
      g.live[i] = 0;
      g.shortest[i] = g.lead[i] = 0x7fffffff;
    }
  }
  bad = __syncthreads_or(bad);
  down = __syncthreads_or(down);
  if (bad && t == 0) set_err(a.err, MEDUSA_DEVERR_LENGTH);
  const bool none = bad || down;
  auto group_of = [&](int b) {  // the last group that starts at or before b: the one that holds it, if any does
    int lo = 0, hi = a.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (g.start[mid] <= b) lo = mid; else hi = mid - 1;
    }
    return g.start[lo] <= b && b < g.start[lo + 1] ? lo : -1;
  };
  for (int b = t; b < a.B; b += kPrepThreads) {
    SeqInfo<> s;
    int code;
    if (none || !seq_info(a, b, s, code)) continue;
    const int k = group_of(b);
    if (k < 0) continue;
    atomicAdd(&g.live[k], 1);
    atomicMin(&g.shortest[k], s.L);
    atomicMin(&g.lead[k], b);
  }
  __syncthreads();
  for (int i = t; i < a.n_groups; i += kPrepThreads) {
    PagedGroup out = {0, 0, 0, 0};
    if (g.live[i] > 0) {
      int keys = a.common[i];
      if (keys < 0 || keys > g.shortest[i]) {
        set_err(a.err, MEDUSA_DEVERR_LENGTH);
        keys = 0;
      }
      if (g.live[i] > 1 && keys >= kMinCommon) {
        const int q0 = max(0, a.q_start[g.start[i]]), q1 = min(a.total_q, a.q_start[g.start[i + 1]]);
        out = PagedGroup{a.rows ? a.rows[g.lead[i]] : g.lead[i], q0, q1 - q0, keys};
      }
    }
    a.groups[i] = out;
    g.live[i] = out.n > 0 ? out.keys : 0;
  }
  __syncthreads();
  for (int b = t; b < a.B; b += kPrepThreads) {
    const int k = none ? -1 : group_of(b);
    a.from[b] = k < 0 ? 0 : g.live[k];
  }
}

template <typename T, int DH, int TOK, bool GROUPS>
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(const __grid_constant__ PagedAttnArgs a) {
  __shared__ __align__(16) float cs[TOK][DH / 2], sn[TOK][DH / 2];
  __shared__ int64_t line0[TOK];  // head 0's line of the token's slot, -1: no page
  __shared__ int use[TOK], pos[TOK], seq[TOK], twice[TOK];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // they wait for this grid's end
  if constexpr (GROUPS) {  // the first column of CTAs: its first one
    __shared__ GroupScratch gs;
    if (blockIdx.x == 0) {
      if (blockIdx.y == 0) find_groups(a, gs);
      return;
    }
  }
  const int t = threadIdx.x, tok0 = (blockIdx.x - (GROUPS ? 1 : 0)) * TOK, nt = min(TOK, a.total_q - tok0);
  if constexpr (GROUPS) {
    if (blockIdx.y == 0)
      for (int e = t; e < a.Hkv * nt * a.g; e += kPrepThreads) {
        const int h = e / (nt * a.g);
        a.parts[((int64_t)h * a.total_q + tok0) * a.g + e - h * nt * a.g] = kNoParts;
      }
  }
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
      SeqInfo<> s;
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
  const size_t few = bf16 ? paged_decode_part_bytes(Dh, sms) : paged_generic_part_bytes(16, Dh, sms);
  const size_t many = bf16 ? paged_chunk_part_bytes(Dh, sms) : paged_generic_part_bytes(64, Dh, sms);
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
template <typename T, int DH, bool GROUPS>
int run_prep(const PagedAttnArgs& a, const PagedKernels& k) {
  const int more = GROUPS ? 1 : 0;
  if (a.total_q >= 16 * 2 * k.sms) {  // two CTAs of 16 tokens for every SM
    launch_kernel(paged_prep_kernel<T, DH, 16, GROUPS>, dim3((a.total_q + 15) / 16 + more), dim3(kPrepThreads), 0,
                  k.stream, a);
  } else {
    const int per = kPrepThreads * kPrepSteps, items = 4 * (a.H + 2 * a.Hkv) * (DH / 16);
    launch_kernel(paged_prep_kernel<T, DH, 4, GROUPS>, dim3((a.total_q + 3) / 4 + more, (items + per - 1) / per),
                  dim3(kPrepThreads), 0, k.stream, a);
  }
  return check_launch(k.name);
}
template <bool GROUPS>
int run_prep_of(const PagedAttnArgs& a, int Dh, medusa_dtype dtype, const PagedKernels& k) {
  if (dtype == MEDUSA_BF16) return Dh == 64 ? run_prep<uint16_t, 64, GROUPS>(a, k) : run_prep<uint16_t, 128, GROUPS>(a, k);
  return Dh == 64 ? run_prep<float, 64, GROUPS>(a, k) : run_prep<float, 128, GROUPS>(a, k);
}
}  // namespace

namespace {
// ---------------------------------------- the common tokens' partials --
// A thread adds four columns of a row's partials, kJoin of them in flight.  FAST:
// the tcgen05 kernel's, where four columns of 128 rows lie side by side, so a warp
// takes 32 rows; else float32 blocks, rows one by one.  Bound by L2: 64 tokens
// behind 16384, 32 heads of 128, 19 partials a row, 20 MB.
constexpr int kJoinThreads = 256, kJoin = 4;

template <int DH, bool FAST>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, int block_rows) {
  // The launch after this one may start: this one begins when kCommon has ended, which
  // has waited for the first launch, so it finds that one's results.  (kCommon letting
  // this one start early: 5 us more for four tokens behind 1024, 7 less for 104
  // behind up to 16384.)
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;\n" ::: "memory");
  constexpr int kQuads = DH / 4;
  const int64_t rows = (int64_t)a.total_q * a.H, e = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int64_t row = FAST ? e / (32 * kQuads) * 32 + e % 32 : e / kQuads;
  const int quad = FAST ? (int)(e / 32 % kQuads) : (int)(e % kQuads);
  if (row >= rows) return;
  const uint32_t w = __ldcg(a.parts + row);
  if (w == kNoParts || w == kNoJoin) return;
  const int r = w & 127, lane = w >> 7 & 1, slot = w >> 8 & 1, first = w >> 9 & 2047, n = w >> 20;
  const int64_t size = (int64_t)block_rows * DH + 2 * block_rows;
  auto part = [&](int i) {
    const int64_t s = 2 * (first + i) + (i == 0 ? slot : 0);
    return a.part + (FAST ? s * 2 + lane : s) * size;
  };
  const int64_t at = FAST ? ((int64_t)quad * block_rows + r) * 4 : (int64_t)r * DH + quad * 4;
  const int64_t ml = (int64_t)block_rows * DH + 2 * r;
  float M = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += kJoin) {
    float2 m[kJoin];
    float4 v[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const float* p = part(min(i0 + j, n - 1));
      m[j] = __ldcg(reinterpret_cast<const float2*>(p + ml));
      v[j] = __ldcg(reinterpret_cast<const float4*>(p + at));
      if (i0 + j >= n) m[j] = make_float2(-INFINITY, 0.f);
    }
    float N = M;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) N = fmaxf(N, m[j].x);
    const float f = M == -INFINITY ? 0.f : exp2f(M - N);
    M = N;
    sum *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      if (m[j].x == -INFINITY) continue;
      const float g = exp2f(m[j].x - N);
      sum += g * m[j].y;
      acc.x += g * v[j].x;
      acc.y += g * v[j].y;
      acc.z += g * v[j].z;
      acc.w += g * v[j].w;
    }
  }
  *reinterpret_cast<float4*>(a.common_o + row * DH + quad * 4) = acc;
  if (quad == 0) a.common_ml[row] = make_float2(M, sum);
}

template <int DH, bool FAST>
int run_join(const PagedAttnArgs& a, int block_rows, const PagedKernels& k) {
  const int64_t rows = ((int64_t)a.total_q * a.H + 31) / 32 * 32;
  launch_after(paged_join_kernel<DH, FAST>, dim3((unsigned)((rows * (DH / 4) + kJoinThreads - 1) / kJoinThreads)),
               dim3(kJoinThreads), 0, k.stream, a, block_rows);
  return check_launch(k.name);
}
}  // namespace

int launch_paged_join(const PagedAttnArgs& a, int Dh, int rows, const PagedKernels& k) {
  if (rows == 128) return Dh == 64 ? run_join<64, true>(a, 128, k) : run_join<128, true>(a, 128, k);
  return Dh == 64 ? run_join<64, false>(a, rows, k) : run_join<128, false>(a, rows, k);
}

int launch_paged_prep(const PagedAttnArgs& a, int Dh, medusa_dtype dtype, bool groups, const PagedKernels& k) {
  return groups ? run_prep_of<true>(a, Dh, dtype, k) : run_prep_of<false>(a, Dh, dtype, k);
}

}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_paged_attn_workspace_size(int B, int total_q, int max_new, int H, int Hkv, int Dh,
                                                   medusa_dtype dtype) {
  if (B < 0 || total_q < 0 || max_new < 0 || H < 1 || Hkv < 1 || Dh < 1) return 0;
  return workspace_of(total_q, H, Dh, dtype, sm_count()).total;
}

namespace {

// The arguments that the three calls have in common.
struct Call {
  const void* q;
  int64_t q_stride;
  const void* k_new;
  int64_t k_stride;
  const void* v_new;
  int64_t v_stride;
  void* k_pages;
  void* v_pages;
  const medusa_pages_t* pages;
  const int32_t* rows;
  const int32_t* q_start;
  int B, total_q, max_new;
  const medusa_tree_t* tree;
  int H, Hkv, Dh;
  float rope_theta, scale;
  medusa_dtype dtype;
  void* out;
  void* workspace;
  size_t workspace_bytes;
  int32_t* err;
  void* stream;
};

// Checks them and fills `a`; a.total_q stays 0 where there is nothing to do.
// `need`: the workspace's least size.
int check_call(const Call& c, size_t need, const char* fn, PagedAttnArgs& a, PagedKernels& k) {
  if (int rc = check_pages(c.pages, fn)) return rc;
  if (int rc = check_pool(c.k_pages, c.v_pages, c.pages->num_pages, c.pages->page_size, c.Hkv, c.Dh, c.dtype, fn))
    return rc;
  if (c.tree)
    if (int rc = check_tree(c.tree, fn)) return rc;
  if (c.B < 0 || c.B > MEDUSA_MAX_ROWS || (!c.rows && c.B > c.pages->rows) || c.total_q < 0 || c.max_new < 0 ||
      c.max_new > (1 << 24))
    return fail(MEDUSA_ERR_INVALID, "%s: B=%d total_q=%d max_new=%d", fn, c.B, c.total_q, c.max_new);
  if (c.H < c.Hkv || c.H % c.Hkv || c.H / c.Hkv > kPagedMaxGroup)
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: H=%d Hkv=%d (H a multiple of Hkv, H / Hkv at most %d)", fn, c.H, c.Hkv,
                kPagedMaxGroup);
  if ((int64_t)c.total_q * c.H >= (1ll << 31))
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: total_q * H must be below 2^31", fn);
  if (!(c.rope_theta > 0.f) || !(c.scale > 0.f)) return fail(MEDUSA_ERR_INVALID, "%s: rope_theta/scale", fn);
  if (c.B == 0 || c.total_q == 0 || c.max_new == 0) return MEDUSA_OK;
  if (!c.q || !c.k_new || !c.v_new || !c.out || !c.q_start) return fail(MEDUSA_ERR_INVALID, "%s: NULL tensor", fn);
  const int es = c.dtype == MEDUSA_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(c.q) | reinterpret_cast<uintptr_t>(c.k_new) | reinterpret_cast<uintptr_t>(c.v_new) |
       reinterpret_cast<uintptr_t>(c.out) | reinterpret_cast<uintptr_t>(c.workspace)) % 16 ||
      ((c.q_stride | c.k_stride | c.v_stride) * es) % 16)
    return fail(MEDUSA_ERR_INVALID, "%s: tensors or strides not 16-byte aligned", fn);
  if (c.total_q > 1 && (c.q_stride < (int64_t)c.H * c.Dh || c.k_stride < (int64_t)c.Hkv * c.Dh ||
                        c.v_stride < (int64_t)c.Hkv * c.Dh))
    return fail(MEDUSA_ERR_INVALID, "%s: a token stride is shorter than a token's heads", fn);
  const int sms = sm_count();
  if (!c.workspace || c.workspace_bytes < need)
    return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, c.workspace_bytes, need);
  const PagedWorkspace w = workspace_of(c.total_q, c.H, c.Dh, c.dtype, sms);
  auto* ws = static_cast<uint8_t*>(c.workspace);
  a.q = c.q; a.k_new = c.k_new; a.v_new = c.v_new;
  a.q_stride = c.q_stride; a.k_stride = c.k_stride; a.v_stride = c.v_stride;
  a.k_pages = c.k_pages; a.v_pages = c.v_pages;
  a.p = pages_dev(c.pages);
  a.rows = c.rows; a.q_start = c.q_start; a.B = c.B; a.total_q = c.total_q; a.max_new = c.max_new;
  if (c.tree) {
    a.T = c.tree->T; a.W = c.tree->W; a.K = c.tree->K; a.depth = c.tree->depth; a.anc = c.tree->anc_mask;
  }
  a.H = c.H; a.Hkv = c.Hkv; a.g = c.H / c.Hkv;
  fill_turns(a.turns, c.rope_theta, c.Dh);
  a.qscale = c.scale * kPagedLog2e;
  a.out = c.out;
  a.q_rot = ws + w.q_rot;
  a.q_low = (int64_t)c.total_q * c.H * c.Dh;
  a.err = c.err;
  a.part = reinterpret_cast<float*>(ws + w.part);
  k = PagedKernels{as_stream(c.stream), sms, fn};
  return MEDUSA_OK;
}

// The counters of the kernels for few query rows and of those for many.
int* counters_of(const Call& c, bool few) { return static_cast<int*>(c.workspace) + (few ? 0 : kPagedCounters); }

// One attention launch for the whole call, by its longest chunk.  A batch
// with both kinds of sequences goes through the kernels for many rows: two
// launches, one per kind, took 14% longer for eleven sequences of 1 .. 700
// tokens (40 heads of 64, prefixes up to 5000).  Up to kFewRows rows per key
// head the kernels for few rows are ahead: 64 single tokens with four heads
// per key head and prefixes up to 8192 take 185 us, 246 us in the other one;
// one token at a prefix of 1024, 12 and 24 us.
template <Keys KEYS>
int attend(const Call& c, PagedAttnArgs& a, const PagedKernels& k) {
  const bool few = (int64_t)a.max_new * a.g <= kFewRows;
  a.counters = counters_of(c, few);
  if (c.dtype == MEDUSA_BF16 && few) return launch_paged_decode<KEYS>(a, c.Dh, k);
  if (int rc = launch_paged_prep(a, c.Dh, c.dtype, false, k)) return rc;
  return c.dtype == MEDUSA_BF16 ? launch_paged_chunk<KEYS>(a, c.Dh, k) : launch_paged_generic<KEYS>(a, c.Dh, few, k);
}

}  // namespace

extern "C" int medusa_paged_attn(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                 const void* v_new, int64_t v_stride, void* k_pages, void* v_pages,
                                 const medusa_pages_t* pages, const int32_t* rows, const int32_t* q_start, int B,
                                 int total_q, int max_new, const medusa_tree_t* tree, int H, int Hkv, int Dh,
                                 float rope_theta, float scale, medusa_dtype dtype, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* err, void* stream) {
  const Call c{q, q_stride, k_new, k_stride, v_new, v_stride, k_pages, v_pages, pages, rows, q_start, B, total_q,
               max_new, tree, H, Hkv, Dh, rope_theta, scale, dtype, out, workspace, workspace_bytes, err, stream};
  PagedAttnArgs a{};
  PagedKernels k{};
  if (int rc = check_call(c, medusa_paged_attn_workspace_size(B, total_q, max_new, H, Hkv, Dh, dtype),
                          "medusa_paged_attn", a, k)) return rc;
  return a.total_q ? attend<kAll>(c, a, k) : MEDUSA_OK;
}

extern "C" int medusa_paged_attn_window(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                        const void* v_new, int64_t v_stride, void* k_pages, void* v_pages,
                                        const medusa_pages_t* pages, const int32_t* rows, const int32_t* q_start,
                                        int B, int total_q, int max_new, const medusa_tree_t* tree, int window,
                                        int sinks, int H, int Hkv, int Dh, float rope_theta, float scale,
                                        medusa_dtype dtype, void* out, void* workspace, size_t workspace_bytes,
                                        int32_t* err, void* stream) {
  const char* fn = "medusa_paged_attn_window";
  if (window < 1 || sinks < 0) return fail(MEDUSA_ERR_INVALID, "%s: window=%d sinks=%d", fn, window, sinks);
  if (tree && window <= tree->K)
    return fail(MEDUSA_ERR_UNSUPPORTED, "%s: a window of %d, a tree of depth %d (the window has to be longer)", fn,
                window, tree->K);
  const Call c{q, q_stride, k_new, k_stride, v_new, v_stride, k_pages, v_pages, pages, rows, q_start, B, total_q,
               max_new, tree, H, Hkv, Dh, rope_theta, scale, dtype, out, workspace, workspace_bytes, err, stream};
  PagedAttnArgs a{};
  PagedKernels k{};
  a.window = window;
  a.sinks = sinks;
  if (int rc = check_call(c, medusa_paged_attn_workspace_size(B, total_q, max_new, H, Hkv, Dh, dtype), fn, a, k)) return rc;
  return a.total_q ? attend<kWindow>(c, a, k) : MEDUSA_OK;
}

namespace {
// Behind the workspace of medusa_paged_attn: the groups, and the common parts.
struct SharedWorkspace {
  size_t groups, from, ml, parts, o, total;
};
SharedWorkspace shared_workspace_of(int B, int n_groups, int total_q, int H, int Dh, medusa_dtype dtype, int sms) {
  SharedWorkspace w;
  w.groups = workspace_of(total_q, H, Dh, dtype, sms).total;
  w.from = align_up(w.groups + (size_t)n_groups * sizeof(PagedGroup), 256);
  w.ml = align_up(w.from + (size_t)B * 4, 256);
  w.parts = align_up(w.ml + (size_t)total_q * H * 8, 256);
  w.o = align_up(w.parts + (size_t)total_q * H * 4, 256);
  w.total = align_up(w.o + (size_t)total_q * H * Dh * 4, 256);
  return w;
}
}  // namespace

extern "C" size_t medusa_paged_attn_shared_workspace_size(int B, int n_groups, int total_q, int max_new, int H, int Hkv,
                                                          int Dh, medusa_dtype dtype) {
  if (B < 0 || n_groups < 0 || total_q < 0 || max_new < 0 || H < 1 || Hkv < 1 || Dh < 1) return 0;
  return shared_workspace_of(B, n_groups, total_q, H, Dh, dtype, sm_count()).total;
}

extern "C" int medusa_paged_attn_shared(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                        const void* v_new, int64_t v_stride, void* k_pages, void* v_pages,
                                        const medusa_pages_t* pages, const int32_t* rows, const int32_t* q_start,
                                        int B, int total_q, int max_new, const medusa_tree_t* tree,
                                        const int32_t* group_start, int n_groups, const int32_t* common, int H, int Hkv,
                                        int Dh, float rope_theta, float scale, medusa_dtype dtype, void* out,
                                        void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  const char* fn = "medusa_paged_attn_shared";
  if (n_groups < 0 || n_groups > MEDUSA_MAX_ROWS) return fail(MEDUSA_ERR_INVALID, "%s: n_groups=%d", fn, n_groups);
  if (n_groups > 0 && (!group_start || !common)) return fail(MEDUSA_ERR_INVALID, "%s: NULL array", fn);
  const Call c{q, q_stride, k_new, k_stride, v_new, v_stride, k_pages, v_pages, pages, rows, q_start, B, total_q,
               max_new, tree, H, Hkv, Dh, rope_theta, scale, dtype, out, workspace, workspace_bytes, err, stream};
  PagedAttnArgs a{};
  PagedKernels k{};
  const size_t bytes = medusa_paged_attn_shared_workspace_size(B, n_groups, total_q, max_new, H, Hkv, Dh, dtype);
  if (int rc = check_call(c, bytes, fn, a, k)) return rc;
  if (!a.total_q) return MEDUSA_OK;
  const int64_t line = 2ll * Hkv * Dh * (dtype == MEDUSA_BF16 ? 2 : 4);
  const int64_t most = (int64_t)pages->max_pages * pages->page_size < INT32_MAX ? (int64_t)pages->max_pages * pages->page_size
                                                                                : INT32_MAX;
  const bool few = (int64_t)max_new * a.g <= kFewRows;
  if (n_groups == 0 || (B - 1) * (most * line) < worth_sharing(total_q, H, Dh, dtype != MEDUSA_BF16, few))
    return attend<kAll>(c, a, k);
  const SharedWorkspace w = shared_workspace_of(B, n_groups, total_q, H, Dh, dtype, k.sms);
  auto* ws = static_cast<uint8_t*>(workspace);
  a.n_groups = n_groups;
  a.group_start = group_start;
  a.common = common;
  a.groups = reinterpret_cast<PagedGroup*>(ws + w.groups);
  a.from = reinterpret_cast<int32_t*>(ws + w.from);
  a.common_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.parts = reinterpret_cast<uint32_t*>(ws + w.parts);
  a.common_o = reinterpret_cast<float*>(ws + w.o);
  if (int rc = launch_paged_prep(a, Dh, dtype, true, k)) return rc;
  const bool few_common = (int64_t)total_q * a.g <= kFewRows;
  if (int rc = dtype == MEDUSA_BF16 ? launch_paged_chunk<kCommon>(a, Dh, k)
                                    : launch_paged_generic<kCommon>(a, Dh, few_common, k))
    return rc;
  if (int rc = launch_paged_join(a, Dh, dtype == MEDUSA_BF16 ? 128 : few_common ? 16 : 64, k)) return rc;
  a.counters = counters_of(c, few);
  if (dtype == MEDUSA_BF16) return few ? launch_paged_decode<kOwn>(a, Dh, k) : launch_paged_chunk<kOwn>(a, Dh, k);
  return launch_paged_generic<kOwn>(a, Dh, few, k);
}

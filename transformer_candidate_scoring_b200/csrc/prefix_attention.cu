// Attention of sequences that share their request's prefix (tr_prefix_attention): the plan, and the
// kernels that add each sequence's own keys and merge.
//
// For query token (s, t) and head h of request r, over the request's prefix keys and then the
// keys of the sequence's own suffix:
//     a_j = scale q.k_j,   m = max_j a_j,   l = sum_j exp(a_j - m),   o = sum_j exp(a_j - m) v_j / l
// with m, l and o carried from key to key (a new maximum rescales l and o), so that no score is
// ever stored.  Exponentials are powers of two: a_j is kept times log2(e).  The prefix part runs
// once per request for all of its sequences (prefix_attention_tc.cu, prefix_attention_f32.cu) and
// leaves one or, of a split prefix, several normalised partial results per row; short prefixes and small
// batches do without it.
#include <math.h>

#include <algorithm>

#include "prefix_attention.cuh"

namespace tr {
namespace attn {
namespace {

__device__ __forceinline__ int request_of(const AttnParams& p, int64_t s) {
  int lo = 0, hi = p.R - 1;        // the last request that starts at or before s and is not empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.req[mid].s0 <= s) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The suffix part of every row (with `simt`, the prefix too), and the merge with the prefix part's partial results.  A team of
// kLanes lanes holds a row, eight of its columns per lane; `parts` teams share a row's suffix
// keys and partial results where rows are few (their results meet in shared memory).  What it
// must read -- each sequence's own keys and values, the partial results -- bounds it: four keys
// are in flight per lane, and the suffix part does not wait for the prefix kernel.
constexpr int kFinishThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// A softmax row in progress: 2^(a - m) summed, and the values so weighted.
struct Running {
  float m = -INFINITY, l = 0.f, o[8] = {};
  __device__ __forceinline__ void rescale(float nm, float* base) {       // *base: what numerators are relative to
    *base = nm == -INFINITY ? 0.f : nm;                                  // keys of -inf weigh nothing, NaN stays NaN
    const float f = exp2f(m - *base);
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f;
    m = nm;
  }
  __device__ __forceinline__ float lse() const { return l == 0.f ? -INFINITY : m * kLn2 + logf(l); }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ bool not_finite(uint32_t w) {       // either of two bf16
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
// Joins the prefix part's results part, part + parts, ... of a row's n (the first at at0, the next `rows`
// further) for columns c0 .. c0 + 7, four at a time.
__device__ __forceinline__ void merge_prefix(const AttnParams& p, int n, int64_t at0, int64_t rows, int c0, bool in,
                                             int part, int parts, Running& x) {
  const int D = p.d.d_head;
  constexpr int kAhead = 4;
  for (int i0 = part; i0 < n; i0 += parts * kAhead) {
    float z[kAhead], oo[kAhead][8];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * parts;
      z[u] = i < n ? p.part_lse[at0 + i * rows] : -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) oo[u][e] = 0.f;
      if (in && i < n) {
        const float4* y = reinterpret_cast<const float4*>(p.part_o + (at0 + i * rows) * D + c0);
        const float4 f = y[0], g = y[1];
        oo[u][0] = f.x; oo[u][1] = f.y; oo[u][2] = f.z; oo[u][3] = f.w;
        oo[u][4] = g.x; oo[u][5] = g.y; oo[u][6] = g.z; oo[u][7] = g.w;
      }
    }
    float base;
    x.rescale(fmaxf(fmaxf(fmaxf(x.m, z[0]), fmaxf(z[1], z[2])), z[3]), &base);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float w = exp2f(z[u] - base);
      x.l += w;
#pragma unroll
      for (int e = 0; e < 8; ++e) x.o[e] = fmaf(w, oo[u][e], x.o[e]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store_row(const AttnParams& p, int64_t row, int c0, const Running& x) {
  const float inv = x.l == 0.f ? 0.f : 1.f / x.l;        // (a NaN score gives a NaN row)
  T* out = static_cast<T*>(p.out) + row * p.d.d_head + c0;
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(out)[0] = make_float4(x.o[0] * inv, x.o[1] * inv, x.o[2] * inv, x.o[3] * inv);
    reinterpret_cast<float4*>(out)[1] = make_float4(x.o[4] * inv, x.o[5] * inv, x.o[6] * inv, x.o[7] * inv);
  } else {
    *reinterpret_cast<uint4*>(out) = make_uint4(bf16x2(x.o[0] * inv, x.o[1] * inv), bf16x2(x.o[2] * inv, x.o[3] * inv),
                                                bf16x2(x.o[4] * inv, x.o[5] * inv), bf16x2(x.o[6] * inv, x.o[7] * inv));
  }
}

template <typename T, int kLanes>
__global__ void __launch_bounds__(kFinishThreads, 3) finish_kernel(const __grid_constant__ AttnParams p, int parts) {
  __shared__ float s_ml[kFinishThreads / kLanes][2];
  __shared__ float s_o[8][kFinishThreads];
  const int team = threadIdx.x / kLanes, tl = threadIdx.x % kLanes;
  const int rows_per = kFinishThreads / kLanes / parts, part = team / rows_per;
  const int64_t row_at = (int64_t)blockIdx.x * rows_per + team % rows_per;
  const bool live = row_at < p.n_rows;
  const int64_t row = live ? row_at : p.n_rows - 1;
  const int D = p.d.d_head, H = p.d.n_head, c0 = tl * 8;
  const bool in = c0 < D;
  const int tk = fast_div((int)row, p.div_h), h = (int)row - tk * H;       // (rows are below 2^31)
  const int64_t st = tk, s = fast_div(tk, p.div_lt);
  const int t = tk - (int)s * p.d.L_t, hk = fast_div(h, p.div_g);
  const RequestPlan& rq = p.req[request_of(p, s)];
  const float c = p.d.scale * kLog2e;
  Running x;
  if (p.d.suffix_cap > 0 || p.simt) {
    float q[8] = {};
    if (in) load8(static_cast<const T*>(p.q) + st * p.d.q_token + (int64_t)h * D + c0, q);
#pragma unroll 1
    for (int own = p.simt ? 0 : 1; own < 2; ++own) {       // the prefix's keys, the sequence's own
      const int n = own ? visible_suffix(p, s, t) : rq.p1 - rq.p0;
      const int64_t token = own ? p.d.suffix_token : p.d.prefix_token;
      const int64_t from = own ? s * p.d.suffix_seq + hk * p.d.suffix_head + c0 : rq.p0 * token + hk * p.d.prefix_head + c0;
      const T *k = static_cast<const T*>(own ? p.k_suffix : p.k_prefix) + from, *v = static_cast<const T*>(own ? p.v_suffix : p.v_prefix) + from;
      const int per = (n + parts - 1) / parts, end = min(n, (part + 1) * per);
      const int steps = __reduce_max_sync(0xffffffffu, max(0, end - part * per));    // of the warp's teams
      constexpr int kAhead = 4;
      for (int i0 = 0; i0 < steps; i0 += kAhead) {
        float a[kAhead], vv[kAhead][8];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int j = part * per + i0 + u;
          float kk[8] = {};
          a[u] = 0.f;
          if (in && j < end) load8(k + j * token, kk);
#pragma unroll
          for (int e = 0; e < 8; ++e) a[u] = fmaf(q[e], kk[e], a[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int j = part * per + i0 + u;
#pragma unroll
          for (int e = 0; e < 8; ++e) vv[u][e] = 0.f;
          if (in && j < end) load8(v + j * token, vv[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
          for (int y = kLanes / 2; y; y >>= 1) a[u] += __shfl_xor_sync(0xffffffffu, a[u], y);
          a[u] = part * per + i0 + u < end ? a[u] * c : -INFINITY;
        }
        float base;
        x.rescale(fmaxf(fmaxf(fmaxf(x.m, a[0]), fmaxf(a[1], a[2])), a[3]), &base);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float w = exp2f(a[u] - base);
          x.l += w;
#pragma unroll
          for (int e = 0; e < 8; ++e) x.o[e] = fmaf(w, vv[u][e], x.o[e]);
        }
      }
    }
  }
  // ---- the prefix part's results
  cudaGridDependencySynchronize();
  const int64_t rows = (int64_t)(rq.s1 - rq.s0) * p.d.L_t * H;
  const int64_t at0 = rq.part + (row - (int64_t)rq.s0 * p.d.L_t * H);
  merge_prefix(p, results_of(p, rq), at0, rows, c0, in, part, parts, x);
  if (parts > 1) {
    if (tl == 0) {
      s_ml[team][0] = x.m;
      s_ml[team][1] = x.l;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s_o[e][threadIdx.x] = x.o[e];
    __syncthreads();
    if (part > 0) return;
    for (int i = 1; i < parts; ++i) {
      const int other = team + i * rows_per;
      float base;
      const float m = s_ml[other][0];
      x.rescale(fmaxf(x.m, m), &base);
      const float w = exp2f(m - base);
      x.l = fmaf(w, s_ml[other][1], x.l);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.o[e] = fmaf(w, s_o[e][other * kLanes + tl], x.o[e]);
    }
  }
  if (!live) return;
  if (in) store_row<T>(p, row, c0, x);
  if (p.lse && tl == 0) p.lse[row] = x.lse();
}

int finish_lanes(int D) { return D <= 8 ? 1 : D <= 16 ? 2 : D <= 32 ? 4 : D <= 64 ? 8 : 16; }
// Teams per row: several while there are few rows and enough keys or partial results to share, about 16 warps per SM.
int finish_parts(const AttnParams& p, int sms, bool simt) {
  const int lanes = finish_lanes(p.d.d_head);
  int parts = 1, items = p.d.suffix_cap;
  for (int r = 0; r < p.R; ++r) items = std::max(items, simt ? p.req[r].p1 - p.req[r].p0 : p.req[r].n_split);
  while (parts < 16 && parts * 2 <= kFinishThreads / lanes && items > 4 * parts &&
         p.n_rows * lanes * parts * 2 <= (int64_t)sms * 16 * 32)
    parts *= 2;
  return parts;
}

template <typename T, int kLanes>
tr_status launch_finish(const AttnParams& p, int sms, cudaStream_t st) {
  const int parts = finish_parts(p, sms, p.simt);
  const int rows_per = kFinishThreads / kLanes / parts;
  return launch_dependent(p.n_units > 0, finish_kernel<T, kLanes>, (unsigned)((p.n_rows + rows_per - 1) / rows_per), kFinishThreads, 0, st,
                          "finish_kernel", p, parts);
}
template <typename T>
tr_status launch_finish(const AttnParams& p, int sms, cudaStream_t st) {
  switch (finish_lanes(p.d.d_head)) {
    case 1: return launch_finish<T, 1>(p, sms, st);
    case 2: return launch_finish<T, 2>(p, sms, st);
    case 4: return launch_finish<T, 4>(p, sms, st);
    case 8: return launch_finish<T, 8>(p, sms, st);
    default: return launch_finish<T, 16>(p, sms, st);
  }
}

// The same for bf16 suffixes of eight tokens and more, on warp-level matrix instructions: of the L_t x
// (n_head / n_kv_head) rows of a sequence that share a key head, eight are the columns of
// S^T = K Q^T (16 keys x 8 rows) and of O^T += V^T P^T, so each key and value is read once for all of them,
// through shared memory, whole rows at a time (the order of d_head within a product is free, so a
// lane's 16 bytes of a key are its share of two slices, and of values its share of eight).  P^T
// turns from a result into an operand by a transpose between lanes.  `parts` warps share a
// sequence's keys; all meet in shared memory, where the prefix part's results join.  The read of the
// keys and values bounds it: a warp has 16 of each in flight.  512 sequences with 61 to 64 tokens, 8 key heads
// of 128: 127 MB in 33 us, the chain of a CTA (its length, its rows, its products, the merge) times seven
// waves at 16 warps per SM.  The call took 107 us with the rows read straight into the products' registers, 16
// bytes of eight rows at a time, against 99; five CTAs per SM at 102 registers 100.5, six with spills 107.
// With the rows in registers, a persistent grid that brings the next unit's rows to L2 meanwhile took 127,
// the same without the persistent grid 114.
constexpr int kSuffixThreads = 128;

__device__ __forceinline__ void mma_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, lane l holding columns 2 (l % 4), + 1 of row l / 4, to its transpose.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

template <int kBlocks, bool kCausal>     // 64-wide blocks of d_head
__global__ void __launch_bounds__(kSuffixThreads, kBlocks == 1 ? 6 : 4)
suffix_kernel(const __grid_constant__ AttnParams p, int log_parts, int r_tiles, const FastDiv div_tiles, const FastDiv div_chunks) {
  constexpr int DP = kBlocks * 64;
  // a warp's 16 keys and 16 values, 16-byte piece c of row r at piece c ^ (r & 7); then its result
  constexpr int kRow = DP * 2, kWarpBytes = 32 * kRow;
  static_assert(8 * (DP + 4) * 4 <= kWarpBytes, "a warp's result");
  __shared__ __align__(128) uint8_t s_kv[kSuffixThreads / 32][kWarpBytes];
  __shared__ float s_m[kSuffixThreads / 32][8], s_l[kSuffixThreads / 32][8];
  auto s_o = [&](int w, int r, int c) { return reinterpret_cast<float*>(s_kv[w]) + r * (DP + 4) + c; };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, qd = lane % 4;
  const int parts = 1 << log_parts, part = warp & (parts - 1), D = p.d.d_head, H = p.d.n_head, Hk = p.d.n_kv_head;
  const int G = p.group, n_rows = p.d.L_t * G;
  const int n_unit = p.req[p.R].s0 * Hk * r_tiles;         // below 2^31: no more than query rows
  const int u_at = (int)(((int64_t)blockIdx.x * (kSuffixThreads / 32) + warp) >> log_parts), u = min(u_at, n_unit - 1);
  const int sh = fast_div(u, div_tiles), s = fast_div(sh, p.div_kv), hk = sh - s * Hk;
  const int row0 = (u - sh * r_tiles) * 8;                 // rows t * G + head in group
  const float c = p.d.scale * kLog2e;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint32_t kv = (uint32_t)__cvta_generic_to_shared(s_kv[warp]);
  auto piece = [&](int r, int c) {                         // rows 0-15 keys, 16-31 values
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(kv + r * kRow + ((c ^ (r & 7)) << 4)));
    return v;
  };
  const int len = visible_suffix(p, s, p.d.L_t - 1);       // what the last query token sees: all of it
  // ---- Q: 16 bytes of row g per 32 columns
  uint4 q[2 * kBlocks];
  {
    const int r = row0 + g, t = fast_div(r, p.div_g);
    const __nv_bfloat16* src =
        static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)s * p.d.L_t + t) * p.d.q_token + (hk * G + r - t * G) * D;
#pragma unroll
    for (int i = 0; i < 2 * kBlocks; ++i)
      q[i] = r < n_rows && i * 32 + qd * 8 < D ? __ldg(reinterpret_cast<const uint4*>(src + i * 32 + qd * 8)) : zero;
  }
  // keys that rows 2 qd and 2 qd + 1 see
  int seen[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    seen[e] = kCausal ? max(0, len - max(0, p.d.L_t - 1 - fast_div(row0 + 2 * qd + e, p.div_g))) : len;
  const int seen_by_all = kCausal ? max(0, len - (p.d.L_t - 1 - fast_div(row0, p.div_g))) : len;
  const RequestPlan& rq = p.req[request_of(p, s)];
  const int pre = p.simt ? rq.p1 - rq.p0 : 0, pre_steps = (pre + 15) / 16, steps = pre_steps + (len + 15) / 16;
  float o[4 * kBlocks][4] = {};                            // O^T: 16 columns of d_head x 8 rows
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int i = part; i < steps; i += parts) {              // of 16 keys: with simt, the prefix's, then the sequence's own
    const bool own = i >= pre_steps;
    const int j0 = (own ? i - pre_steps : i) * 16, n = own ? len : pre;
    const int64_t token = own ? p.d.suffix_token : p.d.prefix_token;
    const int64_t from = own ? (int64_t)s * p.d.suffix_seq + hk * p.d.suffix_head : rq.p0 * token + hk * p.d.prefix_head;
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(own ? p.k_suffix : p.k_prefix) + from;
    const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(own ? p.v_suffix : p.v_prefix) + from;
    __syncwarp();                                          // (the rows of the step before have been read)
    constexpr int kPieces = DP / 8, kRows = 32 / kPieces;  // rows a warp copies at a time
    {
      const int c = lane % kPieces;
#pragma unroll
      for (int r = lane / kPieces; r < 16; r += kRows) {
        const int j = j0 + r, bytes = j < n && c * 8 < D ? 16 : 0;              // 0: zeros
        const int64_t at = bytes ? j * token + c * 8 : 0;
        const uint32_t dst = kv + r * kRow + ((c ^ (r & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(kp + at), "r"(bytes) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * kRow), "l"(vp + at), "r"(bytes) : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    float st[4] = {};                                      // keys g (0, 1) and g + 8 (2, 3) x rows 2 qd, 2 qd + 1
#pragma unroll
    for (int i = 0; i < 2 * kBlocks; ++i) {
      const uint4 k0 = piece(g, qd + 4 * i), k1 = piece(g + 8, qd + 4 * i);
      mma_16816(st, k0.x, k1.x, k0.y, k1.y, q[i].x, q[i].y);
      mma_16816(st, k0.z, k1.z, k0.w, k1.w, q[i].z, q[i].w);
    }
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int sees = own ? seen[e] : n;
      const float a0 = j0 + g < sees ? st[e] * c : -INFINITY, a1 = j0 + g + 8 < sees ? st[2 + e] * c : -INFINITY;
      float top = fmaxf(m[e], fmaxf(a0, a1));
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = top == -INFINITY ? 0.f : top;     // keys of -inf weigh nothing, NaN stays NaN
      f[e] = exp2f(m[e] - base);
      m[e] = top;
      st[e] = exp2f(a0 - base);
      st[2 + e] = exp2f(a1 - base);
      l[e] = l[e] * f[e] + st[e] + st[2 + e];              // (this lane's keys only)
    }
    // Of keys that only the later of the rows see, the product's 0 x V of the others is 0 unless V is
    // infinite or NaN: then every row adds the keys it sees, one by one.
    if (kCausal && own && j0 + 16 > seen_by_all && len > seen_by_all) {
      bool odd = false;
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint4 v = piece(16 + lane / 8 + 4 * h, lane % 8 + 8 * b);
          odd = odd || not_finite(v.x) || not_finite(v.y) || not_finite(v.z) || not_finite(v.w);
        }
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
        for (int i = 0; i < 4 * kBlocks; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= f[e & 1];
        for (int jj = 0; jj < 16 && j0 + jj < len; ++jj) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) w[e] = __shfl_sync(0xffffffffu, jj < 8 ? st[e] : st[2 + e], (jj & 7) * 4 + qd);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            float y[8] = {};
            if (b * 64 + g * 8 < D) load8(vp + (j0 + jj) * token + b * 64 + g * 8, y);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (j0 + jj < seen[e])
#pragma unroll
                for (int x = 0; x < 8; ++x) o[4 * b + x / 2][2 * (x & 1) + e] = fmaf(w[e], y[x], o[4 * b + x / 2][2 * (x & 1) + e]);
          }
        }
        continue;
      }
    }
    const uint32_t b0 = transpose_8x8(bf16x2(st[0], st[1])), b1 = transpose_8x8(bf16x2(st[2], st[3]));
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      uint4 v[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = piece(16 + 2 * qd + (h & 1) + (h >> 1) * 8, g + 8 * b);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // rows of A: columns 8 g' + 2 w and + 1 of the block, g' = 0 .. 7 in lanes' order
        const int i = 4 * b + w;
        uint32_t x[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) x[h] = (&v[h].x)[w];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= f[e & 1];
        mma_16816(o[i], __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x5410),
                  __byte_perm(x[2], x[3], 0x7632), b0, b1);
      }
    }
  }
  __syncwarp();
  // ---- o[i][0], [1]: column b * 64 + 8 g + 2 w of rows 2 qd, 2 qd + 1; [2], [3]: the next column
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
    if (g == 0) {
      s_m[warp][2 * qd + e] = m[e];
      s_l[warp][2 * qd + e] = l[e];
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      float* d = s_o(warp, 2 * qd + e, b * 64 + 8 * g);
      *reinterpret_cast<float4*>(d) = make_float4(o[4 * b][e], o[4 * b][2 + e], o[4 * b + 1][e], o[4 * b + 1][2 + e]);
      *reinterpret_cast<float4*>(d + 4) = make_float4(o[4 * b + 2][e], o[4 * b + 2][2 + e], o[4 * b + 3][e], o[4 * b + 3][2 + e]);
    }
  }
  cudaGridDependencySynchronize();
  __syncthreads();
  // ---- eight columns of a row per thread: the warps' results, then the prefix part's
  if (u_at >= n_unit) return;
  const int64_t rows = (int64_t)(rq.s1 - rq.s0) * p.d.L_t * H;
  const int chunks = D / 8, first = warp - part, n_results = results_of(p, rq);
  const int items = min(8, n_rows - row0) * chunks;
  // `share` neighbouring lanes divide a row's results where threads are to spare
  int share = 1, log_share = 0;
  while (share < 8 && 4 * share < n_results && items * share * 2 <= parts * 32) share = 1 << ++log_share;
  for (int at = part * 32 + lane; at < items * share; at += parts * 32) {
    const int item = at >> log_share, mine = at & (share - 1);
    const int rr = fast_div(item, div_chunks), c0 = (item - rr * chunks) * 8, r = row0 + rr, t = fast_div(r, p.div_g);
    const int64_t row = ((int64_t)s * p.d.L_t + t) * H + hk * G + r - t * G;
    Running x;
    for (int i = mine; i < parts; i += share) {
      const float mm = s_m[first + i][rr];
      float base;
      x.rescale(fmaxf(x.m, mm), &base);
      const float f = exp2f(mm - base);
      x.l = fmaf(f, s_l[first + i][rr], x.l);
      const float4 y = *reinterpret_cast<const float4*>(s_o(first + i, rr, c0)), z = *reinterpret_cast<const float4*>(s_o(first + i, rr, c0 + 4));
      const float w[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) x.o[e] = fmaf(f, w[e], x.o[e]);
    }
    merge_prefix(p, n_results, rq.part + (row - (int64_t)rq.s0 * p.d.L_t * H), rows, c0, true, mine, share, x);
    for (int y = 1; y < share; y <<= 1) {
      const uint32_t group = ((1u << share) - 1) << (lane & ~(share - 1));
      float base;                                          // (both lanes': then their sums add up)
      x.rescale(fmaxf(x.m, __shfl_xor_sync(group, x.m, y)), &base);
      x.l += __shfl_xor_sync(group, x.l, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.o[e] += __shfl_xor_sync(group, x.o[e], y);
    }
    if (mine > 0) continue;
    store_row<__nv_bfloat16>(p, row, c0, x);
    if (p.lse && c0 == 0) p.lse[row] = x.lse();
  }
}

template <int kBlocks, bool kCausal>
tr_status launch_suffix(const AttnParams& p, int sms, cudaStream_t st) {
  const int r_tiles = (p.d.L_t * (p.d.n_head / p.d.n_kv_head) + 7) / 8;
  const int64_t n_unit = (int64_t)p.req[p.R].s0 * p.d.n_kv_head * r_tiles;
  // a warp per 16 own keys or per eight results of the prefix, up to the four of a CTA; where these leave warps
  // to spare, one per 16 keys of the prefix too (with simt)
  int steps = (p.d.suffix_cap + 15) / 16, keys = 0;
  for (int r = 0; r < p.R; ++r) {
    steps = std::max(steps, p.req[r].n_split / 8);
    if (p.simt && p.req[r].s1 > p.req[r].s0) keys = std::max(keys, p.req[r].p1 - p.req[r].p0);
  }
  int log_parts = steps >= 4 ? 2 : steps >= 2 ? 1 : 0;
  while (log_parts < 2 && (2 << log_parts) <= steps + ceil_div(keys, 16) && (n_unit << log_parts) <= (int64_t)sms * 8) ++log_parts;
  const int units = (kSuffixThreads / 32) >> log_parts;
  return launch_dependent(p.n_units > 0, suffix_kernel<kBlocks, kCausal>, (unsigned)((n_unit + units - 1) / units), kSuffixThreads, 0, st, "suffix_kernel", p,
                          log_parts, r_tiles, fast_div_by((uint32_t)r_tiles), fast_div_by((uint32_t)(p.d.d_head / 8)));
}

tr_status check_offsets(const tr_attn_desc* d, const int64_t* seq, const int64_t* prefix, int R) {
  if (!d) return fail(TR_ERR_INVALID_ARG, "desc is null");
  if (d->dtype != TR_F32 && d->dtype != TR_BF16) return fail(TR_ERR_INVALID_ARG, "dtype=%d", (int)d->dtype);
  if (d->n_kv_head < 1 || d->n_head < 1 || d->n_head > 1024 || d->n_head % d->n_kv_head)
    return fail(TR_ERR_INVALID_ARG, "n_head=%d, n_kv_head=%d: need a multiple of n_kv_head, 1..1024", d->n_head, d->n_kv_head);
  if (d->d_head < 8 || d->d_head % 8 || d->d_head > kMaxDHead)
    return fail(TR_ERR_UNSUPPORTED, "d_head=%d: need a multiple of 8 <= %d", d->d_head, kMaxDHead);
  if (d->L_t < 1 || d->L_t > TR_MAX_LT) return fail(TR_ERR_INVALID_ARG, "L_t=%d (need 1..%d)", d->L_t, TR_MAX_LT);
  if (d->causal != 0 && d->causal != 1) return fail(TR_ERR_INVALID_ARG, "causal=%d", d->causal);
  if (d->suffix_cap < 0) return fail(TR_ERR_INVALID_ARG, "suffix_cap=%d", d->suffix_cap);
  if (!(isfinite(d->scale) && d->scale > 0)) return fail(TR_ERR_INVALID_ARG, "scale=%g: need a positive number", (double)d->scale);
  const int64_t unit = d->dtype == TR_F32 ? 4 : 8;
  const int64_t strides[6] = {d->q_token, d->prefix_token, d->prefix_head, d->suffix_seq, d->suffix_token, d->suffix_head};
  for (int i = 0; i < (d->suffix_cap > 0 ? 6 : 3); ++i)
    if (strides[i] <= 0 || strides[i] % unit || strides[i] > (1ll << 38))
      return fail(TR_ERR_INVALID_ARG, "stride %d = %lld elements: need a positive multiple of 16 bytes", i, (long long)strides[i]);
  if (R < 1 || R > TR_MAX_REQUESTS) return fail(TR_ERR_INVALID_ARG, "R=%d (need 1..%d)", R, TR_MAX_REQUESTS);
  if (!seq || !prefix) return fail(TR_ERR_INVALID_ARG, "null host array");
  if (seq[0] != 0) return fail(TR_ERR_INVALID_ARG, "seq_offsets must start at 0");
  if (prefix[0] < 0) return fail(TR_ERR_INVALID_ARG, "prefix_offsets must not be negative");
  for (int r = 0; r < R; ++r) {
    if (seq[r + 1] < seq[r]) return fail(TR_ERR_INVALID_ARG, "seq_offsets decrease at %d", r);
    if (prefix[r + 1] < prefix[r]) return fail(TR_ERR_INVALID_ARG, "prefix_offsets decrease at %d", r);
  }
  if (prefix[R] > INT32_MAX) return fail(TR_ERR_UNSUPPORTED, "2^31 or more prefix tokens");
  if (seq[R] > INT32_MAX || seq[R] * d->L_t * d->n_head > (int64_t)INT32_MAX)
    return fail(TR_ERR_UNSUPPORTED, "2^31 or more query rows (n * L_t * n_head)");
  return TR_OK;
}

// How many steps of keys a unit takes.  Fewer steps give more units to spread over the `slots` (SMs,
// or CTAs that share one), but every unit costs kUnitSteps more and every chunk of a prefix a partial
// result per row.  The candidates are: no split, and the shortest chunks that give one, two or four units per slot.  With `direct`, no split also saves the
// merge's launch (about 4 us), and requests without a prefix have one (empty) unit per 256 rows.
// With `runs`, equal runs of steps are a candidate too, at a unit more per CTA: 16 requests of 2048 to 8192 tokens
// and 32 sequences take 107 us by runs and 122 without, the 18 requests at kUnitSteps 45 and 50.
// Returns the cost.
double plan_units(AttnParams& p, int unit_rows, int step_keys, int slots, bool direct, bool runs) {
  const int G = p.d.n_head / p.d.n_kv_head;
  int steps[TR_MAX_REQUESTS], n_m[TR_MAX_REQUESTS];
  int longest = 0;
  int64_t rows_all = 0;
  bool two = false;
  for (int r = 0; r < p.R; ++r) {
    const int64_t m = (int64_t)(p.req[r].s1 - p.req[r].s0) * p.d.L_t * G;
    steps[r] = m > 0 ? ceil_div(p.req[r].p1 - p.req[r].p0, step_keys) : 0;
    n_m[r] = ceil_div(m, unit_rows);
    two = two || m > unit_rows / 2;
    longest = std::max(longest, steps[r]);
    rows_all += request_rows(p, r);
  }
  auto units = [&](int c) {
    int64_t n = 0;
    for (int r = 0; r < p.R; ++r) {
      const int chunks = ceil_div(steps[r], c);
      n += (int64_t)p.d.n_kv_head * n_m[r] * (direct && c >= longest ? std::max(chunks, 1) : chunks);
    }
    return n;
  };
  int best = std::max(longest, 1);
  double best_cost = 1e300;
  for (int w = 0; w <= 4 && longest > 0; w = w ? 2 * w : 1) {
    int c = longest;
    if (w > 0) {
      int lo = 1, hi = longest;               // units(c) falls with c
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (units(mid) <= (int64_t)w * slots) hi = mid; else lo = mid + 1;
      }
      c = lo;
    }
    // tile steps of the busiest SM (about 0.7 us each), and the partial results' traffic
    const double waves = (double)((units(c) + slots - 1) / slots);
    const double split = (double)ceil_div(longest, c);
    const double bytes = split > 1 ? (double)rows_all * split * p.d.d_head * 8.0 : 0.0;
    const double cost = waves * (c * (two ? 2.0 : 1.0) + kUnitSteps) + bytes / 3.5e6 + (direct && split > 1 ? 6.0 : 0.0);
    if (cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  if (runs && longest > 0 && p.d.n_kv_head <= slots && *std::max_element(n_m, n_m + p.R) == 1) {
    int line = 0, filled = 0;                 // (below 2^24 + R (1 + kUnitSteps))
    for (int r = 0; r < p.R; ++r) {
      line += steps[r] > 0 ? steps[r] + kUnitSteps : 0;
      filled += steps[r] > 0;
    }
    const int run = ceil_div(line, slots / p.d.n_kv_head), n = ceil_div(line, run);
    const double split = 1.0 + (double)line / ((double)run * filled);
    const double cost = run * (two ? 2.0 : 1.0) + kUnitSteps + (double)rows_all * split * p.d.d_head * 8.0 / 3.5e6 +
                        (direct ? 6.0 : 0.0);
    if (cost < best_cost) {
      best_cost = cost;
      p.run = run;
      p.div_run = fast_div_by((uint32_t)run);
      p.n_units = n * p.d.n_kv_head;
    }
  }
  int unit = 0;
  int64_t part = 0;
  for (int r = 0; r < p.R; ++r) {
    RequestPlan& q = p.req[r];
    q.first_unit = unit;
    q.chunk = p.run > 0 ? steps[r] : best;
    // (n places meet at most ceil(n / run) + 1 runs)
    const int places = steps[r] > 0 ? steps[r] + kUnitSteps : 0;
    q.n_split = p.run > 0 ? (places > 0 ? ceil_div(places, p.run) + 1 : 0) : ceil_div(steps[r], best);
    if (direct && p.run == 0 && best >= longest && q.s1 > q.s0) q.n_split = 1;
    q.n_m = n_m[r];
    q.div_m = fast_div_by((uint32_t)std::max(q.n_m, 1));
    q.div_split = fast_div_by((uint32_t)std::max(q.n_split, 1));
    q.part = part;
    unit += p.run > 0 ? places : p.d.n_kv_head * n_m[r] * q.n_split;
    part += request_rows(p, r) * q.n_split;
  }
  p.req[p.R].first_unit = unit;
  p.halves = kNoHalves;
  if (p.run == 0) p.n_units = unit;
  // A last or only wave that leaves half of the SMs idle: its units in halves, one tile of rows each, take half the
  // time (2 requests x 4096 sequences over 4096 tokens, 16 heads of 128 on 4, 3.46 waves: 315 -> 286 us)
  const int rest = unit % slots;
  if (runs && p.run == 0 && two && rest > 0 && 2 * rest <= slots) {
    p.halves = unit - rest;
    p.n_units = unit + rest;
  }
  p.req[p.R].part = part;
  return longest > 0 ? best_cost : 0.0;
}

constexpr int kMmaSuffix = 8;      // own tokens from which suffix_kernel takes them (bf16)

// Whether the kernel of the own keys reads the prefixes too, row by row or sequence by sequence: one launch and no
// partial results, but keys are read again for every row (finish_kernel) or sequence (suffix_kernel).  In us, the prefix
// kernel's cost is 3 and 0.74 (fp32: 1.8) per step of the plan's, and 8 bytes per partial result; finish_kernel takes
// 3.1 ps (fp32: 4.5) per key and lane of a row or 0.27 us per key in turn, and 5 us and 25 ps per lane beside; suffix_kernel
// 0.6 ns (d_head up to 64: 0.4) per 16 keys of a sequence and key head.  Without and with:
//   16 x 300 sequences, 16 heads of 128 on 8, 23 own keys, prefixes of 2, 32, 64 keys    190 and 154, 175, 221 us (the choice changes between 16 and 32)
//   4 x 4, 8 heads of 128, 40 own keys, prefixes of 2, 64, 128                           11.5 and 4.2, 5.2, 6.1
//   5 x 459, 16 heads of 96 on 2, two own keys, prefixes of 2, 8                         43 and 28, 34
//   24 x 77 fp32, 32 heads of 128 on 8, none, prefixes of 2, 8, 16                       112 and 32, 49, 83
//   1 x 4, 8 heads of 64, four own keys, prefixes of 2, 64, 200                          8.8 and 4.7, 5.0, 6.9
bool take_simt(AttnParams& p, int sms, double cost, bool direct) {
  const tr_attn_desc& d = p.d;
  const bool f32 = d.dtype == TR_F32, mma = !f32 && d.suffix_cap >= kMmaSuffix;
  const int lanes = finish_lanes(d.d_head), tiles = ceil_div((int64_t)d.L_t * p.group, 8);
  double simt = 0.0;
  int longest = 0, split = 0;
  for (int r = 0; r < p.R; ++r) {
    const RequestPlan& q = p.req[r];
    const int keys = q.s1 > q.s0 ? q.p1 - q.p0 : 0;
    longest = std::max(longest, keys);
    split = std::max(split, q.n_split);
    simt += mma ? (double)(q.s1 - q.s0) * d.n_kv_head * tiles * ceil_div(keys, 16) * (d.d_head > 64 ? 0.6e-3 : 0.4e-3)
                : (double)request_rows(p, r) * lanes * keys * (f32 ? 4.5e-6 : 3.1e-6);
  }
  simt = mma ? simt + 0.2 * ceil_div(longest, 16) : std::max(simt, 0.27 * ceil_div(longest, finish_parts(p, sms, true)));
  if (direct) simt += 5.0 + 2.5e-5 * p.n_rows * lanes;
  const double partial = direct || split > 1 ? 0.0 : (double)p.n_rows * d.d_head * 8.0 / 3.5e6;
  if (longest > 0 && simt >= 3.0 + (f32 ? 1.8 : 0.74) * (cost + partial)) return false;
  p.simt = true;
  p.n_units = p.run = 0;
  for (int r = 0; r < p.R; ++r) p.req[r].n_split = 0;
  return true;
}

struct Plan {
  bool direct = false;        // the tensor-core kernel writes the results
  size_t bytes = 0;
  int sms = 0, unit_rows = 0;
};
tr_status make_plan(const tr_attn_desc* d, const int64_t* seq, const int64_t* prefix, int R, AttnParams& p, Plan& plan) {
  TR_TRY(check_offsets(d, seq, prefix, R));
  p.d = *d;
  p.R = R;
  p.n_rows = seq[R] * d->L_t * d->n_head;
  p.div_g = fast_div_by((uint32_t)(d->n_head / d->n_kv_head));
  p.div_lt = fast_div_by((uint32_t)d->L_t);
  p.div_kv = fast_div_by((uint32_t)d->n_kv_head);
  p.div_h = fast_div_by((uint32_t)d->n_head);
  p.group = d->n_head / d->n_kv_head;
  for (int r = 0; r <= R; ++r) {
    RequestPlan& q = p.req[r];
    q.s0 = (int)seq[r];
    q.p0 = (int)prefix[r];
    q.s1 = (int)seq[std::min(r + 1, R)];
    q.p1 = (int)prefix[std::min(r + 1, R)];
  }
  TR_TRY(sm_count(&plan.sms));
  if (d->dtype == TR_F32) {
    // two CTAs per SM; units of 16 rows waste less of the few rows of small batches, units of 64
    // read K and V a quarter as often
    int64_t most = 0;
    for (int r = 0; r < R; ++r) most = std::max(most, (seq[r + 1] - seq[r]) * d->L_t * (d->n_head / d->n_kv_head));
    plan.unit_rows = most <= 32 ? 16 : 64;
    const double cost = plan_units(p, plan.unit_rows, kStepKeysF32, 2 * plan.sms, false, false);
    if (take_simt(p, plan.sms, cost, false)) return TR_OK;
    plan.bytes = (size_t)p.req[R].part * (d->d_head + 1) * sizeof(float);
    return TR_OK;
  }
  plan.unit_rows = kUnitRows;
  const double cost = plan_units(p, kUnitRows, kStepKeys, plan.sms, d->suffix_cap <= kDirectSuffix, true);
  plan.direct = d->suffix_cap <= kDirectSuffix && p.run == 0;
  for (int r = 0; r < R; ++r) plan.direct = plan.direct && (p.req[r].n_split == 1 || p.req[r].s0 == p.req[r].s1);
  if (take_simt(p, plan.sms, cost, plan.direct)) {
    plan.direct = false;
    return TR_OK;
  }
  if (!plan.direct) plan.bytes = (size_t)p.req[R].part * (d->d_head + 1) * sizeof(float);
  return TR_OK;
}

}  // namespace
}  // namespace attn
}  // namespace tr

using namespace tr;
using namespace tr::attn;

extern "C" size_t tr_prefix_attention_workspace(const tr_attn_desc* desc, const int64_t* seq_offsets,
                                                const int64_t* prefix_offsets, int R) {
  AttnParams p{};
  Plan plan;
  return make_plan(desc, seq_offsets, prefix_offsets, R, p, plan) == TR_OK ? plan.bytes : SIZE_MAX;
}

extern "C" tr_status tr_prefix_attention(const tr_attn_desc* desc, const void* q, const int64_t* seq_offsets,
                                         const void* k_prefix, const void* v_prefix, const int64_t* prefix_offsets,
                                         const void* k_suffix, const void* v_suffix, const int32_t* suffix_len, int R,
                                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                                         tr_stream stream) {
  TR_TRY(check_offsets(desc, seq_offsets, prefix_offsets, R));
  if (seq_offsets[R] == 0) return TR_OK;
  if (!q || !out) return fail(TR_ERR_INVALID_ARG, "null device pointer");
  if (prefix_offsets[R] > prefix_offsets[0] && (!k_prefix || !v_prefix))
    return fail(TR_ERR_INVALID_ARG, "k_prefix or v_prefix is null");
  if (desc->suffix_cap > 0 && (!k_suffix || !v_suffix || !suffix_len))
    return fail(TR_ERR_INVALID_ARG, "k_suffix, v_suffix or suffix_len is null");
  if (((uintptr_t)q | (uintptr_t)k_prefix | (uintptr_t)v_prefix | (uintptr_t)k_suffix | (uintptr_t)v_suffix |
       (uintptr_t)out) % 16)
    return fail(TR_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  if ((uintptr_t)suffix_len % 4 || (uintptr_t)lse % 4) return fail(TR_ERR_INVALID_ARG, "suffix_len or lse is not aligned to its type");
  AttnParams p{};
  Plan plan;
  TR_TRY(make_plan(desc, seq_offsets, prefix_offsets, R, p, plan));
  if (plan.bytes > 0 && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < plan.bytes))
    return fail(TR_ERR_INVALID_ARG, "workspace: need %zu bytes, 16-byte aligned", plan.bytes);
  DeviceState* ds = nullptr;
  TR_TRY(device_state(&ds));
  const cudaStream_t st = (cudaStream_t)stream;
  p.q = q;
  p.k_prefix = k_prefix;
  p.v_prefix = v_prefix;
  p.k_suffix = k_suffix;
  p.v_suffix = v_suffix;
  p.suffix_len = suffix_len;
  p.out = out;
  p.lse = lse;
  p.status = ds->status;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + p.req[R].part * desc->d_head;
  if (desc->dtype == TR_F32) {
    if (p.n_units > 0) TR_TRY(launch_prefix_f32(p, plan.unit_rows, st));
    return launch_finish<float>(p, plan.sms, st);
  }
  if (p.n_units > 0) TR_TRY(launch_prefix_tc(p, plan.direct, st));
  if (plan.direct) return TR_OK;
  if (desc->suffix_cap >= kMmaSuffix) {
    if (desc->d_head <= 64) return desc->causal ? launch_suffix<1, true>(p, plan.sms, st) : launch_suffix<1, false>(p, plan.sms, st);
    return desc->causal ? launch_suffix<2, true>(p, plan.sms, st) : launch_suffix<2, false>(p, plan.sms, st);
  }
  return launch_finish<__nv_bfloat16>(p, plan.sms, st);
}

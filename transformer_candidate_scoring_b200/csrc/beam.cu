// Beam decoding: selection over beams and vocabulary, and the reordering of beam states.
//
// Selection.  total(b, v) = cum[b] + x[b][v] - log sum_u exp(x[b][u]); the k best (b, v) of each
// request.  The logits are the traffic (2 or 4 bytes per (b, v), read once); the results are a
// few KB.  Two launches:
//   beam_chunk_kernel  one CTA per (row, chunk of 256 threads x 8 16-byte vectors), the chunk
//     held in registers between its uses: the running maximum and the sum of exponentials of
//     the chunk, and the chunk's candidates -- every logit that reaches a threshold below which
//     no chunk element can be among the k best.  The threshold is the k-th largest of the 256
//     threads' own maxima (at least k elements reach it, and for a vocabulary in no particular
//     order not many more than k do), found by bisection with one block-wide count per step.
//   beam_merge_kernel  one CTA per request: the rows' log-sum-exp from the chunks' sums (in 64
//     bits: two beams' totals are compared across rows), the same threshold step over all
//     candidates' totals, then a sort of the few that remain.
// When more elements reach a threshold than its buffer holds (long runs of equal logits), the
// exact k-th key is found by bisection over the elements themselves.
//
// Which thread sums which token depends on the token alone, not on the row's address, so equal
// rows get equal sums and ties between their beams stay ties.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "model.cuh"

namespace tr {
namespace {

constexpr int kChunkThreads = 256;
constexpr int kVecs = 8;                 // 16-byte vectors per thread
constexpr int kMergeThreads = 512;
constexpr int kMergeCap = 2048;          // candidates the final sort takes
constexpr int kTokenBits = 24;

template <typename T> struct Vec { static constexpr int N = 16 / sizeof(T); };
template <typename T> constexpr int chunk_elems() { return kChunkThreads * kVecs * Vec<T>::N; }

// Order-preserving keys (no NaN reaches them).
__device__ __forceinline__ uint32_t okey(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long okey(double d) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(d);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;                      // okey(-inf)
constexpr unsigned long long kKeyNegInf64 = 0x000FFFFFFFFFFFFFull;

struct ChunkStat {
  double sum;      // sum of exp(x - max) over the chunk
  float max;
  int count;       // candidates listed
};
struct Cand {
  float x;
  int token;
};

struct SelectParams {
  const void* logits;
  int64_t ld;
  const float* cum;
  const uint8_t* finished;
  const uint32_t* allowed;
  int64_t allowed_ld;
  int W, V, k, pad_token;
  int n_chunk, cap;
  ChunkStat* stat;     // [rows][n_chunk]
  Cand* cand;          // [rows][n_chunk][cap]
  int32_t *parent, *token;
  float* score;
};

__device__ __forceinline__ bool row_offers(const SelectParams& p, int64_t row) {
  const float c = p.cum[row];
  return isfinite(c) && !(p.finished && p.finished[row]);
}

// One 16-byte vector of tokens v .. v + N - 1 of a row, missing tokens as -inf, NaN as -inf.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int v, int V, float* x) {
  constexpr int N = Vec<T>::N;
  T t[N];
  const T* p = row + v;
  if (v + N <= V) {
    const unsigned a = (unsigned)(uintptr_t)row & 15u;   // the same for the whole row
    if (a == 0) {
      *reinterpret_cast<uint4*>(t) = __ldcs(reinterpret_cast<const uint4*>(p));
    } else if ((a & 3) == 0) {
      uint32_t* w = reinterpret_cast<uint32_t*>(t);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaxf(to_f32(t[i]), -INFINITY);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v + i < V ? fmaxf(to_f32(p[i]), -INFINITY) : -INFINITY;
  }
}

// exp(x - m) with -inf - -inf and inf - inf read as 0 (the limit of equal infinite logits).
__device__ __forceinline__ float exp_diff(float x, float m) { return x == m ? 1.f : __expf(x - m); }

template <typename T>
__global__ void __launch_bounds__(kChunkThreads) beam_chunk_kernel(const __grid_constant__ SelectParams p) {
  constexpr int N = Vec<T>::N;
  const int64_t row = blockIdx.x / p.n_chunk;
  const int chunk = (int)(blockIdx.x % p.n_chunk);
  if (!row_offers(p, row)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* lr = static_cast<const T*>(p.logits) + row * p.ld;
  const int v0 = chunk * chunk_elems<T>() + tid * N;
  constexpr int kStep = kChunkThreads * N;
  float x[kVecs][N];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) load_vec<T>(lr, v0 + i * kStep, p.V, x[i]);

  // the thread's maximum and sum, then the chunk's
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, x[i][e]);
  float s = 0.f;
  if (m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) s += exp_diff(x[i][e], m);
  }
  float gm = m;       // the maximum among the tokens that may be selected
  if (p.allowed) {
    const uint32_t* al = p.allowed + row * p.allowed_ld;
    gm = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = v0 + i * kStep;   // a multiple of N, which divides 32: one word
      const uint32_t bits = v < p.V ? __ldg(al + (v >> 5)) >> (v & 31) : 0u;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (!((bits >> e) & 1u)) x[i][e] = -INFINITY;
        gm = fmaxf(gm, x[i][e]);
      }
    }
  }
  __shared__ float sm_m[kChunkThreads / 32], sm_hi[kChunkThreads / 32];
  __shared__ double sm_s[kChunkThreads / 32];
  __shared__ int sm_count, sm_scan[kChunkThreads / 32];
  extern __shared__ Cand sm_cand[];                 // [cap]
  float wm = m, wh = gm;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    wh = fmaxf(wh, __shfl_xor_sync(0xffffffffu, wh, o));
  }
  double ws = m > -INFINITY ? (double)s * (double)exp_diff(m, wm) : 0.0;
#pragma unroll
  for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
  if (lane == 0) {
    sm_m[warp] = wm;
    sm_s[warp] = ws;
    sm_hi[warp] = wh;
  }
  if (tid == 0) sm_count = 0;
  __syncthreads();
  float bm = -INFINITY, hi_x = -INFINITY;
#pragma unroll
  for (int w = 0; w < kChunkThreads / 32; ++w) {
    bm = fmaxf(bm, sm_m[w]);
    hi_x = fmaxf(hi_x, sm_hi[w]);
  }
  ChunkStat* st = p.stat + row * p.n_chunk + chunk;
  if (tid == 0) {
    double tot = 0.0;
    for (int w = 0; w < kChunkThreads / 32; ++w)
      if (sm_m[w] > -INFINITY) tot += sm_s[w] * (double)exp_diff(sm_m[w], bm);
    st->max = bm;
    st->sum = tot;
  }
  // ---- the threshold: the largest found key that at least k thread maxima reach
  const uint32_t mykey = okey(gm);
  const int k = p.k;
  uint32_t lo = kKeyNegInf + 1, hi = okey(hi_x);
  const int valid = __syncthreads_count(mykey > kKeyNegInf);
  if (valid >= k) {
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int c = __syncthreads_count(mykey >= mid);
      if (c >= k) {
        lo = mid;
        if (c <= k + (k >> 3)) break;
      } else {
        hi = mid - 1;
      }
    }
  }
  // ---- list what reaches it
  Cand* out = p.cand + (row * p.n_chunk + chunk) * (int64_t)p.cap;
  if (mykey >= lo) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (okey(x[i][e]) >= lo) {
          const int at = atomicAdd(&sm_count, 1);
          if (at < p.cap) sm_cand[at] = Cand{x[i][e], v0 + i * kStep + e};
        }
  }
  __syncthreads();
  int count = sm_count;
  if (count > p.cap) {
    // too many: the exact k-th key, everything above it, and its ties in token order
    uint32_t a = lo, b = okey(hi_x);
    while (a < b) {
      const uint32_t mid = a + (b - a + 1) / 2;
      int c = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) c += okey(x[i][e]) >= mid;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) sm_scan[warp] = c;
      __syncthreads();
      int tot = 0;
      for (int w = 0; w < kChunkThreads / 32; ++w) tot += sm_scan[w];
      __syncthreads();
      if (tot >= k) a = mid; else b = mid - 1;
    }
    if (tid == 0) sm_count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (okey(x[i][e]) > a) sm_cand[atomicAdd(&sm_count, 1)] = Cand{x[i][e], v0 + i * kStep + e};   // fewer than k
    __syncthreads();
    int have = sm_count;
    for (int i = 0; i < kVecs && have < k; ++i) {      // `have` is the same in every thread
      int mine = 0;
#pragma unroll
      for (int q = 0; q < kVecs; ++q)
        if (q == i)
#pragma unroll
          for (int e = 0; e < N; ++e) mine += okey(x[q][e]) == a;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sm_scan[warp] = incl;
      __syncthreads();
      int at = have + incl - mine, tot = 0;
      for (int w = 0; w < kChunkThreads / 32; ++w) {
        if (w < warp) at += sm_scan[w];
        tot += sm_scan[w];
      }
#pragma unroll
      for (int q = 0; q < kVecs; ++q)
        if (q == i)
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (okey(x[q][e]) == a) {
              if (at < k) sm_cand[at] = Cand{x[q][e], v0 + i * kStep + e};
              ++at;
            }
      have += tot;
      __syncthreads();
    }
    count = min(have, k);
  }
  for (int i = tid; i < count; i += kChunkThreads) out[i] = sm_cand[i];
  if (tid == 0) st->count = count;
}

// A candidate's place: total first, then lower beam, higher logit, lower token.
struct Rank {
  unsigned long long key, tie;
};
__device__ __forceinline__ bool before(const Rank& a, const Rank& b) {
  return a.key > b.key || (a.key == b.key && a.tie > b.tie);
}
__device__ __forceinline__ unsigned long long tie_of(int beam, float x, int token) {
  return ((unsigned long long)(255 - beam) << 56) | ((unsigned long long)okey(x) << kTokenBits) |
         (unsigned long long)((1 << kTokenBits) - 1 - token);
}

__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const __grid_constant__ SelectParams p) {
  __shared__ float s_max[TR_MAX_BEAMS];
  __shared__ double s_logsum[TR_MAX_BEAMS];
  __shared__ int s_kind[TR_MAX_BEAMS];            // 0 dead, 1 offers tokens, 2 finished
  __shared__ unsigned long long s_hi;
  __shared__ int s_count;
  extern __shared__ Rank s_rank[];                // [kMergeCap]
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)r * p.W;
  for (int b = tid; b < p.W; b += kMergeThreads) {
    const int64_t row = row0 + b;
    int kind = 0;
    float M = -INFINITY;
    double S = 0.0;
    if (isfinite(p.cum[row])) {
      if (p.finished && p.finished[row]) {
        kind = 2;
      } else {
        const ChunkStat* st = p.stat + row * p.n_chunk;
        for (int c = 0; c < p.n_chunk; ++c) M = fmaxf(M, st[c].max);
        for (int c = 0; c < p.n_chunk; ++c)
          if (st[c].max > -INFINITY) S += st[c].sum * (st[c].max == M ? 1.0 : exp((double)st[c].max - (double)M));
        kind = M > -INFINITY ? 1 : 0;
      }
    }
    s_kind[b] = kind;
    s_max[b] = M;
    s_logsum[b] = kind == 1 ? log(S) : 0.0;
  }
  if (tid == 0) {
    s_hi = 0;
    s_count = 0;
  }
  __syncthreads();
  const int n_list = p.W * p.n_chunk;
  constexpr int kWarps = kMergeThreads / 32;
  // f(rank) for every candidate of this thread
  auto each = [&](auto f) {
    for (int l = warp; l < n_list; l += kWarps) {
      const int b = l / p.n_chunk;
      const int64_t row = row0 + b;
      if (s_kind[b] == 1) {
        const int cnt = p.stat[row0 * p.n_chunk + l].count;
        const Cand* c = p.cand + (row0 * p.n_chunk + l) * (int64_t)p.cap;
        const double cum = p.cum[row], ls = s_logsum[b];
        const float M = s_max[b];
        for (int i = lane; i < cnt; i += 32) {
          const Cand q = c[i];
          const double d = q.x == M ? 0.0 : (double)q.x - (double)M;
          if (d > -INFINITY) f(Rank{okey(cum + (d - ls)), tie_of(b, q.x, q.token)});
        }
      } else if (s_kind[b] == 2 && l % p.n_chunk == 0 && lane == 0) {
        f(Rank{okey((double)p.cum[row]), tie_of(b, 0.f, p.pad_token)});
      }
    }
  };
  unsigned long long mine = 0;
  each([&](const Rank& q) {
    if (q.key > mine) mine = q.key;
  });
  if (mine) atomicMax(&s_hi, mine);
  const int k = p.k;
  const int valid = __syncthreads_count(mine != 0);
  unsigned long long lo = kKeyNegInf64 + 1, hi = s_hi;
  if (valid >= k)
    while (lo < hi) {
      const unsigned long long mid = lo + (hi - lo + 1) / 2;
      const int c = __syncthreads_count(mine >= mid);
      if (c >= k) {
        lo = mid;
        if (c <= k + (k >> 3)) break;
      } else {
        hi = mid - 1;
      }
    }
  each([&](const Rank& q) {
    if (q.key >= lo) {
      const int at = atomicAdd(&s_count, 1);
      if (at < kMergeCap) s_rank[at] = q;
    }
  });
  __syncthreads();
  int count = s_count;
  if (count > kMergeCap) {
    // too many: the exact k-th candidate, by its total and then by its tie
    auto count_if = [&](auto pred) {
      int c = 0;
      each([&](const Rank& q) { c += pred(q); });
      __syncthreads();
      if (tid == 0) s_count = 0;
      __syncthreads();
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c) atomicAdd(&s_count, c);
      __syncthreads();
      return s_count;
    };
    unsigned long long a = lo, b = s_hi;
    while (a < b) {
      const unsigned long long mid = a + (b - a + 1) / 2;
      if (count_if([&](const Rank& q) { return q.key >= mid; }) >= k) a = mid; else b = mid - 1;
    }
    unsigned long long ta = 0, tb = ~0ull;
    while (ta < tb) {
      const unsigned long long mid = ta + (tb - ta) / 2 + 1;
      if (count_if([&](const Rank& q) { return q.key > a || (q.key == a && q.tie >= mid); }) >= k) ta = mid; else tb = mid - 1;
    }
    __syncthreads();
    if (tid == 0) s_count = 0;
    __syncthreads();
    each([&](const Rank& q) {
      if (q.key > a || (q.key == a && q.tie >= ta)) s_rank[atomicAdd(&s_count, 1)] = q;   // exactly k (ties differ)
    });
    __syncthreads();
    count = s_count;
  }
  int n = 1;
  while (n < count) n <<= 1;
  for (int i = count + tid; i < n; i += kMergeThreads) s_rank[i] = Rank{0ull, 0ull};
  __syncthreads();
  for (int size = 2; size <= n; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = tid; i < n; i += kMergeThreads) {
        const int j = i ^ stride;
        if (j > i) {
          const Rank a = s_rank[i], b = s_rank[j];
          if ((i & size) == 0 ? before(b, a) : before(a, b)) {
            s_rank[i] = b;
            s_rank[j] = a;
          }
        }
      }
      __syncthreads();
    }
  for (int j = tid; j < k; j += kMergeThreads) {
    int par = -1, tok = -1;
    float sc = -INFINITY;
    if (j < count) {
      const Rank q = s_rank[j];
      par = 255 - (int)(q.tie >> 56);
      tok = (1 << kTokenBits) - 1 - (int)(q.tie & ((1u << kTokenBits) - 1));
      const unsigned long long u = q.key;
      sc = (float)__longlong_as_double((long long)((u >> 63) ? (u & 0x7FFFFFFFFFFFFFFFull) : ~u));
    }
    p.parent[(int64_t)r * k + j] = par;
    p.token[(int64_t)r * k + j] = tok;
    p.score[(int64_t)r * k + j] = sc;
  }
}

// ---------------------------------------------------------------- reorder
// One CTA moves one column slice of one state of one request: every surviving row's slice is
// loaded into registers before the first is stored, and no other CTA touches the slice, so the
// move is safe in place whatever the parents are.  Traffic: each row read once (children of one
// parent read it again from L2) and written once.
constexpr int kMoveThreads = 256;

struct MoveState {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_stride, dst_stride;
  int64_t units;          // of sizeof(U) bytes per row
  int64_t first_block;    // of this state in the grid
  int cols;               // units per slice, a power of two
  int n_slice;
};
struct MoveParams {
  MoveState s[TR_MAX_STATES];
  int n_states, R, W_in, W_out;
  const int32_t* parent;
  int* status;
};

template <typename U, int kUnits>
__global__ void __launch_bounds__(kMoveThreads) beam_move_kernel(const __grid_constant__ MoveParams p) {
  int si = 0;
  while (si + 1 < p.n_states && (int64_t)blockIdx.x >= p.s[si + 1].first_block) ++si;
  const MoveState& s = p.s[si];
  const int64_t local = (int64_t)blockIdx.x - s.first_block;
  const int r = (int)(local / s.n_slice);
  const int64_t c0 = (local % s.n_slice) * (int64_t)s.cols;
  const int col = threadIdx.x & (s.cols - 1);
  const int rows_per = kMoveThreads / s.cols;             // rows per step
  const int row_t = threadIdx.x / s.cols;
  const bool in = c0 + col < s.units;
  const uint8_t* src = s.src + (int64_t)r * p.W_in * s.src_stride + (c0 + col) * (int64_t)sizeof(U);
  uint8_t* dst = s.dst + (int64_t)r * p.W_out * s.dst_stride + (c0 + col) * (int64_t)sizeof(U);
  const int32_t* par = p.parent + (int64_t)r * p.W_out;
  U val[kUnits];
  bool have[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int i = u * rows_per + row_t;
    have[u] = false;
    if (i < p.W_out) {
      const int q = __ldg(par + i);
      if (q >= p.W_in) {
        if (col == 0) atomicOr(p.status, STATUS_KEY_RANGE);
      } else if (q >= 0 && in && !(s.src == s.dst && q == i)) {
        have[u] = true;
        val[u] = *reinterpret_cast<const U*>(src + q * s.src_stride);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int i = u * rows_per + row_t;
    if (have[u]) *reinterpret_cast<U*>(dst + i * s.dst_stride) = val[u];
  }
}

constexpr int kMoveUnits = 8;

template <typename U>
tr_status launch_move(MoveParams& p, cudaStream_t st) {
  int64_t blocks = 0;
  // the widest slice whose W_out rows fit the CTA's registers
  int cols = 1;
  while (cols * 2 <= kMoveThreads && (int64_t)cols * 2 * p.W_out <= (int64_t)kMoveThreads * kMoveUnits) cols *= 2;
  for (int i = 0; i < p.n_states; ++i) {
    MoveState& s = p.s[i];
    s.units /= (int64_t)sizeof(U);
    s.cols = cols;
    const int64_t slices = (s.units + cols - 1) / cols;
    if (slices > INT32_MAX) return fail(TR_ERR_UNSUPPORTED, "state %d: row too long", i);
    s.n_slice = (int)slices;
    s.first_block = blocks;
    blocks += slices * p.R;
  }
  if (blocks > INT32_MAX) return fail(TR_ERR_UNSUPPORTED, "states too large for one call");
  if (blocks == 0) return TR_OK;
  beam_move_kernel<U, kMoveUnits><<<(unsigned)blocks, kMoveThreads, 0, st>>>(p);
  TR_LAUNCH_CHECK("beam_move_kernel");
  return TR_OK;
}

struct Rows {
  const void* base;
  int64_t stride, bytes, n;
};
// Whether two sets of rows share a byte (rows interleaved at one stride do not).
bool overlap(const Rows& a, const Rows& b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.base, b0 = (uintptr_t)b.base;
  if (a0 >= b0 + (b.n - 1) * b.stride + b.bytes || b0 >= a0 + (a.n - 1) * a.stride + a.bytes) return false;
  if (a.stride != b.stride) return true;
  const int64_t d = (int64_t)(a0 > b0 ? (a0 - b0) % a.stride : (a.stride - (b0 - a0) % a.stride) % a.stride);   // a after b
  return !(d >= b.bytes && a.stride - d >= a.bytes);
}

struct SelectPlan {
  int n_chunk, cap;
  size_t stat_bytes, total;
};
SelectPlan plan_select(int64_t rows, int V, int k, bool f32) {
  SelectPlan s;
  const int elems = f32 ? chunk_elems<float>() : chunk_elems<__nv_bfloat16>();
  s.n_chunk = (V + elems - 1) / elems;
  s.cap = std::min(std::max(256, 4 * k), elems);
  s.stat_bytes = ((size_t)rows * s.n_chunk * sizeof(ChunkStat) + 255) / 256 * 256;
  s.total = s.stat_bytes + (size_t)rows * s.n_chunk * s.cap * sizeof(Cand);
  return s;
}

tr_status check_select(int R, int W, int V, int k) {
  if (W < 1 || W > TR_MAX_BEAMS) return fail(TR_ERR_INVALID_ARG, "W=%d (need 1..%d)", W, TR_MAX_BEAMS);
  if (R < 1 || (int64_t)R * W >= (1 << 20)) return fail(TR_ERR_INVALID_ARG, "R=%d (need R >= 1 and R*W < 2^20)", R);
  if (V < 1 || V > (1 << kTokenBits)) return fail(TR_ERR_INVALID_ARG, "V=%d (need 1..2^24)", V);
  if (k < 1 || k > TR_MAX_BEAM_K) return fail(TR_ERR_INVALID_ARG, "k=%d (need 1..%d)", k, TR_MAX_BEAM_K);
  return TR_OK;
}

}  // namespace
}  // namespace tr

using namespace tr;

extern "C" size_t tr_beam_select_workspace(int R, int W, int V, int k) {
  if (check_select(R, W, V, k) != TR_OK) return SIZE_MAX;
  const int64_t rows = (int64_t)R * W;
  return std::max(plan_select(rows, V, k, true).total, plan_select(rows, V, k, false).total);
}

extern "C" tr_status tr_beam_select(const void* logits, tr_dtype logits_dtype, int64_t ld, const float* cum,
                                    const uint8_t* finished, const uint32_t* allowed, int64_t allowed_ld, int R, int W,
                                    int V, int k, int pad_token, int32_t* parent, int32_t* token, float* score,
                                    void* workspace, size_t workspace_bytes, tr_stream stream) {
  TR_TRY(check_select(R, W, V, k));
  if (logits_dtype != TR_F32 && logits_dtype != TR_BF16)
    return fail(TR_ERR_INVALID_ARG, "logits_dtype=%d", (int)logits_dtype);
  const size_t esize = logits_dtype == TR_F32 ? 4 : 2;
  if (ld < V) return fail(TR_ERR_INVALID_ARG, "ld=%lld is less than V=%d", (long long)ld, V);
  if (allowed && allowed_ld < (V + 31) / 32)
    return fail(TR_ERR_INVALID_ARG, "allowed_ld=%lld: need ceil(V/32)", (long long)allowed_ld);
  if (pad_token < 0 || pad_token >= (1 << kTokenBits)) return fail(TR_ERR_INVALID_ARG, "pad_token=%d", pad_token);
  if (!logits || !cum || !parent || !token || !score) return fail(TR_ERR_INVALID_ARG, "null device pointer");
  if ((uintptr_t)logits % esize || (uintptr_t)cum % 4 || (uintptr_t)allowed % 4 || (uintptr_t)parent % 4 ||
      (uintptr_t)token % 4 || (uintptr_t)score % 4)
    return fail(TR_ERR_INVALID_ARG, "a pointer is not aligned to its type");
  const int64_t rows = (int64_t)R * W;
  const SelectPlan sp = plan_select(rows, V, k, logits_dtype == TR_F32);
  if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < sp.total)
    return fail(TR_ERR_INVALID_ARG, "workspace: need %zu bytes, 16-byte aligned", sp.total);
  if (rows * sp.n_chunk > INT32_MAX) return fail(TR_ERR_UNSUPPORTED, "R*W*V is too large for one call");
  const cudaStream_t st = (cudaStream_t)stream;
  SelectParams p{};
  p.logits = logits;
  p.ld = ld;
  p.cum = cum;
  p.finished = finished;
  p.allowed = allowed;
  p.allowed_ld = allowed_ld;
  p.W = W;
  p.V = V;
  p.k = k;
  p.pad_token = pad_token;
  p.n_chunk = sp.n_chunk;
  p.cap = sp.cap;
  p.stat = static_cast<ChunkStat*>(workspace);
  p.cand = reinterpret_cast<Cand*>(static_cast<uint8_t*>(workspace) + sp.stat_bytes);
  p.parent = parent;
  p.token = token;
  p.score = score;
  const unsigned grid = (unsigned)(rows * sp.n_chunk);
  const size_t smem = (size_t)sp.cap * sizeof(Cand);
  if (logits_dtype == TR_F32)
    beam_chunk_kernel<float><<<grid, kChunkThreads, smem, st>>>(p);
  else
    beam_chunk_kernel<__nv_bfloat16><<<grid, kChunkThreads, smem, st>>>(p);
  TR_LAUNCH_CHECK("beam_chunk_kernel");
  beam_merge_kernel<<<R, kMergeThreads, kMergeCap * sizeof(Rank), st>>>(p);
  TR_LAUNCH_CHECK("beam_merge_kernel");
  return TR_OK;
}

extern "C" tr_status tr_beam_reorder(const tr_beam_state* states, int n_states, const int32_t* parent, int R, int W_in,
                                     int W_out, tr_stream stream) {
  if (n_states < 0 || n_states > TR_MAX_STATES)
    return fail(TR_ERR_INVALID_ARG, "n_states=%d (need 0..%d)", n_states, TR_MAX_STATES);
  if (W_in < 1 || W_in > TR_MAX_BEAMS || W_out < 1 || W_out > TR_MAX_BEAMS)
    return fail(TR_ERR_INVALID_ARG, "W_in=%d, W_out=%d (need 1..%d)", W_in, W_out, TR_MAX_BEAMS);
  if (R < 1 || (int64_t)R * std::max(W_in, W_out) >= (1 << 20))
    return fail(TR_ERR_INVALID_ARG, "R=%d (need R >= 1 and R*W < 2^20)", R);
  if (n_states == 0) return TR_OK;
  if (!states || !parent) return fail(TR_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)parent % 4) return fail(TR_ERR_INVALID_ARG, "parent is not aligned to its type");
  MoveParams p{};
  uintptr_t align = 0;
  for (int i = 0; i < n_states; ++i) {
    const tr_beam_state& s = states[i];
    if (s.row_bytes < 0 || (s.row_bytes > 0 && (!s.dst || !s.src)))
      return fail(TR_ERR_INVALID_ARG, "state %d: row_bytes=%lld or null pointer", i, (long long)s.row_bytes);
    if (s.dst_stride < s.row_bytes || s.src_stride < s.row_bytes || std::max(s.dst_stride, s.src_stride) > (1ll << 40))
      return fail(TR_ERR_INVALID_ARG, "state %d: stride below row_bytes or too large", i);
    if (s.dst == s.src && (W_in != W_out || s.dst_stride != s.src_stride))
      return fail(TR_ERR_INVALID_ARG, "state %d: in place needs W_in == W_out and equal strides", i);
    for (int j = 0; j < i + 1 && s.row_bytes > 0; ++j) {
      const tr_beam_state& o = states[j];
      const Rows sd{s.dst, s.dst_stride, s.row_bytes, (int64_t)R * W_out}, ss{s.src, s.src_stride, s.row_bytes, (int64_t)R * W_in};
      const Rows od{o.dst, o.dst_stride, o.row_bytes, (int64_t)R * W_out}, os{o.src, o.src_stride, o.row_bytes, (int64_t)R * W_in};
      const bool bad = i == j ? s.dst != s.src && overlap(sd, ss) : overlap(sd, os) || overlap(sd, od) || overlap(ss, od);
      if (bad) return fail(TR_ERR_INVALID_ARG, "states %d and %d: dst overlaps rows of another state, or its own src", j, i);
    }
    align |= (uintptr_t)s.dst | (uintptr_t)s.src | (uintptr_t)s.dst_stride | (uintptr_t)s.src_stride | (uintptr_t)s.row_bytes;
    p.s[i].src = static_cast<const uint8_t*>(s.src);
    p.s[i].dst = static_cast<uint8_t*>(s.dst);
    p.s[i].src_stride = s.src_stride;
    p.s[i].dst_stride = s.dst_stride;
    p.s[i].units = s.row_bytes;
  }
  DeviceState* ds = nullptr;
  TR_TRY(device_state(&ds));
  p.n_states = n_states;
  p.R = R;
  p.W_in = W_in;
  p.W_out = W_out;
  p.parent = parent;
  p.status = ds->status;
  const cudaStream_t st = (cudaStream_t)stream;
  if (align % 16 == 0) return launch_move<uint4>(p, st);
  if (align % 4 == 0) return launch_move<uint32_t>(p, st);
  return launch_move<uint8_t>(p, st);
}

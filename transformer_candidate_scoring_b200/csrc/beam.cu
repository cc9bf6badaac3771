// Beam decoding: selection over beams and vocabulary, and the reordering of beam states.
//
// Selection.  total(b, v) = cum[b] + x[b][v] - log sum_u exp(x[b][u]); the k best (b, v) of each
// request.  The logits are the traffic (2 or 4 bytes per (b, v), read once); the results are a
// few KB.  Two launches:
//   beam_sum_kernel   one warp per tile of 32 lanes x 8 16-byte vectors of a row, held in
//     registers: the tile's maximum and sum of exponentials, and each lane's best logit (of its
//     "group" of 64 bf16 or 32 fp32 tokens) -- nothing else, no shared memory and no barrier, so
//     that the loads of the next warps are always in flight.
//   beam_pick_kernel  one CTA per request: the rows' log-sum-exp (in 64 bits: two beams' totals
//     are compared across rows), the tiles' best totals, a bound that at least k tiles reach (or
//     groups, of few tiles; the k-th largest of the threads' own best, bisected by one warp), and
//     then only the tiles, groups and logits that reach it -- about k of each -- are looked at,
//     the tokens among them cut down the same way and ranked.
// 64 x 16 rows of 131072 bf16: the sums 48 us (5.6 TB/s, the exponentials' unit 70 % busy), the choice 13 us,
// a chain of some ten barriers that few threads have work between.  Lists of the best per chunk of a row
// took 87 us for the first part, rings filled by cp.async under a persistent grid 108.
// When more tokens reach the bound than the sort holds (long runs of equal logits: beams that have nothing to tell
// their tokens apart, rows filled with a mask's value), the exact k-th candidate is found by bisection over
// the tokens themselves: over the range of their totals, then, among equal ones, in the beam that it falls into.
// 32 beams of 8192 (131072) equal logits: 0.6 ms (9.5), where bisections over all values of a total and of a tie
// took 13.6 (214).
//
// Which lane sums which token depends on the token alone, not on the row's address, so equal
// rows get equal sums and ties between their beams stay ties.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "model.cuh"

namespace tr {
namespace {

constexpr int kSumThreads = 256;
constexpr int kVecs = 8;                 // 16-byte vectors per lane
constexpr int kPickThreads = 1024;
constexpr int kPickTiles = 1024, kPickGroups = 1023;   // tiles and groups noted for a closer look
constexpr int kPickCap = 1536;           // candidates the final sort takes
constexpr int kTokenBits = 24;

template <typename T> constexpr int tile_elems() { return 32 * kVecs * (16 / (int)sizeof(T)); }

// Order-preserving keys (no NaN reaches them; -0 equals 0).
__device__ __forceinline__ uint32_t okey(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long okey(double d) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(d + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;                      // okey(-inf)
__device__ __forceinline__ double of_key(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

struct __align__(16) TileSum {
  float max;
  float sum;       // of exponentials, relative to the maximum (see sum_ref)
  float best;      // the largest logit that may be selected
  float pad;
};

struct SelectParams {
  const void* logits;
  int64_t ld;
  const float* cum;
  const uint8_t* finished;
  const uint32_t* allowed;
  int64_t allowed_ld;
  int W, V, k, pad_token;
  int n_tile;
  bool aligned;        // every row at a 16-byte aligned address
  TileSum* sums;       // [rows][n_tile]
  float* best;         // [rows][n_tile][32]: the groups' largest logits that may be selected
  int32_t *parent, *token;
  float* score;
};

__device__ __forceinline__ bool row_offers(const SelectParams& p, int64_t row) {
  const float c = p.cum[row];
  return isfinite(c) && !(p.finished && p.finished[row]);
}

// Sums of exponentials are held as sum_i 2^(x_i log2 e - ref), ref the rounded log2 of the
// largest term m: subtracting a whole number costs the exponent one rounding of its own size,
// where a subtraction of m log2 e would shift all terms alike by its rounding and so move one
// beam's total against another's.  log2 e is used as hi + lo, hi its fp32 value.  Terms are formed with hi;
// with M the row's maximum, x_i lo = M lo + (x_i - M) lo, and
//     log sum_i exp(x_i) = M + ln 2 (ref - M hi + log2 sum_i 2^(x_i hi - ref) 2^((x_i - M) lo))
// where M hi is exact in 64 bits, whatever M's size.  The last factor is applied as sums are joined, for the maximum m
// of each partial sum in x_i's place (m - M is below 200 in size wherever a sum counts, so 1 + (m - M) lo ln 2 is it to
// 2^-37); what is left, (x_i - m) lo, is below 2^-22 for every term that counts.  Logits beyond 1e9 in size
// are further apart than any exponential reaches: there the sum counts the largest logit's copies (infinite ones
// too).
constexpr float kHuge = 1e9f;
constexpr float kL2eHi = 1.4426950408889634f;                 // rounds to 1.44269502...
constexpr float kL2eLo = (float)(1.4426950408889634 - (double)kL2eHi);
__device__ __forceinline__ bool huge(float m) { return fabsf(m) > kHuge; }
__device__ __forceinline__ float sum_ref(float m) { return rintf(m * kL2eHi); }
// The factor that takes a sum of largest term `m` to one of largest term `to` (to >= m): a power of two and
// the low part of log2 e; terms below 2^-126 of the largest are dropped.
__device__ __forceinline__ float sum_scale(float m, float to) {
  if (m == to) return 1.f;
  if (m == -INFINITY || huge(m) || huge(to)) return 0.f;
  const float n = sum_ref(m) - sum_ref(to);
  return n < -126.f ? 0.f : fmaf(m - to, kL2eLo * 0.693147f, 1.f) * __int_as_float((127 + (int)n) << 23);
}
__device__ __forceinline__ double log_sum(float m, double sum) {   // log sum_i exp(x_i), less m
  return huge(m) ? log(sum) : 0.6931471805599453 * (((double)sum_ref(m) - (double)m * (double)kL2eHi) + log2(sum));
}

__device__ __forceinline__ uint64_t pack2f(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split2f(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The registers of a 16-byte vector of logits: four words of two bf16 or of one fp32.  NaN reads
// as -inf, and so does what lies past the row.
template <typename T> struct Pack;
template <> struct Pack<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;      // (-inf, -inf)
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {      // elementwise, NaN loses
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float top(uint32_t w) { return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
  static __device__ __forceinline__ float at(uint32_t w, int e) { return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16); }
  // of the pair in w: elements whose bit is clear become -inf
  static __device__ __forceinline__ uint32_t mask(uint32_t w, uint32_t bits) {
    const uint32_t lo = bits & 1u ? w & 0xFFFFu : 0xFF80u, hi = bits & 2u ? w & 0xFFFF0000u : 0xFF800000u;
    return lo | hi;
  }
};
template <> struct Pack<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ float top(uint32_t w) { return __uint_as_float(w); }
  static __device__ __forceinline__ float at(uint32_t w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t mask(uint32_t w, uint32_t bits) { return bits & 1u ? w : kNone; }
};

// A vector that the row ends in, or of a row at an odd address.
template <typename T>
__device__ __noinline__ uint4 load_partial(const T* p, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = i < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : Pack<T>::kNone;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p) + 2 * i;
      w[i] = 2 * i < n ? (uint32_t)__ldg(h) : 0xFF80u;
      w[i] |= 2 * i + 1 < n ? (uint32_t)__ldg(h + 1) << 16 : 0xFF800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Tokens v .. of a row, missing ones as -inf.  kAlign: the row's alignment in bytes, 16, 4 or 2.
template <typename T, int kAlign>
__device__ __forceinline__ uint4 load_vec(const T* row, int v, int V) {
  const T* p = row + v;
  if (v + Pack<T>::N <= V) {
    if constexpr (kAlign == 16) {
      return __ldg(reinterpret_cast<const uint4*>(p));
    } else if constexpr (kAlign == 4) {
      const uint32_t* h = reinterpret_cast<const uint32_t*>(p);
      return make_uint4(__ldg(h), __ldg(h + 1), __ldg(h + 2), __ldg(h + 3));
    }
  }
  if (v < V) return load_partial<T>(p, V - v);
  return make_uint4(Pack<T>::kNone, Pack<T>::kNone, Pack<T>::kNone, Pack<T>::kNone);
}
// The mask bits of tokens v .. (v a multiple of 4 or 8, which divide 32: one word).
__device__ __forceinline__ uint32_t allowed_bits(const SelectParams& p, int64_t row, int v) {
  return v < p.V ? __ldg(p.allowed + row * p.allowed_ld + (v >> 5)) >> (v & 31) : 0u;
}

template <typename T, int kAlign>
__global__ void __launch_bounds__(kSumThreads, 4) beam_sum_kernel(const __grid_constant__ SelectParams p) {
  using P = Pack<T>;
  constexpr int N = P::N, PER = N / 4;                  // elements per vector, per word
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, tile = blockIdx.y * (kSumThreads / 32) + (threadIdx.x >> 5);
  if (tile >= p.n_tile || !row_offers(p, row)) return;
  const T* lr = static_cast<const T*>(p.logits) + row * p.ld;
  const int v0 = tile * tile_elems<T>() + lane * N;
  uint32_t x[kVecs][4];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint4 q = load_vec<T, kAlign>(lr, v0 + i * 32 * N, p.V);
    x[i][0] = q.x; x[i][1] = q.y; x[i][2] = q.z; x[i][3] = q.w;
  }
  uint32_t bits[kVecs];
  if (p.allowed) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) bits[i] = allowed_bits(p, row, v0 + i * 32 * N);
  }
  uint32_t top = P::kNone;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = P::max(top, x[i][e]);
  const float m = P::top(top);
  float s = 0.f;
  const float ref = -sum_ref(m);
  if (!huge(m)) {
    const uint64_t ref2 = pack2f(ref, ref), hi2 = pack2f(kL2eHi, kL2eHi);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2 / PER) {
        const uint64_t a = PER == 2 ? pack2f(P::at(x[i][e], 0), P::at(x[i][e], 1))
                                    : pack2f(__uint_as_float(x[i][e]), __uint_as_float(x[i][(e + 1) & 3]));
        float t0, t1;
        split2f(fma2(a, hi2, ref2), t0, t1);
        sum[i & 1] = add2(sum[i & 1], pack2f(ex2(t0), ex2(t1)));
      }
    float t0, t1;
    split2f(add2(sum[0], sum[1]), t0, t1);
    s = t0 + t1;
    if (s != s) {                                       // a NaN logit: leave it out
      s = 0.f;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float y = P::at(x[i][e / PER], e);
          if (y == y) s += ex2(fmaf(y, kL2eHi, ref));
        }
    }
  } else if (m > -INFINITY) {                           // (of all -inf the sum is unused)
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) s += P::at(x[i][e / PER], e) == m ? 1.f : 0.f;
  }
  if (p.allowed) {
    top = P::kNone;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = P::max(top, P::mask(x[i][e], bits[i] >> (e * PER)));
  }
  const float wm = of_key(__reduce_max_sync(0xffffffffu, okey(m)));
  float ws = s * sum_scale(m, wm);
#pragma unroll
  for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
  const int64_t at = row * p.n_tile + tile;
  const float gm = P::top(top);
  const float wg = p.allowed ? of_key(__reduce_max_sync(0xffffffffu, okey(gm))) : wm;
  p.best[at * 32 + lane] = gm;
  if (lane == 0) *reinterpret_cast<float4*>(p.sums + at) = make_float4(wm, ws, wg, 0.f);
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

// One warp, n keys per lane: a key, at least `floor`, that at least `want` of them reach (that many
// are known to reach `floor`), and not many more than that.  A step tries two keys, whose counts
// share one reduction.
template <int n>
__device__ __forceinline__ uint32_t bisect_by(const uint32_t* keys, int want, uint32_t floor) {
  static_assert(n * 32 < 1 << 16, "counts");
  uint32_t key[n], a = ~0u, b = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    key[i] = keys[i * 32 + (threadIdx.x & 31)];
    a = min(a, max(key[i], floor));
    b = max(b, key[i]);
  }
  a = __reduce_min_sync(0xffffffffu, a);
  b = max(a, __reduce_max_sync(0xffffffffu, b));
  while (a < b) {
    const uint32_t q = (b - a + 2) / 3, m1 = min(a + q, b), m2 = min(m1 + q, b);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < n; ++i) c += (key[i] >= m1 ? 1u : 0u) + (key[i] >= m2 ? 1u << 16 : 0u);
    c = __reduce_add_sync(0xffffffffu, c);
    const int c1 = c & 0xFFFF, c2 = c >> 16;
    int got = 0;
    if (c2 >= want) {
      a = m2;
      got = c2;
    } else if (c1 >= want) {
      a = m1;
      b = m2 - 1;
      got = c1;
    } else {
      b = m1 - 1;
    }
    if (got && got <= want + (want >> 3) + 8) break;
  }
  return a;
}
// Over the first `count` of at most 1024 keys (those behind them, up to the next power of two, are 0).
__device__ __noinline__ uint32_t bisect(const uint32_t* keys, int count, int want, uint32_t floor) {
  return count <= 128 ? bisect_by<4>(keys, want, floor) : count <= 512 ? bisect_by<16>(keys, want, floor) : bisect_by<32>(keys, want, floor);
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ SelectParams p) {
  using P = Pack<T>;
  constexpr int N = P::N, kWarps = kPickThreads / 32;
  __shared__ float s_max[TR_MAX_BEAMS], s_off[TR_MAX_BEAMS];
  __shared__ double s_lse[TR_MAX_BEAMS], s_cum[TR_MAX_BEAMS];
  __shared__ uint8_t s_kind[TR_MAX_BEAMS];        // 0 dead, 1 offers tokens, 2 finished
  __shared__ uint32_t s_key[kPickCap], s_best[kPickThreads], s_cut;
  __shared__ __align__(16) uint32_t s_sel_key[kPickCap];
  __shared__ float s_up[kPickGroups];
  __shared__ unsigned long long s_range[2];
  __shared__ int s_count, s_tiles, s_groups, s_tile[kPickTiles], s_group[kPickGroups];
  extern __shared__ Rank s_rank[];                // [kPickCap]
  int* s_sel = reinterpret_cast<int*>(s_rank + kPickCap);
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.k;
  const int64_t row0 = (int64_t)r * p.W;
  const TileSum* sums = p.sums + row0 * p.n_tile;
  cudaGridDependencySynchronize();
  // ---- a warp per beam: the row's maximum and sum, then a thread per beam: its log-sum-exp, less the maximum
  for (int b = warp; b < p.W; b += kWarps) {
    constexpr int kHeld = 4;                            // tiles per lane held between the two steps
    float4 y[kHeld];                                    // (unwritten where the row offers nothing)
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      y[i] = lane + 32 * i < p.n_tile ? __ldcg(reinterpret_cast<const float4*>(sums + b * p.n_tile + lane + 32 * i))
                                      : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    const float cum = p.cum[row0 + b];
    int kind = isfinite(cum) ? p.finished && p.finished[row0 + b] ? 2 : 1 : 0;
    float M = -INFINITY;
    double S = 0.0;
    if (kind == 1) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) M = fmaxf(M, y[i].x);
      for (int c = lane + 32 * kHeld; c < p.n_tile; c += 32) M = fmaxf(M, __ldcg(&sums[b * p.n_tile + c].max));
      M = of_key(__reduce_max_sync(0xffffffffu, okey(M)));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) S += (double)(y[i].y * sum_scale(y[i].x, M));
      for (int c = lane + 32 * kHeld; c < p.n_tile; c += 32) {
        const float4 z = __ldcg(reinterpret_cast<const float4*>(sums + b * p.n_tile + c));
        S += (double)(z.y * sum_scale(z.x, M));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
      if (M == -INFINITY) kind = 0;
    }
    if (lane == 0) {
      s_kind[b] = (uint8_t)kind;
      s_max[b] = M;
      s_cum[b] = (double)cum;
      s_lse[b] = S;
    }
  }
  if (tid == 0) s_count = s_tiles = s_groups = 0;
  __syncthreads();
  if (tid < p.W) {
    const float M = s_max[tid];
    const double lse = s_kind[tid] != 1 ? 0.0 : log_sum(M, s_lse[tid]);
    s_lse[tid] = lse;
    s_off[tid] = (float)(s_cum[tid] - lse);
  }
  __syncthreads();
  // ---- totals.  Exactly, as a 64-bit key (0: not a candidate):
  auto key_of = [&](int b, float x) -> unsigned long long {
    const float M = s_max[b];
    const double d = x == M ? 0.0 : (double)x - (double)M;
    const double t = s_cum[b] + (d - s_lse[b]);
    return t > -INFINITY ? okey(t) : 0ull;
  };
  // In fp32, t, off by at most e: a difference and a sum of two terms, each of which was rounded
  // once, so 2^-22 of their sizes covers them.  A difference or a sum below fp32's range counts as its lowest
  // value: t + e is still no less than the total, and t - e is -inf.
  struct Near { float t, e; };
  auto near_of = [&](int b, float x) -> Near {
    const float M = s_max[b], off = s_off[b], d = x == M ? 0.f : fmaxf(x - M, -FLT_MAX);
    return Near{fmaxf(d + off, -FLT_MAX), 0x1p-22f * (fabsf(d) + fabsf(off))};
  };
  const int per_row = p.n_tile * 32, n_tile = p.W * p.n_tile, n_group = p.W * per_row;
  const float* best = p.best + row0 * per_row;
  // f(beam, tile of the row, t, e) for this thread's tiles; a finished beam counts as its first
  auto each_tile = [&](auto f) {
#pragma unroll 2
    for (int j = tid; j < n_tile; j += kPickThreads) {
      const int b = j / p.n_tile, kind = s_kind[b];
      if (kind == 1) {
        const float x = __ldcg(&sums[j].best);
        if (x > -INFINITY) {
          const Near y = near_of(b, x);
          f(b, j - b * p.n_tile, y.t, y.e);
        }
      } else if (kind == 2 && j % p.n_tile == 0) {
        f(b, 0, s_off[b], 0.f);
      }
    }
  };
  // f(beam, group of the row, t, e) for this thread's groups, four neighbours at a time
  auto each_group = [&](auto f) {
    for (int j = tid * 4; j < n_group; j += kPickThreads * 4) {
      const int b = j / per_row, kind = s_kind[b];
      if (kind == 1) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(best + j));
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (y[e] > -INFINITY) {
            const Near u = near_of(b, y[e]);
            f(b, j - b * per_row + e, u.t, u.e);
          }
      } else if (kind == 2 && j % per_row == 0) {
        f(b, 0, s_off[b], 0.f);
      }
    }
  };
  // A bound that at least k totals reach, from the threads' best (lower ends of) totals; false when
  // fewer than k threads have one.
  uint32_t lo = kKeyNegInf + 1;
  float upper;
  auto bound_of = [&](auto&& each, int keys) {         // keys: threads that may have one, from the first on
    float mine = -INFINITY;
    upper = -INFINITY;
    each([&](int, int, float t, float e) {
      mine = fmaxf(mine, t - e);
      upper = fmaxf(upper, t + e);
    });
    s_key[tid] = okey(mine);
    if (__syncthreads_count(mine > -INFINITY) < k) return false;
    if (warp == 0) {
      const uint32_t cut = bisect(s_key, keys, k, lo);
      if (lane == 0) s_cut = cut;
    }
    __syncthreads();
    lo = s_cut;
    return true;
  };
  float bound = of_key(lo);
  // ---- the groups that may hold a token that reaches it, by way of the tiles
  auto note = [&](int b, int i, float t, float e) {
    if (t + e >= bound) {
      const int at = atomicAdd(&s_groups, 1);
      if (at < kPickGroups) {
        s_group[at] = b << 19 | i;
        s_key[at] = okey(t - e);
        s_up[at] = t + e;
      }
    }
  };
  bool by_tile = bound_of(each_tile, n_tile);
  if (by_tile) {
    bound = of_key(lo);
    if (upper >= bound)
      each_tile([&](int b, int i, float t, float e) {
        if (t + e >= bound) {
          const int at = atomicAdd(&s_tiles, 1);
          if (at < kPickTiles) s_tile[at] = b << 14 | i;
        }
      });
    __syncthreads();
    by_tile = s_tiles <= kPickTiles;
  }
  if (by_tile) {
    constexpr int kAhead = 4;
    for (int i0 = warp; i0 < s_tiles; i0 += kWarps * kAhead) {
      float x[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * kWarps, w = i < s_tiles ? s_tile[i] : 0, b = w >> 14;
        x[q] = i < s_tiles && s_kind[b] == 1 ? __ldcg(best + b * per_row + (w & 16383) * 32 + lane) : -INFINITY;
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * kWarps;
        if (i >= s_tiles) break;
        const int w = s_tile[i], b = w >> 14;
        if (s_kind[b] == 2) {
          if (lane == 0) note(b, 0, s_off[b], 0.f);
        } else if (x[q] > -INFINITY) {
          const Near y = near_of(b, x[q]);
          note(b, (w & 16383) * 32 + lane, y.t, y.e);
        }
      }
    }
  } else {
    each_group(note);
  }
  __syncthreads();
  if (s_groups > kPickGroups) {
    // too many to note: a bound from the groups themselves, and once more
    bound_of(each_group, kPickThreads);
    bound = of_key(lo);
    if (tid == 0) s_groups = 0;
    __syncthreads();
    each_group(note);
    __syncthreads();
  }
  const bool noted = s_groups <= kPickGroups;
  if (noted && s_groups > k + (k >> 2) + 16) {
    // the k-th best of the noted groups is a better bound
    const int n = s_groups;
    for (int i = n + tid; i < kPickGroups + 1; i += kPickThreads) s_key[i] = 0u;
    __syncthreads();
    if (warp == 0) {
      const uint32_t cut = bisect(s_key, n, k, lo);
      if (lane == 0) s_cut = cut;
    }
    __syncthreads();
    lo = s_cut;
    bound = of_key(lo);
  }
  const int n_scan = (noted ? s_groups : n_group) * kVecs;
  // f(beam, logit, token) for every token of those groups that may reach the bound, a vector at a time; a
  // finished beam gives its pad token.  With `again`, of one beam alone where `only` names it: few calls come to this, and
  // its code is kept small (the vectors unrolled here too: 7 x 50 rows of 50257 fp32 29 us instead of 28).
  int only = -1;
  auto each = [&](auto again, auto f) {
    constexpr bool kAgain = decltype(again)::value;
    const bool part = kAgain && !noted && only >= 0;
    const int last = part ? (only + 1) * per_row * kVecs : n_scan;
    for (int j = (part ? only * per_row * kVecs : 0) + tid; j < last; j += kPickThreads) {
      int b, i;
      if (noted) {
        if (s_up[j / kVecs] < bound) continue;
        b = s_group[j / kVecs] >> 19;
        i = s_group[j / kVecs] & ((1 << 19) - 1);
      } else {
        b = j / kVecs / per_row;
        i = j / kVecs % per_row;
      }
      if (kAgain && only >= 0 && b != only) continue;
      const int kind = s_kind[b];
      if (kind == 2 && i == 0 && j % kVecs == 0) f(b, 0.f, p.pad_token);
      if (kind != 1) continue;
      const int v = (i / 32) * tile_elems<T>() + (j % kVecs) * 32 * N + (i % 32) * N;
      if (v >= p.V) continue;
      const T* lr = static_cast<const T*>(p.logits) + (row0 + b) * p.ld;
      const uint4 q = p.aligned ? load_vec<T, 16>(lr, v, p.V) : load_partial<T>(lr + v, p.V - v);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      const uint32_t bits = p.allowed ? allowed_bits(p, row0 + b, v) : ~0u;
      const float above = s_max[b] == INFINITY ? FLT_MAX : -INFINITY;    // beside +inf, the others' totals are -inf
#pragma unroll(kAgain ? 1 : N)
      for (int e = 0; e < N; ++e) {
        const float x = P::at(w[e / (N / 4)], e);
        if (x > above && (bits >> e & 1u)) {
          const Near y = near_of(b, x);
          if (y.t + y.e >= bound) f(b, x, v + e);
        }
      }
    }
  };
  auto rank_of = [&](int b, float x, int token) {
    return Rank{s_kind[b] == 2 ? okey(s_cum[b]) : key_of(b, x), tie_of(b, x, token)};
  };
  each(std::false_type(), [&](int b, float x, int token) {
    const int at = atomicAdd(&s_count, 1);
    if (at < kPickCap) s_rank[at] = Rank{(unsigned long long)__float_as_uint(x), tie_of(b, x, token)};
  });
  __syncthreads();
  int count = s_count;
  if (count <= kPickCap) {
    for (int i = tid; i < count; i += kPickThreads) {      // (their exact totals, now that each has a thread)
      const int b = 255 - (int)(s_rank[i].tie >> 56);
      s_rank[i].key = s_kind[b] == 2 ? okey(s_cum[b]) : key_of(b, __uint_as_float((uint32_t)s_rank[i].key));
    }
    __syncthreads();
  } else {
    // too many: the exact k-th candidate, by its total and then by its tie.  One scan of the tokens per turn:
    // the range of their totals, counts at probes into it, the beams of those equal to the k-th, the range of the
    // ties in the beam that the last of them is from, counts at probes, and what is to be taken.
    enum { kTotals, kTotalCount, kBeams, kTies, kTieCount, kTake };
    unsigned long long a = 0, b = 0, kth = 0, probe = 0;
    int want = k;
    for (int turn = kTotals;;) {
      __syncthreads();
      if (tid == 0) {
        s_count = 0;
        s_range[0] = ~0ull;
        s_range[1] = 0ull;
      }
      if (turn == kBeams && tid < TR_MAX_BEAMS) s_key[tid] = 0u;
      __syncthreads();
      unsigned long long lo64 = ~0ull, hi64 = 0ull;
      int c = 0, run = 0, run_beam = 0;                    // (tokens of one beam counted before they are added)
      each(std::true_type(), [&](int beam, float x, int token) {
        const Rank q = rank_of(beam, x, token);
        if (turn == kTotals || turn == kTies) {
          if (turn == kTotals ? q.key != 0ull : q.key == kth) {
            const unsigned long long y = turn == kTotals ? q.key : q.tie;
            lo64 = min(lo64, y);
            hi64 = max(hi64, y);
          }
        } else if (turn == kTotalCount) {
          c += q.key >= probe;
        } else if (turn == kBeams) {
          c += q.key > kth;
          if (q.key == kth) {
            if (beam != run_beam) {
              if (run) atomicAdd(&s_key[run_beam], (uint32_t)run);
              run = 0;
              run_beam = beam;
            }
            ++run;
          }
        } else if (turn == kTieCount) {
          c += q.key == kth && q.tie >= probe;
        } else if (q.key > kth || (q.key == kth && q.tie >= a)) {
          s_rank[atomicAdd(&s_count, 1)] = q;              // k at most (ties differ)
        }
      });
      if (run) atomicAdd(&s_key[run_beam], (uint32_t)run);
      if (lo64 <= hi64) {
        atomicMin(&s_range[0], lo64);
        atomicMax(&s_range[1], hi64);
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c) atomicAdd(&s_count, c);
      __syncthreads();
      if (turn == kTake) break;
      if (turn == kTotals || turn == kTies) {
        a = s_range[0];
        b = s_range[1];
        if (a > b) {                                       // every total is -inf
          if (tid == 0) s_count = 0;
          break;
        }
        turn = turn == kTotals ? kTotalCount : kTieCount;
      } else if (turn != kBeams) {
        if (s_count >= want) a = probe; else b = probe - 1;
      } else {
        want -= s_count;
        int beam = 0;
        while (beam < p.W && (int)s_key[beam] < want) want -= (int)s_key[beam++];
        only = beam < p.W ? beam : -1;                     // (-1: all of them are taken)
        a = 0;
        turn = only >= 0 ? kTies : kTake;
      }
      if (turn == kTotalCount || turn == kTieCount) {
        if (a < b) {
          probe = a + (b - a) / 2 + 1;
        } else if (turn == kTotalCount) {
          kth = a;
          turn = kBeams;
        } else {
          only = -1;
          turn = kTake;
        }
      }
    }
    __syncthreads();
    count = s_count;
  }
  // the totals rounded to fp32 order the candidates but for ties; those that may be among the k best
  uint32_t cut = 0u, mykey = 0u;
  for (int i = tid; i < count; i += kPickThreads) mykey = max(mykey, s_key[i] = s_rank[i].key ? okey((float)of_key(s_rank[i].key)) : 0u);
  if (tid == 0) s_groups = 0;
  if (count > 2 * k + 32) {
    s_best[tid] = mykey;
    if (__syncthreads_count(mykey > 0u) >= k) {
      if (warp == 0) {
        const uint32_t c = bisect(s_best, count, k, 1u);
        if (lane == 0) s_cut = c;
      }
      __syncthreads();
      cut = s_cut;
    }
  }
  __syncthreads();
  for (int i = tid; i < count; i += kPickThreads)
    if (s_key[i] >= cut) {
      const int at = atomicAdd(&s_groups, 1);
      s_sel[at] = i;
      s_sel_key[at] = s_key[i];
    }
  __syncthreads();
  const int n_sel = s_groups;
  if (tid < (-n_sel & 3)) s_sel_key[n_sel + tid] = 0u;
  __syncthreads();
  auto put = [&](int j, const Rank& q) {
    const int64_t at = (int64_t)r * k + j;
    const bool some = q.key != 0ull;                       // (0: a total of -inf)
    p.parent[at] = some ? 255 - (int)(q.tie >> 56) : -1;
    p.token[at] = some ? (1 << kTokenBits) - 1 - (int)(q.tie & ((1u << kTokenBits) - 1)) : -1;
    p.score[at] = some ? (float)of_key(q.key) : -INFINITY;
  };
  // each of them counts those before it
  const uint4* key4 = reinterpret_cast<const uint4*>(s_sel_key);
  for (int i = tid; i < n_sel; i += kPickThreads) {
    const uint32_t key = s_sel_key[i];
    int at = 0, same = 0;
#pragma unroll 4
    for (int j = 0; j < (n_sel + 3) / 4; ++j) {
      const uint4 o = key4[j];
      at += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
      same += (o.x == key) + (o.y == key) + (o.z == key) + (o.w == key);
    }
    if (at >= k) continue;
    const Rank q = s_rank[s_sel[i]];
    if (same > 1)
      for (int j = 0; j < n_sel; ++j) at += s_sel_key[j] == key && before(s_rank[s_sel[j]], q);
    if (at < k) put(at, q);
  }
  for (int j = count + tid; j < k; j += kPickThreads) {
    const int64_t at = (int64_t)r * k + j;
    p.parent[at] = p.token[at] = -1;
    p.score[at] = -INFINITY;
  }
}

// ---------------------------------------------------------------- reorder
// One CTA moves one column slice of one state of one request: every surviving row's slice is
// loaded into registers before the first is stored, and no other CTA touches the slice, so the
// move is safe in place whatever the parents are.  Traffic: each row read once (children of one
// parent read it again from L2) and written once.  16 states of 32 x 32 rows of 98 KB under random parents:
// 432 us, of 401 that the 63 % of rows with a child, read, and all rows, written, take at a copy's rate.
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
  int n_tile;
  size_t sum_bytes, total;
};
SelectPlan plan_select(int64_t rows, int V, bool f32) {
  SelectPlan s;
  const int elems = f32 ? tile_elems<float>() : tile_elems<__nv_bfloat16>();
  s.n_tile = (V + elems - 1) / elems;
  s.sum_bytes = ((size_t)rows * s.n_tile * sizeof(TileSum) + 255) / 256 * 256;
  s.total = s.sum_bytes + (size_t)rows * s.n_tile * 32 * sizeof(float);
  return s;
}

template <typename T>
tr_status launch_select(const SelectParams& p, int R, uintptr_t align, cudaStream_t st) {
  const dim3 grid((unsigned)(R * p.W), (unsigned)((p.n_tile + kSumThreads / 32 - 1) / (kSumThreads / 32)));
  // rows at 16-byte aligned addresses are read 16 bytes at a time
  if (align % 16 == 0)
    beam_sum_kernel<T, 16><<<grid, kSumThreads, 0, st>>>(p);
  else if (sizeof(T) == 4 || align % 4 == 0)
    beam_sum_kernel<T, 4><<<grid, kSumThreads, 0, st>>>(p);
  else
    beam_sum_kernel<T, 2><<<grid, kSumThreads, 0, st>>>(p);
  TR_LAUNCH_CHECK("beam_sum_kernel");
  constexpr int kPickBytes = kPickCap * (sizeof(Rank) + sizeof(int));
  TR_TRY(ensure_smem_attr((const void*)beam_pick_kernel<T>, kPickBytes));
  return launch_dependent(true, beam_pick_kernel<T>, (unsigned)R, kPickThreads, kPickBytes, st, "beam_pick_kernel", p);
}

tr_status check_select(int R, int W, int V, int k) {
  if (W < 1 || W > TR_MAX_BEAMS) return fail(TR_ERR_INVALID_ARG, "W=%d (need 1..%d)", W, TR_MAX_BEAMS);
  if (R < 1 || (int64_t)R * W >= (1 << 20)) return fail(TR_ERR_INVALID_ARG, "R=%d (need R >= 1 and R*W < 2^20)", R);
  if (V < 1 || V > (1 << kTokenBits)) return fail(TR_ERR_INVALID_ARG, "V=%d (need 1..2^24)", V);
  if (k < 1 || k > TR_MAX_BEAM_K) return fail(TR_ERR_INVALID_ARG, "k=%d (need 1..%d)", k, TR_MAX_BEAM_K);
  return TR_OK;
}

tr_status check_reorder(const tr_beam_state* states, int n_states, const int32_t* parent, int R, int W_in, int W_out) {
  if (n_states < 0) return fail(TR_ERR_INVALID_ARG, "n_states=%d", n_states);
  if (W_in < 1 || W_in > TR_MAX_BEAMS || W_out < 1 || W_out > TR_MAX_BEAMS)
    return fail(TR_ERR_INVALID_ARG, "W_in=%d, W_out=%d (need 1..%d)", W_in, W_out, TR_MAX_BEAMS);
  if (R < 1 || (int64_t)R * std::max(W_in, W_out) >= (1 << 20))
    return fail(TR_ERR_INVALID_ARG, "R=%d (need R >= 1 and R*W < 2^20)", R);
  if (n_states > 0 && (!states || !parent)) return fail(TR_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)parent % 4) return fail(TR_ERR_INVALID_ARG, "parent is not aligned to its type");
  const Rows par{parent, W_out * 4ll, W_out * 4ll, R};
  for (int i = 0; i < n_states; ++i) {
    const tr_beam_state& s = states[i];
    if (s.row_bytes < 0 || (s.row_bytes > 0 && (!s.dst || !s.src)))
      return fail(TR_ERR_INVALID_ARG, "state %d: row_bytes=%lld or null pointer", i, (long long)s.row_bytes);
    if (s.dst_stride < s.row_bytes || s.src_stride < s.row_bytes || std::max(s.dst_stride, s.src_stride) > (1ll << 40))
      return fail(TR_ERR_INVALID_ARG, "state %d: stride below row_bytes or too large", i);
    if (s.dst == s.src && (W_in != W_out || s.dst_stride != s.src_stride))
      return fail(TR_ERR_INVALID_ARG, "state %d: in place needs W_in == W_out and equal strides", i);
    if (overlap(Rows{s.dst, s.dst_stride, s.row_bytes, (int64_t)R * W_out}, par))
      return fail(TR_ERR_INVALID_ARG, "state %d: dst overlaps parent", i);
    for (int j = 0; j < i + 1 && s.row_bytes > 0; ++j) {
      const tr_beam_state& o = states[j];
      const Rows sd{s.dst, s.dst_stride, s.row_bytes, (int64_t)R * W_out}, ss{s.src, s.src_stride, s.row_bytes, (int64_t)R * W_in};
      const Rows od{o.dst, o.dst_stride, o.row_bytes, (int64_t)R * W_out}, os{o.src, o.src_stride, o.row_bytes, (int64_t)R * W_in};
      const bool bad = i == j ? s.dst != s.src && overlap(sd, ss) : overlap(sd, os) || overlap(sd, od) || overlap(ss, od);
      if (bad) return fail(TR_ERR_INVALID_ARG, "states %d and %d: dst overlaps rows of another state, or its own src", j, i);
    }
  }
  return TR_OK;
}

}  // namespace
}  // namespace tr

using namespace tr;

extern "C" size_t tr_beam_select_workspace(int R, int W, int V, int k) {
  if (check_select(R, W, V, k) != TR_OK) return SIZE_MAX;
  const int64_t rows = (int64_t)R * W;
  return std::max(plan_select(rows, V, true).total, plan_select(rows, V, false).total);
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
  const SelectPlan sp = plan_select(rows, V, logits_dtype == TR_F32);
  if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < sp.total)
    return fail(TR_ERR_INVALID_ARG, "workspace: need %zu bytes, 16-byte aligned", sp.total);
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
  p.n_tile = sp.n_tile;
  p.sums = static_cast<TileSum*>(workspace);
  p.best = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.sum_bytes);
  p.parent = parent;
  p.token = token;
  p.score = score;
  const uintptr_t align = (uintptr_t)logits | (uintptr_t)(rows > 1 ? ld * esize : 0);
  p.aligned = align % 16 == 0;
  return logits_dtype == TR_F32 ? launch_select<float>(p, R, align, st) : launch_select<__nv_bfloat16>(p, R, align, st);
}

extern "C" tr_status tr_beam_reorder_check(const tr_beam_state* states, int n_states, const int32_t* parent, int R, int W_in,
                                           int W_out) {
  return check_reorder(states, n_states, parent, R, W_in, W_out);
}

extern "C" tr_status tr_beam_reorder(const tr_beam_state* states, int n_states, const int32_t* parent, int R, int W_in,
                                     int W_out, tr_stream stream) {
  if (n_states > TR_MAX_STATES) return fail(TR_ERR_INVALID_ARG, "n_states=%d (need 0..%d)", n_states, TR_MAX_STATES);
  TR_TRY(check_reorder(states, n_states, parent, R, W_in, W_out));
  if (n_states == 0) return TR_OK;
  MoveParams p{};
  uintptr_t align = 0;
  for (int i = 0; i < n_states; ++i) {
    const tr_beam_state& s = states[i];
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

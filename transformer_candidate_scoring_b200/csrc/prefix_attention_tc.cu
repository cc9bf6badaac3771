// The prefix part of tr_prefix_attention on the tensor cores (bf16).
//
// A request's query rows of one key head -- sequences x query tokens x the heads that share the
// key head -- form one matrix Q against the shared keys, so the prefix is an attention of many
// rows over one K and V:  S = Q K^T (128 rows x 128 keys per step, TMEM), P = 2^(c S - c m) in
// registers with the running row maximum m and sum l, O += P V (P back in TMEM as bf16, the A
// operand; O in TMEM, fp32).  Nothing of S or P leaves the SM.
//
// A CTA holds two row tiles, each with its own softmax warpgroup, so that the tensor core works
// on one tile while the other is in its exponentials.  A unit of more than 128 rows gives the
// two tiles different rows of the same keys; a unit of at most 128 rows gives both the same rows
// and every other step of keys (their results are merged at the unit's end).
//
//   TMEM, 512 columns   S/P of tile 0, S/P of tile 1 (128 each), O of tile 0, O of tile 1
//   shared memory       Q tiles, a ring of K steps and one of V steps; all in the
//                       128-byte-swizzled layout (K-major for Q and K; V is [keys][d_head], the
//                       MN-major form), K and V by TMA, d_head padded to 64 or 128 by TMA's zeros
//   warps 0-3, 4-7      softmax of tile 0 and 1, one row per thread, and the epilogue
//   warps 8, 9, 10      K loads, V loads, MMA issue
//   warp 11             tensor memory; the next unit's Q where shared memory has room for it
//
// A step's chain -- S, softmax, P V, of which the next S waits because P lies where S was -- bounds
// many rows: 2 x 4,096 sequences with 16 heads of 128 on 4 over 4,096 keys take 279 us (985 TFLOP/s),
// the tensor core busy 45 % and the exponentials' unit 45 % of it.  Steps of 64 keys with two S buffers
// per tile, separate S and P with steps of 80 keys, one MMA warp per tile, two threads per row and a part
// of the exponentials on the FMA pipes measured no faster (319 to 427 us against 322 of the kernel then).
// Few rows are bound by the read of K and V: 1 x 16 sequences over 131,072 keys, 268 MB in 51 us.  Short
// prefixes are bound by what a unit costs once (Q, the first S, the result): 16 x 4,096 sequences with 8
// heads of 16 over 16 to 128 keys, 14 units per SM, take 75 us, and took 91 with one Q buffer that the softmax
// warps filled between units.
//
// The row maximum that O and l are relative to is raised only when the new one is more than 2^8
// away (then O is rescaled in TMEM): numerators stay below 2^8 and sums in fp32 range.  Values
// behind a prefix are kept out twice: their scores are replaced by -inf, and the V rows that the
// last 16-key slice would still multiply by 0 are zeroed in shared memory (0 x NaN is NaN).
//
// Every wait is bounded: a stalled barrier sets an error bit and the kernel unwinds, behind its copies and products
// in flight.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "prefix_attention.cuh"
#include "tc_common.cuh"

namespace tr {
namespace attn {
namespace {

using namespace tc;

constexpr int kM = 128, kN = kStepKeys;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kCtlRegs = 56, kSoftmaxRegs = 216;
static_assert(128 * kCtlRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs && kThreads * kLaunchRegs <= 65536,
              "register split");
constexpr float kRaise = 8.f;    // log2 of how far numerators may exceed 1

template <int DH>    // d_head padded to 64 or 128
struct Smem {
  static constexpr int TILE = 128 * DH * 2;
  static constexpr int NK = DH == 128 ? 3 : 4, NV = DH == 128 ? 2 : 4;
  static constexpr int NQ = DH == 128 ? 2 : 4;   // Q tiles
  static constexpr int Q = 0, K = NQ * TILE, V = K + NK * TILE, BAR = V + NV * TILE;
  static constexpr int ML = BAR + 256;           // m and l of tile 1's rows (merge)
  static constexpr int BYTES = ML + 1024 + 1024;   // + alignment of the base
};
static_assert(Smem<128>::BYTES <= 232448 && Smem<64>::BYTES <= 232448, "shared memory plan");

struct TcParams {
  CUtensorMap kmap, vmap;
  AttnParams a;
};

__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {    // K-major, 128-byte swizzle
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// MN-major, 128-byte swizzle: 64 elements of N per 128-byte row, 8 K rows per 1024-byte atom;
// the next 64 of N `n_step` bytes further, the next 8 of K 1024 bytes further.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t n_step) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((n_step >> 4) & 0x3FFF) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
constexpr uint32_t kBMajorMN = 1u << 16;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A warp's wait; every lane gives up when one does.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}
// One lane of a converged warp.  The compiler knows this instruction to pick a single lane and keeps the
// operands of the MMAs under it in uniform registers; under `lane == 0` it does not, and each issue
// took 80 to 120 cycles instead of the product's own 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// acc + the products of two bf16 pairs.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float acc) {
  acc = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), acc);
  return fmaf(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u), acc);
}

// The 16-byte piece c of row r of a Q tile.
__device__ __forceinline__ uint32_t piece(uint32_t tile, int r, int c) {
  return tile + r * 128 + (c >> 3) * (128 * 128) + (((c & 7) ^ (r & 7)) << 4);
}

// Whether Q has two buffers, so that a unit's rows come while the one before it is worked on: d_head up to
// 64 (there the rings leave room for four tiles), or units that all have one tile of rows (kOne; 32 sequences
// with 4 heads of 128 on each key head over 16 ragged prefixes: 119 -> 112 us).
template <int DH, bool kOne>
constexpr bool kQAhead = DH == 64 || kOne;
// Bytes from one Q buffer to the other.
template <int DH, bool kOne>
constexpr uint32_t kQBuffer = (DH == 64 ? 2 : 1) * Smem<DH>::TILE;

struct Bars {
  uint32_t kfull, kempty, vfull, vempty;   // rings, 8 bytes apart
  uint32_t qfull, sfull, pfull, odone;     // per tile (pfull: two per tile; qfull: per buffer if there are two)
  uint32_t qempty;                         // per buffer
  uint32_t ml_full, ml_empty;
  uint32_t drain;                          // unwinding: the products issued so far
};

// One thread: streams the K (or V) steps of every unit into its ring.
template <int DH>
__device__ void load_steps(const AttnParams& p, const CUtensorMap* map, uint32_t ring, int slots, uint32_t full, uint32_t empty,
                           volatile int* abort_flag) {
  int s = 0;
  uint32_t ph = 0;
  bool ok = true;
  uint32_t pending = 0, par = 0;           // bit s: a load of slot s was issued, and its parity
  const int end = end_of(p);
  for (int u = first_of(p); u < end && ok;) {
    const Unit x = unit_at(p, u, kUnitRows, kN);
    u = after(p, u, x);
    for (int j = 0; j < x.steps; ++j) {
      if (!(ok = mbar_wait_idle(empty + 8 * s, ph ^ 1, abort_flag))) break;
      const uint32_t dst = ring + s * Smem<DH>::TILE;
      mbar_arrive_expect_tx(full + 8 * s, Smem<DH>::TILE);
#pragma unroll
      for (int h = 0; h < DH / 64; ++h) tma_load_3d(dst + h * (128 * 128), map, h * 64, x.hk, x.tok + j * kN, full + 8 * s);
      pending |= 1u << s;
      par = (par & ~(1u << s)) | (ph << s);
      if (++s == slots) { s = 0; ph ^= 1; }
    }
  }
  if (!ok) {   // unwinding: let the copies in flight land before the CTA's memory is given back
    int none = 0;
    for (int i = 0; i < slots; ++i)
      if (pending >> i & 1) mbar_wait_idle(full + 8 * i, par >> i & 1, &none, 200000000ull);
  }
}

// The whole warp: one lane issues, all lanes zero V rows behind the prefix.
template <int DH, bool kOne>
__device__ void issue_mmas(const TcParams& p, uint32_t tmem, uint32_t smem, const Bars& b, int lane, volatile int* abort_flag) {
  using L = Smem<DH>;
  const int dk = (p.a.d.d_head + 15) / 16;                 // 16-wide slices of d_head
  const uint32_t id_o = idesc_bf16(kM, dk * 16) | kBMajorMN, id_full = idesc_bf16(kM, kN);
  const uint64_t q0 = desc_k(smem + L::Q), k0 = desc_k(smem + L::K), v0 = desc_mn(smem + L::V, 128 * 128);
  int ks = 0, vs = 0;                                      // ring slots of the current step
  uint32_t kph = 0, vph = 0, qph[2] = {0, 0}, pph[2] = {0, 0};
  constexpr bool kAhead = kQAhead<DH, kOne>;
  int buf = 0;                                             // Q buffer
  bool ok = true;
  const int end = end_of(p.a);
  for (int u = first_of(p.a); u < end && ok;) {
    const Unit x = unit_at(p.a, u, kUnitRows, kN);
    u = after(p.a, u, x);
    const bool two = !kOne && x.two;
    const int n_jobs = two ? 2 * x.steps : x.steps;
    const int last = x.keys - (x.steps - 1) * kN;          // keys of the last step
    auto qk = [&](int i) {
      const int t = i & 1, step = two ? i >> 1 : i;
      if (i < (kAhead ? 1 : 2)) {
        ok = ok && wait_all(b.qfull + 8 * (kAhead ? buf : t), qph[kAhead ? buf : t], abort_flag);
        qph[kAhead ? buf : t] ^= 1;
      }
      ok = ok && wait_all(b.kfull + 8 * ks, kph, abort_flag);
      if (!ok) return;
      const bool done = !two || t == 1;                    // nothing reads these keys any more
      tc_fence_after();
      if (elect_one()) {
        const uint64_t qa = q0 + (kAhead ? buf * (kQBuffer<DH, kOne> >> 4) + (two ? t * (L::TILE >> 4) : 0) : t * (L::TILE >> 4)), ka = k0 + ks * (L::TILE >> 4);
        const uint32_t id = step == x.steps - 1 ? idesc_bf16(kM, (last + 15) & ~15) : id_full;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
          if (kk < dk) {
            const uint64_t o = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
            mma_bf16(tmem + t * kN, qa + o, ka + o, id, kk > 0);
          }
        mma_commit(b.sfull + 8 * t);
        if (done) mma_commit(b.kempty + 8 * ks);
        if (kAhead && i == n_jobs - 1) mma_commit(b.qempty + 8 * buf);
      }
      if (done && ++ks == L::NK) { ks = 0; kph ^= 1; }
    };
    if (n_jobs > 0) qk(0);
    if (n_jobs > 1) qk(1);
    if (kAhead && n_jobs == 0) {                           // (no prefix)
      ok = ok && wait_all(b.qfull + 8 * buf, qph[buf], abort_flag);     // (else a later unit's wait could meet this phase)
      qph[buf] ^= 1;
      if (lane == 0) mbar_arrive(b.qempty + 8 * buf);
    }
    for (int i = 0; i < n_jobs && ok; ++i) {
      const int t = i & 1, k = i >> 1, step = two ? k : i;
      const int valid = step == x.steps - 1 ? last : kN;
      const bool done = !two || t == 1;
      if (t == 0 || !two) {
        ok = wait_all(b.vfull + 8 * vs, vph, abort_flag);
        if (ok && (valid & 15)) {
          // rows valid .. the end of their 16-key slice: 16-byte pieces of the 128-byte rows
          const uint32_t va = smem + L::V + vs * L::TILE;
          const int n_rows = 16 - (valid & 15);
          for (int c = lane; c < n_rows * 8 * (DH / 64); c += 32) {
            const int h = c / (n_rows * 8), rr = (c / 8) % n_rows;
            st_shared_v4(va + h * (128 * 128) + (valid + rr) * 128 + (c & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      const uint64_t va = v0 + vs * (L::TILE >> 4);
      const int nk = (valid + 15) / 16;
#pragma unroll
      for (int half = 0; half < 2; ++half) {               // P comes in two halves of 64 keys
        ok = ok && wait_all(b.pfull + 8 * (2 * t + half), pph[t], abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = half * (kN / 32); kk < (half + 1) * (kN / 32); ++kk)
            if (kk < nk)
              mma_bf16_ta(tmem + 2 * kN + t * 128, tmem + t * kN + kk * 8, va + kk * (2048 >> 4), id_o, (k > 0 || kk > 0) ? 1u : 0u);
          if (half == 1) {
            if (done) mma_commit(b.vempty + 8 * vs);
            if (i + 2 >= n_jobs) mma_commit(b.odone + 8 * t);
          }
        }
      }
      pph[t] ^= 1;
      if (!ok) break;
      if (done && ++vs == L::NV) { vs = 0; vph ^= 1; }
      if (i + 2 < n_jobs) qk(i + 2);
    }
    buf ^= 1;
  }
  if (!ok) {   // unwinding: products in flight end before tensor and shared memory are given back
    int none = 0;
    if (elect_one()) mma_commit(b.drain);
    mbar_wait_idle(b.drain, 0, &none, 200000000ull);
  }
}

// What a softmax thread knows of its row of a unit.
struct Row {
  Unit x;
  int base, jobs;        // the tile's first row in the unit, its steps
  bool live, warp_live;
  int token, head;       // query token of the batch, head
};
__device__ __forceinline__ Row row_at(const AttnParams& p, int u, int t, int tid) {
  Row r;
  r.x = unit_at(p, u, kUnitRows, kN);
  r.base = r.x.two ? t * kM : 0;
  r.jobs = r.x.jobs(t);
  r.live = r.base + tid < r.x.rows;
  r.warp_live = r.base + (tid & ~31) < r.x.rows;
  const int G = p.group, m = r.x.m0 + r.base + tid;     // row within (request, key head)
  const int tok = fast_div(m, p.div_g);
  r.token = p.req[r.x.r].s0 * p.d.L_t + tok;
  r.head = r.x.hk * G + m - tok * G;
  return r;
}
// Where a row's own key begins (and its value).
__device__ __forceinline__ int64_t own_at(const AttnParams& p, const Row& r) {
  return (int64_t)fast_div(r.token, p.div_lt) * p.d.suffix_seq + (int64_t)r.x.hk * p.d.suffix_head;
}
// Asks for a row's own key and value to be brought to L2, a unit ahead of their use.
__device__ __forceinline__ void ask_own(const AttnParams& p, const Row& r) {
  if (!r.live || p.d.suffix_cap == 0) return;
  const int64_t at = own_at(p, r);
  for (int i = 0; i < p.d.d_head; i += 64) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __nv_bfloat16*>(p.k_suffix) + at + i));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __nv_bfloat16*>(p.v_suffix) + at + i));
  }
}
// This thread's row of Q into the Q tile, eight 16-byte pieces in flight.
template <int DH>
__device__ __forceinline__ void fill_q(const AttnParams& p, const Row& r, uint32_t tile, int tid) {
  const int D = p.d.d_head;
  const bool in = r.live;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                  (in ? r.token * p.d.q_token + r.head * D : 0));
#pragma unroll
  for (int i0 = 0; i0 < DH / 8; i0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = in && (i0 + i) * 8 < D ? __ldg(q + i0 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i0 + i) * 8 < D + 8) st_shared_v4(piece(tile, tid, i0 + i), v[i].x, v[i].y, v[i].z, v[i].w);
  }
}

// The whole warp: brings the Q rows of every unit but the first (which the softmax warps, idle till then, fill in) into its
// buffer, and asks for their own keys and values.
template <int DH, bool kDirect, bool kOne>
__device__ void load_q(const AttnParams& p, uint32_t smem, const Bars& b, int lane, volatile int* abort_flag) {
  const int D = p.d.d_head, pieces = (D + 15) / 16 * 2, G = p.group;     // 16-byte pieces, two per slice
  const int per = 32 / pieces, own_c = lane % pieces, own_r = lane / pieces;
  const int end = end_of(p);
  uint32_t ph[2] = {1, 1};
  int buf = 0;
  for (int u = first_of(p); u < end;) {
    const Unit x = unit_at(p, u, kUnitRows, kN);
    const bool first = u == first_of(p);
    u = after(p, u, x);
    if (!wait_all(b.qempty + 8 * buf, ph[buf], abort_flag)) return;
    ph[buf] ^= 1;
    if (first) {
      buf ^= 1;
      continue;
    }
    const uint32_t tiles = smem + Smem<DH>::Q + buf * kQBuffer<DH, kOne>;
    const int token0 = p.req[x.r].s0 * p.d.L_t;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)x.hk * G * D + own_c * 8;
    if (own_r < per)                                       // (what a tile holds behind its rows reaches no result)
      for (int r = own_r; r < x.rows; r += per) {
        const int m = x.m0 + r, tok = fast_div(m, p.div_g);
        const bool in = own_c * 8 < D;
        const __nv_bfloat16* src = q + (in ? (token0 + tok) * p.d.q_token + (m - tok * G) * D : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(piece(tiles + (r >> 7) * Smem<DH>::TILE, r & 127, own_c)),
                     "l"(src - (in ? 0 : own_c * 8)), "r"(in ? 16 : 0)
                     : "memory");
      }
    if (kDirect && p.d.suffix_cap > 0)
      for (int r = lane; r < x.rows; r += 32) {
        const int tok = token0 + fast_div(x.m0 + r, p.div_g);
        const int64_t at = (int64_t)fast_div(tok, p.div_lt) * p.d.suffix_seq + (int64_t)x.hk * p.d.suffix_head;
        for (int i = 0; i < D; i += 64) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __nv_bfloat16*>(p.k_suffix) + at + i));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __nv_bfloat16*>(p.v_suffix) + at + i));
        }
      }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    mbar_arrive(b.qfull + 8 * buf);
    buf ^= 1;
  }
}

// A softmax warpgroup (tile t): turns S into P step by step and writes the result.  Where Q has one buffer,
// its next rows are filled in here once the unit's products are done.
template <int DH, bool kDirect, bool kOne>
__device__ void softmax_tile(const TcParams& tp, int t, uint32_t tmem, uint32_t smem, float* sml, const Bars& b,
                             volatile int* abort_flag) {
  using L = Smem<DH>;
  const AttnParams& p = tp.a;
  const int tid = threadIdx.x & 127, lane = tid & 31, wrow = tid & ~31;    // wrow: the warp's first row
  const uint32_t lanes = (uint32_t)wrow << 16;                              // its TMEM lanes
  constexpr bool kAhead = kQAhead<DH, kOne>;
  uint32_t q_tile = smem + L::Q + t * L::TILE, qph = 0;
  int buf = 0;
  const uint32_t s_addr = tmem + t * kN + lanes, o_addr = tmem + 2 * kN + t * 128 + lanes;
  const int D = p.d.d_head;
  const float c = p.d.scale * kLog2e;
  const uint64_t c2 = f32x2(c, c);
  uint32_t sph = 0, oph = 0, xph = 0;
  bool ok = true;
  const int end = end_of(p);
  int u = first_of(p);
  Row next = row_at(p, u, t, tid);
  if (!kOne || t == 0) fill_q<DH>(p, next, q_tile, tid);
  if (kDirect) ask_own(p, next);
  if constexpr (kAhead) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane < 4) mbar_arrive(b.qfull);                    // 32 in all
  }
  while (u < end && ok) {
    const Row rw = kAhead ? row_at(p, u, t, tid) : next;
    const Unit& x = rw.x;
    const RequestPlan& rq = p.req[x.r];
    const bool live = rw.live, warp_live = rw.warp_live;
    const int jobs = rw.jobs;
    if (!kAhead && jobs > 0) {
      fence_proxy_async_smem();
      mbar_arrive(b.qfull + 8 * t);
    }
    float mx = -INFINITY;          // the reference maximum of S, unscaled
    float l = 0.f;
    for (int k = 0; k < jobs; ++k) {
      const int valid = min(kN, x.keys - x.step_of(t, k) * kN);
      if (!(ok = wait_all(b.sfull + 8 * t, sph, abort_flag))) break;
      sph ^= 1;
      tc_fence_after();
      float mc = 0.f;
      float s[kN];
      if (warp_live) {
#pragma unroll
        for (int i = 0; i < kN / 32; ++i)
          if (i * 32 < valid) tmem_ld32(s_addr + 32 * i, s + 32 * i);
        tmem_wait_ld();
        reg_fence<kN>(s);
        if (valid < kN) {
#pragma unroll
          for (int i = 0; i < kN; i += 32)
            if (i + 32 > valid) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (i + e >= valid) s[i + e] = -INFINITY;
            }
        }
        float n0 = mx, n1 = s[0], n2 = s[1], n3 = s[2];
#pragma unroll
        for (int i = 3; i + 7 < kN; i += 8) {
          n0 = max3(n0, s[i], s[i + 1]);
          n1 = max3(n1, s[i + 2], s[i + 3]);
          n2 = max3(n2, s[i + 4], s[i + 5]);
          n3 = max3(n3, s[i + 6], s[i + 7]);
        }
        n0 = max3(n0, s[123], s[124]);
        n1 = max3(n1, s[125], s[126]);
        const float nm = max3(fmaxf(n0, s[127]), n1, fmaxf(n2, n3));
        const bool raise = k == 0 || (nm - mx) * c > kRaise;
        if (__any_sync(0xffffffffu, raise)) {
          // (the first step has no O yet; S of this step was committed after the last P V)
          const float f = raise ? (nm == mx ? 1.f : ex2((mx - nm) * c)) : 1.f;
          if (raise) mx = nm;
          if (k > 0) {
            l *= f;
            for (int i = 0; i * 16 < D; ++i) {
              float o[16];
              tmem_ld16(o_addr + 16 * i, o);
              tmem_wait_ld();
              reg_fence<16>(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tmem_st16(o_addr + 16 * i, o);
            }
            tmem_wait_st();
          }
        }
        mc = mx == -INFINITY ? 0.f : mx * c;              // keys of -inf weigh nothing, NaN stays NaN
      }
      const uint64_t mc2 = f32x2(-mc, -mc);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (warp_live) {
#pragma unroll
          for (int i = 2 * half; i < 2 * half + 2; ++i)
            if (i * 32 < valid) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float a, bb;
                f32x2_split(fma_f32x2(f32x2(s[32 * i + 2 * e], s[32 * i + 2 * e + 1]), c2, mc2), a, bb);
                a = ex2(a);
                bb = ex2(bb);
                sum[e & 1] = add_f32x2(sum[e & 1], f32x2(a, bb));
                w[e] = pack_bf16(a, bb);
              }
              asm volatile(
                  "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                      s_addr + 16 * i),
                  "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]),
                  "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
                  : "memory");
            }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b.pfull + 8 * (2 * t + half));
      }
      float a0, a1;
      f32x2_split(add_f32x2(sum[0], sum[1]), a0, a1);
      l += a0 + a1;
    }
    if (!ok) break;
    // ---- with kDirect, the row's own key: its score, from the Q row in shared memory
    bool own = false;
    float a = -INFINITY;
    const uint4* own_v = nullptr;
    if constexpr (kDirect) {
      if constexpr (kAhead) {        // (every warp waits, also for rows it does not have: none gets units ahead)
        q_tile = smem + L::Q + buf * kQBuffer<DH, kOne> + t * L::TILE;
        if (!(ok = wait_all(b.qfull + 8 * buf, qph, abort_flag))) break;
      }
      if (warp_live && (x.two || t == 0) && p.d.suffix_cap > 0) {
        const int seq = fast_div(rw.token, p.div_lt);
        own = live && visible_suffix(p, seq, rw.token - seq * p.d.L_t) > 0;
        const int64_t at = own_at(p, rw);
        own_v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v_suffix) + at);
        if (own) {
          const uint4* kr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_suffix) + at);
          float acc = 0.f;
#pragma unroll 8
          for (int i = 0; i < D / 8; ++i) {
            const uint4 kv = __ldg(kr + i);
            uint4 qv;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(qv.x), "=r"(qv.y), "=r"(qv.z), "=r"(qv.w)
                         : "r"(piece(q_tile, tid, i)));
            acc = dot2(qv.x, kv.x, dot2(qv.y, kv.y, dot2(qv.z, kv.z, dot2(qv.w, kv.w, acc))));
          }
          a = acc * c;
        }
      }
      if constexpr (kAhead) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b.qempty + 8 * buf);
      }
    }
    if (buf) qph ^= 1;
    buf ^= 1;
    u = after(p, u, x);
    const bool more = !kAhead && u < end;
    if (more) next = row_at(p, u, t, tid);
    // ---- the result of the unit's rows
    if (jobs > 0) {
      if (!(ok = wait_all(b.odone + 8 * t, oph, abort_flag))) break;
      oph ^= 1;
    }
    if (!x.two && t == 1) {
      // both tiles hold these rows: tile 1 hands its maximum and sum over, tile 0 reads its O
      sml[tid] = jobs > 0 ? mx : -INFINITY;
      sml[128 + tid] = l;
      tc_fence_before();
      mbar_arrive(b.ml_full);
      ok = wait_all(b.ml_empty, xph, abort_flag);
      xph ^= 1;
    } else {
      float w0 = 1.f, w1 = 0.f, lsum = l, mref = mx;
      if (!x.two) {
        if (!(ok = wait_all(b.ml_full, xph, abort_flag))) break;
        xph ^= 1;
        const float m1 = sml[tid], l1 = sml[128 + tid];
        mref = fmaxf(mx, m1);
        const float mb = mref == -INFINITY ? 0.f : mref;
        w0 = mx == mref ? 1.f : ex2((mx - mb) * c);
        w1 = m1 == mref ? 1.f : ex2((m1 - mb) * c);
        lsum = w0 * l + w1 * l1;
      }
      tc_fence_after();
      const bool second = !x.two && x.steps > 1;             // tile 1 has an O
      if (warp_live) {
        const int64_t row = (int64_t)rw.token * p.d.n_head + rw.head;
        float ref = __fmul_rn(mref, c);
        if (kDirect && own) {
          const float top = fmaxf(ref, a), tb = top == -INFINITY ? 0.f : top, f = ref == top ? 1.f : ex2(ref - tb);
          a = ex2(a - tb);
          lsum = lsum * f + a;
          w0 *= f;
          w1 *= f;
          ref = top;
        } else {
          a = 0.f;
        }
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        const float lse2 = lsum == 0.f ? -INFINITY : ref + log2f(lsum);
        const int64_t part = rq.part + x.split * request_rows(p, x.r) + (row - (int64_t)rq.s0 * p.d.L_t * p.d.n_head);
        w0 *= inv;
        w1 *= inv;
        a *= inv;
#pragma unroll 2
        for (int i = 0; i < (D + 15) / 16; ++i) {
          uint4 v[2];
          if constexpr (kDirect) {
#pragma unroll
            for (int h = 0; h < 2; ++h) v[h] = own && 16 * i + 8 * h < D ? __ldg(own_v + 2 * i + h) : make_uint4(0, 0, 0, 0);
          }
          float o[16], o1[16];
          tmem_ld16(o_addr + 16 * i, o);
          if (second) tmem_ld16(o_addr + 128 + 16 * i, o1);
          tmem_wait_ld();
          reg_fence<16>(o);
          reg_fence<16>(o1);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = x.steps == 0 ? 0.f : second ? o[e] * w0 + o1[e] * w1 : o[e] * w0;
          if constexpr (kDirect) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t vw[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
              if (own)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  o[8 * h + 2 * e] = fmaf(a, __uint_as_float(vw[e] << 16), o[8 * h + 2 * e]);
                  o[8 * h + 2 * e + 1] = fmaf(a, __uint_as_float(vw[e] & 0xFFFF0000u), o[8 * h + 2 * e + 1]);
                }
            }
          }
          if (live) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (16 * i + 8 * h < D) {
                if (kDirect) {
                  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * D + 16 * i + 8 * h) =
                      make_uint4(pack_bf16(o[8 * h], o[8 * h + 1]), pack_bf16(o[8 * h + 2], o[8 * h + 3]),
                                 pack_bf16(o[8 * h + 4], o[8 * h + 5]), pack_bf16(o[8 * h + 6], o[8 * h + 7]));
                } else {
                  float4* d = reinterpret_cast<float4*>(p.part_o + part * D + 16 * i + 8 * h);
                  d[0] = make_float4(o[8 * h], o[8 * h + 1], o[8 * h + 2], o[8 * h + 3]);
                  d[1] = make_float4(o[8 * h + 4], o[8 * h + 5], o[8 * h + 6], o[8 * h + 7]);
                }
              }
          }
        }
        if (live) {
          if (!kDirect)
            p.part_lse[part] = lse2;
          else if (p.lse)
            p.lse[row] = lse2 * kLn2;
        }
      }
      tc_fence_before();
      if (!x.two) mbar_arrive(b.ml_empty);
    }
    if (more) {
      fill_q<DH>(p, next, q_tile, tid);
      if (kDirect) ask_own(p, next);
    }
  }
}

template <int DH, bool kDirect, bool kOne>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ TcParams p) {
  using L = Smem<DH>;
  extern __shared__ uint8_t raw[];
  const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* gbase = raw + (smem - smem_u32(raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Bars b;
  uint32_t at = smem + L::BAR;
  auto take = [&](int n) { const uint32_t r = at; at += 8 * n; return r; };
  b.kfull = take(L::NK); b.kempty = take(L::NK); b.vfull = take(L::NV); b.vempty = take(L::NV);
  b.qfull = take(2); b.sfull = take(2); b.pfull = take(4); b.odone = take(2);
  b.ml_full = take(1); b.ml_empty = take(1); b.qempty = take(2); b.drain = take(1);
  constexpr bool kAhead = kQAhead<DH, kOne>;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::BAR + 248);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::BAR + 252);
  static_assert((2 * L::NK + 2 * L::NV + 15) * 8 <= 248, "barriers");
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::NK; ++i) { mbar_init(b.kfull + 8 * i, 1); mbar_init(b.kempty + 8 * i, 1); }
    for (int i = 0; i < L::NV; ++i) { mbar_init(b.vfull + 8 * i, 1); mbar_init(b.vempty + 8 * i, 1); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(b.qfull + 8 * t, kAhead ? 32 : 128);
      mbar_init(b.qempty + 8 * t, kDirect ? 9 : 1);
      mbar_init(b.sfull + 8 * t, 1);
      mbar_init(b.pfull + 16 * t, 4);
      mbar_init(b.pfull + 16 * t + 8, 4);
      mbar_init(b.odone + 8 * t, 1);
    }
    mbar_init(b.ml_full, 128);
    mbar_init(b.ml_empty, 128);
    mbar_init(b.drain, 1);
    mbar_fence_init();
  }
  if (warp == 11) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  cudaTriggerProgrammaticLaunchCompletion();   // the merge kernel's own part may start where SMs fall idle
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    if (warp == 8 && lane == 0) load_steps<DH>(p.a, &p.kmap, smem + L::K, L::NK, b.kfull, b.kempty, abort_flag);
    if (warp == 9 && lane == 0) load_steps<DH>(p.a, &p.vmap, smem + L::V, L::NV, b.vfull, b.vempty, abort_flag);
    if (warp == 10) issue_mmas<DH, kOne>(p, tmem, smem, b, lane, abort_flag);
    if (kAhead && warp == 11) load_q<DH, kDirect, kOne>(p.a, smem, b, lane, abort_flag);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_tile<DH, kDirect, kOne>(p, warp >> 2, tmem, smem, reinterpret_cast<float*>(gbase + L::ML), b, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.a.status, STATUS_KERNEL_TIMEOUT);
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// [tokens][key heads][d_head] with the caller's strides; boxes of 128 tokens x 64 columns of one
// head, columns past d_head and tokens past the end read as zeros.
tr_status encode_map(CUtensorMap* map, const void* base, const AttnParams& p) {
  auto encode = get_encode();
  if (!encode) return fail(TR_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int64_t row = p.d.d_head;
  const int tokens = p.req[p.R].p0;                        // (some request has a prefix, or no unit would be there)
  // a dimension of one entry may come with any stride: it is never multiplied
  const int64_t hs = p.d.n_kv_head > 1 ? p.d.prefix_head : row, ts = tokens > 1 ? p.d.prefix_token : row;
  cuuint64_t gdim[3] = {(cuuint64_t)row, (cuuint64_t)p.d.n_kv_head, (cuuint64_t)tokens};
  cuuint64_t gstride[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2};
  cuuint32_t box[3] = {64, 1, 128};
  cuuint32_t estride[3] = {1, 1, 1};
  CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estride,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TR_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return TR_OK;
}

template <int DH, bool kDirect, bool kOne>
tr_status launch(const TcParams& p, int sms, cudaStream_t st) {
  TR_TRY(ensure_smem_attr((const void*)prefix_kernel<DH, kDirect, kOne>, Smem<DH>::BYTES));
  prefix_kernel<DH, kDirect, kOne><<<std::min(p.a.n_units, sms), kThreads, Smem<DH>::BYTES, st>>>(p);
  TR_LAUNCH_CHECK("prefix_kernel");
  return TR_OK;
}

}  // namespace

tr_status launch_prefix_tc(const AttnParams& a, bool direct, cudaStream_t st) {
  TcParams p;
  memset(&p, 0, sizeof p);
  p.a = a;
  TR_TRY(encode_map(&p.kmap, a.k_prefix, a));
  TR_TRY(encode_map(&p.vmap, a.v_prefix, a));
  int sms = 0;
  TR_TRY(sm_count(&sms));
  if (a.d.d_head <= 64) return direct ? launch<64, true, false>(p, sms, st) : launch<64, false, false>(p, sms, st);
  bool one = true;
  for (int r = 0; r < a.R; ++r) one = one && request_rows(a, r) / a.d.n_kv_head <= kM;
  if (one) return direct ? launch<128, true, true>(p, sms, st) : launch<128, false, true>(p, sms, st);
  return direct ? launch<128, true, false>(p, sms, st) : launch<128, false, false>(p, sms, st);
}

}  // namespace attn
}  // namespace tr

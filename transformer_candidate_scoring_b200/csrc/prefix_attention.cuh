// Shared by the kernels of tr_prefix_attention: the call's parameters, and how the work over a
// request's prefix is cut into units and its partial results are stored.
#pragma once

#include "common.cuh"

namespace tr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxDHead = 128;
// Query rows of a unit and keys of a step: of the tensor-core kernel (two tiles of 128 rows), and
// of the fp32 one, whose units are 64 rows, or 16 where no key head has more than 32.
constexpr int kUnitRows = 256, kStepKeys = 128;
constexpr int kStepKeysF32 = 64;
// What a unit costs beside its keys (Q, the first scores, the result), in steps.  (18 requests of 0 to 5990
// tokens, 4 sequences each, 32 heads of 128 on 8: with 3, 5 and 8 steps 47, 45 and 46 us.)
constexpr int kUnitSteps = 5;

// The prefix part of one request: rows = sequences x query tokens x heads of a key head.  A unit
// is up to `unit_rows` of them of one key head over `chunk` steps of keys; a prefix of several chunks
// gives each row several partial results.
//
// Where no key head has more rows than a unit (each key is read by one CTA), the cut may be by runs
// instead (`run` > 0): the steps of all requests stand in one line, each request's behind kUnitSteps places
// without keys, and a team of n_kv_head CTAs, one per key head, takes `run` places of it; a unit is what of a
// run belongs to one request.  However the prefixes' lengths differ, every CTA has the same share.

// n / d for 0 <= n < 2^31 as a multiplication: (mulhi(n, mul) + n) >> shift, after Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication".
struct FastDiv {
  uint32_t mul = 1, shift = 0;
};
inline FastDiv fast_div_by(uint32_t d) {       // 1 <= d < 2^31
  FastDiv f;
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((1ull << f.shift) - d) << 32) / d + 1);
  return f;
}
__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
  return (int)((__umulhi((uint32_t)n, f.mul) + (uint32_t)n) >> f.shift);
}

constexpr int kNoHalves = 0x7FFFFFFF;

struct RequestPlan {
  int first_unit;      // units (with runs: places) of request r: first_unit[r] .. first_unit[r+1]-1
  int n_split;         // partial results per row, with runs at most (0: no prefix or no sequences)
  int chunk;           // steps per chunk; with runs, of the prefix
  int p0, p1;          // prefix tokens
  int s0, s1;          // sequences
  int64_t part;        // the request's first partial result
  int n_m;             // units of rows per key head and chunk
  FastDiv div_m, div_split;
};

struct AttnParams {
  const void *q, *k_suffix, *v_suffix, *k_prefix, *v_prefix;
  const int32_t* suffix_len;
  void* out;
  float* lse;
  int* status;
  tr_attn_desc d;
  int R, n_units;      // (with runs, the CTAs)
  bool simt;           // no prefix kernel: the kernel of the own keys reads the prefixes too
  int halves;          // from this unit on, each is two of half the rows (kNoHalves: none)
  int run;             // steps per CTA, 0: units of `chunk` steps
  int64_t n_rows;      // query rows of all requests: n * L_t * n_head
  FastDiv div_g, div_lt;   // by n_head / n_kv_head, by L_t
  FastDiv div_run, div_kv, div_h;   // by run, n_kv_head, n_head
  int group;           // n_head / n_kv_head
  // partial result i of row `row` of request r (its rows counted from 0, head fastest) is
  // part_o[(part + i * rows of r + row) * d_head ..] and part_lse[the same] (times log2 e)
  float *part_o, *part_lse;
  RequestPlan req[TR_MAX_REQUESTS + 1];
};

__host__ __device__ inline int64_t request_rows(const AttnParams& p, int r) {
  return (int64_t)(p.req[r].s1 - p.req[r].s0) * p.d.L_t * p.d.n_head;
}

// Partial results of a row of request q.
__device__ __forceinline__ int results_of(const AttnParams& p, const RequestPlan& q) {
  if (p.run == 0 || q.n_split == 0) return q.n_split;
  return fast_div(q.first_unit + kUnitSteps + q.chunk - 1, p.div_run) - fast_div(q.first_unit, p.div_run) + 1;
}

struct Unit {
  int r, hk, m0, rows, split;
  int tok, keys;       // first key token, keys of this chunk
  int steps;
  bool two;            // tensor-core kernel: the two tiles hold different rows
  __device__ int jobs(int t) const { return two ? steps : (steps + 1 - t) / 2; }
  __device__ int step_of(int t, int k) const { return two ? k : 2 * k + t; }   // step of tile t's k-th job
};

__device__ __forceinline__ Unit unit_at(const AttnParams& p, int u, int unit_rows, int step_keys) {
  const bool halved = u >= p.halves;
  int half = 0;
  if (halved) {
    half = (u - p.halves) & 1;
    u = p.halves + ((u - p.halves) >> 1);
    unit_rows /= 2;
  }
  int lo = 0, hi = p.R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.req[mid].first_unit <= u) lo = mid; else hi = mid - 1;
  }
  const RequestPlan& q = p.req[lo];
  const int m_all = (q.s1 - q.s0) * p.d.L_t * p.group;
  const int i = u - q.first_unit;
  Unit x;
  x.r = lo;
  if (p.run > 0) {
    const int team = fast_div(blockIdx.x, p.div_kv);
    x.hk = blockIdx.x - team * p.d.n_kv_head;
    x.m0 = 0;
    x.split = team - fast_div(q.first_unit, p.div_run);
    const int step = max(i - kUnitSteps, 0);
    x.tok = q.p0 + step * step_keys;
    x.steps = max(min(q.chunk, (team + 1) * p.run - q.first_unit - kUnitSteps) - step, 0);
  } else {
    const int im = fast_div(i, q.div_m);
    x.m0 = (i - im * q.n_m) * (unit_rows << halved) + half * unit_rows;      // units that share keys are neighbours
    x.hk = fast_div(im, q.div_split);
    x.split = im - x.hk * q.n_split;
    x.tok = q.p0 + x.split * q.chunk * step_keys;
    x.steps = q.chunk;
  }
  x.rows = min(unit_rows, m_all - x.m0);
  x.two = !halved && x.rows > unit_rows / 2;
  x.keys = min(x.steps * step_keys, q.p1 - x.tok);         // (none where a run ends before a request's first key)
  x.steps = (x.keys + step_keys - 1) / step_keys;
  return x;
}

// The units of this CTA: for (u = first_of(p); u < end_of(p); u = after(p, u, the unit)).
__device__ __forceinline__ int first_of(const AttnParams& p) { return p.run > 0 ? fast_div(blockIdx.x, p.div_kv) * p.run : blockIdx.x; }
__device__ __forceinline__ int end_of(const AttnParams& p) {
  return p.run > 0 ? min((fast_div(blockIdx.x, p.div_kv) + 1) * p.run, p.req[p.R].first_unit) : p.n_units;
}
__device__ __forceinline__ int after(const AttnParams& p, int u, const Unit& x) {
  if (p.run == 0) return u + gridDim.x;
  const RequestPlan& q = p.req[x.r];          // the request's end or the run's, whichever is first
  return min(q.first_unit + kUnitSteps + q.chunk, (x.split + fast_div(q.first_unit, p.div_run) + 1) * p.run);
}

// Suffix keys that query token t of sequence s sees; a length outside the buffer is clamped.
__device__ __forceinline__ int visible_suffix(const AttnParams& p, int64_t s, int t) {
  if (p.d.suffix_cap == 0) return 0;
  int len = p.suffix_len[s];
  if (len < 0 || len > p.d.suffix_cap) {
    atomicOr(p.status, STATUS_KEY_RANGE);
    len = min(max(len, 0), p.d.suffix_cap);
  }
  return p.d.causal ? max(0, len - (p.d.L_t - 1 - t)) : len;
}

// Launches the tensor-core kernel over every unit of the plan (bf16).  With `direct`, every row
// has exactly one partial result and suffix buffers hold at most one token: the kernel adds
// the row's own key and writes out and lse instead.
constexpr int kDirectSuffix = 1;
tr_status launch_prefix_tc(const AttnParams& p, bool direct, cudaStream_t st);
// The fp32 kernel over every unit (of 64 or 16 rows).
tr_status launch_prefix_f32(const AttnParams& p, int unit_rows, cudaStream_t st);

}  // namespace attn
}  // namespace tr

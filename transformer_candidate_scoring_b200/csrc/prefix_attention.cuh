// Shared by the kernels of tr_prefix_attention: the call's parameters, and how the work over a
// request's prefix is cut into units and its partial results are stored.
#pragma once

#include "common.cuh"

namespace tr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxDHead = 128;
constexpr int kStepKeys = 128;      // keys of one step of the tensor-core kernel
constexpr int kUnitRows = 256;      // query rows of a unit (two tiles of 128)

// The prefix part of one request: rows = sequences x query tokens x heads of a key head.  A unit
// is up to 256 rows of one key head over `chunk` steps of 128 keys; a prefix of several chunks
// gives each row several partial results.
struct RequestPlan {
  int first_unit;      // units of request r: first_unit[r] .. first_unit[r+1]-1
  int n_split;         // chunks of the prefix (0: no prefix or no sequences)
  int chunk;           // steps per chunk
  int p0, p1;          // prefix tokens
  int s0, s1;          // sequences
  int64_t part;        // the request's first partial result
};

struct AttnParams {
  const void *q, *k_suffix, *v_suffix, *k_prefix, *v_prefix;
  const int32_t* suffix_len;
  void* out;
  float* lse;
  int* status;
  tr_attn_desc d;
  int R, n_units;
  int64_t n_rows;      // query rows of all requests: n * L_t * n_head
  // partial result i of row `row` of request r (its rows counted from 0, head fastest) is
  // part_o[(part + i * rows of r + row) * d_head ..] and part_lse[the same] (times log2 e)
  float *part_o, *part_lse;
  RequestPlan req[TR_MAX_REQUESTS + 1];
};

__host__ __device__ inline int64_t request_rows(const AttnParams& p, int r) {
  return (int64_t)(p.req[r].s1 - p.req[r].s0) * p.d.L_t * p.d.n_head;
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
// has exactly one partial result and suffix buffers hold at most kDirectSuffix tokens: the kernel adds
// the row's own keys and writes out and lse instead.
constexpr int kDirectSuffix = 4;
tr_status launch_prefix_tc(const AttnParams& p, bool direct, cudaStream_t st);

}  // namespace attn
}  // namespace tr

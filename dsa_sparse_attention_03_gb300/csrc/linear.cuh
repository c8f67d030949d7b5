// Launchers of the linear attention kernels (linear.cu, linear_step.cu), used by api.cu.
#pragma once

#include "common.cuh"
#include "dsa_linear.h"

namespace dsa {

struct LinearArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* log_decay;
  const int32_t* row_offsets;
  const int32_t* state_idx;
  const float* state_in;    // or null
  float* state_out;         // or null
  uint16_t* out;
  float* seg_state;         // workspace [split_segs, H, D_k, D_v]: each segment's end state
  uint32_t* status;
  int64_t q_stride, k_stride, v_stride;
  uint64_t wait_ns;
  int R, B, H, D_k, D_v, n_states;
  int seg_len;              // tokens of a segment (a multiple of 128)
  int segs, split_segs;     // segments of the call, at most, and those of split requests
  float scale;
  int test_no_load;         // test hook: arm the first chunk, issue no copy
  int status_known;         // the status word is this value whatever the kernel finds (-1: it is cleared before, and raised)
};

// Tokens of a segment: a request with more is split, its segments run on
// different SMs (INT32_MAX - 127, a multiple of 128: no request is split).
int linear_seg_len(const dsa_linear_problem& p);
// Segments of the call, at most.
int64_t linear_segs(const dsa_linear_problem& p, int seg_len);
// Those of split requests: one of n > seg_len tokens has less than 2 n / seg_len.
inline int64_t linear_split_segs(const dsa_linear_problem& p, int seg_len) { return 2 * (int64_t)p.R / seg_len; }

cudaError_t launch_linear(const LinearArgs& a, bool f16, bool split, cudaStream_t st);
cudaError_t launch_linear_step(const LinearArgs& a, bool f16, cudaStream_t st);

// The place of request b's state: its index, or -1 where the request is to be
// skipped (unused, out of range, or the same place as an earlier request).  The
// whole block calls it with the same b; `scratch` is a shared int.
static __device__ inline int state_place(const LinearArgs& a, int b, int* scratch, bool report) {
  if (!a.state_idx) {
    const int ok = b < a.n_states;
    if (!ok && report && threadIdx.x == 0 && a.status_known < 0) {
      pdl_wait();
      raise_status(a.status, DSA_DEVICE_BAD_INDEX);
    }
    return ok ? b : -1;
  }
  const int at = a.state_idx[b];
  if (threadIdx.x == 0) *scratch = 0;
  __syncthreads();
  if (at < 0) return -1;
  bool twice = at >= a.n_states;
  for (int i = threadIdx.x; i < b; i += blockDim.x) twice |= a.state_idx[i] == at;
  if (twice) *scratch = 1;
  __syncthreads();
  if (*scratch) {
    if (report && threadIdx.x == 0) {
      pdl_wait();
      raise_status(a.status, DSA_DEVICE_BAD_INDEX);
    }
    return -1;
  }
  return at;
}

// log2 of a head's decay, at most 0 and bounded below (2^-300 is 0 in fp32), so
// that a power of it is never 0 * inf.
static __device__ __forceinline__ float log2_decay(float log_decay) {
  const float x = log_decay * 1.44269504088896341f;
  return x > 0.f ? 0.f : (x < -300.f ? -300.f : x);
}

}  // namespace dsa

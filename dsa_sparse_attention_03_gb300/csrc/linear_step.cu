// Linear attention, one token of each request (dsa_linear_step).
//
//   S' = lambda S + k^T v,   o = scale * q S'
//
// Reading and writing the states is the traffic (8 bytes per element against
// two multiply-adds), so the kernel is one pass over each state: a CTA of 256
// threads per request and head, a thread holding 4 adjacent columns of every
// (256 / (D_v / 4))-th row, with all its loads issued before the first use.  The
// output's partial sums over rows meet in shared memory, in a fixed order.
// Measured: 96 requests of 64 heads of 128 x 128, 117 to 119 us for 812 MB, 6.8 to 6.9
// TB/s (the copy rate); one request 2.9 us in a graph.
#include "linear.cuh"
#include "tc.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

template <int DK, int DV, bool F16>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const LinearArgs a) {
  constexpr int C4 = DV / 4;               // threads along a row
  constexpr int RG = kThreads / C4;        // rows at a time
  constexpr int N = DK / RG;               // rows of a thread
  __shared__ float qs[DK], ks[DK];
  __shared__ float4 part[kThreads];
  __shared__ int twice;
  const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
  const int tid = threadIdx.x, c = tid % C4, r = tid / C4;
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0 && a.status_known >= 0) *a.status = (uint32_t)a.status_known;
  const int at = state_place(a, b, &twice, h == 0);
  if (at < 0) return;
  const int64_t base = ((int64_t)at * a.H + h) * DK * DV;
  float4 s[N];
  if (a.state_in) {
    const float4* in = reinterpret_cast<const float4*>(a.state_in + base);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = in[(i * RG + r) * C4 + c];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (tid < DK) {
    qs[tid] = to_float<F16>(a.q[b * a.q_stride + h * DK + tid]);
  } else if (tid - DK < DK) {
    ks[tid - DK] = to_float<F16>(a.k[b * a.k_stride + h * DK + tid - DK]);
  }
  const uint2 vw = *reinterpret_cast<const uint2*>(a.v + b * a.v_stride + h * DV + 4 * c);
  const float4 v = make_float4(to_float<F16>((uint16_t)vw.x), to_float<F16>((uint16_t)(vw.x >> 16)),
                               to_float<F16>((uint16_t)vw.y), to_float<F16>((uint16_t)(vw.y >> 16)));
  const float lambda = exp2f(log2_decay(a.log_decay[h]));
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float4* dst = reinterpret_cast<float4*>(a.state_out + base);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = ks[i * RG + r], q = qs[i * RG + r];
    float4 x = s[i];
    x.x = fmaf(k, v.x, lambda * x.x);
    x.y = fmaf(k, v.y, lambda * x.y);
    x.z = fmaf(k, v.z, lambda * x.z);
    x.w = fmaf(k, v.w, lambda * x.w);
    dst[(i * RG + r) * C4 + c] = x;
    o.x = fmaf(q, x.x, o.x);
    o.y = fmaf(q, x.y, o.y);
    o.z = fmaf(q, x.z, o.z);
    o.w = fmaf(q, x.w, o.w);
  }
  part[tid] = o;
  __syncthreads();
  if (tid < C4) {
#pragma unroll
    for (int i = 1; i < RG; ++i) {
      const float4 p = part[i * C4 + tid];
      o.x += p.x; o.y += p.y; o.z += p.z; o.w += p.w;
    }
    *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + h) * DV + 4 * tid) =
        make_uint2(pack16<F16>(o.x * a.scale, o.y * a.scale), pack16<F16>(o.z * a.scale, o.w * a.scale));
  }
}

template <int DK, int DV>
cudaError_t launch_one(const LinearArgs& a, bool f16, cudaStream_t st) {
  const unsigned grid = (unsigned)a.B * (unsigned)a.H;
  return f16 ? launch_pdl(linear_step_kernel<DK, DV, true>, dim3(grid), dim3(kThreads), 0, st, a)
             : launch_pdl(linear_step_kernel<DK, DV, false>, dim3(grid), dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_linear_step(const LinearArgs& a, bool f16, cudaStream_t st) {
  if (a.D_k == 64) return a.D_v == 64 ? launch_one<64, 64>(a, f16, st) : launch_one<64, 128>(a, f16, st);
  return a.D_v == 64 ? launch_one<128, 64>(a, f16, st) : launch_one<128, 128>(a, f16, st);
}

}  // namespace dsa

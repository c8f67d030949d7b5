// Norms of queries and keys for each head and the position rotation (dsa_qk_norm_rope).
//
//   y = x w / sqrt(mean x^2 + eps), then pairs of columns turned by position * inv_freq.
//
// Every element is read once and written once (4 bytes against about ten operations), so
// what bounds the kernel is HBM, or for few rows latency.  A CTA takes one row and some of
// its heads: the row's angles are the same for all heads, so its cos and sin are computed
// once, by as many threads as there are frequencies, while the heads' loads are under way.  A
// head is held by 8 to 32 lanes with both columns of a pair in one lane (rope.cuh), so the
// rotation needs no exchange and the norm three to five shuffles.
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const TurnArgs t) {
  constexpr int L = kHeadLanes<D>, S = kThreads / L, U = 4;   // lanes to a head, heads at a time, in flight
  __shared__ float2 cs[128];
  const int tid = threadIdx.x, j = tid % L, slot = tid / L;
  const int row = blockIdx.x / t.chunks, chunk = blockIdx.x - row * t.chunks;
  const int heads = t.H_q + t.H_kv;
  const int h0 = (int)((int64_t)heads * chunk / t.chunks), h1 = (int)((int64_t)heads * (chunk + 1) / t.chunks);
  const HeadLane l = head_lane<D>(t, j);
  pdl_wait();
  pdl_trigger();
  const int pos = t.positions[row];
  float2 c[4];
  for (int base = h0; base < h1; base += U * S) {
    uint2 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = base + u * S + slot;
      const uint16_t* p = x < t.H_q ? t.q + row * t.q_stride + (int64_t)x * D
                                    : t.k + row * t.k_stride + (int64_t)(x - t.H_q) * D;
      v[u][0] = x < h1 ? load4(p, l.a) : make_uint2(0, 0);
      v[u][1] = x < h1 ? load4(p, l.b) : make_uint2(0, 0);
    }
    if (base == h0) {
      if (pos < 0) return;
      if (tid < t.rot / 2) cs[tid] = turn(turn_fraction(t.inv_freq[tid]), pos);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = l.f >= 0 ? cs[l.f + i] : make_float2(1.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * S >= h1) break;   // (the same for a whole CTA)
      const int x = base + u * S + slot;
      const bool is_q = x < t.H_q;
      float y[8];
      unpack4<F16>(v[u][0], y);
      unpack4<F16>(v[u][1], y + 4);
      turn_head<D, F16, false>(t, is_q ? t.q_weight : t.k_weight, l, c, y, nullptr);
      if (x < h1 && l.a >= 0) {
        uint16_t* p = is_q ? t.q_out + row * t.q_out_stride + (int64_t)x * D
                           : t.k_out + row * t.k_out_stride + (int64_t)(x - t.H_q) * D;
        *reinterpret_cast<uint2*>(p + l.a) = make_uint2(pack16<F16>(y[0], y[1]), pack16<F16>(y[2], y[3]));
        *reinterpret_cast<uint2*>(p + l.b) = make_uint2(pack16<F16>(y[4], y[5]), pack16<F16>(y[6], y[7]));
      }
    }
  }
}

template <int D>
cudaError_t launch_width(TurnArgs t, bool f16, cudaStream_t st) {
  // CTAs to a row: as many as keep four heads in flight a thread; few rows are spread
  // further, one head a thread, to fill the GPU.
  constexpr int S = kThreads / kHeadLanes<D>;
  const int heads = t.H_q + t.H_kv;
  const int most = (heads + S - 1) / S, least = (heads + 4 * S - 1) / (4 * S);
  t.chunks = least;
  while (t.chunks < most && (int64_t)t.R * t.chunks < 608) ++t.chunks;
  const dim3 grid((unsigned)((int64_t)t.R * t.chunks));
  return f16 ? launch_pdl(qk_norm_rope_kernel<D, true>, grid, dim3(kThreads), 0, st, t)
             : launch_pdl(qk_norm_rope_kernel<D, false>, grid, dim3(kThreads), 0, st, t);
}

}  // namespace

cudaError_t launch_qk_norm_rope(TurnArgs a, int D, bool f16, cudaStream_t st) {
  if (a.R == 0 || a.H_q + a.H_kv == 0) return cudaSuccess;
  switch (D) {
    case 64: return launch_width<64>(a, f16, st);
    case 128: return launch_width<128>(a, f16, st);
    case 192: return launch_width<192>(a, f16, st);
    default: return launch_width<256>(a, f16, st);
  }
}

}  // namespace dsa

// Norms of queries and keys for each head and the position rotation (dsa_qk_norm_rope).
//
//   y = x w / sqrt(mean x^2 + eps), then pairs of columns turned by position * inv_freq.
//
// Every element is read once and written once (4 bytes against about ten operations), so
// what bounds the kernel is HBM, or for few rows latency.  A CTA takes up to eight rows, whose
// angles' cos and sin its threads work out first, one each (by every warp for itself they were
// 40% of its instructions), and its warps runs of a row's heads, with the norm's weights in registers.  A
// head is held by 8 to 32 lanes with both columns of a pair in one lane (rope.cuh), so the
// rotation needs no exchange and the norm three to five shuffles.
//
// Measured: 9601 rows of 64 + 8 heads of 128 out of a fused projection 62.5 us, 5.7 TB/s (83% of the
// copy rate; 67% of the issue slots are taken); one row 2.3 us in a graph.
#include "rope.cuh"

namespace dsa {
namespace {

template <int D, bool F16>
__global__ void __launch_bounds__(kTurnThreads) qk_norm_rope_kernel(const __grid_constant__ TurnArgs t) {
  __shared__ RowTurns cs;
  const int lane = threadIdx.x & 31, runs = t.q_runs + t.k_runs;
  int row0, u0, u1;
  cta_units(t, runs, row0, u0, u1);
  pdl_wait();
  pdl_trigger();
  row_turns(t, cs, row0);
  __syncthreads();
  for (int u = u0 + (threadIdx.x >> 5); u < u1; u += kTurnThreads / 32) {
    const int c = u >> t.rows_log2, i = u - (c << t.rows_log2), row = row0 + i;
    if (row >= t.R || t.positions[row] < 0) continue;
    const bool is_q = c < t.q_runs;
    int h0, h1;
    run_heads(t, is_q ? t.H_q : t.H_kv, is_q ? c : c - t.q_runs, h0, h1);
    turn_row<D, F16>(t, is_q ? t.q_weight : t.k_weight, cs[i], is_q ? t.q + row * t.q_stride : t.k + row * t.k_stride,
                     is_q ? t.q_out + row * t.q_out_stride : t.k_out + row * t.k_out_stride, h0, h1, lane);
  }
}

template <int D>
cudaError_t launch_width(TurnArgs t, bool f16, cudaStream_t st) {
  deal_heads(t, 32 / kHeadLanes<D>, 8, t.H_kv, 0);
  const dim3 grid((unsigned)((t.R + (1 << t.rows_log2) - 1) >> t.rows_log2), (unsigned)t.split);
  return f16 ? launch_pdl(qk_norm_rope_kernel<D, true>, grid, dim3(kTurnThreads), 0, st, t)
             : launch_pdl(qk_norm_rope_kernel<D, false>, grid, dim3(kTurnThreads), 0, st, t);
}

}  // namespace

// Many rows: up to eight to a CTA, whose angles its threads work out together, and `most` heads to a
// run.  Few rows: a row's heads over several CTAs, as few to a warp as fit it, as long as that
// leaves every CTA's warps a run.
void deal_heads(TurnArgs& t, int at_once, int most, int H_k, int H_v) {
  int runs = 0;
  auto cut = [&](int log2) {
    const int heads = 1 << log2;
    t.run_log2 = log2;
    t.q_runs = (t.H_q + heads - 1) / heads;
    t.k_runs = (H_k + heads - 1) / heads;
    t.v_runs = (H_v + heads - 1) / heads;
    runs = t.q_runs + t.k_runs + t.v_runs;
  };
  int log2 = 0, least = 0;
  while (1 << log2 < most || 1 << log2 < at_once) ++log2;
  while (1 << least < at_once) ++least;
  cut(log2);
  while (log2 > least && (int64_t)t.R * runs < 9728) cut(--log2);
  t.rows_log2 = t.R >= 8 * 608 ? 3 : t.R >= 4 * 608 ? 2 : t.R >= 2 * 608 ? 1 : 0;
  t.split = 1;
  if (t.rows_log2 == 0)
    while (t.split < (runs + 7) / 8 && (int64_t)t.R * (t.split + 1) <= 1216) ++t.split;
  t.units = ((runs << t.rows_log2) + t.split - 1) / t.split;
}

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

// How the roles of the linear attention kernel share buffers (linear.cu): which
// buffer a chunk uses and which phase of a barrier stands for that use.  The kernel
// and a model of its waits that runs on the host (tests/c/linear_protocol_check.cc) take
// them from here.  Plain C++: no CUDA headers needed.
//
// A wait names a phase by its parity alone.  It is sound only where the barrier's next
// phase cannot complete before the waiter went on: a waiter that is lapped sees the
// parity it started from and waits for a phase that may never come.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define DSA_PIPE_FN __host__ __device__ __forceinline__ static constexpr
#else
#define DSA_PIPE_FN static constexpr
#endif

namespace dsa {

// STATE: the launch that computes the segments' end states alone (no Q, no output).
template <bool STATE>
struct ChunkPipe {
  static constexpr int stages = STATE ? 3 : 2;     // K and V (and Q) tiles in shared memory
  static constexpr int dh_bufs = STATE ? 2 : 1;    // accumulators of dH
  static constexpr int v_bufs = STATE ? 4 : 2;     // buffers of the decayed V: quarter g of a chunk uses g % v_bufs
  // Arrivals that give a stage's K and V back: the last read of the dH products, and
  // where there are outputs that of P V.  One barrier for each stage, whose next phase
  // needs the producer's own load.
  static constexpr int kv_releases = STATE ? 1 : 2;
  // Barriers for the output tiles that wait for their store, one for each stage whose Q
  // tile they lie in: the next tile there needs the stage that the store gives back.
  static constexpr int o_tiles = STATE ? 0 : stages;
  // Slots of the scales of the decayed V's columns (fp16).  Chunk c's are written once the
  // first product of chunk c - 1 is through, which waited for the state warps to be through
  // with chunk c - 1 - dh_bufs: they may still read those of the dh_bufs chunks before c.
  static constexpr int scale_slots = STATE ? 4 : 2;

  DSA_PIPE_FN int stage(int c) { return (int)((unsigned)c % stages); }
  DSA_PIPE_FN uint32_t stage_phase(int c) { return (unsigned)c / stages & 1u; }
  DSA_PIPE_FN int dh(int c) { return (int)((unsigned)c % dh_bufs); }
  DSA_PIPE_FN uint32_t dh_phase(int c) { return (unsigned)c / dh_bufs & 1u; }
  DSA_PIPE_FN int scale(int c) { return (int)((unsigned)c % scale_slots); }
  DSA_PIPE_FN int v(int g) { return (int)((unsigned)g % v_bufs); }
  DSA_PIPE_FN bool v_first(int c, int g) { return c == 0 && g < v_bufs; }   // the buffer's first use
  // Phase of use (c, g), and of the buffer's use before it.
  DSA_PIPE_FN uint32_t v_phase(int c, int g) { return ((unsigned)c * (4 / v_bufs) + (unsigned)g / v_bufs) & 1u; }
  DSA_PIPE_FN uint32_t v_phase_before(int c, int g) { return v_phase(c, g) ^ 1u; }
};

}  // namespace dsa

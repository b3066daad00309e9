// Arguments of lt_attn_prompt's kernels and the map from a launch's tiles to
// the sequences, read on the device.
#pragma once

#include "attn_common.cuh"

namespace lt {

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  long long sq, sk, sv, so;  // elements between tokens
  const int32_t* q_off;
  const int32_t* kv_off;
  int n_seqs, n_q, n_kv, heads, kv_heads, group;
  float scale;
  int* status;
};

// Tile `t` of the packed batch in units of `tok` tokens: its sequence and its
// tile within that (from the last one down: the longest rows start first).
// Run by a whole warp; false when there is no such tile.
struct PromptTile {
  int q0, lq, k0, lk, tile;
};
__device__ __forceinline__ bool prompt_tile(const PromptArgs& a, int t, int tok, PromptTile& out) {
  const int lane = threadIdx.x & 31;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int2 r = {0, 0};
    if (s < a.n_seqs) r = off_range(a.q_off, s, a.n_q, a.status);
    const int n = cdiv(r.y - r.x, tok);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned here = __ballot_sync(0xffffffffu, incl > t);
    if (here) {
      const int w = __ffs(here) - 1;
      int2 kr = {0, 0};
      if (lane == w) kr = off_range(a.kv_off, s, a.n_kv, a.status);
      out.q0 = __shfl_sync(0xffffffffu, r.x, w);
      out.lq = __shfl_sync(0xffffffffu, r.y - r.x, w);
      out.k0 = __shfl_sync(0xffffffffu, kr.x, w);
      out.lk = __shfl_sync(0xffffffffu, kr.y - kr.x, w);
      out.tile = __shfl_sync(0xffffffffu, incl - 1 - t, w);
      return true;
    }
    t -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

}  // namespace lt

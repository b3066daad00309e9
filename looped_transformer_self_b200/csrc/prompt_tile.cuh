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
  int splits;        // key ranges of a pair of tiles, each an item of its own (bf16)
  float2* part_ml;   // partials of the ranges: [pairs * splits][256] maximum (log2 units) and sum
  int o_wide;        // output rows start on 32-byte boundaries
  float* part;       // [pairs * splits][256][head_dim] unnormalised outputs
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

// Pairs of 128-row tiles per key/value head, at most.
inline long long prompt_pairs(int n_q, int n_seqs, int group) { return n_q / (2 * (128 / group)) + (long long)n_seqs; }

// Key ranges of a pair of tiles, at most: an item for every SM.
inline int prompt_max_splits(int n_q, int n_seqs, int heads, int kv_heads) {
  const long long pairs = prompt_pairs(n_q, n_seqs, heads / kv_heads) * kv_heads;
  const int sms = attn_sm_count();
  return pairs <= 0 || pairs * 2 > sms ? 1 : (int)(sms / pairs);
}
// Key ranges taken: partials cost a write, a read and a second kernel (6 us for
// 48 pairs of 5 blocks, 16.6 us whole), a block about 1.6 us, so a range keeps
// at least 6 blocks of an average sequence's keys (32 pairs of up to 47 blocks:
// 80 us whole, 34 us in 4 ranges).
inline int prompt_splits(int n_q, int n_kv, int n_seqs, int heads, int kv_heads) {
  const long long blocks = (long long)n_kv / (n_seqs > 0 ? n_seqs : 1) / 128;
  const long long most = prompt_max_splits(n_q, n_seqs, heads, kv_heads);
  return (int)(blocks / 6 < 1 ? 1 : blocks / 6 < most ? blocks / 6 : most);
}

}  // namespace lt

// Work partition of lt_attn_prefix, shared by its kernels and its merge.
//
// A tile is (group of rows, key/value head, up to MT packed query rows); its
// keys are the group's prefix slots followed by the tail slots of the tile's
// own rows, in blocks of BN.  The (tile, block) units of all tiles are
// laid end to end and CTA c of n takes units [c U / n, (c + 1) U / n),
// so every CTA streams the same number of blocks whatever the lengths are.
// Lengths are read on the device: a captured call follows them.
//
// CTA c's part of tile t goes to partial slot c + t: along the units either c
// or t grows by one from a part to the next, so the slots are distinct and at
// most grid + tiles of them are used.
#pragma once

#include "attn_common.cuh"

namespace lt {


struct PrefixArgs {
  const void* q;
  const void* cache;  // [n_slots][2][kv_heads * hd]
  void* o;
  long long sq, so;
  const int32_t* row_off;     // [n_groups + 1]
  const int32_t* prefix;      // slots
  const int32_t* prefix_off;  // [n_groups + 1]
  const int32_t* tail;        // slots
  const int32_t* tail_off;    // [n_rows + 1]
  int n_groups, n_rows, n_slots, n_prefix, n_tail, heads, kv_heads, group;
  float scale;
  // scratch
  long long* head;  // [0]: U
  int4* tile_tab;   // per tile: first unit (x low, y high), blocks, 0
  int4* row_tab;    // per row: tile of key/value head 0, tiles per head, first packed row, partials of a part
  float2* part_ml;  // [slots][MT]: maximum (log2 units) and sum
  float* part;      // [slots][MT][hd] unnormalised outputs
  int max_tiles;
  int* status;
};

struct PrefixGroup {
  int r0, m, p0, np;
};
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixArgs& a, int g) {
  const int2 r = off_range(a.row_off, g, a.n_rows, a.status);
  const int2 p = off_range(a.prefix_off, g, a.n_prefix, a.status);
  return {r.x, r.y - r.x, p.x, p.y - p.x};
}
// Tail entries of rows [row, row + n).
__device__ __forceinline__ int2 prefix_tail(const PrefixArgs& a, int row, int n) {
  const int x = off_range(a.tail_off, row, a.n_tail, a.status).x;
  const int y = off_range(a.tail_off, row + n - 1, a.n_tail, a.status).y;
  return {x, max(x, y)};
}
template <int BN>
__device__ __forceinline__ int prefix_blocks(int np, int nt) {
  return max(1, cdiv(np + nt, BN));
}

// Blocks of all row tiles of one group (one key/value head).
template <int BN>
__device__ __forceinline__ int prefix_group_blocks(const PrefixArgs& a, const PrefixGroup& g, int tok) {
  int n = 0;
  for (int i = 0; i < g.m; i += tok) {
    const int2 t = prefix_tail(a, g.r0 + i, min(tok, g.m - i));
    n += prefix_blocks<BN>(g.np, t.y - t.x);
  }
  return n;
}

__device__ __forceinline__ long long warp_incl_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// Units of all groups (every warp computes it alike).
template <int BN>
__device__ __forceinline__ long long prefix_total(const PrefixArgs& a, int tok) {
  const int lane = threadIdx.x & 31;
  long long n = 0;
  for (int g = lane; g < a.n_groups; g += 32) {
    const PrefixGroup pg = prefix_group(a, g);
    n += (long long)a.kv_heads * prefix_group_blocks<BN>(a, pg, tok);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

template <int BN>
struct PrefixPos {
  PrefixGroup g;
  int gi, kh, mt, nmt;   // group, key/value head, row tile, row tiles of the group
  int t;                 // tile index
  long long u0;          // first unit of the tile
  int nb;                // its blocks
  int row0, nrow;        // its rows
  int2 tail;             // its rows' tail entries
  __device__ __forceinline__ void set_tile(const PrefixArgs& a, int tok) {
    row0 = g.r0 + mt * tok;
    nrow = min(tok, g.m - mt * tok);
    tail = prefix_tail(a, row0, nrow);
    nb = prefix_blocks<BN>(g.np, tail.y - tail.x);
  }
  // The tile that holds unit u (u below the total).
  __device__ __forceinline__ void find(const PrefixArgs& a, int tok, long long u) {
    const int lane = threadIdx.x & 31;
    long long base = 0, tiles = 0;
    for (int s0 = 0; s0 < a.n_groups; s0 += 32) {
      long long units = 0, nt = 0;
      PrefixGroup pg = {0, 0, 0, 0};
      int blocks = 0;
      if (s0 + lane < a.n_groups) {
        pg = prefix_group(a, s0 + lane);
        blocks = prefix_group_blocks<BN>(a, pg, tok);
        units = (long long)a.kv_heads * blocks;
        nt = (long long)a.kv_heads * cdiv(pg.m, tok);
      }
      const long long iu = warp_incl_scan(units), it = warp_incl_scan(nt);
      const unsigned here = __ballot_sync(0xffffffffu, base + iu > u);
      if (here) {
        const int w = __ffs(here) - 1;
        gi = s0 + w;
        g.r0 = __shfl_sync(0xffffffffu, pg.r0, w);
        g.m = __shfl_sync(0xffffffffu, pg.m, w);
        g.p0 = __shfl_sync(0xffffffffu, pg.p0, w);
        g.np = __shfl_sync(0xffffffffu, pg.np, w);
        blocks = __shfl_sync(0xffffffffu, blocks, w);
        u0 = base + __shfl_sync(0xffffffffu, iu - units, w);
        t = (int)(tiles + __shfl_sync(0xffffffffu, it - nt, w));
        nmt = cdiv(g.m, tok);
        kh = (int)((u - u0) / blocks);
        u0 += (long long)kh * blocks;
        t += kh * nmt;
        mt = 0;
        set_tile(a, tok);
        while (u >= u0 + nb && mt + 1 < nmt) {
          u0 += nb;
          ++t;
          ++mt;
          set_tile(a, tok);
        }
        return;
      }
      base += __shfl_sync(0xffffffffu, iu, 31);
      tiles += __shfl_sync(0xffffffffu, it, 31);
    }
  }
  // The next tile (there is one: the caller still has units).
  __device__ __forceinline__ void next(const PrefixArgs& a, int tok) {
    u0 += nb;
    ++t;
    if (++mt == nmt) {
      mt = 0;
      if (++kh == a.kv_heads) {
        kh = 0;
        do {
          if (gi + 1 >= a.n_groups) return;
          g = prefix_group(a, ++gi);
        } while (g.m == 0);
        nmt = cdiv(g.m, tok);
      }
    }
    set_tile(a, tok);
  }
  // Entries of the tables that the merge reads, written by the CTA with the tile's first block
  // (threads `id` of n; `half`: rows of a 128-row half of the tile, 0 for tiles in one piece;
  // `two`: a part of more than one block has two partials, see TcSpan).
  __device__ __forceinline__ void publish(const PrefixArgs& a, int id, int n, int half = 0, bool two = false) const {
    if (id == 0)
      a.tile_tab[t] = make_int4((int)(unsigned)(u0 & 0xffffffffll), (int)(u0 >> 32), nb, 0);
    if (kh == 0)
      for (int i = id; i < nrow; i += n) {
        const int r = half ? i / half * 128 + i % half * a.group : i * a.group;
        a.row_tab[row0 + i] = make_int4(t, nmt, r, two ? 2 : 1);
      }
  }
};

// CTAs that get units: with fewer units than CTAs, one each (a CTA without units has no part).
__device__ __forceinline__ int prefix_ctas(long long U, int grid) { return (int)min(U, (long long)grid); }
__device__ __forceinline__ long long prefix_u0(int c, long long U, int ctas) { return c * U / ctas; }
__device__ __forceinline__ int prefix_cta_of(long long u, long long U, int ctas) {
  int c = (int)(u * ctas / U);
  while (c > 0 && prefix_u0(c, U, ctas) > u) --c;
  while (c + 1 < ctas && prefix_u0(c + 1, U, ctas) <= u) ++c;
  return c;
}

}  // namespace lt

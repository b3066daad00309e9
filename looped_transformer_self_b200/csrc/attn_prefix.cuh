// Work partition of lt_attn_prefix, shared by its kernels and its merge.
//
// A tile is (group of rows, key/value head, up to MT packed query rows); its
// keys are the group's prefix slots followed by the tail slots of the tile's
// own rows, in blocks of BN.  Where each tile can have CTAs of its own, a CTA
// takes one range of one tile (leaving a tile
// costs a CTA a start-up and a partial: 14 us of 90 at 27.7 blocks of 512 per
// CTA).  Otherwise the (tile, block) units of all tiles are laid end to end and
// CTA c of n takes units [c U / n, (c + 1) U / n).  Lengths are read on the
// device: a captured call follows them.
//
// CTA c's part of tile t goes to partial slot c + t: from a part to the next
// one of c and t grows, so the slots are distinct and at most grid + tiles of
// them are used.
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
  int4* tile_tab;   // per tile: first CTA, CTAs
  int4* row_tab;    // per row: tile of key/value head 0, tiles per head, first packed row, partials of a part
  float2* part_ml;  // [slots][MT]: maximum (log2 units) and sum
  float* part;      // [slots][MT][hd] unnormalised outputs
  int max_tiles;
  int* status;
};

// What the merge takes from the tables for one (row, head).  Entries that no CTA wrote hold whatever the
// scratch held (offsets that are not as promised, a wait that gave up), so nothing is assumed of them.
struct PrefixPlace {
  int t, r;             // tile, packed row in it
  int first, parts, two;  // first CTA, partials in all, partials of a part
};
__host__ __device__ __forceinline__ bool prefix_place(int4 row, int head, int group, int max_tiles, int mt,
                                                      PrefixPlace& p) {
  const long long t = row.x + (long long)(head / group) * row.y, r = (long long)row.z + head % group;
  p.two = row.w == 2 ? 2 : 1;
  if (t < 0 || t >= max_tiles || row.z < 0 || r >= (p.two == 2 ? mt / 2 : mt)) return false;
  p.t = (int)t;
  p.r = (int)r;
  return true;
}
__host__ __device__ __forceinline__ bool prefix_parts(int4 tile, int grid, PrefixPlace& p) {
  if (tile.x < 0 || tile.x >= grid || tile.y <= 0 || tile.y > grid - tile.x) return false;
  p.first = tile.x;
  p.parts = tile.y * p.two;
  return true;
}

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

template <int BN>
struct PrefixPos {
  PrefixGroup g;
  int gi, kh, mt, nmt;   // group, key/value head, row tile, row tiles of the group
  int t;                 // tile index
  int u0;                // first unit of the tile
  int nb;                // its blocks
  int row0, nrow;        // its rows
  int2 tail;             // its rows' tail entries
  __device__ __forceinline__ void set_tile(const PrefixArgs& a, int tok) {
    row0 = g.r0 + mt * tok;
    nrow = min(tok, g.m - mt * tok);
    tail = prefix_tail(a, row0, nrow);
    nb = prefix_blocks<BN>(g.np, tail.y - tail.x);
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
};

// floor(a b / c) of non-negative numbers; a 32-bit division where the product allows.
__device__ __forceinline__ int mul_div(int a, int b, int c) {
  const unsigned long long p = (unsigned long long)(unsigned)a * (unsigned)b;
  return p >> 32 ? (int)(p / (unsigned)c) : (int)((unsigned)p / (unsigned)c);
}
__device__ __forceinline__ int prefix_u0(int c, int U, int ctas) { return mul_div(c, U, ctas); }
__device__ __forceinline__ int prefix_cta_of(int u, int U, int ctas) {
  int c = mul_div(u, ctas, U);
  while (c > 0 && prefix_u0(c, U, ctas) > u) --c;
  while (c + 1 < ctas && prefix_u0(c + 1, U, ctas) <= u) ++c;
  return c;
}
__device__ __forceinline__ int warp_incl_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// The parts of one CTA, walked through by every warp alike.  The host bounds
// the units of as many tiles as the scratch holds by 2^30, so they are counted in
// 32 bits (the 64-bit divisions and scans of a first form took 4 us of each call).
template <int BN>
struct PrefixWalk {
  PrefixPos<BN> pos;
  int b0, n;              // the part's blocks of pos's tile
  int first_cta, n_ctas;  // the tile's CTAs
  int u, hi, U;           // units of this CTA, of all (units laid end to end)
  int ctas;               // CTAs with units
  int most;               // where the tiles have CTAs of their own: the blocks one takes at most
  bool own;

  // What a lane knows of group s0 + lane; blocks and shares are of one key/value head.
  struct Group {
    PrefixGroup g;
    int nmt, blocks, shares;
  };
  // CTAs of a tile of nb blocks that has its own.
  __device__ __forceinline__ int share(int nb) const { return cdiv(nb, most); }
  __device__ __forceinline__ void load(const PrefixArgs& a, int tok, int s0, Group& x) const {
    const int g = s0 + (threadIdx.x & 31);
    x = {{0, 0, 0, 0}, 0, 0, 0};
    if (g >= a.n_groups) return;
    x.g = prefix_group(a, g);
    x.nmt = cdiv(x.g.m, tok);
    x.blocks = prefix_group_blocks<BN>(a, x.g, tok);
  }
  __device__ __forceinline__ void set_shares(const PrefixArgs& a, int tok, Group& x) const {
    x.shares = 0;
    if (x.nmt <= 1) {
      x.shares = share(x.blocks);  // none for an empty group
    } else {
      for (int i = 0; i < x.g.m; i += tok) {
        const int2 t = prefix_tail(a, x.g.r0 + i, min(tok, x.g.m - i));
        x.shares += share(prefix_blocks<BN>(x.g.np, t.y - t.x));
      }
    }
  }
  __device__ __forceinline__ int sum(int v) const { return (int)__reduce_add_sync(0xffffffffu, (unsigned)v); }
  // The same of numbers up to 2^31 - 1 whose sum may pass 32 bits.
  __device__ __forceinline__ long long sum_wide(int v) const {
    return ((long long)sum(v >> 16) << 16) + sum(v & 0xffff);
  }

  // Sets the tile `left` (CTAs where the tiles own them, else blocks) into the tiles: `left` becomes
  // what remains within the tile.  False if there is none.  `first`: the first 32 groups.
  __device__ __forceinline__ bool locate(const PrefixArgs& a, int tok, const Group& first, int& left) {
    int tiles = 0;
    pos.u0 = 0;
    for (int s0 = 0; s0 < a.n_groups; s0 += 32) {
      Group x = first;
      if (s0 > 0) {
        load(a, tok, s0, x);
        if (own) set_shares(a, tok, x);
      }
      const int mine = a.kv_heads * (own ? x.shares : x.blocks), nt = a.kv_heads * x.nmt, nb = a.kv_heads * x.blocks;
      const int is = warp_incl_scan(mine);
      const unsigned here = __ballot_sync(0xffffffffu, is > left);
      const int w = here ? __ffs(here) - 1 : 32;  // the group's lane
      const bool before = (int)(threadIdx.x & 31) < w;
      tiles += sum(before ? nt : 0);
      pos.u0 += sum(before ? nb : 0);
      if (here) {
        pos.gi = s0 + w;
        pos.g.r0 = __shfl_sync(0xffffffffu, x.g.r0, w);
        pos.g.m = __shfl_sync(0xffffffffu, x.g.m, w);
        pos.g.p0 = __shfl_sync(0xffffffffu, x.g.p0, w);
        pos.g.np = __shfl_sync(0xffffffffu, x.g.np, w);
        left -= __shfl_sync(0xffffffffu, is - mine, w);
        pos.nmt = __shfl_sync(0xffffffffu, x.nmt, w);
        const int per = __shfl_sync(0xffffffffu, own ? x.shares : x.blocks, w);  // of one head
        pos.kh = left / per;
        left -= pos.kh * per;
        pos.t = tiles + pos.kh * pos.nmt;
        pos.u0 += pos.kh * __shfl_sync(0xffffffffu, x.blocks, w);
        for (pos.mt = 0;; ++pos.mt) {
          pos.set_tile(a, tok);
          const int here_n = own ? share(pos.nb) : pos.nb;
          if (left < here_n || pos.mt + 1 >= pos.nmt) break;
          left -= here_n;
          pos.u0 += pos.nb;
          ++pos.t;
        }
        return true;
      }
      left -= __shfl_sync(0xffffffffu, is, 31);
    }
    return false;
  }
  __device__ __forceinline__ void set_part() {
    b0 = u - pos.u0;
    n = min(pos.nb - b0, hi - u);
    first_cta = prefix_cta_of(pos.u0, U, ctas);
    n_ctas = prefix_cta_of(pos.u0 + pos.nb - 1, U, ctas) - first_cta + 1;
  }
  // The first part of CTA `cta` of `grid`; false: it has none.
  __device__ __forceinline__ bool start(const PrefixArgs& a, int tok, int cta, int grid) {
    Group first, x;
    load(a, tok, 0, first);
    unsigned units = first.blocks;
    int nmt = first.nmt;
    for (int s0 = 32; s0 < a.n_groups; s0 += 32) {
      load(a, tok, s0, x);
      units += x.blocks;
      nmt = min(nmt + x.nmt, a.max_tiles + 1);
    }
    // Groups that overlap make more tiles than the scratch has room for, and more units than 32 bits
    // count: none of them is worked on.
    const long long all = a.kv_heads * sum_wide(nmt);
    if (all > a.max_tiles) {
      if ((threadIdx.x & 31) == 0) set_err(a.status, DEV_BAD_INDEX);
      return false;
    }
    const int tiles = (int)all;
    U = a.kv_heads * sum((int)units);
    if (U == 0) return false;
    // CTAs of their own where the tiles are few: the longest part as short as the CTAs allow, to
    // within a few blocks.
    own = false;
    if (2 * tiles <= grid)
      for (int more = 0; more <= 16 && !own; more = more ? 2 * more : 1) {
        most = cdiv(U, grid) + more;
        set_shares(a, tok, first);
        int shares = first.shares;
        for (int s0 = 32; s0 < a.n_groups; s0 += 32) {
          load(a, tok, s0, x);
          set_shares(a, tok, x);
          shares += x.shares;
        }
        own = a.kv_heads * sum(shares) <= grid;
      }
    if (own) {
      int k = cta;
      if (!locate(a, tok, first, k)) return false;
      n_ctas = share(pos.nb);
      first_cta = cta - k;
      b0 = mul_div(k, pos.nb, n_ctas);
      n = mul_div(k + 1, pos.nb, n_ctas) - b0;
      return true;
    }
    ctas = min(U, grid);  // with fewer units than CTAs, one each (a CTA without units has no part)
    if (cta >= ctas) return false;
    u = prefix_u0(cta, U, ctas);
    hi = prefix_u0(cta + 1, U, ctas);
    int left = u;
    if (!locate(a, tok, first, left)) return false;
    set_part();
    return true;
  }
  // The next part; false: there is none.
  __device__ __forceinline__ bool next(const PrefixArgs& a, int tok) {
    if (own || (u += n) >= hi) return false;
    pos.next(a, tok);
    set_part();
    return true;
  }
  // Entries of the tables that the merge reads, written with the tile's first block (threads `id` of
  // `threads`; `half`: rows of a 128-row half of the tile, 0 for tiles in one piece; `two`: a part has
  // two partials, see TcSpan).
  __device__ __forceinline__ void publish(const PrefixArgs& a, int id, int threads, int half = 0,
                                          bool two = false) const {
    if (b0 != 0) return;
    if (id == 0) a.tile_tab[pos.t] = make_int4(first_cta, n_ctas, 0, 0);
    if (pos.kh == 0)
      for (int i = id; i < pos.nrow; i += threads) {
        const int r = half ? i / half * 128 + i % half * a.group : i * a.group;
        a.row_tab[pos.row0 + i] = make_int4(pos.t, pos.nmt, r, two ? 2 : 1);
      }
  }
};

}  // namespace lt

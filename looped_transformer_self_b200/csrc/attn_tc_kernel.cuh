// Attention of 128-row tiles on the 5th-generation tensor cores (bf16): the
// kernel of lt_attn_prompt and lt_attn_prefix.
//
// A resident CTA per SM takes work items one after the other: two tiles of 128
// packed query rows of one key/value head and a range of the keys they see, in
// blocks of 128 that pass through a ring of shared-memory slots.  Warps 0-3 and
// 4-7 hold one tile each, a row per thread; warps 9 and 10 issue the tiles'
// MMAs, warp 11 fetches items, warp 8 loads queries and (prompt) keys and values
// by TMA; for the slot cache warps 12-15 gather the rows (cp.async: one TMA
// request per row ran at half the speed in the decode attention).  Per tile and
// block:
//   S = Q K^T      tcgen05.mma, both from shared memory, S in TMEM (fp32)
//   P = 2^(S' - m) in registers, bf16 into the TMEM columns S stood in
//   O += P V       tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// The tensor core runs the other tile's products while one tile is in its
// softmax.  P is handed over in quarters, so that its product starts while the
// rest is still being computed.
// O is only rescaled when a row's maximum has grown by more than 2^8 since its
// reference was taken: weights stay below 2^8 and sums are fp32, so nothing
// overflows and the relative rounding of a weight is the same at any scale.
//
// What bounds it: a tile's chain of load S, maximum, 128 exponentials a thread,
// product and next S, about 3400 cycles per block of both tiles at head size 128
// against 2048 of the tensor pipe (1536 at 96) and as many of the exponential
// unit (32768 a block, 16 a cycle; counted on a long prefix: 1045 warp
// instructions a block, 1024 of them these).  Measured and not faster: two threads per row (16 softmax warps);
// exponentials on the FMA pipe (polynomial of degree 5); P in halves; half
// blocks of 64 keys with two S buffers a tile, so that a tile's next S runs
// under its softmax (11 % faster at head size 96, 5 to 11 % slower at 128 and
// for the slot cache: products of 64 columns take 3/4 of the tensor rate);
// outputs turned in shared memory before they are stored.
#pragma once

#include "attn_tc.cuh"
#include "attn_prefix.cuh"
#include "prompt_tile.cuh"

namespace lt {

template <int HD>
struct TcShape {
  static constexpr int CHUNKS = (HD + 63) / 64;       // 128-byte column chunks of a row
  static constexpr int TILE = CHUNKS * 128 * 128;     // bytes of a 128-row tile
  static constexpr int SLOTS = HD > 64 ? 5 : 8;       // ring slots (K and V blocks in turn)
  static constexpr int OCOLS = CHUNKS * 64;           // TMEM columns of an output tile
  static constexpr size_t TILES = (size_t)(2 + SLOTS) * TILE;  // queries, ring
};

constexpr int TC_ITEMS = 3;      // items handed over ahead
constexpr int TC_VALID = 8;      // blocks whose marks of present keys are kept

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 scores x of a row to weights 2^(x sl + nms), as bf16 pairs in the first half
// of x, and their fp32 values added to `sum`.  The weights are rounded because the
// product takes both operands in 16 bits; against 64 bits an output is then off by
// 0.0019 to 0.0023 of its size (rms) where fp32 weights and the one rounding of the
// output leave 0.0015 to 0.0017.
__device__ __forceinline__ void softmax_chunk(uint32_t* x, uint64_t sl2, uint64_t nms2, uint64_t* sum) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float e0, e1;
    unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sl2, nms2), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    sum[i & 1] = add2(sum[i & 1], pack2(e0, e1));
    x[i] = pack_bf16(e0, e1);
  }
}
// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}\n" : "=r"(p));
  return p != 0;
}

// Asks for a CTA that has not started; the answer lands in `to` and completes 16 bytes on `bar`.
__device__ __forceinline__ void clc_request(uint32_t to, uint32_t bar) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last answer has been read
  mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
      "r"(bar)
      : "memory");
}
// The block index it gave, or -1.
__device__ __forceinline__ int clc_answer(uint32_t at) {
  uint32_t x, ok;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}\n"
      : "=r"(x), "=r"(ok)
      : "r"(at)
      : "memory");
  return ok ? (int)x : -1;
}

// What an item covers: per tile first token, tokens and blocks, and the ring's
// blocks jb .. jb + n - 1.  The tiles share every block (step 1), except that
// where the second tile is empty its rows may be the first's (step 2): then the
// tiles take the blocks in turn and leave a partial each.
struct TcSpan {
  int t0[2], nt[2], nb[2], n, jb, step;
  __device__ __forceinline__ void share_rows() {
    step = 2;
    t0[1] = t0[0];
    nt[1] = nt[0];
    nb[1] = n >> 1;
    nb[0] = n - nb[1];
  }
  // ring block of the tile's k-th block, from jb
  __device__ __forceinline__ int at(int t, int k) const { return step == 2 ? 2 * k + t : k; }
};

// lt_attn_prompt: a pair of tiles of one sequence, or one of `splits` ranges of
// the keys it sees.  Items are the launch's CTAs: one that is done cancels one
// that has not started and takes its place (clusterlaunchcontrol), which
// balances items of different lengths and lets loads and the first product of
// the next item run under the softmax and output of the last.
struct PromptItem {
  int q0, k0, lq, lk;        // the sequence
  int tile, kh, split, part; // its pair of tiles, head, key range, place of its partial
};
struct PromptWork {
  using Args = PromptArgs;
  using Item = PromptItem;
  static constexpr bool GATHER = false;
  static constexpr int THREADS = 384;
  static __device__ __forceinline__ bool partial(const Args& a) { return a.splits > 1; }
  static __device__ __forceinline__ TcSpan span(const Item& it, int tok, int splits) {
    TcSpan s;
    int full[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.t0[i] = (it.tile * 2 + i) * tok;
      s.nt[i] = max(0, min(tok, it.lq - s.t0[i]));
      full[i] = s.nt[i] ? cdiv(max(0, it.lk - it.lq + s.t0[i] + s.nt[i]), 128) : 0;
    }
    const int chunk = cdiv(max(full[0], full[1]), splits);
    s.jb = it.split * chunk;
#pragma unroll
    for (int i = 0; i < 2; ++i) s.nb[i] = max(0, min(full[i] - s.jb, chunk));
    s.n = max(s.nb[0], s.nb[1]);
    s.step = 1;
    if (splits > 1 && s.nt[1] == 0) s.share_rows();
    return s;
  }
  static __device__ __forceinline__ TcSpan span(const Item& it, int tok, const Args& a) {
    return span(it, tok, a.splits);
  }
};

// lt_attn_prefix: a CTA's share of a tile's blocks (see attn_prefix.cuh).
struct PrefixItem {
  int q0, lq;             // first row, rows
  int p0, np, tail0, nk;  // prefix list, its length, the rows' tail list, keys together
  int jb, n;              // blocks
  int tile, kh, part;     // tile >= 0; head, place of its partial
};
struct PrefixWork {
  using Args = PrefixArgs;
  using Item = PrefixItem;
  static constexpr bool GATHER = true;
  static constexpr int THREADS = 512;
  static __device__ __forceinline__ bool partial(const Args&) { return true; }
  static __device__ __forceinline__ TcSpan span(const Item& it, int tok, const Args&) {
    TcSpan s;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.t0[i] = i * tok;
      s.nt[i] = max(0, min(tok, it.lq - s.t0[i]));
      s.nb[i] = s.nt[i] ? it.n : 0;
    }
    s.n = it.n;
    s.jb = it.jb;
    s.step = 1;
    if (s.nt[1] == 0) s.share_rows();
    return s;
  }
};

template <class W>
struct TcSmem {
  typename W::Item item[TC_ITEMS];
  alignas(16) uint4 clc;  // answer of a cancel request
  uint64_t clc_full, loaded;
  uint64_t item_full[TC_ITEMS], item_empty[TC_ITEMS];
  uint64_t q_full, q_empty, kv_full[8], kv_empty[8], s_full[2], p_full[2][4], o_done[2], turn[2], fin;
  uint32_t tmem;
  int abort_flag;
  int poison[4];  // by item: (its number + 1) once a masked block held an infinity or NaN among its values
  uint64_t valid_full[W::GATHER ? TC_VALID : 1];
  uint32_t valid[W::GATHER ? TC_VALID : 1][4];  // keys of a block that are there, one bit each
};
template <int HD, class W>
constexpr size_t tc_smem() { return TcShape<HD>::TILES + sizeof(TcSmem<W>); }

// Bits [lo, hi) of 32.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  const uint32_t below_hi = hi == 32 ? 0xffffffffu : (1u << hi) - 1;
  return lo == 32 ? 0u : below_hi & (0xffffffffu << lo);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

template <int HD, class W>
__global__ void __launch_bounds__(W::THREADS, 1)
    k_attn_tc(const __grid_constant__ typename W::Args a, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = TcShape<HD>;
  using Item = typename W::Item;
  constexpr bool GATHER = W::GATHER;
  extern __shared__ __align__(1024) char smem_raw[];
  TcSmem<W>& sb = *reinterpret_cast<TcSmem<W>*>(smem_raw + C::TILES);
  if (smem_u32(smem_raw) & 1023) {  // swizzle atoms are 1024 bytes
    pdl_wait();
    set_err(a.status, DEV_STATE);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group, tok = 128 / group;

  const uint32_t q_s = smem_u32(smem_raw), ring = q_s + 2 * C::TILE;
  const uint32_t q_full = smem_u32(&sb.q_full), q_empty = smem_u32(&sb.q_empty), fin = smem_u32(&sb.fin);
  auto kv_full = [&](int s) { return smem_u32(&sb.kv_full[s]); };
  auto kv_empty = [&](int s) { return smem_u32(&sb.kv_empty[s]); };
  auto s_full = [&](int t) { return smem_u32(&sb.s_full[t]); };
  auto p_full = [&](int t, int c) { return smem_u32(&sb.p_full[t][c]); };
  auto o_done = [&](int t) { return smem_u32(&sb.o_done[t]); };
  volatile int* abort_flag = &sb.abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(fin, 2);
    mbar_init(smem_u32(&sb.clc_full), 1);
    mbar_init(smem_u32(&sb.loaded), 1);
    for (int s = 0; s < TC_ITEMS; ++s) {
      mbar_init(smem_u32(&sb.item_full[s]), 1);
      mbar_init(smem_u32(&sb.item_empty[s]), GATHER ? 15 : 11);  // eight softmax warps, the loaders, two MMA warps
    }
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(kv_full(s), GATHER ? 128 : 1);
      mbar_init(kv_empty(s), 2);  // both tiles
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      for (int c = 0; c < 4; ++c) mbar_init(p_full(t, c), 4);  // four warps
      mbar_init(o_done(t), 1);
      mbar_init(smem_u32(&sb.turn[t]), 4);  // four warps of the other tile
    }
    if (GATHER)
      for (int i = 0; i < TC_VALID; ++i) mbar_init(smem_u32(&sb.valid_full[i]), 4);
    sb.abort_flag = 0;
    for (int i = 0; i < 4; ++i) sb.poison[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sb.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // What follows may be launched: it waits for this grid's end before it reads.  Not before this CTA has
  // its TMEM: a kernel that took the columns first and then waited for this grid would never end.
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = sb.tmem;
  auto s_col = [&](int t) { return tmem + (uint32_t)t * 128; };
  auto o_col = [&](int t) { return tmem + 256 + (uint32_t)t * C::OCOLS; };
  // use u of the ring: K and V of the items' blocks in turn
  auto slot_of = [&](int u) { return u % C::SLOTS; };
  auto par_of = [&](int u) { return (uint32_t)(u / C::SLOTS) & 1; };
  // the next item of this CTA (its `it`-th); false at the end
  auto take = [&](int it, Item& item) -> bool {
    const int e = it % TC_ITEMS;
    if (!mbar_wait(smem_u32(&sb.item_full[e]), (uint32_t)(it / TC_ITEMS) & 1, abort_flag)) return false;
    item = sb.item[e];
    return item.tile >= 0;
  };
  auto give_back = [&](int it) { mbar_arrive(smem_u32(&sb.item_empty[it % TC_ITEMS])); };

  // Registers a thread: 168 at launch with three warps per scheduler, of which the softmax
  // warpgroups take 216 and the third keeps 72 (216 + 216 + 72 = 3 * 168); 128 with four, 192, 192,
  // 72 and 56 (= 4 * 128; 200, 200, 56 and 56 spilled in the third: 1 % slower).
  if (GATHER && warp >= 12) {
    if constexpr (GATHER) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      // Keys 32 w + lane of every block: a lane holds one key's slot, and the warp copies the rows of
      // its 32 keys, LPR lanes per row with a 16-byte piece each.  The slots of a lane's rows are
      // spread once for keys and values.  A ring slot counts as full when the copies of all lanes have
      // landed (the barrier follows them); the MMA warps put the proxy fence between the copies and
      // their products.  Waiting for copies here delayed their use by up to three slots.
      constexpr int PIECES = HD / 8, LPR = PIECES > 8 ? 16 : PIECES > 4 ? 8 : 4;
      const int p = lane % LPR, r0 = lane / LPR * LPR;  // piece, first of the lane's LPR rows
      const int w = warp - 12;
      const size_t width = (size_t)a.kv_heads * HD, stride = 2 * width;
      int u = 0;  // ring uses issued
      bool ok = true;
      Item item;
      for (int it = 0;; ++it) {
        ok = __all_sync(0xffffffffu, take(it, item));
        if (!ok) break;
        __syncwarp();
        if (lane == 0) give_back(it);
        const __nv_bfloat16* base = (const __nv_bfloat16*)a.cache + (size_t)item.kh * HD;
        auto fetch = [&](int j) {
          const int x = (item.jb + j) * 128 + w * 32 + lane;
          int s = -1;
          if (j < item.n) {
            if (x < item.np) s = a.prefix[item.p0 + x];
            else if (x < item.nk) s = a.tail[x - item.np + item.tail0];
          }
          return s >= 0 && s < a.n_slots ? s : -1;
        };
        int ahead = fetch(0);
        for (int j = 0; ok && j < item.n; ++j) {
          const int mine = ahead;
          ahead = fetch(j + 1);
          const uint32_t here = __ballot_sync(0xffffffffu, mine >= 0);
          int slots[LPR];
#pragma unroll
          for (int i = 0; i < LPR; ++i) slots[i] = __shfl_sync(0xffffffffu, mine, r0 + i);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++u) {
            const int s = slot_of(u);
            if (u >= C::SLOTS &&
                !(ok = __all_sync(0xffffffffu, mbar_wait(kv_empty(s), par_of(u) ^ 1, abort_flag))))
              break;
            if (kv == 0 && lane == 0) {
              const int b = (u >> 1) & (TC_VALID - 1);
              sb.valid[b][w] = here;
              mbar_arrive(smem_u32(&sb.valid_full[b]));
            }
            const uint32_t dst = ring + s * C::TILE + (w * 32 + r0) * 128 + (p >> 3) * 16384;
            const __nv_bfloat16* src = base + (kv ? width : 0) + p * 8;
            if (PIECES == LPR || p < PIECES) {
              if (here == 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < LPR; ++i)
                  cp_async16(dst + i * 128 + (((p & 7) ^ ((r0 + i) & 7)) << 4), src + (size_t)slots[i] * stride);
              } else {  // absent keys' rows are zero
#pragma unroll
                for (int i = 0; i < LPR; ++i)
                  cp_async16(dst + i * 128 + (((p & 7) ^ ((r0 + i) & 7)) << 4),
                             src + (size_t)max(slots[i], 0) * stride, slots[i] >= 0);
              }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(kv_full(s)) : "memory");
          }
        }
        if (!ok) break;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // copies in flight land before the CTA leaves
    }
  } else if (warp >= 8) {
    if constexpr (GATHER)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      if (lane == 0) {
        int u = 0, qn = 0;
        bool ok = true;
        Item item;
        for (int it = 0; ok && take(it, item); ++it) {
          const TcSpan sp = W::span(item, tok, a);
          auto load_q = [&] {
            if (qn > 0 && !(ok = mbar_wait(q_empty, (uint32_t)(qn - 1) & 1, abort_flag))) return;
            const int qt = (sp.nt[0] > 0) + (sp.nt[1] > 0);
            mbar_expect_tx(q_full, (uint32_t)(qt * C::CHUNKS * tok * group * 128));
            for (int t = 0; t < qt; ++t) {
              const int at = item.q0 + sp.t0[t];
              tma_load_4d(q_s + t * C::TILE, &mq, 0, item.kh * group, at, 0, q_full);
              if (HD == 96) tma_load_4d(q_s + t * C::TILE + 16384, &mq, 64, item.kh * group, at, 0, q_full);
              if (HD == 128) tma_load_4d(q_s + t * C::TILE + 16384, &mq, 0, item.kh * group, at, 1, q_full);
            }
            ++qn;
          };
          if constexpr (GATHER) {
            load_q();
          } else {
            const int ub = u;
            for (; ok && u < ub + 2 * sp.n; ++u) {
              if (u == ub + 1) load_q();  // behind the first key block
              const int s = slot_of(u);
              if (!ok || (u >= C::SLOTS && !(ok = mbar_wait(kv_empty(s), par_of(u) ^ 1, abort_flag)))) break;
              const CUtensorMap* m = ((u - ub) & 1) ? &mv : &mk;
              const int key = item.k0 + (sp.jb + ((u - ub) >> 1)) * 128;
              mbar_expect_tx(kv_full(s), C::TILE);
              tma_load_4d(ring + s * C::TILE, m, 0, item.kh, key, 0, kv_full(s));
              if (HD == 96) tma_load_4d(ring + s * C::TILE + 16384, m, 64, item.kh, key, 0, kv_full(s));
            }
          }
          if (!ok) break;
          give_back(it);
          if constexpr (!GATHER) mbar_arrive(smem_u32(&sb.loaded));
        }
        if (*abort_flag) {  // copies in flight land before the CTA leaves
          int none = 0;
          if (qn > 0) mbar_wait(q_full, (uint32_t)(qn - 1) & 1, &none);
          for (int i = max(0, u - C::SLOTS); i < u; ++i) mbar_wait(kv_full(slot_of(i)), par_of(i), &none);
        }
      }
    } else if (warp < 11) {
      // One warp per tile, so that neither tile's products wait for the other's weights.  The whole
      // warp walks through the items and waits; one elected lane issues (a loop run by one lane alone
      // cost up to 250 cycles per MMA here: its operands do not stay in uniform registers).  MMAs of
      // one thread run in order, so S may be written over the P of the product before it.
      constexpr uint32_t IS = attn_idesc(128, false), IO = attn_idesc(HD, true);
      const int t = warp - 9;
      // descriptors count 16-byte units: a step along an operand is an addition
      const uint64_t dq = smem_desc(q_s + t * C::TILE), dk = smem_desc(ring), dv = smem_desc_mn(ring, 16384);
      const uint32_t st = s_col(t), ot = o_col(t), s_bar = s_full(t), o_bar = o_done(t);
      auto wait = [&](uint32_t bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, par)) ||
               __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag));
      };
      int slot = 0, done = 0, qn = 0;
      uint32_t ring_par = 0;
      auto next_slot = [&] {
        if (++slot == C::SLOTS) {
          slot = 0;
          ring_par ^= 1;
        }
      };
      bool ok = true;
      Item item;
      for (int it = 0; ok; ++it) {
        ok = __all_sync(0xffffffffu, take(it, item));
        if (!ok) break;
        const TcSpan sp = W::span(item, tok, a);
        __syncwarp();
        if (lane == 0) give_back(it);
        if (sp.n == 0) continue;
        const int nb = t ? sp.nb[1] : sp.nb[0];
        if (!(ok = wait(q_full, (uint32_t)qn & 1))) break;
        ++qn;
        // Step j: the product of block j - 1's weights, then S of block j.  A slot is given back by
        // both tiles, used or not, and not before it is full: no tile gets a turn of the ring ahead.
        int v_slot = 0, s_next = 0, p_next = 0;  // blocks whose S is out; the one whose product follows, + 1
        uint32_t v_par = 0;
        for (int j = 0; j <= sp.n; ++j) {
          const int k_slot = slot;
          const uint32_t k_par = ring_par;
          if (j > 0 && !(ok = wait(kv_full(v_slot), v_par))) break;
          if (GATHER) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (p_next > 0) {
            const uint64_t v = dv + (uint32_t)(v_slot * (C::TILE >> 4));
            const uint32_t par = (uint32_t)(done + p_next - 1) & 1;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (!(ok = ok && wait(p_full(t, c), par))) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int i = 2 * c; i < 2 * c + 2; ++i)
                  tc_mma_ts(ot, st + i * 8, v + i * 128, IO, p_next > 1 || i > 0);
                if (c == 3) tc_commit(o_bar);
              }
              __syncwarp();
            }
            if (!ok) break;
            p_next = 0;
          }
          if (j < sp.n) {
            if (!(ok = wait(kv_full(k_slot), k_par))) break;
            if (GATHER) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (s_next < nb && j == sp.at(t, s_next)) {
              p_next = ++s_next;
              tc_fence_after();
              const uint64_t k = dk + (uint32_t)(k_slot * (C::TILE >> 4));
              if (elect_one()) {
#pragma unroll
                for (int i = 0; i < HD / 16; ++i) {
                  const uint32_t at = ((uint32_t)(i >> 2) * 16384 + (i & 3) * 32) >> 4;
                  tc_mma<false>(st, dq + at, k + at, IS, i > 0);
                }
                tc_commit(s_bar);
              }
              __syncwarp();
            }
            next_slot();
          }
          if (elect_one()) {
            if (j > 0) tc_commit(kv_empty(v_slot));
            if (j < sp.n) tc_commit(kv_empty(k_slot));
            if (j + 1 == sp.n) tc_commit(q_empty);
          }
          __syncwarp();
          if (j < sp.n) {
            v_slot = slot;
            v_par = ring_par;
            next_slot();
          }
        }
        done += nb;
      }
      if (*abort_flag) {  // MMAs in flight end before TMEM is freed
        int none = 0;
        if (elect_one()) tc_commit(fin);
        __syncwarp();
        mbar_wait(fin, 0, &none);
        __syncwarp();
      }
    } else {
      auto wait = [&](uint32_t bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag)) != 0;
      };
      auto hand_over = [&](int it, const Item& item) {
        const int e = it % TC_ITEMS;
        if (it >= TC_ITEMS && !wait(smem_u32(&sb.item_empty[e]), (uint32_t)(it / TC_ITEMS - 1) & 1)) return false;
        if (lane == 0) {
          sb.item[e] = item;
          mbar_arrive(smem_u32(&sb.item_full[e]));
        }
        return true;
      };
      if constexpr (GATHER) {
        const int rows = 2 * tok;  // of a pair of tiles
        int it = 0;
        PrefixWalk<128> walk;
        if (walk.start(a, rows, blockIdx.x, gridDim.x)) {
          do {
            const PrefixPos<128>& pos = walk.pos;
            walk.publish(a, lane, 32, tok, pos.nrow <= tok);
            if (!hand_over(it, PrefixItem{pos.row0, pos.nrow, pos.g.p0, pos.g.np, pos.tail.x,
                                          pos.g.np + pos.tail.y - pos.tail.x, walk.b0, walk.n, 0, pos.kh,
                                          (int)blockIdx.x + pos.t}))
              break;
            ++it;
          } while (walk.next(a, rows));
        }
        hand_over(it, PrefixItem{0, 0, 0, 0, 0, 0, 0, 0, -1, 0, 0});
      } else {
        // An item is asked for when the loads of the one before are out: the ring holds two blocks or
        // more then, which covers the answer, and no CTA takes work that another could start sooner.
        int idx = blockIdx.x, it = 0;
        const uint32_t clc = smem_u32(&sb.clc), clc_full = smem_u32(&sb.clc_full);
        for (uint32_t asked = 0;; ++asked) {
          PromptTile pt;
          const int pair = idx / a.splits;
          const bool have = idx >= 0 && prompt_tile(a, pair / a.kv_heads, 2 * tok, pt);
          if (have || idx < 0) {
            PromptItem item = {0, 0, 0, 0, -1, 0, 0, 0};
            if (have) item = {pt.q0, pt.k0, pt.lq, pt.lk, pt.tile, pair % a.kv_heads, idx % a.splits, idx};
            if (!hand_over(it, item)) break;
            if (idx < 0 || !wait(smem_u32(&sb.loaded), (uint32_t)it & 1)) break;
            ++it;
          }
          if (lane == 0) clc_request(clc, clc_full);
          __syncwarp();
          if (!wait(clc_full, asked & 1)) {  // nothing writes to shared memory after the CTA is gone
            int none = 0;
            mbar_wait(clc_full, asked & 1, &none);
            break;
          }
          idx = clc_answer(clc);
          __syncwarp();
        }
      }
    }
  } else {
    if constexpr (GATHER)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sc = s_col(t) + lane_off, oc = o_col(t) + lane_off;
    const int tl = r / group;                        // token within the tile
    const float sl = a.scale * 1.4426950408889634f;  // scores in log2 units
    const float slack = fminf(8.f / sl, 1e30f);
    int ub = 0, done = 0;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_try_wait(bar, par)) ||
             __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag));
    };
    // The tiles take turns with their exponentials, one turn per block of the item (a tile without the
    // block passes): left alone they fall into step, both in their softmax and then both waiting for
    // the tensor core.
    int turns = 0;
    const uint32_t my_turn = smem_u32(&sb.turn[t]), other_turn = smem_u32(&sb.turn[t ^ 1]);
    auto take_turn = [&](int k) { return wait(my_turn, (uint32_t)(turns + k + (t ^ 1)) & 1); };
    auto pass_turn = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(other_turn);
    };
    for (int it = 0; ok; ++it) {
      Item item;
      ok = __all_sync(0xffffffffu, take(it, item));
      if (!ok) break;
      if (lane == 0) give_back(it);
      const TcSpan sp = W::span(item, tok, a);
      const int t0 = t ? sp.t0[1] : sp.t0[0], nt = t ? sp.nt[1] : sp.nt[0], nb = t ? sp.nb[1] : sp.nb[0];
      const bool valid = tl < nt && r < tok * group;
      // Keys a row sees: [0, see) and, of the slot cache, also [own.x, own.y).  Keys from `shared` on
      // are not seen by all rows of the tile, keys from `scanned` on not by all rows of both tiles.
      int see, shared, scanned;
      int2 own = {0, 0};
      if constexpr (GATHER) {
        see = shared = scanned = item.np;
        if (valid) {
          const int2 t2 = off_range(a.tail_off, item.q0 + t0 + tl, a.n_tail, a.status);
          own = {item.np + t2.x - item.tail0, item.np + t2.y - item.tail0};
        }
      } else {
        const int ctx = item.lk - item.lq;
        see = valid ? ctx + t0 + tl + 1 : 0;  // may be <= 0
        shared = ctx + t0 + 1;
        scanned = ctx + sp.t0[0] + 1;
      }
      float m = -INFINITY, l = 0.f;                   // m: reference maximum of the raw scores
      for (int jj = 0; jj < nb; ++jj) {
        const int jr = sp.at(t, jj), j = sp.jb + jr, ph = done + jj;
        if (!(ok = wait(s_full(t), ph & 1))) break;
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(sc + c * 32, x + c * 32);
        tmem_wait_ld();
        const bool mixed = (j + 1) * 128 > shared;  // holds keys that some row does not see
        bool masked = mixed;
        const uint32_t* there = nullptr;
        if constexpr (GATHER) {
          // the loads are fewer than TC_VALID blocks ahead, so the marks stay
          const int b = (ub >> 1) + jr;
          if (!(ok = wait(smem_u32(&sb.valid_full[b & (TC_VALID - 1)]), (uint32_t)(b / TC_VALID) & 1))) break;
          there = sb.valid[b & (TC_VALID - 1)];
          masked = mixed || (there[0] & there[1] & there[2] & there[3]) != 0xffffffffu;
        }
        if (masked) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int x0 = j * 128 + c * 32;
            uint32_t seen = bit_range(0, see - x0);
            if constexpr (GATHER) seen = (seen | bit_range(own.x - x0, own.y - x0)) & there[c];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen & (1u << i))) x[c * 32 + i] = 0xff800000u;  // -inf
          }
        }
        if ((j + 1) * 128 > scanned) {
          // Values that some row must not see: rows behind the keys (other sequences, padding)
          // are zeroed, infinities and NaN taken out (0 * inf is NaN) and given back to the rows
          // that see them at the end.  A thread goes over one key's row.  Both tiles do this for the
          // same blocks, each before its own product, so that neither multiplies what the other may
          // have taken out or not; and every thread fences, since a row that it finds clean may have
          // been cleaned by the other tile a moment before.
          const int u = ub + 2 * jr + 1;
          if (!(ok = wait(kv_full(slot_of(u)), par_of(u)))) break;
          char* row = smem_raw + (2 + slot_of(u)) * C::TILE + r * 128;
          bool gone = false;  // an absent slot's row is zero already
          if constexpr (!GATHER) gone = j * 128 + r >= item.lk;
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < HD / 8; ++k) {
            // a key's 16-byte pieces lie at places given by its row (the swizzle)
            const uint4 v = *reinterpret_cast<const uint4*>(row + (k >> 3) * 16384 + (((k & 7) ^ (r & 7)) << 4));
            bad |= nonfinite_bits(v.x) | nonfinite_bits(v.y) | nonfinite_bits(v.z) | nonfinite_bits(v.w);
          }
          if (gone || bad) {
            if (!gone) {
              *(volatile int*)&sb.poison[it & 3] = it + 1;
              __threadfence_block();  // a warp that finds the value gone finds the flag set
            }
#pragma unroll 1
            for (int k = 0; k < HD / 8; ++k) {
              uint4* q = reinterpret_cast<uint4*>(row + (k >> 3) * 16384 + (((k & 7) ^ (r & 7)) << 4));
              uint4 v = *q;
              if (gone) v = make_uint4(0u, 0u, 0u, 0u);
              drop_nonfinite(v.x);
              drop_nonfinite(v.y);
              drop_nonfinite(v.z);
              drop_nonfinite(v.w);
              *q = v;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        float mx4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx4[e] = __uint_as_float(x[e]);
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx4[e] = fmaxf(fmaxf(mx4[e], __uint_as_float(x[c + e])), __uint_as_float(x[c + 4 + e]));
#pragma unroll
        for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], __uint_as_float(x[124 + e]));
        // (a NaN score leaves the maximum and comes out in its weight and the sum)
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const bool grow = mx > m + slack;
        if (jj == 0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2((m - mx) * sl) : 1.f;
          if (grow) m = mx;
          l *= f;
          if (!(ok = wait(o_done(t), (ph - 1) & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < HD; c += 16) {
            uint32_t o[16];
            tmem_ld16(oc + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(oc + c, o);
          }
        }
        // nothing seen yet: every weight is 0; an infinite or NaN maximum makes the row NaN
        float ms = m * sl;
        if (!(fabsf(ms) < INFINITY)) ms = m == -INFINITY ? 0.f : NAN;
        const uint64_t sl2 = pack2(sl, sl), ms2 = pack2(-ms, -ms);
        uint64_t sum[2] = {0, 0};
        if (!(ok = take_turn(jj))) break;
        // a quarter's store is waited for after the next quarter's exponentials
#pragma unroll
        for (int c = 0; c <= 4; ++c) {
          if (c < 4) softmax_chunk(x + c * 32, sl2, ms2, sum);
          if (c == 3) pass_turn();
          if (c > 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(t, c - 1));
          }
          if (c < 4) tmem_st16(sc + c * 16, x + c * 32);
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      const int most = max(sp.nb[0], sp.nb[1]);
      for (int k = nb; ok && k < most; ++k) {
        ok = take_turn(k);
        pass_turn();
      }
      turns += most;
      if (!ok) break;
      const bool partial = W::partial(a);
      if (GATHER && nb == 0 && valid) a.part_ml[(size_t)item.part * 256 + t * 128 + r] = make_float2(-INFINITY, 0.f);
      if (nt > 0 && (nb > 0 || !partial)) {
        if (nb > 0) {
          if (!(ok = wait(o_done(t), (done + nb - 1) & 1))) break;
          tc_fence_after();
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t prow = (size_t)item.part * 256 + t * 128 + r;  // row of the partial
        if (partial && valid) a.part_ml[prow] = make_float2(m * sl, l);
        __nv_bfloat16* o = (__nv_bfloat16*)a.o + (size_t)(item.q0 + t0 + tl) * a.so +
                           (size_t)(item.kh * group + r % group) * HD;
        const bool poison = nb > 0 && *(volatile int*)&sb.poison[it & 3] == it + 1;
        // keys of mixed blocks of either tile
        int from, to;
        if constexpr (GATHER) {
          from = item.np & ~127;
          to = item.nk;
        } else {
          from = max(0, (item.lk - item.lq + sp.t0[0] + 1) & ~127);
          to = item.lk - item.lq + t0 + nt;
        }
        from = max(from, sp.jb * 128);
        to = min(to, (sp.jb + sp.n) * 128);
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t x[32];
          if (nb > 0) {
            tmem_ld32(oc + c, x);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0;
          }
          if (poison) {
            for (int key = from; key < to; ++key) {
              if (sp.step == 2 && (((key >> 7) - sp.jb) & 1) != t) continue;  // the other tile's
              const __nv_bfloat16* v;
              if constexpr (GATHER) {
                const int slot = key < item.np ? a.prefix[item.p0 + key] : a.tail[key - item.np + item.tail0];
                if (slot < 0 || slot >= a.n_slots) continue;
                v = (const __nv_bfloat16*)a.cache + ((size_t)slot * 2 + 1) * a.kv_heads * HD;
              } else {
                v = (const __nv_bfloat16*)a.v + (size_t)(item.k0 + key) * a.sv;
              }
              v += (size_t)item.kh * HD + c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float f = __bfloat162float(v[i]);
                if (!(fabsf(f) < INFINITY) && (key < see || (key >= own.x && key < own.y))) x[i] = __float_as_uint(__uint_as_float(x[i]) + f);
              }
            }
          }
          if (!valid) continue;
          if (partial) {
            float* dst = a.part + prow * HD + c;
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global32(dst + 8 * i, x + 8 * i);
          } else if constexpr (!GATHER) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = pack_bf16(__uint_as_float(x[2 * i]) * inv, __uint_as_float(x[2 * i + 1]) * inv);
            if (a.o_wide) {  // a row's 64 bytes in two stores of whole 32-byte sectors
              st_global32(o + c, x);
              st_global32(o + c + 16, x + 8);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(o + c + 8 * i) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
          }
        }
        tc_fence_before();  // O is read before the next item's first product overwrites it
      }
      done += nb;
      ub += 2 * sp.n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) set_err(a.status, DEV_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the key ranges of a pair of tiles: with M the largest maximum of a row's
// partials, o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, in range order.
// One thread per four columns of a row; JOIN_ROWS rows of a pair per CTA.
template <int HD>
constexpr int prompt_join_rows() { return 256 / (HD / 4); }
template <int HD>
__global__ void __launch_bounds__(256) k_attn_prompt_join(PromptArgs a, int parts) {
  pdl_wait();
  constexpr int PER = HD / 4, ROWS = prompt_join_rows<HD>();
  const int tok = 128 / a.group, pair = blockIdx.x / parts;
  PromptTile pt;
  if (!prompt_tile(a, pair / a.kv_heads, 2 * tok, pt)) return;
  const int kh = pair % a.kv_heads;
  const int row = (blockIdx.x % parts) * ROWS + (int)threadIdx.x / PER, c = ((int)threadIdx.x % PER) * 4;
  const int t = row >> 7, r = row & 127, token = (pt.tile * 2 + t) * tok + r / a.group;
  if ((int)threadIdx.x >= ROWS * PER || row >= 256 || r >= tok * a.group || token >= pt.lq) return;
  const PromptItem it = {pt.q0, pt.k0, pt.lq, pt.lk, pt.tile, kh, 0, 0};
  const TcSpan whole = PromptWork::span(it, tok, 1);
  const int blocks = t ? whole.nb[1] : whole.nb[0], chunk = cdiv(whole.n, a.splits);
  // a range's partial, or its two where both tiles took the rows (blocks in turn)
  const int two = whole.nt[1] == 0 ? 2 : 1;
  const size_t p0 = (size_t)pair * a.splits * 256 + row;
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int B = 8;  // partials in flight
  for (int k0 = 0; (k0 / two) * chunk < blocks; k0 += B) {
    float2 ml[B];
    float4 v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int s = (k0 + i) / two, e = (k0 + i) % two;
      const bool there = s * chunk + e < blocks && e < chunk;
      const size_t p = p0 + (size_t)s * 256 + e * 128;
      ml[i] = there ? a.part_ml[p] : make_float2(-INFINITY, 0.f);
      v[i] = there ? *reinterpret_cast<const float4*>(a.part + p * HD + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = M;
#pragma unroll
    for (int i = 0; i < B; ++i) mx = max_nan(mx, ml[i].x);
    const float ms = mx == -INFINITY ? 0.f : mx, f = ex2(M - ms);
    M = mx;
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const float w = ex2(ml[i].x - ms);
      l += w * ml[i].y;
      o.x = fmaf(w, v[i].x, o.x);
      o.y = fmaf(w, v[i].y, o.y);
      o.z = fmaf(w, v[i].z, o.z);
      o.w = fmaf(w, v[i].w, o.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>((__nv_bfloat16*)a.o + (size_t)(pt.q0 + token) * a.so +
                            (size_t)(kh * a.group + r % a.group) * HD + c) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

}  // namespace lt

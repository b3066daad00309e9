// lt_attn_prompt for bf16 on the 5th-generation tensor cores.
//
// One CTA takes two tiles of 128 packed query rows of one key/value head and
// streams the keys they see in blocks of 128 through a ring of shared-memory
// slots (TMA).  Warps 0-3 and 4-7 hold one tile each, a row per thread; warp 8
// loads, warp 9 issues the MMAs.  Per tile and block:
//   S = Q K^T      tcgen05.mma, both from shared memory, S in TMEM (fp32)
//   P = e^(S - m)  in registers, bf16 into the TMEM columns S stood in
//   O += P V       tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// The tensor core runs the other tile's products while one tile is in its
// softmax.  O is only rescaled when a row's maximum has grown by more than 2^8
// since its reference was taken (the weights stay below 2^8 and the sums are
// fp32, so nothing overflows and the relative rounding of a weight is the same
// at any scale); that is rare after the first blocks, so O stays in TMEM.
#pragma once

#include "attn_tc.cuh"
#include "prompt_tile.cuh"

namespace lt {

template <int HD>
struct PromptTc {
  static constexpr int NT = 2;                        // tiles of a CTA
  static constexpr int CHUNKS = (HD + 63) / 64;       // 128-byte column chunks of a row
  static constexpr int TILE = CHUNKS * 128 * 128;     // bytes of a 128-row tile
  static constexpr int SLOTS = HD > 64 ? 5 : 8;       // ring slots (K and V blocks in turn)
  static constexpr int OCOLS = CHUNKS * 64;           // TMEM columns of an output tile
  static constexpr int THREADS = NT * 128 + 128;      // two softmax warpgroups, one for loads and MMAs
  static constexpr size_t SMEM = 1024 + (size_t)(NT + SLOTS) * TILE;
};

struct PromptBars {
  uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_full[2], o_done[2], fin;
  uint32_t tmem;
  int abort_flag;
  int poison;  // a masked block held an infinity or NaN among its values
};

template <int HD>
__global__ void __launch_bounds__(PromptTc<HD>::THREADS, 1)
    k_attn_prompt_tc(PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv) {
  using C = PromptTc<HD>;
  extern __shared__ char smem_raw[];
  __shared__ PromptBars sb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = blockIdx.x % a.kv_heads, group = a.group, tok = 128 / group;
  PromptTile pt;
  if (!prompt_tile(a, blockIdx.x / a.kv_heads, C::NT * tok, pt)) return;
  const int ctx = pt.lk - pt.lq;
  // per tile: first token, tokens, keys its last row sees, key blocks
  int t0[2], nt[2], nb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t0[i] = (pt.tile * 2 + i) * tok;
    nt[i] = max(0, min(tok, pt.lq - t0[i]));
    nb[i] = nt[i] ? cdiv(max(0, ctx + t0[i] + nt[i]), 128) : 0;
  }
  const int n = max(nb[0], nb[1]);

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_s = base, ring = base + C::NT * C::TILE;
  const uint32_t q_full = smem_u32(&sb.q_full), fin = smem_u32(&sb.fin);
  auto kv_full = [&](int s) { return smem_u32(&sb.kv_full[s]); };
  auto kv_empty = [&](int s) { return smem_u32(&sb.kv_empty[s]); };
  auto s_full = [&](int t) { return smem_u32(&sb.s_full[t]); };
  auto p_full = [&](int t) { return smem_u32(&sb.p_full[t]); };
  auto o_done = [&](int t) { return smem_u32(&sb.o_done[t]); };
  volatile int* abort_flag = &sb.abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(fin, 1);
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 128);
      mbar_init(o_done(t), 1);
    }
    sb.abort_flag = 0;
    sb.poison = 0;
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
  const uint32_t tmem = sb.tmem;
  auto s_col = [&](int t) { return tmem + (uint32_t)t * 128; };
  auto o_col = [&](int t) { return tmem + 256 + (uint32_t)t * C::OCOLS; };
  // use u of the ring: K_0, V_0, K_1, V_1, ...
  auto slot_of = [&](int u) { return u % C::SLOTS; };
  auto par_of = [&](int u) { return (uint32_t)(u / C::SLOTS) & 1; };

  // 168 registers a thread at launch (3 warps per scheduler): the softmax warpgroups take 216, the
  // third keeps 72 (216 + 216 + 72 = 3 * 168).
  if (warp >= 8) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
   if (warp == 8) {
    if (lane == 0 && n > 0) {
      const int qt = (nt[0] > 0) + (nt[1] > 0);
      mbar_expect_tx(q_full, (uint32_t)(qt * C::CHUNKS * tok * group * 128));
      for (int t = 0; t < qt; ++t) {
        tma_load_4d(q_s + t * C::TILE, &mq, 0, kh * group, pt.q0 + t0[t], 0, q_full);
        if (HD == 96) tma_load_4d(q_s + t * C::TILE + 16384, &mq, 64, kh * group, pt.q0 + t0[t], 0, q_full);
      }
      int u = 0;
      for (; u < 2 * n; ++u) {
        const int s = slot_of(u);
        if (u >= C::SLOTS && !mbar_wait(kv_empty(s), par_of(u) ^ 1, abort_flag)) break;
        const CUtensorMap* m = (u & 1) ? &mv : &mk;
        const int key = pt.k0 + (u >> 1) * 128;
        mbar_expect_tx(kv_full(s), C::TILE);
        tma_load_4d(ring + s * C::TILE, m, 0, kh, key, 0, kv_full(s));
        if (HD == 96) tma_load_4d(ring + s * C::TILE + 16384, m, 64, kh, key, 0, kv_full(s));
      }
      if (*abort_flag) {  // copies in flight land before the CTA leaves
        int none = 0;
        mbar_wait(q_full, 0, &none);
        for (int i = max(0, u - C::SLOTS); i < u; ++i) mbar_wait(kv_full(slot_of(i)), par_of(i), &none);
      }
    }
   } else if (warp == 9) {
    if (lane == 0 && n > 0) {
      constexpr uint32_t IS = attn_idesc(128, false), IO = attn_idesc(HD, true);
      auto issue_s = [&](int t, int u) {
        const uint32_t k = ring + slot_of(u) * C::TILE, q = q_s + t * C::TILE;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          const uint32_t at = (uint32_t)(i >> 2) * 16384 + (i & 3) * 32;
          tc_mma<false>(s_col(t), smem_desc(q + at), smem_desc(k + at), IS, i > 0);
        }
        tc_commit(s_full(t));
      };
      auto issue_o = [&](int t, int u, bool acc) {
        const uint32_t v = ring + slot_of(u) * C::TILE;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tc_mma_ts(o_col(t), s_col(t) + i * 8, smem_desc_mn(v + i * 2048, 16384), IO, acc || i > 0);
        tc_commit(o_done(t));
      };
      bool ok = mbar_wait(q_full, 0, abort_flag) && mbar_wait(kv_full(0), 0, abort_flag);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < 2; ++t)
          if (nb[t] > 0) issue_s(t, 0);
        tc_commit(kv_empty(0));
      }
      for (int j = 0; ok && j < n; ++j) {
        const int uv = 2 * j + 1, uk = 2 * j + 2;
        for (int t = 0; ok && t < 2; ++t) {
          if (j >= nb[t]) continue;
          ok = mbar_wait(kv_full(slot_of(uv)), par_of(uv), abort_flag) &&
               mbar_wait(p_full(t), j & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue_o(t, uv, j > 0);
          if (j + 1 < nb[t]) {
            ok = mbar_wait(kv_full(slot_of(uk)), par_of(uk), abort_flag);
            if (!ok) break;
            issue_s(t, uk);
          }
        }
        if (!ok) break;
        tc_commit(kv_empty(slot_of(uv)));
        if (j + 1 < n) tc_commit(kv_empty(slot_of(uk)));
      }
      if (!ok) {  // MMAs in flight end before TMEM is freed
        int none = 0;
        tc_commit(fin);
        mbar_wait(fin, 0, &none);
      }
    }
   }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sc = s_col(t) + lane_off, oc = o_col(t) + lane_off;
    const int tl = r / group;                         // token within the tile
    const bool valid = tl < nt[t] && r < tok * group;
    const int see = valid ? ctx + t0[t] + tl + 1 : 0;  // keys this row sees (may be <= 0)
    const int see_first = ctx + t0[t] + 1;             // keys the tile's first row sees
    const float sl = a.scale * 1.4426950408889634f;    // scores in log2 units
    float m = -INFINITY, l = 0.f;                      // m: reference maximum of the raw scores
    bool ok = true;
    for (int j = 0; j < nb[t]; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(s_full(t), j & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t x[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(sc + c * 32, x + c * 32);
      tmem_wait_ld();
      const bool masked = (j + 1) * 128 > see_first;
      if (masked) {
        const int lim = see - j * 128;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= lim) x[c] = 0xff800000u;  // -inf
      }
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 128; ++c) mx = fmaxf(mx, __uint_as_float(x[c]));
      const bool grow = (mx - m) * sl > 8.f;  // false where both are -inf
      if (j == 0) {
        m = mx;
      } else if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2((m - mx) * sl) : 1.f;
        if (grow) m = mx;
        l *= f;
        ok = __all_sync(0xffffffffu, mbar_wait(o_done(t), (j - 1) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(oc + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(oc + c, o);
        }
      }
      const float ms = m == -INFINITY ? 0.f : m * sl;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e0 = ex2(fmaf(__uint_as_float(x[c * 32 + 2 * i]), sl, -ms));
          const float e1 = ex2(fmaf(__uint_as_float(x[c * 32 + 2 * i + 1]), sl, -ms));
          sum[i & 3] += e0 + e1;
          p[i] = pack_bf16(e0, e1);
        }
        tmem_st16(sc + c * 16, p);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (masked) {
        // Values that some row must not see: rows behind the keys (other sequences, padding) are
        // zeroed, infinities and NaN taken out (0 * inf is NaN) and given back to the rows that
        // see them at the end.  A thread goes over one key's row.
        const int u = 2 * j + 1;
        ok = __all_sync(0xffffffffu, mbar_wait(kv_full(slot_of(u)), par_of(u), abort_flag));
        if (!ok) break;
        char* row = smem_raw + (ring - smem_u32(smem_raw)) + slot_of(u) * C::TILE + r * 128;
        const bool gone = j * 128 + r >= pt.lk;
#pragma unroll
        for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint4* p = reinterpret_cast<uint4*>(row + c * 16384 + ((i + r) & 7) * 16);
            uint4 v = *p;
            if (gone) {
              *p = make_uint4(0u, 0u, 0u, 0u);
            } else {
              const bool b0 = drop_nonfinite(v.x), b1 = drop_nonfinite(v.y), b2 = drop_nonfinite(v.z),
                         b3 = drop_nonfinite(v.w);
              if (b0 || b1 || b2 || b3) {
                *(volatile int*)&sb.poison = 1;
                __threadfence_block();  // a warp that finds the value gone finds the flag set
                *p = v;
              }
            }
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full(t));
    }
    if (ok && nt[t] > 0) {
      if (nb[t] > 0) ok = __all_sync(0xffffffffu, mbar_wait(o_done(t), (nb[t] - 1) & 1, abort_flag));
      if (ok) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16* o = (__nv_bfloat16*)a.o + (size_t)(pt.q0 + t0[t] + tl) * a.so +
                           (size_t)(kh * group + r % group) * HD;
        const bool poison = nb[t] > 0 && *(volatile int*)&sb.poison;
        // masked keys of either tile start here
        const int from = max(0, (ctx + t0[0] + 1) & ~127);
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t x[32];
          if (nb[t] > 0) {
            tmem_ld32(oc + c, x);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0;
          }
          if (poison) {
            for (int key = from; key < ctx + t0[t] + nt[t]; ++key) {
              const __nv_bfloat16* v =
                  (const __nv_bfloat16*)a.v + (size_t)(pt.k0 + key) * a.sv + (size_t)kh * HD + c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float f = __bfloat162float(v[i]);
                if (!(fabsf(f) < INFINITY) && key < see) x[i] = __float_as_uint(__uint_as_float(x[i]) + f);
              }
            }
          }
          if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 w;
              w.x = pack_bf16(__uint_as_float(x[8 * i]) * inv, __uint_as_float(x[8 * i + 1]) * inv);
              w.y = pack_bf16(__uint_as_float(x[8 * i + 2]) * inv, __uint_as_float(x[8 * i + 3]) * inv);
              w.z = pack_bf16(__uint_as_float(x[8 * i + 4]) * inv, __uint_as_float(x[8 * i + 5]) * inv);
              w.w = pack_bf16(__uint_as_float(x[8 * i + 6]) * inv, __uint_as_float(x[8 * i + 7]) * inv);
              *reinterpret_cast<uint4*>(o + c + 8 * i) = w;
            }
          }
        }
      }
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

template <int HD>
static int prompt_tc(const PromptArgs& a, cudaStream_t st) {
  using C = PromptTc<HD>;
  const int tok = 128 / a.group;
  CUtensorMap mq, mk, mv;
  // no keys: nothing is loaded, and the maps stand on the queries
  const void* k = a.n_kv > 0 ? a.k : a.q;
  const void* v = a.n_kv > 0 ? a.v : a.q;
  const long long nk = a.n_kv > 0 ? a.n_kv : 1;
  if (attn_tmap(&mq, a.q, HD, a.heads, a.n_q, a.sq, a.group, tok) ||
      attn_tmap(&mk, k, HD, a.kv_heads, nk, a.sk, 1, 128) || attn_tmap(&mv, v, HD, a.kv_heads, nk, a.sv, 1, 128))
    return LT_ERR_CUDA;
  static bool set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (cudaFuncSetAttribute(k_attn_prompt_tc<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) !=
        cudaSuccess)
      return LT_ERR_CUDA;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const unsigned tiles = (unsigned)(a.n_q / (C::NT * tok) + a.n_seqs);
  k_attn_prompt_tc<HD><<<tiles * a.kv_heads, C::THREADS, C::SMEM, st>>>(a, mq, mk, mv);
  return cudaGetLastError() == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

}  // namespace lt

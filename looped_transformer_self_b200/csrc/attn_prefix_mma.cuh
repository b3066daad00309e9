// lt_attn_prefix for bf16 with few packed rows per key/value head: warp-level
// MMAs (m16n8k16) over a cp.async ring of gathered cache rows.
//
// Few rows make this a stream of the cache (2 MT flops per byte of it), so the
// tensor rate does not bound it; what counts is bytes in flight.  Warps are
// WM x WK: each holds 16 packed rows and every WK-th 16-key slice of a block,
// with its own running maximum, sum and output, merged when the CTA leaves the
// tile.  Rows of shared memory are 16 bytes longer than a cache row, so eight
// rows' pieces of one column lie in different banks (ldmatrix).  Weights are
// rounded to bf16 for their product, as the MMA takes them; their sum is of the
// fp32 values.  Measured with the merge: 8 rows on 601 shared slots (16 heads of
// 128, 5.1 MB) 10.0 us, bound by its start and the merge; 1 row on 6000 slots
// 22.2 us (49 MB, 2.2 TB/s).
#pragma once

#include "attn_tc_kernel.cuh"

namespace lt {

constexpr int PREFIX_N = 64;  // keys of a block

template <int HD, int MT>
struct PrefixMma {
  static constexpr int WARPS = 4, THREADS = 128;
  static constexpr int WM = MT / 16, WK = WARPS / WM;
  static constexpr int STAGES = 3;
  static constexpr int PITCH = HD * 2 + 16;                // bytes
  static constexpr int STAGE = 2 * PREFIX_N * PITCH;       // K rows, then V rows
  static constexpr int KEYS = PREFIX_N / WK;               // keys of a warp in a block
  static constexpr int RING = 8;                           // slot lists kept
  static constexpr size_t SMEM = (size_t)STAGES * STAGE;
  static_assert((size_t)WARPS * 16 * (HD + 4) * 4 <= SMEM, "the merge reuses the ring");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int HD, int MT>
__global__ void __launch_bounds__(128, 2) k_attn_prefix_mma(PrefixArgs a) {
  using C = PrefixMma<HD, MT>;
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ int sslot[C::RING][PREFIX_N];
  __shared__ uint32_t svalid[C::RING][2];
  __shared__ float2 sml[C::WARPS][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wm = warp / C::WK, wk = warp % C::WK;
  const int gr = lane >> 2, gc = (lane & 3) * 2;
  const uint32_t smem = smem_u32(smem_raw);
  const int group = a.group, tok = MT / group;
  pdl_trigger();
  pdl_wait();
  PrefixWalk<PREFIX_N> walk;
  if (!walk.start(a, tok, blockIdx.x, gridDim.x)) return;
  const PrefixPos<PREFIX_N>& pos = walk.pos;
  const size_t width = (size_t)a.kv_heads * HD;
  const float sl = a.scale * 1.4426950408889634f;  // scores in log2 units
  do {
    walk.publish(a, threadIdx.x, C::THREADS);
    const int b0 = walk.b0, b1 = b0 + walk.n;
    const int rows = pos.nrow * group;
    const int np = pos.g.np, nk = np + pos.tail.y - pos.tail.x;
    const __nv_bfloat16* kc = (const __nv_bfloat16*)a.cache + (size_t)pos.kh * HD;
    // one key's slot of block b, for threads 0 .. PREFIX_N - 1
    auto fetch = [&](int b) -> int {
      const int x = b * PREFIX_N + (int)threadIdx.x;
      int s = -1;
      if (b < b1) {
        if (x < np) s = a.prefix[pos.g.p0 + x];
        else if (x < nk) s = a.tail[x - np + pos.tail.x];
      }
      return s >= 0 && s < a.n_slots ? s : -1;
    };
    auto put = [&](int b, int s) {
      const unsigned v = __ballot_sync(0xffffffffu, s >= 0);
      sslot[b & (C::RING - 1)][threadIdx.x] = s;
      if (lane == 0) svalid[b & (C::RING - 1)][warp] = v;
    };
    auto load = [&](int b) {  // K and V rows of block b into its stage
      const uint32_t st = smem + (uint32_t)((b - b0) % C::STAGES) * C::STAGE;
      constexpr int PIECES = HD / 8;  // 16-byte pieces of a row
#pragma unroll
      for (int e = threadIdx.x; e < PREFIX_N * PIECES; e += C::THREADS) {
        const int j = e / PIECES, c = e % PIECES, s = sslot[b & (C::RING - 1)][j];
        const __nv_bfloat16* src = kc + (size_t)max(s, 0) * 2 * width + c * 8;
        const uint32_t dst = st + j * C::PITCH + c * 16;
        cp_async16(dst, src, s >= 0);
        cp_async16(dst + PREFIX_N * C::PITCH, src + width, s >= 0);
      }
    };
    __syncthreads();  // the previous tile's ring and slot lists are consumed
    int ahead = -1;   // slot of block b + STAGES, fetched one block before it is put down
    if (warp < 2) {
#pragma unroll
      for (int i = 0; i < C::STAGES; ++i) put(b0 + i, fetch(b0 + i));
      ahead = fetch(b0 + C::STAGES);
    }
    // query fragments and the rows' tail keys
    uint32_t q[HD / 16][4];
    int2 mine[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = wm * 16 + gr + h * 8;
      const bool have = r < rows;
      mine[h] = {0, 0};
      const __nv_bfloat16* p = (const __nv_bfloat16*)a.q;
      if (have) {
        const int row = pos.row0 + r / group;
        const int2 t = off_range(a.tail_off, row, a.n_tail, a.status);
        mine[h] = {np + t.x - pos.tail.x, np + t.y - pos.tail.x};
        p += (size_t)row * a.sq + (size_t)(pos.kh * group + r % group) * HD + gc;
      }
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        q[i][h] = have ? *reinterpret_cast<const uint32_t*>(p + i * 16) : 0u;
        q[i][h + 2] = have ? *reinterpret_cast<const uint32_t*>(p + i * 16 + 8) : 0u;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      if (b0 + i < b1) load(b0 + i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    bool poison = false;
    for (int b = b0; b < b1; ++b) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
      __syncthreads();
      if (b + C::STAGES - 1 < b1) load(b + C::STAGES - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (warp < 2) {
        put(b + C::STAGES, ahead);
        ahead = fetch(b + C::STAGES + 1);
      }
      const uint32_t st = smem + (uint32_t)((b - b0) % C::STAGES) * C::STAGE;
      const uint32_t ks = st + wk * C::KEYS * C::PITCH, vs = ks + PREFIX_N * C::PITCH;
      float s[C::KEYS / 8][4];
#pragma unroll
      for (int j = 0; j < C::KEYS / 16; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[2 * j][e] = s[2 * j + 1][e] = 0.f;
        // matrices: keys 0-7 / 8-15 of the slice by columns 0-7 / 8-15
        const uint32_t at = ks + (j * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * C::PITCH + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          uint32_t k[4];
          ldsm4(at + i * 32, k);
          mma16816(s[2 * j], q[i], k[0], k[1]);
          mma16816(s[2 * j + 1], q[i], k[2], k[3]);
        }
      }
      const uint32_t v0 = svalid[b & (C::RING - 1)][0], v1 = svalid[b & (C::RING - 1)][1];
      const bool tailed = (b + 1) * PREFIX_N > np;
      if (tailed || (v0 & v1) != 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < C::KEYS / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = wk * C::KEYS + j * 8 + gc + (e & 1), x = b * PREFIX_N + c;
            const bool there = ((c < 32 ? v0 >> c : v1 >> (c - 32)) & 1u) != 0;
            const int2 w = mine[e >> 1];
            if (!there || !(x < np || (x >= w.x && x < w.y))) s[j][e] = -INFINITY;
          }
      }
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < C::KEYS / 8; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * h], s[j][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[h], mx * sl);
        f[h] = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
        m[h] = mn;
        const float ms = mn == -INFINITY ? 0.f : mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < C::KEYS / 8; ++j)
#pragma unroll
          for (int e = 2 * h; e < 2 * h + 2; ++e) {
            s[j][e] = ex2(fmaf(s[j][e], sl, -ms));
            sum += s[j][e];
          }
        l[h] = l[h] * f[h] + sum;
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= f[e >> 1];
      }
#pragma unroll
      for (int j = 0; j < C::KEYS / 16; ++j) {
        uint32_t p[4];
        p[0] = pack_bf16(s[2 * j][0], s[2 * j][1]);
        p[1] = pack_bf16(s[2 * j][2], s[2 * j][3]);
        p[2] = pack_bf16(s[2 * j + 1][0], s[2 * j + 1][1]);
        p[3] = pack_bf16(s[2 * j + 1][2], s[2 * j + 1][3]);
        // matrices: keys 0-7 / 8-15 of the slice by columns 0-7 / 8-15, transposed
        const uint32_t at = vs + (j * 16 + (lane & 15)) * C::PITCH + ((lane >> 4) & 1) * 16;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          uint32_t v[4];
          ldsm4_t(at + i * 32, v);
          if (tailed) {
            // Tail values belong to one row each: infinities and NaN stay out of the products
            // (0 * inf is NaN) and go to their rows below.
#pragma unroll
            for (int e = 0; e < 4; ++e) poison |= drop_nonfinite(v[e]);
          }
          mma16816(o[2 * i], p, v[0], v[1]);
          mma16816(o[2 * i + 1], p, v[2], v[3]);
        }
      }
    }
    if (__any_sync(0xffffffffu, poison)) {
      for (int x = max(b0, np / PREFIX_N) * PREFIX_N; x < min(b1 * PREFIX_N, nk); ++x) {
        const int c = x % PREFIX_N;
        if (c / C::KEYS != wk) continue;
        const int s = x < np ? a.prefix[pos.g.p0 + x] : a.tail[x - np + pos.tail.x];
        if (s < 0 || s >= a.n_slots) continue;
        const __nv_bfloat16* v = kc + ((size_t)s * 2 + 1) * width + gc;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = __bfloat162float(v[i * 8 + (e & 1)]);
            const int2 w = mine[e >> 1];
            if (!(fabsf(y) < INFINITY) && (x < np || (x >= w.x && x < w.y))) o[i][e] += y;
          }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    const size_t part = (size_t)(blockIdx.x + pos.t);
    if (C::WK == 1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = wm * 16 + gr + h * 8;
        if (r >= rows) continue;
        if ((lane & 3) == 0) a.part_ml[part * MT + r] = make_float2(m[h], l[h]);
        float* dst = a.part + (part * MT + r) * HD + gc;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
      }
    } else {
      // merge of the WK key slices: through shared memory, in slice order
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      float* so = reinterpret_cast<float*>(smem_raw);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = gr + h * 8;
        if ((lane & 3) == 0) sml[warp][r] = make_float2(m[h], l[h]);
        float* dst = so + (warp * 16 + r) * (HD + 4) + gc;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < rows * (HD / 4); e += C::THREADS) {
        const int r = e / (HD / 4), c = (e % (HD / 4)) * 4, w0 = (r >> 4) * C::WK, rr = r & 15;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < C::WK; ++k) M = fmaxf(M, sml[w0 + k][rr].x);
        const float ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < C::WK; ++k) {
          const float2 ml = sml[w0 + k][rr];
          const float w = ex2(ml.x - ms);
          const float4 v = *reinterpret_cast<const float4*>(so + ((w0 + k) * 16 + rr) * (HD + 4) + c);
          L += w * ml.y;
          acc.x = fmaf(w, v.x, acc.x);
          acc.y = fmaf(w, v.y, acc.y);
          acc.z = fmaf(w, v.z, acc.z);
          acc.w = fmaf(w, v.w, acc.w);
        }
        if (c == 0) a.part_ml[part * MT + r] = make_float2(M, L);
        *reinterpret_cast<float4*>(a.part + (part * MT + r) * HD + c) = acc;
      }
    }
  } while (walk.next(a, tok));
}

}  // namespace lt

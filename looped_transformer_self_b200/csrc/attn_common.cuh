// Shared parts of the stand-alone attention operators (lt_attn_prompt,
// lt_attn_prefix): which rows and keys a tile covers, the fp32 tile kernel's
// arithmetic, and small host helpers.
//
// Query rows are packed: the G = n_heads / n_kv_heads query heads that read one
// key/value head sit side by side in a tile, so that a key/value row is loaded
// once for all of them.  Packed row r of a tile is (token or branch r / G,
// head r % G within the group).
#pragma once

#include "common.cuh"

namespace lt {

constexpr int ATTN_MAX_GROUP = 64;  // query heads per key/value head (they share a 64-row tile)
constexpr int COUNT_MAX = 0x7fffffff - 1023;  // rows or keys: kernels count some blocks past them in 32 bits

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// The element range of entry i of an offset array, clamped into [0, n] and
// ascending.  Offsets that had to be clamped are reported once in `status`.
__device__ __forceinline__ int2 off_range(const int32_t* off, int i, int n, int* status) {
  const int a = off[i], b = off[i + 1];
  int2 r = {min(max(a, 0), n), min(max(b, 0), n)};
  r.y = max(r.x, r.y);
  if (r.x != a || r.y != b) set_err(status, DEV_BAD_INDEX);
  return r;
}

// ---- one tile of attention in fp32 (256 threads, 64 packed rows x 64 keys) ----
// The flash recurrence: with m the running row maximum and l the running sum,
// a block of scores s gives m' = max(m, max s), p = exp(s - m'),
// l' = l exp(m - m') + sum p, O' = O exp(m - m') + p V.  Thread (ty, tx) of a
// 16 x 16 grid holds scores of rows 4 ty + i and keys tx + 16 j, and output
// columns 2 tx + 32 c.  A block's keys are copied while the block before is
// multiplied with its values and its values during its scores (cp.async); at
// head size 128 the four arrays are just half of an SM's shared memory, so two
// CTAs fit.
constexpr int SIMT_M = 64, SIMT_N = 64, SIMT_THREADS = 256;

template <int HD>
struct SimtSmem {
  float k[SIMT_N][HD + 4];  // pitch HD + 4: eight rows read as float4 touch all banks once
  float q[SIMT_M][HD];
  float v[SIMT_N][HD];
  float p[SIMT_M][SIMT_N];  // column c of row r at c ^ 16 (r / 4 % 2): a warp's two row groups in different banks
};
__device__ __forceinline__ int simt_p_col(int r, int c) { return c ^ ((r >> 2 & 1) << 4); }

// Row state of one tile: 4 rows per thread, replicated over the 16 threads of a row.
template <int HD>
struct SimtState {
  float m[4], l[4], o[4][HD / 16];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) o[i][c] = 0.f;
    }
  }
};

// Copies the tile's query rows (scaled) to shared memory; rows without a pointer are zero.
template <int HD, typename RowPtr>
__device__ __forceinline__ void simt_load_q(SimtSmem<HD>& sm, RowPtr row, float scale) {
  for (int e = threadIdx.x; e < SIMT_M * (HD / 4); e += SIMT_THREADS) {
    const int r = e / (HD / 4), c = (e % (HD / 4)) * 4;
    const float* p = row(r);
    float4 v = p ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
    *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
  }
}
// Starts the copy of 64 rows (a copy group of its own); rows without a pointer become zero.  `any`:
// a valid address, not read for those.
template <int HD, int PITCH, typename RowPtr>
__device__ __forceinline__ void simt_fetch(float* dst, RowPtr row, const float* any) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  for (int e = threadIdx.x; e < SIMT_N * (HD / 4); e += SIMT_THREADS) {
    const int r = e / (HD / 4), c = (e % (HD / 4)) * 4;
    const float* p = row(r);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (r * PITCH + c) * 4),
                 "l"(p ? p + c : any), "r"(p ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void simt_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void simt_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// O += P V of one block.  GUARD: the weight of a key that the row does not see
// is -0, which takes nothing from its value row, so that an infinity or NaN
// there stays out (0 * inf is NaN).  A key that it sees with a finite score has a
// weight of +0 at the least, and its value reaches the row.
template <int HD, bool GUARD>
__device__ __forceinline__ void simt_pv(SimtSmem<HD>& sm, SimtState<HD>& st) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
  for (int k = 0; k < SIMT_N; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = *reinterpret_cast<const float4*>(&sm.p[ty * 4 + i][simt_p_col(ty * 4, k)]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        const float2 v = *reinterpret_cast<const float2*>(&sm.v[k + u][tx * 2 + 32 * c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
          const bool take = !GUARD || (int)__float_as_uint(w) >= 0;  // not -0
          st.o[i][2 * c] = fmaf(w, take ? v.x : 0.f, st.o[i][2 * c]);
          st.o[i][2 * c + 1] = fmaf(w, take ? v.y : 0.f, st.o[i][2 * c + 1]);
        }
      }
  }
}

// One block of 64 keys whose copies were started as the group before last (keys) and the last
// (values).  `seen(r, j)` says whether packed row r sees key j; `masked` (uniform): some row may not
// see some key of the block.  next_k() / next_v() start the next block's copies, a group each (empty
// at the end), where their buffers are free; before_k() runs between the scores and next_k, with a
// barrier on both sides.
template <int HD, typename Seen, typename Before, typename NextK, typename NextV>
__device__ __forceinline__ void simt_block(SimtSmem<HD>& sm, SimtState<HD>& st, Seen seen, bool masked,
                                           Before before_k, NextK next_k, NextV next_v) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  simt_wait1();
  __syncthreads();
  float s[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < HD; d += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&sm.q[ty * 4 + i][d]);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][d]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
        s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
        s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
        s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!seen(ty * 4 + i, tx + 16 * j)) s[i][j] = -INFINITY;
  before_k();
  __syncthreads();  // the keys are consumed
  next_k();
  simt_commit();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(st.m[i], mx);
    const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every p is 0
    const float f = expf(st.m[i] - ms);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e = expf(s[i][j] - ms), p = masked && s[i][j] == -INFINITY ? -0.f : e;
      sum += p;
      sm.p[r][simt_p_col(r, tx + 16 * j)] = p;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    st.l[i] = st.l[i] * f + sum;
    st.m[i] = mn;
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) st.o[i][c] *= f;
  }
  simt_wait1();
  __syncthreads();  // P is complete, the values are there
  if (masked)
    simt_pv<HD, true>(sm, st);
  else
    simt_pv<HD, false>(sm, st);
  __syncthreads();  // the values are consumed
  next_v();
  simt_commit();
}

// ---- host helpers --------------------------------------------------------------
inline bool attn_shape_ok(int n_heads, int n_kv_heads, int head_dim) {
  if (head_dim != 32 && head_dim != 64 && head_dim != 96 && head_dim != 128) return false;
  return n_kv_heads > 0 && n_kv_heads <= 1024 && n_heads > 0 && n_heads % n_kv_heads == 0 &&
         n_heads / n_kv_heads <= ATTN_MAX_GROUP;
}
// Launches with programmatic dependence on the work before it on the stream: the kernel may start
// while that drains, and waits for it (pdl_wait) before it reads or writes global memory.  What it reads
// may be written while it already runs, so its loads are ordinary ones: __ldg is for memory that nothing
// writes in a kernel's lifetime, and the compiler may move it in front of the wait.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid_x, unsigned grid_y, int threads, size_t smem,
                              cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Lets kernel K take `bytes` of dynamic shared memory (the attribute belongs to a device).
template <auto K>
inline cudaError_t allow_smem(size_t bytes) {
  static bool set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) set[dev] = true;
  return e;
}
// Rows start on 16-byte boundaries (vector loads and TMA).
inline bool attn_aligned(int dtype, const void* p, long long stride) {
  return ((uintptr_t)p & 15) == 0 && (stride * (dtype == 0 ? 4 : 2)) % 16 == 0;
}
inline int attn_sm_count() {
  static int cached[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 148;
  if (!cached[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = n > 0 ? n : 148;
  }
  return cached[dev];
}

}  // namespace lt

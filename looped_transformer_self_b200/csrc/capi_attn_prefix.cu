// Attention of a batch of rows that share long prefixes over the slot cache:
// the keys of a group's prefix are read once for all of its rows (the branches
// of one committed prefix, or the samples of one prompt), and each row's own
// tail is read for it alone.
#include "../../include/looped_spec.h"
#include "attn_prefix_mma.cuh"

namespace lt {

// fp32 arithmetic throughout (CUDA cores): the form of fp32 models.  Bound by
// its start, the partition and one block's chain where the cache is short (2 and
// 9 rows on 777 and 289 shared slots, 4 heads of 32: 12 to 13 us with the merge).
// Two CTAs per SM leave 128 registers a thread, which the walk and the tile pass by
// about 70, 150 and 220 bytes of spills at head sizes 64, 96 and 128.
template <int HD>
__global__ void __launch_bounds__(SIMT_THREADS, 2) k_attn_prefix_simt(PrefixArgs a) {
  extern __shared__ __align__(16) char smem_raw[];
  SimtSmem<HD>& sm = *reinterpret_cast<SimtSmem<HD>*>(smem_raw);
  // The slots of two blocks' keys stand in the key rows' padding: two CTAs fill an SM's shared memory.
  auto slot_at = [&](int b, int j) -> int& { return reinterpret_cast<int&>(sm.k[j][HD + (b & 1)]); };
  const int tok = SIMT_M / a.group, group = a.group;
  pdl_trigger();
  pdl_wait();
  PrefixWalk<PREFIX_N> walk;
  if (!walk.start(a, tok, blockIdx.x, gridDim.x)) return;
  const PrefixPos<PREFIX_N>& pos = walk.pos;
  const size_t width = (size_t)a.kv_heads * HD;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  do {
    walk.publish(a, threadIdx.x, SIMT_THREADS);
    const int b0 = walk.b0, b1 = b0 + walk.n;
    const int rows = pos.nrow * group, h0 = pos.kh * group;
    const float* q = (const float*)a.q + (size_t)pos.row0 * a.sq + (size_t)h0 * HD;
    const int np = pos.g.np, nk = np + pos.tail.y - pos.tail.x;
    const float* kc = (const float*)a.cache + (size_t)pos.kh * HD;
    auto slot_of = [&](int b) {  // of this thread's key of block b
      const int x = b * PREFIX_N + threadIdx.x;
      int s = -1;
      if (threadIdx.x < PREFIX_N && b < b1) {
        if (x < np) s = a.prefix[pos.g.p0 + x];
        else if (x < nk) s = a.tail[x - np + pos.tail.x];
      }
      return s >= 0 && s < a.n_slots ? s : -1;
    };
    auto put = [&](int b, int s) {
      if (threadIdx.x < PREFIX_N) slot_at(b, threadIdx.x) = s;
    };
    auto fetch_k = [&](int b) {
      if (b < b1)
        simt_fetch<HD, HD + 4>(&sm.k[0][0], [&](int j) {
          const int s = slot_at(b, j);
          return s >= 0 ? kc + (size_t)s * 2 * width : nullptr;
        }, q);
    };
    auto fetch_v = [&](int b) {
      if (b < b1)
        simt_fetch<HD, HD>(&sm.v[0][0], [&](int j) {
          const int s = slot_at(b, j);
          return s >= 0 ? kc + ((size_t)s * 2 + 1) * width : nullptr;
        }, q);
    };
    __syncthreads();  // the previous tile is done with the shared arrays
    put(b0, slot_of(b0));
    __syncthreads();
    fetch_k(b0);
    simt_commit();
    fetch_v(b0);
    simt_commit();
    simt_load_q<HD>(sm, [&](int r) {
      return r < rows ? q + (size_t)(r / group) * a.sq + (r % group) * HD : nullptr;
    }, a.scale);
    int2 mine[4];  // tail entries of this thread's rows, as key indices of the tile
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      mine[i] = {0, 0};
      if (r < rows) {
        const int2 t = off_range(a.tail_off, pos.row0 + r / group, a.n_tail, a.status);
        mine[i] = {np + t.x - pos.tail.x, np + t.y - pos.tail.x};
      }
    }
    SimtState<HD> st;
    st.clear();
    for (int b = b0; b < b1; ++b) {
      const int x0 = b * PREFIX_N, next = slot_of(b + 1);
      simt_block<HD>(
          sm, st,
          [&](int r, int j) {
            const int2 m = mine[r & 3];
            return slot_at(b, j) >= 0 && (x0 + j < np || (x0 + j >= m.x && x0 + j < m.y));
          },
          x0 + PREFIX_N > np, [&] { put(b + 1, next); }, [&] { fetch_k(b + 1); }, [&] { fetch_v(b + 1); });
    }
    const size_t part = (size_t)(blockIdx.x + pos.t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      if (tx == 0) a.part_ml[part * SIMT_M + r] = make_float2(st.m[i] * 1.4426950408889634f, st.l[i]);
      float* o = a.part + (part * SIMT_M + r) * HD;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c)
        *reinterpret_cast<float2*>(o + tx * 2 + 32 * c) = make_float2(st.o[i][2 * c], st.o[i][2 * c + 1]);
    }
  } while (walk.next(a, tok));
}

// N consecutive values, moved at once where N is a power of two.
template <typename T, int N>
struct alignas(N == 3 ? sizeof(T) : N * sizeof(T)) MergeVec {
  T x[N];
};

// Merge of a row's partials: with M the largest m, o = sum_i 2^(m_i - M) O_i /
// sum_i 2^(m_i - M) l_i.  One warp per (row, head); bound by
// its chain of table, maxima and partials (3 us, 5 us for 19 partials of 64 rows of 32
// heads).
template <typename T, int HD, int MT>
__global__ void __launch_bounds__(256) k_attn_prefix_merge(PrefixArgs a, int grid) {
  constexpr int PER = HD / 32;
  const int row = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (h >= a.heads) return;
  pdl_wait();
  // rows before the first group or behind the last one are left as they were
  const int first = max(*a.row_off, 0), last = min(a.row_off[a.n_groups], a.n_rows);
  const int4 rt = a.row_tab[row];  // asked for together with the offsets
  if (row < first || row >= last) return;
  PrefixPlace at;
  if (!prefix_place(rt, h, a.group, a.max_tiles, MT, at) || !prefix_parts(a.tile_tab[at.t], grid, at)) {
    set_err(a.status, DEV_BAD_INDEX);  // rows that the offsets do not reach
    return;
  }
  float M = -INFINITY, l = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  constexpr int B = 16;  // partials in flight
  for (int k0 = 0; k0 < at.parts; k0 += B) {
    float2 ml[B];
    MergeVec<float, PER> v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const bool there = k0 + k < at.parts;
      const size_t p = (size_t)(at.first + (k0 + k) / at.two + at.t) * MT + (k0 + k) % at.two * (MT / 2) + at.r;
      ml[k] = there ? a.part_ml[p] : make_float2(-INFINITY, 0.f);
      v[k] = {};
      if (there) v[k] = *reinterpret_cast<const MergeVec<float, PER>*>(a.part + p * HD + lane * PER);
    }
    float mx = M;
#pragma unroll
    for (int k = 0; k < B; ++k) mx = max_nan(mx, ml[k].x);
    const float ms = mx == -INFINITY ? 0.f : mx, f = ex2(M - ms);  // nothing seen yet: the sum is 0
    M = mx;
    l *= f;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] *= f;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      // A partial that saw nothing has no outputs.  NaN scores alone leave no maximum either, but a NaN
      // sum, which has to reach the row.
      if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
      const float w = ex2(ml[k].x - ms);
      l += w * ml[k].y;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = fmaf(w, v[k].x[i], o[i]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  MergeVec<T, PER> out;
#pragma unroll
  for (int i = 0; i < PER; ++i) out.x[i] = from_f<T>(o[i] * inv);
  *reinterpret_cast<MergeVec<T, PER>*>((T*)a.o + (size_t)row * a.so + (size_t)h * HD + lane * PER) = out;
}

template <typename T, int HD, int MT>
static cudaError_t prefix_merge(const PrefixArgs& a, int grid, cudaStream_t st) {
  return launch_pdl(k_attn_prefix_merge<T, HD, MT>, a.n_rows, cdiv(a.heads, 8), 256, 0, st, a, grid);
}

template <int HD>
static cudaError_t prefix_f32(const PrefixArgs& a, int grid, cudaStream_t st) {
  if (cudaError_t e = allow_smem<k_attn_prefix_simt<HD>>(sizeof(SimtSmem<HD>))) return e;
  if (cudaError_t e = launch_pdl(k_attn_prefix_simt<HD>, grid, 1, SIMT_THREADS, sizeof(SimtSmem<HD>), st, a))
    return e;
  return prefix_merge<float, HD, SIMT_M>(a, grid, st);
}

template <int HD, int MT>
static cudaError_t prefix_mma(const PrefixArgs& a, int grid, cudaStream_t st) {
  using C = PrefixMma<HD, MT>;
  if (cudaError_t e = allow_smem<k_attn_prefix_mma<HD, MT>>(C::SMEM)) return e;
  if (cudaError_t e = launch_pdl(k_attn_prefix_mma<HD, MT>, grid, 1, C::THREADS, C::SMEM, st, a)) return e;
  return prefix_merge<__nv_bfloat16, HD, MT>(a, grid, st);
}

template <int HD>
static cudaError_t prefix_tc(const PrefixArgs& a, int grid, cudaStream_t st) {
  using W = PrefixWork;
  CUtensorMap mq;
  if (attn_tmap(&mq, a.q, HD, a.heads, a.n_rows, a.sq, a.group, 128 / a.group, 1)) return cudaErrorInvalidValue;
  if (cudaError_t e = allow_smem<k_attn_tc<HD, W>>(tc_smem<HD, W>())) return e;
  if (cudaError_t e = launch_pdl(k_attn_tc<HD, W>, grid, 1, W::THREADS, tc_smem<HD, W>(), st, a, mq, mq, mq)) return e;
  return prefix_merge<__nv_bfloat16, HD, 256>(a, grid, st);
}

template <int HD>
static cudaError_t prefix_any(int dtype, int mt, const PrefixArgs& a, int grid, cudaStream_t st) {
  if (dtype == LT_F32) return prefix_f32<HD>(a, grid, st);
  switch (mt) {
    case 16: return prefix_mma<HD, 16>(a, grid, st);
    case 32: return prefix_mma<HD, 32>(a, grid, st);
    case 64: return prefix_mma<HD, 64>(a, grid, st);
    default: return prefix_tc<HD>(a, grid, st);
  }
}

// Scratch layout: tile table, row table, (m, l) pairs, partial outputs.
struct PrefixPlan {
  int mt, grid;
  long long max_tiles;
  size_t row_at, ml_at, part_at, bytes;
};
static PrefixPlan prefix_plan(int mt, int n_rows, int n_groups, int n_heads, int n_kv_heads, int hd) {
  PrefixPlan p;
  const int group = n_heads / n_kv_heads, tok = mt == 256 ? 2 * (128 / group) : mt / group;
  p.mt = mt;
  p.grid = (mt == 256 ? 1 : 2) * attn_sm_count();
  p.max_tiles = (long long)n_kv_heads * (n_rows / tok + (long long)n_groups);
  const size_t slots = (size_t)p.max_tiles + p.grid;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.row_at = up((size_t)p.max_tiles * sizeof(int4));
  p.ml_at = p.row_at + up((size_t)n_rows * sizeof(int4));
  p.part_at = p.ml_at + up(slots * mt * sizeof(float2));
  p.bytes = p.part_at + up(slots * mt * (size_t)hd * sizeof(float));
  return p;
}
// The smallest tile of the few-rows kernels that holds an average group's packed rows (a group may
// take several tiles).
static int prefix_small_tile(int dtype, int n_rows, int n_groups, int group) {
  const long long avg = (long long)group * n_rows / (n_groups > 0 ? n_groups : 1);
  if (dtype == LT_F32) return SIMT_M;
  return avg <= 16 && group <= 16 ? 16 : avg <= 32 && group <= 32 ? 32 : 64;
}
// The tensor-core tiles (256 packed rows) cost up to 4 us more to start and less per key; the more
// rows the few-rows kernel holds, the fewer keys it takes to make that up.  The sizes are those that the
// host knows: the lengths of the lists, not what the offsets take of them.  Measured at head size 128
// (few rows / tiles, us): 16 heads, 1 row, 2500 keys 13.0 / 16.7, 6000 keys 22.2 / 22.4, 10000 keys
// 30.3 / 29.1, 20000 keys 48.4 / 42.3; 32 rows, 1000 keys 13.8 / 14.1, 2500 keys 16.6 / 17.7, 3500 keys
// 20.4 / 19.2, 6000 keys 27.4 / 23.2; 64 rows, 400 keys 14.3 / 13.7, 600 keys 14.3 / 14.2; 32 heads on 8,
// 32 rows (128 packed), 300 keys 14.2 / 13.3, 1000 keys 16.6 / 15.0, 20000 keys 74.1 / 35.4.  Near the
// bounds the two differ by a microsecond either way.  Smaller heads make fewer bytes of a key, and the
// tiles come a little early: 1 row of 55 heads of 96, 4000 keys 32.4 / 33.9; 16 heads of 32, 10000 keys
// 15.2 / 20.7; 8 heads of 64 on 2, 8 rows, 30000 keys 20.2 / 23.8, 80000 keys 32.8 / 33.1.
static bool prefix_use_tc(int mt, long long keys, int n_kv_heads) {
  return keys * n_kv_heads >= (mt == 64 ? 8000 : mt == 32 ? 48000 : 160000);
}

}  // namespace lt

using namespace lt;

extern "C" int lt_attn_prefix_scratch_bytes(int dtype, int n_rows, int n_groups, int n_heads,
                                            int n_kv_heads, int head_dim, size_t* bytes) {
  if (!bytes || (dtype != LT_F32 && dtype != LT_BF16) || n_rows < 0 || n_groups < 0) return LT_ERR_ARG;
  if (!attn_shape_ok(n_heads, n_kv_heads, head_dim) || n_rows > 65535) return LT_ERR_SHAPE;
  const int small = prefix_small_tile(dtype, n_rows, n_groups, n_heads / n_kv_heads);
  const PrefixPlan p = prefix_plan(small, n_rows, n_groups, n_heads, n_kv_heads, head_dim);
  if (p.max_tiles > (1 << 30)) return LT_ERR_SHAPE;
  *bytes = p.bytes;
  if (dtype == LT_BF16) {  // either kernel may run: the number of keys decides
    const size_t tc = prefix_plan(256, n_rows, n_groups, n_heads, n_kv_heads, head_dim).bytes;
    if (tc > *bytes) *bytes = tc;
  }
  return LT_OK;
}

extern "C" int lt_attn_prefix(int dtype, const void* d_q, long long stride_q, const void* d_cache,
                              int n_slots, void* d_o, long long stride_o, const int32_t* d_row_off,
                              int n_groups, int n_rows, const int32_t* d_prefix,
                              const int32_t* d_prefix_off, int n_prefix, const int32_t* d_tail,
                              const int32_t* d_tail_off, int n_tail, int n_heads, int n_kv_heads,
                              int head_dim, float scale, void* d_scratch, size_t scratch_bytes,
                              int32_t* d_status, void* stream) {
  size_t need = 0;
  const int e = lt_attn_prefix_scratch_bytes(dtype, n_rows, n_groups, n_heads, n_kv_heads, head_dim, &need);
  if (e != LT_OK) return e;
  if (n_slots < 0 || n_prefix < 0 || n_tail < 0 || !(scale > 0.f) || !(scale < INFINITY)) return LT_ERR_ARG;
  if ((long long)n_prefix + n_tail > COUNT_MAX) return LT_ERR_SHAPE;
  if (n_rows == 0 || n_groups == 0) return LT_OK;
  if (!d_q || !d_o || !d_row_off || !d_prefix_off || !d_tail_off || !d_scratch ||
      (n_slots > 0 && !d_cache) || (n_prefix > 0 && !d_prefix) || (n_tail > 0 && !d_tail))
    return LT_ERR_ARG;
  const long long w = (long long)n_heads * head_dim;
  if (stride_q < w || stride_o < w) return LT_ERR_ARG;
  if (!attn_aligned(dtype, d_q, stride_q) || !attn_aligned(dtype, d_o, stride_o) ||
      ((uintptr_t)d_cache & 15) || ((uintptr_t)d_scratch & 31))
    return LT_ERR_SHAPE;
  if (scratch_bytes < need) return LT_ERR_CAPACITY;
  int mt = prefix_small_tile(dtype, n_rows, n_groups, n_heads / n_kv_heads);
  if (dtype == LT_BF16 && prefix_use_tc(mt, (long long)n_prefix + n_tail, n_kv_heads)) mt = 256;
  const PrefixPlan p = prefix_plan(mt, n_rows, n_groups, n_heads, n_kv_heads, head_dim);
  // the kernels count blocks of all tiles in 32 bits
  if ((((long long)n_prefix + n_tail) / PREFIX_N + 1) * p.max_tiles > (1 << 30)) return LT_ERR_SHAPE;
  char* s = (char*)d_scratch;
  PrefixArgs a = {d_q, d_cache, d_o, stride_q, stride_o, d_row_off, d_prefix, d_prefix_off, d_tail,
                  d_tail_off, n_groups, n_rows, n_slots, n_prefix, n_tail, n_heads, n_kv_heads,
                  n_heads / n_kv_heads, scale, (int4*)s,
                  (int4*)(s + p.row_at), (float2*)(s + p.ml_at), (float*)(s + p.part_at),
                  (int)p.max_tiles, d_status};
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t r;
  switch (head_dim) {
    case 32: r = prefix_any<32>(dtype, p.mt, a, p.grid, st); break;
    case 64: r = prefix_any<64>(dtype, p.mt, a, p.grid, st); break;
    case 96: r = prefix_any<96>(dtype, p.mt, a, p.grid, st); break;
    default: r = prefix_any<128>(dtype, p.mt, a, p.grid, st); break;
  }
  return r == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

// Causal attention over whole prompts: packed sequences of different lengths,
// grouped heads, keys that may start before the queries (a prompt taken in
// pieces).  Query t of a sequence with lq queries and lk keys sees keys
// 0 .. lk - lq + t.
#include "../../include/looped_spec.h"
#include "attn_tc_kernel.cuh"

namespace lt {

// fp32 arithmetic throughout (CUDA cores): the form of fp32 models.  A tile of
// 64 rows per CTA keeps its keys' and values' copies under the arithmetic; bound
// by the chain of blocks of the longest tile where tiles are few (9 sequences, 700
// tokens in all, 4 heads of 32: 60 CTAs of work, 23.5 us).
template <int HD>
__global__ void __launch_bounds__(SIMT_THREADS, 2) k_attn_prompt_simt(PromptArgs a) {
  extern __shared__ __align__(16) char smem_raw[];
  SimtSmem<HD>& sm = *reinterpret_cast<SimtSmem<HD>*>(smem_raw);
  const int kh = blockIdx.x % a.kv_heads, tok = SIMT_M / a.group;
  pdl_trigger();
  pdl_wait();
  PromptTile pt;
  if (!prompt_tile(a, blockIdx.x / a.kv_heads, tok, pt)) return;
  const int t0 = pt.tile * tok, nt = min(tok, pt.lq - t0), rows = nt * a.group;
  const int ctx = pt.lk - pt.lq;  // keys before the first query
  const int group = a.group, h0 = kh * group;
  const float* q = (const float*)a.q + (size_t)(pt.q0 + t0) * a.sq + (size_t)h0 * HD;
  const float* k = (const float*)a.k + (size_t)pt.k0 * a.sk + (size_t)kh * HD;
  const float* v = (const float*)a.v + (size_t)pt.k0 * a.sv + (size_t)kh * HD;
  const int see_first = ctx + t0 + 1, see_last = min(ctx + t0 + nt, pt.lk);  // keys of the first / last row
  auto fetch_k = [&](int b) {
    if (b < see_last)
      simt_fetch<HD, HD + 4>(&sm.k[0][0],
                             [&](int j) { return b + j < see_last ? k + (size_t)(b + j) * a.sk : nullptr; }, q);
  };
  auto fetch_v = [&](int b) {
    if (b < see_last)
      simt_fetch<HD, HD>(&sm.v[0][0],
                         [&](int j) { return b + j < see_last ? v + (size_t)(b + j) * a.sv : nullptr; }, q);
  };
  fetch_k(0);
  simt_commit();
  fetch_v(0);
  simt_commit();
  simt_load_q<HD>(sm, [&](int r) {
    return r < rows ? q + (size_t)(r / group) * a.sq + (r % group) * HD : nullptr;
  }, a.scale);
  SimtState<HD> st;
  st.clear();
  for (int b = 0; b < see_last; b += SIMT_N) {
    simt_block<HD>(
        sm, st, [&](int r, int j) { return b + j <= ctx + t0 + r / group && b + j < see_last; },
        b + SIMT_N > see_first, [] {}, [&] { fetch_k(b + SIMT_N); }, [&] { fetch_v(b + SIMT_N); });
  }
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    if (r >= rows) continue;
    const float inv = st.l[i] > 0.f ? 1.f / st.l[i] : st.l[i] == 0.f ? 0.f : st.l[i];
    float* o = (float*)a.o + (size_t)(pt.q0 + t0 + r / group) * a.so + (size_t)(h0 + r % group) * HD;
#pragma unroll
    for (int c = 0; c < HD / 32; ++c)
      *reinterpret_cast<float2*>(o + tx * 2 + 32 * c) = make_float2(st.o[i][2 * c] * inv, st.o[i][2 * c + 1] * inv);
  }
}

template <int HD>
static cudaError_t prompt_simt(const PromptArgs& a, cudaStream_t st) {
  const int tok = SIMT_M / a.group;
  const unsigned tiles = (unsigned)(a.n_q / tok + a.n_seqs);
  if (cudaError_t e = allow_smem<k_attn_prompt_simt<HD>>(sizeof(SimtSmem<HD>))) return e;
  return launch_pdl(k_attn_prompt_simt<HD>, tiles * a.kv_heads, 1, SIMT_THREADS, sizeof(SimtSmem<HD>), st, a);
}

template <int HD>
static int prompt_tc(const PromptArgs& a, cudaStream_t st) {
  using W = PromptWork;
  const int tok = 128 / a.group;
  CUtensorMap mq, mk, mv;
  // no keys: nothing is loaded, and the maps stand on the queries
  const void* k = a.n_kv > 0 ? a.k : a.q;
  const void* v = a.n_kv > 0 ? a.v : a.q;
  const long long nk = a.n_kv > 0 ? a.n_kv : 1;
  if (attn_tmap(&mq, a.q, HD, a.heads, a.n_q, a.sq, a.group, tok, 1) ||
      attn_tmap(&mk, k, HD, a.kv_heads, nk, a.sk, 1, 128, 2) || attn_tmap(&mv, v, HD, a.kv_heads, nk, a.sv, 1, 128, 2))
    return LT_ERR_CUDA;
  if (allow_smem<k_attn_tc<HD, W>>(tc_smem<HD, W>()) != cudaSuccess) return LT_ERR_CUDA;
  const unsigned pairs = (unsigned)prompt_pairs(a.n_q, a.n_seqs, a.group) * a.kv_heads;
  if (launch_pdl(k_attn_tc<HD, W>, pairs * a.splits, 1, W::THREADS, tc_smem<HD, W>(), st, a, mq, mk, mv) != cudaSuccess)
    return LT_ERR_CUDA;
  if (a.splits > 1) {
    const int parts = cdiv(256, prompt_join_rows<HD>());
    if (launch_pdl(k_attn_prompt_join<HD>, pairs * parts, 1, 256, 0, st, a, parts) != cudaSuccess) return LT_ERR_CUDA;
  }
  return LT_OK;
}

template <int HD>
static int prompt_any(int dtype, const PromptArgs& a, cudaStream_t st) {
  if (dtype == LT_BF16) return prompt_tc<HD>(a, st);
  return prompt_simt<HD>(a, st) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

}  // namespace lt

using namespace lt;

extern "C" int lt_attn_prompt_scratch_bytes(int dtype, int n_q, int n_seqs, int n_heads, int n_kv_heads,
                                            int head_dim, size_t* bytes) {
  if (!bytes || (dtype != LT_F32 && dtype != LT_BF16) || n_q < 0 || n_seqs < 0) return LT_ERR_ARG;
  if (!attn_shape_ok(n_heads, n_kv_heads, head_dim)) return LT_ERR_SHAPE;
  // the launch grid counts tiles of at least 64 / group tokens
  if (n_q > COUNT_MAX || ((long long)n_q / (SIMT_M / (n_heads / n_kv_heads)) + n_seqs) * n_kv_heads > 0x7fffffff)
    return LT_ERR_SHAPE;
  *bytes = 256;
  if (dtype == LT_BF16) {
    const long long splits = prompt_max_splits(n_q, n_seqs, n_heads, n_kv_heads);
    if (splits > 1)
      *bytes = (size_t)(prompt_pairs(n_q, n_seqs, n_heads / n_kv_heads) * n_kv_heads * splits) * 256 *
               (sizeof(float2) + (size_t)head_dim * sizeof(float));
  }
  return LT_OK;
}

extern "C" int lt_attn_prompt(int dtype, const void* d_q, long long stride_q, const void* d_k,
                              long long stride_k, const void* d_v, long long stride_v, void* d_o,
                              long long stride_o, const int32_t* d_q_off, const int32_t* d_kv_off,
                              int n_seqs, int n_q, int n_kv, int n_heads, int n_kv_heads, int head_dim,
                              float scale, void* d_scratch, size_t scratch_bytes, int32_t* d_status,
                              void* stream) {
  if (dtype != LT_F32 && dtype != LT_BF16) return LT_ERR_ARG;
  if (n_seqs < 0 || n_q < 0 || n_kv < 0 || !(scale > 0.f) || !(scale < INFINITY)) return LT_ERR_ARG;
  if (!attn_shape_ok(n_heads, n_kv_heads, head_dim)) return LT_ERR_SHAPE;
  size_t need = 0;
  if (int e = lt_attn_prompt_scratch_bytes(dtype, n_q, n_seqs, n_heads, n_kv_heads, head_dim, &need)) return e;
  if (n_kv > COUNT_MAX) return LT_ERR_SHAPE;
  if (n_seqs == 0 || n_q == 0) return LT_OK;
  if (!d_q || !d_o || !d_q_off || !d_scratch || (n_kv > 0 && (!d_k || !d_v))) return LT_ERR_ARG;
  const long long w = (long long)n_heads * head_dim, wk = (long long)n_kv_heads * head_dim;
  if (stride_q < w || stride_o < w || stride_k < wk || stride_v < wk) return LT_ERR_ARG;
  if (((uintptr_t)d_scratch & 31) || !attn_aligned(dtype, d_q, stride_q) || !attn_aligned(dtype, d_k, stride_k) ||
      !attn_aligned(dtype, d_v, stride_v) || !attn_aligned(dtype, d_o, stride_o))
    return LT_ERR_SHAPE;
  if (scratch_bytes < need) return LT_ERR_CAPACITY;
  PromptArgs a = {d_q, d_k, d_v, d_o, stride_q, stride_k, stride_v, stride_o, d_q_off,
                  d_kv_off ? d_kv_off : d_q_off, n_seqs, n_q, n_kv, n_heads, n_kv_heads,
                  n_heads / n_kv_heads, scale, d_status, 1, nullptr,
                  ((uintptr_t)d_o & 31) == 0 && stride_o % 16 == 0, nullptr};
  if (dtype == LT_BF16) {
    a.splits = prompt_splits(n_q, n_kv, n_seqs, n_heads, n_kv_heads);
    const size_t slots = (size_t)(prompt_pairs(n_q, n_seqs, a.group) * n_kv_heads * a.splits) * 256;
    a.part = (float*)d_scratch;
    a.part_ml = (float2*)(a.part + slots * head_dim);
  }
  cudaStream_t st = (cudaStream_t)stream;
  switch (head_dim) {
    case 32: return prompt_any<32>(dtype, a, st);
    case 64: return prompt_any<64>(dtype, a, st);
    case 96: return prompt_any<96>(dtype, a, st);
    default: return prompt_any<128>(dtype, a, st);
  }
}

// Verification of drafted tokens against the target's probabilities, from
// given random numbers (LoopSpec page, section 2.2, Eqs. 2-4: accept a draft x
// with probability min(1, p(x) / q(x)), else draw from the residual
// max(0, p - q)).
#include <cooperative_groups.h>

#include "../../include/looped_spec.h"
#include "attn_common.cuh"

namespace lt {

namespace cg = cooperative_groups;

constexpr int VERIFY_THREADS = 256, VERIFY_WARPS = VERIFY_THREADS / 32;
constexpr int VERIFY_SEG = 512;      // vocabulary entries one warp sums at a time
constexpr int VERIFY_MAX_SEGS = 256; // segments of one CTA whose sums are kept

struct VerifyArgs {
  const float* p;
  const float* q;
  long long sp, sq;
  const int32_t* draft;
  const int32_t* off;
  int n_seqs, n_drafts, V;
  const float* u_acc;
  const float* u_draw;
  int32_t* n_acc;
  int32_t* tok;
  int* status;
};

// Weight of entry j of a draw: max(0, p - q) (rounded once, as fp32 does), p
// where no q is given; the excluded entry, non-finite and negative ones weigh 0.
__device__ __forceinline__ float verify_weight(float p, float q, int j, int excl) {
  const float w = p - q;
  return (w > 0.f && w < INFINITY && j != excl) ? w : 0.f;
}

// One segment's weights, 16 per lane: entries base + i * 128 + lane * 4 + e
// (VEC: rows on 16-byte boundaries), or base + i * 32 + lane.
template <bool VEC>
__device__ __forceinline__ int seg_index(int base, int k) {
  const int lane = threadIdx.x & 31;
  return VEC ? base + (k >> 2) * 128 + lane * 4 + (k & 3) : base + k * 32 + lane;
}
template <bool VEC>
__device__ __forceinline__ void seg_load(const float* __restrict__ p, const float* __restrict__ q, int base,
                                         int V, int excl, float w[16]) {
  __align__(16) float a[16], b[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) a[k] = b[k] = 0.f;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = seg_index<VEC>(base, 4 * i);
      if (j + 4 <= V) {
        *reinterpret_cast<float4*>(a + 4 * i) = *reinterpret_cast<const float4*>(p + j);
        if (q) *reinterpret_cast<float4*>(b + 4 * i) = *reinterpret_cast<const float4*>(q + j);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < V) {
            a[4 * i + e] = p[j + e];
            if (q) b[4 * i + e] = q[j + e];
          }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int j = seg_index<VEC>(base, k);
      if (j < V) {
        a[k] = p[j];
        if (q) b[k] = q[j];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = verify_weight(a[k], b[k], seg_index<VEC>(base, k), excl);
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_scan_d(double v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// The lowest entry of a segment whose running sum (from `before`) exceeds
// `target`; the segment's last entry with a weight where rounding leaves none.
template <bool VEC>
__device__ __forceinline__ int seg_pick(const float w[16], int base, double before, double target) {
  constexpr int GRP = VEC ? 4 : 1;  // consecutive entries a lane holds
  int last = -1;
#pragma unroll
  for (int i = 0; i < 16 / GRP; ++i) {
    double s = 0;
#pragma unroll
    for (int e = 0; e < GRP; ++e) s += (double)w[i * GRP + e];
    const double incl = warp_scan_d(s);
    double run = before + (incl - s);
    int pick = 0x7fffffff, mine = -1;
#pragma unroll
    for (int e = 0; e < GRP; ++e) {
      run += (double)w[i * GRP + e];
      const int j = seg_index<VEC>(base, i * GRP + e);
      if (w[i * GRP + e] > 0.f) {
        mine = j;
        if (run > target && pick == 0x7fffffff) pick = j;
      }
    }
    pick = __reduce_min_sync(0xffffffffu, pick);
    if (pick != 0x7fffffff) return pick;
    last = max(last, __reduce_max_sync(0xffffffffu, mine));
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return last;
}

// A cluster per sequence.  Each CTA decides the chain by itself (a few loads),
// sums its slice of the stopping row's weights segment by segment in 64 bits
// (the running sum decides a token, so its rounding must stay far below a
// weight), and the CTA that holds the crossing reads that one segment again.
// Bound by HBM for a batch (one row of p and one of q per sequence) and by the
// chain of dependent loads for one sequence.
template <bool VEC>
__global__ void __launch_bounds__(VERIFY_THREADS, 4) k_verify(VerifyArgs a, int seg_units) {
  __shared__ double seg_sum[VERIFY_MAX_SEGS];
  __shared__ double total;
  __shared__ double run_at;
  __shared__ int seg_at;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), nr = cl.num_blocks();
  const int s = blockIdx.x / nr, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  const int o0 = __ldg(a.off + s), o1 = __ldg(a.off + s + 1);
  const bool bad = o0 < 0 || o1 < o0 || o1 > a.n_drafts;  // the same in every CTA of the cluster
  if (bad) {
    if (threadIdx.x == 0 && rank == 0) {
      set_err(a.status, DEV_BAD_INDEX);
      a.n_acc[s] = -1;
    }
    return;
  }
  const int k = o1 - o0;
  // the first draft that is not accepted
  int acc = k, x = -1;
  for (int i0 = 0; i0 < k; i0 += 32) {
    const int i = i0 + lane;
    int xi = -1;
    bool ok = i < k;
    if (ok) {
      xi = __ldg(a.draft + o0 + i);
      ok = xi >= 0 && xi < a.V;
      if (ok) {
        const double pv = a.p[(size_t)(o0 + s + i) * a.sp + xi];
        const double qv = a.q ? a.q[(size_t)(o0 + i) * a.sq + xi] : 1.0;
        ok = (double)a.u_acc[o0 + i] * qv < pv;
      }
    }
    const unsigned no = __ballot_sync(0xffffffffu, !ok);
    if (no) {
      const int f = __ffs(no) - 1;
      if (i0 + f < k) {
        acc = i0 + f;
        x = __shfl_sync(0xffffffffu, xi, f);
      }
      break;
    }
  }
  if (rank == 0) {
    const size_t base = (size_t)o0 + s;
    for (int i = threadIdx.x; i <= k; i += VERIFY_THREADS)
      if (i != acc) a.tok[base + i] = i < acc ? __ldg(a.draft + o0 + i) : -1;
    if (threadIdx.x == 0) a.n_acc[s] = acc;
  }
  const float* p = a.p + (size_t)(o0 + s + acc) * a.sp;
  const float* q = acc < k && a.q ? a.q + (size_t)(o0 + acc) * a.sq : nullptr;
  int excl = acc < k && !a.q ? x : -1;  // a one-hot draft: its residual is p without it
  const int SEG = seg_units * VERIFY_SEG;
  const int segs = (a.V + SEG - 1) / SEG, per = (segs + nr - 1) / nr;
  const int s0 = min(segs, rank * per), s1 = min(segs, s0 + per);
  for (int pass = 0; pass < 2; ++pass) {
    for (int g = s0 + w; g < s1; g += VERIFY_WARPS) {
      double sum = 0;
      for (int b = 0; b < seg_units; ++b) {
        float wt[16];
        seg_load<VEC>(p, q, g * SEG + b * VERIFY_SEG, a.V, excl, wt);
        double part = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) part += (double)wt[e];
        sum += part;
      }
      sum = warp_sum_d(sum);
      if (lane == 0) seg_sum[g - s0] = sum;
    }
    __syncthreads();
    if (w == 0) {
      double t = 0;
      for (int g = lane; g < s1 - s0; g += 32) t += seg_sum[g];
      t = warp_sum_d(t);
      if (lane == 0) total = t;
    }
    cl.sync();
    double all = 0, before = 0;
    for (int r = 0; r < nr; ++r) {
      const double t = *cl.map_shared_rank(&total, r);
      if (r < rank) before += t;
      all += t;
    }
    const double target = (double)a.u_draw[s] * all;
    // the first CTA whose inclusive sum exceeds the target, else the last with a weight
    int owner = -1, lastw = -1;
    double run = 0;
    for (int r = 0; r < nr; ++r) {
      const double t = *cl.map_shared_rank(&total, r);
      run += t;
      if (t > 0) lastw = r;
      if (owner < 0 && run > target) owner = r;
    }
    if (owner < 0) owner = lastw;
    cl.sync();  // every CTA has read the totals
    if (owner < 0) {  // no mass: a residual falls back to the row itself, a row gives -1
      if (pass == 0 && (q || excl >= 0)) {
        q = nullptr;
        excl = -1;
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) a.tok[(size_t)o0 + s + acc] = -1;
      return;
    }
    if (owner != rank) return;
    if (threadIdx.x == 0) {
      double r = before;
      int at = -1;
      double at_run = 0;
      for (int g = 0; g < s1 - s0; ++g) {
        if (seg_sum[g] > 0) {
          at = g;
          at_run = r;
        }
        r += seg_sum[g];
        if (seg_sum[g] > 0 && r > target) break;
      }
      seg_at = s0 + at;
      run_at = at_run;
    }
    __syncthreads();
    if (w == 0) {
      double r = run_at;
      int pick = -1;
      for (int b = 0; b < seg_units; ++b) {
        float wt[16];
        const int base = seg_at * SEG + b * VERIFY_SEG;
        seg_load<VEC>(p, q, base, a.V, excl, wt);
        double part = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) part += (double)wt[e];
        part = warp_sum_d(part);
        if (part > 0) {
          pick = seg_pick<VEC>(wt, base, r, target);
          r += part;
          if (r > target) break;
        }
      }
      if (lane == 0) a.tok[(size_t)o0 + s + acc] = pick;
    }
    return;
  }
}

}  // namespace lt

using namespace lt;

extern "C" int lt_verify_drafts(const float* d_p, long long stride_p, const float* d_q, long long stride_q,
                                const int32_t* d_draft, const int32_t* d_off, int n_seqs, int n_drafts,
                                int V, const float* d_u_accept, const float* d_u_draw,
                                int32_t* d_n_accepted, int32_t* d_tokens, int32_t* d_status,
                                void* stream) {
  if (n_seqs < 0 || n_drafts < 0 || V <= 0 || (long long)n_drafts + n_seqs > 0x7fffffff) return LT_ERR_ARG;
  if (n_seqs == 0) return LT_OK;
  if (!d_p || !d_off || !d_u_draw || !d_n_accepted || !d_tokens || stride_p < V ||
      (n_drafts > 0 && (!d_draft || !d_u_accept)) || (d_q && stride_q < V))
    return LT_ERR_ARG;
  // Eight CTAs a sequence for latency (one chain at a vocabulary of 49152: 6.9 us, 18.2 us with one),
  // fewer where all of them would not be resident at once with room to place the clusters (148 chains
  // at 65536: 23.0 us with two, 25.7 us with four, which would just fit; 192 chains: 26.2 us with two,
  // 33.2 us with eight) or would have less than a segment per warp.
  int nr = 8;
  while (nr > 1 && ((long long)n_seqs * nr > 3ll * attn_sm_count() || (long long)(nr / 2) * VERIFY_WARPS * VERIFY_SEG >= V)) nr /= 2;
  const long long segs = ((long long)V + VERIFY_SEG - 1) / VERIFY_SEG;
  const int units = (int)((segs + (long long)nr * VERIFY_MAX_SEGS - 1) / ((long long)nr * VERIFY_MAX_SEGS));
  VerifyArgs a = {d_p, d_q, stride_p, stride_q, d_draft, d_off, n_seqs, n_drafts, V, d_u_accept,
                  d_u_draw, d_n_accepted, d_tokens, d_status};
  const bool vec = ((uintptr_t)d_p & 15) == 0 && stride_p % 4 == 0 &&
                   (!d_q || (((uintptr_t)d_q & 15) == 0 && stride_q % 4 == 0));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_seqs * (long long)nr));
  cfg.blockDim = dim3(VERIFY_THREADS);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nr;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, k_verify<true>, a, units)
                            : cudaLaunchKernelEx(&cfg, k_verify<false>, a, units);
  return e == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

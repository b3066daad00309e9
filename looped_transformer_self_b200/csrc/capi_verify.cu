// Verification of drafted tokens against the target's probabilities, from
// given random numbers (LoopSpec page, section 2.2, Eqs. 2-4: accept a draft x
// with probability min(1, p(x) / q(x)), else draw from the residual
// max(0, p - q)).
#include <cooperative_groups.h>

#include <algorithm>

#include "../../include/looped_spec.h"
#include "attn_common.cuh"

namespace lt {

namespace cg = cooperative_groups;

constexpr int VERIFY_THREADS = 256, VERIFY_WARPS = VERIFY_THREADS / 32;
constexpr int VERIFY_SEG = 512;        // vocabulary entries one warp loads at a time
constexpr int VERIFY_MAX_GROUPS = 256; // groups of segments of one CTA, whose sums are kept
constexpr int VERIFY_MAX_CTAS = 8;     // of a cluster

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
__device__ __forceinline__ void seg_raw(const float* p, int base, int V, float a[16]) {
  if (VEC && base + VERIFY_SEG <= V) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(p + seg_index<VEC>(base, 4 * i));
      a[4 * i] = x.x, a[4 * i + 1] = x.y, a[4 * i + 2] = x.z, a[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int j = seg_index<VEC>(base, k);
      a[k] = j < V ? p[j] : 0.f;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void seg_load(const float* p, const float* q, int base,
                                         int V, int excl, float w[16]) {
  float b[16];
  seg_raw<VEC>(p, base, V, w);
#pragma unroll
  for (int k = 0; k < 16; ++k) b[k] = 0.f;
  if (q) seg_raw<VEC>(q, base, V, b);
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = verify_weight(w[k], b[k], seg_index<VEC>(base, k), excl);
}
// A lane's share of a segment's weights, in 64 bits.
template <bool VEC>
__device__ __forceinline__ double seg_sum_exact(const float* p, const float* q, int base,
                                                int V, int excl) {
  float w[16];
  seg_load<VEC>(p, q, base, V, excl, w);
  double s = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += (double)w[k];
  return s;
}
// The same without the tests of an excluded entry and of infinite weights (then the sum is infinite).
template <bool VEC>
__device__ __forceinline__ double seg_sum_fast(const float* p, const float* q, int base,
                                               int V) {
  float a[16], b[16];
  seg_raw<VEC>(p, base, V, a);
  double s[4] = {0, 0, 0, 0};
  if (q) {
    seg_raw<VEC>(q, base, V, b);
#pragma unroll
    for (int k = 0; k < 16; ++k) a[k] -= b[k];
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) s[k & 3] += (double)fmaxf(a[k], 0.f);  // a NaN weighs 0
  return (s[0] + s[1]) + (s[2] + s[3]);
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

// Cluster barrier in two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// A cluster per sequence.  Each CTA decides the chain by itself (a few loads) and
// sums its slice of the stopping row's weights in 64 bits, a group of segments
// per warp (the running sum decides a token, so its rounding must stay far below
// a weight); the CTA that holds the crossing reads that one group again, a
// segment per warp.
// Bound by HBM for a batch (one row of p and, unless all drafts are accepted, one of
// q per sequence: 192 chains at 65536, 90 MB read, take 22 us, and 6 us with a row of
// 64: 5.6 TB/s between the two) and by the chain of dependent loads for one sequence
// (6.7 us at 49152: offsets, drafts, their probabilities, the row, two barriers, the
// group again).
// Testing every entry for the excluded one and for infinities, and a sum per
// segment, cost 4 us of the batch (25 instructions an entry against 6).
template <bool VEC>
__global__ void __launch_bounds__(VERIFY_THREADS, 3) k_verify(VerifyArgs a, int units) {
  __shared__ double group_sum[VERIFY_MAX_GROUPS];
  __shared__ double seg_part[VERIFY_WARPS];
  __shared__ double total;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), nr = cl.num_blocks();
  const int s = blockIdx.x / nr, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  const int o0 = a.off[s], o1 = a.off[s + 1];
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
      xi = a.draft[o0 + i];
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
      if (i != acc) a.tok[base + i] = i < acc ? a.draft[o0 + i] : -1;
    if (threadIdx.x == 0) a.n_acc[s] = acc;
  }
  const float* p = a.p + (size_t)(o0 + s + acc) * a.sp;
  const float* q = acc < k && a.q ? a.q + (size_t)(o0 + acc) * a.sq : nullptr;
  int excl = acc < k && !a.q ? x : -1;  // a one-hot draft: its residual is p without it
  const int span = units * VERIFY_SEG;  // entries of a group
  const int groups = (a.V + span - 1) / span, per = (groups + nr - 1) / nr;
  const int g0 = min(groups, rank * per), g1 = min(groups, g0 + per);
  for (int pass = 0; pass < 2; ++pass) {
    for (int g = g0 + w; g < g1; g += VERIFY_WARPS) {
      double sum = 0;
#pragma unroll 2
      for (int base = g * span; base < min(a.V, (g + 1) * span); base += VERIFY_SEG)
        sum += excl >= base && excl < base + VERIFY_SEG ? seg_sum_exact<VEC>(p, q, base, a.V, excl)
                                                        : seg_sum_fast<VEC>(p, q, base, a.V);
      sum = warp_sum_d(sum);
      if (!(sum < INFINITY)) {  // an infinite weight, which counts for nothing
        sum = 0;
        for (int base = g * span; base < min(a.V, (g + 1) * span); base += VERIFY_SEG)
          sum += seg_sum_exact<VEC>(p, q, base, a.V, excl);
        sum = warp_sum_d(sum);
      }
      if (lane == 0) group_sum[g - g0] = sum;
    }
    __syncthreads();
    if (w == 0) {
      double t = 0;
      for (int g = lane; g < g1 - g0; g += 32) t += group_sum[g];
      t = warp_sum_d(t);
      if (lane == 0) total = t;
    }
    cluster_arrive();
    cluster_wait();
    const double theirs = lane < nr ? *cl.map_shared_rank(&total, lane) : 0.0;
    cluster_arrive();  // waited for before `total` is written again or the CTA ends
    double all = 0;
    for (int r = 0; r < nr; ++r) all += __shfl_sync(0xffffffffu, theirs, r);
    const double target = (double)a.u_draw[s] * all;
    // the first CTA whose inclusive sum exceeds the target, else the last with a weight
    int owner = -1, lastw = -1;
    double run = 0, before = 0;
    for (int r = 0; r < nr; ++r) {
      const double t = __shfl_sync(0xffffffffu, theirs, r);
      if (r == rank) before = run;
      run += t;
      if (t > 0) lastw = r;
      if (owner < 0 && run > target) owner = r;
    }
    if (owner < 0) owner = lastw;
    if (owner < 0 && pass == 0 && (q || excl >= 0)) {  // a residual without mass: the row itself
      q = nullptr;
      excl = -1;
      cluster_wait();
      continue;
    }
    int at = -1;  // the group
    double at_run = before;
    if (owner == rank)
      for (int g = 0; g < g1 - g0; ++g) {
        const double t = group_sum[g];
        if (t > 0) {
          at = g0 + g;
          at_run = before;
        }
        before += t;
        if (t > 0 && before > target) break;
      }
    if (at >= 0) {
      int hit = -1;  // the segment in it
      double hit_run = at_run;
      float wt[16];
      for (int b0 = 0; b0 < units; b0 += VERIFY_WARPS) {
        double part = 0;
        if (b0 + w < units) {
          seg_load<VEC>(p, q, at * span + (b0 + w) * VERIFY_SEG, a.V, excl, wt);
#pragma unroll
          for (int e = 0; e < 16; ++e) part += (double)wt[e];
        }
        part = warp_sum_d(part);
        if (lane == 0) seg_part[w] = part;
        __syncthreads();
        bool found = false;
        for (int i = 0; i < VERIFY_WARPS && !found; ++i) {
          const double t = seg_part[i];
          if (t > 0) {
            hit = b0 + i;
            hit_run = at_run;
          }
          at_run += t;
          found = t > 0 && at_run > target;
        }
        if (found) break;
        __syncthreads();
      }
      if (hit >= 0 && w == hit % VERIFY_WARPS) {
        const int base = at * span + hit * VERIFY_SEG;
        seg_load<VEC>(p, q, base, a.V, excl, wt);
        const int pick = seg_pick<VEC>(wt, base, hit_run, target);
        if (lane == 0) a.tok[(size_t)o0 + s + acc] = pick;
      }
    } else if (owner < 0 && rank == 0 && threadIdx.x == 0) {
      a.tok[(size_t)o0 + s + acc] = -1;  // no mass
    }
    cluster_wait();
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
  if (n_seqs < 0 || n_drafts < 0 || V <= 0 || V > (1 << 30) || (long long)n_drafts + n_seqs > COUNT_MAX) return LT_ERR_ARG;
  if (n_seqs == 0) return LT_OK;
  if (!d_p || !d_off || !d_u_draw || !d_n_accepted || !d_tokens || stride_p < V ||
      (n_drafts > 0 && (!d_draft || !d_u_accept)) || (d_q && stride_q < V))
    return LT_ERR_ARG;
  // Eight CTAs a sequence for latency (one chain at a vocabulary of 49152: 6.4 to 6.7 us, 6.8 us with four,
  // 12.0 us with one), fewer where all of them would not be resident at once with room to place the
  // clusters (148 chains at 65536: 19.2 us with two, 22.7 us with four, which would just fit; 192 chains:
  // 21.9 us with two, 24.6 us with one, 24.8 us with four) or would have less than a segment per warp.
  int nr = VERIFY_MAX_CTAS;
  while (nr > 1 && ((long long)n_seqs * nr > 3ll * attn_sm_count() || (long long)(nr / 2) * VERIFY_WARPS * VERIFY_SEG >= V)) nr /= 2;
  // Segments a warp sums before it reduces and keeps a sum: all of its own, at most eight (a group is
  // read again by the CTA's eight warps) as long as the groups' sums fit.
  const long long segs = ((long long)V + VERIFY_SEG - 1) / VERIFY_SEG, mine = (segs + nr * VERIFY_WARPS - 1) / (nr * VERIFY_WARPS);
  const long long rounds = (mine + VERIFY_WARPS - 1) / VERIFY_WARPS;
  const long long least = (segs + (long long)nr * VERIFY_MAX_GROUPS - 1) / ((long long)nr * VERIFY_MAX_GROUPS);
  const int units = (int)std::max((mine + rounds - 1) / rounds, least);
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

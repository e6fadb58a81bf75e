// Routing of any number of tokens, and the routes grouped by expert.
//
// Per token ("mega_moe" _MegaKernel.top_k_pick, as route_topk): s = sigmoid(logits), key = s + bias, the top_k
// largest keys (ties: lower expert), weights s / (sum of the picked s) * scale. The T * top_k routes, numbered
// t * top_k + r, are then sorted by expert, ascending within one: a counting sort.
//
// The tokens are cut into contiguous shares, one a CTA, and a CTA's share into contiguous
// runs, one a warp, so counts per (CTA, warp, expert) give every route its place
// without an order-dependent atomic.
//   1  route_pick_kernel     picks, weights, and the CTA's routes per expert -> counts[CTA][E]
//   2  route_place_kernel    expert starts from all counts, then each route to its place
#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kRtWarps = 16;
constexpr int kRtThreads = 32 * kRtWarps;
constexpr int kRtMaxCtas = 152;

struct RtArgs {
  const void* logits;
  const float* bias;
  int logits_f32, T, E, top_k;
  float scale;
  int per_cta, per_warp;  // tokens
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* tokens;
  uint16_t* counts;  // [CTAs][E]: a share holds fewer than 65,536 tokens
};

// The picks of token t: lane r < top_k gets rank r's expert and weight. Lane l holds experts l + 32 j.
template <int J>
__device__ __forceinline__ void rt_pick(const RtArgs& a, const float (&bias)[J], int t, int lane, int& my_e, float& my_w) {
  float sc[J];
  uint32_t ky[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 32 * j;
    sc[j] = 0.0f;
    if (e < a.E)
      sc[j] = a.logits_f32
                  ? __ldg(static_cast<const float*>(a.logits) + static_cast<size_t>(t) * a.E + e)
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[static_cast<size_t>(t) * a.E + e]);
  }
  uint32_t best = 0u;
  int best_j = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    sc[j] = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-sc[j])));
    // At least 1, so that an expert (a NaN key, too) always stands above a lane's empty places.
    ky[j] = (lane + 32 * j < a.E) ? max(1u, ordered_key(__fadd_rn(sc[j], bias[j]))) : 0u;
    if (ky[j] > best) {
      best = ky[j];
      best_j = j;
    }
  }
  float total = 0.0f, mine = 0.0f;
  int mine_e = 0;
#pragma unroll 1
  for (int r = 0; r < a.top_k; ++r) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t cand = best == top ? static_cast<uint32_t>(lane + 32 * best_j) : 0xFFFFFFFFu;
    const int win = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, cand));
    float sv = 0.0f;
    if (lane == (win & 31)) {
      // Only the winner's lane takes its pick out and looks for its next best.
      best = 0u;
      int next = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j == best_j) {
          sv = sc[j];
          ky[j] = 0u;
        }
        if (ky[j] > best) {
          best = ky[j];
          next = j;
        }
      }
      best_j = next;
    }
    const float s = __shfl_sync(0xFFFFFFFFu, sv, win & 31);
    total = __fadd_rn(total, s);
    if (lane == r) {
      mine = s;
      mine_e = win;
    }
  }
  my_e = mine_e;
  my_w = __fmul_rn(__fdiv_rn(mine, total), a.scale);
}

template <int J>
__global__ void __launch_bounds__(kRtThreads) route_pick_kernel(const RtArgs a) {
  __shared__ int hist[kMaxExperts];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += kRtThreads) hist[e] = 0;
  float bias[J];
#pragma unroll
  for (int j = 0; j < J; ++j) bias[j] = lane + 32 * j < a.E ? __ldg(a.bias + lane + 32 * j) : 0.0f;
  __syncthreads();
  const int c0 = blockIdx.x * a.per_cta, c1 = min(a.T, c0 + a.per_cta);
  const int t0 = c0 + warp * a.per_warp, t1 = min(c1, t0 + a.per_warp);
  for (int t = t0; t < t1; ++t) {
    int e;
    float w;
    rt_pick<J>(a, bias, t, lane, e, w);
    if (lane < a.top_k) {
      a.ids[static_cast<size_t>(t) * a.top_k + lane] = e;
      a.weights[static_cast<size_t>(t) * a.top_k + lane] = w;
      atomicAdd(&hist[e], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRtThreads)
    a.counts[static_cast<size_t>(blockIdx.x) * a.E + e] = static_cast<uint16_t>(hist[e]);
}

__global__ void __launch_bounds__(kRtThreads) route_place_kernel(const RtArgs a) {
  __shared__ int start[kMaxExperts];              // where this CTA's routes of an expert go
  __shared__ uint16_t before[kRtWarps][kMaxExperts];  // this warp's next place among them
  __shared__ int warp_sum[kRtWarps];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x;
  // Two experts a thread: routes of all CTAs, and of those before this one.
  int all[2], prev[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * threadIdx.x + i;
    all[i] = prev[i] = 0;
    if (e < a.E)
#pragma unroll 8
      for (int c = 0; c < G; ++c) {
        const int n = a.counts[static_cast<size_t>(c) * a.E + e];
        all[i] += n;
        prev[i] += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
  }
  int scan = all[0] + all[1];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  for (int e = lane; e < a.E; e += 32) before[warp][e] = 0;
  __syncthreads();
  int at = scan - all[0] - all[1];
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * threadIdx.x + i;
    if (e < a.E) {
      start[e] = at + prev[i];
      if (blockIdx.x == 0) a.offsets[e] = at;
    }
    at += all[i];
    if (e == a.E - 1 && blockIdx.x == 0) a.offsets[a.E] = at;
  }
  const int c0 = blockIdx.x * a.per_cta, c1 = min(a.T, c0 + a.per_cta);
  const int t0 = min(c1, c0 + warp * a.per_warp), t1 = min(c1, t0 + a.per_warp);
  // A token's picks are distinct, so its lanes never meet on one counter.
  for (int t = t0; t < t1; ++t) {
    if (lane < a.top_k) ++before[warp][a.ids[static_cast<size_t>(t) * a.top_k + lane]];
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRtThreads) {
    int sum = 0;
    for (int w = 0; w < kRtWarps; ++w) {
      const int n = before[w][e];
      before[w][e] = static_cast<uint16_t>(sum);
      sum += n;
    }
  }
  __syncthreads();
  for (int t = t0; t < t1; ++t) {
    if (lane < a.top_k) {
      const int route = t * a.top_k + lane;
      const int e = a.ids[route];
      const int place = start[e] + before[warp][e]++;
      a.rows[place] = route;
      a.tokens[place] = t;
    }
    __syncwarp();
  }
}

static int rt_ctas(int T) {
  const int n = (T + kRtWarps - 1) / kRtWarps;
  return n < kRtMaxCtas ? n : kRtMaxCtas;
}

size_t route_workspace_bytes(int T, int E) {
  return 256 + ((static_cast<size_t>(rt_ctas(T)) * E * sizeof(uint16_t) + 255) & ~size_t(255));
}

int route(const void* logits, int logits_dtype, const float* bias, int T, int E, int top_k, float scale, int32_t* ids,
          float* weights, int32_t* offsets, int32_t* rows, int32_t* tokens, void* workspace, size_t workspace_bytes,
          cudaStream_t st) {
  const size_t need = route_workspace_bytes(T, E);
  if (workspace == nullptr || workspace_bytes < need)
    return set_last_error(FME_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (T == 0) {
    const cudaError_t err = cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), st);
    if (err != cudaSuccess) return set_last_error(FME_ECUDA, "cudaMemsetAsync: %s", cudaGetErrorString(err));
    return FME_OK;
  }
  RtArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.logits_f32 = logits_dtype == FME_F32;
  a.T = T;
  a.E = E;
  a.top_k = top_k;
  a.scale = scale;
  const int ctas = rt_ctas(T);
  a.per_cta = (T + ctas - 1) / ctas;
  a.per_warp = (a.per_cta + kRtWarps - 1) / kRtWarps;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.tokens = tokens;
  a.counts = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + 256);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kRtThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t err;
  if (E <= 64)
    err = cudaLaunchKernelEx(&cfg, route_pick_kernel<2>, a);
  else if (E <= 256)
    err = cudaLaunchKernelEx(&cfg, route_pick_kernel<8>, a);
  else
    err = cudaLaunchKernelEx(&cfg, route_pick_kernel<32>, a);
  if (err == cudaSuccess) err = cudaLaunchKernelEx(&cfg, route_place_kernel, a);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "route launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

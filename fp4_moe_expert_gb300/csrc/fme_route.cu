// Routing of any number of tokens, and the routes grouped by expert, in one launch.
//
// Per token ("mega_moe" _MegaKernel.top_k_pick, as route_topk): s = sigmoid(logits), key = s + bias, the top_k
// largest keys (ties: lower expert), weights s / (sum of the picked s) * scale. The T * top_k routes, numbered
// t * top_k + r, are then sorted by expert, ascending within one: a counting sort.
//
// The tokens are cut into contiguous shares, one a CTA, and a share into contiguous runs, one a warp. A warp picks
// for its run and counts its routes per expert in shared memory; the CTAs publish their counts, meet once (bounded
// wait), and each derives the expert starts and its own places from all counts. So every route has its place without
// an atomic whose order could show.
// What bounds it: 16384 tokens of 256 experts, 24 us: of a CTA's 43,000 clocks the picks take 27,100 (three or four
// tokens a warp, one after another), the sums over all CTAs' counts 6,600, the meeting 4,300, the places 3,000; issue slots
// are half used, and the largest stall is the CTA barrier. 1533 tokens of 896 experts, 23 us (96 CTAs, 39,800 clocks):
// picks 19,100, sums 8,500, meeting 8,300. One token 6 us: latency.
#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kRtMaxCtas = 152;
constexpr int kRtTokens = 16;  // least tokens a CTA is given, where there are as many
// Set in the arrival word by a CTA whose wait gave up or met a word that was not left clean: no later call of this
// workspace takes stale counts for its own until the workspace is cleared.
constexpr uint32_t kRtBroken = 1u << 30;
constexpr int kRtIds = 64;     // picks of its run that a warp keeps in shared memory; the rest it reads back
// Warps a CTA: 32 where a lane's experts (J) leave 64 registers enough, else 16.
template <int J>
__host__ __device__ constexpr int rt_warps() { return J <= 8 ? 32 : 16; }

struct RtArgs {
  const void* logits;
  const float* bias;
  int logits_f32, vec, T, E, top_k;
  float scale;
  int per_cta, per_warp;  // tokens
  int pitch;              // experts in a row of counts: E rounded up to 8
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* tokens;
  uint16_t* counts;  // [CTAs][pitch]: a share holds fewer than 65,536 tokens, an expert at most one route of each
  uint32_t* err;
  uint32_t* sync;  // CTAs arrived (and kRtBroken), CTAs past the wait; zero between calls
  unsigned long long timeout_ns;
};

__device__ __noinline__ float rt_recip_far(float d) { return __fdiv_rn(1.0f, d); }
// route_topk's sigmoid, bit for bit.
__device__ __forceinline__ float rt_sigmoid(float l) {
  const float d = __fadd_rn(1.0f, expf(-l));
  return d <= 0x1p125f ? recip_rn(d) : rt_recip_far(d);
}
__device__ __forceinline__ float rt_value(const void* from, bool f32, size_t i) {
  return f32 ? __ldg(static_cast<const float*>(from) + i)
             : __bfloat162float(static_cast<const __nv_bfloat16*>(from)[i]);
}

// Values J * lane .. J * lane + J - 1 of the row of E that starts at element `row` (J a multiple of 8: in 16-byte loads
// where rows allow).
template <int J>
__device__ __forceinline__ void rt_load(const RtArgs& a, const void* from, bool f32, size_t row, int lane, float (&l)[J]) {
  const int e0 = J * lane;
  if (J >= 8 && a.vec) {
#pragma unroll
    for (int j = 0; j < J; j += 8)
      if (e0 + j < a.E) {
        if (f32) {
          const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(from) + row + e0 + j);
          const float4 p = __ldg(src), q = __ldg(src + 1);
          l[j] = p.x, l[j + 1] = p.y, l[j + 2] = p.z, l[j + 3] = p.w;
          l[j + 4] = q.x, l[j + 5] = q.y, l[j + 6] = q.z, l[j + 7] = q.w;
        } else {
          const uint4 p =
              __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(from) + row + e0 + j));
          const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            l[j + 2 * k] = __uint_as_float(w[k] << 16);
            l[j + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
          }
        }
      }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (e0 + j < a.E) l[j] = rt_value(from, f32, row + e0 + j);
  }
}

// Sorts v over the warp, largest in lane 0 (bitonic).
template <typename V>
__device__ __forceinline__ V rt_sort(V v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d >= 1; d >>= 1) {
      const V o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
      const bool keep_larger = ((lane & d) == 0) == ((lane & size) == 0 || size == 32);
      v = (v > o) == keep_larger ? v : o;
    }
  return v;
}

// The picks of token t: lane r < top_k gets rank r's expert and weight. `cand`: 32 words of this warp's.
//
// The top_k-th largest of the 32 lane maxima is at most the top_k-th largest key. The keys from it up are few (about
// 9 of 256 for 8 picks, 22 of 896 for 16): they move to one a lane and are sorted, key first, lower expert first.
// Where they are more than 32, the picks are taken one after another instead.
template <int J>
__device__ __forceinline__ void rt_pick(const RtArgs& a, const float (&bias)[J], const float (&l)[J], int t, int lane,
                                        unsigned long long* cand, int& my_e, float& my_w) {
  uint32_t ky[J];
  uint32_t best = 0u;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    // At least 1, so that an expert (a NaN key, too) always stands above a lane's empty places.
    ky[j] = J * lane + j < a.E ? max(1u, ordered_key(__fadd_rn(rt_sigmoid(l[j]), bias[j]))) : 0u;
    best = max(best, ky[j]);
  }
  const uint32_t floor_key = max(1u, __shfl_sync(0xFFFFFFFFu, rt_sort(best, lane), a.top_k - 1));
  int count = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, ky[j] >= floor_key);
    if (m != 0u) {
      const int at = count + __popc(m & ((1u << lane) - 1u));
      if (ky[j] >= floor_key && at < 32)
        cand[at] = (static_cast<unsigned long long>(ky[j]) << 32) | (0xFFFFFFFFu - (J * lane + j));
      count += __popc(m);
    }
  }
  __syncwarp();
  int mine;
  if (count <= 32) {
    mine = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(rt_sort(lane < count ? cand[lane] : 0ull, lane)));
    __syncwarp();
  } else {
    mine = 0;
#pragma unroll 1
    for (int r = 0; r < a.top_k; ++r) {
      uint32_t top = 0u;
      int top_j = 0;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (ky[j] > top) {
          top = ky[j];
          top_j = j;
        }
      // Lower lanes hold lower experts, and a lane's best is its lowest of equals.
      const int win = __ffs(__ballot_sync(0xFFFFFFFFu, top == __reduce_max_sync(0xFFFFFFFFu, top))) - 1;
      const int e = __shfl_sync(0xFFFFFFFFu, J * lane + top_j, win);
      if (lane == r) mine = e;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (lane == win && j == top_j) ky[j] = 0u;
    }
  }
  const float s =
      lane < a.top_k ? rt_sigmoid(rt_value(a.logits, a.logits_f32, static_cast<size_t>(t) * a.E + mine)) : 0.0f;
  float total = 0.0f;
  for (int r = 0; r < a.top_k; ++r) total = __fadd_rn(total, __shfl_sync(0xFFFFFFFFu, s, r));
  my_e = mine;
  my_w = __fmul_rn(__fdiv_rn(s, total), a.scale);
}

template <int J>
__global__ void __launch_bounds__(32 * rt_warps<J>()) route_kernel(const RtArgs a) {
  constexpr int kRtWarps = rt_warps<J>(), kRtThreads = 32 * kRtWarps;
  __shared__ uint16_t seen[kRtWarps][32 * J];    // routes of a warp's run per expert, then its next place
  __shared__ uint16_t picks[kRtWarps][kRtIds];   // the first picks of the run
  __shared__ union {
    unsigned long long cand[kRtWarps][32];  // while picking
    int start[32 * J];                      // then: where this CTA's routes of an expert go
  } u;
  __shared__ int all[32 * J], prev[32 * J];      // routes of every CTA, and of those before this one
  __shared__ int warp_sum[kRtWarps];
  __shared__ int gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = gridDim.x;
  for (int e = lane; e < a.E; e += 32) seen[warp][e] = 0;
  for (int e = threadIdx.x; e < a.E; e += kRtThreads) all[e] = prev[e] = 0;
  if (threadIdx.x == 0) gave_up = 0;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  const int c0 = min(a.T, static_cast<int>(blockIdx.x) * a.per_cta), c1 = min(a.T, c0 + a.per_cta);
  const int t0 = min(c1, c0 + warp * a.per_warp), t1 = min(c1, t0 + a.per_warp);
  if (t0 < t1) {
    float bias[J], l[J], next[J];
#pragma unroll
    for (int j = 0; j < J; ++j) bias[j] = l[j] = next[j] = 0.0f;
    rt_load<J>(a, a.logits, a.logits_f32, static_cast<size_t>(t0) * a.E, lane, l);
    rt_load<J>(a, a.bias, true, 0, lane, bias);
    __syncwarp();
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) rt_load<J>(a, a.logits, a.logits_f32, static_cast<size_t>(t + 1) * a.E, lane, next);
      int e;
      float w;
      rt_pick<J>(a, bias, l, t, lane, u.cand[warp], e, w);
      if (lane < a.top_k) {
        a.ids[static_cast<size_t>(t) * a.top_k + lane] = e;
        a.weights[static_cast<size_t>(t) * a.top_k + lane] = w;
        const int i = (t - t0) * a.top_k + lane;
        if (i < kRtIds) picks[warp][i] = static_cast<uint16_t>(e);
        ++seen[warp][e];  // a token's picks are distinct: its lanes never meet on one counter
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < J; ++j) l[j] = next[j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.pitch; e += kRtThreads) {
    int sum = 0;
    if (e < a.E)
      for (int w = 0; w < kRtWarps; ++w) {
        const int n = seen[w][e];
        seen[w][e] = static_cast<uint16_t>(sum);
        sum += n;
      }
    if (G > 1)
      a.counts[static_cast<size_t>(blockIdx.x) * a.pitch + e] = static_cast<uint16_t>(sum);
    else if (e < a.E)
      all[e] = sum;
  }
  if (G > 1) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      red_release_gpu_add(a.sync, 1u);
      const uint64_t begin = globaltimer_ns();
      int arrived;
      while ((arrived = static_cast<int>(ld_acquire_gpu(a.sync))) < G)
        if (globaltimer_ns() - begin > a.timeout_ns) break;
      // More than G: the word held something before this call's first arrival (the last CTA to arrive sees it at least).
      if (arrived != G) {
        atomicOr(a.err, kErrCrossWait);
        atomicOr(a.sync, kRtBroken);
        gave_up = 1;
      }
      // The last CTA past the wait leaves both words zero for the next call.
      if (!gave_up && atomicAdd(a.sync + 1, 1u) == static_cast<uint32_t>(G) - 1u) {
        a.sync[0] = 0u;
        a.sync[1] = 0u;
      }
    }
    __syncthreads();
    if (gave_up) {
      if (blockIdx.x == 0)  // groups without rows: the products that read them have nothing to do
        for (int e = threadIdx.x; e <= a.E; e += kRtThreads) a.offsets[e] = 0;
      return;
    }
    // Eight experts a load; the CTAs' rows are dealt to as many threads as there are to a column.
    const int words = a.pitch / 8, lanes = kRtThreads / words, col = threadIdx.x % words, first = threadIdx.x / words;
    if (first < lanes) {
      int sum[8], sum_prev[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = sum_prev[k] = 0;
#pragma unroll 4
      for (int c = first; c < G; c += lanes) {
        const uint4 p = __ldcg(reinterpret_cast<const uint4*>(a.counts + static_cast<size_t>(c) * a.pitch) + col);
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
        const bool before = c < static_cast<int>(blockIdx.x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int n = (w[k / 2] >> (16 * (k & 1))) & 0xFFFFu;
          sum[k] += n;
          sum_prev[k] += before ? n : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (8 * col + k < a.E) {
          if (sum[k] != 0) atomicAdd(&all[8 * col + k], sum[k]);
          if (sum_prev[k] != 0) atomicAdd(&prev[8 * col + k], sum_prev[k]);
        }
    }
  }
  __syncthreads();
  // Expert starts: two experts a thread (512 threads hold them all), a block scan.
  const int e0 = 2 * threadIdx.x;
  const int n0 = e0 < a.E ? all[e0] : 0, n1 = e0 + 1 < a.E ? all[e0 + 1] : 0;
  int scan = n0 + n1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int at = scan - n0 - n1;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  if (e0 < a.E) u.start[e0] = at + prev[e0];
  if (e0 + 1 < a.E) u.start[e0 + 1] = at + n0 + prev[e0 + 1];
  if (blockIdx.x == 0) {
    if (e0 < a.E) a.offsets[e0] = at;
    if (e0 + 1 < a.E) a.offsets[e0 + 1] = at + n0;
    if (e0 < a.E && e0 + 2 >= a.E) a.offsets[a.E] = at + n0 + n1;
  }
  __syncthreads();
  for (int t = t0; t < t1; ++t) {
    if (lane < a.top_k) {
      const int r = t * a.top_k + lane;
      const int i = (t - t0) * a.top_k + lane;
      const int e = i < kRtIds ? picks[warp][i] : a.ids[r];  // this lane's own store
      const int place = u.start[e] + seen[warp][e]++;
      if (static_cast<uint32_t>(place) < static_cast<uint32_t>(a.T * a.top_k)) {
        a.rows[place] = r;
        a.tokens[place] = t;
      } else {
        atomicOr(a.err, kErrCrossWait);  // counts of another call: this one passed the wait before its own were there
      }
    }
    __syncwarp();
  }
}

static int rt_ctas(int T) {
  const int n = (T + kRtTokens - 1) / kRtTokens;
  return n < 1 ? 1 : n < kRtMaxCtas ? n : kRtMaxCtas;
}
static int rt_pitch(int E) { return (E + 7) & ~7; }

size_t route_workspace_bytes(int T, int E) {
  return 256 + ((static_cast<size_t>(rt_ctas(T)) * rt_pitch(E) * sizeof(uint16_t) + 255) & ~size_t(255));
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
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return set_last_error(FME_ECUDA, "cudaGetDevice failed");
  const int sms = device_sm_count(dev);
  if (sms <= 0) return set_last_error(FME_ECUDA, "no SM count for device %d", dev);
  RtArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.logits_f32 = logits_dtype == FME_F32;
  a.vec = E % 8 == 0;  // rows of logits are then whole 16-byte units
  a.T = T;
  a.E = E;
  a.top_k = top_k;
  a.scale = scale;
  // All CTAs of a launch meet, so there are no more than SMs.
  const int ctas = rt_ctas(T) < sms ? rt_ctas(T) : sms;
  a.per_cta = (T + ctas - 1) / ctas;
  const int warps = E <= 256 ? rt_warps<8>() : rt_warps<32>();
  a.per_warp = (a.per_cta + warps - 1) / warps;
  a.pitch = rt_pitch(E);
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.tokens = tokens;
  a.err = static_cast<uint32_t*>(workspace);
  a.sync = a.err + 16;
  a.counts = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + 256);
  a.timeout_ns = wait_timeout_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // CTAs that meet run all or none: beside another stream's kernel that waits on its own CTAs, each could otherwise hold
  // SMs that the other needs. (16384 tokens: 24.6 us instead of 22.0 in a stream, 21.9 either way in a graph.)
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  void (*kernel)(RtArgs) = E <= 64 ? route_kernel<2> : E <= 256 ? route_kernel<8> : E <= 512 ? route_kernel<16> : route_kernel<32>;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "route launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

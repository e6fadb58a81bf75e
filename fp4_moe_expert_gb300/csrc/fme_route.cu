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
// The scored form (SCORED, fme_moe_route_groups) differs in the picks alone: sigmoid or softmax scores p, keys p + bias or, without
// a bias, the logits themselves (their order is the scores', and neither saturates nor underflows); the experts of the
// groups whose best one or two keys sum to less than those of the top_groups best groups are out; weights p / (sum of the
// picked p) * scale or p * scale. A softmax row's picks are weighed by exp(l - max): the sum over the row cancels.
//
// What bounds it: 16384 tokens of 256 experts, 18 us: of a CTA's 37,600 clocks the picks take 25,000 (three or four tokens a
// warp, one after another), the meeting 4,100, the sums over all CTAs' counts 3,200 (7,400 without adding them in pairs), the places
// 2,900. 1533 tokens of 896 experts, 14 us (96 CTAs, 27,200 clocks): picks 14,200, of which the rows' arrival 4,200, sums
// 6,200, meeting 3,200. One token 3.8 us: latency. Four of eight groups: 16384 x 256 4 us more, 1533 x 896 5 us; the groups'
// sums by a tree over the lanes that hold them (16384 x 256 16 us more with a loop over the groups, 1533 x 896 15), which groups
// that several of share a lane take.
#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kRtMaxCtas = 152;
constexpr int kRtTokens = 16;  // least tokens a CTA is given, where there are as many
// Set in the arrival word by a CTA whose wait gave up or met a word that was not left clean: no later call of this
// workspace takes stale counts for its own until the workspace is cleared.
constexpr uint32_t kRtBroken = 1u << 30;
constexpr int kRtIds = 64;     // picks of its run that a warp keeps in shared memory; the rest it reads back
constexpr int kRtStaged = 16;  // a lane's experts (J) from which rows come through shared memory
// Warps a CTA: 32 where a lane's experts (J) leave 64 registers enough, 24 where 80 (10922 tokens of 384 experts 19.8 us, with 16
// warps 23.0; 1000 tokens 10.2 and 9.5), else 16.
template <int J>
__host__ __device__ constexpr int rt_warps() { return J <= 8 ? 32 : J <= 16 ? 24 : 16; }

struct RtArgs {
  const void* logits;
  const float* bias;  // scored form: may be null
  int logits_f32, vec, T, E, top_k;
  float scale;
  int softmax, groups, group_size, top_groups, group_top, renormalise;  // scored form
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

// Rows of more than 256 experts come through shared memory: a lane's own experts are 64 bytes and more, and loads that far apart
// take a cycle of L1 each (1533 x 896, FP32: 4,200 clocks until a CTA's rows are there, 13,000 with a lane's own loads; up to 256
// experts a lane's loads are neighbours', and 16384 x 256 takes 18.1 us without, 20.1 with). A row is `each` units of 16 bytes a
// lane; unit c of a lane's stands where eight neighbours' units c are in different banks.
__device__ __forceinline__ int rt_unit(int lane, int c, int each) {
  return lane * each + (c ^ (lane * each / 8 & (each - 1)));
}
// Begins copying the row of E values of `size` (2 or 4) bytes at `from`: thread `first` of `step`.
template <int J>
__device__ __forceinline__ void rt_stage(const RtArgs& a, const void* from, int size, uint4* to, int first, int step) {
  const int shift = (J == 32 ? 2 : 1) + (size == 4), each = 1 << shift;  // units a lane: J * size / 16
  if (a.vec) {
    const uint4* src = static_cast<const uint4*>(from);
    for (int u = first; u < a.E * size / 16; u += step) cp_async_16(to + rt_unit(u >> shift, u & (each - 1), each), src + u);
  } else {
    const int in = 16 / size;  // values a unit
    for (int e = first; e < a.E; e += step) {
      uint4* unit = to + rt_unit(e / J, e % J / in, each);
      if (size == 4)
        reinterpret_cast<float*>(unit)[e % in] = __ldg(static_cast<const float*>(from) + e);
      else
        reinterpret_cast<uint16_t*>(unit)[e % in] = __ldg(static_cast<const uint16_t*>(from) + e);
    }
  }
  cp_async_commit();
}
// This lane's values of a staged row, 0 past the last expert.
template <int J>
__device__ __forceinline__ void rt_take(const RtArgs& a, const uint4* row, int size, int lane, float (&l)[J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] = 0.0f;
  if (size == 4) {
#pragma unroll
    for (int j = 0; j < J; j += 4) {
      const uint4 p = row[rt_unit(lane, j / 4, J / 4)];
      l[j] = __uint_as_float(p.x), l[j + 1] = __uint_as_float(p.y);
      l[j + 2] = __uint_as_float(p.z), l[j + 3] = __uint_as_float(p.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j + 8 <= J; j += 8) {
      const uint4 p = row[rt_unit(lane, j / 8, J / 8)];
      const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l[j + 2 * k] = __uint_as_float(w[k] << 16);
        l[j + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
    if (J * lane + j >= a.E) l[j] = 0.0f;
}

// p = rt_sigmoid of each of l. The rare far case stands outside the loop, so that the values' chains overlap.
template <int J>
__device__ __forceinline__ void rt_sigmoids(const float (&l)[J], float (&p)[J]) {
  bool near = true;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float d = __fadd_rn(1.0f, expf(-l[j]));
    near = near && d <= 0x1p125f;
    p[j] = recip_rn(d);
  }
  if (!near) {
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = rt_sigmoid(l[j]);
  }
}

// s's sum over the lanes below top_k, in their order (s is 0 above).
__device__ __forceinline__ float rt_sum(float s, int top_k) {
  float total = 0.0f;
  for (int r = 0; r < top_k; r += 8)
#pragma unroll
    for (int i = 0; i < 8; ++i) total = __fadd_rn(total, __shfl_sync(0xFFFFFFFFu, s, r + i));
  return total;
}

// The expert of rank `lane` (lanes below top_k) among the keys ky of experts J * lane .., and its logit; key 0: no expert. At least
// top_k keys are not 0. `most`: the largest of this lane's; `w`: 64 words of this warp's.
//
// The top_k-th largest of the 32 lane maxima is at most the top_k-th largest key. The keys from it up are few (about 9 of
// 256 for 8 picks, 22 of 896 for 16); where they are more than 32 (fewer than top_k lanes have keys, or a lane has many large
// ones), bisection finds a higher limit. They move to shared memory in the experts' order, and a key's rank is the number of
// those above it: every lane compares its own with all, which has no chain of shuffles (a token of 256 experts alone on its
// SM 3900 clocks, 5900 with both sets sorted in a bitonic network). Equal keys that no limit parts are picked one after another.
template <int J>
__device__ __forceinline__ int rt_select(const RtArgs& a, int t, uint32_t (&ky)[J], uint32_t most, int lane, uint32_t* w,
                                         float& logit) {
  const uint4* quads = reinterpret_cast<const uint4*>(w);
  w[lane] = most;
  __syncwarp();
  int above = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 q = quads[i];
    above += (q.x > most) + (q.y > most) + (q.z > most) + (q.w > most);
  }
  uint32_t floor_key = max(1u, __reduce_min_sync(0xFFFFFFFFu, above < a.top_k ? most : 0xFFFFFFFFu));
  __syncwarp();
  w[lane] = 0u;
  auto own = [&](uint32_t least) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) n += ky[j] >= least;
    return n;
  };
  int at = own(floor_key), count = __reduce_add_sync(0xFFFFFFFFu, at);
  if (count > 32) {
    // More than 32 keys from `low` up, fewer than top_k from `high` + 1 up.
    uint32_t low = floor_key, high = __reduce_max_sync(0xFFFFFFFFu, most);
    while (low < high) {
      floor_key = low + (high - low + 1) / 2;
      at = own(floor_key);
      count = __reduce_add_sync(0xFFFFFFFFu, at);
      if (count > 32)
        low = floor_key;
      else if (count < a.top_k)
        high = floor_key - 1;
      else
        break;
    }
    if (low >= high) count = 33;  // equal keys across the limit
  }
  int mine = 0;
  const int before = at;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, at, d);
    if (lane >= d) at += v;
  }
  at -= before;
  __syncwarp();
  if (count <= 32) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (ky[j] >= floor_key) {
        w[at] = ky[j];
        w[32 + at] = J * lane + j;
        ++at;
      }
    __syncwarp();
    const uint32_t key = w[lane], e = w[32 + lane];
    float v = 0.0f;
    if (lane < count) v = rt_value(a.logits, a.logits_f32, static_cast<size_t>(t) * a.E + e);
    int rank = 0;
#pragma unroll 2
    for (int i = 0; i < count; i += 4) {
      const uint4 q = quads[i / 4];
      // Of equal keys the lower expert's, which stands before, goes first.
      rank += q.x > key - (i < lane);
      rank += q.y > key - (i + 1 < lane);
      rank += q.z > key - (i + 2 < lane);
      rank += q.w > key - (i + 3 < lane);
    }
    __syncwarp();
    if (lane < count && rank < a.top_k) {
      w[rank] = e;
      w[32 + rank] = __float_as_uint(v);
    }
    __syncwarp();
    mine = static_cast<int>(w[lane]);
    logit = __uint_as_float(w[32 + lane]);
  } else {
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
    if (lane < a.top_k) logit = rt_value(a.logits, a.logits_f32, static_cast<size_t>(t) * a.E + mine);
  }
  return mine;
}

// The picks of token t: lane r < top_k gets rank r's expert and weight.
template <int J, typename Bias>
__device__ __forceinline__ void rt_pick(const RtArgs& a, Bias load_bias, const float (&l)[J], int t, int lane, uint32_t* w,
                                        int& my_e, float& my_w) {
  uint32_t ky[J];
  uint32_t most = 0u;
  float p[J], bias[J];
  rt_sigmoids<J>(l, p);
  load_bias(bias);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    // At least 1, so that an expert (a NaN key, too) always stands above a lane's empty places.
    ky[j] = J * lane + j < a.E ? max(1u, ordered_key(__fadd_rn(p[j], bias[j]))) : 0u;
    most = max(most, ky[j]);
  }
  float v = 0.0f;
  my_e = rt_select<J>(a, t, ky, most, lane, w, v);
  const float s = lane < a.top_k ? rt_sigmoid(v) : 0.0f;
  my_w = __fmul_rn(__fdiv_rn(s, rt_sum(s, a.top_k)), a.scale);
}

// The float of an ordered key.
__device__ __forceinline__ float rt_from_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Bit g: group g is among the top_groups whose best group_top keys sum to the most (ties: lower group). gk: keys of what the
// groups are compared by, 0 past the last expert; a group has group_top experts at least.
template <int J>
__device__ __forceinline__ uint32_t rt_groups(const RtArgs& a, const uint32_t (&gk)[J], int lane) {
  uint32_t mine = 0u;  // lane g: group g's sum, as a key
  auto sum_of = [&](uint32_t first, uint32_t second) {
    return a.group_top == 1 ? first : max(1u, ordered_key(__fadd_rn(rt_from_key(first), rt_from_key(second))));
  };
  uint32_t first = 0u, second = 0u;
  auto merge = [&](uint32_t f, uint32_t s) {
    second = max(min(first, f), max(second, s));
    first = max(first, f);
  };
  if (a.group_size % J == 0) {
    // A lane's experts are of one group, and a group those of `seg` lanes: a tree over them.
    const int seg = a.group_size / J, at = lane % seg;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      second = max(second, min(first, gk[j]));
      first = max(first, gk[j]);
    }
    for (int d = 1; d < seg; d <<= 1) {
      const uint32_t f = __shfl_down_sync(0xFFFFFFFFu, first, d), s = __shfl_down_sync(0xFFFFFFFFu, second, d);
      if (at + d < seg) merge(f, s);
    }
    mine = __shfl_sync(0xFFFFFFFFu, sum_of(first, second), lane * seg & 31);
    if (lane >= a.groups) mine = 0u;
  } else if (a.group_size >= J) {
    // A lane's experts are of one group or two neighbours. What it has of the second goes to the next lane, which begins in that
    // group; then a tree over the lanes that begin in one group.
    const int g0 = J * lane / a.group_size, own = (g0 + 1) * a.group_size - J * lane;
    uint32_t next = 0u, next2 = 0u;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t k = j < own ? gk[j] : 0u, n = j < own ? 0u : gk[j];
      second = max(second, min(first, k));
      first = max(first, k);
      next2 = max(next2, min(next, n));
      next = max(next, n);
    }
    next = __shfl_up_sync(0xFFFFFFFFu, next, 1);
    next2 = __shfl_up_sync(0xFFFFFFFFu, next2, 1);
    if (lane > 0) merge(next, next2);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t f = __shfl_down_sync(0xFFFFFFFFu, first, d), s = __shfl_down_sync(0xFFFFFFFFu, second, d);
      const int g = __shfl_down_sync(0xFFFFFFFFu, g0, d);
      if (lane + d < 32 && g == g0) merge(f, s);
    }
    mine = __shfl_sync(0xFFFFFFFFu, sum_of(first, second), (lane * a.group_size + J - 1) / J & 31);
    if (lane >= a.groups) mine = 0u;
  } else {
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      const int lo = g * a.group_size, hi = lo + a.group_size;
      first = second = 0u;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t k = J * lane + j >= lo && J * lane + j < hi ? gk[j] : 0u;
        second = max(second, min(first, k));
        first = max(first, k);
      }
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, first);
      uint32_t next = 0u;
      if (a.group_top == 2) {
        const int win = __ffs(__ballot_sync(0xFFFFFFFFu, first == top)) - 1;
        next = __reduce_max_sync(0xFFFFFFFFu, lane == win ? second : first);
      }
      if (lane == g) mine = sum_of(top, next);
    }
  }
  int rank = 0;
#pragma unroll 8
  for (int g = 0; g < a.groups; ++g) {
    const uint32_t k = __shfl_sync(0xFFFFFFFFu, mine, g);
    rank += k > mine || (k == mine && g < lane);
  }
  return __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank < a.top_groups);
}

// rt_pick of the scored form.
template <int J, typename Bias>
__device__ __forceinline__ void rt_pick_scored(const RtArgs& a, Bias load_bias, const float (&l)[J], int t, int lane,
                                               uint32_t* w, int& my_e, float& my_w) {
  float m = 0.0f, inv = 1.0f;  // softmax: scores are exp(l - m) * inv
  float p[J];
  if (a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (J * lane + j < a.E) m = fmaxf(m, l[j]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (m == -INFINITY) m = 0.0f;  // nothing but -inf: every score is 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      p[j] = J * lane + j < a.E ? expf(__fsub_rn(l[j], m)) : 0.0f;
      sum = __fadd_rn(sum, p[j]);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, d));
    inv = sum == 0.0f ? 0.0f : recip_rn(sum);  // sum in [1, 1024], or 0 (or NaN)
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = __fmul_rn(p[j], inv);
  } else {
    rt_sigmoids<J>(l, p);
  }
  if (a.bias != nullptr) {
    float bias[J];
    load_bias(bias);
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = __fadd_rn(p[j], bias[j]);
  }
  uint32_t ky[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    // (Adding 0 makes -0 the same key as 0; score + bias is never -0.)
    ky[j] = J * lane + j < a.E ? max(1u, ordered_key(a.bias != nullptr ? p[j] : __fadd_rn(l[j], 0.0f))) : 0u;
  }
  if (a.top_groups < a.groups) {
    uint32_t open;
    if (a.bias != nullptr || a.group_top == 1) {
      open = rt_groups<J>(a, ky, lane);
    } else {
      uint32_t gk[J];
#pragma unroll
      for (int j = 0; j < J; ++j) gk[j] = ky[j] == 0u ? 0u : max(1u, ordered_key(p[j]));
      open = rt_groups<J>(a, gk, lane);
    }
    int g = J * lane / a.group_size;
    if (a.group_size % J == 0) {  // one group a lane (past the last expert: keys are 0 already)
      const bool out = !(open >> (g & 31) & 1u);
#pragma unroll
      for (int j = 0; j < J; ++j) ky[j] = out ? 0u : ky[j];
    } else if (a.group_size >= J) {  // or two
      const int own = (g + 1) * a.group_size - J * lane;
      const bool out = !(open >> (g & 31) & 1u), out2 = !(open >> (g + 1 & 31) & 1u);
#pragma unroll
      for (int j = 0; j < J; ++j) ky[j] = (j < own ? out : out2) ? 0u : ky[j];
    } else {
      int next = (g + 1) * a.group_size;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (J * lane + j == next) {
          ++g;
          next += a.group_size;
        }
        if (g < 32 && !(open >> g & 1u)) ky[j] = 0u;
      }
    }
  }
  uint32_t most = 0u;
#pragma unroll
  for (int j = 0; j < J; ++j) most = max(most, ky[j]);
  float v = 0.0f;
  my_e = rt_select<J>(a, t, ky, most, lane, w, v);
  float s = 0.0f;
  if (lane < a.top_k) s = a.softmax ? expf(__fsub_rn(v, m)) : rt_sigmoid(v);
  if (a.renormalise) {
    const float total = rt_sum(s, a.top_k);
    my_w = total == 0.0f ? 0.0f : __fmul_rn(__fdiv_rn(s, total), a.scale);
  } else {
    my_w = __fmul_rn(a.softmax ? __fmul_rn(s, inv) : s, a.scale);
  }
}

template <int J, bool SCORED>
__global__ void __launch_bounds__(32 * rt_warps<J>()) route_kernel(const RtArgs a) {
  constexpr int kRtWarps = rt_warps<J>(), kRtThreads = 32 * kRtWarps;
  __shared__ uint16_t seen[kRtWarps][32 * J];    // routes of a warp's run per expert, then its next place
  __shared__ uint16_t picks[kRtWarps][kRtIds];   // the first picks of the run
  __shared__ union {
    uint4 keys[kRtWarps][16];               // while picking: rt_select's words
    int start[32 * J];                      // then: where this CTA's routes of an expert go
  } u;
  // Routes of every CTA, and of those before this one. A thread adds the counts of eight experts: theirs stand in eight rows
  // (or, two to a word, in four), so that neighbouring threads add to neighbouring words.
  __shared__ int all[32 * J], prev[32 * J];
  const bool pairs = gridDim.x > 1 && a.T < 65536;  // sums of 16 bits are enough
  auto count_of = [&](const int* sums, int e) {
    return pairs ? sums[(e & 7) / 2 * (4 * J) + (e >> 3)] >> (16 * (e & 1)) & 0xFFFF : sums[(e & 7) * (4 * J) + (e >> 3)];
  };
  __shared__ int warp_sum[kRtWarps];
  __shared__ int gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = gridDim.x;
  for (int e = lane; e < a.E; e += 32) seen[warp][e] = 0;
  for (int i = threadIdx.x; i < 32 * J; i += kRtThreads) all[i] = prev[i] = 0;
  if (threadIdx.x == 0) gave_up = 0;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  const int c0 = min(a.T, static_cast<int>(blockIdx.x) * a.per_cta), c1 = min(a.T, c0 + a.per_cta);
  const int t0 = min(c1, c0 + warp * a.per_warp), t1 = min(c1, t0 + a.per_warp);
  auto pick = [&](auto load_bias, const float(&l)[J], int t) {
    int e;
    float w;
    uint32_t* words = reinterpret_cast<uint32_t*>(u.keys[warp]);
    if (SCORED)
      rt_pick_scored<J>(a, load_bias, l, t, lane, words, e, w);
    else
      rt_pick<J>(a, load_bias, l, t, lane, words, e, w);
    if (lane < a.top_k) {
      a.ids[static_cast<size_t>(t) * a.top_k + lane] = e;
      a.weights[static_cast<size_t>(t) * a.top_k + lane] = w;
      const int i = (t - t0) * a.top_k + lane;
      if (i < kRtIds) picks[warp][i] = static_cast<uint16_t>(e);
      ++seen[warp][e];  // a token's picks are distinct: its lanes never meet on one counter
    }
    __syncwarp();
  };
  if constexpr (J >= kRtStaged) {
    extern __shared__ uint4 staged[];  // the bias, then a row a warp
    const int size = a.logits_f32 ? 4 : 2;
    uint4* row = staged + (1 + warp) * (32 * J / 4);
    auto stage = [&](int t) {
      rt_stage<J>(a, static_cast<const char*>(a.logits) + static_cast<size_t>(t) * a.E * size, size, row, lane, 32);
    };
    if (!SCORED || a.bias != nullptr) rt_stage<J>(a, a.bias, 4, staged, threadIdx.x, kRtThreads);
    if (t0 < t1) stage(t0);
    cp_async_wait<0>();
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
      float l[J];
      rt_take<J>(a, row, size, lane, l);
      __syncwarp();
      if (t + 1 < t1) stage(t + 1);
      pick([&](float(&bias)[J]) { rt_take<J>(a, staged, 4, lane, bias); }, l, t);
      cp_async_wait<0>();
      __syncwarp();
    }
  } else if (t0 < t1) {
    float bias[J], l[J], next[J];
#pragma unroll
    for (int j = 0; j < J; ++j) bias[j] = l[j] = next[j] = 0.0f;
    rt_load<J>(a, a.logits, a.logits_f32, static_cast<size_t>(t0) * a.E, lane, l);
    if (!SCORED || a.bias != nullptr) rt_load<J>(a, a.bias, true, 0, lane, bias);
    __syncwarp();
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) rt_load<J>(a, a.logits, a.logits_f32, static_cast<size_t>(t + 1) * a.E, lane, next);
      pick([&](float(&b)[J]) {
#pragma unroll
        for (int j = 0; j < J; ++j) b[j] = bias[j];
      }, l, t);
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
      all[(e & 7) * (4 * J) + (e >> 3)] = sum;
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
    // Eight experts a load; the CTAs' rows are dealt to as many threads as there are to a column, those that get none have
    // nothing to add (of few experts most: 8 experts, 1533 tokens 10.4 us with their zeros, 7.0 without).
    const int words = a.pitch / 8, lanes = min(kRtThreads / words, G), col = threadIdx.x % words, first = threadIdx.x / words;
    if (first < lanes) {
      constexpr int kRows = J <= 8 ? 5 : 12;  // on their way at once
      uint32_t pair[4] = {0u, 0u, 0u, 0u}, pair_prev[4] = {0u, 0u, 0u, 0u};
      int* const to[2] = {all + col, prev + col};
#pragma unroll 1
      for (int c0 = first; c0 < G; c0 += kRows * lanes) {
        uint4 p[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (c0 + i * lanes < G)
            p[i] = __ldcg(reinterpret_cast<const uint4*>(a.counts + static_cast<size_t>(c0 + i * lanes) * a.pitch) + col);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (c0 + i * lanes < G) {
            const uint32_t w[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
            const bool before = c0 + i * lanes < static_cast<int>(blockIdx.x);
            if (pairs) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                pair[k] += w[k];
                if (before) pair_prev[k] += w[k];
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int n = w[k / 2] >> (16 * (k & 1)) & 0xFFFFu;
                atomicAdd(to[0] + 4 * J * k, n);
                if (before) atomicAdd(to[1] + 4 * J * k, n);
              }
            }
          }
      }
      if (pairs) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          atomicAdd(to[0] + 4 * J * k, static_cast<int>(pair[k]));
          atomicAdd(to[1] + 4 * J * k, static_cast<int>(pair_prev[k]));
        }
      }
    }
  }
  __syncthreads();
  // Expert starts: two experts a thread (512 threads hold them all), a block scan.
  const int e0 = 2 * threadIdx.x;
  const int n0 = e0 < a.E ? count_of(all, e0) : 0, n1 = e0 + 1 < a.E ? count_of(all, e0 + 1) : 0;
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
  if (e0 < a.E) u.start[e0] = at + count_of(prev, e0);
  if (e0 + 1 < a.E) u.start[e0 + 1] = at + n0 + count_of(prev, e0 + 1);
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
  return kWorkspaceWords + ((static_cast<size_t>(rt_ctas(T)) * rt_pitch(E) * sizeof(uint16_t) + 255) & ~size_t(255));
}

int route(const void* logits, int logits_dtype, const float* bias, int T, int E, int top_k, const RouteScores* scored,
          float scale, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* tokens, void* workspace,
          size_t workspace_bytes, cudaStream_t st) {
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
  if (scored != nullptr) {
    a.softmax = scored->softmax ? 1 : 0;
    a.groups = scored->groups;
    a.group_size = E / scored->groups;
    a.top_groups = scored->top_groups;
    a.group_top = scored->group_top;
    a.renormalise = scored->renormalise ? 1 : 0;
  }
  // All CTAs of a launch meet, so there are no more than SMs.
  const int ctas = rt_ctas(T) < sms ? rt_ctas(T) : sms;
  a.per_cta = (T + ctas - 1) / ctas;
  const int warps = E <= 256 ? rt_warps<8>() : E <= 512 ? rt_warps<16>() : rt_warps<32>();
  a.per_warp = (a.per_cta + warps - 1) / warps;
  a.pitch = rt_pitch(E);
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.tokens = tokens;
  a.err = static_cast<uint32_t*>(workspace);
  a.sync = a.err + 16;
  a.counts = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + kWorkspaceWords);
  a.timeout_ns = wait_timeout_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // CTAs that meet run all or none: beside another stream's kernel that waits on its own CTAs, each could otherwise hold
  // SMs that the other needs. (2.6 us more in a stream, nothing in a graph.)
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const bool is_scored = scored != nullptr;
  void (*kernel)(RtArgs) = E <= 64    ? is_scored ? route_kernel<2, true> : route_kernel<2, false>
                           : E <= 256 ? is_scored ? route_kernel<8, true> : route_kernel<8, false>
                           : E <= 512 ? is_scored ? route_kernel<16, true> : route_kernel<16, false>
                                      : is_scored ? route_kernel<32, true> : route_kernel<32, false>;
  if (E > 256) {
    const int J = E <= 512 ? 16 : 32;
    cfg.dynamicSmemBytes = static_cast<size_t>(1 + warps) * 32 * J * sizeof(float);
    if (!ensure_smem_attr(dev, reinterpret_cast<const void*>(kernel), cfg.dynamicSmemBytes))
      return set_last_error(FME_ECUDA, "shared memory for the route kernel");
  }
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "route launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

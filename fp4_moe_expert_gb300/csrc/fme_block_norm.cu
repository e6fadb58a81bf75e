// What stands between a block and the next, in one pass over a token's row:
//
//   o = x[t]  or, combining routes,  sum_r w[t, r] x[t * top_k + r] (+ shared_out[t])   (FP32, ascending r)
//   p = o * rstd(o) * post_gamma       rstd(v) = 1 / sqrt(sum v^2 / H + eps); without post_gamma p = o
//   h = residual_scale * residual + gate * p
//   y = h * rstd(h) * gamma
//   residual_out = bf16(h), normed = bf16(y), and y in E4M3 per 128 (FP32 scales) or 32 (E8M0) values
//
// Everything between the loads and the stores is FP32 and stays in registers; the second norm takes the FP32 h, not its
// BF16 rounding, and the combined o is not rounded either: one rounding fewer at each, and the row need not be read
// again. Products and sums of the combination are rounded one by one as fme_moe_finalize's, the norm and the codes as
// fme_add_rmsnorm_fp8's.
//
// HBM-bound: 2 bytes a value for each row read, 4 to 5 written; what stands in the way are instructions, so values are worked
// on in pairs (f32x2), divisions are taken by one residual step, and rows that fill every thread's chunks have a kernel of their
// own (16384 x 7168 with a gate for every value 270 -> 201 us with the copies ahead and all three, 6.4 TB/s; 4096 tokens of 8
// routes 137 -> 109 us, 6.7 TB/s, the copy rate). Measured and left out (against 213 us of the gated form before the last
// step): four chunks a thread 229, one 284, five rows ahead 217, a CTA a row without copies ahead 269.
#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kBnChunks = 2;       // chunks of eight values a thread (wide rows)
constexpr int kBnAhead = 3;        // rows that it asks for ahead
constexpr int kBnThreads = 1024;   // threads an SM: 64 registers each
constexpr int kBnSmallRows = 8;  // rows a CTA, one a warp, where one warp holds a row

struct BnArgs {
  const __nv_bfloat16* x;
  const float* route_weights;
  const __nv_bfloat16* shared_out;
  const __nv_bfloat16* post_gamma;
  const __nv_bfloat16* gate;
  const __nv_bfloat16* residual;
  const __nv_bfloat16* gamma;
  long long ldx, ldg, ldr;
  int top_k, T, H;
  long long jump_x, step_shared, step_gate, step_residual;  // from a CTA's token's rows to its next one's, in 16 bytes
  float residual_scale, eps, inv_h;
  int quant, ue8m0;
  uint8_t* q;
  void* scales;
  __nv_bfloat16* normed;
  __nv_bfloat16* residual_out;
};

// Two FP32 values, worked on by one instruction (each as alone).
typedef unsigned long long BnPair;
__device__ __forceinline__ BnPair bn_pair(float lo, float hi) {
  BnPair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void bn_split(BnPair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ BnPair bn_mul(BnPair a, BnPair b) {
  BnPair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ BnPair bn_add(BnPair a, BnPair b) {
  BnPair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ BnPair bn_fma(BnPair a, BnPair b, BnPair c) {
  BnPair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// c + a b with both results rounded, value by value: the compiler fuses the pairs' multiplication and addition.
__device__ __forceinline__ BnPair bn_mul_add(float a, BnPair b, BnPair c) {
  float b0, b1, c0, c1;
  bn_split(b, b0, b1);
  bn_split(c, c0, c1);
  return bn_pair(__fadd_rn(c0, __fmul_rn(a, b0)), __fadd_rn(c1, __fmul_rn(a, b1)));
}
__device__ __forceinline__ void bn_unpack(const uint4& p, BnPair (&v)[4]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = bn_pair(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 bn_pack(const BnPair (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo, hi;
    bn_split(v[k], lo, hi);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(hi), "f"(lo));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / sqrt(mean square + eps) of a row, whose sum of squares is `total` over the row's threads. part: a warp's sum each,
// for rows of several warps.
template <bool SMALL>
__device__ __forceinline__ float bn_rstd(float total, float inv_h, float eps, float* part) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xFFFFFFFFu, total, d));
  if (!SMALL) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = total;
    __syncthreads();
    total = lane < blockDim.x / 32 ? part[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xFFFFFFFFu, total, d));
  }
  return rsqrtf(__fmaf_rn(total, inv_h, eps));
}

__device__ __noinline__ float bn_recip_far(float s) { return __fdiv_rn(1.0f, s); }
// 1 / s correctly rounded, for the scales of blocks: 1e-10 / 448 at least.
__device__ __forceinline__ float bn_recip(float s) {
  return s <= 0x1p80f ? __fmul_rn(recip_rn(__fmul_rn(s, 0x1p40f)), 0x1p40f) : bn_recip_far(s);
}

// Walks the rows that tokens' sums need, in the order of their use: of a token the block's (top_k of them or one), the
// shared expert's, the gate, the residual.
struct BnWalk {
  const uint4 *x, *shared, *gate, *residual;  // of the token, at this thread's first chunk
  int i;                                      // the next row
};
__device__ __forceinline__ BnWalk bn_walk(const BnArgs& a, int t, int first) {
  BnWalk w;
  const int n = a.top_k == 0 ? 1 : a.top_k;
  w.x = reinterpret_cast<const uint4*>(a.x + static_cast<long long>(t) * n * a.ldx) + first;
  w.shared = reinterpret_cast<const uint4*>(a.shared_out + static_cast<size_t>(t) * a.H) + first;
  w.gate = reinterpret_cast<const uint4*>(a.gate + t * a.ldg) + first;
  w.residual = reinterpret_cast<const uint4*>(a.residual + t * a.ldr) + first;
  w.i = 0;
  return w;
}
__device__ __forceinline__ const uint4* bn_next(const BnArgs& a, BnWalk& w) {
  int i = w.i++ - (a.top_k == 0 ? 1 : a.top_k);
  if (i < 0) {
    const uint4* r = w.x;
    w.x += a.ldx / 8;
    return r;
  }
  if (a.shared_out != nullptr && i-- == 0) return w.shared;
  if (a.gate != nullptr && i-- == 0) return w.gate;
  return w.residual;
}

// Token t, from o on: this thread's CH chunks of eight values, chunk c at 16-byte unit first + c * step of a row where mine[c].
// load(use) calls use(c, chunk) for the chunks of the next row of bn_row.
template <int CH, bool SMALL, typename Load>
__device__ __forceinline__ void bn_token(const BnArgs& a, int t, int first, int step, const bool (&mine)[CH],
                                         float (&part)[2][32], Load load) {
  BnPair v[CH][4];
  if (a.top_k == 0) {
    load([&](int c, const uint4& p) { bn_unpack(p, v[c]); });
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c][k] = 0ull;
    const float* weights = a.route_weights + static_cast<size_t>(t) * a.top_k;
    for (int r = 0; r < a.top_k; ++r) {
      const float w = __ldg(weights + r);
      load([&](int c, const uint4& p) {
        BnPair o[4];
        bn_unpack(p, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[c][k] = bn_mul_add(w, o[k], v[c][k]);
      });
    }
    if (a.shared_out != nullptr)
      load([&](int c, const uint4& p) {
        BnPair o[4];
        bn_unpack(p, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[c][k] = bn_add(v[c][k], o[k]);
      });
  }
  // Sum of squares and the vector of the norm, which is asked for before the sum is waited for.
  auto norm = [&](const __nv_bfloat16* gamma, float* sums) {
    uint4 g[CH];
    BnPair total = 0ull;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (mine[c]) {
        g[c] = __ldg(reinterpret_cast<const uint4*>(gamma) + first + c * step);
#pragma unroll
        for (int k = 0; k < 4; ++k) total = bn_fma(v[c][k], v[c][k], total);
      }
    float lo, hi;
    bn_split(total, lo, hi);
    const float rstd = bn_rstd<SMALL>(__fadd_rn(lo, hi), a.inv_h, a.eps, sums);
    const BnPair rr = bn_pair(rstd, rstd);
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (mine[c]) {
        BnPair w[4];
        bn_unpack(g[c], w);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[c][k] = bn_mul(bn_mul(v[c][k], rr), w[k]);
      }
  };
  if (a.post_gamma != nullptr) norm(a.post_gamma, part[0]);
  if (a.gate != nullptr)
    load([&](int c, const uint4& p) {
      BnPair g[4];
      bn_unpack(p, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c][k] = bn_mul(v[c][k], g[k]);
    });
  // residual_out may be the residual's buffer: this thread alone reads and writes these bytes.
  if (a.residual != nullptr) {
    const BnPair scale = bn_pair(a.residual_scale, a.residual_scale);
    load([&](int c, const uint4& p) {
      BnPair r[4];
      bn_unpack(p, r);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c][k] = bn_fma(scale, r[k], v[c][k]);
    });
  }
  const size_t row = static_cast<size_t>(t) * (a.H / 8) + first;  // in units of eight values
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (mine[c]) __stcs(reinterpret_cast<uint4*>(a.residual_out) + row + c * step, bn_pack(v[c]));
  if (a.gamma == nullptr) return;
  norm(a.gamma, part[1]);
  if (a.normed != nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (mine[c]) *(reinterpret_cast<uint4*>(a.normed) + row + c * step) = bn_pack(v[c]);
  }
  if (a.quant == FME_QUANT_NONE) return;
  const bool mx = a.quant == FME_QUANT_MXFP8;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float y[8], amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bn_split(v[c][k], y[2 * k], y[2 * k + 1]);
      if (mine[c]) amax = fmaxf(amax, fmaxf(fabsf(y[2 * k]), fabsf(y[2 * k + 1])));
    }
    // A block's chunks lie in neighbouring lanes and are all inside or all past the row's end.
    if (!mx) {
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 8));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    if (!mine[c]) continue;
    const int ch = first + c * step;
    float inv;
    if (mx) {
      const int ef = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
      const int e = ef == 0 ? -127 : max(-127, min(127, ef - 127 - 8));
      inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, -e in [-119, 127]
      if ((ch & 3) == 0)
        static_cast<uint8_t*>(a.scales)[static_cast<size_t>(t) * (a.H / 32) + ch / 4] = static_cast<uint8_t>(e + 127);
    } else {
      float s = quotient_rn(fmaxf(amax, 1e-10f), 448.0f, 1.0f / 448.0f);
      if (amax == INFINITY) s = INFINITY;  // (whose residual is NaN)
      if (a.ue8m0) s = ue8m0_ceil(s);
      inv = bn_recip(s);
      if ((ch & 15) == 0) static_cast<float*>(a.scales)[static_cast<size_t>(t) * (a.H / 128) + ch / 16] = s;
    }
    const BnPair ii = bn_pair(inv, inv);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) bn_split(bn_mul(v[c][k], ii), y[2 * k], y[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = f32x2_to_e4m3x2(y[4 * k], y[4 * k + 1]) | (f32x2_to_e4m3x2(y[4 * k + 2], y[4 * k + 3]) << 16);
    *(reinterpret_cast<uint2*>(a.q) + row + c * step) = make_uint2(w[0], w[1]);
  }
}

// Narrow rows: a warp a row.
template <int CH, bool WHOLE>
__global__ void __launch_bounds__(32 * kBnSmallRows) block_norm_small_kernel(const BnArgs a) {
  __shared__ float part[2][32];
  const int lane = threadIdx.x & 31, t = blockIdx.x * kBnSmallRows + (threadIdx.x >> 5);
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  if (t >= a.T) return;
  bool mine[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) mine[c] = WHOLE || lane + 32 * c < a.H / 8;
  BnWalk walk = bn_walk(a, t, lane);
  bn_token<CH, true>(a, t, lane, 32, mine, part, [&](auto use) {
    const uint4* from = bn_next(a, walk);
    uint4 p[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) p[c] = mine[c] ? __ldg(from + 32 * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int c = 0; c < CH; ++c) use(c, p[c]);
  });
}

// Wide rows: persistent CTAs, a token at a time. A thread's chunks are the same columns in every row, so it copies them itself,
// kBnAhead rows ahead (of this token or the next), into places of shared memory that are its own, and no barrier stands
// between a copy and its use.
template <int MOST, bool WHOLE>
__global__ void __launch_bounds__(MOST, kBnThreads / MOST) block_norm_kernel(const BnArgs a, const int rows) {
  constexpr int CH = kBnChunks, S = kBnAhead + 1;
  extern __shared__ uint4 ring[];  // [S][CH][threads]
  __shared__ float part[2][2][32];
  const int tid = threadIdx.x, threads = blockDim.x;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  bool mine[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) mine[c] = WHOLE || tid + threads * c < a.H / 8;
  uint4* const begin = ring + tid;
  uint4* const end = begin + S * CH * threads;
  int at = blockIdx.x;  // the token of the next row to ask for
  BnWalk walk = bn_walk(a, at, tid);
  uint4* into = begin;
  auto ask = [&]() {
    if (at < a.T) {
      const uint4* from = bn_next(a, walk);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (mine[c]) cp_async_16(into + threads * c, from + threads * c);
    }
    cp_async_commit();
    into += CH * threads;
    if (into == end) into = begin;
    if (walk.i == rows) {
      at += gridDim.x;
      walk.x += a.jump_x;
      walk.shared += a.step_shared;
      walk.gate += a.step_gate;
      walk.residual += a.step_residual;
      walk.i = 0;
    }
  };
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) ask();
  const uint4* slot = begin;
  int parity = 0;
#pragma unroll 1
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 1)
    bn_token<CH, false>(a, t, tid, threads, mine, part[parity], [&](auto use) {
      cp_async_wait<S - 2>();
#pragma unroll
      for (int c = 0; c < CH; ++c) use(c, mine[c] ? slot[threads * c] : make_uint4(0, 0, 0, 0));
      slot += CH * threads;
      if (slot == end) slot = begin;
      ask();  // into the slot before, whose row this thread has used
    });
}

template <int MOST, bool WHOLE>
static cudaError_t bn_launch(BnArgs a, int rows, int sms, int dev, cudaStream_t st) {
  const int threads = (a.H / 8 + 32 * kBnChunks - 1) / (32 * kBnChunks) * 32;
  const size_t place = (kBnAhead + 1) * kBnChunks * sizeof(uint4), smem = place * threads;  // place: a thread's
  const void* kernel = reinterpret_cast<const void*>(block_norm_kernel<MOST, WHOLE>);
  if (!ensure_smem_attr(dev, kernel, place * MOST)) return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  const int most = sms * (kBnThreads / threads);  // as many as an SM's registers hold
  const long long grid = a.T < most ? a.T : most, n = a.top_k == 0 ? 1 : a.top_k;
  a.jump_x = (grid - 1) * n * (a.ldx / 8);
  a.step_shared = grid * (a.H / 8);
  a.step_gate = grid * (a.ldg / 8);
  a.step_residual = grid * (a.ldr / 8);
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_norm_kernel<MOST, WHOLE>, a, rows);
}

template <int CH, bool WHOLE>
static cudaError_t bn_launch_small(const BnArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T + kBnSmallRows - 1) / kBnSmallRows));
  cfg.blockDim = dim3(32 * kBnSmallRows);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_norm_small_kernel<CH, WHOLE>, a);
}

int block_norm(const BlockNorm& b, cudaStream_t st) {
  BnArgs a = {};
  a.x = static_cast<const __nv_bfloat16*>(b.x);
  a.route_weights = b.route_weights;
  a.shared_out = static_cast<const __nv_bfloat16*>(b.shared_out);
  a.post_gamma = static_cast<const __nv_bfloat16*>(b.post_gamma);
  a.gate = static_cast<const __nv_bfloat16*>(b.gate);
  a.residual = static_cast<const __nv_bfloat16*>(b.residual);
  a.gamma = static_cast<const __nv_bfloat16*>(b.gamma);
  a.ldx = b.ldx;
  a.ldg = b.ldg;
  a.ldr = b.ldr;
  a.top_k = b.top_k;
  a.T = b.T;
  a.H = b.H;
  a.residual_scale = b.residual_scale;
  a.eps = b.eps;
  a.inv_h = 1.0f / static_cast<float>(b.H);
  a.quant = b.quant;
  a.ue8m0 = b.ue8m0 ? 1 : 0;
  a.q = b.q;
  a.scales = b.scales;
  a.normed = static_cast<__nv_bfloat16*>(b.normed);
  a.residual_out = static_cast<__nv_bfloat16*>(b.residual_out);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return set_last_error(FME_ECUDA, "cudaGetDevice failed");
  const int sms = device_sm_count(dev);
  if (sms <= 0) return set_last_error(FME_ECUDA, "no SM count for device %d", dev);
  const int chunks = a.H / 8;
  const int rows = (a.top_k == 0 ? 1 : a.top_k) + (a.shared_out != nullptr) + (a.gate != nullptr) + (a.residual != nullptr);
  // A warp a row up to 1024 values (16384 tokens of 1024: 26 us, of the wide kernel 29). Rows that fill every thread's chunks
  // have no values to ask about (16384 x 7168 with a gate 213 -> 201 us).
  cudaError_t err;
  if (chunks <= 32)
    err = chunks == 32 ? bn_launch_small<1, true>(a, st) : bn_launch_small<1, false>(a, st);
  else if (chunks <= 64)
    err = chunks == 64 ? bn_launch_small<2, true>(a, st) : bn_launch_small<2, false>(a, st);
  else if (chunks <= 128)
    err = chunks == 128 ? bn_launch_small<4, true>(a, st) : bn_launch_small<4, false>(a, st);
  else if (chunks <= 1024)
    err = chunks % (32 * kBnChunks) == 0 ? bn_launch<512, true>(a, rows, sms, dev, st)
                                         : bn_launch<512, false>(a, rows, sms, dev, st);
  else
    err = chunks % (32 * kBnChunks) == 0 ? bn_launch<1024, true>(a, rows, sms, dev, st)
                                         : bn_launch<1024, false>(a, rows, sms, dev, st);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "block norm launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

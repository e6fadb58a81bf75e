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
// HBM-bound: 2 bytes a value for each row read, 4 to 5 written.
#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kBnChunks = 4;     // chunks of eight values a thread
constexpr int kBnRowWarps = 16;  // most warps a row: 16384 values
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
  float residual_scale, eps;
  int quant, ue8m0;
  uint8_t* q;
  void* scales;
  __nv_bfloat16* normed;
  __nv_bfloat16* residual_out;
};

__device__ __forceinline__ void bn_unpack(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 bn_pack(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * k]))) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * k + 1]))) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / sqrt(mean square + eps) of a row, whose sum of squares is `total` over the row's threads.
template <bool SMALL>
__device__ __forceinline__ float bn_rstd(float total, int warps, int H, float eps, float* part) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xFFFFFFFFu, total, d));
  if (!SMALL) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = total;
    __syncthreads();
    total = 0.0f;
    for (int w = 0; w < warps; ++w) total = __fadd_rn(total, part[w]);
  }
  return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(total, static_cast<float>(H)), eps)));
}

// SMALL: a warp a row, kBnSmallRows a CTA; otherwise the CTA is the row's.
template <bool SMALL>
__global__ void __launch_bounds__(SMALL ? 32 * kBnSmallRows : 32 * kBnRowWarps) block_norm_kernel(const BnArgs a) {
  __shared__ float part[2][kBnRowWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = SMALL ? blockIdx.x * kBnSmallRows + warp : blockIdx.x;
  const int rt = SMALL ? lane : threadIdx.x, width = SMALL ? 32 : blockDim.x;  // thread of the row, threads a row
  const int chunks = t < a.T ? a.H / 8 : 0;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  float v[kBnChunks][8];
  if (a.top_k == 0) {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + t * a.ldx);
#pragma unroll
    for (int c = 0; c < kBnChunks; ++c)
      bn_unpack(rt + width * c < chunks ? __ldcs(x + rt + width * c) : make_uint4(0, 0, 0, 0), v[c]);
  } else {
#pragma unroll
    for (int c = 0; c < kBnChunks; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[c][k] = 0.0f;
    const long long first = static_cast<long long>(t) * a.top_k;
    if (t < a.T)
#pragma unroll 2
      for (int r = 0; r < a.top_k; ++r) {
        const float w = __ldg(a.route_weights + first + r);
        const uint4* x = reinterpret_cast<const uint4*>(a.x + (first + r) * a.ldx);
        uint4 p[kBnChunks];
#pragma unroll
        for (int c = 0; c < kBnChunks; ++c)
          if (rt + width * c < chunks) p[c] = __ldcs(x + rt + width * c);
#pragma unroll
        for (int c = 0; c < kBnChunks; ++c)
          if (rt + width * c < chunks) {
            float o[8];
            bn_unpack(p[c], o);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[c][k] = __fadd_rn(v[c][k], __fmul_rn(w, o[k]));
          }
      }
    if (a.shared_out != nullptr) {
      const uint4* s = reinterpret_cast<const uint4*>(a.shared_out + static_cast<size_t>(t) * a.H);
#pragma unroll
      for (int c = 0; c < kBnChunks; ++c)
        if (rt + width * c < chunks) {
          float o[8];
          bn_unpack(__ldcs(s + rt + width * c), o);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[c][k] = __fadd_rn(v[c][k], o[k]);
        }
    }
  }
  uint4 res[kBnChunks];
  if (a.residual != nullptr) {
    // residual_out may be the same buffer: this thread alone reads and writes these bytes.
    const uint4* r = reinterpret_cast<const uint4*>(a.residual + t * a.ldr);
#pragma unroll
    for (int c = 0; c < kBnChunks; ++c)
      if (rt + width * c < chunks) res[c] = __ldcs(r + rt + width * c);
  }
  if (a.post_gamma != nullptr) {
    float total = 0.0f;
#pragma unroll
    for (int c = 0; c < kBnChunks; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) total = __fmaf_rn(v[c][k], v[c][k], total);
    const float rstd = bn_rstd<SMALL>(total, width / 32, a.H, a.eps, part[0]);
#pragma unroll
    for (int c = 0; c < kBnChunks; ++c)
      if (rt + width * c < chunks) {
        float g[8];
        bn_unpack(__ldg(reinterpret_cast<const uint4*>(a.post_gamma) + rt + width * c), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = __fmul_rn(__fmul_rn(v[c][k], rstd), g[k]);
      }
  }
  if (a.gate != nullptr) {
    const uint4* gate = reinterpret_cast<const uint4*>(a.gate + t * a.ldg);
#pragma unroll
    for (int c = 0; c < kBnChunks; ++c)
      if (rt + width * c < chunks) {
        float g[8];
        bn_unpack(__ldg(gate + rt + width * c), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = __fmul_rn(v[c][k], g[k]);
      }
  }
  float total = 0.0f;
#pragma unroll
  for (int c = 0; c < kBnChunks; ++c)
    if (rt + width * c < chunks) {
      if (a.residual != nullptr) {
        float r[8];
        bn_unpack(res[c], r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = __fadd_rn(__fmul_rn(a.residual_scale, r[k]), v[c][k]);
      }
      *(reinterpret_cast<uint4*>(a.residual_out + static_cast<size_t>(t) * a.H) + rt + width * c) = bn_pack(v[c]);
#pragma unroll
      for (int k = 0; k < 8; ++k) total = __fmaf_rn(v[c][k], v[c][k], total);
    }
  if (a.gamma == nullptr) return;
  const float rstd = bn_rstd<SMALL>(total, width / 32, a.H, a.eps, part[1]);
#pragma unroll
  for (int c = 0; c < kBnChunks; ++c) {
    const int ch = rt + width * c;
    const bool mine = ch < chunks;
    float amax = 0.0f;
    if (mine) {
      float g[8];
      bn_unpack(__ldg(reinterpret_cast<const uint4*>(a.gamma) + ch), g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[c][k] = __fmul_rn(__fmul_rn(v[c][k], rstd), g[k]);
        amax = fmaxf(amax, fabsf(v[c][k]));
      }
      if (a.normed != nullptr)
        *(reinterpret_cast<uint4*>(a.normed + static_cast<size_t>(t) * a.H) + ch) = bn_pack(v[c]);
    }
    if (a.quant == FME_QUANT_NONE) continue;
    // A block's chunks lie in neighbouring lanes and are all inside or all past the row's end.
    const bool mx = a.quant == FME_QUANT_MXFP8;
    if (!mx) {
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 8));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    if (!mine) continue;
    float inv;
    if (mx) {
      const int ef = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
      const int e = ef == 0 ? -127 : max(-127, min(127, ef - 127 - 8));
      inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, -e in [-119, 127]
      if ((ch & 3) == 0)
        static_cast<uint8_t*>(a.scales)[static_cast<size_t>(t) * (a.H / 32) + ch / 4] = static_cast<uint8_t>(e + 127);
    } else {
      float s = __fdiv_rn(fmaxf(amax, 1e-10f), 448.0f);
      if (a.ue8m0) s = ue8m0_ceil(s);
      inv = __fdiv_rn(1.0f, s);
      if ((ch & 15) == 0) static_cast<float*>(a.scales)[static_cast<size_t>(t) * (a.H / 128) + ch / 16] = s;
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = f32x2_to_e4m3x2(__fmul_rn(v[c][4 * k], inv), __fmul_rn(v[c][4 * k + 1], inv)) |
             (f32x2_to_e4m3x2(__fmul_rn(v[c][4 * k + 2], inv), __fmul_rn(v[c][4 * k + 3], inv)) << 16);
    *(reinterpret_cast<uint2*>(a.q + static_cast<size_t>(t) * a.H) + ch) = make_uint2(w[0], w[1]);
  }
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
  a.quant = b.quant;
  a.ue8m0 = b.ue8m0 ? 1 : 0;
  a.q = b.q;
  a.scales = b.scales;
  a.normed = static_cast<__nv_bfloat16*>(b.normed);
  a.residual_out = static_cast<__nv_bfloat16*>(b.residual_out);
  const int warps = (a.H / 8 + 32 * kBnChunks - 1) / (32 * kBnChunks);
  const bool small = warps == 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(small ? (a.T + kBnSmallRows - 1) / kBnSmallRows : a.T));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * (small ? kBnSmallRows : warps)));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = small ? cudaLaunchKernelEx(&cfg, block_norm_kernel<true>, a)
                                : cudaLaunchKernelEx(&cfg, block_norm_kernel<false>, a);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "block norm launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

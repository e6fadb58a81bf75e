// Residual addition, RMSNorm and 8-bit quantisation of BF16 rows in one pass.
//
//   z = bf16(x + residual)                     (FP32 addition, one rounding; z = x without a residual)
//   rstd = 1 / sqrt(sum z^2 / H + eps),  y = (z * rstd) * gamma        (FP32)
//   FP8    per 128 values: s = max(amax |y|, 1e-10) / 448 (a power of two when ue8m0), q = e4m3(y * (1 / s))
//   MXFP8  per 32 values: e = floor(log2 amax |y|) - 8 in [-127, 127], q = e4m3(y * 2^-e), scale byte e + 127
//   normed = bf16(y), residual_out = z
//
// HBM-bound: 2 (4 with a residual) bytes a value read, 1 to 5 written. Each row is
// read once, into registers as the BF16 values z are (16 registers a thread: four
// chunks of eight values), by the fewest warps that hold it so; a block's amax takes
// shuffles over its 16 (4) threads. 16384 x 7168 with residual and BF16 norm: 156 us,
// 6.8 TB/s, the rate of a plain copy; one row: about 4 us, its latency.
#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kNqChunks = 4;     // chunks of eight values a thread
constexpr int kNqRowWarps = 16;  // most warps a row: 16384 values
constexpr int kNqSmallRows = 8;  // rows a CTA, one a warp, where one warp holds a row

struct NqArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;  // null: none
  const __nv_bfloat16* gamma;
  long long ldx, ldr;
  int T, H;
  float eps;
  int ue8m0;
  uint8_t* q;
  float* scales;      // FP8
  uint8_t* mxscales;  // MXFP8
  __nv_bfloat16* normed;
  __nv_bfloat16* residual_out;
};

__device__ __forceinline__ void nq_unpack(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 nq_pack(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * k]))) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * k + 1]))) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// SMALL: a warp a row, kNqSmallRows a CTA; otherwise the CTA is the row's.
template <bool MX, bool SMALL>
__global__ void __launch_bounds__(SMALL ? 32 * kNqSmallRows : 32 * kNqRowWarps) add_rmsnorm_quant_kernel(const NqArgs a) {
  __shared__ float part[kNqRowWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = SMALL ? blockIdx.x * kNqSmallRows + warp : blockIdx.x;
  const int rt = SMALL ? lane : threadIdx.x, width = SMALL ? 32 : blockDim.x;  // thread of the row, threads a row
  const int chunks = t < a.T ? a.H / 8 : 0;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  const uint4* x = reinterpret_cast<const uint4*>(a.x + t * a.ldx);
  uint4 z[kNqChunks];
#pragma unroll
  for (int c = 0; c < kNqChunks; ++c) {
    z[c] = make_uint4(0, 0, 0, 0);
    if (rt + width * c < chunks) z[c] = __ldcs(x + rt + width * c);
  }
  if (a.residual != nullptr) {
    const uint4* res = reinterpret_cast<const uint4*>(a.residual + t * a.ldr);
    uint4* res_out = reinterpret_cast<uint4*>(a.residual_out + static_cast<size_t>(t) * a.H);
    uint4 r[kNqChunks];
    // residual_out may be the same buffer: this thread alone reads and writes these bytes.
#pragma unroll
    for (int c = 0; c < kNqChunks; ++c)
      if (rt + width * c < chunks) r[c] = __ldcs(res + rt + width * c);
#pragma unroll
    for (int c = 0; c < kNqChunks; ++c)
      if (rt + width * c < chunks) {
        float v[8], w[8];
        nq_unpack(z[c], v);
        nq_unpack(r[c], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __fadd_rn(v[k], w[k]);
        z[c] = nq_pack(v);
        res_out[rt + width * c] = z[c];
      }
  }
  float total = 0.0f;
#pragma unroll
  for (int c = 0; c < kNqChunks; ++c) {
    float v[8];
    nq_unpack(z[c], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) total = __fmaf_rn(v[k], v[k], total);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xFFFFFFFFu, total, d));
  if (!SMALL) {
    if (lane == 0) part[warp] = total;
    __syncthreads();
    total = 0.0f;
    for (int w = 0; w < width / 32; ++w) total = __fadd_rn(total, part[w]);
  }
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(total, static_cast<float>(a.H)), a.eps)));
#pragma unroll
  for (int c = 0; c < kNqChunks; ++c) {
    const int ch = rt + width * c;
    const bool mine = ch < chunks;
    float amax = 0.0f, y[8];
    if (mine) {
      float g[8];
      nq_unpack(z[c], y);
      nq_unpack(__ldg(reinterpret_cast<const uint4*>(a.gamma) + ch), g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y[k] = __fmul_rn(__fmul_rn(y[k], rstd), g[k]);
        amax = fmaxf(amax, fabsf(y[k]));
      }
      if (a.normed != nullptr)
        *(reinterpret_cast<uint4*>(a.normed + static_cast<size_t>(t) * a.H) + ch) = nq_pack(y);
    }
    // A block's chunks lie in neighbouring lanes and are all inside or all past the row's end.
#pragma unroll
    for (int d = (MX ? 2 : 8); d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    if (!mine) continue;
    float inv;
    if (MX) {
      const int ef = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
      const int e = ef == 0 ? -127 : max(-127, min(127, ef - 127 - 8));
      inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, -e in [-119, 127]
      if ((ch & 3) == 0) a.mxscales[static_cast<size_t>(t) * (a.H / 32) + ch / 4] = static_cast<uint8_t>(e + 127);
    } else {
      float s = __fdiv_rn(fmaxf(amax, 1e-10f), 448.0f);
      if (a.ue8m0) s = ue8m0_ceil(s);
      inv = __fdiv_rn(1.0f, s);
      if ((ch & 15) == 0) a.scales[static_cast<size_t>(t) * (a.H / 128) + ch / 16] = s;
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = f32x2_to_e4m3x2(__fmul_rn(y[4 * k], inv), __fmul_rn(y[4 * k + 1], inv)) |
             (f32x2_to_e4m3x2(__fmul_rn(y[4 * k + 2], inv), __fmul_rn(y[4 * k + 3], inv)) << 16);
    *(reinterpret_cast<uint2*>(a.q + static_cast<size_t>(t) * a.H) + ch) = make_uint2(w[0], w[1]);
  }
}

template <bool MX>
static cudaError_t nq_launch(const NqArgs& a, cudaStream_t st) {
  const int warps = (a.H / 8 + 32 * kNqChunks - 1) / (32 * kNqChunks);
  const bool small = warps == 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(small ? (a.T + kNqSmallRows - 1) / kNqSmallRows : a.T));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * (small ? kNqSmallRows : warps)));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return small ? cudaLaunchKernelEx(&cfg, add_rmsnorm_quant_kernel<MX, true>, a)
               : cudaLaunchKernelEx(&cfg, add_rmsnorm_quant_kernel<MX, false>, a);
}

int add_rmsnorm_quant(const void* x, long long ldx, const void* residual, long long ldr, const void* gamma, int T, int H,
                      float eps, int ue8m0, uint8_t* q, float* scales, uint8_t* mxscales, void* normed,
                      void* residual_out, cudaStream_t st) {
  NqArgs a = {};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.residual = static_cast<const __nv_bfloat16*>(residual);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.ldx = ldx;
  a.ldr = ldr;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.ue8m0 = ue8m0 ? 1 : 0;
  a.q = q;
  a.scales = scales;
  a.mxscales = mxscales;
  a.normed = static_cast<__nv_bfloat16*>(normed);
  a.residual_out = static_cast<__nv_bfloat16*>(residual_out);
  const cudaError_t err = mxscales != nullptr ? nq_launch<true>(a, st) : nq_launch<false>(a, st);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "add rmsnorm launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

// out = act(x W^T + bias) + residual, BF16 x [M, K] and W [N, K], FP32 sums, one rounding to the output's type.
//
// Three kernels.
//
// linear_one_kernel, one token: a warp (or 2, 4, 8 that share its K range) multiplies kLnRows weight rows, 16 bytes of each
// a lane and load. Bound by latency where the weights are few (256 x 7168: 2.7 us, from HBM 3.8) and by their stream where they are many
// (4096 x 7168: 13 us, 4.4 TB/s).
//
// linear_few_kernel, up to 16 tokens (ln_few): warps hold 16 tokens x 8 weight rows in mma.sync fragments, loaded straight
// from global memory. A tcgen05 tile needs its operands in shared memory, tensor memory allocated and a pipeline filled,
// which is 3 us before the first result; here 8 tokens of 256 x 7168 take 4.6 us instead of 6.3.
//
// linear_tc_kernel, the rest: one persistent CTA per SM walks units, tiles of up to 128 tokens x tile_n weight rows (a
// multiple of 16 up to 256) times a share of K. Twelve warps: two load by TMA (tokens and weights, 128-byte swizzle), one
// issues tcgen05.mma kind::f16, eight read the accumulators (two buffers in tensor memory, so that a tile's epilogue runs
// beside the next tile's products). Where the tiles are fewer than SMs, K is cut, too: a unit's epilogue warps then store their
// FP32 sums to the workspace, and of a tile's units the last to have a warp's part there adds them in K order, whichever it is,
// so the result does not hang on the order of arrival, and no unit waits for another. Counts that no call left are found and the
// workspace refused until it is cleared. (A warp's parts in 16-byte pieces, counted by one release and acquire a warp: 128 x 256
// x 7168 FP32 9.2 us; value by value behind barriers and fences of the CTA 11.8.)
// * A stage holds as many K blocks of 64 values as fit 64 KB: a TMA instruction costs its warp about 100 ns whatever it
//   brings (16 tokens x 7168 x 2048: 12.3 us with one block a stage and one loading warp, 7.8 with eight and two).
// * FP32 outputs: the tensor core's accumulation truncates, so a chain of 448 instructions (K = 7168) is 8e-6 of the result
//   off. Accumulations of about kLnChunk blocks are added with rounding instead: 5e-7. They stand side by side in tensor memory
//   where a unit's fit (128 x 256 x 7168 9.2 -> 7.8 us), else they are added in registers as they end (CHUNKED: 16384 x 256 x
//   7168 57.5 us, the chain 53.8). BF16 outputs, whose rounding is 250 times that, take the chain.
// (Times of 64 x 7168 x 2048 below are with its weights in L2, as repeated calls find them; from HBM it takes 9.1 us.)
// What bounds it: large products shared memory's 128 bytes a clock. A K block of a 128 x 256 tile is written there (48 KB)
// and read by the MMAs (48 KB), 750 clocks against 512 of MMA; measured 744 (16384 x 4096 x 7168: 575 us, 1670 TFLOP/s, in a
// burst; 615 to 640 at the power limit. The tiles' order counts: 771 us with the row tiles of one weight tile one after
// another). Small tiles the same: an MMA reads its 128 (up to 64 tokens: 64) token rows whatever it has of them, so one of
// 48 columns takes 70 clocks as one of 256 takes 190 (64 x 7168 x 2048: 8.1 us with 128 rows, 7.0 with 64). Measured and
// left out: 256 x 256 tiles, two accumulators that share the weights, with three stages of 64 KB (626 us against 577) and
// with six of half as many values (809: TMA takes rows of 64 bytes no faster than rows of 128); prefetches into L2 ahead of
// the ring (router of 16384 tokens 57.8 against 57.4 us, 64 x 4096 x 7168 18.1 against 17.4); CTAs that start at different
// places of K (no difference); two CTAs an SM with half the ring (64 x 7168 x 2048 11.2 us against 9.1); partial sums with a
// row's columns together (512 x 256 x 7168 17 us against 12.5). Rows whose stride is an odd multiple of 16 bytes cost more:
// 128 bytes of a row then lie in five sectors (1533 x 895 x 3581 22.8 us, with strides of whole sectors 17.3).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

struct LnEpilogue {
  const float* bias;     // null: none
  const void* residual;  // null: none; the output's type
  long long ldr, ldo;
  void* out;
  int act, out_f32;
  int bias16;  // bias is 16-byte aligned
  int wide;    // bytes that out (and residual) rows start at multiples of, where those are 32 or 16
  int M, N;
};

// ---------------------------------------------------------------- epilogue
// Sigmoid by the exponential of -|z|, which never overflows: 1 / (1 + exp(-z)) is 0 below z = -88.72, where SiLU, z times
// it, is still 2e-37. The divisor is in [1, 2].
__device__ __forceinline__ float ln_sigmoid(float z) {
  const float e = expf(-fabsf(z)), r = recip_rn(__fadd_rn(1.0f, e));
  return z < 0.0f ? __fmul_rn(e, r) : r;
}

// NaN stays NaN in each.
__device__ __forceinline__ float ln_act(float z, int act) {
  switch (act) {
    case FME_ACT_RELU:
      return z < 0.0f ? 0.0f : z;
    case FME_ACT_SILU:
      return __fmul_rn(z, ln_sigmoid(z));
    case FME_ACT_GELU:  // z P(N(0, 1) < z); erfc keeps the tail's relative precision, which 1 + erf loses
      return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(z, -0.70710678f)));
    case FME_ACT_SIGMOID:
      return ln_sigmoid(z);
    default:
      return z;
  }
}

// One value at (row, n).
__device__ __forceinline__ void ln_store(const LnEpilogue& e, float z, int row, int n) {
  if (e.bias != nullptr) z = __fadd_rn(z, __ldg(e.bias + n));
  z = ln_act(z, e.act);
  const size_t r = static_cast<size_t>(row) * e.ldr + n, o = static_cast<size_t>(row) * e.ldo + n;
  if (e.out_f32) {
    if (e.residual != nullptr) z = __fadd_rn(z, static_cast<const float*>(e.residual)[r]);
    static_cast<float*>(e.out)[o] = z;
  } else {
    if (e.residual != nullptr) z = __fadd_rn(z, __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[r]));
    static_cast<__nv_bfloat16*>(e.out)[o] = __float2bfloat16_rn(z);
  }
}

__device__ __forceinline__ void ln_st32(void* p, const uint32_t (&w)[8], bool sector) {
  if (sector) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void ln_ld32(const void* p, uint32_t (&w)[8], bool sector) {
  if (sector) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 lo = static_cast<const uint4*>(p)[0], hi = static_cast<const uint4*>(p)[1];
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
    w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
  }
}
__device__ __forceinline__ uint32_t ln_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 256 sigmoid(z) for outputs of 8 bits' precision: the hardware's approximate exponential and reciprocal, of the divisor by
// 256, so that neither overflows nor is flushed to zero before SiLU is below the normal numbers (z = -92.9). Argument,
// exponential and reciprocal together: 4 + 1.2 |z| units of 2^-23.
__device__ __forceinline__ float ln_sigmoid256(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(z, -1.44269504f, -8.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(0x1p-8f, e)));
  return r;
}

// Sixteen sums of one row, columns n .. n + 15: bias and activation. (The cases stand outside the loops: inside them each
// value's code holds every case's.) BF16 outputs take exp and reciprocal by the hardware's approximations.
__device__ __forceinline__ void ln_finish16(const LnEpilogue& e, const float* bias, int act, float (&z)[16], int n) {
  if (bias != nullptr && e.bias16 && n + 16 <= e.N) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(bias + n) + i);
      z[4 * i] = __fadd_rn(z[4 * i], b.x);
      z[4 * i + 1] = __fadd_rn(z[4 * i + 1], b.y);
      z[4 * i + 2] = __fadd_rn(z[4 * i + 2], b.z);
      z[4 * i + 3] = __fadd_rn(z[4 * i + 3], b.w);
    }
  } else if (bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __fadd_rn(z[i], n + i < e.N ? __ldg(bias + n + i) : 0.0f);
  }
  if (act == FME_ACT_NONE) return;
  if (act == FME_ACT_SILU && !e.out_f32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __fmul_rn(__fmul_rn(z[i], 0x1p-8f), ln_sigmoid256(z[i]));
  } else if (act == FME_ACT_SIGMOID && !e.out_f32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __fmul_rn(ln_sigmoid256(z[i]), 0x1p-8f);
  } else if (act == FME_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = ln_act(z[i], FME_ACT_RELU);
  } else if (act == FME_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = ln_act(z[i], FME_ACT_SILU);
  } else if (act == FME_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = ln_act(z[i], FME_ACT_SIGMOID);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = ln_act(z[i], FME_ACT_GELU);
  }
}

// A chunk is sixteen columns of a warp's 32 rows. Whole chunks of rows that start at multiples of 16 bytes are loaded and
// stored as the accumulator gives them, a lane a row, 32 (sector) or 16 bytes at a time.
__device__ __forceinline__ void ln_load_whole(uint32_t (&raw)[16], const char* from, int size, bool sector) {
  uint32_t w[8];
  ln_ld32(from, w, sector);
#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i] = w[i];
  if (size == 4) {
    ln_ld32(from + 32, w, sector);
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[8 + i] = w[i];
  }
}
__device__ __forceinline__ void ln_add_whole(float (&z)[16], const uint32_t (&raw)[16], int size) {
  if (size == 4) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __fadd_rn(z[i], __uint_as_float(raw[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[2 * i] = __fadd_rn(z[2 * i], __uint_as_float(raw[i] << 16));
      z[2 * i + 1] = __fadd_rn(z[2 * i + 1], __uint_as_float(raw[i] & 0xFFFF0000u));
    }
  }
}
__device__ __forceinline__ void ln_store_whole(const float (&z)[16], char* to, int size, bool sector) {
  uint32_t w[8];
  if (size == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(z[8 * h + i]);
      ln_st32(to + 32 * h, w, sector);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ln_bf16x2(z[2 * i], z[2 * i + 1]);
    ln_st32(to, w, sector);
  }
}

// Other chunks (columns n .. n + 15, the first `cols` of them; rows from `row`, the first `rows` of them) are turned through
// shared memory, so that neighbouring lanes store neighbouring values (1533 x 895 x 3584: 16.4 us; a lane a row, value by value,
// 41.7).
struct LnChunk {
  int row, rows, n, cols;
};
// The residual of a chunk, asked for before its sums are read: bits of the values this lane stores.
__device__ __forceinline__ void ln_load_turned(const LnEpilogue& e, const LnChunk& c, int lane, uint32_t (&raw)[16]) {
  if ((lane & 15) >= c.cols) return;
  const int r0 = lane >> 4;
  const size_t at = static_cast<size_t>(c.row + r0) * e.ldr + c.n + (lane & 15);
  if (e.out_f32) {
    const float* from = static_cast<const float*>(e.residual) + at;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i + r0 < c.rows) raw[i] = __float_as_uint(from[2 * i * e.ldr]);
  } else {
    const uint16_t* from = static_cast<const uint16_t*>(e.residual) + at;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i + r0 < c.rows) raw[i] = from[2 * i * e.ldr];
#pragma unroll
    for (int i = 0; i < 16; ++i) raw[i] <<= 16;
  }
}
// Adds the residual to a chunk and stores it. z: the sums of row `lane`.
__device__ __forceinline__ void ln_store_turned(const LnEpilogue& e, const LnChunk& c, float (&z)[16],
                                                const uint32_t (&raw)[16], float* turn, int lane) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) turn[lane * 17 + i] = z[i];
  __syncwarp();
  const int col = lane & 15, r0 = lane >> 4;
  if (col >= c.cols) return;
  // All loads before the first store: the compiler cannot know that they do not meet.
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = turn[(2 * i + r0) * 17 + col];
  if (e.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __fadd_rn(z[i], __uint_as_float(raw[i]));
  }
  const size_t at = static_cast<size_t>(c.row + r0) * e.ldo + c.n + col;
  if (e.out_f32) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i + r0 < c.rows) static_cast<float*>(e.out)[at + 2 * i * e.ldo] = z[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (2 * i + r0 < c.rows) static_cast<__nv_bfloat16*>(e.out)[at + 2 * i * e.ldo] = __float2bfloat16_rn(z[i]);
  }
}

// ---------------------------------------------------------------- one token
constexpr int kLnRows = 2;      // weight rows a warp
constexpr int kLnRowWarps = 8;  // warps a CTA

struct LnRowsArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  long long ldx, ldw;
  int K;
  int share;  // warps that share a weight row's K range: 1, 2, 4 or 8
  LnEpilogue e;
};

__device__ __forceinline__ void ln_unpack(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
// Values 8 c .. 8 c + 7 of a row, those from K up as zeros (and not read).
__device__ __forceinline__ uint4 ln_chunk(const __nv_bfloat16* row, int c, int K) {
  if (8 * c + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row) + c);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (8 * c + k < K)
      w[k / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(row[8 * c + k])) << (16 * (k & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(32 * kLnRowWarps) linear_one_kernel(const LnRowsArgs a) {
  __shared__ float part[kLnRowWarps][kLnRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = kLnRowWarps / a.share;  // of warps, kLnRows weight rows each
  const int n0 = (blockIdx.x * groups + warp / a.share) * kLnRows;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  float acc[kLnRows];
#pragma unroll
  for (int r = 0; r < kLnRows; ++r) acc[r] = 0.0f;
  if (n0 < a.e.N) {
    const int chunks = (a.K + 7) / 8;
    const __nv_bfloat16* w[kLnRows];  // (past the last row: the last again, dropped below)
#pragma unroll
    for (int r = 0; r < kLnRows; ++r) w[r] = a.w + min(n0 + r, a.e.N - 1) * a.ldw;
#pragma unroll 4
    for (int c = (warp % a.share) * 32 + lane; c < chunks; c += 32 * a.share) {
      float wv[kLnRows][8], xv[8];
#pragma unroll
      for (int r = 0; r < kLnRows; ++r) ln_unpack(ln_chunk(w[r], c, a.K), wv[r]);
      ln_unpack(ln_chunk(a.x, c, a.K), xv);
#pragma unroll
      for (int r = 0; r < kLnRows; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[r] = __fmaf_rn(xv[k], wv[r][k], acc[r]);
    }
#pragma unroll
    for (int r = 0; r < kLnRows; ++r)
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) acc[r] = __fadd_rn(acc[r], __shfl_xor_sync(0xFFFFFFFFu, acc[r], d));
  }
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < kLnRows; ++r) part[warp][r] = acc[r];
  __syncthreads();
  if (threadIdx.x < groups * kLnRows) {
    const int r = threadIdx.x % kLnRows, g = threadIdx.x / kLnRows;
    const int n = (blockIdx.x * groups + g) * kLnRows + r;
    if (n < a.e.N) {
      float z = 0.0f;
      for (int s = 0; s < a.share; ++s) z = __fadd_rn(z, part[g * a.share + s][r]);
      ln_store(a.e, z, 0, n);
    }
  }
}

// ---------------------------------------------------------------- a few tokens
constexpr int kLnFewMax = 16;    // most tokens
constexpr int kLnFewWarps = 16;  // warps a CTA
constexpr int kLnFewSteps = 4;   // steps of 32 values that a warp loads at once

// D += A B^T, 16 tokens x 8 weight rows x 16 values of K, in registers.
__device__ __forceinline__ void ln_mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// share: warps that share a weight row's K range (1 to 16, a power of two). BOTH: more than 8 tokens.
template <bool BOTH>
__global__ void __launch_bounds__(32 * kLnFewWarps) linear_few_kernel(const LnRowsArgs a) {
  __shared__ float part[kLnFewWarps][16][8];  // [token][weight row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int groups = kLnFewWarps / a.share;  // of 8 weight rows
  const int n0 = (blockIdx.x * groups + warp / a.share) * 8;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n0 < a.e.N) {
    // A lane's fragments are 8 neighbouring values of token g (and g + 8) and weight row g: which of the instruction's K
    // slots they take is the same for both, so their order does not matter. (Past the last row: the last again, dropped
    // below.)
    const __nv_bfloat16* w = a.w + min(n0 + g, a.e.N - 1) * a.ldw;
    const __nv_bfloat16* x0 = a.x + min(g, a.e.M - 1) * a.ldx;
    const __nv_bfloat16* x1 = a.x + min(g + 8, a.e.M - 1) * a.ldx;
    const int steps = (a.K + 31) / 32;
    for (int s = warp % a.share; s < steps; s += kLnFewSteps * a.share) {
      uint4 wp[kLnFewSteps], xp[kLnFewSteps], yp[kLnFewSteps];
#pragma unroll
      for (int i = 0; i < kLnFewSteps; ++i) {
        wp[i] = xp[i] = yp[i] = make_uint4(0, 0, 0, 0);
        const int c = 4 * (s + i * a.share) + q;
        if (s + i * a.share < steps) {
          wp[i] = ln_chunk(w, c, a.K);
          xp[i] = ln_chunk(x0, c, a.K);
          if (BOTH) yp[i] = ln_chunk(x1, c, a.K);
        }
      }
      // Chains of eight instructions in the tensor core, which truncates; their sums are added with rounding.
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kLnFewSteps; ++i) {
        ln_mma_16x8(d, xp[i].x, yp[i].x, xp[i].y, yp[i].y, wp[i].x, wp[i].y);
        ln_mma_16x8(d, xp[i].z, yp[i].z, xp[i].w, yp[i].w, wp[i].z, wp[i].w);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] = __fadd_rn(sum[k], d[k]);
    }
  }
  part[warp][g][2 * q] = sum[0];
  part[warp][g][2 * q + 1] = sum[1];
  part[warp][g + 8][2 * q] = sum[2];
  part[warp][g + 8][2 * q + 1] = sum[3];
  __syncthreads();
  for (int i = threadIdx.x; i < groups * 8 * a.e.M; i += 32 * kLnFewWarps) {
    const int r = i % 8, m = i / 8 % a.e.M, grp = i / (8 * a.e.M);
    const int n = (blockIdx.x * groups + grp) * 8 + r;
    if (n >= a.e.N) continue;
    float z = 0.0f;
    for (int s = 0; s < a.share; ++s) z = __fadd_rn(z, part[grp * a.share + s][m][r]);
    ln_store(a.e, z, m, n);
  }
}

// ---------------------------------------------------------------- tiles
constexpr int kLnThreads = 384;
constexpr int kLnEpiWarps = 8;
// Registers a thread: 384 x 168 at launch, then 8 epilogue warps x 216 and 4 others x 72 (the same sum): a thread of the
// epilogue holds 128 sums.
constexpr int kLnLaunchRegs = 168, kLnEpiRegs = 216, kLnOtherRegs = 72;
static_assert(2 * kLnEpiRegs + kLnOtherRegs == 3 * kLnLaunchRegs, "register split");
constexpr int kLnMaxUnits = 160;           // units of a call that cuts K (one a CTA)
constexpr int kLnKBlock = 64;              // values of a K block: 128 bytes a row; a stage holds up to eight blocks
constexpr int kLnMaxStages = 12;
constexpr int kLnRingBytes = 196608;       // 4 stages of 128 + 256 rows
constexpr int kLnStageBytes = 65536;
constexpr int kLnChunk = 8;
constexpr int kLnGroup = 8;                // weight tiles that are walked together
constexpr int kLnCountsAt = 256;           // byte of the workspace where the counts of cut tiles begin, one a warp of a tile
constexpr int kLnCounts = kLnMaxUnits / 2 * kLnEpiWarps;  // (a tile that is cut has two units at least)
constexpr uint32_t kLnBegun = 1u << 16;    // a count: units begun, and in the lower half arrived
constexpr uint32_t kLnRefused = 1u << 31;  // in every count: products that cut K write nothing until the workspace is cleared
static_assert(kLnCountsAt + kLnCounts * 4 <= kWorkspaceWords, "counts");

struct LnTcArgs {
  CUtensorMap mapx, mapx1;  // x [M, K], box box_m rows x 64 values, `slices` (1) K blocks of them
  CUtensorMap mapw, mapw1;  // w [N, K], box tile_n rows x 64 values, likewise
  int tile_m, box_m, tile_n, tiles_m, tiles_n;
  int blocks;  // K blocks of a row
  int slices;  // K blocks a stage
  int groups;  // stages of a row
  int single;  // first stage that is loaded block by block
  int chunk;   // stages that one accumulation in tensor memory takes
  int split;   // units a tile
  int half_m;  // MMAs of 64 token rows
  int units, stages;
  uint32_t tmem_cols;  // allocated: both buffers, or the only one
  float4* partial;     // [units][rows / 32][tile_n / 4][32] of four columns
  int rows;            // rows of a partial tile: 32 a quarter
  uint32_t* err;
  uint32_t* counts;  // [tiles][warps], zero between calls
  unsigned long long timeout_ns;
  LnEpilogue e;
};

struct LnShared {
  uint64_t full[kLnMaxStages];  // a stage's operands have landed
  uint64_t done[kLnMaxStages];  // its MMAs have completed: the stage is free
  uint64_t tfull[2];            // an accumulator buffer is complete
  uint64_t tempty[2];           // and has been read
  uint64_t drain;
  uint32_t tmem;
  int abort;
  float turn[kLnEpiWarps][32 * 17];
};
constexpr size_t kLnSmemBytes = kLnRingBytes + 1024 + sizeof(LnShared);
static_assert(kLnSmemBytes <= 232448, "shared memory per CTA");
static_assert(sizeof(LnShared) >= 128 * 128, "an MMA of the last stage reads 128 rows");

// Instruction descriptor of tcgen05.mma kind::f16 with BF16 A and B, both K-major, FP32 accumulation, shape M x N.
__device__ __forceinline__ uint32_t ln_idesc(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[smem] x B[smem]^T, 16 values of K, issued by one thread.
__device__ __forceinline__ void ln_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Counts an arrival: what this warp wrote before stands for whoever counts after.
__device__ __forceinline__ uint32_t ln_arrive(uint32_t* counter) {
  uint32_t before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  return before;
}

struct LnUnit {
  int m, n, tile, g0, g1;  // tile, and the unit's stages of K
};
__device__ __forceinline__ LnUnit ln_unit(const LnTcArgs& a, int u) {
  LnUnit t;
  t.tile = u / a.split;
  const int s = u - t.tile * a.split;
  // Weight tiles in groups of kLnGroup, within a group the tiles of one row tile are neighbours: CTAs running at the same
  // time share both operands through L2.
  const int each = kLnGroup * a.tiles_m, g = t.tile / each, in = t.tile - g * each;
  const int width = min(kLnGroup, a.tiles_n - g * kLnGroup);
  t.m = in / width;
  t.n = g * kLnGroup + in - t.m * width;
  t.g0 = s * a.groups / a.split;
  t.g1 = (s + 1) * a.groups / a.split;
  return t;
}

template <bool CHUNKED>
__global__ void __launch_bounds__(kLnThreads, 1) linear_tc_kernel(const __grid_constant__ LnTcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  LnShared& S = *reinterpret_cast<LnShared*>(ring + kLnRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // A stage: its blocks' token rows, then its blocks' weight rows. The MMA reads 128 token rows whatever the box has: what it
  // finds past them (other rows, at the ring's end this CTA's variables) goes to rows that are not stored.
  const uint32_t a_block = a.box_m * 128, b_block = a.tile_n * 128;
  const uint32_t a_bytes = a.slices * a_block, stage_bytes = a_bytes + a.slices * b_block;

  if (tid == 0) {
    for (int s = 0; s < kLnMaxStages; ++s) {
      mbar_init(&S.full[s], 2);
      mbar_init(&S.done[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.tfull[b], 1);
      mbar_init(&S.tempty[b], kLnEpiWarps);
    }
    mbar_init(&S.drain, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&S.tmem, a.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&a.mapx);
    prefetch_tmap(&a.mapw);
  }
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const volatile int* abort = &S.abort;
  const int first = blockIdx.x, step = gridDim.x;
  constexpr int JOIN = CHUNKED ? 2 : 4;  // partial sums on their way at once, as the registers allow

  if (CHUNKED && warp >= kLnEpiWarps) reg_dec<kLnOtherRegs>();

  if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------ loads: one warp the tokens, the other the weights
    const bool tokens = warp == 8;
    const uint32_t block_bytes = tokens ? a_block : b_block;
    const CUtensorMap* map = tokens ? &a.mapx : &a.mapw;
    const CUtensorMap* map1 = tokens ? &a.mapx1 : &a.mapw1;
    uint32_t it = 0, s = 0, phase = 0;
    bool ok = true;
    for (int u = first; u < a.units && ok; u += step) {
      const LnUnit t = ln_unit(a, u);
      const int y = tokens ? a.tile_m * t.m : a.tile_n * t.n;
      for (int g = t.g0; g < t.g1; ++g, ++it) {
        ok = mbar_wait_spin(&S.done[s], phase ^ 1, a.timeout_ns, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint8_t* st = ring + s * stage_bytes + (tokens ? 0 : a_bytes);
        const int j = g * a.slices;
        if (elect_one()) {
          if (g >= a.single) {
            const int n = min(a.slices, a.blocks - j);
            mbar_arrive_expect_tx(&S.full[s], n * block_bytes);
            for (int k = 0; k < n; ++k) tma_load_2d(st + k * block_bytes, map1, kLnKBlock * (j + k), y, &S.full[s]);
          } else {
            mbar_arrive_expect_tx(&S.full[s], a.slices * block_bytes);
            tma_load_3d(st, map, 0, y, j, &S.full[s]);
          }
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(a.stages)) s = 0, phase ^= 1;
      }
    }
    // The last stages' arrivals have to land before the CTA leaves its shared memory: the MMAs' of a good end, the
    // copies' of a bad one (given 10 ms each, a thousand times a copy's latency: the other loads may be missing).
    if (lane == 0) {
      const uint32_t n = a.stages;
      for (uint32_t k = it > n ? it - n : 0; k < it; ++k) {
        if (ok) ok = mbar_wait_spin(&S.done[k % n], (k / n) & 1, a.timeout_ns, abort);
        if (!ok) mbar_wait_spin(&S.full[k % n], (k / n) & 1, 10000000ull, nullptr);
      }
      if (!ok) {
        atomicOr(a.err, kErrRingWait);
        S.abort = 1;
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA
    uint32_t s = 0, phase = 0, n = 0, b = 0, d = 0;  // n: buffers begun, b and d: the current one and its accumulator
    bool ok = true;
    const uint32_t idesc = ln_idesc(a.half_m ? 64 : 128, a.tile_n);
    const uint64_t desc0 = sw128_desc(smem_u32(ring));
    for (int u = first; u < a.units && ok; u += step) {
      const LnUnit t = ln_unit(a, u);
      for (int c0 = t.g0; c0 < t.g1 && ok; c0 += a.chunk) {
        const int c1 = min(t.g1, c0 + a.chunk);
        if (CHUNKED || c0 == t.g0) {
          b = n & 1;
          d = tmem + b * (a.tmem_cols / 2);
          ok = mbar_wait_spin(&S.tempty[b], ((n >> 1) & 1) ^ 1, a.timeout_ns, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          ++n;
        } else {
          d += a.tile_n;
        }
        for (int g = c0; g < c1 && ok; ++g) {
          ok = mbar_wait_spin(&S.full[s], phase, a.timeout_ns, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const int blocks = min(a.slices, a.blocks - g * a.slices);
          if (elect_one()) {
            // The start address is the descriptor's low field, in units of 16 bytes.
            uint64_t ad = desc0 + ((s * stage_bytes) >> 4), bd = ad + (a_bytes >> 4);
#pragma unroll 1
            for (int j = 0; j < blocks; ++j, ad += a_block >> 4, bd += b_block >> 4)
#pragma unroll
              for (int i = 0; i < 4; ++i) ln_mma(d, ad + 2 * i, bd + 2 * i, idesc, g > c0 || j + i != 0);
            tc_commit(&S.done[s]);
            if (g == (CHUNKED ? c1 : t.g1) - 1) tc_commit(&S.tfull[b]);
          }
          __syncwarp();
          if (++s == static_cast<uint32_t>(a.stages)) s = 0, phase ^= 1;
        }
      }
    }
    if (!ok && elect_one()) {
      atomicOr(a.err, kErrRingWait);
      S.abort = 1;
      tc_commit(&S.drain);
      if (!mbar_wait_spin(&S.drain, 0, a.timeout_ns, nullptr)) atomicOr(a.err, kErrDrain);
    }
    __syncwarp();
  } else if (warp < kLnEpiWarps) {
    // ------------------------------------------------------------ epilogue
    if (CHUNKED) reg_inc<kLnEpiRegs>();
    // A warp reads the 32 tensor-memory lanes (rows) its number allows; the two warps of a quarter share the columns.
    const int quad = warp & 3, half = warp >> 2;
    // Of 128 rows a warp's lanes hold 32; of 64 rows the first 16 of its lanes hold 16.
    const int each_quad = a.half_m ? 16 : 32;
    float* turn = S.turn[warp];
    const float* bias = a.e.bias;
    const int size = CHUNKED || a.e.out_f32 ? 4 : 2, wide = a.e.wide, act = a.e.act;
    // (The branches' likelihoods place the code of activations and of ragged chunks behind the loop, which then runs on without
    // jumps: 300 x 7168 x 2048 13.2 -> 12.7 us, 64 x 7168 x 2048 7.0 -> 6.8.)
    const bool more = bias != nullptr || act != FME_ACT_NONE;
    uint32_t n = 0;
    bool ok = true, refuse = false;
    for (int u = first; u < a.units && ok; u += step) {
      const LnUnit t = ln_unit(a, u);
      const int m0 = a.tile_m * t.m, n0 = a.tile_n * t.n;
      const int rows = min(each_quad, min(a.tile_m, a.e.M - m0) - each_quad * quad);  // of this warp
      // A warp's count of a cut tile: begun is counted here, long before the result is needed, arrived where its part is stored.
      // So at any moment no more have arrived than begun and no more begun than there are units, and a count that no call left
      // shows, if not to the unit that begins first then to one that finds too many begun. (300 x 896 x 3584 FP32 10.2 -> 10.3
      // us, 20 x 16 x 3584 4.9 -> 5.1, 64 x 256 x 7168 FP32 6.75 either way and, with a mark of its own that every warp reads,
      // one address for all, 7.1.)
      uint32_t* const count = a.counts + t.tile * kLnEpiWarps + warp;
      uint32_t begun = 0;
      if (a.split > 1 && rows > 0 && lane == 0) begun = atomicAdd(count, kLnBegun);
      uint32_t base = 0;  // this thread's row of the accumulator, from the columns of its half
      auto wait = [&]() {
        ok = mbar_wait_spin(&S.tfull[n & 1], (n >> 1) & 1, a.timeout_ns, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        base = tmem + (n & 1) * (a.tmem_cols / 2) + (static_cast<uint32_t>(32 * quad) << 16) + 16 * half;
        return ok;
      };
      auto release = [&]() {  // the MMA may write the buffer again
        __syncwarp();
        tc_fence_before();
        if (lane == 0) mbar_arrive(&S.tempty[n & 1]);
        ++n;
      };
      // This thread's column chunks: 32 i + 16 half.
      auto has = [&](int c) { return c + 16 * half < a.tile_n && n0 + c + 16 * half < a.e.N; };
      if (CHUNKED) {
        // The accumulations' sums meet in registers, 16 columns 32 i + 16 half each; the tile's go back over the last one's.
        float z[8][16];
        for (int c0 = t.g0; c0 < t.g1; c0 += a.chunk) {
          if (!wait()) break;
          if (rows > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (32 * i + 16 * half < a.tile_n) {
                float d[16];
                tmem_ld_issue(base + 32 * i, d);
                tmem_ld_join(d);
                if (c0 == t.g0) {
#pragma unroll
                  for (int k = 0; k < 16; ++k) z[i][k] = d[k];
                } else {
#pragma unroll
                  for (int k = 0; k < 16; ++k) z[i][k] = __fadd_rn(z[i][k], d[k]);
                }
                if (c0 + a.chunk >= t.g1) tmem_st16(base + 32 * i, reinterpret_cast<const uint32_t(&)[16]>(z[i]));
              }
          }
          if (c0 + a.chunk < t.g1) release();
        }
        tc_wait_st();
      } else {
        wait();
      }
      // 16 columns of the unit's sums: of one accumulator, or of all that it has.
      auto sums = [&](int c, float (&z)[16]) {
        tmem_ld_issue(base + c, z);
        tmem_ld_join(z);
        if (!CHUNKED)
#pragma unroll 1
          for (int c0 = t.g0 + a.chunk, at = base + c; c0 < t.g1; c0 += a.chunk) {
            float d[16];
            tmem_ld_issue(at += a.tile_n, d);
            tmem_ld_join(d);
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] = __fadd_rn(z[k], d[k]);
          }
      };
      if (!ok) break;
      bool mine = rows > 0;  // this warp finishes its part of the tile
      // Partial sums: of a unit a part for each quarter of the rows, of that 16 columns at a time, of those four at a time,
      // of those a row a lane.
      const size_t each = static_cast<size_t>(a.tile_n) * a.rows;
      float4* tile = a.partial + (static_cast<size_t>(t.tile) * a.split * each + (a.tile_n * quad + 16 * half) * 32) / 4 + lane;
      if (mine && a.split > 1) {
        float4* part = tile + (u - t.tile * a.split) * (each / 4);
        for (int c = 0; has(c); c += 32) {
          float z[16];
          sums(c, z);
          if (lane < rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              __stcg(part + (c / 4 + k) * 32, make_float4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]));
          }
        }
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0) {
          const uint32_t n = a.split;
          if (begun < kLnRefused) {
            before = ln_arrive(count);
            if (before == n * kLnBegun + n - 1u) atomicAnd(count, kLnRefused);
            refuse = begun / kLnBegun >= n || begun % kLnBegun > begun / kLnBegun || before / kLnBegun > n ||
                     before % kLnBegun >= before / kLnBegun;
          } else {
            atomicOr(a.err, kErrCrossWait);
            atomicSub(count, kLnBegun);
          }
        }
        mine = __shfl_sync(0xFFFFFFFFu, before, 0) == a.split * kLnBegun + a.split - 1u;
        __syncwarp();  // the other lanes' reads of the parts stand behind lane 0's acquire (a shuffle orders no memory)
      }
      auto join = [&](int c, float (&z)[16]) {
        if (a.split == 1) {
          sums(c, z);
          return;
        }
        // In K's order, JOIN units' partial sums on their way at once; lanes past the rows read the last row's.
        const float4* from = tile + (c / 4) * 32 - max(lane - (rows - 1), 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.0f;
#pragma unroll 1
        for (int s = 0; s < a.split; s += JOIN, from += JOIN * (each / 4)) {
          float4 p[JOIN][4];
#pragma unroll
          for (int b = 0; b < JOIN; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              p[b][i] = s + b < a.split ? __ldcg(from + b * (each / 4) + i * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int b = 0; b < JOIN; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              z[4 * i] = __fadd_rn(z[4 * i], p[b][i].x);
              z[4 * i + 1] = __fadd_rn(z[4 * i + 1], p[b][i].y);
              z[4 * i + 2] = __fadd_rn(z[4 * i + 2], p[b][i].z);
              z[4 * i + 3] = __fadd_rn(z[4 * i + 3], p[b][i].w);
            }
        }
      };
      if (mine) {
        const size_t row = m0 + each_quad * quad + lane, col = n0 + 16 * half;
        char* to = static_cast<char*>(a.e.out) + (row * a.e.ldo + col) * size;
        const char* from =
            a.e.residual == nullptr ? nullptr : static_cast<const char*>(a.e.residual) + (row * a.e.ldr + col) * size;
        for (int c = 0; has(c); c += 32) {
          const LnChunk k = {m0 + each_quad * quad, rows, n0 + c + 16 * half, min(16, a.e.N - n0 - c - 16 * half)};
          const bool whole = wide != 0 && k.cols == 16;
          uint32_t raw[16];
          if (from != nullptr) {
            if (__builtin_expect(!whole, 0))
              ln_load_turned(a.e, k, lane, raw);
            else if (lane < rows)
              ln_load_whole(raw, from + c * size, size, wide == 32);
          }
          float z[16];
          join(c, z);
          if (__builtin_expect(more, 0)) ln_finish16(a.e, bias, act, z, k.n);
          if (__builtin_expect(whole, 1)) {
            if (from != nullptr) ln_add_whole(z, raw, size);
            if (lane < rows) ln_store_whole(z, to + c * size, size, wide == 32);
          } else {
            ln_store_turned(a.e, k, z, raw, turn, lane);
          }
        }
      }
      release();
    }
    if (__any_sync(0xFFFFFFFFu, !ok || refuse)) {
      if (!ok) S.abort = 1;
      if (lane == 0) atomicOr(a.err, ok ? kErrCrossWait : kErrRingWait);
      // Counts that stay incomplete, or are of no call, would let a later call take a unit for the last one too early.
#pragma unroll 1
      for (int i = lane; a.split > 1 && i < kLnCounts; i += 32) atomicOr(a.counts + i, kLnRefused);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, a.tmem_cols);
}

// ---------------------------------------------------------------- host side
static PFN_cuTensorMapEncodeTiled_v12000 ln_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// BF16 tensor [rows, cols] with row stride ld, 128-byte swizzle, zeros outside. slices = 0: box box_rows x 64 values; else
// the whole 64-value blocks of its rows as a third dimension, box 64 values x box_rows x slices.
static bool ln_map(CUtensorMap* map, const void* base, int rows, int cols, long long ld, int box_rows, int slices) {
  auto fn = ln_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t n = static_cast<cuuint64_t>(rows), pitch = static_cast<cuuint64_t>(ld) * 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), n, 0};
  cuuint64_t strides[2] = {pitch, 128};
  cuuint32_t box[3] = {kLnKBlock, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(slices)};
  cuuint32_t estr[3] = {1, 1, 1};
  if (slices > 0) {
    dims[0] = kLnKBlock;
    dims[2] = static_cast<cuuint64_t>(cols / kLnKBlock);
  }
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, slices > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether a product goes to the kernels of few tokens. Measured with the weights out of L2, they against tiles (us): 8 tokens of
// 256 x 7168 4.6 / 6.3, of 7168 x 2048 8.4 / 8.9, of 4096 x 7168 13.1 / 14.6; 16 tokens of 256 x 7168 5.8 / 6.4, of 1024 x
// 4096 4.9 / 5.8, of 7168 x 1024 9.3 / 6.6, of 4096 x 7168 23 / 14.5. (Weights above 4096 x 7168 were not measured.)
static bool ln_few(int M, int N, int K) {
  return M <= 8 || (M <= kLnFewMax && static_cast<long long>(N) * K <= (1 << 22));
}

// How a product in tiles is cut: by what the ways cost, in clocks, to within 1 % on average of the best way of 42 shapes that
// were swept with their operands out of L2 (tokens 17 to 16384, 8 to 7168 outputs, K 64 to 7168); the worst are 17 x 256 x 7168
// FP32, 7.5 % off (16 columns in 9 cuts for 8), and 200 x 256 x 7168 FP32, 6.9 % (16 columns in 4 for 32 in 8). A K block costs shared
// memory's time at 128 bytes a clock: what is written, the box's token rows and the weight rows, and what an MMA reads, 128 (or
// 64) token rows and the weight rows again, each of them 128 bytes; all blocks together at least HBM's, 3500 bytes a clock.
// Cutting K costs 2500 clocks and the partial sums' way at 20 bytes a clock.
struct LnPlan {
  int tile_m, tile_n, tiles_m, tiles_n, blocks, split;
};
static LnPlan ln_plan(int M, int N, int K, int sms) {
  LnPlan p;
  p.blocks = (K + kLnKBlock - 1) / kLnKBlock;
  p.tiles_m = (M + 127) / 128;
  p.tile_m = p.tiles_m == 1 ? M : ((M + p.tiles_m - 1) / p.tiles_m + 7) / 8 * 8;
  p.tiles_m = (M + p.tile_m - 1) / p.tile_m;
  const int box_m = (p.tile_m + 7) / 8 * 8;
  const long long hbm = 2ll * K * (static_cast<long long>(M) + N) / 3500;
  long long best = -1;
  for (int tile_n = 16; tile_n <= 256 && tile_n < N + 16; tile_n += 16) {
    const int tiles_n = (N + tile_n - 1) / tile_n;
    const long long tiles = static_cast<long long>(p.tiles_m) * tiles_n;
    const long long block = box_m + (p.tile_m <= 64 ? 64 : 128) + 2 * tile_n;
    for (int split = 1; split <= 16 && split <= p.blocks && (split == 1 || tiles * split <= sms); ++split) {
      long long cost = (tiles * split + sms - 1) / sms * ((p.blocks + split - 1) / split) * block;
      if (cost < hbm) cost = hbm;
      if (split > 1) cost += 2500 + split * (4ll * p.tile_m * tile_n) / 20;
      if (best < 0 || cost < best) {
        best = cost;
        p.tile_n = tile_n;
        p.tiles_n = tiles_n;
        p.split = split;
      }
    }
  }
  return p;
}

// The plan of these sizes; the last ones' are kept, since a search is up to 256 ways (64 x 7168 x 2048
// in a stream 15.8 us, searched twice a call and with four tensor maps; 12.9 with one search kept and two maps).
static LnPlan ln_plan_kept(int M, int N, int K, int sms) {
  struct Kept {
    int M = -1, N, K, sms;
    LnPlan plan;
  };
  constexpr unsigned kKept = 64;
  thread_local Kept kept[kKept];
  const unsigned h = (static_cast<unsigned>(M) * 31u + static_cast<unsigned>(N)) * 31u + static_cast<unsigned>(K);
  Kept& k = kept[(h ^ (h >> 8)) % kKept];
  if (k.M != M || k.N != N || k.K != K || k.sms != sms) {
    k.plan = ln_plan(M, N, K, sms);
    k.M = M;
    k.N = N;
    k.K = K;
    k.sms = sms;
  }
  return k.plan;
}

// Rows of a partial tile: 32 for each of its quarters of 32 (or 16).
static int ln_partial_rows(const LnPlan& p) {
  const int quarter = p.tile_m <= 64 ? 16 : 32;
  return (p.tile_m + quarter - 1) / quarter * 32;
}

static int ln_sms(int dev) {
  const int sms = device_sm_count(dev);
  return sms < kLnMaxUnits ? sms : kLnMaxUnits;
}

// Powers of two where K is cut, so that a program's products need few sizes.
static size_t ln_plan_bytes(const LnPlan& p) {
  if (p.split == 1) return kWorkspaceWords;
  const size_t part = static_cast<size_t>(p.tile_n) * ln_partial_rows(p) * sizeof(float);  // of a unit
  const size_t need = kWorkspaceWords + part * p.tiles_m * p.tiles_n * p.split;
  size_t bytes = 65536;
  while (bytes < need) bytes *= 2;
  return bytes;
}
size_t linear_workspace_bytes(int M, int N, int K) {
  if (ln_few(M, N, K)) return kWorkspaceWords;
  int dev = 0, sms = -1;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = ln_sms(dev);
  return ln_plan_bytes(ln_plan_kept(M, N, K, sms > 0 ? sms : 152));
}

static LnEpilogue ln_epilogue(const Linear& l) {
  LnEpilogue e = {};
  e.bias = l.bias;
  e.bias16 = reinterpret_cast<uintptr_t>(l.bias) % 16 == 0;
  e.residual = l.residual;
  e.ldr = l.ldr;
  e.ldo = l.ldo;
  e.out = l.out;
  e.act = l.act;
  e.out_f32 = l.out_f32 ? 1 : 0;
  e.M = l.M;
  e.N = l.N;
  const long long size = l.out_f32 ? 4 : 2;
  const long long any = static_cast<long long>(reinterpret_cast<uintptr_t>(l.out)) | l.ldo * size |
                        (l.residual != nullptr ? static_cast<long long>(reinterpret_cast<uintptr_t>(l.residual)) | l.ldr * size : 0);
  e.wide = any % 32 == 0 ? 32 : any % 16 == 0 ? 16 : 0;
  return e;
}

static int ln_launch(const void* kernel, int grid, int threads, size_t smem, void* args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* params[1] = {args};
  const cudaError_t err = cudaLaunchKernelExC(&cfg, kernel, params);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "linear launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

static int linear_few(const Linear& l, int sms, cudaStream_t st) {
  LnRowsArgs a = {};
  a.x = static_cast<const __nv_bfloat16*>(l.x);
  a.w = static_cast<const __nv_bfloat16*>(l.w);
  a.ldx = l.ldx;
  a.ldw = l.ldw;
  a.K = l.K;
  a.e = ln_epilogue(l);
  // More warps share a row's K range while there are fewer than 16 warps an SM and each keeps one 16-byte load a lane and row
  // (one token) or one step of 32 values (a few).
  a.share = 1;
  if (l.M == 1) {
    const int pairs = (l.N + kLnRows - 1) / kLnRows;
    while (a.share < kLnRowWarps && pairs * a.share < 16 * sms && l.K >= 512 * a.share) a.share *= 2;
    const int groups = kLnRowWarps / a.share;
    return ln_launch(reinterpret_cast<const void*>(linear_one_kernel), (pairs + groups - 1) / groups, 32 * kLnRowWarps, 0,
                     &a, st);
  }
  const int rows8 = (l.N + 7) / 8;
  while (a.share < kLnFewWarps && rows8 * a.share < 16 * sms && l.K >= 64 * a.share) a.share *= 2;
  const int groups = kLnFewWarps / a.share;
  return ln_launch(reinterpret_cast<const void*>(l.M > 8 ? linear_few_kernel<true> : linear_few_kernel<false>),
                   (rows8 + groups - 1) / groups, 32 * kLnFewWarps, 0, &a, st);
}

int linear(const Linear& l, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  const bool few = ln_few(l.M, l.N, l.K);
  int dev = 0, sms = -1;
  const bool has_device = cudaGetDevice(&dev) == cudaSuccess;
  if (has_device) sms = ln_sms(dev);
  LnPlan p = {};
  if (!few) p = ln_plan_kept(l.M, l.N, l.K, sms > 0 ? sms : 152);
  const size_t need = few ? kWorkspaceWords : ln_plan_bytes(p);
  if (workspace == nullptr || workspace_bytes < need)
    return set_last_error(FME_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (l.M == 0) return FME_OK;
  if (!has_device) return set_last_error(FME_ECUDA, "cudaGetDevice failed");
  if (sms <= 0) return set_last_error(FME_ECUDA, "no SM count for device %d", dev);
  if (few) return linear_few(l, sms, st);
  LnTcArgs a = {};
  a.e = ln_epilogue(l);
  a.rows = ln_partial_rows(p);
  a.tile_m = p.tile_m;
  a.half_m = p.tile_m <= 64;
  a.box_m = (p.tile_m + 7) / 8 * 8;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.tile_n = p.tile_n;
  a.blocks = p.blocks;
  const int block = (a.box_m + a.tile_n) * 128;  // bytes of a K block
  a.slices = kLnStageBytes / block;
  if (a.slices < 4 && 8 * block <= kLnRingBytes) a.slices = 4;
  if (a.slices > 8) a.slices = 8;
  if (a.slices > p.blocks) a.slices = p.blocks;
  a.groups = (p.blocks + a.slices - 1) / a.slices;
  // A box of several blocks cannot end inside one.
  a.single = a.slices == 1 ? 0 : l.K % kLnKBlock == 0 ? a.groups : a.groups - 1;
  a.chunk = l.out_f32 ? (kLnChunk + a.slices - 1) / a.slices : a.groups;
  a.split = p.split < a.groups ? p.split : a.groups;
  a.units = p.tiles_m * p.tiles_n * a.split;
  a.stages = kLnRingBytes / (a.slices * block);
  if (a.stages > kLnMaxStages) a.stages = kLnMaxStages;
  // A unit's accumulations stay side by side in tensor memory where they fit (two buffers of them for CTAs of several units), and
  // meet in registers as they end where not.
  const int most = (a.groups + a.split - 1) / a.split, each = (most + a.chunk - 1) / a.chunk * a.tile_n;
  const int beside = a.units <= sms ? each : 2 * each;
  const bool chunked = beside > 512;
  a.tmem_cols = 32;
  while (a.tmem_cols < static_cast<uint32_t>(chunked ? 2 * a.tile_n : beside)) a.tmem_cols *= 2;
  // Maps for the stages that are loaded whole, and for those block by block, where there are any.
  const bool whole = a.single > 0, blocks = a.single < a.groups;
  if ((whole && (!ln_map(&a.mapx, l.x, l.M, l.K, l.ldx, a.box_m, a.slices) ||
                 !ln_map(&a.mapw, l.w, l.N, l.K, l.ldw, a.tile_n, a.slices))) ||
      (blocks && (!ln_map(&a.mapx1, l.x, l.M, l.K, l.ldx, a.box_m, 0) ||
                  !ln_map(&a.mapw1, l.w, l.N, l.K, l.ldw, a.tile_n, 0))))
    return set_last_error(FME_ECUDA, "cuTensorMapEncodeTiled failed or unavailable");
  if (!whole) {
    a.mapx = a.mapx1;
    a.mapw = a.mapw1;
  }
  a.err = static_cast<uint32_t*>(workspace);
  a.counts = a.err + kLnCountsAt / 4;
  a.partial = reinterpret_cast<float4*>(static_cast<uint8_t*>(workspace) + kWorkspaceWords);
  a.timeout_ns = wait_timeout_ns();
  const void* kernel = reinterpret_cast<const void*>(chunked ? linear_tc_kernel<true> : linear_tc_kernel<false>);
  if (!ensure_smem_attr(dev, kernel, kLnSmemBytes)) return FME_ECUDA;
  return ln_launch(kernel, a.units < sms ? a.units : sms, kLnThreads,
                   kLnSmemBytes, &a, st);
}

}  // namespace fme

// out = act(x W^T + bias) + residual, BF16 x [M, K] and W [N, K], FP32 sums, one rounding to the output's type.
//
// Two kernels.
//
// Up to kLnRowsMax tokens, linear_rows_kernel: a warp (or 2, 4, 8 that share its K range) holds kLnRows weight rows' sums
// for every token in registers, 16 bytes of a row a lane and load. Bound by the weights' stream, and by latency where they
// are few.
//
// Above, linear_tc_kernel: one persistent CTA per SM walks units, tiles of 128 tokens x tile_n weight rows (a multiple of
// 16 up to 256) times a share of K. Ten warps: one loads by TMA (64 values of the tile's rows a stage, 128-byte swizzle),
// one issues tcgen05.mma kind::f16, eight read the accumulators (two buffers in tensor memory, so that a tile's epilogue
// runs beside the next tile's products). Where the tiles are fewer than SMs, K is cut, too: a unit then stores its FP32
// sums to the workspace and the last of a tile's units to arrive adds them in K order, whichever it is, so the result
// does not hang on the order of arrival, and no unit waits for another.
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
  int wide;  // out (and residual) rows start at multiples of 32 bytes: whole sectors a store
  int M, N;
};

// ---------------------------------------------------------------- epilogue
// NaN stays NaN in each.
__device__ __forceinline__ float ln_act(float z, int act) {
  switch (act) {
    case FME_ACT_RELU:
      return z < 0.0f ? 0.0f : z;
    case FME_ACT_SILU:
      return silu_rn(z);
    case FME_ACT_GELU:  // z P(N(0, 1) < z); erfc keeps the tail's relative precision, which 1 + erf loses
      return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(z, -0.70710678f)));
    case FME_ACT_SIGMOID:
      return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-z)));
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

__device__ __forceinline__ void ln_st32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void ln_ld32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ uint32_t ln_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sixteen sums of one row, columns n .. n + 15 (those below N).
__device__ __forceinline__ void ln_store16(const LnEpilogue& e, float (&z)[16], int row, int n) {
  if (!e.wide || n + 16 > e.N) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < e.N) ln_store(e, z[i], row, n + i);
    return;
  }
  if (e.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __fadd_rn(z[i], __ldg(e.bias + n + i));
  }
  if (e.act != FME_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = ln_act(z[i], e.act);
  }
  const size_t r = static_cast<size_t>(row) * e.ldr + n, o = static_cast<size_t>(row) * e.ldo + n;
  uint32_t w[8];
  if (e.out_f32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (e.residual != nullptr) {
        ln_ld32(static_cast<const float*>(e.residual) + r + 8 * h, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[8 * h + i] = __fadd_rn(z[8 * h + i], __uint_as_float(w[i]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(z[8 * h + i]);
      ln_st32(static_cast<float*>(e.out) + o + 8 * h, w);
    }
  } else {
    if (e.residual != nullptr) {
      ln_ld32(static_cast<const __nv_bfloat16*>(e.residual) + r, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[2 * i] = __fadd_rn(z[2 * i], __uint_as_float(w[i] << 16));
        z[2 * i + 1] = __fadd_rn(z[2 * i + 1], __uint_as_float(w[i] & 0xFFFF0000u));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ln_bf16x2(z[2 * i], z[2 * i + 1]);
    ln_st32(static_cast<__nv_bfloat16*>(e.out) + o, w);
  }
}

// ---------------------------------------------------------------- a few tokens
constexpr int kLnRowsMax = 8;   // most tokens
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

template <int MT>
__global__ void __launch_bounds__(32 * kLnRowWarps) linear_rows_kernel(const LnRowsArgs a) {
  __shared__ float part[kLnRowWarps][kLnRows * MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = kLnRowWarps / a.share;  // of warps, kLnRows weight rows each
  const int n0 = (blockIdx.x * groups + warp / a.share) * kLnRows;
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  float acc[kLnRows][MT];
#pragma unroll
  for (int r = 0; r < kLnRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0.0f;
  if (n0 < a.e.N) {
    const int chunks = (a.K + 7) / 8;
    // (Past the last weight or token row: the last again, dropped below.)
    const __nv_bfloat16* w[kLnRows];
#pragma unroll
    for (int r = 0; r < kLnRows; ++r) w[r] = a.w + min(n0 + r, a.e.N - 1) * a.ldw;
#pragma unroll 4
    for (int c = (warp % a.share) * 32 + lane; c < chunks; c += 32 * a.share) {
      uint4 wp[kLnRows];
#pragma unroll
      for (int r = 0; r < kLnRows; ++r) wp[r] = ln_chunk(w[r], c, a.K);
      float wv[kLnRows][8];
#pragma unroll
      for (int r = 0; r < kLnRows; ++r) ln_unpack(wp[r], wv[r]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float xv[8];
        ln_unpack(ln_chunk(a.x + min(m, a.e.M - 1) * a.ldx, c, a.K), xv);
#pragma unroll
        for (int r = 0; r < kLnRows; ++r)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[r][m] = __fmaf_rn(xv[k], wv[r][k], acc[r][m]);
      }
    }
#pragma unroll
    for (int r = 0; r < kLnRows; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
          acc[r][m] = __fadd_rn(acc[r][m], __shfl_xor_sync(0xFFFFFFFFu, acc[r][m], d));
  }
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < kLnRows; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m) part[warp][r * MT + m] = acc[r][m];
  __syncthreads();
  for (int i = threadIdx.x; i < groups * kLnRows * MT; i += 32 * kLnRowWarps) {
    const int r = i % kLnRows, g = i / kLnRows % groups, m = i / (kLnRows * groups);
    const int n = (blockIdx.x * groups + g) * kLnRows + r;
    if (n >= a.e.N || m >= a.e.M) continue;
    float z = 0.0f;
    for (int s = 0; s < a.share; ++s) z = __fadd_rn(z, part[g * a.share + s][r * MT + m]);
    ln_store(a.e, z, m, n);
  }
}

// ---------------------------------------------------------------- tiles
constexpr int kLnThreads = 320;
constexpr int kLnEpiWarps = 8;
constexpr int kLnMaxUnits = 160;           // units of a call that cuts K (one a CTA)
constexpr int kLnKBlock = 64;              // values a stage: 128 bytes a row
constexpr int kLnABytes = 128 * 128;       // a stage's token rows
constexpr int kLnMaxStages = 12;
constexpr int kLnRingBytes = 196608;       // 4 stages of 128 + 256 rows, 10 of 128 + 16
constexpr int kLnHeader = 4096;            // workspace: error word, then from byte 256 the tiles' arrival counters

struct LnTcArgs {
  CUtensorMap mapx;  // x [M, K], box box_m rows x 64 values
  CUtensorMap mapw;  // w [N, K], box tile_n rows x 64 values
  int box_m, tile_n, tiles_m, tiles_n;
  int blocks;  // K blocks of a row
  int split;   // units a tile
  int units, stages;
  uint32_t tmem_cols;  // allocated: both buffers
  float* partial;      // [units][tile_n][rows]
  int rows;            // rows of a partial tile: min(M, 128)
  uint32_t* err;
  uint32_t* arrived;  // [tiles], zero between calls
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
  int last;
};
constexpr size_t kLnSmemBytes = kLnRingBytes + 1024 + sizeof(LnShared);

// Instruction descriptor of tcgen05.mma kind::f16 with BF16 A and B, both K-major, FP32 accumulation, shape 128 x N.
__device__ __forceinline__ uint32_t ln_idesc(int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (128u >> 4 << 24);
}
// D[tmem] (+)= A[smem] x B[smem]^T, 16 values of K, issued by one thread.
__device__ __forceinline__ void ln_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct LnUnit {
  int m, n, tile, kb0, kb1;
};
__device__ __forceinline__ LnUnit ln_unit(const LnTcArgs& a, int u) {
  LnUnit t;
  t.tile = u / a.split;
  const int s = u - t.tile * a.split;
  t.n = t.tile / a.tiles_m;
  t.m = t.tile - t.n * a.tiles_m;
  t.kb0 = static_cast<int>(static_cast<long long>(s) * a.blocks / a.split);
  t.kb1 = static_cast<int>(static_cast<long long>(s + 1) * a.blocks / a.split);
  return t;
}

__global__ void __launch_bounds__(kLnThreads, 1) linear_tc_kernel(const __grid_constant__ LnTcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  LnShared& S = *reinterpret_cast<LnShared*>(ring + kLnRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stage_bytes = kLnABytes + a.tile_n * 128;

  if (tid == 0) {
    for (int s = 0; s < kLnMaxStages; ++s) {
      mbar_init(&S.full[s], 1);
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
  if (warp == 1) {
    tmem_alloc(&S.tmem, a.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
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

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    uint32_t it = 0, s = 0, phase = 0;
    bool ok = true;
    const uint32_t bytes = (a.box_m + a.tile_n) * 128;
    for (int u = first; u < a.units && ok; u += step) {
      const LnUnit t = ln_unit(a, u);
      for (int j = t.kb0; j < t.kb1; ++j, ++it) {
        ok = mbar_wait_spin(&S.done[s], phase ^ 1, a.timeout_ns, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint8_t* st = ring + s * stage_bytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&S.full[s], bytes);
          tma_load_2d(st, &a.mapx, kLnKBlock * j, 128 * t.m, &S.full[s]);
          tma_load_2d(st + kLnABytes, &a.mapw, kLnKBlock * j, a.tile_n * t.n, &S.full[s]);
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(a.stages)) s = 0, phase ^= 1;
      }
    }
    // The last stages' arrivals have to land before the CTA leaves its shared memory: the MMAs' of a good end, the
    // copies' of a bad one (given 10 ms each, a thousand times a copy's latency).
    if (lane == 0) {
      const uint32_t n = a.stages;
      for (uint32_t k = it > n ? it - n : 0; k < it; ++k) {
        if (ok)
          ok = mbar_wait_spin(&S.done[k % n], (k / n) & 1, a.timeout_ns, abort);
        if (!ok) mbar_wait_spin(&S.full[k % n], (k / n) & 1, 10000000ull, nullptr);
      }
      if (!ok) {
        atomicOr(a.err, kErrRingWait);
        S.abort = 1;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    uint32_t s = 0, phase = 0, n = 0;
    bool ok = true;
    const uint32_t idesc = ln_idesc(a.tile_n);
    const uint64_t desc0 = sw128_desc(smem_u32(ring));
    for (int u = first; u < a.units && ok; u += step, ++n) {
      const LnUnit t = ln_unit(a, u);
      const uint32_t b = n & 1, d = tmem + b * (a.tmem_cols / 2);
      ok = mbar_wait_spin(&S.tempty[b], ((n >> 1) & 1) ^ 1, a.timeout_ns, abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      for (int j = t.kb0; j < t.kb1 && ok; ++j) {
        ok = mbar_wait_spin(&S.full[s], phase, a.timeout_ns, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          // The start address is the descriptor's low field, in units of 16 bytes.
          const uint64_t ad = desc0 + ((s * stage_bytes) >> 4), bd = ad + (kLnABytes >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) ln_mma(d, ad + 2 * i, bd + 2 * i, idesc, j > t.kb0 || i != 0);
          tc_commit(&S.done[s]);
          if (j == t.kb1 - 1) tc_commit(&S.tfull[b]);
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(a.stages)) s = 0, phase ^= 1;
      }
    }
    if (!ok && elect_one()) {
      atomicOr(a.err, kErrRingWait);
      S.abort = 1;
      tc_commit(&S.drain);
      if (!mbar_wait_spin(&S.drain, 0, a.timeout_ns, nullptr)) atomicOr(a.err, kErrDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // A warp reads the 32 tensor-memory lanes (rows) its number allows; the two warps of a quarter share the columns.
    const int quad = warp & 3, half = (warp - 2) >> 2, etid = tid - 64;
    const int row = 32 * quad + lane;
    uint32_t n = 0;
    bool ok = true;
    for (int u = first; u < a.units && ok; u += step, ++n) {
      const LnUnit t = ln_unit(a, u);
      const uint32_t b = n & 1;
      ok = mbar_wait_spin(&S.tfull[b], (n >> 1) & 1, a.timeout_ns, abort);
      // Uniform over the eight warps, so that none is left waiting at a barrier below.
      ok = !named_bar_or(1, 32 * kLnEpiWarps, !ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + b * (a.tmem_cols / 2) + (static_cast<uint32_t>(32 * quad) << 16);
      const int m = 128 * t.m + row, n0 = a.tile_n * t.n;
      const bool live = 128 * t.m + 32 * quad < a.e.M;  // this warp has rows
      float* part = a.partial + static_cast<size_t>(u) * a.tile_n * a.rows + row;
      if (live) {
        for (int c = 16 * half; c < a.tile_n; c += 32) {
          float z[16];
          tmem_ld_issue(base + c, z);
          tmem_ld_join(z);
          if (a.split > 1) {
            if (row < a.rows) {
#pragma unroll
              for (int i = 0; i < 16; ++i) __stcg(part + static_cast<size_t>(c + i) * a.rows, z[i]);
            }
          } else if (m < a.e.M && n0 + c < a.e.N) {
            ln_store16(a.e, z, m, n0 + c);
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      if (lane == 0) mbar_arrive(&S.tempty[b]);
      if (a.split > 1) {
        __threadfence();
        named_bar_sync(1, 32 * kLnEpiWarps);
        if (etid == 0) {
          __threadfence();
          S.last = atomicAdd(a.arrived + t.tile, 1u) == static_cast<uint32_t>(a.split) - 1u;
          __threadfence();
        }
        named_bar_sync(1, 32 * kLnEpiWarps);
        if (S.last) {
          __threadfence();
          if (etid == 0) a.arrived[t.tile] = 0u;
          const size_t each = static_cast<size_t>(a.tile_n) * a.rows;
          const float* from = a.partial + static_cast<size_t>(t.tile) * a.split * each + row;
          if (row < a.rows && m < a.e.M)
            for (int c = 16 * half; c < a.tile_n && n0 + c < a.e.N; c += 32) {
              float z[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) z[i] = 0.0f;
#pragma unroll 2
              for (int s = 0; s < a.split; ++s)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  z[i] = __fadd_rn(z[i], __ldcg(from + s * each + static_cast<size_t>(c + i) * a.rows));
              ln_store16(a.e, z, m, n0 + c);
            }
        }
      }
    }
    if (!ok && lane == 0) {
      atomicOr(a.err, kErrRingWait);
      S.abort = 1;
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, a.tmem_cols);
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

// BF16 tensor [rows, cols] with row stride ld, box box_rows x 64 values, 128-byte swizzle, zeros outside.
static bool ln_map(CUtensorMap* map, const void* base, int rows, int cols, long long ld, int box_rows) {
  auto fn = ln_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {kLnKBlock, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product of more than kLnRowsMax tokens is cut.
struct LnPlan {
  int tile_n, tiles_m, tiles_n, blocks, split, rows;
};
static LnPlan ln_plan(int M, int N, int K, int sms) {
  LnPlan p;
  p.rows = M < 128 ? M : 128;
  p.tiles_m = (M + 127) / 128;
  p.blocks = (K + kLnKBlock - 1) / kLnKBlock;
  p.tile_n = N < 256 ? (N + 15) / 16 * 16 : 256;
  p.tiles_n = (N + p.tile_n - 1) / p.tile_n;
  const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
  p.split = 1;
  if (tiles < sms) {
    p.split = sms / static_cast<int>(tiles);
    if (p.split > p.blocks) p.split = p.blocks;
  }
  return p;
}

static int ln_sms(int dev) {
  const int sms = device_sm_count(dev);
  return sms < kLnMaxUnits ? sms : kLnMaxUnits;
}

// Powers of two where K is cut, so that a program's products need few sizes.
size_t linear_workspace_bytes(int M, int N, int K) {
  if (M <= kLnRowsMax) return kLnHeader;
  int dev = 0, sms = -1;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = ln_sms(dev);
  const LnPlan p = ln_plan(M, N, K, sms > 0 ? sms : 152);
  if (p.split == 1) return kLnHeader;
  const size_t need =
      kLnHeader + static_cast<size_t>(p.tiles_m) * p.tiles_n * p.split * p.tile_n * p.rows * sizeof(float);
  size_t bytes = 65536;
  while (bytes < need) bytes *= 2;
  return bytes;
}

static LnEpilogue ln_epilogue(const Linear& l) {
  LnEpilogue e = {};
  e.bias = l.bias;
  e.residual = l.residual;
  e.ldr = l.ldr;
  e.ldo = l.ldo;
  e.out = l.out;
  e.act = l.act;
  e.out_f32 = l.out_f32 ? 1 : 0;
  e.M = l.M;
  e.N = l.N;
  const long long size = l.out_f32 ? 4 : 2;
  e.wide = reinterpret_cast<uintptr_t>(l.out) % 32 == 0 && l.ldo * size % 32 == 0 &&
           (l.residual == nullptr || (reinterpret_cast<uintptr_t>(l.residual) % 32 == 0 && l.ldr * size % 32 == 0));
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

static int linear_rows(const Linear& l, int sms, cudaStream_t st) {
  LnRowsArgs a = {};
  a.x = static_cast<const __nv_bfloat16*>(l.x);
  a.w = static_cast<const __nv_bfloat16*>(l.w);
  a.ldx = l.ldx;
  a.ldw = l.ldw;
  a.K = l.K;
  a.e = ln_epilogue(l);
  // More warps a row while there are fewer than 16 an SM and each keeps 32 chunks.
  const int pairs = (l.N + kLnRows - 1) / kLnRows;
  a.share = 1;
  while (a.share < kLnRowWarps && pairs * a.share < 16 * sms && l.K >= 512 * a.share) a.share *= 2;
  const int groups = kLnRowWarps / a.share;
  void (*kernel)(LnRowsArgs) = l.M == 1   ? linear_rows_kernel<1>
                               : l.M == 2 ? linear_rows_kernel<2>
                               : l.M <= 4 ? linear_rows_kernel<4>
                                          : linear_rows_kernel<8>;
  return ln_launch(reinterpret_cast<const void*>(kernel), (pairs + groups - 1) / groups, 32 * kLnRowWarps, 0, &a, st);
}

int linear(const Linear& l, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  const size_t need = linear_workspace_bytes(l.M, l.N, l.K);
  if (workspace == nullptr || workspace_bytes < need)
    return set_last_error(FME_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (l.M == 0) return FME_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return set_last_error(FME_ECUDA, "cudaGetDevice failed");
  const int sms = ln_sms(dev);
  if (sms <= 0) return set_last_error(FME_ECUDA, "no SM count for device %d", dev);
  if (l.M <= kLnRowsMax) return linear_rows(l, sms, st);
  const LnPlan p = ln_plan(l.M, l.N, l.K, sms);
  LnTcArgs a = {};
  a.e = ln_epilogue(l);
  a.rows = p.rows;
  a.box_m = (p.rows + 7) / 8 * 8;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.tile_n = p.tile_n;
  a.blocks = p.blocks;
  a.split = p.split;
  a.units = p.tiles_m * p.tiles_n * p.split;
  const int stage = kLnABytes + a.tile_n * 128;
  a.stages = kLnRingBytes / stage < kLnMaxStages ? kLnRingBytes / stage : kLnMaxStages;
  a.tmem_cols = 32;
  while (a.tmem_cols < 2u * a.tile_n) a.tmem_cols *= 2;
  if (!ln_map(&a.mapx, l.x, l.M, l.K, l.ldx, a.box_m) || !ln_map(&a.mapw, l.w, l.N, l.K, l.ldw, a.tile_n))
    return set_last_error(FME_ECUDA, "cuTensorMapEncodeTiled failed or unavailable");
  a.err = static_cast<uint32_t*>(workspace);
  a.arrived = a.err + 64;
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kLnHeader);
  a.timeout_ns = wait_timeout_ns();
  if (!ensure_smem_attr(dev, reinterpret_cast<const void*>(linear_tc_kernel), kLnSmemBytes)) return FME_ECUDA;
  return ln_launch(reinterpret_cast<const void*>(linear_tc_kernel), a.units < sms ? a.units : sms, kLnThreads,
                   kLnSmemBytes, &a, st);
}

}  // namespace fme

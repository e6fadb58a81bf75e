// Matrix products grouped by expert, E4M3 x E4M3 with FP32 block scales, for
// any number of tokens: the prompt-side counterpart of the routed decode
// kernel, on the same resident weights.
//
// Group e holds rows p in [offsets[e], offsets[e + 1]). Per row and weight row n
//   y[p, n] = sum_b (sum_{k in block b} W[e, n, k] a[r, k]) * (sw[e, n/128, b] * sa[r, b]),
// r = in_rows[p]. Two epilogues:
//   gemm    out[out_rows[p], n] = bf16(y[p, n]);
//   swiglu  h = silu(min(gate, limit)) * clamp(up, -limit, limit),
//           s = max(amax over 128 hidden values, 1e-10) / 448, q = e4m3(h / s).
//
// One persistent CTA per SM walks tiles of 128 rows of a group x 256 weight rows
// (swiglu: the 128 up rows and the 128 gate rows of one 128-value hidden
// block, so its quantisation block is inside the tile and one thread holds
// both halves of a value). Twelve warps: 0-7 accumulate, 8 loads by TMA, 9 issues
// the MMA, 10-11 copy activation rows by index.
// * Loads: per 128-value K block two 128-row boxes of weights by TMA, and the tile's
//   rows: a full tile of consecutive rows as one box, others row by row with cp.async
//   (only the rows the group has; two warps, whose pace tells: predicates on a full tile cost 3 %). TMA's own row gather
//   (tile::gather4) measured 90 clocks for four rows, 2900 a tile and K block against 512 of MMA work.
// * The scales are FP32 and not powers of two, so the MMA cannot apply them: each
//   K block is one 128 x 256 accumulation in tensor memory (two buffers), and the
//   accumulate warps add D * (sw * sa) into 128 registers a thread. A row is a
//   tensor-memory lane, so sa is one scalar a thread and sw one or two a tile.
// * Why 128 x 256: the largest tile whose FP32 sums fit the registers of eight warps, and the fewest bytes loaded for
//   the work. 128-column MMAs read the activation rows twice from shared memory (238 us where this takes 216).
//
// What bounds it: with few rows a group, DRAM (gate/up of the DeepSeek-V3 shape: 8 experts, one row each, 44 us,
// 5.3 TB/s; 226 experts, 7 rows each, 945-975 us, 6.8-7.0 TB/s, the copy rate). With many, the accumulate warps, about 735
// clocks of waits, tensor-memory loads and multiply-adds a K block alone and 950 beside the loads, against 512 of MMA (16
// experts x 512 rows: gate/up 208 us, 2310 TFLOP/s; down 119 us, 2025 TFLOP/s), tiles that a group does not fill (256
// experts x 512 rows on average hold 1.12 times their rows: gate/up 1920 TFLOP/s of rows; 256 on average 1.25: down 1390),
// and under sustained load the power limit (the 16 experts again and again: 225 and 128 us).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "fme_common.cuh"
#include "fme_internal.h"

namespace fme {

constexpr int kGrThreads = 384;
constexpr int kGrAccWarps = 8;
constexpr int kGrGatherThreads = 64;
// Registers a thread: 384 x 168 at launch, then 8 accumulate warps x 216 and 4 others x 72 (the same sum): without the
// split the accumulators spill (16 experts x 512 rows: gate/up 218 -> 228 us, down 123 -> 138 us).
constexpr int kGrLaunchRegs = 168, kGrAccRegs = 216, kGrOtherRegs = 72;
static_assert(2 * kGrAccRegs + kGrOtherRegs == 3 * kGrLaunchRegs, "register split");
// Scales travel in groups of up to four K blocks of a tile. The producer fills a group's slot once the MMA of the K block
// four before its first is done, which waited for the accumulate warps to leave the K block two before that: the
// groups still read are at most five back.
constexpr int kGrSlots = 6;
constexpr int kGrABytes = 128 * 128;    // 128 activation rows of a K block
constexpr int kGrBoxBytes = 128 * 128;  // 128 weight rows
constexpr int kGrStages = 4;
constexpr int kGrStageBytes = kGrABytes + 2 * kGrBoxBytes;

struct GrArgs {
  CUtensorMap mapa;  // a as [a_rows, K bytes], box 128 rows x 128 bytes (full tiles of consecutive rows)
  CUtensorMap mapw;  // weights as [E * N, K bytes], box 128 rows x 128 bytes
  const uint8_t* a;
  const float* sa;
  const float* sw;
  const int32_t* offsets;
  const int32_t* in_rows;   // null: row p
  const int32_t* out_rows;  // null: row p
  int a_rows, R, out_n, K, N, E;
  int up0, gate0;  // first up / gate weight row (swiglu)
  int tile_n;      // weight rows a tile: 256, or 128 (gemm)
  uint32_t most;   // tiles that ascending offsets make at most
  float limit;
  int ue8m0;
  int wide;  // out is 32-byte aligned: whole sectors a store
  uint8_t* q;
  float* sq;
  __nv_bfloat16* out;
  uint32_t* err;
  unsigned long long timeout_ns;
};

struct GrShared {
  float4 sx[kGrSlots][128];  // activation scales of the rows, four K blocks
  float4 sw[kGrSlots][2];    // weight scales of the two 128-row boxes
  uint64_t full[kGrStages];  // a stage's operands have landed
  uint64_t done[kGrStages];  // its MMAs have completed: the stage is free and the accumulator complete
  uint64_t tempty[2];        // an accumulator buffer has been read
  uint64_t sfull[kGrSlots];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  uint32_t warp_sum[kGrThreads / 32];
  int off[kMaxExperts + 1];     // group starts, clamped to [0, R] and ascending
  int tiles[kMaxExperts + 1];   // tiles before group e
  float amax[2][2][128];        // [tile parity][column half][row]
};

constexpr size_t kGrSmemBytes = static_cast<size_t>(kGrStages) * kGrStageBytes + 1024 + sizeof(GrShared);
static_assert(kGrSmemBytes <= 232448, "shared memory per CTA");

struct GrTile {
  int e, n, p0, rows;  // expert, weight tile, first row and row count
};

// Tile t: groups in order, within a group the row tiles of one weight tile are
// neighbours, so CTAs running at the same time share the weights through L2. `from`:
// a group not after t's, where the search starts (the last tile's group).
__device__ __forceinline__ GrTile gr_tile(const GrShared& S, int E, int t, int from) {
  int lo = from, hi = E;  // tiles[lo] <= t < tiles[hi]
  // Usually a step or two on; else halving what is left.
  for (int i = 0; i < 3 && hi - lo > 1; ++i) {
    if (S.tiles[lo + 1] <= t)
      ++lo;
    else
      hi = lo + 1;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (S.tiles[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int mt = (S.off[lo + 1] - S.off[lo] + 127) / 128;
  const int local = t - S.tiles[lo];
  GrTile g;
  g.e = lo;
  g.n = local / mt;
  g.p0 = S.off[lo] + 128 * (local - g.n * mt);
  g.rows = min(128, S.off[lo + 1] - g.p0);
  return g;
}

// Row of a that place i of the tile reads (past its end: its last row's; a bad index: row 0, the result is dropped).
__device__ __forceinline__ int gr_row(const GrArgs& a, const GrTile& g, int i) {
  const int p = g.p0 + min(i, g.rows - 1);
  const int r = a.in_rows != nullptr ? __ldg(a.in_rows + p) : p;
  return r >= 0 && r < a.a_rows ? r : 0;
}

// (lo, hi) rounded to BF16, lo in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kGrThreads, 1) grouped_fp8_kernel(const __grid_constant__ GrArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  GrShared& S = *reinterpret_cast<GrShared*>(ring + kGrStages * kGrStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int KB = a.K / 128;
  const int n_tiles = SWIGLU ? a.N / 256 : (a.N + a.tile_n - 1) / a.tile_n;

  if (tid == 0) {
    for (int s = 0; s < kGrStages; ++s) {
      mbar_init(&S.full[s], 1 + kGrGatherThreads);
      mbar_init(&S.done[s], 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(&S.tempty[b], kGrAccWarps);
    for (int s = 0; s < kGrSlots; ++s) mbar_init(&S.sfull[s], 32);
    mbar_init(&S.drain, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&S.tmem, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&a.mapa);
    prefetch_tmap(&a.mapw);
  }
  griddep_launch_dependents();  // the next kernel's start may overlap this one's end; it waits before it reads
  griddep_wait();
  // Tiles before each group: every thread a few groups, then a block scan. A group has 2^25 tiles at most and a warp 96
  // groups, so a warp's sum fits 32 bits; the warps' sums are cut at one more than ascending offsets can make.
  constexpr int kPer = (kMaxExperts + kGrThreads - 1) / kGrThreads;
  const int first = blockIdx.x, step = gridDim.x;
  uint32_t own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    own[i] = 0;
    if (e < a.E) {
      const int lo = max(0, min(a.R, __ldg(a.offsets + e)));
      const int hi = max(lo, min(a.R, __ldg(a.offsets + e + 1)));
      S.off[e] = lo;
      own[i] = (hi - lo + 127) / 128 * n_tiles;
      if (e == a.E - 1) S.off[a.E] = hi;
    }
    sum += own[i];
  }
  uint32_t scan = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 31) S.warp_sum[warp] = min(scan, a.most + 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t before = scan - sum;
  for (int w = 0; w < warp; ++w) before += S.warp_sum[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e <= a.E) S.tiles[e] = static_cast<int>(before);
    before += own[i];
  }
  __syncthreads();
  int total = S.tiles[a.E];
  if (static_cast<uint32_t>(total) > a.most) {  // the offsets overlap: nothing is computed
    total = 0;
    if (blockIdx.x == 0 && tid == 0) atomicOr(a.err, kErrRoute);
  }
  const uint32_t tmem = S.tmem;
  const volatile int* abort = &S.abort;
  if (warp >= kGrAccWarps) reg_dec<kGrOtherRegs>();

  if (warp == 8) {
    // ------------------------------------------------------------ loads
    uint32_t it = 0, group = 0;
    int from = 0;
    const bool vec = KB % 4 == 0;  // rows of scales are whole 16-byte units
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const GrTile g = gr_tile(S, a.E, t, from);
      from = g.e;
      const bool box = a.in_rows == nullptr && g.rows == 128;
      const float* sa[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sa[i] = a.sa + static_cast<size_t>(gr_row(a, g, 4 * lane + i)) * KB;
      // Lane i < 2: the scales of weight box i.
      const int wb =
          SWIGLU ? (lane == 0 ? a.up0 : a.gate0) / 128 + g.n : min(g.n * (a.tile_n / 128) + lane, a.N / 128 - 1);
      const float* sw = a.sw + (static_cast<size_t>(g.e) * (a.N / 128) + wb) * KB;
      const int row0 = SWIGLU ? a.up0 + 128 * g.n : a.tile_n * g.n, row1 = SWIGLU ? a.gate0 + 128 * g.n : row0 + 128;
      const bool two = SWIGLU || (a.tile_n == 256 && row1 < a.N);  // the last tile may have one box only
      const uint32_t bytes = (box ? kGrABytes : 0) + (two ? 2 : 1) * kGrBoxBytes;
      for (int j = 0; j < KB; ++j, ++it) {
        const uint32_t s = it % kGrStages;
        ok = mbar_wait_spin(&S.done[s], ((it / kGrStages) & 1) ^ 1, a.timeout_ns, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint8_t* st = ring + s * kGrStageBytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&S.full[s], bytes);
          tma_load_2d(st + kGrABytes, &a.mapw, 128 * j, g.e * a.N + row0, &S.full[s]);
          if (two) tma_load_2d(st + kGrABytes + kGrBoxBytes, &a.mapw, 128 * j, g.e * a.N + row1, &S.full[s]);
          if (box) tma_load_2d(st, &a.mapa, 128 * j, g.p0, &S.full[s]);
        }
        __syncwarp();
        if ((j & 3) == 0) {
          const uint32_t slot = group++ % kGrSlots;
          if (vec) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async_l1_16(&S.sx[slot][4 * lane + i], sa[i] + j);
            if (lane < 2) cp_async_l1_16(&S.sw[slot][lane], sw + j);
          } else {
            for (int k = 0; k < 4 && j + k < KB; ++k) {
#pragma unroll
              for (int i = 0; i < 4; ++i) cp_async_l1_4(&S.sx[slot][4 * lane + i].x + k, sa[i] + j + k);
              if (lane < 2) cp_async_l1_4(&S.sw[slot][lane].x + k, sw + j + k);
            }
          }
          cp_async_arrive(&S.sfull[slot]);
        }
      }
    }
    if (!ok) {
      // Copies in flight must land before the CTA leaves its shared memory. A stage's barrier may never complete (the
      // gather warps have left, too), so each is given 10 ms, a thousand times a copy's latency.
      cp_async_wait_all();
      if (lane == 0) {
        atomicOr(a.err, kErrRingWait);
        S.abort = 1;
        for (uint32_t k = it > kGrStages ? it - kGrStages : 0; k < it; ++k)
          mbar_wait_spin(&S.full[k % kGrStages], (k / kGrStages) & 1, 10000000ull, nullptr);
      }
      __syncwarp();
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA
    uint32_t it = 0;
    bool ok = true;
    const uint64_t desc0 = sw128_desc(smem_u32(ring));
    const uint32_t idesc = SWIGLU || a.tile_n == 256 ? f8_idesc(128, 256) : f8_idesc(128, 128);
    for (int t = first; t < total && ok; t += step) {
      for (int j = 0; j < KB; ++j, ++it) {
        const uint32_t s = it % kGrStages, b = it & 1;
        ok = mbar_wait_spin2(&S.full[s], (it / kGrStages) & 1, &S.tempty[b], ((it >> 1) & 1) ^ 1, a.timeout_ns, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        // The gather's copies, complete by their arrivals on the stage's barrier, before the MMA's reads. (A fence in the
        // gather warps would hold each K block's copies up for the last one's: gate/up 217 us instead of 211.)
        fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          // The start address is the descriptor's low field, in units of 16 bytes.
          const uint64_t ad = desc0 + s * (kGrStageBytes >> 4), bd = ad + (kGrABytes >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) tc_mma_f8(tmem + 256 * b, ad + 2 * i, bd + 2 * i, idesc, i != 0);
          tc_commit(&S.done[s]);
        }
        __syncwarp();
      }
    }
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok && elect_one()) {
      atomicOr(a.err, kErrRingWait);
      S.abort = 1;
      tc_commit(&S.drain);
      if (!mbar_wait_spin(&S.drain, 0, a.timeout_ns, nullptr)) atomicOr(a.err, kErrDrain);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------------------------ activation rows by index
    // Eight threads copy a row's 128 bytes, swizzled as the MMA's descriptor says.
    const int gt = tid - 320, chunk = gt & 7, r0 = gt >> 3;
    const uint32_t dst0 = r0 * 128 + ((chunk ^ (r0 & 7)) << 4);
    uint32_t it = 0;
    int from = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const GrTile g = gr_tile(S, a.E, t, from);
      from = g.e;
      const bool box = a.in_rows == nullptr && g.rows == 128;
      int row[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) row[i] = gr_row(a, g, r0 + 8 * i);
      const int n = box ? 0 : (g.rows - r0 + 7) / 8;  // rows this thread copies
      const uint8_t* src = a.a + 16 * chunk;
      for (int j = 0; j < KB;) {
        // Two K blocks a turn: one wait and one address for both.
        const bool two = j + 1 < KB;
        const uint32_t s0 = it % kGrStages, s1 = (it + 1) % kGrStages, last = it + (two ? 1 : 0);
        ok = mbar_wait_spin(&S.done[last % kGrStages], ((last / kGrStages) & 1) ^ 1, a.timeout_ns, abort);
        if (!ok) break;
        uint8_t* st0 = ring + s0 * kGrStageBytes + dst0;
        uint8_t* st1 = ring + s1 * kGrStageBytes + dst0;
        if (two) {
          if (n == 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint8_t* p = src + static_cast<size_t>(row[i]) * a.K;
              cp_async_16(st0 + 1024 * i, p);
              cp_async_16(st1 + 1024 * i, p + 128);
            }
            cp_async_arrive(&S.full[s0]);
            cp_async_arrive(&S.full[s1]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < n) {
                const uint8_t* p = src + static_cast<size_t>(row[i]) * a.K;
                cp_async_16(st0 + 1024 * i, p);
                cp_async_16(st1 + 1024 * i, p + 128);
              }
            cp_async_arrive(&S.full[s0]);
            cp_async_arrive(&S.full[s1]);
          }
          j += 2, it += 2, src += 256;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (i < n) cp_async_16(st0 + 1024 * i, src + static_cast<size_t>(row[i]) * a.K);
          cp_async_arrive(&S.full[s0]);
          ++j, ++it, src += 128;
        }
      }
    }
    if (!ok) {
      atomicOr(a.err, kErrRingWait);
      S.abort = 1;
      cp_async_wait_all();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ accumulate and epilogue
    reg_inc<kGrAccRegs>();
    const int half = warp >> 2, quad = warp & 3;
    const int row = 32 * quad + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    // The MMA may write buffer b again.
    auto release = [&](uint32_t b) {
      tc_fence_before();
      if (lane == 0) mbar_arrive(&S.tempty[b]);
    };
    uint32_t it = 0, group = 0, slot = 0;
    int parity = 0, from = 0;
    bool ok = true;
    for (int t = first; t < total; t += step, parity ^= 1) {
      const GrTile g = gr_tile(S, a.E, t, from);
      from = g.e;
      const bool columns = SWIGLU || (128 * half < a.tile_n && a.tile_n * g.n + 128 * half < a.N);
      const bool live = 32 * quad < g.rows && columns;  // this warp has rows (and columns) to hold
      const int p = g.p0 + min(row, g.rows - 1);
      const int r = a.in_rows != nullptr ? __ldg(a.in_rows + p) : p;
      const bool bad = r < 0 || r >= a.a_rows;
      const int o = SWIGLU || a.out_rows == nullptr ? p : __ldg(a.out_rows + p);
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.0f;
      for (int j = 0; j < KB; ++j, ++it) {
        const uint32_t b = it & 1;
        if ((j & 3) == 0) {
          slot = group % kGrSlots;
          ok = ok && mbar_wait_spin(&S.sfull[slot], (group++ / kGrSlots) & 1, a.timeout_ns, abort);
        }
        const float sx = (&S.sx[slot][row].x)[j & 3];
        const float s0 = __fmul_rn((&S.sw[slot][SWIGLU ? 0 : half].x)[j & 3], sx);
        const float s1 = SWIGLU ? __fmul_rn((&S.sw[slot][1].x)[j & 3], sx) : s0;
        // One vote over the first try (20 us at most); the bounded wait and its vote only behind a failed one (gate/up
        // 203.8 us instead of 205.7, down alike).
        if (!__all_sync(0xFFFFFFFFu, ok && mbar_try_wait_for(&S.done[it % kGrStages], (it / kGrStages) & 1, 20000))) {
          ok = ok && mbar_wait_spin(&S.done[it % kGrStages], (it / kGrStages) & 1, a.timeout_ns, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
        }
        if (live) {
          tc_fence_after();
          const uint32_t base = lanes + 256 * b + (SWIGLU ? 64 : 128) * half;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float d[16];
            tmem_ld_issue(base + (SWIGLU && c >= 4 ? 64 : 0) + 16 * c, d);
            tmem_ld_join(d);
            if (c == 7) release(b);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[16 * c + i] = __fmaf_rn(d[i], c < 4 ? s0 : s1, acc[16 * c + i]);
          }
        } else {
          __syncwarp();
          release(b);
        }
      }
      if (bad) {
        if (row < g.rows && half == 0) atomicOr(a.err, kErrRoute);
#pragma unroll
        for (int c = 0; c < 128; ++c) acc[c] = 0.0f;
      }
      if (SWIGLU) {
        // acc[0..63] up, acc[64..127] gate of hidden values 64 * half .. + 63.
        float amax = 0.0f;
        if (live) {
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            const float up = min_nan(max_nan(acc[c], -a.limit), a.limit);
            const float gate = min_nan(acc[64 + c], a.limit);
            acc[c] = __fmul_rn(silu_rn(gate), up);
            amax = fmaxf(amax, fabsf(acc[c]));
          }
        }
        S.amax[parity][half][row] = amax;
        // Uniform over the eight warps, so none is left waiting at the next tile's barrier.
        if (named_bar_or(1, 32 * kGrAccWarps, !ok)) {
          ok = false;
          break;
        }
        if (row < g.rows) {
          amax = fmaxf(amax, S.amax[parity][half ^ 1][row]);
          float s = __fdiv_rn(fmaxf(amax, 1e-10f), 448.0f);
          if (a.ue8m0) s = ue8m0_ceil(s);
          const float inv = __fdiv_rn(1.0f, s);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = quotient_rn(acc[4 * i + k], s, inv);
            w[i] = f32x2_to_e4m3x2(v[0], v[1]) | (f32x2_to_e4m3x2(v[2], v[3]) << 16);
          }
          const int I = a.N / 2;
          uint4* dst = reinterpret_cast<uint4*>(a.q + static_cast<size_t>(p) * I + 128 * g.n + 64 * half);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if (half == 0) a.sq[static_cast<size_t>(p) * (I / 128) + g.n] = s;
        }
      } else {
        if (!ok) break;
        if (row < g.rows && columns) {
          if (o < 0 || o >= a.out_n) {
            atomicOr(a.err, kErrRoute);
          } else {
            __nv_bfloat16* dst = a.out + static_cast<size_t>(o) * a.N + a.tile_n * g.n + 128 * half;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = bf16x2(acc[16 * i + 2 * k], acc[16 * i + 2 * k + 1]);
              if (a.wide) {
                st_global_32(dst + 16 * i, w);
              } else {
                reinterpret_cast<uint4*>(dst)[2 * i] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst)[2 * i + 1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
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
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side
static PFN_cuTensorMapEncodeTiled_v12000 gr_encode_fn() {
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

// Byte tensor [rows, cols], box box_rows x 128 bytes, 128-byte swizzle.
static bool gr_map(CUtensorMap* map, const void* base, unsigned long long rows, unsigned long long cols,
                   unsigned box_rows) {
  auto fn = gr_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t grouped_fp8_workspace_bytes() { return 256; }

int grouped_fp8(const GroupedFp8& g, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  if (workspace == nullptr || workspace_bytes < grouped_fp8_workspace_bytes())
    return set_last_error(FME_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes,
                          grouped_fp8_workspace_bytes());
  if (g.R == 0) return FME_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return set_last_error(FME_ECUDA, "cudaGetDevice failed");
  const int sms = device_sm_count(dev);
  if (sms <= 0) return set_last_error(FME_ECUDA, "no SM count for device %d", dev);
  GrArgs a = {};
  if (!gr_map(&a.mapa, g.a, g.a_rows, g.K, 128) ||
      !gr_map(&a.mapw, g.w, static_cast<unsigned long long>(g.E) * g.N, g.K, 128))
    return set_last_error(FME_ECUDA, "cuTensorMapEncodeTiled failed or unavailable");
  a.a = g.a;
  a.sa = g.sa;
  a.sw = g.sw;
  a.offsets = g.offsets;
  a.in_rows = g.in_rows;
  a.out_rows = g.out_rows;
  a.a_rows = g.a_rows;
  a.R = g.R;
  a.out_n = g.out_n;
  a.K = g.K;
  a.N = g.N;
  a.E = g.E;
  a.up0 = g.gate_first ? g.N / 2 : 0;
  a.gate0 = g.gate_first ? 0 : g.N / 2;
  a.limit = g.limit;
  a.ue8m0 = g.ue8m0 ? 1 : 0;
  a.q = g.q;
  a.sq = g.sq;
  a.out = static_cast<__nv_bfloat16*>(g.out);
  a.wide = (reinterpret_cast<uintptr_t>(g.out) & 31u) == 0;
  a.err = static_cast<uint32_t*>(workspace);
  a.timeout_ns = wait_timeout_ns();
  const bool swiglu = g.q != nullptr;
  // At most so many row tiles (a group's last may be part empty).
  const long long row_tiles = static_cast<long long>(g.R) / 128 + (g.R < g.E ? g.R : g.E);
  auto tiles = [&](int tile_n) { return row_tiles * ((g.N + tile_n - 1) / tile_n); };
  // Half as wide gemm tiles where they all run at once: a tile's time is what counts then (8 experts of 512 x 256, 512
  // tokens 5.3 us instead of 6.2; 40 of 1024 x 384, one token 4.8 instead of 5.2). Otherwise wide ones, which read the
  // activations once for twice the columns (256 of 7168 x 2048, 2 tokens 38.8 us instead of 44.6).
  a.tile_n = !swiglu && tiles(128) <= sms ? 128 : 256;
  const long long most = tiles(a.tile_n);
  a.most = static_cast<uint32_t>(most);  // (2^18 + 2^10) row tiles of 128 weight tiles, or fewer
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < sms ? most : sms));
  cfg.blockDim = dim3(kGrThreads);
  cfg.dynamicSmemBytes = kGrSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*kernel)(GrArgs) = swiglu ? grouped_fp8_kernel<true> : grouped_fp8_kernel<false>;
  if (!ensure_smem_attr(dev, reinterpret_cast<const void*>(kernel), kGrSmemBytes)) return FME_ECUDA;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err != cudaSuccess) return set_last_error(FME_ECUDA, "grouped fp8 launch: %s", cudaGetErrorString(err));
  return FME_OK;
}

}  // namespace fme

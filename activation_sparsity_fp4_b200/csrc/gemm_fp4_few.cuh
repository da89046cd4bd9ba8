// gemm_fp4_few.cuh -- the plain FP4 product for few activation rows (decode).
//
//   y[t][n] = r_x[t] r_w[n] sum_j (E2M1 x S)(t, j) (E2M1 x S)(n, j)
//
// With few rows the product is a stream of the weight, so the weight is the
// 128-row operand A and the rows, padded to TN = 32, 64 or 128, are operand B:
// D[n][t].  The K loop of a 128-row weight tile is cut into slices on different
// SMs, the CTAs of one cluster; each leaves its sums in its shared memory, and
// the CTAs add them up in slice order (so results repeat bit for bit), each for
// its share of the rows, through distributed shared memory.
//
// Per CTA (192 threads): warp 0 TMA producer, warp 1 MMAs, warps 2-5 the scale
// chunks into tensor memory, then the accumulator out of it.  Every wait is
// bounded in time and reports through the device error word.
//
// 1 x 14336 -> 4096 NVFP4 9.1 us (33 MB of weight, 3.6 TB/s), 16 x 4096 x 4096 6.0 us:
// bound by the launch, the first loads and the two cluster barriers.
#pragma once
#include "gemm_fp4.cuh"

namespace sharq {

constexpr int kFp4FewMaxSplit = 8;  // the portable cluster size

template <int KIND, int TN>
struct Fp4FewCfg {
  static_assert(TN == 32 || TN == 64 || TN == 128, "rows of operand B");
  static constexpr int BM = 128, BK = 256;
  static constexpr int kVec = KIND == GK_NVF4 ? 16 : 32, kChunks = BK / kVec / 4;
  static constexpr int oW = 0, oX = BM * 128, oSfw = oX + TN * 128, oSfx = oSfw + kChunks * 512;
  static constexpr int kStageBytes = ((oSfx + kChunks * 512 + 1023) / 1024) * 1024;
  static constexpr int kStages = TN == 128 ? 6 : 8;
  static constexpr int kSlotCols = 8 * kChunks;  // weight scales, then activation scales
  static constexpr int kTmemCols = 512;
  static_assert(TN + kStages * kSlotCols <= kTmemCols, "tensor memory budget");
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(TN * BM * 4 <= kStages * kStageBytes, "the slice's sums take the stages' place");
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(TN >> 3) << 17) |
                                     ((KIND == GK_NVF4 ? 0u : 1u) << 23) | ((uint32_t)(BM >> 4) << 24);
};

struct Fp4FewMaps {
  CUtensorMap w, x;
};

struct Fp4FewParams {
  int64_t t, n, k;
  int32_t split;  // K slices of a weight tile = CTAs of a cluster
  const uint8_t* sf_w;
  const uint8_t* sf_x;
  const float* row_w;
  const float* row_x;
  void* y;
  int y_bf16;
  uint64_t timeout_ns;
};

template <int KIND, int TN>
__global__ void __launch_bounds__(192, 1) gemm_fp4_few_kernel(const __grid_constant__ Fp4FewMaps maps,
                                                              const Fp4FewParams p) {
  using C = Fp4FewCfg<KIND, TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* ready = empty + C::kStages;  // the stage's scales are in tensor memory
  uint64_t* acc_full = ready + C::kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // blockIdx: (weight tile x K slice) fastest, then the tile of TN rows
  const int n_tiles = (int)((p.n + C::BM - 1) / C::BM), k_tiles = (int)((p.k + C::BK - 1) / C::BK);
  const int item = (int)(blockIdx.x / p.split), slice = (int)(blockIdx.x % p.split);
  const int64_t n0 = (int64_t)(item % n_tiles) * C::BM, t0 = (int64_t)(item / n_tiles) * TN;
  const int k0 = (int)((int64_t)slice * k_tiles / p.split), k1 = (int)((int64_t)(slice + 1) * k_tiles / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&ready[s], 4);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch(&maps.w);
      tma_prefetch(&maps.x);
    }
    // while the kernel before this one finishes: warm L2 with this slice of the
    // weight (no data reaches the SM, so it may even be that kernel's output)
    for (int kt = k0 + lane; kt < k1; kt += 32) tma_prefetch_l2_2d(&maps.w, kt * 128, (int32_t)n0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dep_wait();
  grid_dep_launch();

  const int64_t s_blocks = (p.k / C::kVec + 3) / 4;  // 512-byte chunks per 128 rows
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t smem0 = smem_u32(smem), full0 = smem_u32(full);
      const uint8_t* g_w = p.sf_w + (n0 / 128) * s_blocks * 512;
      const uint8_t* g_x = p.sf_x + (t0 / 128) * s_blocks * 512;
      uint32_t issued = 0, issued_par = 0, stage = 0, phase = 0;
      for (int kt = k0; kt < k1 && !*abort_flag; kt++) {
        if (!mbar_wait(&empty[stage], phase ^ 1, p.timeout_ns, abort_flag)) { *abort_flag = 1; break; }
        const uint32_t sb = smem0 + stage * (uint32_t)C::kStageBytes, fb = full0 + stage * 8;
        const int64_t left = s_blocks - (int64_t)kt * C::kChunks, so = (int64_t)kt * C::kChunks * 512;
        const uint32_t bytes = (uint32_t)(left < C::kChunks ? left : C::kChunks) * 512u;
        mbar_arrive_expect_tx_u32(fb, (uint32_t)((C::BM + TN) * 128) + 2 * bytes);
        tma_load_2d_u32(sb + C::oW, &maps.w, kt * 128, (int32_t)n0, fb);
        tma_load_2d_u32(sb + C::oX, &maps.x, kt * 128, (int32_t)t0, fb);
        bulk_load_u32(sb + C::oSfw, g_w + so, bytes, fb);
        bulk_load_u32(sb + C::oSfx, g_x + so, bytes, fb);
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == C::kStages) { stage = 0; phase ^= 1; }
      }
      if (*abort_flag) {  // let every load already issued land before the block can exit
        for (int i = 0; i < C::kStages; i++)
          if ((issued >> i) & 1u) (void)mbar_wait(&full[i], (issued_par >> i) & 1u, 1000000000ull, nullptr, true);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    constexpr uint32_t kHi128 = desc_hi(1024, 2), kLbo = 1u << 16;
    const uint32_t lo0 = __shfl_sync(0xffffffffu, smem_u32(smem) >> 4, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    uint32_t stage = 0, phase = 0;
    for (int kt = k0; kt < k1; kt++) {
      if (!mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag) ||
          !mbar_wait(&ready[stage], phase, p.timeout_ns, abort_flag)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t ls = lo0 + stage * (uint32_t)(C::kStageBytes >> 4);
      const uint32_t sl = tm + TN + stage * (uint32_t)C::kSlotCols;
      const int left = (int)((p.k + 63) / 64) - kt * (C::BK / 64);  // beyond K there are no scales
      if (elect_one()) {
#pragma unroll
        for (int kb = 0; kb < C::BK / 64; kb++) {
          if (kb < left) {
            constexpr int kScales = 64 / C::kVec;
            const uint32_t chunk = (kb * kScales) / 4, byte = (kb * kScales) % 4;
            const uint32_t idesc = C::kIdesc | (byte << 29) | (byte << 4);
            const uint64_t a = desc_lohi((ls + (C::oW >> 4) + 2 * kb) | kLbo, kHi128);
            const uint64_t b = desc_lohi((ls + (C::oX >> 4) + 2 * kb) | kLbo, kHi128);
            const uint32_t sfa = (sl + 4 * chunk) | (byte << 30);
            const uint32_t sfb = (sl + 4 * C::kChunks + 4 * chunk) | (byte << 30);
            fp4_mma<KIND, 1>(tm, a, b, idesc, sfa, sfb, kt > k0 || kb > 0 ? 1u : 0u);
          }
        }
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == C::kStages) { stage = 0; phase ^= 1; }
    }
    if (elect_one()) tc_commit(acc_full);
    __syncwarp();
    // the MMAs are complete before their operands' place or tensor memory is used otherwise
    (void)mbar_wait(acc_full, 0, 1000000000ull, nullptr, true);
  } else {
    // ----------------------------------------- scales, then the sums (warps 2-5)
    const int q = warp & 3;  // tensor-memory lanes 32 q .. 32 q + 31
    const uint32_t tq = tmem_base + ((uint32_t)(32 * q) << 16);
    uint32_t stage = 0, phase = 0;
    for (int kt = k0; kt < k1; kt++) {
      if (!mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag)) { *abort_flag = 1; break; }
      const uint8_t* sb = smem + stage * C::kStageBytes + 16 * lane;
      const uint32_t sl = tq + TN + stage * (uint32_t)C::kSlotCols;
      uint4 v[2 * C::kChunks];
#pragma unroll
      for (int c = 0; c < C::kChunks; c++) {
        v[c] = *reinterpret_cast<const uint4*>(sb + C::oSfw + 512 * c);
        v[C::kChunks + c] = *reinterpret_cast<const uint4*>(sb + C::oSfx + 512 * c);
      }
#pragma unroll
      for (int c = 0; c < 2 * C::kChunks; c += 4) tmem_st16(sl + 4 * c, v + c);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[stage]);
      if (++stage == C::kStages) { stage = 0; phase ^= 1; }
    }
    if (!*abort_flag && !mbar_wait(acc_full, 0, p.timeout_ns, abort_flag)) *abort_flag = 1;
    if (!*abort_flag) {
      // this slice's sums, [row of the activations][weight row], in the idle stages' place
      tc_fence_after();
      float* part = reinterpret_cast<float*>(smem) + 32 * q + lane;
#pragma unroll
      for (int c = 0; c < TN; c += 32) {
        uint32_t v[32];
        tmem_ld32_nowait(tq + (uint32_t)c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i++) part[(c + i) * C::BM] = __uint_as_float(v[i]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync_all();  // every slice's sums are in place
  if (warp >= 2 && !*abort_flag) {
    // a warp takes a row of the tile at a time, a lane four adjacent columns; all
    // slices' sums are on their way before the first is added
    const int64_t n = n0 + 4 * lane;  // n is a multiple of 8: four columns are inside or outside together
    const int rows = (int)(p.t - t0 < TN ? p.t - t0 : TN);
    const uint32_t part = smem_u32(smem) + (uint32_t)(16 * lane);
    if (n < p.n) {
      const float4 rw = __ldg(reinterpret_cast<const float4*>(p.row_w + n));
      uint32_t peer[kFp4FewMaxSplit];
#pragma unroll
      for (int r = 0; r < kFp4FewMaxSplit; r++) peer[r] = p.split > 1 && r < p.split ? mapa_u32(part, (uint32_t)r) : part;
#pragma unroll 2
      for (int t = slice + p.split * (warp - 2); t < rows; t += 4 * p.split) {
        float4 v[kFp4FewMaxSplit];
#pragma unroll
        for (int r = 0; r < kFp4FewMaxSplit; r++)
          if (r < p.split) v[r] = ld_cluster_f32x4(peer[r] + (uint32_t)(t * C::BM * 4));
        const float rf = __ldg(p.row_x + t0 + t);
        const bool far = KIND == GK_NVF4 && rf >= kFp4FarRow;
        const float rx = far ? rf * kFp4FarDown : rf, up = far ? kFp4FarUp : 1.0f;
        float4 f = v[0];
#pragma unroll
        for (int r = 1; r < kFp4FewMaxSplit; r++)
          if (r < p.split)
            f = make_float4(__fadd_rn(f.x, v[r].x), __fadd_rn(f.y, v[r].y), __fadd_rn(f.z, v[r].z), __fadd_rn(f.w, v[r].w));
        f = make_float4(__fmul_rn(__fmul_rn(f.x, rx), rw.x) * up, __fmul_rn(__fmul_rn(f.y, rx), rw.y) * up,
                        __fmul_rn(__fmul_rn(f.z, rx), rw.z) * up, __fmul_rn(__fmul_rn(f.w, rx), rw.w) * up);
        const int64_t at = (t0 + t) * p.n + n;
        if (p.y_bf16) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(f.x, f.y), hi = __floats2bfloat162_rn(f.z, f.w);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = f;
        }
      }
    }
  }
  __syncwarp();
  if (p.split > 1) cluster_sync_all();  // no CTA's shared memory goes before all have read it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace sharq

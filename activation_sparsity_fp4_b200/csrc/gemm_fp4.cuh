// gemm_fp4.cuh -- the plain FP4 product y = X W^T on tcgen05 block-scaled MMAs.
//
//   y[t][n] = r_x[t] r_w[n] sum_j (E2M1 x S)(t, j) (E2M1 x S)(n, j)
//
// Each block-scaled MMA multiplies 64 K elements of both operands by their
// block scales and adds into an fp32 accumulator in tensor memory; the rows'
// second-level scales are applied to it once, in the epilogue.
#pragma once
#include "fp4.cuh"
#include "gemm_pair.cuh"

namespace sharq {

// CTAS = 1: a CTA computes 128 x 256 outputs; CTAS = 2: two CTAs of a cluster
// compute 256 x 256, each holding 128 activation rows and half of the weight rows.
template <int KIND, int CTAS>
struct Fp4Cfg {
  static_assert(KIND == GK_NVF4 || KIND == GK_MXF4, "packed FP4 kinds");
  static constexpr int BM = 128, BN = 256, BNh = BN / CTAS, BK = 256;
  static constexpr int kVec = KIND == GK_NVF4 ? 16 : 32;
  static constexpr int kChunks = BK / kVec / 4;  // 512-byte scale chunks per 128 rows and stage
  static constexpr int kNRB = BN / 128;          // 128-row blocks of weight scales, all in every CTA
  static constexpr int kWBytes = BNh * 128, kXBytes = BM * 128;
  static constexpr int kSfx = kChunks * 512, kSfw = kNRB * kChunks * 512;
  static constexpr int oW = 0, oX = oW + kWBytes, oSfx = oX + kXBytes, oSfw = oSfx + kSfx;
  static constexpr int kStageBytes = ((oSfw + kSfw + 1023) / 1024) * 1024;
  static constexpr int kStages = CTAS == 2 ? 5 : 4;
  // tensor memory: accumulator, then a scale slot per stage
  static constexpr int cSfx = 0, cSfw = 4 * kChunks, kSlotCols = 4 * (1 + kNRB) * kChunks;
  static constexpr int kTmemCols = 512;
  static_assert(BN + kStages * kSlotCols <= kTmemCols, "tensor memory budget");
  static constexpr int kYRow = CTAS == 2 ? 64 : 32;   // bytes of an output row staged at a time, per warp
  static constexpr int kYBuf = 8 * 32 * kYRow;
  static constexpr int kSmemBytes = kStages * kStageBytes + kYBuf + 1024 /*align*/ + 256 /*barriers*/;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                     ((KIND == GK_NVF4 ? 0u : 1u) << 23) | ((uint32_t)((BM * CTAS) >> 4) << 24);
  static constexpr int kBandTiles = 2048 / (BM * CTAS);  // row tiles per raster band
};

struct Fp4Maps {
  CUtensorMap x, w, y;
};

struct Fp4GemmParams {
  int64_t t, n, k;
  int32_t experts;
  const int32_t* group_offsets;  // grouped form, else null
  const uint8_t* sf_x;
  const uint8_t* sf_w;
  const float* row_x;
  const float* row_w;
  int y_bf16;
  uint64_t timeout_ns;
};

template <int KIND, int CTAS>
__device__ __forceinline__ void fp4_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (CTAS == 2) {
    if constexpr (KIND == GK_NVF4) mma_nvf4_pair(d, a, b, idesc, sfa, sfb, accumulate);
    else mma_mxf4_pair(d, a, b, idesc, sfa, sfb, accumulate);
  } else {
    if constexpr (KIND == GK_NVF4) mma_nvf4(d, a, b, idesc, sfa, sfb, accumulate);
    else mma_mxf4(d, a, b, idesc, sfa, sfb, accumulate);
  }
}

// Per CTA (448 threads, one CTA per SM, persistent over output tiles):
//   warp 0      TMA producer: activation and weight tiles (counted on the leader's
//               full[]), this CTA's scale chunks (on its own sfull[]);
//   warp 1      tensor memory; in the leader one thread issues the MMAs;
//   warps 2-9   epilogue, two warps per 32-lane quadrant, 128 columns each;
//   warps 10-13 scale chunks, shared memory -> the stage's tensor-memory slot.
// Every wait is bounded in time; a timeout sets the abort flag of both CTAs and
// the device error word.
template <int KIND, int CTAS, bool GROUPED>
__global__ void __launch_bounds__(448, 1) gemm_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Fp4GemmParams p) {
  using C = Fp4Cfg<KIND, CTAS>;
  static_assert(!GROUPED || CTAS == 1, "expert segments are multiples of 128 rows");
  constexpr bool kPair = CTAS == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ybuf = smem + C::kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ybuf + C::kYBuf);  // leader: both CTAs' tiles
  uint64_t* empty = full + C::kStages;       // this CTA: the stage's MMAs have retired
  uint64_t* sfull = empty + C::kStages;      // this CTA: its scale chunks have landed
  uint64_t* sf_ready = sfull + C::kStages;   // leader: both CTAs' scale slots are in tensor memory
  uint64_t* acc_full = sf_ready + C::kStages;
  uint64_t* acc_empty = acc_full + 1;        // leader: both CTAs have drained their accumulator
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const int cluster = (int)(blockIdx.x / CTAS), nclusters = (int)(gridDim.x / CTAS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&sf_ready[s], 4 * CTAS);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 8 * CTAS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_holder, C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, C::kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch(&maps.x);
    tma_prefetch(&maps.w);
    tma_prefetch(&maps.y);
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  auto at_leader = [&](uint32_t a) { return kPair ? mapa_u32(a, 0) : a; };
  auto arrive_leader = [&](uint32_t a) {
    if constexpr (kPair) mbar_arrive_remote(a);
    else asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
  };
  auto give_up = [&]() {
    *abort_flag = 1;
    if constexpr (kPair) st_cluster_u32(mapa_u32(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
  };
  grid_dep_wait();
  grid_dep_launch();

  const int m_tiles = (int)((p.t + C::BM * CTAS - 1) / (C::BM * CTAS));
  const int n_tiles = (int)((p.n + C::BN - 1) / C::BN);
  const int num_tiles = m_tiles * n_tiles;
  const int k_tiles = (int)((p.k + C::BK - 1) / C::BK);
  const int64_t s_blocks = (p.k / C::kVec + 3) / 4;  // 512-byte chunks per 128 rows
  const int64_t w_blocks = (p.n + 127) / 128, x_blocks = (p.t + 127) / 128;
  // expert of a row tile; -1 = rows outside every group
  auto tile_expert = [&](int64_t m0) -> int {
    if constexpr (!GROUPED) return 0;
    if (m0 >= (int64_t)__ldg(p.group_offsets + p.experts)) return -1;
    int lo = 0, hi = p.experts;  // off[lo] <= m0 < off[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)__ldg(p.group_offsets + mid) <= m0) lo = mid;
      else hi = mid;
    }
    return lo;
  };

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t g = 0, issued = 0, issued_par = 0;
      const uint32_t smem0 = smem_u32(smem);
      const uint32_t full_leader = at_leader(smem_u32(full));
      for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
        const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
        const int64_t m0 = (int64_t)xy.mt * C::BM * CTAS + C::BM * (int64_t)rank;
        const int e = tile_expert(m0);
        if (e < 0) continue;
        const int32_t wrow = (int32_t)(e * p.n + (int64_t)xy.nt * C::BN + C::BNh * (int64_t)rank);
        // a block past the last one holds no row that is stored: any block stands in for its scales
        const int64_t xb = m0 / 128 < x_blocks ? m0 / 128 : x_blocks - 1;
        const uint8_t* g_sfx = p.sf_x + xb * s_blocks * 512;
        const uint8_t* g_sfw[C::kNRB];
#pragma unroll
        for (int rb = 0; rb < C::kNRB; rb++) {
          int64_t wb = (int64_t)xy.nt * C::kNRB + rb;
          if (wb >= w_blocks) wb = w_blocks - 1;
          g_sfw[rb] = p.sf_w + (e * w_blocks + wb) * s_blocks * 512;
        }
        for (int kt = 0; kt < k_tiles; kt++, g++) {
          const int stage = (int)(g % C::kStages);
          const uint32_t ph = (g / C::kStages) & 1u;
          if (!mbar_wait(&empty[stage], ph ^ 1u, p.timeout_ns, abort_flag)) { give_up(); break; }
          const uint32_t sb = smem0 + (uint32_t)(stage * C::kStageBytes);
          const uint32_t fl = full_leader + (uint32_t)(stage * 8);
          const uint32_t sf = smem_u32(&sfull[stage]);
          if (rank == 0) mbar_arrive_expect_tx_u32(smem_u32(&full[stage]), (uint32_t)(CTAS * (C::kWBytes + C::kXBytes)));
          if constexpr (kPair) {
            tma_load_2d_pair(sb + C::oW, &maps.w, kt * 128, wrow, fl);
            tma_load_2d_pair(sb + C::oX, &maps.x, kt * 128, (int32_t)m0, fl);
          } else {
            tma_load_2d_u32(sb + C::oW, &maps.w, kt * 128, wrow, fl);
            tma_load_2d_u32(sb + C::oX, &maps.x, kt * 128, (int32_t)m0, fl);
          }
          const int64_t left = s_blocks - (int64_t)kt * C::kChunks;
          const uint32_t bytes = (uint32_t)(left < C::kChunks ? left : C::kChunks) * 512u;
          const int64_t so = (int64_t)kt * C::kChunks * 512;
          mbar_arrive_expect_tx_u32(sf, bytes * (1 + C::kNRB));
          bulk_load_u32(sb + C::oSfx, g_sfx + so, bytes, sf);
#pragma unroll
          for (int rb = 0; rb < C::kNRB; rb++)
            bulk_load_u32(sb + C::oSfw + rb * C::kChunks * 512, g_sfw[rb] + so, bytes, sf);
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (ph << stage);
        }
      }
      if (*abort_flag) {
        // let every load already issued land before the block can exit
        for (int i = 0; i < C::kStages; i++)
          if ((issued >> i) & 1u) {
            (void)mbar_wait(&sfull[i], (issued_par >> i) & 1u, 1000000000ull, nullptr, true);
            if (rank == 0) (void)mbar_wait(&full[i], (issued_par >> i) & 1u, 1000000000ull, nullptr, true);
          }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    if (rank == 0 && lane == 0) {
      uint32_t g = 0;
      int it = 0;
      constexpr uint32_t kHi128 = desc_hi(1024, 2), kLbo = 1u << 16;
      const uint32_t lo0 = smem_u32(smem) >> 4;
      auto commit = [&](uint64_t* bar) {
        if constexpr (kPair) {
          tc_commit_pair(smem_u32(bar));
          tc_commit_pair(mapa_u32(smem_u32(bar), 1));
        } else {
          tc_commit(bar);
        }
      };
      for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
        const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
        if (tile_expert((int64_t)xy.mt * C::BM * CTAS) < 0) continue;
        if (!mbar_wait(acc_empty, (uint32_t)(it & 1) ^ 1u, p.timeout_ns, abort_flag)) { give_up(); break; }
        it++;
        tc_fence_after();
        uint32_t accumulate = 0;
        for (int kt = 0; kt < k_tiles; kt++, g++) {
          const int stage = (int)(g % C::kStages);
          const uint32_t ph = (g / C::kStages) & 1u;
          if (!mbar_wait(&full[stage], ph, p.timeout_ns, abort_flag)) { give_up(); break; }
          if (!mbar_wait(&sf_ready[stage], ph, p.timeout_ns, abort_flag)) { give_up(); break; }
          tc_fence_after();
          const uint32_t ls = lo0 + (uint32_t)(stage * (C::kStageBytes >> 4));
          const uint32_t sl = tmem_base + C::BN + (uint32_t)(stage * C::kSlotCols);
          const int64_t left = p.k - (int64_t)kt * C::BK;
#pragma unroll
          for (int kb = 0; kb < C::BK / 64; kb++) {
            if (64 * kb < left) {  // beyond K there are no scales
              constexpr int kScales = 64 / C::kVec;
              const uint32_t chunk = (kb * kScales) / 4, byte = (kb * kScales) % 4;
              const uint32_t idesc = C::kIdesc | (byte << 29) | (byte << 4);
              const uint64_t a = desc_lohi((ls + (C::oX >> 4) + 2 * kb) | kLbo, kHi128);
              const uint64_t b = desc_lohi((ls + (C::oW >> 4) + 2 * kb) | kLbo, kHi128);
              const uint32_t sfa = (sl + C::cSfx + 4 * chunk) | (byte << 30);
              const uint32_t sfb = (sl + C::cSfw + 4 * C::kNRB * chunk) | (byte << 30);
              fp4_mma<KIND, CTAS>(tmem_base, a, b, idesc, sfa, sfb, accumulate);
              accumulate = 1;
            }
          }
          commit(&empty[stage]);
        }
        if (*abort_flag) break;
        commit(acc_full);
      }
      // every MMA is complete before either CTA frees tensor memory or exits
      if constexpr (kPair) tc_commit_pair(smem_u32(drain));
      else tc_commit(drain);
      (void)mbar_wait(drain, 0, 1000000000ull, nullptr, true);
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------- epilogue
    // accumulator lanes 32q..32q+31 (output rows), columns 128h..128h+127
    constexpr int kCols = C::BN / 2;
    const int q = warp & 3, hcol = (warp - 2) >> 2;
    const uint32_t tq = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(kCols * hcol);
    const uint32_t acc_empty_leader = at_leader(smem_u32(acc_empty));
    uint8_t* yb = ybuf + (warp - 2) * 32 * C::kYRow;
    int it = 0;
    for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
      const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
      const int64_t m0 = (int64_t)xy.mt * C::BM * CTAS + C::BM * (int64_t)rank;
      const int e = tile_expert((int64_t)xy.mt * C::BM * CTAS);
      if (e < 0) continue;
      const int64_t row = m0 + 32 * q + lane;
      const float rx = row < p.t ? __ldg(p.row_x + row) : 0.0f;
      const int64_t n0 = (int64_t)xy.nt * C::BN + kCols * hcol;
      const float* rw = p.row_w + e * p.n;
      if (!mbar_wait(acc_full, (uint32_t)(it & 1), p.timeout_ns, abort_flag)) { give_up(); break; }
      it++;
      tc_fence_after();
      const int32_t row0 = (int32_t)(row - lane);
#pragma unroll 1
      for (int c = 0; c < kCols / 32; c++) {
        uint32_t v[32];
        tmem_ld32_nowait(tq + (uint32_t)(32 * c), v);
        tmem_ld_wait();
        float f[32];
#pragma unroll
        for (int j = 0; j < 8; j++) {  // n is a multiple of 8: four columns are inside or outside together
          const int64_t col = n0 + 32 * c + 4 * j;
          const float4 s = col < p.n ? __ldg(reinterpret_cast<const float4*>(rw + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
          f[4 * j] = __fmul_rn(__fmul_rn(__uint_as_float(v[4 * j]), rx), s.x);
          f[4 * j + 1] = __fmul_rn(__fmul_rn(__uint_as_float(v[4 * j + 1]), rx), s.y);
          f[4 * j + 2] = __fmul_rn(__fmul_rn(__uint_as_float(v[4 * j + 2]), rx), s.z);
          f[4 * j + 3] = __fmul_rn(__fmul_rn(__uint_as_float(v[4 * j + 3]), rx), s.w);
        }
        if (c == kCols / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(acc_empty_leader);
        }
        if (row0 >= p.t) continue;
        // kYRow bytes of each row at a time through shared memory, written by TMA
        // stores (whole lines; rows at or beyond t and columns from n on are clipped)
        const int es = p.y_bf16 ? 2 : 4, per = C::kYRow / es;
#pragma unroll
        for (int h = 0; h < 32 * 4 / C::kYRow; h++) {
          if (p.y_bf16 && h >= 32 * 2 / C::kYRow) break;
          if (lane == 0) bulk_wait_group_read0();  // the previous store has read the buffer
          __syncwarp();
          uint4* d = reinterpret_cast<uint4*>(yb + C::kYRow * lane);
#pragma unroll
          for (int j = 0; j < C::kYRow / 16; j++) {
            uint32_t o[4];
            if (p.y_bf16) {
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int at = (h * (C::kYRow / 2) + 8 * j + 2 * i) & 31;
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(f[at], f[at + 1]);
                o[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; i++) o[i] = __float_as_uint(f[h * (C::kYRow / 4) + 4 * j + i]);
            }
            d[j] = make_uint4(o[0], o[1], o[2], o[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          const int64_t col = n0 + 32 * c + h * per;
          if (lane == 0 && col < p.n) {
            tma_store_2d(&maps.y, smem_u32(yb), (int32_t)(es * col), row0);
            bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group0();  // output stores complete
  } else {
    // ------------------------------------------------ scale-slot staging
    const int q = warp & 3;
    const uint32_t tq = tmem_base + ((uint32_t)(32 * q) << 16);
    const uint32_t ready_leader = at_leader(smem_u32(sf_ready));
    uint32_t g = 0;
    for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
      const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
      if (tile_expert((int64_t)xy.mt * C::BM * CTAS) < 0) continue;
      for (int kt = 0; kt < k_tiles; kt++, g++) {
        const int stage = (int)(g % C::kStages);
        // the chunks were loaded into a stage, and so into a slot, whose MMAs have retired
        if (!mbar_wait(&sfull[stage], (g / C::kStages) & 1u, p.timeout_ns, abort_flag)) { give_up(); break; }
        tc_fence_after();
        const uint8_t* sb = smem + stage * C::kStageBytes;
        const uint32_t st = tq + C::BN + (uint32_t)(stage * C::kSlotCols);
#pragma unroll
        for (int c = 0; c < C::kChunks; c++) {
          tmem_st4(st + C::cSfx + 4 * c, *reinterpret_cast<const uint4*>(sb + C::oSfx + 512 * c + 16 * lane));
#pragma unroll
          for (int rb = 0; rb < C::kNRB; rb++)
            tmem_st4(st + C::cSfw + 4 * C::kNRB * c + 4 * rb,
                     *reinterpret_cast<const uint4*>(sb + C::oSfw + (rb * C::kChunks + c) * 512 + 16 * lane));
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(ready_leader + (uint32_t)(stage * 8));
      }
    }
  }

  // the leader's MMAs read the other CTA's shared memory and write its tensor
  // memory: neither frees tensor memory or exits before both are done
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace sharq

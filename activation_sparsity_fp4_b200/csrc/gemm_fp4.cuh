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
  // a ring of operand stages of BK each
  static constexpr int oW = 0, oX = oW + kWBytes, kStageBytes = oX + kXBytes;
  static constexpr int kStages = CTAS == 2 ? 5 : 3;
  // The scales go a step further, shared -> tensor memory, by warps whose waits
  // and barriers cost more than the copy: they move two K tiles' worth at a
  // time, in rings of their own in both memories.
  static constexpr int kSfTiles = 2, kSfChunks = kSfTiles * kChunks;
  static constexpr int kSfx = kSfChunks * 512, kSfw = kNRB * kSfChunks * 512;
  static constexpr int oSfx = 0, oSfw = oSfx + kSfx, kSfBytes = oSfw + kSfw;
  static constexpr int kSfStages = 2;
  // tensor memory: accumulator, then the scale slots
  static constexpr int cSfx = 0, cSfw = 4 * kSfChunks, kSlotCols = 4 * (1 + kNRB) * kSfChunks;
  static constexpr int kSlots = 2;
  static_assert(kNRB == 2, "256 weight rows");
  static constexpr int kTmemCols = 512;
  static_assert(BN + kSlots * kSlotCols <= kTmemCols, "tensor memory budget");
  static constexpr int kYRow = 128;             // bytes of an output row staged at a time, per epilogue warp
  static constexpr int kYBuf = 8 * 32 * kYRow;
  static constexpr int kTable = CTAS == 1 ? 1024 : 0;  // experts whose offsets are held in shared memory
  static constexpr int kSmemBytes = kStages * kStageBytes + kSfStages * kSfBytes + kYBuf + 8 * 128 * 4 + 4 * kTable + 1024 /*align*/ + 256 /*barriers*/;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                     ((KIND == GK_NVF4 ? 0u : 1u) << 23) | ((uint32_t)((BM * CTAS) >> 4) << 24);
  static constexpr int kBandTiles = 2048 / (BM * CTAS);  // row tiles per raster band
};

// 128 registers a thread at launch; the epilogue's two warpgroups hold 128 sums
// and more, the other two give up what they can spare.
constexpr int kFp4GemmThreads = 512, kFp4GemmRegs = 128, kFp4RegsLow = 72, kFp4RegsHigh = 184;
static_assert(2 * kFp4RegsLow + 2 * kFp4RegsHigh == 4 * kFp4GemmRegs, "no more than the block was launched with");

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

// A sum is up to 2^23 k, so that its product with a row factor near fp32's end leaves
// fp32 where the column's factor would bring it back.  From 2^72 on a factor is taken
// at 2^-56 of its size, and the output brought up at last (exact, 1 otherwise).  MXFP4's
// row factors are 1.
constexpr float kFp4FarRow = 0x1p72f, kFp4FarDown = 0x1p-56f, kFp4FarUp = 0x1p56f;

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

// Per CTA (512 threads, one CTA per SM, persistent over output tiles):
//   warp 0      TMA producer of activation and weight tiles (counted on the
//               leader's full[]);
//   warp 1      tensor memory; in the leader it issues the MMAs;
//   warp 2      producer of this CTA's scale chunks (sfull[]); warp 3 has no part;
//   warps 4-7   scale chunks, shared memory -> a tensor-memory slot;
//   warps 8-15  epilogue, two warps per 32-lane quadrant, 128 columns each: the
//               raw sums into registers, so that the next tile's MMAs wait for
//               the tensor-memory loads alone; the factors, the rounding and the
//               stores run under those MMAs.
// Every wait is bounded in time; a timeout sets the abort flag of both CTAs and
// the device error word.
// CTAS = 1 is the grouped form (expert segments are multiples of 128 rows, so two
// row tiles need not share a weight), CTAS = 2 the plain one (with one CTA a tile it
// was 398 us where it was 362, and no size was faster).
//
// 32768 x 5120 x 5120: NVFP4 328 to 335 us (5.1 PFLOP/s), MXFP4 306 us (5.6), bound by
// the issue of one warp (about 80 cycles an MMA, with its waits near the 128 that an
// MMA runs) and by the operands' and scales' way into shared and tensor memory.
// 2048 x 4096 x 4096: 18.1 us, of which two rounds of tiles are 8.3 us of MMAs and the rest
// launch, first loads and the last epilogue, which nothing overlaps.
// 40832 routed rows x 1536 x 2048 of 128 experts, NVFP4: 90 us, 400 MB (4.4 TB/s): the
// waits for a tile's loads, with three stages in flight (DRAM 53 % busy, the pipe 32 %).
// NVFP4's instantiations spill 80 bytes a thread at 128 registers, once a tile.
template <int KIND, int CTAS>
__global__ void __launch_bounds__(kFp4GemmThreads, 1) gemm_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Fp4GemmParams p) {
  using C = Fp4Cfg<KIND, CTAS>;
  constexpr bool kPair = CTAS == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sfbuf = smem + C::kStages * C::kStageBytes;
  uint8_t* ybuf = sfbuf + C::kSfStages * C::kSfBytes;
  float* rwbuf = reinterpret_cast<float*>(ybuf + C::kYBuf);        // the epilogue warps' column factors
  int32_t* table = reinterpret_cast<int32_t*>(rwbuf + 8 * 128);
  uint64_t* full = reinterpret_cast<uint64_t*>(table + C::kTable);  // leader: both CTAs' tiles
  uint64_t* empty = full + C::kStages;       // this CTA: the stage's MMAs have retired
  uint64_t* sfull = empty + C::kStages;      // this CTA: its scale chunks have landed
  uint64_t* sfree = sfull + C::kSfStages;    // this CTA: they have been copied
  uint64_t* sf_ready = sfree + C::kSfStages; // leader: both CTAs' scale slots are in tensor memory
  uint64_t* slot_empty = sf_ready + C::kSlots;  // this CTA: the slot's MMAs have retired
  uint64_t* acc_full = slot_empty + C::kSlots;
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
    }
    for (int s = 0; s < C::kSlots; s++) {
      mbar_init(&sf_ready[s], 4 * CTAS);
      mbar_init(&slot_empty[s], 1);
    }
    for (int s = 0; s < C::kSfStages; s++) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], 4);
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

  // Grouped: the rows in use end at the last offset, and a tile's expert is found
  // in a table in shared memory.  (Looked up in global memory, with hardly any L1
  // beside this much shared memory, the search took every role 2800 of a tile's
  // 10500 cycles; 40832 rows x 1536 x 2048 of 128 experts: 92.3 us where it is 90.2.)
  int64_t t_used = p.t, t_first = 0;
  if constexpr (!kPair) {
    const int64_t last = (int64_t)__ldg(p.group_offsets + p.experts);
    t_used = last < 0 ? 0 : last < p.t ? last : p.t;
    t_first = (int64_t)__ldg(p.group_offsets);
    for (int e = threadIdx.x; e < p.experts && e < C::kTable; e += kFp4GemmThreads) table[e] = __ldg(p.group_offsets + e);
    __syncthreads();
  }
  const int m_tiles = (int)((t_used + C::BM * CTAS - 1) / (C::BM * CTAS));
  const int n_tiles = (int)((p.n + C::BN - 1) / C::BN);
  const int num_tiles = m_tiles * n_tiles;
  const int k_tiles = (int)((p.k + C::BK - 1) / C::BK);
  const int k_groups = (k_tiles + C::kSfTiles - 1) / C::kSfTiles;  // of scales
  const int64_t s_blocks = (p.k / C::kVec + 3) / 4;  // 512-byte chunks per 128 rows
  const int64_t w_blocks = (p.n + 127) / 128, x_blocks = (p.t + 127) / 128;
  // rows in front of the first group belong to no expert
  auto outside = [&](int64_t m0) { return !kPair && m0 < t_first; };
  auto tile_expert = [&](int64_t m0) -> int {
    if constexpr (kPair) return 0;
    int lo = 0, hi = p.experts;  // off[lo] <= m0 < off[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      const int32_t at = mid < C::kTable ? table[mid] : __ldg(p.group_offsets + mid);
      if ((int64_t)at <= m0) lo = mid;
      else hi = mid;
    }
    return lo;
  };

  if (warp < 4) regs_down<kFp4RegsLow>();
  if (warp == 0) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      uint32_t g = 0, issued = 0, issued_par = 0;
      const uint32_t smem0 = smem_u32(smem);
      const uint32_t full_leader = at_leader(smem_u32(full));
      for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
        const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
        const int64_t m0 = (int64_t)xy.mt * C::BM * CTAS + C::BM * (int64_t)rank;
        if (outside(m0)) continue;
        const int e = tile_expert(m0);
        const int32_t wrow = (int32_t)(e * p.n + (int64_t)xy.nt * C::BN + C::BNh * (int64_t)rank);
        for (int kt = 0; kt < k_tiles; kt++, g++) {
          const int stage = (int)(g % C::kStages);
          const uint32_t ph = (g / C::kStages) & 1u;
          if (!mbar_wait(&empty[stage], ph ^ 1u, p.timeout_ns, abort_flag)) { give_up(); break; }
          const uint32_t sb = smem0 + (uint32_t)(stage * C::kStageBytes);
          const uint32_t fl = full_leader + (uint32_t)(stage * 8);
          if (rank == 0) mbar_arrive_expect_tx_u32(smem_u32(&full[stage]), (uint32_t)(CTAS * (C::kWBytes + C::kXBytes)));
          if constexpr (kPair) {
            tma_load_2d_pair(sb + C::oW, &maps.w, kt * 128, wrow, fl);
            tma_load_2d_pair(sb + C::oX, &maps.x, kt * 128, (int32_t)m0, fl);
          } else {
            tma_load_2d_u32(sb + C::oW, &maps.w, kt * 128, wrow, fl);
            tma_load_2d_u32(sb + C::oX, &maps.x, kt * 128, (int32_t)m0, fl);
          }
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (ph << stage);
        }
      }
      if (*abort_flag) {
        // let every load already issued land before the block can exit (the pair's are all counted here)
        for (int i = 0; i < C::kStages; i++)
          if (rank == 0 && ((issued >> i) & 1u)) (void)mbar_wait(&full[i], (issued_par >> i) & 1u, 1000000000ull, nullptr, true);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    // the whole warp runs the loop, so that its addresses and descriptors stay
    // uniform; one lane issues (a branch on the lane number cost 112 cycles an
    // MMA in moves to uniform registers, more than the MMA's own 124 leave room for)
    if (rank == 0) {
      uint32_t stage = 0, ph = 0, slot = 0, sph = 0, acc_ph = 1;
      constexpr uint32_t kHi128 = desc_hi(1024, 2), kLbo = 1u << 16;
      const uint32_t lo0 = __shfl_sync(0xffffffffu, smem_u32(smem) >> 4, 0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
      auto commit = [&](uint64_t* bar) {
        if constexpr (kPair) tc_commit_pair_both(smem_u32(bar));
        else tc_commit(bar);
      };
      // votes, so that the compiler sees one way through the loop
      auto waited = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.timeout_ns, abort_flag)) != 0;
      };
      for (int tile = cluster; tile < num_tiles; tile += nclusters) {
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
        if (outside((int64_t)xy.mt * C::BM * CTAS)) continue;
        if (!waited(acc_empty, acc_ph)) { give_up(); break; }
        acc_ph ^= 1u;
        tc_fence_after();
        int left = (int)((p.k + 63) / 64);  // MMAs of this tile still to come (beyond K there are no scales)
        bool ok = true;
        // A group's two stages and scales are asked after together: a wait costs the
        // issuing warp 75 cycles and more though nothing is missing, an MMA 80 of
        // the 128 that it runs for, so one wait a stage left the pipe idle.
        for (int kt = 0; ok && kt < k_tiles; kt += C::kSfTiles) {
          static_assert(C::kSfTiles == 2, "two stages a group");
          const bool two = kt + 1 < k_tiles, end = kt + C::kSfTiles >= k_tiles;
          const uint32_t wrap = stage + 1 == C::kStages, stage1 = wrap ? 0u : stage + 1, ph1 = ph ^ wrap;
          const uint32_t seen = __reduce_and_sync(
              0xffffffffu, mbar_test3(&full[stage], ph, &sf_ready[slot], sph, &full[stage1], ph1));
          if ((seen & 3u) != 3u) ok = waited(&full[stage], ph) && waited(&sf_ready[slot], sph);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sl = tm + C::BN + slot * (uint32_t)C::kSlotCols;
          auto issue = [&](uint32_t st, uint32_t half, int left) {  // the MMAs of a stage
            const uint32_t ls = lo0 + st * (uint32_t)(C::kStageBytes >> 4);
            const uint32_t slx = sl + C::cSfx + 4 * C::kChunks * half;
            const uint32_t slw = sl + C::cSfw + 4 * C::kNRB * C::kChunks * half;
#pragma unroll
            for (int kb = 0; kb < C::BK / 64; kb++) {
              if (kb < left) {
                constexpr int kScales = 64 / C::kVec;
                const uint32_t chunk = (kb * kScales) / 4, byte = (kb * kScales) % 4;
                const uint32_t idesc = C::kIdesc | (byte << 29) | (byte << 4);
                const uint64_t a = desc_lohi((ls + (C::oX >> 4) + 2 * kb) | kLbo, kHi128);
                const uint64_t b = desc_lohi((ls + (C::oW >> 4) + 2 * kb) | kLbo, kHi128);
                const uint32_t sfa = (slx + 4 * chunk) | (byte << 30);
                const uint32_t sfb = (slw + 4 * C::kNRB * chunk) | (byte << 30);
                fp4_mma<KIND, CTAS>(tm, a, b, idesc, sfa, sfb, kt > 0 || half > 0 || kb > 0 ? 1u : 0u);
              }
            }
          };
          if (two && (seen & 4u)) {  // the usual case: all of the group at once
            if (elect_one()) {
              issue(stage, 0, left);
              commit(&empty[stage]);
              issue(stage1, 1, left - C::BK / 64);
              commit(&empty[stage1]);
              commit(&slot_empty[slot]);
              if (end) commit(acc_full);
            }
            __syncwarp();
          } else {
            if (elect_one()) {
              issue(stage, 0, left);
              commit(&empty[stage]);
              if (!two) {
                commit(&slot_empty[slot]);
                commit(acc_full);
              }
            }
            __syncwarp();
            if (two) {
              ok = waited(&full[stage1], ph1);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                issue(stage1, 1, left - C::BK / 64);
                commit(&empty[stage1]);
                commit(&slot_empty[slot]);
                if (end) commit(acc_full);
              }
              __syncwarp();
            }
          }
          left -= C::kSfTiles * (C::BK / 64);
          if (two) {
            ph = ph1;
            stage = stage1;
          }
          if (++stage == C::kStages) {
            stage = 0;
            ph ^= 1u;
          }
          if (++slot == C::kSlots) {
            slot = 0;
            sph ^= 1u;
          }
        }
        if (!ok) { give_up(); break; }
      }
      // every MMA is complete before either CTA frees tensor memory or exits
      if (elect_one()) {
        if constexpr (kPair) tc_commit_pair(smem_u32(drain));
        else tc_commit(drain);
      }
      __syncwarp();
      (void)mbar_wait(drain, 0, 1000000000ull, nullptr, true);
    }
  } else if (warp >= 8) {
    regs_up<kFp4RegsHigh>();
    // ------------------------------------------------------------- epilogue
    // accumulator lanes 32q..32q+31 (output rows), columns 128h..128h+127
    constexpr int kCols = C::BN / 2;
    const int q = warp & 3, hcol = (warp - 8) >> 2;
    const uint32_t tq = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(kCols * hcol);
    const uint32_t acc_empty_leader = at_leader(smem_u32(acc_empty));
    uint8_t* yb = ybuf + (warp - 8) * 32 * C::kYRow;
    int it = 0;
    for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
      const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
      const int64_t m0 = (int64_t)xy.mt * C::BM * CTAS + C::BM * (int64_t)rank;
      if (outside(m0)) continue;
      const int e = tile_expert(m0);
      const int64_t row = m0 + 32 * q + lane;
      const float rx = row < p.t ? __ldg(p.row_x + row) : 0.0f;
      const int64_t n0 = (int64_t)xy.nt * C::BN + kCols * hcol;
      // this warp's 128 column factors, one lane's four at a time (n is a multiple of 8)
      float* rws = rwbuf + (warp - 8) * kCols;
      __syncwarp();  // the previous tile's have been read
      const int64_t cw = n0 + 4 * lane;
      *reinterpret_cast<float4*>(rws + 4 * lane) =
          cw < p.n ? __ldg(reinterpret_cast<const float4*>(p.row_w + e * p.n + cw)) : make_float4(0.f, 0.f, 0.f, 0.f);
      __syncwarp();
      if (!mbar_wait(acc_full, (uint32_t)(it & 1), p.timeout_ns, abort_flag)) { give_up(); break; }
      it++;
      tc_fence_after();
      const int32_t row0 = (int32_t)(row - lane);
      // 128 bytes of each row at a time through shared memory (in the tensor map's
      // 128-byte swizzle, so that neither side meets bank conflicts), written by a
      // TMA store: whole lines; rows at or beyond t and columns from n on are clipped
      auto store = [&](const uint32_t* w, int64_t col) {
        if (lane == 0) bulk_wait_group_read0();  // the previous store has read the buffer
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; j++)
          *reinterpret_cast<uint4*>(yb + C::kYRow * lane + ((j ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && col < p.n) {
          tma_store_2d(&maps.y, smem_u32(yb), (int32_t)((p.y_bf16 ? 2 : 4) * col), row0);
          bulk_commit_group();
        }
      };
      uint32_t v[kCols];
#pragma unroll
      for (int c = 0; c < kCols / 32; c++)
        tmem_ld32_nowait(tq + (uint32_t)(32 * c), *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(acc_empty_leader);
      if (row0 >= p.t) continue;
      auto times = [&](float r, float up) {  // the row factors, read while the tile's MMAs ran
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const float4 s = *reinterpret_cast<const float4*>(rws + c);
          v[c] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(v[c]), r), s.x) * up);
          v[c + 1] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(v[c + 1]), r), s.y) * up);
          v[c + 2] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(v[c + 2]), r), s.z) * up);
          v[c + 3] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(v[c + 3]), r), s.w) * up);
        }
      };
      if (KIND == GK_NVF4 && __any_sync(0xffffffffu, rx >= kFp4FarRow))
        times(rx >= kFp4FarRow ? rx * kFp4FarDown : rx, rx >= kFp4FarRow ? kFp4FarUp : 1.0f);
      else
        times(rx, 1.0f);
      if (p.y_bf16) {
#pragma unroll
        for (int i = 0; i < kCols / 2; i++) {
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          v[i] = *reinterpret_cast<const uint32_t*>(&h2);
        }
#pragma unroll
        for (int i = 0; i < kCols / 2; i += C::kYRow / 4) store(v + i, n0 + 2 * i);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; i += C::kYRow / 4) store(v + i, n0 + i);
      }
    }
    if (lane == 0) bulk_wait_group0();  // output stores complete
  } else if (warp == 2) {
    // ------------------------------------------------------ scale producer
    if (lane == 0) {
      uint32_t g = 0, issued = 0, issued_par = 0;
      const uint32_t sf0 = smem_u32(sfbuf);
      for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
        const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
        const int64_t m0 = (int64_t)xy.mt * C::BM * CTAS + C::BM * (int64_t)rank;
        if (outside(m0)) continue;
        const int e = tile_expert(m0);
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
        for (int q = 0; q < k_groups; q++, g++) {
          const int ss = (int)(g % C::kSfStages);
          const uint32_t ph = (g / C::kSfStages) & 1u;
          if (!mbar_wait(&sfree[ss], ph ^ 1u, p.timeout_ns, abort_flag)) { give_up(); break; }
          const uint32_t sb = sf0 + (uint32_t)(ss * C::kSfBytes), sf = smem_u32(&sfull[ss]);
          const int64_t left = s_blocks - (int64_t)q * C::kSfChunks;
          const uint32_t bytes = (uint32_t)(left < C::kSfChunks ? left : C::kSfChunks) * 512u;
          const int64_t so = (int64_t)q * C::kSfChunks * 512;
          mbar_arrive_expect_tx_u32(sf, bytes * (1 + C::kNRB));
          bulk_load_u32(sb + C::oSfx, g_sfx + so, bytes, sf);
#pragma unroll
          for (int rb = 0; rb < C::kNRB; rb++)
            bulk_load_u32(sb + C::oSfw + rb * C::kSfChunks * 512, g_sfw[rb] + so, bytes, sf);
          issued |= 1u << ss;
          issued_par = (issued_par & ~(1u << ss)) | (ph << ss);
        }
      }
      if (*abort_flag) {
        for (int i = 0; i < C::kSfStages; i++)
          if ((issued >> i) & 1u) (void)mbar_wait(&sfull[i], (issued_par >> i) & 1u, 1000000000ull, nullptr, true);
      }
    }
  } else if (warp >= 4) {
    regs_down<kFp4RegsLow>();
    // ------------------------------------------------ scale-slot staging
    const int q = warp & 3;
    const uint32_t tq = tmem_base + ((uint32_t)(32 * q) << 16);
    const uint32_t ready_leader = at_leader(smem_u32(sf_ready));
    uint32_t g = 0;
    for (int tile = cluster; tile < num_tiles && !*abort_flag; tile += nclusters) {
      const TileXY xy = tile_xy(tile, m_tiles, n_tiles, C::kBandTiles);
      if (outside((int64_t)xy.mt * C::BM * CTAS)) continue;
      for (int kq = 0; kq < k_groups; kq++, g++) {
        const uint32_t ss = g % C::kSfStages, slot = g % C::kSlots;
        bool ok = true;
        if (!mbar_wait(&sfull[ss], (g / C::kSfStages) & 1u, p.timeout_ns, abort_flag)) { give_up(); break; }
        const uint8_t* sb = sfbuf + ss * C::kSfBytes + 16 * lane;
        const uint32_t st = tq + C::BN + slot * (uint32_t)C::kSlotCols;
        constexpr int kPieces = (1 + C::kNRB) * C::kSfChunks;  // of 16 bytes a lane, in the slot's order of columns
        auto piece = [&](int i) {
          const int c = (i - C::kSfChunks) / C::kNRB, rb = (i - C::kSfChunks) % C::kNRB;
          return *reinterpret_cast<const uint4*>(i < C::kSfChunks ? sb + C::oSfx + 512 * i
                                                                  : sb + C::oSfw + (rb * C::kSfChunks + c) * 512);
        };
#pragma unroll
        for (int h = 0; h < 2; h++) {
          uint4 v[kPieces / 2];
#pragma unroll
          for (int i = 0; i < kPieces / 2; i++) v[i] = piece(h * (kPieces / 2) + i);
          if (h == 0) {  // the MMAs that used the slot before have retired
            ok = mbar_wait(&slot_empty[slot], ((g / C::kSlots) & 1u) ^ 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            tc_fence_after();
          }
          static_assert(kPieces % 4 == 0, "halves of stores of 16 and 8 columns");
#pragma unroll
          for (int i = 0; i + 4 <= kPieces / 2; i += 4) tmem_st16(st + 4 * (h * (kPieces / 2) + i), v + i);
          if constexpr ((kPieces / 2) % 4 == 2)
            tmem_st8(st + 4 * (h * (kPieces / 2) + kPieces / 2 - 2), v[kPieces / 2 - 2], v[kPieces / 2 - 1]);
        }
        if (!ok) { give_up(); break; }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_leader(ready_leader + slot * 8);
          mbar_arrive(&sfree[ss]);
        }
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

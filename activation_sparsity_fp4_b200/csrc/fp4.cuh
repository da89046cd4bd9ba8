// fp4.cuh -- rows to microscaled FP4 (one operand a row, no split): MXFP4 and
// NVFP4 codes, tiled scales and the row's second-level scale in one pass.
#pragma once
#include "prep.cuh"
#include "route.cuh"

namespace sharq {

constexpr int64_t kFp4MaxHeld = 16384;  // longest row that fp4_kernel holds in registers (32 warps x 32 units)

enum { FRONT_NONE = 0, FRONT_NORM = 1, FRONT_SWIGLU = 2 };

struct Fp4Params {
  const void* x;      // SwiGLU: the gate
  const void* x2;     // SwiGLU: the up input
  int64_t x_rows, stride;
  const int32_t* rows;
  const int32_t* count;
  const void* gamma;
  float eps, amax;
  int64_t rows_out, k;      // all experts' rows; per expert rows_expert
  int64_t rows_expert;
  uint8_t* codes;
  uint8_t* scales;
  float* row_scale;
};

// 16 consecutive values of the input row(s) in front of the norm.
template <int FRONT, bool XBF16>
__device__ __forceinline__ void fp4_load16(const Fp4Params& p, int64_t at, float (&v)[16]) {
  float a[8], b[8];
  load8<XBF16>(p.x, at, a);
  load8<XBF16>(p.x, at + 8, b);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = a[i];
    v[8 + i] = b[i];
  }
  if constexpr (FRONT == FRONT_SWIGLU) {
    load8<XBF16>(p.x2, at, a);
    load8<XBF16>(p.x2, at + 8, b);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      v[i] = __fmul_rn(dev_silu(v[i]), a[i]);
      v[8 + i] = __fmul_rn(dev_silu(v[8 + i]), b[i]);
    }
  }
}

// ------------------------------------------------- a row in registers
// wpr warps share a row, a lane holds NJ units of 16 adjacent values (unit
// w * 32 + lane + 32 wpr j of the row), read once.  The row's sum of squares and
// largest magnitude are reduced by shuffles and, across its warps, through
// shared memory behind a barrier of those warps alone.

// Largest magnitude.  WIDE: up to 32 warps a row, else up to 8.
template <bool WIDE>
__device__ __forceinline__ float row_max(float v, float* red /* wpr floats, a multiple of 8 */, int wr, int wpr,
                                         int barrier) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  if (wpr > 1) {
    const int lane = threadIdx.x & 31, slots = WIDE ? (wpr + 7) & ~7 : 8;
    if (lane == 0) red[wr] = v;
    if (wr == 0 && lane >= wpr && lane < slots) red[lane] = 0.0f;  // no magnitude is smaller
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(wpr * 32) : "memory");
    for (int i = 0; i < (WIDE ? slots : 8); i += 8) {
      const float4 c = *reinterpret_cast<const float4*>(red + i), d = *reinterpret_cast<const float4*>(red + i + 4);
      const float t = fmaxf(fmaxf(fmaxf(c.x, c.y), fmaxf(c.z, c.w)), fmaxf(fmaxf(d.x, d.y), fmaxf(d.z, d.w)));
      v = i == 0 ? t : fmaxf(v, t);
    }
  }
  return v;
}

// Sum over a row's units, s[j] that of this lane's unit j.  The order is that of
// sharq_prepare and of the oracle, a tree of adjacent units whatever warps and lanes
// hold them, so that a row has one sum in every batch: adjacent lanes first, which
// gives the sums of chunks of 32 units, then adjacent chunks.  The first shuffles
// halve the number of sums as they go (a lane keeps those of chunks whose low bits
// are its own), so two or four units a lane cost no more shuffles than one.
// LANES: the chunks are added by shuffles again, else by every lane from 16-byte reads.
// NVFP4 takes the first and MXFP4 the second for the registers that the compiler
// then needs, which decide between three and four blocks of five warps an SM
// (32768 x 5120: NVFP4 128 us with 96 registers against 147 with 102, MXFP4 110 with
// 88 against 124 with 98).
template <int NJ, bool LANES>
__device__ __forceinline__ float row_sum(const float (&s)[NJ], float* red /* a float a chunk, a multiple of 8 */, int wr,
                                         int wpr, int barrier) {
  static_assert(NJ == 1 || NJ == 2 || NJ == 4, "units a lane");
  const int lane = threadIdx.x & 31;
  float a[NJ];
#pragma unroll
  for (int j = 0; j < NJ; j++) a[j] = s[j];
  int m = 1;
#pragma unroll
  for (int n = NJ; n > 1; n /= 2, m *= 2)
#pragma unroll
    for (int j = 0; j < n; j += 2) {
      const bool odd = (lane & m) != 0;
      const float keep = odd ? a[j + 1] : a[j], give = odd ? a[j] : a[j + 1];
      a[j / 2] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, m));
    }
  float v = a[0];
#pragma unroll
  for (int q = NJ; q < 32; q *= 2) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, q));
  // lane l: the chunk of units l % NJ of this warp's lanes, chunk wr + wpr (l % NJ) of the row
  if (wpr == 1) {
#pragma unroll
    for (int q = 1; q < NJ; q *= 2) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, q));
    return v;
  }
  const int slots = (NJ * wpr + 3) & ~3;  // at most 32
  if (lane < NJ) red[wr + wpr * lane] = v;
  if (wr == 0 && lane >= NJ * wpr && lane < slots) red[lane] = 0.0f;
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(wpr * 32) : "memory");
  if constexpr (LANES) {
    v = lane < slots ? red[lane] : 0.0f;
#pragma unroll
    for (int q = 1; q < 32; q *= 2) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, q));
    return v;
  }
  auto four = [&](int i) {
    const float4 c = *reinterpret_cast<const float4*>(red + i);
    return __fadd_rn(__fadd_rn(c.x, c.y), __fadd_rn(c.z, c.w));
  };
  auto eight = [&](int i) { return slots > i + 4 ? __fadd_rn(four(i), four(i + 4)) : four(i); };
  v = eight(0);
  if (slots > 8) v = __fadd_rn(v, eight(8));
  if (slots > 16) v = __fadd_rn(v, slots > 24 ? __fadd_rn(eight(16), eight(24)) : eight(16));
  return v;
}

// mean(x^2) + eps and 1 / sqrt of it, every step rounded once as in sharq_prepare (the reciprocal of a root is its
// quotient).
__device__ __forceinline__ float fp4_mean(float sumsq, int64_t k, float eps) {
  return __fadd_rn(__fdiv_rn(sumsq, (float)k), eps);
}
__device__ __forceinline__ float fp4_rstd(float mean) { return __frcp_rn(__fsqrt_rn(mean)); }

// Rows whose squares leave fp32 (values from about 2^64 / sqrt(k) on, or below 2^-45
// where eps is as small) are summed again at 2^-80 or 2^90 of their size.
__device__ __forceinline__ bool fp4_mean_in_range(float mean) { return mean >= 0x1p-90f && mean <= 3.402823466e38f; }
__device__ __forceinline__ float fp4_norm_scale(float mean) { return mean < 1.0f ? 0x1p90f : 0x1p-80f; }

// NVFP4's second-level scales of a row with the largest magnitude `top`: 2688 / top,
// but at most 2^118, so that neither it nor its quotient by a block's scale (2^-9 at
// the least) leaves fp32, and what undoes it.
__device__ __forceinline__ float fp4_row_enc(float top) {
  return top > 0.0f ? fminf(__fdiv_rn(2688.0f, top), 0x1p118f) : 1.0f;
}
__device__ __forceinline__ float fp4_row_dec(float top) {
  return top > 0.0f ? fmaxf(__fdiv_rn(top, 2688.0f), 0x1p-118f) : 1.0f;
}

// Scale code of a block with the largest magnitude a, and the factor onto the E2M1 grid.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_scale(float a, float g_enc, float& mul) {
  if constexpr (FMT == FMT_MX) {
    const int ex = mx_exponent(a);
    mul = pow2f(-ex);
    return (uint32_t)(ex + 127);
  } else {
    const uint32_t sc = cvt_e4m3(__fmul_rn(div6_rn(a), g_enc));
    mul = sc == 0 ? 0.0f : __fdiv_rn(g_enc, e4m3_value(sc));
    return sc;
  }
}

// The 16 values of a unit as they are in memory.
template <int FRONT, bool XBF16>
struct Fp4Raw {
  static constexpr int kWords = (XBF16 ? 2 : 4) * (FRONT == FRONT_SWIGLU ? 2 : 1);
  uint4 q[kWords];
  __device__ __forceinline__ void load(const Fp4Params& p, int64_t at) {
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + at * (XBF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (XBF16 ? 2 : 4); i++) q[i] = __ldg(x + i);
    if constexpr (FRONT == FRONT_SWIGLU) {
      const uint4* y = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x2) + at * (XBF16 ? 2 : 4));
#pragma unroll
      for (int i = 0; i < (XBF16 ? 2 : 4); i++) q[kWords / 2 + i] = __ldg(y + i);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; i++) q[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ static void unpack(const uint4* w, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < (XBF16 ? 2 : 4); i++) {
      const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if constexpr (XBF16) {
          v[8 * i + 2 * j] = __uint_as_float(ws[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
        } else {
          v[4 * i + j] = __uint_as_float(ws[j]);
        }
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[16]) const {
    unpack(q, v);
    if constexpr (FRONT == FRONT_SWIGLU) {
      uint32_t any = 0;  // padding rows hold zeros: SiLU(0) * 0 = 0 without the exponentials
#pragma unroll
      for (int i = 0; i < kWords; i++) any |= q[i].x | q[i].y | q[i].z | q[i].w;
      if (any == 0) return;
      float u[16];
      unpack(q + kWords / 2, u);
#pragma unroll
      for (int i = 0; i < 16; i++) v[i] = __fmul_rn(dev_silu(v[i]), u[i]);
    }
  }
};

// Persistent over rows; the next row's loads are issued before the present
// row's arithmetic, so that both the memory and the issue slots stay busy.  32768 x
// 5120 bf16: MXFP4 66 us (the copy rate), NVFP4 84, behind a norm 107 and 126: 290
// instructions for the 16 elements of each of a warp's lanes keep two thirds of the
// issue slots busy, with the 19 warps an SM that the registers leave.  (Asking for a
// number of resident blocks, even one, had the compiler take more registers: 136.)
template <int FMT, int FRONT, bool XBF16, int NJ>
__global__ void __launch_bounds__(NJ == 1 ? 1024 : 256) fp4_kernel(const Fp4Params p, const int wpr) {
  // [row parity][sum, sum again, largest magnitude][a multiple of eight for each row of the block, 32 in all at most]
  __shared__ __align__(16) float red[2][3][64];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, group = w / wpr, wr = w - group * wpr;
  const int groups = (int)(blockDim.x / (32 * wpr)), bar = 1 + group;
  const int units = (int)(p.k / 16), u0 = wr * 32 + lane, step = 32 * wpr;
  const int chunks = (NJ * wpr + 7) & ~7;
  int64_t end = p.rows_out;
  if (p.count) {
    const int64_t c = (int64_t)__ldg(p.count);
    end = c < end ? c : end;
  }
  const int64_t stride = (int64_t)gridDim.x * groups;
  int64_t r = (int64_t)blockIdx.x * groups + group;
  auto source = [&](int64_t row) -> int64_t {
    if (row >= end) return -1;
    const int64_t src = p.rows ? (int64_t)__ldg(p.rows + row) : row;
    return src < p.x_rows ? src : -1;
  };
  Fp4Raw<FRONT, XBF16> raw[NJ];
  auto fetch = [&](int64_t src) {
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const int u = u0 + step * j;
      if (src >= 0 && u < units) raw[j].load(p, src * p.stride + 16 * u);
      else raw[j].zero();
    }
  };
  fetch(source(r));
  int64_t next = source(r + stride);
  constexpr int kStep = FMT == FMT_NV ? 1 : 2;  // lanes per scale
  const int64_t S = p.k / (16 * kStep);
  for (int par = 0; r < end; r += stride, par ^= 1) {
    float v[NJ][16];
#pragma unroll
    for (int j = 0; j < NJ; j++) raw[j].values(v[j]);
    fetch(next);
    next = source(r + 2 * stride);
    if constexpr (FRONT == FRONT_NORM) {
      auto sumsq = [&](float f, float* buf) {
        float s[NJ];
#pragma unroll
        for (int j = 0; j < NJ; j++) {
          s[j] = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; i++) s[j] = __fmaf_rn(v[j][i] * f, v[j][i] * f, s[j]);
        }
        return row_sum<NJ, FMT == FMT_NV>(s, buf + chunks * group, wr, wpr, bar);
      };
      const float mean = fp4_mean(sumsq(1.0f, red[par][0]), p.k, p.eps);
      float rs;
      if (fp4_mean_in_range(mean)) {
        rs = fp4_rstd(mean);
      } else {
        const float f = fp4_norm_scale(mean);
        rs = f * fp4_rstd(fp4_mean(sumsq(f, red[par][1]), p.k, p.eps * f * f));
      }
#pragma unroll
      for (int j = 0; j < NJ; j++) {
        const int u = u0 + step * j;
        if (u >= units || isinf(rs)) continue;  // r beyond fp32: the row as it is
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float g[8];
          load8<XBF16>(p.gamma, 16 * u + 8 * h, g);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            mul2(v[j][8 * h + i], v[j][8 * h + i + 1], rs, rs);
            mul2(v[j][8 * h + i], v[j][8 * h + i + 1], g[i], g[i + 1]);
          }
        }
      }
    }
    float a[NJ], top = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      a[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i++) a[j] = fmaxf(a[j], fabsf(v[j][i]));
      top = fmaxf(top, a[j]);
    }
    float g_enc = 1.0f;
    if constexpr (FMT == FMT_NV) {
      // with an amax given too, a row that does not exist is one of zeros, as fp4_gather_kernel writes it
      if (p.amax > 0.0f) top = p.rows && (uint32_t)__ldg(p.rows + r) >= (uint64_t)p.x_rows ? 0.0f : p.amax;
      else top = row_max<NJ == 1>(top, red[par][2] + 8 * group, wr, wpr, bar);
      g_enc = fp4_row_enc(top);
      if (u0 == 0) p.row_scale[r] = fp4_row_dec(top);
    } else if (u0 == 0) {
      p.row_scale[r] = 1.0f;
    }
    int64_t e = 0, re = r;
    if (p.rows_expert != p.rows_out) {
      e = r / p.rows_expert;
      re = r % p.rows_expert;
    }
    uint8_t* sf = p.scales + e * tiled_sf_bytes(p.rows_expert, S) + tiled_sf_offset(re, u0 / kStep, S);
    uint8_t* codes = p.codes + r * (p.k / 2) + 8 * u0;
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const bool in = u0 + step * j < units;
      float am = a[j], mul;
      if constexpr (FMT == FMT_MX) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      uint32_t sc = fp4_scale<FMT>(am, g_enc, mul);
      if (in) {
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float* vv = v[j] + 8 * h;
#pragma unroll
          for (int i = 0; i < 8; i += 2) mul2(vv[i], vv[i + 1], mul, mul);
          q[h] = mul == 0.0f ? 0u : cvt_e2m1x8(vv);
        }
        *reinterpret_cast<uint2*>(codes + (int64_t)8 * step * j) = make_uint2(q[0], q[1]);
      } else {
        sc = 0;  // the places of a group of four past the row's last scale
      }
      // four adjacent scales of a row are one word of the tiled layout (512 bytes on: the next four)
      sc |= __shfl_down_sync(0xffffffffu, sc, kStep) << 8;
      sc |= __shfl_down_sync(0xffffffffu, sc, 2 * kStep) << 16;
      if (lane % (4 * kStep) == 0 && in)
        *reinterpret_cast<uint32_t*>(sf + (int64_t)(step / (4 * kStep)) * 512 * j) = sc;
    }
  }
}

// ------------------------------------- rows too long for the registers
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {  // 128 threads
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, m);
    v = MAX ? fmaxf(v, o) : __fadd_rn(v, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return MAX ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]))
             : __fadd_rn(__fadd_rn(red[0], red[1]), __fadd_rn(red[2], red[3]));
}

// One block of 128 threads per row; a thread takes 16 values at a time and reads
// them again (from L1 or L2) for each pass over the row, of which there are up to
// three.  4096 x 28672 bf16 NVFP4 83 us, behind a norm 111, behind a gate 322 (46, 46
// and 82 by bytes): the passes' arithmetic.
template <int FMT, int FRONT, bool XBF16>
__global__ void __launch_bounds__(128) fp4_long_kernel(const Fp4Params p) {
  __shared__ float red[4];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t r = blockIdx.x;
  if (p.count && r >= (int64_t)*p.count) return;
  int64_t src = p.rows ? (int64_t)p.rows[r] : r;
  if (src >= p.x_rows) src = -1;
  const int64_t off = src * p.stride;
  const int units = (int)(p.k / 16), span = (units + 127) & ~127;
  auto value = [&](int u, float rs, float (&v)[16]) {
    if (src < 0 || u >= units) {
#pragma unroll
      for (int i = 0; i < 16; i++) v[i] = 0.0f;
      return;
    }
    fp4_load16<FRONT, XBF16>(p, off + 16 * (int64_t)u, v);
    if constexpr (FRONT == FRONT_NORM) {
      if (isinf(rs)) return;  // r beyond fp32: the row as it is
      float g[8];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        load8<XBF16>(p.gamma, 16 * (int64_t)u + 8 * h, g);
#pragma unroll
        for (int i = 0; i < 8; i++) v[8 * h + i] = __fmul_rn(__fmul_rn(v[8 * h + i], rs), g[i]);
      }
    }
  };
  float rs = 1.0f;
  if constexpr (FRONT == FRONT_NORM) {
    auto sumsq = [&](float f) {
      float s = 0.0f;
      for (int u = threadIdx.x; u < units && src >= 0; u += 128) {
        float v[16];
        fp4_load16<FRONT, XBF16>(p, off + 16 * (int64_t)u, v);
#pragma unroll
        for (int i = 0; i < 16; i++) s = __fmaf_rn(v[i] * f, v[i] * f, s);
      }
      return block_reduce<false>(s, red);
    };
    const float mean = fp4_mean(sumsq(1.0f), p.k, p.eps);
    if (fp4_mean_in_range(mean)) {
      rs = fp4_rstd(mean);
    } else {
      const float f = fp4_norm_scale(mean);
      rs = f * fp4_rstd(fp4_mean(sumsq(f), p.k, p.eps * f * f));
    }
  }
  float g_enc = 1.0f, g_dec = 1.0f;
  if constexpr (FMT == FMT_NV) {
    float top = src < 0 ? 0.0f : p.amax;
    if (!(top > 0.0f)) {
      top = 0.0f;
      for (int u = threadIdx.x; u < units; u += 128) {
        float v[16];
        value(u, rs, v);
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(v[i]));
      }
      top = block_reduce<true>(top, red);
    }
    g_enc = fp4_row_enc(top);
    g_dec = fp4_row_dec(top);
  }
  if (threadIdx.x == 0) p.row_scale[r] = g_dec;
  const int64_t S = p.k / (FMT == FMT_NV ? 16 : 32);
  const int64_t e = r / p.rows_expert, re = r % p.rows_expert;
  uint8_t* sf = p.scales + e * tiled_sf_bytes(p.rows_expert, S);
  for (int u = threadIdx.x; u < span; u += 128) {
    float v[16];
    value(u, rs, v);
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) a = fmaxf(a, fabsf(v[i]));
    if constexpr (FMT == FMT_MX) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    float mul;
    const uint32_t sc = fp4_scale<FMT>(a, g_enc, mul);
    if (u < units) {
      const uint2 q = make_uint2(quant8(v, mul), quant8(v + 8, mul));
      *reinterpret_cast<uint2*>(p.codes + r * (p.k / 2) + 8 * (int64_t)u) = q;
    }
    // scales of the row, and zeros up to the end of its last group of four
    if constexpr (FMT == FMT_NV) {
      if (u < ((units + 3) & ~3)) sf[tiled_sf_offset(re, u, S)] = u < units ? (uint8_t)sc : 0;
    } else {
      if ((u & 1) == 0 && (u >> 1) < (((int)S + 3) & ~3)) sf[tiled_sf_offset(re, u >> 1, S)] = u < units ? (uint8_t)sc : 0;
    }
  }
}

// ------------------------------------------------------ gather of rows
// FP4 rows laid out again by index.  Every row has its own scales, so this is
// what quantizing the gathered rows gives, at a quarter of the bytes read and
// none of the arithmetic for each copy (32768 routed rows of 2048 from 4096
// tokens: 43 us when every copy was quantized).  A block takes 128 rows, a whole
// tile of the scale layout, and a part of their columns.
struct Fp4GatherParams {
  const uint8_t *s_codes, *s_scales;
  const float* s_row;
  uint8_t *d_codes, *d_scales;
  float* d_row;
  const int32_t* rows;
  const int32_t* count;
  int64_t src_rows, dst_rows;
  int32_t pieces, blocks;  // 16-byte pieces of a row's codes; 512-byte scale blocks of a row tile
};

__global__ void __launch_bounds__(256) fp4_gather_kernel(const Fp4GatherParams p) {
  __shared__ int32_t src[128];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t r0 = (int64_t)blockIdx.x * 128;
  int64_t end = p.dst_rows;
  if (p.count) {
    const int64_t c = (int64_t)__ldg(p.count);
    end = c < end ? c : end;
  }
  if (r0 >= end) return;
  const int live = (int)(end - r0 < 128 ? end - r0 : 128);
  for (int i = threadIdx.x; i < 128; i += 256) {
    int32_t s = i < live ? __ldg(p.rows + r0 + i) : -1;
    if (s < 0 || s >= p.src_rows) s = -1;
    src[i] = s;
    if (blockIdx.y == 0 && i < live) p.d_row[r0 + i] = s >= 0 ? __ldg(p.s_row + s) : 1.0f;  // a zero row's factor is 1
  }
  __syncthreads();
  const int parts = (int)gridDim.y, part = (int)blockIdx.y;
  // codes: a warp takes a row's share of pieces, lane by lane
  const int c0 = (int)((int64_t)p.pieces * part / parts), c1 = (int)((int64_t)p.pieces * (part + 1) / parts);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int c = c0 + lane; c < c1; c += 32) {
    for (int i0 = w; i0 < live; i0 += 32) {  // four rows' loads in flight
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int i = i0 + 8 * u;
        const int64_t s = i < live ? src[i] : -1;
        v[u] = s >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.s_codes) + s * p.pieces + c) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < 4; u++)
        if (i0 + 8 * u < live) reinterpret_cast<uint4*>(p.d_codes)[(r0 + i0 + 8 * u) * p.pieces + c] = v[u];
    }
  }
  // scales: 16 bytes of a block are the words of rows q, q + 32, q + 64, q + 96
  const int b0 = (int)((int64_t)p.blocks * part / parts), b1 = (int)((int64_t)p.blocks * (part + 1) / parts);
  for (int64_t j = (int64_t)b0 * 32 + threadIdx.x; j < (int64_t)b1 * 32; j += 256) {
    const int64_t b = j >> 5;
    const int q = (int)(j & 31);
    uint32_t v[4];
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int64_t s = src[q + 32 * g];
      v[g] = s >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(p.s_scales + ((s >> 7) * p.blocks + b) * 512 + (s & 31) * 16 +
                                                              ((s >> 5) & 3) * 4))
                    : 0u;
    }
    uint8_t* to = p.d_scales + ((int64_t)blockIdx.x * p.blocks + b) * 512 + q * 16;
    if (live == 128) {
      *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int g = 0; g < 4; g++)
        if (q + 32 * g < live) *reinterpret_cast<uint32_t*>(to + 4 * g) = v[g];
    }
  }
}

}  // namespace sharq

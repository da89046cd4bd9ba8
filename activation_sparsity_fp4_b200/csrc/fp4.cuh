// fp4.cuh -- rows to microscaled FP4 (one operand a row, no split): MXFP4 and
// NVFP4 codes, tiled scales and the row's second-level scale in one pass.
#pragma once
#include "prep.cuh"
#include "route.cuh"

namespace sharq {

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

// One block of 128 threads per row; a thread takes 16 values at a time.
template <int FMT, int FRONT, bool XBF16>
__global__ void __launch_bounds__(128) fp4_kernel(const Fp4Params p) {
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
    const float s = sumsq(1.0f);
    // squares beyond fp32 (values from about 2^64 / sqrt(k) on): again at 2^-80 of their size, where eps is nothing
    rs = isinf(s) ? __fmul_rn(0x1p-80f, rstd_from_sumsq(sumsq(0x1p-80f), p.k, 0.0f)) : rstd_from_sumsq(s, p.k, p.eps);
  }
  float g_enc = 1.0f, g_dec = 1.0f;
  if constexpr (FMT == FMT_NV) {
    float top = p.amax;
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
    tensor_scales(top, g_enc, g_dec);
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
    uint32_t sc;
    float mul;
    if constexpr (FMT == FMT_MX) {
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      const int ex = mx_exponent(a);
      sc = (uint32_t)(ex + 127);
      mul = pow2f(-ex);
    } else {
      sc = cvt_e4m3(__fmul_rn(div6_rn(a), g_enc));
      const float sv = e4m3_value(sc);
      mul = sv == 0.0f ? 0.0f : __fdiv_rn(g_enc, sv);
    }
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

}  // namespace sharq

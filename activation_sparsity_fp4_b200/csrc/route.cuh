// route.cuh -- mixture-of-experts routing: scores and top-k, the routed-row
// layout, and the weighted sum of the experts' rows.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace sharq {

constexpr int kMaxExperts = 512;
constexpr int kMaxGroups = 32;
constexpr int kMaxTopK = 32;

struct RouteParams {
  const void* logits;
  int64_t t, stride;
  const float* bias;
  int32_t experts, groups, top_groups, group_top, top_k;
  int softmax, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// One warp per token; lane l holds the experts l, l + 32, ... (VPL of them).
template <int VPL, bool XBF16>
__global__ void __launch_bounds__(128) route_kernel(const RouteParams p) {
  extern __shared__ double route_smem[];  // per warp: the experts' selection scores (grouped form)
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const double ninf = -__longlong_as_double(0x7FF0000000000000ll);
  grid_dep_wait();
  grid_dep_launch();
  const int64_t tok = (int64_t)blockIdx.x * 4 + w;
  if (tok >= p.t) return;
  float l[VPL];
  double s[VPL], c[VPL];  // score p, selection value
  double m = ninf;
#pragma unroll
  for (int i = 0; i < VPL; i++) {
    const int e = lane + 32 * i;
    float v = -INFINITY;
    if (e < p.experts) {
      const int64_t at = tok * p.stride + e;
      if constexpr (XBF16) v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at]);
      else v = static_cast<const float*>(p.logits)[at];
    }
    if (!(v > -INFINITY)) v = -INFINITY;  // NaN: not eligible
    l[i] = v;
    m = fmax(m, (double)v);
  }
  if (p.softmax) {
    m = warp_max(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
      s[i] = (double)l[i] == ninf ? 0.0 : ((double)l[i] == m ? 1.0 : exp((double)l[i] - m));
      sum += s[i];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < VPL; i++) s[i] = s[i] / sum;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; i++) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
#pragma unroll
  for (int i = 0; i < VPL; i++) {
    const int e = lane + 32 * i;
    double v = s[i];
    if (p.bias && e < p.experts) v += (double)p.bias[e];
    c[i] = l[i] > -INFINITY && v > ninf ? v : ninf;
  }
  if (p.groups > 1) {
    double* sc = route_smem + w * p.experts;
    const int per = p.experts / p.groups;
#pragma unroll
    for (int i = 0; i < VPL; i++)
      if (lane + 32 * i < p.experts) sc[lane + 32 * i] = c[i];
    __syncwarp();
    double gv = ninf;
    if (lane < p.groups) {
      double a = ninf, b = ninf;
      for (int j = 0; j < per; j++) {
        const double v = sc[lane * per + j];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      gv = p.group_top == 2 && b > ninf ? a + b : a;
    }
    int before = 0;  // groups that come before this lane's
    for (int g = 0; g < p.groups; g++) {
      const double o = __shfl_sync(0xffffffffu, gv, g);
      before += o > gv || (o == gv && g < lane);
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, lane < p.groups && before < p.top_groups);
#pragma unroll
    for (int i = 0; i < VPL; i++) {
      const int e = lane + 32 * i;
      if (e < p.experts && !((kept >> (e / per)) & 1u)) c[i] = ninf;
    }
  }
  if (!p.bias) {
#pragma unroll
    for (int i = 0; i < VPL; i++)
      if (c[i] > ninf) c[i] = (double)l[i];
  }
  double sum = 0.0, mine = 0.0;
  int my_id = -1;
  for (int j = 0; j < p.top_k; j++) {
    double best = ninf, bs = 0.0;
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < VPL; i++)
      if (c[i] > best) {
        best = c[i];
        bs = s[i];
        be = lane + 32 * i;
      }
#pragma unroll
    for (int msk = 16; msk >= 1; msk >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, msk), os = __shfl_xor_sync(0xffffffffu, bs, msk);
      const int oe = __shfl_xor_sync(0xffffffffu, be, msk);
      if (ob > best || (ob == best && oe < be)) {
        best = ob;
        bs = os;
        be = oe;
      }
    }
    if (be == 0x7FFFFFFF) break;  // no eligible expert left (the same in every lane)
#pragma unroll
    for (int i = 0; i < VPL; i++)
      if (lane + 32 * i == be) c[i] = ninf;
    sum += bs;
    if (lane == j) {
      my_id = be;
      mine = bs;
    }
  }
  if (lane < p.top_k) {
    double wv = mine;
    if (p.renormalize) wv = sum > 0.0 ? wv / sum : 0.0;
    p.ids[tok * p.top_k + lane] = my_id;
    p.weights[tok * p.top_k + lane] = (float)(wv * (double)p.scale);
  }
}

// ------------------------------------------------------------ row layout
// A stable counting sort by one cluster of CTAs: each CTA takes a contiguous
// share of the ids, each warp a contiguous share of that.  Pass 1 counts every
// warp's ids per expert (a warp's equal ids found by match, so no atomics and
// one order only); the counts are prefixed over the warps of a CTA, then over
// the cluster's CTAs through distributed shared memory, and the experts'
// padded sizes give the offsets.  Pass 2 walks the same ids again and hands
// out the rows.
struct RowsParams {
  const int32_t* ids;
  int64_t n;  // t * top_k
  int32_t top_k, experts;
  int32_t* rows;
  int64_t capacity;
  int32_t* offsets;
  int32_t* slots;
};
constexpr int kRowsWarps = 32;

__global__ void __launch_bounds__(kRowsWarps * 32) route_rows_kernel(const RowsParams p) {
  extern __shared__ int32_t rows_smem[];
  const int E = p.experts;
  int32_t* hist = rows_smem;                // [warp][E]
  int32_t* total = hist + kRowsWarps * E;   // this CTA's ids per expert
  int32_t* count = total + E;               // the cluster's
  int32_t* off = count + E;                 // E + 1 padded offsets
  __shared__ int32_t wsum[kRowsWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster
  grid_dep_wait();
  grid_dep_launch();
  const int64_t parts = (int64_t)ctas * kRowsWarps, part = (int64_t)rank * kRowsWarps + w;
  const int64_t lo = p.n * part / parts, hi = p.n * (part + 1) / parts;
  int32_t* hw = hist + w * E;
  for (int e = lane; e < E; e += 32) hw[e] = 0;
  __syncwarp();
  for (int64_t i0 = lo; i0 < hi; i0 += 32) {
    const int64_t i = i0 + lane;
    int e = i < hi ? p.ids[i] : -1;
    if (e < 0 || e >= E) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) hw[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {  // exclusive prefix over the warps
    int run = 0;
    for (int q = 0; q < kRowsWarps; q++) {
      const int v = hist[q * E + e];
      hist[q * E + e] = run;
      run += v;
    }
    total[e] = run;
  }
  __syncthreads();
  cluster_sync_all();
  int padded = 0;
  if (threadIdx.x < (unsigned)E) {  // E <= 512 threads
    const int e = threadIdx.x;
    int all = 0, before = 0;
    for (int r = 0; r < ctas; r++) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_u32(smem_u32(total + e), (uint32_t)r)) : "memory");
      if (r < rank) before += v;
      all += v;
    }
    count[e] = all;
    padded = (all + 127) / 128 * 128;
    hist[e] += before;  // warp 0's prefix; the other warps' below
    for (int q = 1; q < kRowsWarps; q++) hist[q * E + e] += before;
  }
  // inclusive scan of the padded sizes over the block
  int run = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, d);
    if (lane >= d) run += v;
  }
  if (lane == 31) wsum[w] = run;
  __syncthreads();
  int base = 0;
  for (int q = 0; q < w; q++) base += wsum[q];
  if (threadIdx.x < (unsigned)E) off[threadIdx.x + 1] = base + run;
  if (threadIdx.x == 0) off[0] = 0;
  __syncthreads();
  cluster_sync_all();  // every CTA has read the others' totals: they may exit from here on
  if (rank == 0)
    for (int e = threadIdx.x; e <= E; e += blockDim.x) p.offsets[e] = off[e];
  for (int64_t i0 = lo; i0 < hi; i0 += 32) {
    const int64_t i = i0 + lane;
    int e = i < hi ? p.ids[i] : -1;
    if (e < 0 || e >= E) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    int slot = -1;
    if (e >= 0) slot = off[e] + hw[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) hw[e] += __popc(same);
    __syncwarp();
    if (i < hi) {
      p.slots[i] = slot;
      if (slot >= 0) p.rows[slot] = (int32_t)(i / p.top_k);
    }
  }
  // padding rows of the experts, and the rows behind the last one
  for (int e = (int)part; e < E; e += (int)parts)
    for (int r = off[e] + count[e] + lane; r < off[e + 1]; r += 32) p.rows[r] = -1;
  for (int64_t r = off[E] + part * 32 + lane; r < p.capacity; r += parts * 32) p.rows[r] = -1;
}

// ---------------------------------------------------------------- combine
struct CombineParams {
  const void* y;
  int64_t y_rows, n;
  const int32_t* slots;
  const float* weights;
  int64_t t;
  int32_t top_k;
  const void* add;
  void* out;
};

// 8 consecutive values of a row as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t ws[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = __uint_as_float(ws[j] << 16);
      v[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// One thread per 8 columns of a token.
template <bool YBF16, bool OBF16>
__global__ void __launch_bounds__(128) combine_kernel(const CombineParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t per = p.n / 8;
  const int64_t g = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (g >= p.t * per) return;
  const int64_t tok = g / per, col = (g % per) * 8;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (p.add) load8<YBF16>(p.add, tok * p.n + col, acc);
  for (int j = 0; j < p.top_k; j++) {
    const int64_t slot = p.slots[tok * p.top_k + j];
    if (slot < 0 || slot >= p.y_rows) continue;
    const float wv = p.weights[tok * p.top_k + j];
    float v[8];
    load8<YBF16>(p.y, slot * p.n + col, v);
#pragma unroll
    for (int i = 0; i < 8; i++) acc[i] = __fmaf_rn(wv, v[i], acc[i]);
  }
  store8<OBF16>(p.out, tok * p.n + col, acc);
}

}  // namespace sharq

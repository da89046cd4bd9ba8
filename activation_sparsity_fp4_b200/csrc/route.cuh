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
  int32_t smem_doubles;     // shared memory of a warp (grouped form)
  int32_t lanes_per_group;  // a power of two
  uint32_t per_magic;       // ceil(2^32 / (experts / groups)): e / per = umulhi(e, per_magic) for e <= 512; 0: per = 1
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

// Scores, selection and weights of one token in 64 bits, by one warp; lane l holds the experts l, l + 32, ....
template <int VPL, bool XBF16>
__device__ __noinline__ void route_exact(const RouteParams& p, int64_t tok, double* sc /* experts, grouped form */) {
  const int lane = threadIdx.x & 31;
  const double ninf = -__longlong_as_double(0x7FF0000000000000ll);
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
    const int per = p.experts / p.groups;
#pragma unroll
    for (int i = 0; i < VPL; i++)
      if (lane + 32 * i < p.experts) sc[lane + 32 * i] = c[i];
    __syncwarp();
    const int lpg = p.lanes_per_group, g = lane / lpg, sub = lane & (lpg - 1);
    double a = ninf, b = ninf;  // the group's two largest
    if (g < p.groups)
      for (int j = sub; j < per; j += lpg) {
        const double v = sc[g * per + j];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
    for (int d = 1; d < lpg; d <<= 1) {
      const double oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    const double gv = p.group_top == 2 && b > ninf ? a + b : a;
    int before = 0;  // groups that come before this lane's
    for (int o = 0; o < p.groups; o++) {
      const double ov = __shfl_sync(0xffffffffu, gv, o * lpg);
      before += ov > gv || (ov == gv && o < g);
    }
    const uint32_t kept =
        __reduce_or_sync(0xffffffffu, g < p.groups && sub == 0 && before < p.top_groups ? 1u << g : 0u);
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
  // ordered bits of the values, 0 for none
  uint64_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i++) {
    const uint64_t u = (uint64_t)__double_as_longlong(c[i] + 0.0);
    key[i] = c[i] > ninf ? u ^ ((u >> 63) ? ~0ull : 1ull << 63) : 0;
  }
  double sum = 0.0, mine = 0.0;
  int my_id = -1;
  for (int j = 0; j < p.top_k; j++) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < VPL; i++) best = key[i] > best ? key[i] : best;
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const uint64_t top = (uint64_t)hi << 32 | lo;
    if (top == 0) break;  // no eligible expert left (the same in every lane)
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; i--)
      if (key[i] == top) e = (uint32_t)(lane + 32 * i);
    e = __reduce_min_sync(0xffffffffu, e);
    double bs = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; i++)
      if ((uint32_t)(lane + 32 * i) == e) {
        key[i] = 0;
        bs = s[i];
      }
    bs = __shfl_sync(0xffffffffu, bs, (int)(e & 31u));
    sum += bs;
    if (lane == j) {
      my_id = (int)e;
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

// Order-preserving bits of a float (0 stands for "not eligible": no value but a NaN maps to it).
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and 0 are one value
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered_bits(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Sorts N values (a power of two) in descending order by Batcher's odd-even merges.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; i++)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = a > b ? a : b;
            v[i + j + k] = a > b ? b : a;
          }
}

// One warp per token.  Scores are formed in fp32, ranked by redux.sync on their
// ordered bits, and the ranking is taken where it is certain: neighbours that
// decide (the top_k and the one after, the groups on either side of the border)
// further apart than fp32's error, or equal in all that makes them.  Places taken
// that are too close to each other are put in order in 64 bits, a lane each; a
// token where it is open what is taken is ranked again in 64 bits as a whole.
// Without a bias the logits themselves are ranked, which is exact.
//
// Error of a score made for ranking: __expf(x) is within 2 + 1.2 |x| units of
// 2^-23; of that e^x a sigmoid 1 / (1 + e^-l) = s passes on the part 1 - s and adds
// 1 + 4 units of 2^-24; the softmax adds at most 16 + 5 for its sum, what the sum's
// own exponentials are off by (their mean, under 2^-20) and 3 more, 2^-19 in all;
// the bias 2^-24 of c.  The weights are formed in fp32, the type they are returned in (expf,
// their sum, the quotient): off by about 5e-8 where 64 bits rounded once are off by half of that.
//
// Bound by ALU issue (the lanes' sort, 19 exchanges at 256 experts, and top_k + 1
// rounds): 4096 tokens x 128 bf16 4.4 us, 16384 x 256 fp32 12.4 us, with scores, a
// bias and 8 groups 28 to 35 us, as many tokens go to 64 bits (all of them: 55 us);
// one token 2.2 us.
template <int VPL, bool XBF16>
__global__ void __launch_bounds__(128, VPL == 16 ? 5 : 10) route_kernel(const RouteParams p) {
  extern __shared__ double route_smem[];  // per warp: the experts' selection values (grouped form)
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t tok = (int64_t)blockIdx.x * 4 + w;
  if (tok >= p.t) return;
  const int64_t row = tok * p.stride;
  auto logit = [&](int e) {
    if constexpr (XBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[row + e]);
    else return static_cast<const float*>(p.logits)[row + e];
  };
  const bool scores = p.bias != nullptr || p.groups > 1;  // whether the scores take part in the selection
  float l[VPL], c[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; i++) {
    const int e = lane + 32 * i;
    l[i] = e < p.experts ? logit(e) : -INFINITY;
    m = fmaxf(m, l[i]);  // a NaN is passed over
  }
  float sum = 1.0f;
  if (p.softmax) {
    m = from_ordered_bits(__reduce_max_sync(0xffffffffu, ordered_bits(m)));
    if (scores || !p.renormalize) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; i++) {
        // not renormalized, the weights are divided by this sum: of the same terms as theirs
        const float x = l[i] - m;
        c[i] = l[i] == m ? 1.0f : (l[i] > -INFINITY ? (p.renormalize ? __expf(x) : expf(x)) : 0.0f);
        sum += c[i];
      }
#pragma unroll
      for (int msk = 16; msk >= 1; msk >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, msk);
    }
  }
  const float scale_p = p.softmax ? 1.0f / sum : 1.0f;
  auto score = [&](float v) -> float {
    if (p.softmax) return (v == m ? 1.0f : expf(v - m)) * scale_p;
    return 1.0f / (1.0f + expf(-v));
  };
  // no score, fast or not, is further off than this: s (1 - s) (2 + 1.2 |l|) < 0.56 and e^x (2 + 1.2 |x|) <= 2
  const float off = p.softmax ? scale_p * (0x1p-22f + 0x1p-19f) : 0.56f * 0x1p-23f + 0x1p-21f;
  const float exact_off = p.softmax ? off : 0x1p-22f;  // of score(): expf 2 units of 2^-23, of which s (1 - s) <= 1/4 pass
  uint32_t key[VPL];
  bool unsure = false;
#pragma unroll
  for (int i = 0; i < VPL; i++) key[i] = l[i] > -INFINITY ? ordered_bits(l[i]) : 0u;
  if (scores) {
    uint32_t kept = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
      const int e = lane + 32 * i;
      const float s = p.softmax ? c[i] * scale_p : __fdividef(1.0f, 1.0f + __expf(-l[i]));
      c[i] = key[i] ? s + (p.bias ? __ldg(p.bias + e) : 0.0f) : -INFINITY;
      if (!(c[i] > -INFINITY)) {
        c[i] = -INFINITY;
        key[i] = 0;
      }
    }
    if (p.groups > 1) {
      // lanes [g lpg, (g + 1) lpg) find group g's two largest; lpg floats between
      // the groups in shared memory keep their reads on different banks
      const int lpg = p.lanes_per_group, per = p.experts / p.groups, g = lane / lpg, sub = lane & (lpg - 1);
      // one expert a group and no bias: the groups' best logits rank them as their scores do
      const bool by_logit = p.group_top == 1 && !p.bias;
      float* sc = reinterpret_cast<float*>(route_smem + (size_t)w * p.smem_doubles);
      auto group_of = [&](int e) { return p.per_magic ? (int)__umulhi((uint32_t)e, p.per_magic) : e; };
#pragma unroll
      for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        if (e < p.experts) sc[e + lpg * group_of(e)] = by_logit ? (key[i] ? l[i] : -INFINITY) : c[i];
      }
      __syncwarp();
      float a = -INFINITY, b = -INFINITY;
      if (g < p.groups) {
        const float* sg = sc + g * (per + lpg);
        for (int j = sub; j < per; j += lpg) {
          const float v = sg[j];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
      }
      for (int d = 1; d < lpg; d <<= 1) {
        const float oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
      }
      const float gv = p.group_top == 2 && b > -INFINITY ? a + b : a;
      int before = 0;  // groups ahead of this lane's
      for (int o = 0; o < p.groups; o++) {
        const float ov = __shfl_sync(0xffffffffu, gv, o * lpg);
        before += ov > gv || (ov == gv && o < g);
      }
      // The border.  A group's value is off by its scores' errors and by the rounding
      // of its terms (each c, and their sum), which may be far larger than it: two of
      // opposite signs cancel.  It is taken where the least that a group inside may
      // be worth is above the most that one outside may; a sum beyond fp32 may be
      // anything.  Without a bias a score is the whole term, off by 110 of 2^-23 of
      // itself at most (|x| to 88).
      const bool head = g < p.groups && sub == 0, inside = before < p.top_groups;
      float err = 0.0f;
      if (!by_logit) {
        const float terms = a > -INFINITY ? fabsf(a) + (p.group_top == 2 && b > -INFINITY ? fabsf(b) : 0.0f) : 0.0f;
        err = (p.bias ? 2.0f * off : fminf(2.0f * off, 0x1p-15f * terms)) + 0x1p-22f * terms + 0x1p-120f;
      }
      const float in = from_ordered_bits(__reduce_min_sync(
          0xffffffffu, head && inside ? ordered_bits(err < INFINITY ? gv - err : -INFINITY) : 0xFFFFFFFFu));
      const float out = from_ordered_bits(__reduce_max_sync(
          0xffffffffu, head && !inside ? ordered_bits(err < INFINITY ? gv + err : INFINITY) : 0u));
      if (p.top_groups < p.groups && out > -INFINITY) {
        if (!by_logit)
          unsure = !(in > out);
        else if (in < INFINITY)  // except where even 64 bits may round the scores of different logits to one value
          unsure = in != out && (in - out < 0x1p-24f || (p.softmax ? m - in > 700.0f : in > 15.0f || in < -700.0f));
      }
      uint32_t mine = head && before < p.top_groups ? 1u << g : 0u;
      kept = __reduce_or_sync(0xffffffffu, mine);
#pragma unroll
      for (int i = 0; i < VPL; i++)
        if (!((kept >> (group_of(lane + 32 * i) & 31)) & 1u)) key[i] = 0;
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < VPL; i++)
        if (key[i]) key[i] = ordered_bits(c[i]);
    }
  }
  // The top_k keys in order, and with a bias the one after them.  First on words
  // of the key's upper 23 bits and the expert (lower experts larger): all words
  // differ, each lane keeps its own sorted, and a round takes the largest head.
  int my_id = -1;
  int after_id = -1;  // lane top_k - 1: the one after
  const int rounds = p.top_k + 1;
  uint32_t last = 0, mine = 0;  // the last word taken; lane j's, of round j
  bool close = false;           // neighbours that the upper bits do not tell apart
  {
    uint32_t word[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i++)
      word[i] = key[i] ? (key[i] & 0xFFFFFE00u) | (511u - (uint32_t)(lane + 32 * i)) : 0u;
    sort_desc<VPL>(word);
    for (int j = 0; j < rounds; j++) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, word[0]);
      if (top == 0) break;
      if (word[0] == top) {
#pragma unroll
        for (int i = 0; i + 1 < VPL; i++) word[i] = word[i + 1];
        word[VPL - 1] = 0;
      }
      // bf16 logits have 16 bits: equal here is equal, and the lower expert is first
      if ((!XBF16 || p.bias) && j > 0 && ((last ^ top) >> 9) == 0) close = true;
      last = top;
      if (lane == j) mine = top;
    }
    const uint32_t next = p.top_k < 32 ? __shfl_sync(0xffffffffu, mine, p.top_k & 31) : last;
    if (lane < p.top_k && mine) my_id = 511 - (int)(mine & 511u);
    // with all 32 places taken the last word is the one after only if it was not the last place's own
    if (next && next != __shfl_sync(0xffffffffu, mine, p.top_k - 1)) after_id = 511 - (int)(next & 511u);
  }
  if (close) {  // the same on whole keys
    my_id = after_id = -1;
    for (int j = 0; j < rounds; j++) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < VPL; i++) best = key[i] > best ? key[i] : best;
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      if (top == 0) break;
      uint32_t e = 0xFFFFFFFFu;
#pragma unroll
      for (int i = VPL - 1; i >= 0; i--)
        if (key[i] == top) e = (uint32_t)(lane + 32 * i);
      e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
      for (int i = 0; i < VPL; i++)
        if ((uint32_t)(lane + 32 * i) == e) key[i] = 0;
      if (j == p.top_k) after_id = (int)e;
      else if (lane == j) my_id = (int)e;
    }
  }
  const float ml = my_id >= 0 ? logit(my_id) : -INFINITY;
  float wv = my_id >= 0 ? score(ml) : 0.0f;
  if (p.bias) {
    // Every place against the next one, by these scores (each within exact_off), and
    // the last one against the one after.  For an expert z behind that one only the
    // ranking's scores (within off) say that it is no larger: the two of z and of the
    // one after more.  And that no place taken is worth less than the last holds by
    // these scores only while every place is certainly above the next; where one is not
    // (order), it holds by the ranking's, of that place and of the last: two more.  The
    // slack is the rounding of c, 2^-24 of it for each score in question.
    const float mb = my_id >= 0 ? __ldg(p.bias + my_id) : 0.0f, mc = wv + mb;
    float nl = __shfl_down_sync(0xffffffffu, ml, 1), nb = __shfl_down_sync(0xffffffffu, mb, 1);
    float nw = __shfl_down_sync(0xffffffffu, wv, 1);
    int ni = __shfl_down_sync(0xffffffffu, my_id, 1);
    const bool border = lane == p.top_k - 1;
    if (border) {
      ni = after_id;
      if (ni >= 0) {
        nl = logit(ni);
        nb = __ldg(p.bias + ni);
        nw = score(nl);
      }
    }
    bool order = false, near = false;
    if (my_id >= 0 && ni >= 0 && lane < p.top_k) {
      const bool same = ml == nl && mb == nb;
      const float gap = mc - (nw + nb), slack = 0x1p-22f * fabsf(mc);
      if (!same && mc < INFINITY) {
        if (border || p.softmax) unsure = unsure || gap <= 2.0f * (exact_off + off) + 1.25f * slack;
        else order = gap <= 2.0f * exact_off + slack;
        near = border && gap <= 2.0f * exact_off + 4.0f * off + 2.0f * slack;
      }
    }
    if (__any_sync(0xffffffffu, order) && __any_sync(0xffffffffu, near)) unsure = true;
    if (__any_sync(0xffffffffu, order) && !__any_sync(0xffffffffu, unsure)) {
      // the right experts, perhaps in the wrong order: a lane's own in 64 bits (sigmoid), and its rank
      const double cd = my_id >= 0 ? 1.0 / (1.0 + exp(-(double)ml)) + (double)mb : -INFINITY;
      int rank = 0, from = lane;
      for (int i = 0; i < p.top_k; i++) {
        const double oc = __shfl_sync(0xffffffffu, cd, i);
        const int oi = __shfl_sync(0xffffffffu, my_id, i);
        rank += oi >= 0 && (oc > cd || (oc == cd && oi < my_id));
      }
      for (int i = 0; i < p.top_k; i++)
        if (__shfl_sync(0xffffffffu, my_id >= 0 ? rank : -1, i) == lane) from = i;
      my_id = __shfl_sync(0xffffffffu, my_id, from);
      wv = __shfl_sync(0xffffffffu, wv, from);
    }
  }
  float total = wv;
  if (p.renormalize) {
#pragma unroll
    for (int msk = 16; msk >= 1; msk >>= 1) total += __shfl_xor_sync(0xffffffffu, total, msk);
    // so small a sum has lost bits to underflow
    if (total < 0x1p-90f && __any_sync(0xffffffffu, my_id >= 0)) unsure = true;
  }
  if (__any_sync(0xffffffffu, unsure)) {
    route_exact<VPL, XBF16>(p, tok, route_smem + (size_t)w * p.smem_doubles);
    return;
  }
  if (lane < p.top_k) {
    if (p.renormalize) wv = my_id >= 0 ? wv / total : 0.0f;
    p.ids[tok * p.top_k + lane] = my_id;
    p.weights[tok * p.top_k + lane] = wv * p.scale;
  }
}

// ------------------------------------------------------------ row layout
// A stable counting sort by one cluster of CTAs: each CTA takes a contiguous
// share of the ids, each warp a contiguous share of that.  Pass 1 counts every
// warp's ids per expert; the counts are prefixed over the warps of a CTA, then over
// the cluster's CTAs through distributed shared memory, and the experts'
// padded sizes give the offsets.  Pass 2 walks the same ids again and hands
// out the rows.  One launch and no workspace: 104 ids 4.8 us, 131072 ids with 256
// experts 12.9 us by 16 CTAs (20 us by 8), bound by their scattered row stores.
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

constexpr int kRowsBits = 10;  // an expert below kMaxExperts, or -1
static_assert(kMaxExperts <= 1 << (kRowsBits - 1), "the last bit tells -1 apart");
constexpr int kRowsBatch = 8;  // steps of a warp whose ids are loaded together

__global__ void __launch_bounds__(kRowsWarps * 32) route_rows_kernel(const RowsParams p) {
  extern __shared__ int32_t rows_smem[];
  const int E = p.experts;
  int32_t* hist = rows_smem;               // [warp][E]
  int32_t* total = hist + kRowsWarps * E;  // this CTA's ids per expert
  int32_t* count = total + E;              // the cluster's
  int32_t* base = count + E;               // first row of this CTA's
  int32_t* off = base + E;                 // E + 1 padded offsets
  __shared__ int32_t wsum[kRowsWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster
  int32_t* hw = hist + w * E;
  for (int e = lane; e < E; e += 32) hw[e] = 0;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t parts = (int64_t)ctas * kRowsWarps, part = (int64_t)rank * kRowsWarps + w;
  // shares in whole steps of 32 ids
  const int64_t steps = (p.n + 31) / 32, lo = steps * part / parts * 32, hi_ = steps * (part + 1) / parts * 32;
  const int64_t hi = hi_ < p.n ? hi_ : p.n;
  // the ids of kRowsBatch steps from i0 on: -1 for none
  auto load = [&](int64_t i0, int (&e)[kRowsBatch]) {
#pragma unroll
    for (int b = 0; b < kRowsBatch; b++) {
      const int64_t i = i0 + 32 * b + lane;
      e[b] = i < hi ? __ldg(p.ids + i) : -1;
    }
#pragma unroll
    for (int b = 0; b < kRowsBatch; b++)
      if (e[b] < 0 || e[b] >= E) e[b] = -1;
  };
  __syncwarp();
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kRowsBatch) {
    int ids[kRowsBatch];
    load(i0, ids);
#pragma unroll
    for (int b = 0; b < kRowsBatch; b++)
      if (ids[b] >= 0) atomicAdd(hw + ids[b], 1);  // counts alone: their order changes nothing
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {  // exclusive prefix over the warps
    int run = 0;
    for (int q0 = 0; q0 < kRowsWarps; q0 += 8) {
      int v[8];
#pragma unroll
      for (int q = 0; q < 8; q++) v[q] = hist[(q0 + q) * E + e];
#pragma unroll
      for (int q = 0; q < 8; q++) {
        hist[(q0 + q) * E + e] = run;
        run += v[q];
      }
    }
    total[e] = run;
  }
  __syncthreads();
  cluster_sync_all();
  int padded = 0, before = 0;
  if (threadIdx.x < (unsigned)E) {  // E <= 512 threads
    const int e = threadIdx.x;
    int all = 0;
    for (int r = 0; r < ctas; r++) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_u32(smem_u32(total + e), (uint32_t)r)) : "memory");
      if (r < rank) before += v;
      all += v;
    }
    count[e] = all;
    padded = (all + 127) / 128 * 128;
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
  // what the warps before this one add up to
  int ahead = lane < w ? wsum[lane] : 0;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, m);
  if (threadIdx.x < (unsigned)E) {
    off[threadIdx.x + 1] = ahead + run;
    base[threadIdx.x] = ahead + run - padded + before;
  }
  if (threadIdx.x == 0) off[0] = 0;
  __syncthreads();
  cluster_sync_all();  // every CTA has read the others' totals: they may exit from here on
  if (rank == 0)
    for (int e = threadIdx.x; e <= E; e += blockDim.x) p.offsets[e] = off[e];
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kRowsBatch) {
    int ids[kRowsBatch];
    load(i0, ids);
#pragma unroll
    for (int b = 0; b < kRowsBatch; b++) {
      const int64_t i = i0 + 32 * b + lane;
      if (i0 + 32 * b >= hi) break;
      const int e = ids[b];
      // lanes of the same expert, one ballot a bit (match.any takes a turn for every
      // expert in the warp: 300 cycles a step)
      uint32_t same = 0xFFFFFFFFu;
#pragma unroll
      for (int bit = 0; bit < kRowsBits; bit++) {
        const uint32_t on = __ballot_sync(0xffffffffu, (e >> bit) & 1);
        same &= (e >> bit) & 1 ? on : ~on;
      }
      int at = -1;
      if (e >= 0) at = base[e] + hw[e] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (e >= 0 && lane == __ffs(same) - 1) hw[e] += __popc(same);
      __syncwarp();
      if (i < hi) {
        p.slots[i] = at;
        if (at >= 0) p.rows[at] = (int32_t)((uint32_t)i / (uint32_t)p.top_k);
      }
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

// One thread per 8 columns of a token; the loads of up to eight places (bf16; four in
// fp32) are on their way before the first is added.  Bound by DRAM: 4096 tokens x 8 places x
// 2048 bf16 columns onto a residual, 168 MB in 31.3 us (5.4 TB/s).
template <bool YBF16, bool OBF16>
__global__ void __launch_bounds__(128) combine_kernel(const CombineParams p) {
  constexpr int kAhead = YBF16 ? 8 : 4, kWords = YBF16 ? 1 : 2;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t per = p.n / 8;
  const int64_t g = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (g >= p.t * per) return;
  const int64_t tok = g / per, col = (g % per) * 8;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (p.add) load8<YBF16>(p.add, tok * p.n + col, acc);
  const int32_t* slots = p.slots + tok * p.top_k;
  const float* weights = p.weights + tok * p.top_k;
  for (int j0 = 0; j0 < p.top_k; j0 += kAhead) {
    uint4 raw[kAhead][kWords];
    bool on[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const int64_t slot = j0 + j < p.top_k ? __ldg(slots + j0 + j) : -1;
      on[j] = slot >= 0 && slot < p.y_rows;
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.y) +
                                                         ((on[j] ? slot : 0) * p.n + col) * (YBF16 ? 2 : 4));
      if (on[j])
#pragma unroll
        for (int q = 0; q < kWords; q++) raw[j][q] = __ldg(from + q);
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      if (!on[j]) continue;
      const float wv = __ldg(weights + j0 + j);
      float v[8];
      load8<YBF16>(raw[j], 0, v);
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] = __fmaf_rn(wv, v[i], acc[i]);
    }
  }
  store8<OBF16>(p.out, tok * p.n + col, acc);
}

}  // namespace sharq

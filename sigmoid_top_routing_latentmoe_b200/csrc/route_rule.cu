// Routing of given logits with the experts in groups, and its gradient.
//
//   s = sigmoid(l) or softmax(l) over all experts;  key = s + b
//   group score = the largest key of the group, or the sum of its two largest
//   T = the top-k keys among the experts of the topk_groups best groups
//   w_i = scale * s_i / max(sum_T s, 1e-9)   (renormalise), or scale * s_i
//
// Ties go to the lower group and the lower expert; a key that is NaN ranks
// with -inf, so that every row has k distinct experts.  b only selects.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace lmoe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kMinSum = 1e-9f;  // the least sum that weights are divided by
constexpr int kWarps = 4;

__device__ __forceinline__ float sigmoid_f(float l) { return 1.0f / (1.0f + expf(-l)); }

// Order-preserving code of a key, above 0 for every key: -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t key_code(float f) {
  if (isnan(f)) f = -INFINITY;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
// Bitonic sort of 32 codes across the warp, the largest in lane 0.
__device__ __forceinline__ uint32_t warp_sort_desc(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const uint32_t pv = __shfl_xor_sync(kAll, v, stride);
      const bool desc = (lane & size) == 0 || size == 32;
      v = ((lane & stride) == 0) == desc ? max(v, pv) : min(v, pv);
    }
  }
  return v;
}

// Groups of experts in shared memory, per warp: the keys (a padding of `pad`
// floats after each group keeps the lanes that share a group's scan on
// different banks), the groups' codes, and a bit per kept group.
struct Groups {
  int n, kept, size, lanes, top2;  // lanes: how many lanes scan one group (a power of two)
  float inv_size;
  __host__ __device__ int key_words() const { return n * (size + lanes); }
  __host__ __device__ int words() const { return key_words() + n + (n + 31) / 32; }
};
// Group of expert e: (e + 1/2) / size lies at least 1 / (2 size) from a whole
// number, the rounding of the product below 1e-3 / size (e < 4096).
__device__ __forceinline__ int group_of(const Groups& g, int e) {
  return (int)(((float)e + 0.5f) * g.inv_size);
}

// Marks the topk_groups best groups in the warp's bits.
template <int VPL>
__device__ __forceinline__ const uint32_t* keep_groups(const Groups& g, const float (&key)[VPL],
                                                       int R, float* sm) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    if (e < R) sm[e + group_of(g, e) * g.lanes] = key[j];
  }
  uint32_t* code = reinterpret_cast<uint32_t*>(sm) + g.key_words();
  uint32_t* bits = code + g.n;
  __syncwarp();
  const int per = 32 / g.lanes, sub = lane & (g.lanes - 1);
  for (int g0 = 0; g0 < g.n; g0 += per) {
    const int gi = g0 + lane / g.lanes;
    float a = -INFINITY, b = -INFINITY;  // the two largest keys
    if (gi < g.n)
      for (int i = sub; i < g.size; i += g.lanes) {
        float v = sm[gi * (g.size + g.lanes) + i];
        if (isnan(v)) v = -INFINITY;
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    for (int off = g.lanes >> 1; off > 0; off >>= 1) {
      const float oa = __shfl_xor_sync(kAll, a, off), ob = __shfl_xor_sync(kAll, b, off);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    if (gi < g.n && sub == 0) code[gi] = key_code(g.top2 && g.size > 1 ? a + b : a);
  }
  __syncwarp();
  for (int g0 = 0; g0 < g.n; g0 += 32) {
    const int gi = g0 + lane;
    int rank = g.kept;
    if (gi < g.n) {
      const uint32_t c = code[gi];
      rank = 0;
      for (int o = 0; o < g.n; ++o) rank += code[o] > c || (code[o] == c && o < gi);
    }
    const uint32_t m = __ballot_sync(kAll, rank < g.kept);
    if (lane == 0) bits[g0 >> 5] = m;
  }
  __syncwarp();
  return bits;
}

// One warp per token; expert j * 32 + lane is value j of the lane.
// k <= 32 of many experts: the k-th largest of the 32 lane maxima bounds the
// k-th largest key from below, so only the keys at or above it (a few dozen)
// go into the k rounds of selection, two per lane.  Clustered keys (more than
// 64 above the bound) and k > 32 take the rounds over every key.
template <int VPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kWarps) route_rule_kernel(
    const float* __restrict__ logits, int64_t ld, const float* __restrict__ bias, int64_t n, int R,
    int k, Groups g, int renormalise, float scale, int32_t* __restrict__ ids,
    float* __restrict__ probs) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint32_t cand_code[kWarps][64];
  __shared__ int cand_e[kWarps][64];
  extern __shared__ float sm_keys[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t >= n) return;
  const float* lr = logits + t * ld;
  float key[VPL];
  float top = 0.0f, inv = 0.0f;  // softmax: the largest logit, 1 / sum of the exponentials
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    key[j] = e < R ? lr[e] : -INFINITY;
  }
  if (SOFTMAX) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) top = fmaxf(top, key[j]);
    top = warp_max(top);
    if (top == -INFINITY) top = 0.0f;  // no expert is open: every score is 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      key[j] = expf(key[j] - top);
      sum += key[j];
    }
    sum = warp_sum(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    const float s = SOFTMAX ? key[j] * inv : sigmoid_f(key[j]);
    key[j] = s + (bias != nullptr && e < R ? bias[e] : 0.0f);
  }
  const uint32_t* bits = nullptr;
  if (g.kept < g.n) bits = keep_groups<VPL>(g, key, R, sm_keys + warp * g.words());
  uint32_t code[VPL];  // 0: not to be chosen
  uint32_t lmax = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    bool open = e < R;
    if (open && bits != nullptr) {
      const int gi = group_of(g, e);
      open = (bits[gi >> 5] >> (gi & 31)) & 1u;
    }
    code[j] = open ? key_code(key[j]) : 0u;
    lmax = max(lmax, code[j]);
  }
  // candidates: two codes per lane, or all of them
  uint32_t c0 = 0, c1 = 0;
  int e0 = 0, e1 = 0;
  bool few = VPL <= 2;
  if (VPL <= 2) {
    c0 = code[0];
    e0 = lane;
    if (VPL == 2) {
      c1 = code[VPL - 1];
      e1 = 32 + lane;
    }
  } else if (k <= 32) {
    const uint32_t least = max(1u, __shfl_sync(kAll, warp_sort_desc(lmax), k - 1));
    int mine = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) mine += code[j] >= least ? 1 : 0;
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += o;
    }
    const int total = __shfl_sync(kAll, incl, 31);
    few = total <= 64;
    if (few) {
      int at = incl - mine;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (code[j] >= least) {
          cand_code[warp][at] = code[j];
          cand_e[warp][at++] = j * 32 + lane;
        }
      __syncwarp();
      if (lane < total) {
        c0 = cand_code[warp][lane];
        e0 = cand_e[warp][lane];
      }
      if (lane + 32 < total) {
        c1 = cand_code[warp][lane + 32];
        e1 = cand_e[warp][lane + 32];
      }
    }
  }
  int32_t* ids_row = ids + t * k;
  float* probs_row = probs + t * k;
  float sum = 0.0f;
  for (int base = 0; base < k; base += 32) {
    const int slots = min(32, k - base);
    int chosen = 0;
    for (int slot = 0; slot < slots; ++slot) {
      uint32_t best = max(c0, c1);
      if (!few) {
        best = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) best = max(best, code[j]);
      }
      const uint32_t m = __reduce_max_sync(kAll, best);
      int at = 0x7fffffff;
      if (few) {
        if (c0 == m) at = e0;
        if (c1 == m) at = min(at, e1);
      } else {
#pragma unroll
        for (int j = VPL - 1; j >= 0; --j)
          if (code[j] == m) at = j * 32 + lane;
      }
      const int e = __reduce_min_sync(kAll, at);
      if (few) {
        if (e0 == e) c0 = 0;
        if (e1 == e) c1 = 0;
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          if (j * 32 + lane == e) code[j] = 0;
      }
      if (slot == lane) chosen = e;
    }
    float s = 0.0f;
    if (lane < slots) {
      const float l = lr[chosen];
      s = SOFTMAX ? expf(l - top) * inv : sigmoid_f(l);
    }
    if (renormalise)  // in slot order
      for (int slot = 0; slot < slots; ++slot) sum += __shfl_sync(kAll, s, slot);
    if (lane < slots) {
      ids_row[base + lane] = chosen;
      if (k <= 32) s = scale * (renormalise ? s / fmaxf(sum, kMinSum) : s);
      probs_row[base + lane] = s;
    }
  }
  if (k > 32)  // each lane's own values
    for (int slot = lane; slot < k; slot += 32)
      probs_row[slot] = scale * (renormalise ? probs_row[slot] / fmaxf(sum, kMinSum)
                                             : probs_row[slot]);
}

// The gradient, one warp per token.  With g = scale * dw, D = max(sum_T s, 1e-9):
//   ds_i = (g_i - [sum_T s > 1e-9] sum_j g_j s_j / D) / D (renormalise), or g_i
//   sigmoid: dl_i = ds_i s_i (1 - s_i) for i in T, 0 elsewhere
//   softmax: dl_e = s_e ([e in T] ds_e - c), c = sum_T ds_j s_j; renormalised
//   weights do not change when every selected score is scaled, so c = 0 there
//   (unless D is the floor).
// A sigmoid row reads the k selected logits only.
template <int VPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kWarps) route_rule_backward_kernel(
    const float* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const float* __restrict__ dprobs, int64_t n, int R, int k, int renormalise, float scale,
    float* __restrict__ dlogits, int64_t ldd) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= n) return;
  const float* lr = logits + t * ld;
  const int32_t* ids_row = ids + t * k;
  const float* dp = dprobs + t * k;
  float* dl = dlogits + t * ldd;
  float s_all[VPL];
  float top = 0.0f, inv = 0.0f;
  if (SOFTMAX) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * 32 + lane;
      s_all[j] = e < R ? lr[e] : -INFINITY;
      top = fmaxf(top, s_all[j]);
    }
    top = warp_max(top);
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      s_all[j] = expf(s_all[j] - top);
      sum += s_all[j];
    }
    sum = warp_sum(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  // sums over the selected experts
  float sum_s = 0.0f, sum_gs = 0.0f;
  for (int slot = lane; slot < k; slot += 32) {
    const int e = ids_row[slot];
    if (e < 0 || e >= R) continue;
    const float s = SOFTMAX ? expf(lr[e] - top) * inv : sigmoid_f(lr[e]);
    sum_s += s;
    sum_gs += scale * dp[slot] * s;
  }
  sum_s = warp_sum(sum_s);
  sum_gs = warp_sum(sum_gs);
  const float d = fmaxf(sum_s, kMinSum);
  const bool floored = !(sum_s > kMinSum);
  const float mean = renormalise && !floored ? sum_gs / d : 0.0f;
  const float c = !SOFTMAX || (renormalise && !floored) ? 0.0f : renormalise ? sum_gs / d : sum_gs;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    if (e < R) dl[e] = SOFTMAX ? -(s_all[j] * inv) * c : 0.0f;
  }
  __syncwarp();
  for (int slot = lane; slot < k; slot += 32) {
    const int e = ids_row[slot];
    if (e < 0 || e >= R) continue;
    const float s = SOFTMAX ? expf(lr[e] - top) * inv : sigmoid_f(lr[e]);
    const float gi = scale * dp[slot];
    const float ds = renormalise ? (gi - mean) / d : gi;
    dl[e] = SOFTMAX ? s * (ds - c) : ds * s * (1.0f - s);
  }
}

int values_per_lane(int R) {
  int v = 1;
  while (v * 32 < R) v *= 2;
  return v;
}

}  // namespace

#define LMOE_VPL(V, CALL) \
  case V: {               \
    constexpr int kV = V; \
    return CALL;          \
  }
#define LMOE_VPL_SWITCH(R, CALL)                                              \
  switch (values_per_lane(R)) {                                               \
    LMOE_VPL(1, CALL) LMOE_VPL(2, CALL) LMOE_VPL(4, CALL) LMOE_VPL(8, CALL)   \
    LMOE_VPL(16, CALL) LMOE_VPL(32, CALL) LMOE_VPL(64, CALL) LMOE_VPL(128, CALL) \
  }

template <int VPL, bool SOFTMAX>
static cudaError_t launch_rule(const RouteRule& rule, const Groups& g, const float* logits,
                               int64_t ld, const float* bias, int64_t n, int R, int k, int32_t* ids,
                               float* probs, cudaStream_t st) {
  const size_t smem = g.kept < g.n ? (size_t)kWarps * g.words() * 4 : 0;
  if (smem > 40 * 1024) {  // with the candidates' 2 KB, more than a kernel gets unasked
    cudaError_t e = cudaFuncSetAttribute(route_rule_kernel<VPL, SOFTMAX>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  count_launch();
  return launch_pdl(route_rule_kernel<VPL, SOFTMAX>, dim3((unsigned)((n + kWarps - 1) / kWarps)),
                    dim3(32 * kWarps), smem, st, 1, logits, ld, bias, n, R, k, g, rule.renormalise,
                    rule.scale, ids, probs);
}

cudaError_t launch_route_rule(const RouteRule& rule, const float* logits, int64_t ld,
                              const float* bias, int64_t n, int R, int k, int32_t* ids,
                              float* probs, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  Groups g;
  g.n = rule.n_groups;
  g.kept = rule.topk_groups;
  g.size = R / rule.n_groups;
  g.lanes = 1;
  while (g.lanes * 2 * g.n <= 32) g.lanes *= 2;
  g.top2 = rule.top2;
  g.inv_size = 1.0f / (float)g.size;
  LMOE_VPL_SWITCH(R, (rule.softmax ? launch_rule<kV, true>(rule, g, logits, ld, bias, n, R, k, ids,
                                                           probs, st)
                                   : launch_rule<kV, false>(rule, g, logits, ld, bias, n, R, k, ids,
                                                            probs, st)))
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_rule_backward(const RouteRule& rule, const float* logits, int64_t ld,
                                       const int32_t* ids, const float* dprobs, int64_t n, int R,
                                       int k, float* dlogits, int64_t ldd, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  const dim3 grid((unsigned)((n + kWarps - 1) / kWarps)), block(32 * kWarps);
  count_launch();
  LMOE_VPL_SWITCH(R, (rule.softmax
                          ? launch_pdl(route_rule_backward_kernel<kV, true>, grid, block, 0, st, 1,
                                       logits, ld, ids, dprobs, n, R, k, rule.renormalise,
                                       rule.scale, dlogits, ldd)
                          : launch_pdl(route_rule_backward_kernel<kV, false>, grid, block, 0, st, 1,
                                       logits, ld, ids, dprobs, n, R, k, rule.renormalise,
                                       rule.scale, dlogits, ldd)))
  return cudaErrorInvalidValue;
}

}  // namespace lmoe

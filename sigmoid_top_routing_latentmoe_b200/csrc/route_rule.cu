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
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace lmoe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kMinSum = 1e-9f;  // the least sum that weights are divided by
constexpr int kWarps = 4;

// What weights are divided by.  A NaN stays one (fmaxf would give the floor, and
// the row's other weights 1e9 times their score).
__device__ __forceinline__ float divisor(float sum) { return sum < kMinSum ? kMinSum : sum; }

__device__ __forceinline__ float sigmoid_f(float l) { return 1.0f / (1.0f + expf(-l)); }

// Order-preserving code of a key, above 0 for every key: -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t key_code(float f) {
  if (isnan(f)) f = -INFINITY;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// The key of a code (0 for -0).
__device__ __forceinline__ float decode_key(uint32_t c) {
  return __uint_as_float((c & 0x80000000u) ? c & 0x7fffffffu : ~c);
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

// Keys take expf and one approximate reciprocal (1 ulp; a score under 2^-126 counts
// as 0 there), so that a score is as good as any in 32 bits wherever its logit lies;
// equal logits give equal keys.  (The exponential of a product with log2 e, rounded
// once, was off by 2^-24 for each unit of |l|: far from zero neighbouring logits
// changed places.  That took 25 us where this takes 26, 8192 x 896.)  The weights of the chosen experts take a division.
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Shared memory of a warp: the keys, group by group (a padding of `lanes` floats
// after each group keeps the lanes that share a group's scan on different
// banks), the groups' codes and the kept groups in ascending order.
struct Groups {
  int n, kept, size, lanes, top2;  // lanes: how many lanes scan one group (a power of two)
  uint32_t magic;                  // ceil(2^32 / size): e / size = umulhi(e, magic) for e < 4096, size > 1
  __host__ __device__ int key_words() const { return n * (size + lanes); }
  __host__ __device__ int words() const { return key_words() + 2 * n; }
  __device__ int group_of(int e) const { return (int)__umulhi((uint32_t)e, magic); }
};

// Puts the topk_groups best groups in ascending order into `list`.
__device__ __forceinline__ void keep_groups(const Groups& g, const float* key, uint32_t* code,
                                            int* list) {
  const int lane = threadIdx.x & 31;
  const int per = 32 / g.lanes, sub = lane & (g.lanes - 1);
  for (int g0 = 0; g0 < g.n; g0 += per) {
    const int gi = g0 + lane / g.lanes;
    float a = -INFINITY, b = -INFINITY;  // the two largest keys (a NaN counts as -inf)
    if (gi < g.n) {
      const float* k = key + gi * (g.size + g.lanes) + sub;
#pragma unroll 8
      for (int i = 0; i < g.size - sub; i += g.lanes) {
        const float v = fmaxf(k[i], -INFINITY);
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    }
    for (int off = g.lanes >> 1; off > 0; off >>= 1) {
      const float oa = __shfl_xor_sync(kAll, a, off), ob = __shfl_xor_sync(kAll, b, off);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    if (gi < g.n && sub == 0) code[gi] = key_code(g.top2 ? a + b : a);
  }
  __syncwarp();
  int kept = 0;
  for (int g0 = 0; g0 < g.n; g0 += 32) {
    const int gi = g0 + lane;
    int rank = g.kept;
    if (gi < g.n) {
      const uint32_t c = code[gi];
      rank = 0;
#pragma unroll 4
      for (int o = 0; o < g.n; ++o) rank += code[o] > c || (code[o] == c && o < gi);
    }
    const uint32_t m = __ballot_sync(kAll, rank < g.kept);
    if (rank < g.kept) list[kept + __popc(m & ((1u << lane) - 1u))] = gi;
    kept += __popc(m);
  }
  __syncwarp();
}

constexpr uint32_t kTaken = 0xffffffffu;  // bits of a key that has its slot

// One warp per token; its keys stay in shared memory, so that the groups may
// have any size and the registers go to warps in flight.
// With k <= 32 and more than 64 open experts, the k-th largest of the 32 lane
// maxima bounds the k-th largest key from below, so only the keys at or above
// it (a few dozen) are put in order: each by counting the ones before it, or in
// k rounds of a warp maximum where k is small.  Clustered keys (more than 64
// above the bound) and k > 32 take the rounds over every open key.
// Bound by issue slots, not bytes: 8192 x 896, top 16, in 14 groups takes 26 us, 4.7
// at the copy rate; 64 tokens take one warp's chain, 8 us.
template <bool SOFTMAX, bool GROUPED>
__global__ void __launch_bounds__(32 * kWarps) route_rule_kernel(
    const float* __restrict__ logits, int64_t ld, const float* __restrict__ bias, int64_t n, int R,
    int k, Groups g, int renormalise, float scale, int32_t* __restrict__ ids,
    float* __restrict__ probs) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint64_t cands[kWarps][64];  // code, then ~expert: the larger comes first
  __shared__ int slots_e[kWarps][32];
  extern __shared__ float sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t >= n) return;
  const float* lr = logits + t * ld;
  float* key = sm + warp * g.words();
  uint32_t* code = reinterpret_cast<uint32_t*>(key + g.key_words());
  int* list = reinterpret_cast<int*>(code + g.n);
  uint64_t* cand = cands[warp];
  int* slot_e = slots_e[warp];
  // R <= 64 without groups: two experts a lane, in registers
  const bool small = !GROUPED && R <= 64;
  uint64_t c0 = 0, c1 = 0;  // this lane's candidates
  float lmax = -INFINITY;   // its largest key (NaN left out)

  float top = 0.0f, den = 0.0f, inv = 0.0f;  // softmax: the largest logit, sum of the exponentials, 1 / sum
  float l0 = -INFINITY, l1 = -INFINITY, bias0 = 0.0f, bias1 = 0.0f;  // small: this lane's
  if (small) {
    if (lane < R) l0 = lr[lane];
    if (lane + 32 < R) l1 = lr[lane + 32];
    if (bias != nullptr) {
      if (lane < R) bias0 = bias[lane];
      if (lane + 32 < R) bias1 = bias[lane + 32];
    }
  }
  if (SOFTMAX) {
    top = fmaxf(l0, l1);
    if (!small) {
#pragma unroll 16
      for (int e = lane; e < R; e += 32) top = fmaxf(top, lr[e]);
    }
    top = warp_max(top);
    if (top == -INFINITY) top = 0.0f;  // no expert is open: every score is 0
    if (small) {
      den = expf(l0 - top) + expf(l1 - top);
    } else {
      constexpr int kBatch = 8;
      for (int e0 = lane; e0 < R; e0 += 32 * kBatch) {  // from L1
        float l[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) l[j] = e0 + 32 * j < R ? lr[e0 + 32 * j] : -INFINITY;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) den += expf(l[j] - top);
      }
    }
    den = warp_sum(den);
    if (den == 0.0f) den = 1.0f;  // every exponential is 0
    inv = 1.0f / den;
  }
  auto key_of = [&](float l, float b) {
    return (SOFTMAX ? expf(l - top) * inv : rcp(1.0f + expf(-l))) + b;
  };
  auto candidate = [&](float v, int e) { return (uint64_t)key_code(v) << 32 | (uint32_t)~e; };
  if (small) {
    const float v0 = key_of(l0, bias0), v1 = key_of(l1, bias1);
    if (lane < R) c0 = candidate(v0, lane);
    if (lane + 32 < R) c1 = candidate(v1, lane + 32);
    if (k > 32) {
      if (lane < R) key[lane] = v0;
      if (lane + 32 < R) key[lane + 32] = v1;
      __syncwarp();
    }
  } else {
    // kBatch keys a lane at a time, their loads in flight together
    constexpr int kBatch = 7;
    auto put = [&](int e, float v) {
      key[GROUPED ? e + g.group_of(e) * g.lanes : e] = v;
      if (!GROUPED) lmax = fmaxf(lmax, v);
    };
    for (int e0 = lane; e0 < R; e0 += 32 * kBatch) {
      float l[kBatch], b[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int e = e0 + 32 * j;
        l[j] = e < R ? lr[e] : 0.0f;
        b[j] = bias != nullptr && e < R ? bias[e] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (e0 + 32 * j < R) put(e0 + 32 * j, key_of(l[j], b[j]));
    }
    __syncwarp();
    if (GROUPED) keep_groups(g, key, code, list);
  }

  // open expert c of `open`: its place among the keys, its number
  const int open = GROUPED ? g.kept * g.size : R;
  auto place = [&](int c) {
    if (!GROUPED) return c;
    const int a = g.group_of(c);
    return list[a] * (g.size + g.lanes) + c - a * g.size;
  };
  auto expert = [&](int c) {
    if (!GROUPED) return c;
    const int a = g.group_of(c);
    return list[a] * g.size + c - a * g.size;
  };
  int32_t* ids_row = ids + t * k;
  float* probs_row = probs + t * k;
  float sum = 0.0f;
  // slots base ... base + slots - 1 go to the experts that lanes 0 ... hold
  auto write_slots = [&](int base, int slots, int chosen) {
    float s = 0.0f;
    if (lane < slots) {
      const float l = lr[chosen];
      s = SOFTMAX ? expf(l - top) / den : sigmoid_f(l);
    }
    if (renormalise) sum += warp_sum(s);
    if (lane < slots) {
      ids_row[base + lane] = chosen;
      if (k <= 32) s = scale * (renormalise ? s / divisor(sum) : s);
      probs_row[base + lane] = s;
    }
  };

  int total = small ? R : 65;  // candidates
  if (!small && k <= 32) {
    float least = -INFINITY;  // NaN counts as -inf
    if (open > 64) {
      if (GROUPED) {
#pragma unroll 4
        for (int c = lane; c < open; c += 32) lmax = fmaxf(lmax, key[place(c)]);
      }
      least = decode_key(__shfl_sync(kAll, warp_sort_desc(key_code(lmax)), k - 1));
    }
    total = 0;
#pragma unroll 4
    for (int base = 0; base < open; base += 32) {
      const int c = base + lane;
      const float v = c < open ? key[place(c)] : 0.0f;
      const bool in = c < open && !(v < least) && (v == v || least == -INFINITY);
      const uint32_t m = __ballot_sync(kAll, in);
      if (m == 0) continue;
      const int at = total + __popc(m & ((1u << lane) - 1u));
      if (in && at < 64) cand[at] = candidate(v, expert(c));
      total += __popc(m);
    }
    __syncwarp();
    if (lane < total) c0 = cand[lane];
    if (lane + 32 < total) c1 = cand[lane + 32];
  }
  if (total <= 64 && k <= 32) {
    int chosen = 0;
    if (small || 3 * k < total) {  // k rounds of two reductions, some 14 instructions each
      for (int slot = 0; slot < k; ++slot) {
        const uint32_t h0 = (uint32_t)(c0 >> 32), h1 = (uint32_t)(c1 >> 32);
        const uint32_t m = __reduce_max_sync(kAll, max(h0, h1));
        const uint32_t l0 = h0 == m ? (uint32_t)c0 : 0u, l1 = h1 == m ? (uint32_t)c1 : 0u;
        const uint32_t best = __reduce_max_sync(kAll, max(l0, l1));
        if (h0 == m && (uint32_t)c0 == best) c0 = 0;
        if (h1 == m && (uint32_t)c1 == best) c1 = 0;
        if (slot == lane) chosen = (int)~best;
      }
    } else {  // some 5 instructions a candidate
      int r0 = 0, r1 = 0;
#pragma unroll 4
      for (int i = 0; i < total; ++i) {
        const uint64_t c = cand[i];
        r0 += c > c0;
        r1 += c > c1;
      }
      if (c0 != 0 && r0 < k) slot_e[r0] = (int)~(uint32_t)c0;
      if (c1 != 0 && r1 < k) slot_e[r1] = (int)~(uint32_t)c1;
      __syncwarp();
      if (lane < k) chosen = slot_e[lane];
    }
    write_slots(0, k, chosen);
    return;
  }
  for (int base = 0; base < k; base += 32) {
    const int slots = min(32, k - base);
    int chosen = 0;
    for (int slot = 0; slot < slots; ++slot) {
      uint32_t best = 0, at = 0;
      for (int c = lane; c < open; c += 32) {  // ascending: a tie keeps the lower one
        const float v = key[place(c)];
        const uint32_t u = __float_as_uint(v) == kTaken ? 0u : key_code(v);
        if (u > best) {
          best = u;
          at = c;
        }
      }
      const uint32_t m = __reduce_max_sync(kAll, best);
      const int c = (int)__reduce_min_sync(kAll, best == m ? at : 0x7fffffffu);
      if (lane == (c & 31)) key[place(c)] = __uint_as_float(kTaken);
      if (slot == lane) chosen = expert(c);
    }
    write_slots(base, slots, chosen);
  }
  if (k > 32)  // each lane's own values
    for (int slot = lane; slot < k; slot += 32)
      probs_row[slot] = scale * (renormalise ? probs_row[slot] / divisor(sum)
                                             : probs_row[slot]);
}

// The gradient, one warp per token.  With g = scale * dw, D = max(sum_T s, 1e-9):
//   ds_i = (g_i - [sum_T s > 1e-9] sum_j g_j s_j / D) / D (renormalise), or g_i
//   sigmoid: dl_i = ds_i s_i (1 - s_i) for i in T, 0 elsewhere
//   softmax: dl_e = s_e ([e in T] ds_e - c), c = sum_T ds_j s_j; renormalised
//   weights do not change when every selected score is scaled, so c = 0 there
//   (unless D is the floor).
// A sigmoid row reads the k selected logits only.
// Bound by bytes: 8192 x 896 takes 10.6 us softmax (9.2 at the copy rate), 7.5 sigmoid.
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
  const float d = divisor(sum_s);
  const bool floored = sum_s <= kMinSum;
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

// Dynamic shared memory that the rule kernels may need: 4096 experts in 2048
// groups of two.  The limit of a kernel is raised to it once per device: set to
// each call's own size, one host thread could lower it between another's setting
// and its launch.
constexpr int kMaxExperts = 4096, kMaxDevices = 64;
constexpr int kMaxSmem = kWarps * 4 * (kMaxExperts + 3 * (kMaxExperts / 2));

template <bool SOFTMAX, bool GROUPED>
static cudaError_t raise_smem_limit() {
  static std::mutex mu;
  static bool raised[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!raised[dev]) {
    e = cudaFuncSetAttribute(route_rule_kernel<SOFTMAX, GROUPED>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    raised[dev] = e == cudaSuccess;
  }
  return e;
}

template <bool SOFTMAX, bool GROUPED>
static cudaError_t launch_rule(const RouteRule& rule, const Groups& g, const float* logits,
                               int64_t ld, const float* bias, int64_t n, int R, int k, int32_t* ids,
                               float* probs, cudaStream_t st) {
  const size_t smem = (size_t)kWarps * g.words() * 4;
  if (smem > 40 * 1024) {  // with the candidates' 3 KB, more than a kernel gets unasked
    const cudaError_t e = raise_smem_limit<SOFTMAX, GROUPED>();
    if (e != cudaSuccess) return e;
  }
  count_launch();
  return launch_pdl(route_rule_kernel<SOFTMAX, GROUPED>, dim3((unsigned)((n + kWarps - 1) / kWarps)),
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
  // Every group is kept: as one.  So are groups of one expert: the top_k keys of
  // the topk_groups >= top_k best groups are the top_k keys, ties included (4096
  // of them would need 256 KB of shared memory a block).
  if (g.kept == g.n || g.n == R) g.n = g.kept = 1;
  g.size = R / g.n;
  g.lanes = 1;
  while (g.lanes * 2 * g.n <= 32) g.lanes *= 2;
  g.top2 = rule.top2;
  g.magic = g.size == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + g.size - 1) / g.size);
  const bool grouped = g.kept < g.n;
  const auto run = rule.softmax ? (grouped ? launch_rule<true, true> : launch_rule<true, false>)
                                : (grouped ? launch_rule<false, true> : launch_rule<false, false>);
  return run(rule, g, logits, ld, bias, n, R, k, ids, probs, st);
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

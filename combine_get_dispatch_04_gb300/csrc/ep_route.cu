// ep_route.cu -- the router (logits -> topk_idx, topk_weights) and its
// gradient.
//
// One warp per token.  Lane j holds VPL consecutive experts, so that among
// equal keys the lowest lane, and in it the lowest register, is the lowest
// index.  Keys are kept as unsigned integers in the keys' order (0: not to be
// chosen), so that one warp-wide integer maximum finds the best key of a
// round; K rounds give the choice in descending order.
#include <cuda_bf16.h>

#include "ep_common.cuh"

namespace ep {
namespace {

constexpr int kWarps = 4;  // tokens per block
constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxGroups = 64;

struct RouteArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int64_t T;
  int E, K, G, keep;
  bool sigmoid, renorm;
  float scale;
  int64_t* idx;
  float* w;
};

template <bool kBF16>
__device__ __forceinline__ float load_logit(const void* base, int64_t i) {
  if (kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  return static_cast<const float*>(base)[i];
}

// 1 / (1 + exp(-l)) with every step rounded once: the keys of the choice must
// not depend on how the compiler contracts them.
__device__ __forceinline__ float sigmoid_rn(float l) {
  return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l)));
}

// exp(l - m) for m = max l; at m = +inf the limit: the logits at +inf share.
__device__ __forceinline__ float exp_from(float l, float m) {
  return m == INFINITY ? (l == INFINITY ? 1.0f : 0.0f) : expf(l - m);
}

// Unsigned integer in the order of the float (-0 counts as +0); never 0 for a
// number, so 0 can mark what is not to be chosen.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return u == 0 ? -INFINITY : __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Lane k < K holds the chosen expert of slot k (-1: none); writes the slots.
// m, z: the softmax's maximum and sum (read when !renorm && !sigmoid).
template <bool kBF16>
__device__ __forceinline__ void write_slots(const RouteArgs& a, int64_t t, int lane, int mine,
                                            float m, float z) {
  const bool live = lane < a.K && mine >= 0;
  const float l = live ? load_logit<kBF16>(a.logits, t * a.stride + mine) : -INFINITY;
  float u = 0.0f;
  if (a.sigmoid) {
    u = live ? sigmoid_rn(l) : 0.0f;
  } else if (a.renorm) {
    const float top = warp_max(l);
    u = live ? exp_from(l, top) : 0.0f;
  } else {
    u = live ? exp_from(l, m) / z : 0.0f;
  }
  if (a.renorm) {
    const float s = warp_sum(u);
    u = s > 0.0f ? u / s : 0.0f;
  }
  if (lane < a.K) {
    a.idx[t * a.K + lane] = mine;
    a.w[t * a.K + lane] = u * a.scale;
  }
}

// E <= 32 * VPL, groups (if any) of a power of two of whole lanes.
template <int VPL, bool kBF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a, int group_lanes) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int e0 = lane * VPL;

  float l[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    l[v] = e0 + v < a.E ? load_logit<kBF16>(a.logits, t * a.stride + e0 + v) : -INFINITY;

  float m = -INFINITY, z = 1.0f;
  if (!a.sigmoid && (a.bias || !a.renorm)) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) m = fmaxf(m, l[v]);  // fmaxf passes over NaN
    m = warp_max(m);
    z = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) z += l[v] > -INFINITY ? exp_from(l[v], m) : 0.0f;
    z = warp_sum(z);
  }
  uint32_t key[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float c = l[v];
    if (a.sigmoid) c = sigmoid_rn(c);
    if (a.bias && l[v] > -INFINITY) {
      if (!a.sigmoid) c = exp_from(c, m) / z;
      c = __fadd_rn(c, a.bias[e0 + v]);
    }
    key[v] = l[v] > -INFINITY ? ordered(c) : 0u;  // false for NaN
  }

  if (a.G > 1) {
    uint32_t m1 = 0, m2 = 0;  // the two largest keys of the group
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      m2 = max(m2, min(m1, key[v]));
      m1 = max(m1, key[v]);
    }
    for (int o = 1; o < group_lanes; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
      m2 = max(min(m1, o1), max(m2, o2));
      m1 = max(m1, o1);
    }
    float g = from_ordered(m1);
    if (a.sigmoid && m2) g = __fadd_rn(g, from_ordered(m2));
    const int mine = lane / group_lanes;
    int better = 0;
    for (int j = 0; j < a.G; ++j) {
      const float other = __shfl_sync(kFull, g, j * group_lanes);
      better += other > g || (other == g && j < mine);
    }
    if (better >= a.keep) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) key[v] = 0;
    }
  }

  int chosen = -1;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) best = max(best, key[v]);
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;  // uniform: nothing left to choose
    const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
    int e = 0;
    bool taken = lane != owner;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (!taken && key[v] == top) {
        e = e0 + v;
        key[v] = 0;
        taken = true;
      }
    }
    e = __shfl_sync(kFull, e, owner);
    if (lane == k) chosen = e;
  }
  write_slots<kBF16>(a, t, lane, chosen, m, z);
}

// Any E and any groups: the keys in shared memory, lanes over experts and
// over groups.
template <bool kBF16>
__global__ void route_any_kernel(RouteArgs a) {
  pdl_wait_then_release();
  extern __shared__ uint32_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  uint32_t* key = smem + warp * (a.E + kMaxGroups);
  float* gscore = reinterpret_cast<float*>(key + a.E);

  float m = -INFINITY, z = 1.0f;
  if (!a.sigmoid && (a.bias || !a.renorm)) {
    for (int e = lane; e < a.E; e += 32)
      m = fmaxf(m, load_logit<kBF16>(a.logits, t * a.stride + e));
    m = warp_max(m);
    z = 0.0f;
    for (int e = lane; e < a.E; e += 32) {
      const float l = load_logit<kBF16>(a.logits, t * a.stride + e);
      z += l > -INFINITY ? exp_from(l, m) : 0.0f;
    }
    z = warp_sum(z);
  }
  for (int e = lane; e < a.E; e += 32) {
    const float l = load_logit<kBF16>(a.logits, t * a.stride + e);
    float c = l;
    if (a.sigmoid) c = sigmoid_rn(c);
    if (a.bias && l > -INFINITY) {
      if (!a.sigmoid) c = exp_from(c, m) / z;
      c = __fadd_rn(c, a.bias[e]);
    }
    key[e] = l > -INFINITY ? ordered(c) : 0u;
  }
  __syncwarp();

  if (a.G > 1) {
    const int size = a.E / a.G;
    for (int g = lane; g < a.G; g += 32) {
      uint32_t m1 = 0, m2 = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t c = key[g * size + i];
        m2 = max(m2, min(m1, c));
        m1 = max(m1, c);
      }
      float s = from_ordered(m1);
      if (a.sigmoid && m2) s = __fadd_rn(s, from_ordered(m2));
      gscore[g] = s;
    }
    __syncwarp();
    bool drop[kMaxGroups / 32] = {};
#pragma unroll
    for (int i = 0; i < kMaxGroups / 32; ++i) {
      const int g = lane + 32 * i;
      if (g >= a.G) continue;
      int better = 0;
      for (int j = 0; j < a.G; ++j)
        better += gscore[j] > gscore[g] || (gscore[j] == gscore[g] && j < g);
      drop[i] = better >= a.keep;
    }
#pragma unroll
    for (int i = 0; i < kMaxGroups / 32; ++i) {
      const int g = lane + 32 * i;
      if (g < a.G && drop[i])
        for (int j = 0; j < size; ++j) key[g * size + j] = 0;
    }
    __syncwarp();
  }

  int chosen = -1;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < a.E; e += 32) {
      if (key[e] > best) {
        best = key[e];
        at = e;
      }
    }
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;
    const int e = (int)__reduce_min_sync(kFull, best == top ? (unsigned)at : 0x7FFFFFFFu);
    if (lane == (e & 31)) key[e] = 0;
    __syncwarp();
    if (lane == k) chosen = e;
  }
  write_slots<kBF16>(a, t, lane, chosen, m, z);
}

struct GradArgs {
  const float* dw;
  const void* logits;
  int64_t stride;
  const int64_t* idx;
  int64_t T;
  int E, K;
  bool sigmoid, renorm;
  float scale;
  void* dl;
  int32_t* err;
};

template <bool kBF16>
__device__ __forceinline__ void store_grad(void* base, int64_t i, float v) {
  if (kBF16)
    static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(base)[i] = v;
}

// One warp per token; lane k holds slot k.  Only the chosen experts have a
// gradient unless the weights are softmax scores that are not renormalised.
template <bool kBF16>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(GradArgs a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int64_t row = t * a.E;

  const int64_t id = lane < a.K ? a.idx[t * a.K + lane] : -1;
  const bool bad = id < -1 || id >= a.E;
  if (__any_sync(kFull, bad) && lane == 0 && a.err) atomicOr(a.err, EP_ERRBIT_BAD_EXPERT);
  const int e = (id >= 0 && !bad) ? (int)id : -1;
  const float l = e >= 0 ? load_logit<kBF16>(a.logits, t * a.stride + e) : -INFINITY;
  const bool live = e >= 0 && l > -INFINITY;
  const float dw = live ? a.scale * a.dw[t * a.K + lane] : 0.0f;

  // g: the gradient with respect to this slot's logit, before the slots of
  // one expert are added up; dense: minus the factor of every score
  float g, m = 0.0f, rz = 0.0f, dense = 0.0f;
  if (a.sigmoid) {
    const float u = live ? sigmoid_rn(l) : 0.0f;
    float du = dw;
    if (a.renorm) {
      const float s = warp_sum(u), r = s > 0.0f ? 1.0f / s : 0.0f;
      du = (dw - warp_sum(dw * (u * r))) * r;
    }
    g = du * u * (1.0f - u);
  } else if (a.renorm) {
    const float top = warp_max(live ? l : -INFINITY);
    const float x = live ? exp_from(l, top) : 0.0f, s = warp_sum(x);
    const float w = s > 0.0f ? x / s : 0.0f;
    g = w * (dw - warp_sum(w * dw));
  } else {
    m = -INFINITY;
    for (int i = lane; i < a.E; i += 32)
      m = fmaxf(m, load_logit<kBF16>(a.logits, t * a.stride + i));
    m = warp_max(m);
    float z = 0.0f;
    for (int i = lane; i < a.E; i += 32) {
      const float li = load_logit<kBF16>(a.logits, t * a.stride + i);
      z += li > -INFINITY ? exp_from(li, m) : 0.0f;
    }
    z = warp_sum(z);
    rz = z > 0.0f ? 1.0f / z : 0.0f;
    const float p = live ? exp_from(l, m) * rz : 0.0f;
    dense = warp_sum(p * dw);
    g = p * dw;  // the dense part is added below, once per expert
  }

  if (!a.sigmoid && !a.renorm) {
    for (int i = lane; i < a.E; i += 32) {
      const float li = load_logit<kBF16>(a.logits, t * a.stride + i);
      store_grad<kBF16>(a.dl, row + i, li > -INFINITY ? -(exp_from(li, m) * rz) * dense : 0.0f);
    }
    if (live) g -= exp_from(l, m) * rz * dense;
  } else {
    for (int i = lane; i < a.E; i += 32) store_grad<kBF16>(a.dl, row + i, 0.0f);
  }

  // slots that name the same expert are added in the order of k
  const unsigned same = __match_any_sync(kFull, live ? e : -1 - lane);
  const bool dup = __any_sync(kFull, __popc(same) > 1);
  if (dup) {
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k) {
      const float gk = __shfl_sync(kFull, g, k), pd = __shfl_sync(kFull, dense, k);
      const float pk = __shfl_sync(kFull, live ? exp_from(l, m) * rz : 0.0f, k);
      if (same >> k & 1) {
        // the dense part belongs to the expert, not to each of its slots
        sum += (k == __ffs(same) - 1) ? gk : gk + pk * pd;
      }
    }
    g = sum;
  }
  __syncwarp();
  if (live && lane == __ffs(same) - 1) store_grad<kBF16>(a.dl, row + e, g);
}

template <bool kBF16>
void launch_route(const RouteArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.T + kWarps - 1) / kWarps);
  const int size = a.E / a.G;
  // the smallest register tile that holds E and, with groups, splits them
  // into a power of two of whole lanes
  const auto fits = [&](int vpl) {
    if (a.E > 32 * vpl) return false;
    if (a.G == 1) return true;
    if (size % vpl) return false;
    const int n = size / vpl;
    return (n & (n - 1)) == 0 && n <= 32;
  };
#define EP_ROUTE_CASE(V)                                                                         \
  if (fits(V)) {                                                                                 \
    launch_pdl(route_kernel<V, kBF16>, blocks, kWarps * 32, 0, st, a, a.G > 1 ? size / V : 32); \
    return;                                                                                      \
  }
  EP_ROUTE_CASE(1)
  EP_ROUTE_CASE(2)
  EP_ROUTE_CASE(4)
  EP_ROUTE_CASE(5)
  EP_ROUTE_CASE(8)
  EP_ROUTE_CASE(16)
#undef EP_ROUTE_CASE
  const int warps = a.E <= 1024 ? 4 : 1;  // at most 17 KB of keys a block
  launch_pdl(route_any_kernel<kBF16>, (unsigned)((a.T + warps - 1) / warps), warps * 32,
             (size_t)warps * (a.E + kMaxGroups) * 4, st, a);
}

bool score_ok(int score) { return score == EP_SCORE_SOFTMAX || score == EP_SCORE_SIGMOID; }

// Shapes that both directions share; the element type's alignment is all the
// logits need.
bool router_ok(const void* logits, int bf16, int64_t stride, int64_t T, int E, int K) {
  if (T < 0 || T >= (int64_t(1) << 31) || E < 1 || E > EP_MAX_EXPERTS) return false;
  if (K < 1 || K > EP_MAX_TOPK || stride < E) return false;
  if (T > 0 && (!logits || reinterpret_cast<uintptr_t>(logits) % (bf16 ? 2 : 4))) return false;
  return true;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" ep_status_t ep_route(const void* logits, int logits_bf16, int64_t row_stride,
                                const float* bias, int64_t num_tokens, int num_experts,
                                int num_topk, int score, int num_groups, int topk_groups,
                                int renormalize, float scale, int64_t* topk_idx,
                                float* topk_weights, ep_stream_t stream) {
  if (!router_ok(logits, logits_bf16, row_stride, num_tokens, num_experts, num_topk))
    return EP_ERR_INVALID_ARG;
  if (num_topk > num_experts || !score_ok(score)) return EP_ERR_INVALID_ARG;
  if (num_groups < 1 || num_groups > kMaxGroups || num_experts % num_groups ||
      topk_groups < 1 || topk_groups > num_groups)
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!topk_idx || !topk_weights || !aligned16(topk_idx) || !aligned16(topk_weights) ||
      !aligned16(bias))
    return EP_ERR_INVALID_ARG;
  RouteArgs a = {logits,    row_stride,  bias, num_tokens,  num_experts, num_topk,     num_groups,
                 topk_groups, score == EP_SCORE_SIGMOID, renormalize != 0, scale, topk_idx,
                 topk_weights};
  if (a.keep == a.G) a.G = a.keep = 1;  // every group is kept
  cudaStream_t st = to_cuda(stream);
  if (logits_bf16)
    launch_route<true>(a, st);
  else
    launch_route<false>(a, st);
  return launch_status();
}

extern "C" ep_status_t ep_route_backward(const float* dweights, const void* logits,
                                         int logits_bf16, int64_t row_stride,
                                         const int64_t* topk_idx, int64_t num_tokens,
                                         int num_experts, int num_topk, int score,
                                         int renormalize, float scale, void* dlogits,
                                         int32_t* err_word, ep_stream_t stream) {
  if (!router_ok(logits, logits_bf16, row_stride, num_tokens, num_experts, num_topk))
    return EP_ERR_INVALID_ARG;
  if (!score_ok(score)) return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!dweights || !topk_idx || !dlogits || !aligned16(dweights) || !aligned16(topk_idx) ||
      !aligned16(dlogits))
    return EP_ERR_INVALID_ARG;
  const GradArgs a = {dweights,    logits,           row_stride,       topk_idx,
                      num_tokens,  num_experts,      num_topk,         score == EP_SCORE_SIGMOID,
                      renormalize != 0, scale,       dlogits,          err_word};
  const unsigned blocks = (unsigned)((num_tokens + kWarps - 1) / kWarps);
  if (logits_bf16)
    launch_pdl(route_grad_kernel<true>, blocks, kWarps * 32, 0, to_cuda(stream), a);
  else
    launch_pdl(route_grad_kernel<false>, blocks, kWarps * 32, 0, to_cuda(stream), a);
  return launch_status();
}

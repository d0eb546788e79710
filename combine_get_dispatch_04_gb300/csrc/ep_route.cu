// ep_route.cu -- the router (logits -> topk_idx, topk_weights) and its
// gradient.
//
// The choice takes more instructions than bytes, so a warp works on as many
// tokens as fit: LANES lanes hold a token, VPL consecutive experts each, and
// all tokens of the warp go through the same rounds.  Keys are kept as
// unsigned integers in the keys' order (0: not to be chosen); a round finds
// the largest key of the token and then the lowest index that has it, K
// rounds give the choice in descending order.  What bounds it is the integer
// pipe: some 40 instructions a round for 8 experts a lane, two cycles each,
// and below a few thousand tokens the chain of K reductions.  Time on the
// device: 4096 tokens, sigmoid scores, 256 experts in 8 groups, 8 chosen:
// 10.2 us; 32768 such tokens 41 us; one token 3.9 us.  bf16 logits that are
// the keys themselves need no rounds (below).
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
  return __frcp_rn(__fadd_rn(1.0f, expf(-l)));
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

// The weights of the slots of one token, by the LANES lanes that hold it.
// slots: this token's chosen experts (-1: none); u: room for K scores.
// m, z: the softmax's maximum and sum (read when !renorm && !sigmoid).
template <int LANES, bool kBF16>
__device__ __forceinline__ void write_slots(const RouteArgs& a, int64_t t, bool in, int sl,
                                            const int* slots, float* u, float m, float z) {
  float top = -INFINITY, sum = 0.0f;
  if (!a.sigmoid && a.renorm) {
    for (int k = sl; k < a.K; k += LANES)
      if (slots[k] >= 0) top = fmaxf(top, load_logit<kBF16>(a.logits, t * a.stride + slots[k]));
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  }
  for (int k = sl; k < a.K; k += LANES) {
    float v = 0.0f;
    if (slots[k] >= 0) {
      const float l = load_logit<kBF16>(a.logits, t * a.stride + slots[k]);
      v = a.sigmoid ? sigmoid_rn(l) : a.renorm ? exp_from(l, top) : exp_from(l, m) / z;
    }
    u[k] = v;
    sum += v;
  }
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (!in) return;
  for (int k = sl; k < a.K; k += LANES) {
    a.idx[t * a.K + k] = slots[k];
    a.w[t * a.K + k] = (a.renorm ? (sum > 0.0f ? u[k] / sum : 0.0f) : u[k]) * a.scale;
  }
}

// This lane's VPL logits (-inf beyond E).  vec: rows are 16-byte aligned and
// hold whole lanes.
template <int VPL, bool kBF16>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int e0, bool vec,
                                            float (&l)[VPL]) {
  if (VPL == 8 && vec) {
    if (e0 < a.E) {
      if (kBF16) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(
            static_cast<const __nv_bfloat16*>(a.logits) + row + e0));
        float f[8];
        unpack_bf16x8(v, f);
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = f[i & 7];
      } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row + e0);
        const float4 v[2] = {__ldg(p), __ldg(p + 1)};
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = (&v[i >> 2 & 1].x)[i & 3];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = -INFINITY;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    l[i] = e0 + i < a.E ? load_logit<kBF16>(a.logits, row + e0 + i) : -INFINITY;
}

// E <= LANES * VPL, groups (if any) of a power of two of whole lanes.
template <int LANES, int VPL, bool kBF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a, int group_lanes, bool vec) {
  pdl_wait_then_release();
  constexpr int kTokens = 32 / LANES;  // of a warp
  __shared__ int slots[kWarps][kTokens][EP_MAX_TOPK];
  __shared__ float score[kWarps][kTokens][EP_MAX_TOPK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sl = lane % LANES, mine = lane / LANES, lane0 = lane - sl;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * kTokens;
  if (first >= a.T) return;  // the whole warp
  const bool in = first + mine < a.T;
  const int64_t t = in ? first + mine : a.T - 1;  // lanes without a token repeat the last one
  const int e0 = sl * VPL;

  float l[VPL];
  load_logits<VPL, kBF16>(a, t * a.stride, e0, vec, l);

  float m = -INFINITY, z = 1.0f;
  if (!a.sigmoid && (a.bias || !a.renorm)) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) m = fmaxf(m, l[v]);  // fmaxf passes over NaN
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    z = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) z += l[v] > -INFINITY ? exp_from(l[v], m) : 0.0f;
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
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
    key[v] = l[v] > -INFINITY && c > -INFINITY ? ordered(c) : 0u;  // false for NaN
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
    const int own = sl / group_lanes;
    int better = 0;
    for (int j = 0; j < a.G; ++j) {
      const float other = __shfl_sync(kFull, g, lane0 + j * group_lanes);
      better += other > g || (other == g && j < own);
    }
    if (better >= a.keep) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) key[v] = 0;
    }
  }

  const unsigned below = ((1u << sl) - 1u) << lane0;  // the token's lanes of lower experts
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) best = max(best, key[v]);
    uint32_t top = best;
    if (LANES == 32) {
      top = __reduce_max_sync(kFull, best);
    } else {
#pragma unroll
      for (int o = LANES / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    }
    // the first lane that has it gives its first key that is it
    const unsigned have = __ballot_sync(kFull, best == top);
    const bool look = best == top && !(have & below);
    int e = -1;
    bool open = look && top;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const bool hit = open && key[v] == top;
      open = open && key[v] != top;
      if (hit) {
        e = e0 + v;
        key[v] = 0;
      }
    }
    if (look) slots[warp][mine][k] = e;
  }
  __syncwarp();
  write_slots<LANES, kBF16>(a, t, in, sl, slots[warp][mine], score[warp][mine], m, z);
}

// --- bf16 logits as keys, at most eight experts a token ---------------------------
// A key is 32 bits: the logit in the order of unsigned integers above, 0xFFFF
// - index below, so keys differ and ties go to the lowest index.  A lane sorts
// the 8 keys of a 16-byte chunk with a network of 19 exchanges, and joins
// two sorted lists into their eight largest with 8 maxima and 12 exchanges
// (the larger of a[i] and b[7 - i] are the eight, in a bitonic order): first
// its own chunks, then other lanes' lists.  That takes about 9 integer
// instructions a key, and no step waits for a reduction over the warp.
// 131072 tokens of 64 experts, 6 chosen: 10.3 us (25 us with rounds; its
// bytes take 3.9), 32768 of 256, 8 chosen: 11.1 (25.7).  The same with 64-bit
// keys, for other scores, takes three instructions for one here and was
// slower than the rounds (32768 tokens of 256 experts: 39.8 against 32.2 us).
constexpr int kBest = 8;    // experts a token
constexpr int kChunks = 4;  // chunks a lane

__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}
__device__ __forceinline__ void sort8(uint32_t (&k)[8]) {
  exchange(k[0], k[1]), exchange(k[2], k[3]), exchange(k[4], k[5]), exchange(k[6], k[7]);
  exchange(k[0], k[2]), exchange(k[1], k[3]), exchange(k[4], k[6]), exchange(k[5], k[7]);
  exchange(k[1], k[2]), exchange(k[5], k[6]);
  exchange(k[0], k[4]), exchange(k[1], k[5]), exchange(k[2], k[6]), exchange(k[3], k[7]);
  exchange(k[2], k[4]), exchange(k[3], k[5]);
  exchange(k[1], k[2]), exchange(k[3], k[4]), exchange(k[5], k[6]);
}
__device__ __forceinline__ void join8(uint32_t (&a)[8], const uint32_t (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) exchange(a[i], a[i + d]);
}

// Keys of the chunk of experts e0 .. e0 + 7, two logits at a time: -0 becomes
// +0 (adding 0), NaN becomes -inf (the maximum with -inf), then negative
// numbers are inverted and positive ones get the sign bit.  -inf is 0x007F,
// below every number.
__device__ __forceinline__ void chunk_keys(const uint4& raw, int e0, uint32_t (&k)[8]) {
  uint32_t index = (uint32_t)(0xFFFF - e0 - 1) << 16 | (uint32_t)(0xFFFF - e0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = (&raw.x)[i];
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0u));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0xFF80FF80u));
    uint32_t sign;
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(sign) : "r"(v));  // each half's, 16 times
    v ^= sign | 0x80008000u;
    k[2 * i] = __byte_perm(index, v, 0x5410);
    k[2 * i + 1] = __byte_perm(index, v, 0x7632);
    index -= 0x00020002u;
  }
}
__device__ __forceinline__ bool key_is_number(uint32_t k) { return k >> 16 > 0x007Fu; }
__device__ __forceinline__ float key_logit(uint32_t k) {
  // a negative number is inverted, so its lower half is ones here
  return from_ordered(k & 0x80000000u ? k & 0xFFFF0000u : k | 0xFFFFu);
}

// Softmax scores of bf16 logits without a bias.  LANES lanes hold a token,
// chunks LANES apart; K <= kBest, E <= 8 * kChunks * LANES.
template <int LANES>
__global__ void __launch_bounds__(kWarps * 32) route_sort_kernel(RouteArgs a, bool vec) {
  pdl_wait_then_release();
  constexpr int kTokens = 32 / LANES;  // of a warp
  __shared__ int slots[kWarps][kTokens * kBest];
  __shared__ float weight[kWarps][kTokens * kBest];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sl = lane % LANES, mine = lane / LANES;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * kTokens;
  if (first >= a.T) return;  // the whole warp
  const int64_t t = min(first + mine, a.T - 1);  // lanes without a token repeat the last one
  const uint16_t* row = static_cast<const uint16_t*>(a.logits) + t * a.stride;

  uint4 raw[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int e0 = (c * LANES + sl) * 8;
    raw[c] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    if (e0 >= a.E) continue;
    if (vec) {
      raw[c] = __ldg(reinterpret_cast<const uint4*>(row + e0));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i < a.E)
          (&raw[c].x)[i >> 1] = __byte_perm((&raw[c].x)[i >> 1], __ldg(row + e0 + i),
                                            i & 1 ? 0x5410 : 0x3254);
    }
  }
  uint32_t best[8];
  chunk_keys(raw[0], sl * 8, best);
  sort8(best);
#pragma unroll
  for (int c = 1; c < kChunks; ++c) {
    if (c * LANES * 8 >= a.E) break;
    uint32_t k[8];
    chunk_keys(raw[c], (c * LANES + sl) * 8, k);
    sort8(k);
    join8(best, k);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    uint32_t k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = __shfl_xor_sync(kFull, best[i], o);
    join8(best, k);
  }

  // every lane of the token has the list now
  const float m = key_is_number(best[0]) ? key_logit(best[0]) : -INFINITY;
  float u[kBest], sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kBest; ++k) {
    u[k] = k < a.K && key_is_number(best[k]) ? exp_from(key_logit(best[k]), m) : 0.0f;
    sum += u[k];
  }
  if (!a.renorm) {  // over all experts instead
    sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (c * LANES * 8 >= a.E) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = (&raw[c].x)[i >> 1];
        const float l = __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
        sum += l > -INFINITY ? exp_from(l, m) : 0.0f;
      }
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  // through shared memory, so that a warp writes its tokens' slots in order
  if (sl == 0) {
#pragma unroll
    for (int k = 0; k < kBest; ++k) {
      if (k < a.K) {
        slots[warp][mine * a.K + k] = key_is_number(best[k]) ? 0xFFFF - (int)(best[k] & 0xFFFF) : -1;
        weight[warp][mine * a.K + k] = (sum > 0.0f ? u[k] / sum : 0.0f) * a.scale;
      }
    }
  }
  __syncwarp();
  const int n = (int)min((int64_t)kTokens, a.T - first) * a.K;
  for (int i = lane; i < n; i += 32) {
    a.idx[first * a.K + i] = slots[warp][i];
    a.w[first * a.K + i] = weight[warp][i];
  }
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
  uint32_t* key = smem + warp * (a.E + kMaxGroups + 2 * EP_MAX_TOPK);
  float* gscore = reinterpret_cast<float*>(key + a.E);
  int* slots = reinterpret_cast<int*>(gscore + kMaxGroups);
  float* score = reinterpret_cast<float*>(slots + EP_MAX_TOPK);

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
    key[e] = l > -INFINITY && c > -INFINITY ? ordered(c) : 0u;
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
    const int e = (int)__reduce_min_sync(kFull, best == top ? (unsigned)at : 0x7FFFFFFFu);
    if (top && lane == (e & 31)) key[e] = 0;
    if (lane == 0) slots[k] = top ? e : -1;
    __syncwarp();
  }
  write_slots<32, kBF16>(a, t, true, lane, slots, score, m, z);
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
  bool vec;  // logits' rows are 16-byte aligned and whole vectors
};

// SL lanes hold a token, one slot each (K <= SL), and its row of gradients in
// shared memory, where the slots are added; then the row is written in
// 16-byte stores.  The rows written are most of the traffic: only the chosen
// experts have a gradient, and only their logits are read, unless the weights
// are softmax scores that are not renormalised (kDense: the row is read, and
// kept in shared memory as exp(l - max)).  Everything stays within a warp.
// Bound by DRAM, and by the passes over the row in shared memory where that is
// kept: 32768 tokens of 256 experts, float32, sigmoid scores: 12.0 us (its
// bytes take 5.7); 131072 tokens of 64 experts, bf16, dense: 20.4 us (6.4).
template <int SL>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int o = SL / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int SL>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
  for (int o = SL / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// A row's place in shared memory: 16-byte aligned, and eight banks further
// for every token of a warp.
inline __host__ __device__ int grad_pitch(int E) { return (E + 7) / 8 * 8 + 8; }

template <int SL, bool kBF16, bool kDense>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(GradArgs a) {
  pdl_wait_then_release();
  extern __shared__ __align__(16) float sm[];
  constexpr int kTokens = 32 / SL, kVec = kBF16 ? 8 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % SL;
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x >> 5) + warp) * kTokens;
  if (first >= a.T) return;  // the whole warp
  const bool in = first + lane / SL < a.T;
  const int64_t t = in ? first + lane / SL : a.T - 1;  // a spare token repeats the last one
  float* row = sm + (warp * kTokens + lane / SL) * grad_pitch(a.E);

  const int64_t id = sub < a.K ? a.idx[t * a.K + sub] : -1;
  const bool bad = id < -1 || id >= a.E;
  if (bad && a.err) atomicOr(a.err, EP_ERRBIT_BAD_EXPERT);
  const int e = id >= 0 && !bad ? (int)id : -1;
  const float l = e >= 0 ? load_logit<kBF16>(a.logits, t * a.stride + e) : -INFINITY;
  const bool live = l > -INFINITY;  // false for NaN
  const float dw = live ? a.scale * a.dw[t * a.K + sub] : 0.0f;

  float m = -INFINITY, rz = 0.0f;
  if (kDense) {
    if (a.vec) {
      for (int i = sub * kVec; i < a.E; i += SL * kVec) {
        float f[8];
        const int4 v = __ldg(reinterpret_cast<const int4*>(
            static_cast<const char*>(a.logits) + (t * a.stride + i) * (kBF16 ? 2 : 4)));
        if (kBF16) {
          unpack_bf16x8(v, f);
        } else {
          f[0] = __int_as_float(v.x), f[1] = __int_as_float(v.y);
          f[2] = __int_as_float(v.z), f[3] = __int_as_float(v.w);
        }
#pragma unroll
        for (int j = 0; j < kVec; j += 4)
          *reinterpret_cast<float4*>(row + i + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
#pragma unroll
        for (int j = 0; j < kVec; ++j) m = fmaxf(m, f[j]);
      }
    } else {
      for (int i = sub; i < a.E; i += SL) {
        const float li = load_logit<kBF16>(a.logits, t * a.stride + i);
        row[i] = li;
        m = fmaxf(m, li);
      }
    }
    m = part_max<SL>(m);
    __syncwarp();
    float z = 0.0f;
    for (int i = sub; i < a.E; i += SL) {
      const float x = row[i] > -INFINITY ? exp_from(row[i], m) : 0.0f;
      row[i] = x;
      z += x;
    }
    z = part_sum<SL>(z);
    rz = z > 0.0f ? 1.0f / z : 0.0f;
  } else {
    for (int i = sub * 4; i < a.E; i += SL * 4)
      *reinterpret_cast<float4*>(row + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }

  float g;  // this slot's part of its logit's gradient
  if (kDense) {
    const float p = live ? exp_from(l, m) * rz : 0.0f;
    g = p * dw;
    const float dot = part_sum<SL>(g) * -rz;
    __syncwarp();
    for (int i = sub; i < a.E; i += SL) row[i] *= dot;
  } else if (a.sigmoid) {
    const float u = live ? sigmoid_rn(l) : 0.0f;
    if (a.renorm) {
      const float s = part_sum<SL>(u);
      const float w = s > 0.0f ? u / s : 0.0f;  // 1 / s may overflow where u / s does not
      g = w * (dw - part_sum<SL>(w * dw));
    } else {
      g = u * dw;
    }
    g *= sigmoid_rn(-l);  // 1 - u would cancel: 0 from l = 17 on
  } else {
    const float top = part_max<SL>(l);
    const float x = live ? exp_from(l, top) : 0.0f, s = part_sum<SL>(x);
    const float w = s > 0.0f ? x / s : 0.0f;
    g = w * (dw - part_sum<SL>(w * dw));
  }
  __syncwarp();
  // an expert that a token names twice gets its slots in the order of k
  const unsigned same = __match_any_sync(kFull, live ? lane / SL << 16 | e : -1 - lane);
  if (__any_sync(kFull, live && (same & (same - 1)))) {
    for (int k = 0; k < SL; ++k) {
      if (sub == k && live) row[e] += g;
      __syncwarp();
    }
  } else if (live) {
    row[e] += g;
  }
  __syncwarp();
  if (!in) return;
  const int64_t out = t * a.E;
  if (a.E % kVec == 0) {  // rows of whole vectors
    for (int i = sub * kVec; i < a.E; i += SL * kVec) {
      int4 v;
      const float4 f = *reinterpret_cast<const float4*>(row + i);
      if (kBF16) {
        const float4 h = *reinterpret_cast<const float4*>(row + i + 4);
        const __nv_bfloat162 w[4] = {__floats2bfloat162_rn(f.x, f.y), __floats2bfloat162_rn(f.z, f.w),
                                     __floats2bfloat162_rn(h.x, h.y), __floats2bfloat162_rn(h.z, h.w)};
        v = *reinterpret_cast<const int4*>(w);
        st_stream_v4(reinterpret_cast<int4*>(static_cast<__nv_bfloat16*>(a.dl) + out + i), v);
      } else {
        v = make_int4(__float_as_int(f.x), __float_as_int(f.y), __float_as_int(f.z),
                      __float_as_int(f.w));
        st_stream_v4(reinterpret_cast<int4*>(static_cast<float*>(a.dl) + out + i), v);
      }
    }
  } else {
    for (int i = sub; i < a.E; i += SL) {
      if (kBF16)
        static_cast<__nv_bfloat16*>(a.dl)[out + i] = __float2bfloat16_rn(row[i]);
      else
        static_cast<float*>(a.dl)[out + i] = row[i];
    }
  }
}

template <int SL, bool kBF16, bool kDense>
ep_status_t launch_grad(const GradArgs& a, cudaStream_t st) {
  const int warps = a.E <= 512 ? kWarps : 1;  // at most 33 KB of rows a block
  const int64_t per = warps * (32 / SL);
  launch_pdl(route_grad_kernel<SL, kBF16, kDense>, (unsigned)((a.T + per - 1) / per), warps * 32,
             (size_t)per * grad_pitch(a.E) * 4, st, a);
  return launch_status();
}

template <bool kBF16, bool kDense>
ep_status_t launch_grad_lanes(const GradArgs& a, cudaStream_t st) {
  // eight lanes a token where its slots fit them and four rows a warp fit
  // shared memory
  return a.K <= 8 && a.E <= 512 ? launch_grad<8, kBF16, kDense>(a, st)
                                : launch_grad<32, kBF16, kDense>(a, st);
}

template <bool kBF16>
void launch_route(const RouteArgs& a, int sm_count, cudaStream_t st) {
  const int size = a.E / a.G;
  const bool vec = a.E % 8 == 0 && aligned16(a.logits) && a.stride * (kBF16 ? 2 : 4) % 16 == 0;
  // The first tile below that holds E and, with groups, splits them into a power
  // of two of whole lanes.  Tiles of eight experts a lane, which are loaded in
  // 16-byte vectors, come first, from few lanes a token to many: 32768 float32
  // tokens of 16 / 64 / 128 experts, 8 chosen (of 16: 4), take 4.4 / 10.5 / 19.3 us,
  // and 21 / 26 / 26 with 32 lanes each.  Then other widths of 32 lanes, for sizes
  // and groups that eight does not divide and up to 512 experts (384: 74 us), then
  // the keys in shared memory (600: 85 us).
  const auto fits = [&](int lanes, int vpl) {
    if (a.E > lanes * vpl) return false;
    if (a.G == 1) return true;
    if (size % vpl) return false;
    const int n = size / vpl;
    return (n & (n - 1)) == 0 && n <= lanes;
  };
  if (kBF16 && !a.sigmoid && !a.bias && a.G == 1 && a.K <= kBest && a.E <= 8 * kChunks * 32) {
    // the fewest lanes that hold E, so that most of the joining is a lane's
    // own, unless there are too few tokens for every scheduler to have a warp
    // (one token of 256 experts: 2.1 against 2.4 us)
    const int64_t few = 4 * (int64_t)sm_count;  // one for each scheduler
    int lanes = 1;
    while (lanes < 32 && (a.E > 8 * kChunks * lanes ||
                          (a.E > 8 * lanes && a.T * lanes < few * 32)))
      lanes *= 2;
#define EP_ROUTE_SORT(L)                                                                       \
  case L: {                                                                                    \
    const int64_t per = kWarps * (32 / L);                                                     \
    launch_pdl(route_sort_kernel<L>, (unsigned)((a.T + per - 1) / per), kWarps * 32, 0, st, a, \
               vec);                                                                           \
    return;                                                                                    \
  }
    switch (lanes) {
      EP_ROUTE_SORT(1)
      EP_ROUTE_SORT(2)
      EP_ROUTE_SORT(4)
      EP_ROUTE_SORT(8)
      EP_ROUTE_SORT(16)
      EP_ROUTE_SORT(32)
    }
#undef EP_ROUTE_SORT
  }
#define EP_ROUTE_CASE(L, V)                                                              \
  if (fits(L, V)) {                                                                      \
    const int64_t per = kWarps * (32 / L);                                               \
    launch_pdl(route_kernel<L, V, kBF16>, (unsigned)((a.T + per - 1) / per), kWarps * 32, \
               0, st, a, a.G > 1 ? size / V : L, vec);                                   \
    return;                                                                              \
  }
  EP_ROUTE_CASE(2, 8)
  EP_ROUTE_CASE(8, 8)
  EP_ROUTE_CASE(16, 8)
  EP_ROUTE_CASE(32, 5)
  EP_ROUTE_CASE(32, 8)
  EP_ROUTE_CASE(32, 2)
  EP_ROUTE_CASE(32, 4)
  EP_ROUTE_CASE(32, 16)
#undef EP_ROUTE_CASE
  const int warps = a.E <= 1024 ? 4 : 1;  // at most 18 KB of keys a block
  launch_pdl(route_any_kernel<kBF16>, (unsigned)((a.T + warps - 1) / warps), warps * 32,
             (size_t)warps * (a.E + kMaxGroups + 2 * EP_MAX_TOPK) * 4, st, a);
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
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  cudaStream_t st = to_cuda(stream);
  if (logits_bf16)
    launch_route<true>(a, props.sm_count, st);
  else
    launch_route<false>(a, props.sm_count, st);
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
  const uint64_t size = logits_bf16 ? 2 : 4;
  if (overlap(dlogits, num_tokens * num_experts * size, logits,
              ((num_tokens - 1) * row_stride + num_experts) * size))
    return EP_ERR_INVALID_ARG;
  const GradArgs a = {dweights,    logits,           row_stride,       topk_idx,
                      num_tokens,  num_experts,      num_topk,         score == EP_SCORE_SIGMOID,
                      renormalize != 0, scale,       dlogits,          err_word,
                      aligned16(logits) && row_stride * (logits_bf16 ? 2 : 4) % 16 == 0 &&
                          num_experts % (logits_bf16 ? 8 : 4) == 0};
  const bool dense = score == EP_SCORE_SOFTMAX && !renormalize;
  cudaStream_t st = to_cuda(stream);
  if (logits_bf16)
    return dense ? launch_grad_lanes<true, true>(a, st) : launch_grad_lanes<true, false>(a, st);
  return dense ? launch_grad_lanes<false, true>(a, st) : launch_grad_lanes<false, false>(a, st);
}

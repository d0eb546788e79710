// ep_route.cuh -- the router's choice of experts for one token, by a warp or a
// part of one: shared by the router (ep_route.cu) and the layer for a few tokens
// (ep_layer_w4.cu), which so choose alike.
#pragma once

#include <cuda_bf16.h>

#include "ep_common.cuh"

namespace ep {

constexpr unsigned kFull = 0xFFFFFFFFu;  // every lane of a warp
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

// The tile in registers that holds a choice (vpl 0: none, the keys go to shared memory):
// the first that holds E and, with groups, splits them into a power of two of whole
// lanes.  Tiles of eight experts a lane, which are loaded in 16-byte vectors, come
// first, from few lanes a token to many: 32768 float32 tokens of 16 / 64 / 128
// experts, 8 chosen (of 16: 4), take 4.4 / 10.5 / 19.3 us, and 21 / 26 / 26 with 32 lanes
// each.  Then other widths of 32 lanes, for sizes and groups that eight does not
// divide and up to 512 experts (384: 74 us), then the keys in shared memory (600: 85 us).
struct RouteTile {
  int lanes, vpl;
};
inline RouteTile route_tile(int E, int G) {
  constexpr RouteTile kTiles[] = {{2, 8}, {8, 8}, {16, 8}, {32, 5}, {32, 8}, {32, 2}, {32, 4}, {32, 16}};
  for (const RouteTile& t : kTiles) {
    if (E > t.lanes * t.vpl) continue;
    if (G == 1) return t;
    if (E / G % t.vpl) continue;
    const int n = E / G / t.vpl;  // lanes of a group
    if ((n & (n - 1)) == 0 && n <= t.lanes) return t;
  }
  return {32, 0};
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

// The choice of token t by the LANES lanes that hold it, VPL experts each: E <=
// LANES * VPL, groups (if any) of a power of two of whole lanes.  Its experts
// go to `slots`; m and z are the softmax's maximum and sum where those are needed.
template <int LANES, int VPL, bool kBF16>
__device__ __forceinline__ void choose_in_registers(const RouteArgs& a, int64_t t, int lane,
                                                    int group_lanes, bool vec, int* slots,
                                                    float& m, float& z) {
  const int sl = lane % LANES, lane0 = lane - sl, e0 = sl * VPL;
  float l[VPL];
  load_logits<VPL, kBF16>(a, t * a.stride, e0, vec, l);

  m = -INFINITY, z = 1.0f;
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
    if (look) slots[k] = e;
  }
}

// The same for any E and any groups, by a warp: the keys in shared memory, lanes
// over experts and over groups.  key: E words, gscore: kMaxGroups.  kUnroll: of its
// loops (1 where the code's size counts more than its speed).  run: consecutive experts
// that a lane adds up to z, or 0 for every 32nd.  With the VPL of a tile, z has the bits that
// choose_in_registers gives it there: a lane's sum is its lane's, and where fewer than 32 lanes
// hold a token there, the others add zeros here.
template <bool kBF16, int kUnroll>
__device__ __forceinline__ void choose_in_shared(const RouteArgs& a, int64_t t, int lane, int run,
                                                 uint32_t* key, float* gscore, int* slots,
                                                 float& m, float& z) {
  m = -INFINITY, z = 1.0f;
  if (!a.sigmoid && (a.bias || !a.renorm)) {
#pragma unroll kUnroll
    for (int e = lane; e < a.E; e += 32)
      m = fmaxf(m, load_logit<kBF16>(a.logits, t * a.stride + e));
    m = warp_max(m);
    z = 0.0f;
    const int end = run ? min(a.E, (lane + 1) * run) : a.E, step = run ? 1 : 32;
#pragma unroll kUnroll
    for (int e = run ? lane * run : lane; e < end; e += step) {
      const float l = load_logit<kBF16>(a.logits, t * a.stride + e);
      z += l > -INFINITY ? exp_from(l, m) : 0.0f;
    }
    z = warp_sum(z);
  }
#pragma unroll kUnroll
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
#pragma unroll kUnroll
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
#pragma unroll kUnroll
      for (int j = 0; j < a.G; ++j)
        better += gscore[j] > gscore[g] || (gscore[j] == gscore[g] && j < g);
      drop[i] = better >= a.keep;
    }
#pragma unroll
    for (int i = 0; i < kMaxGroups / 32; ++i) {
      const int g = lane + 32 * i;
      if (g < a.G && drop[i])
#pragma unroll kUnroll
        for (int j = 0; j < size; ++j) key[g * size + j] = 0;
    }
    __syncwarp();
  }

  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF;
#pragma unroll kUnroll
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
}

}  // namespace ep

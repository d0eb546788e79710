// ep_block_norm.cu -- what stands between two blocks: the norm after a block,
// its gate and residual scale, the addition to the residual stream and the norm
// before the next block, in one pass over the row; with the combine of the
// experts' rows in front of it, and its gradient.
//
//   n = y / rms(y) * post,  z = x + scale * gate * n,  h = z / rms(z) * pre
//
// Forward: a block takes one token and keeps its row in registers, in 32
// bits, between the two sums of squares.
//
// Backward: with d = dh * pre, q = y * post * gate, r = 1 / rms and c = r_z^3
// mean(z d),
//   dx = dz + r_z d - c z                    =: t
//   dy = scale (r_y post gate t - r_y^3 mean(q t) y)
// The sum of q t needs t, and so the sum of z d first; but it is sum(q dz) + r_z sum(q d)
// - c sum(q z), so one reduction of six sums serves both norms.  The sums over
// the tokens (of dh z r_z and of t y r_y) stay in the registers of a persistent
// block and are joined by a second kernel in a fixed order.
#include <cuda_bf16.h>

#include "ep_common.cuh"

namespace ep {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxHidden = 16384;
constexpr int kMaxWarps = 16;

enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };

struct NormArgs {
  const void* x;  // the stream (backward: its result z)
  const uint8_t* y;
  const int32_t* slot;  // [T, K]: y is the expert-major rows
  const float* w;
  int K;
  int64_t rows, T;
  int H, nvec;
  const void *gate, *post, *pre;
  int gate_kind;
  bool bf16;  // type of gate, post and pre
  float scale, eps;
  void* z;
  uint8_t *h, *comb;
  int32_t* err;
  // backward
  const void* dz;
  const uint8_t* dh;
  void* dx;
  uint8_t* dy;
  void* dgate;
  float *dpost, *dpre;
  float* part;  // [blocks][2][H]
};

__device__ __forceinline__ int4 pack8(const float (&f)[8]) {
  int4 v;
  uint32_t* p = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    p[i] = *reinterpret_cast<const uint32_t*>(&two);
  }
  return v;
}

// Eight values of a weight (kept in L1: every token reads them).
__device__ __forceinline__ void weight8(const void* p, bool bf16, int64_t v, float (&f)[8]) {
  if (bf16) {
    unpack_bf16x8(__ldg(static_cast<const int4*>(p) + v), f);
  } else {
    const float4* q = static_cast<const float4*>(p) + 2 * v;
    const float4 a = __ldg(q), b = __ldg(q + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}
__device__ __forceinline__ float weight1(const void* p, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}

// Eight values of the stream, read once.
template <bool kF32>
struct Stream8 {
  int4 v[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
#pragma unroll
    for (int i = 0; i < (kF32 ? 2 : 1); ++i)
      v[i] = ld_stream_v4(static_cast<const int4*>(p) + at * (kF32 ? 2 : 1) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kF32 ? 2 : 1); ++i) v[i] = make_int4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (kF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __int_as_float((&v[i >> 2].x)[i & 3]);
    } else {
      unpack_bf16x8(v[0], f);
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t at, const float (&f)[8]) {
    if constexpr (kF32) {
      int4* q = static_cast<int4*>(p) + 2 * at;
      st_stream_v4(q, make_int4(__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]),
                                __float_as_int(f[3])));
      st_stream_v4(q + 1, make_int4(__float_as_int(f[4]), __float_as_int(f[5]),
                                    __float_as_int(f[6]), __float_as_int(f[7])));
    } else {
      st_stream_v4(static_cast<int4*>(p) + at, pack8(f));
    }
  }
};

// Sums of kN values over the block; every thread gets them.  `part` is not
// written again before the caller's next barrier.
template <int kN>
__device__ __forceinline__ void block_sums(float (&v)[kN], float (*part)[kN]) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int o = 16; o; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) part[threadIdx.x >> 5][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    v[i] = lane < warps ? part[lane][i] : 0.0f;
#pragma unroll
    for (int o = kMaxWarps / 2; o; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
    v[i] = __shfl_sync(kFull, v[i], 0);
  }
}

// The token's live rows and their weights; run by one warp.
__device__ __forceinline__ int live_rows(const NormArgs& a, int64_t t, int lane, int32_t* row,
                                         float* weight) {
  int32_t r = lane < a.K ? a.slot[t * a.K + lane] : -1;
  const bool over = r >= a.rows;
  if (over && a.err) atomicOr(a.err, EP_ERRBIT_CAPACITY);
  const bool live = r >= 0 && !over;
  const unsigned all = __ballot_sync(kFull, live);
  if (live) {
    const int at = __popc(all & ((1u << lane) - 1u));
    row[at] = r;
    weight[at] = a.w ? a.w[t * a.K + lane] : 1.0f;
  }
  return __popc(all);
}

// NV vectors of 8 channels a thread.
template <int NV, bool kF32, bool kRows>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a) {
  pdl_wait_then_release();
  __shared__ float part[2][kMaxWarps][1];
  __shared__ int32_t row[EP_MAX_TOPK];
  __shared__ float weight[EP_MAX_TOPK];
  __shared__ int live;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t t = blockIdx.x, base = t * a.nvec;

  Stream8<kF32> xv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * threads;
    if (v < a.nvec) xv[i].load(a.x, base + v);
    else xv[i].zero();
  }
  float y[NV][8];
  if (kRows) {
    if (tid < 32) {
      const int n = live_rows(a, t, tid, row, weight);
      if (tid == 0) live = n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) y[i][c] = 0.0f;
    const int n = live;
    const int4* src = reinterpret_cast<const int4*>(a.y);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const int4* p = src + (int64_t)row[k] * a.nvec;
      const float w = weight[k];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * threads;
        if (v < a.nvec) {
          float f[8];
          unpack_bf16x8(ld_stream_v4(p + v), f);
#pragma unroll
          for (int c = 0; c < 8; ++c) y[i][c] = fmaf(w, f[c], y[i][c]);
        }
      }
    }
    if (a.comb) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * threads;
        if (v < a.nvec) st_stream_v4(reinterpret_cast<int4*>(a.comb) + base + v, pack8(y[i]));
      }
    }
  } else if (a.y) {
    int4 yv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * threads;
      yv[i] = make_int4(0, 0, 0, 0);
      if (v < a.nvec) yv[i] = ld_stream_v4(reinterpret_cast<const int4*>(a.y) + base + v);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack_bf16x8(yv[i], y[i]);
  }

  if (kRows || a.y) {
    float f = a.scale;
    if (a.gate_kind == kGateToken) f *= weight1(a.gate, a.bf16, t);
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) s[0] = fmaf(y[i][c], y[i][c], s[0]);
      block_sums<1>(s, part[0]);
      f *= rsqrtf(s[0] / (float)a.H + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * threads;
      float g[8], x[8];
      if (v < a.nvec) {
        if (a.post) {
          weight8(a.post, a.bf16, v, g);
#pragma unroll
          for (int c = 0; c < 8; ++c) y[i][c] *= g[c];
        }
        if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
          weight8(a.gate, a.bf16, a.gate_kind == kGateFull ? base + v : v, g);
#pragma unroll
          for (int c = 0; c < 8; ++c) y[i][c] *= g[c];
        }
        xv[i].get(x);
#pragma unroll
        for (int c = 0; c < 8; ++c) y[i][c] = fmaf(f, y[i][c], x[c]);
        Stream8<kF32>::store(a.z, base + v, y[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) xv[i].get(y[i]);
  }
  if (!a.h) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) s[0] = fmaf(y[i][c], y[i][c], s[0]);
  block_sums<1>(s, part[1]);
  const float r = rsqrtf(s[0] / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * threads;
    if (v < a.nvec) {
      float g[8];
      weight8(a.pre, a.bf16, v, g);
#pragma unroll
      for (int c = 0; c < 8; ++c) g[c] *= y[i][c] * r;
      st_stream_v4(reinterpret_cast<int4*>(a.h) + base + v, pack8(g));
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
template <int NV, bool kF32>
__global__ void __launch_bounds__(512) norm_grad_kernel(NormArgs a) {
  pdl_wait_then_release();
  __shared__ float part[2][kMaxWarps][6];
  const int tid = threadIdx.x, threads = blockDim.x;
  const bool need_y = a.post || a.gate_kind != kGateNone;
  const float inv_h = 1.0f / (float)a.H;
  float cpre[NV][8], cpost[NV][8];  // this block's sums over its tokens
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) cpre[i][c] = cpost[i][c] = 0.0f;

  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const int64_t base = t * a.nvec;
    Stream8<kF32> zv[NV], dzv[NV];
    int4 yv[NV], dhv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * threads;
      zv[i].zero();
      dzv[i].zero();
      yv[i] = dhv[i] = make_int4(0, 0, 0, 0);
      if (v < a.nvec) {
        if (a.dh) zv[i].load(a.x, base + v);
        if (a.dz) dzv[i].load(a.dz, base + v);
        if (need_y) yv[i] = ld_stream_v4(reinterpret_cast<const int4*>(a.y) + base + v);
        if (a.dh) dhv[i] = ld_stream_v4(reinterpret_cast<const int4*>(a.dh) + base + v);
      }
    }
    const float gt = a.gate_kind == kGateToken ? weight1(a.gate, a.bf16, t) : 1.0f;
    // z z, y y, z d, q dz, q d, q z
    float s[6] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = min(tid + i * threads, a.nvec - 1);
      float z[8], dz[8], y[8], d[8], g[8];
      zv[i].get(z);
      dzv[i].get(dz);
      unpack_bf16x8(yv[i], y);
      unpack_bf16x8(dhv[i], d);
      if (a.dh) {
        weight8(a.pre, a.bf16, v, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) d[c] *= g[c];
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        s[0] = fmaf(z[c], z[c], s[0]);
        s[1] = fmaf(y[c], y[c], s[1]);
        s[2] = fmaf(z[c], d[c], s[2]);
      }
      if (need_y) {
        if (a.post) {
          weight8(a.post, a.bf16, v, g);
#pragma unroll
          for (int c = 0; c < 8; ++c) y[c] *= g[c];
        }
        if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
          weight8(a.gate, a.bf16, a.gate_kind == kGateFull ? base + v : v, g);
#pragma unroll
          for (int c = 0; c < 8; ++c) y[c] *= g[c];
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          s[3] = fmaf(y[c], dz[c], s[3]);
          s[4] = fmaf(y[c], d[c], s[4]);
          s[5] = fmaf(y[c], z[c], s[5]);
        }
      }
    }
    block_sums<6>(s, part[turn]);
    const float rz = a.dh ? rsqrtf(s[0] * inv_h + a.eps) : 0.0f;
    const float cz = rz * rz * rz * (s[2] * inv_h);
    const float ry = a.post ? rsqrtf(s[1] * inv_h + a.eps) : 1.0f;
    const float qt = s[3] + rz * s[4] - cz * s[5];  // sum of q t
    const float f = a.scale * gt;
    const float cy = a.post ? f * ry * ry * ry * (qt * inv_h) : 0.0f;
    if (a.gate_kind == kGateToken && tid == 0 && a.dgate)
      static_cast<float*>(a.dgate)[t] = a.scale * ry * qt;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * threads;
      if (v >= a.nvec) continue;
      float tt[8], z[8], dh[8], y[8], g[8], o[8];
      dzv[i].get(tt);
      if (a.dh) {
        zv[i].get(z);
        unpack_bf16x8(dhv[i], dh);
        weight8(a.pre, a.bf16, v, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float hr = dh[c] * rz;
          cpre[i][c] = fmaf(hr, z[c], cpre[i][c]);
          tt[c] = fmaf(hr, g[c], fmaf(-cz, z[c], tt[c]));
        }
      }
      Stream8<kF32>::store(a.dx, base + v, tt);
      if (need_y) unpack_bf16x8(yv[i], y);
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = f * tt[c];  // the gradient of gate n / gate
      if (a.gate_kind == kGateFull) {
        float p[8];
        weight8(a.gate, a.bf16, base + v, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) p[c] = 1.0f;
        if (a.post) weight8(a.post, a.bf16, v, p);
#pragma unroll
        for (int c = 0; c < 8; ++c) p[c] *= o[c] * y[c] * ry;
        if (a.dgate) {
          if (a.bf16)
            st_stream_v4(static_cast<int4*>(a.dgate) + base + v, pack8(p));
          else
            Stream8<true>::store(a.dgate, base + v, p);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] *= g[c];
      }
      if (need_y) {  // without the channel's gate, which the second kernel knows
#pragma unroll
        for (int c = 0; c < 8; ++c) cpost[i][c] = fmaf(o[c], y[c] * ry, cpost[i][c]);
      }
      if (a.gate_kind == kGateChannel) {
        weight8(a.gate, a.bf16, v, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] *= g[c];
      }
      if (a.post) {
        weight8(a.post, a.bf16, v, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = fmaf(ry * g[c], o[c], -cy * y[c]);
      }
      if (a.dy) st_stream_v4(reinterpret_cast<int4*>(a.dy) + base + v, pack8(o));
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * threads;
    if (v >= a.nvec) continue;
    float4* p = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * 2 * a.H) + 2 * v;
    p[0] = make_float4(cpre[i][0], cpre[i][1], cpre[i][2], cpre[i][3]);
    p[1] = make_float4(cpre[i][4], cpre[i][5], cpre[i][6], cpre[i][7]);
    p += a.H / 4;
    p[0] = make_float4(cpost[i][0], cpost[i][1], cpost[i][2], cpost[i][3]);
    p[1] = make_float4(cpost[i][4], cpost[i][5], cpost[i][6], cpost[i][7]);
  }
}

// The blocks' sums, added up channel by channel: 32 channels a block, 8
// warps over the blocks of the first kernel.
__global__ void __launch_bounds__(256) norm_columns_kernel(NormArgs a, int blocks) {
  pdl_wait_then_release();
  __shared__ float sum[8][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float s0 = 0.0f, s1 = 0.0f;
  if (h < a.H) {
#pragma unroll 4
    for (int b = warp; b < blocks; b += 8) {
      s0 += a.part[(int64_t)b * 2 * a.H + h];
      s1 += a.part[(int64_t)b * 2 * a.H + a.H + h];
    }
  }
  sum[warp][0][lane] = s0;
  sum[warp][1][lane] = s1;
  __syncthreads();
  if (warp >= 2 || h >= a.H) return;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += sum[i][warp][lane];
  if (warp == 0) {
    if (a.dpre) a.dpre[h] = s;
    return;
  }
  const bool channel = a.gate_kind == kGateChannel;
  if (a.dpost) a.dpost[h] = channel ? s * weight1(a.gate, a.bf16, h) : s;
  if (channel && a.dgate)
    static_cast<float*>(a.dgate)[h] = a.post ? s * weight1(a.post, a.bf16, h) : s;
}

// Vectors a thread and threads a block for rows of nvec vectors.
struct Shape {
  int nv, threads;
};
Shape forward_shape(int nvec) {
  const int nv = nvec <= 64 ? 1 : nvec <= 256 ? 2 : 4;
  return {nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}
Shape backward_shape(int nvec) {
  const int nv = nvec <= 128 ? 1 : nvec <= 1024 ? 2 : 4;
  return {nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}
int backward_blocks(int64_t T, int threads, int sm_count) {
  const int64_t most = (int64_t)sm_count * (1024 / threads > 8 ? 8 : 1024 / threads < 1 ? 1 : 1024 / threads);
  return (int)(T < most ? T : most);
}

template <int NV, bool kF32>
void launch_forward(const NormArgs& a, int threads, cudaStream_t st) {
  if (a.slot)
    launch_pdl(norm_kernel<NV, kF32, true>, (unsigned)a.T, threads, 0, st, a);
  else
    launch_pdl(norm_kernel<NV, kF32, false>, (unsigned)a.T, threads, 0, st, a);
}

bool common_ok(const NormArgs& a, int64_t T, int H, int gate_kind, float eps) {
  if (T < 0 || T >= (int64_t(1) << 31) || H < 8 || H % 8 || H > kMaxHidden) return false;
  if (gate_kind < kGateNone || gate_kind > kGateFull) return false;
  if (!(eps > 0.0f)) return false;
  return aligned16(a.post) && aligned16(a.pre) &&
         (gate_kind == kGateToken
              ? reinterpret_cast<uintptr_t>(a.gate) % (a.bf16 ? 2 : 4) == 0
              : aligned16(a.gate));
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" ep_status_t ep_block_norm(const void* x, int stream_f32, const void* y,
                                     int64_t num_rows, const float* topk_weights, int num_topk,
                                     const int32_t* ll_slot, int64_t num_tokens, int hidden,
                                     const void* gate, int gate_kind, const void* post_weight,
                                     const void* pre_weight, int weights_bf16, float scale,
                                     float eps, void* z, void* h, void* combined,
                                     int32_t* err_word, ep_stream_t stream) {
  NormArgs a = {};
  a.x = x;
  a.y = static_cast<const uint8_t*>(y);
  a.slot = ll_slot;
  a.w = topk_weights;
  a.K = num_topk;
  a.rows = ll_slot ? num_rows : num_tokens;
  a.T = num_tokens;
  a.H = hidden;
  a.nvec = hidden / 8;
  a.gate = gate;
  a.post = post_weight;
  a.pre = pre_weight;
  a.gate_kind = gate_kind;
  a.bf16 = weights_bf16 != 0;
  a.scale = scale;
  a.eps = eps;
  a.z = z;
  a.h = static_cast<uint8_t*>(h);
  a.comb = static_cast<uint8_t*>(combined);
  a.err = err_word;
  if (!common_ok(a, num_tokens, hidden, gate_kind, eps)) return EP_ERR_INVALID_ARG;
  if (ll_slot && (num_topk < 1 || num_topk > EP_MAX_TOPK || num_rows < 0 ||
                  num_rows >= (int64_t(1) << 31)))
    return EP_ERR_INVALID_ARG;
  if (!ll_slot && (combined || topk_weights)) return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  const bool block = ll_slot || y;  // there is a block's output to add
  if (!x || !pre_weight != !h || !block != !z || (!block && !h)) return EP_ERR_INVALID_ARG;
  if (!block && (post_weight || gate_kind != kGateNone)) return EP_ERR_INVALID_ARG;
  if (ll_slot && num_rows > 0 && !y) return EP_ERR_INVALID_ARG;
  if (!gate != (gate_kind == kGateNone)) return EP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(z) || !aligned16(h) || !aligned16(combined))
    return EP_ERR_INVALID_ARG;
  // a token's outputs are written while others still read: nothing may overlap,
  // but z may be x itself, which each token reads before it writes
  const uint64_t n = (uint64_t)num_tokens * hidden, xs = n * (stream_f32 ? 4 : 2);
  const uint64_t ys = (uint64_t)a.rows * hidden * 2;
  const uint64_t gs = gate_kind == kGateFull ? n * (a.bf16 ? 2 : 4) : 0;
  if ((z != x && overlap(z, xs, x, xs)) || overlap(z, xs, y, ys) || overlap(h, 2 * n, x, xs) ||
      overlap(h, 2 * n, y, ys) || overlap(h, 2 * n, z, xs) || overlap(combined, 2 * n, x, xs) ||
      overlap(combined, 2 * n, y, ys) || overlap(combined, 2 * n, z, xs) ||
      overlap(combined, 2 * n, h, 2 * n) || overlap(z, xs, gate, gs) || overlap(h, 2 * n, gate, gs) ||
      overlap(combined, 2 * n, gate, gs))
    return EP_ERR_INVALID_ARG;
  const Shape s = forward_shape(a.nvec);
  cudaStream_t st = to_cuda(stream);
  if (stream_f32)
    s.nv == 1   ? launch_forward<1, true>(a, s.threads, st)
    : s.nv == 2 ? launch_forward<2, true>(a, s.threads, st)
                : launch_forward<4, true>(a, s.threads, st);
  else
    s.nv == 1   ? launch_forward<1, false>(a, s.threads, st)
    : s.nv == 2 ? launch_forward<2, false>(a, s.threads, st)
                : launch_forward<4, false>(a, s.threads, st);
  return launch_status();
}

extern "C" size_t ep_block_norm_backward_workspace_bytes(int64_t num_tokens, int hidden) {
  if (num_tokens < 1 || hidden < 8 || hidden % 8 || hidden > kMaxHidden) return 0;
  DeviceProps props;
  if (!device_props(&props)) return 0;
  return (size_t)backward_blocks(num_tokens, backward_shape(hidden / 8).threads, props.sm_count) *
         2 * hidden * sizeof(float);
}

extern "C" ep_status_t ep_block_norm_backward(
    const void* dz, const void* dh, const void* z, int stream_f32, const void* y,
    int64_t num_tokens, int hidden, const void* gate, int gate_kind, const void* post_weight,
    const void* pre_weight, int weights_bf16, float scale, float eps, void* dx, void* dy,
    void* dgate, float* dpost_weight, float* dpre_weight, void* workspace, size_t workspace_bytes,
    ep_stream_t stream) {
  NormArgs a = {};
  a.x = z;
  a.y = static_cast<const uint8_t*>(y);
  a.T = num_tokens;
  a.H = hidden;
  a.nvec = hidden / 8;
  a.gate = gate;
  a.post = post_weight;
  a.pre = pre_weight;
  a.gate_kind = gate_kind;
  a.bf16 = weights_bf16 != 0;
  a.scale = scale;
  a.eps = eps;
  a.dz = dz;
  a.dh = static_cast<const uint8_t*>(dh);
  a.dx = dx;
  a.dy = static_cast<uint8_t*>(dy);
  a.dgate = dgate;
  a.dpost = dpost_weight;
  a.dpre = dpre_weight;
  if (!common_ok(a, num_tokens, hidden, gate_kind, eps)) return EP_ERR_INVALID_ARG;
  if ((dpost_weight && !post_weight) || (dpre_weight && !pre_weight) || (dgate && !gate))
    return EP_ERR_INVALID_ARG;
  if (!aligned16(dz) || !aligned16(dh) || !aligned16(z) || !aligned16(y) || !aligned16(dx) ||
      !aligned16(dy) || !aligned16(dgate) || !aligned16(dpost_weight) || !aligned16(dpre_weight) ||
      !aligned16(workspace))
    return EP_ERR_INVALID_ARG;
  const bool columns = dpre_weight || dpost_weight || (dgate && gate_kind == kGateChannel);
  cudaStream_t st = to_cuda(stream);
  if (num_tokens == 0) {  // the sums over no tokens
    if (dpre_weight && cudaMemsetAsync(dpre_weight, 0, hidden * 4, st) != cudaSuccess) return EP_ERR_CUDA;
    if (dpost_weight && cudaMemsetAsync(dpost_weight, 0, hidden * 4, st) != cudaSuccess) return EP_ERR_CUDA;
    if (dgate && gate_kind == kGateChannel && cudaMemsetAsync(dgate, 0, hidden * 4, st) != cudaSuccess)
      return EP_ERR_CUDA;
    return EP_OK;
  }
  const bool need_y = post_weight || gate_kind != kGateNone;
  if (!gate != (gate_kind == kGateNone) || !dh != !pre_weight) return EP_ERR_INVALID_ARG;
  if (!dx || (!dz && !dh) || (dh && !z) || (need_y && !y)) return EP_ERR_INVALID_ARG;
  const uint64_t n = (uint64_t)num_tokens * hidden, ss = n * (stream_f32 ? 4 : 2);
  const uint64_t gs = gate_kind == kGateFull ? n * (a.bf16 ? 2 : 4) : 0;
  const struct {
    const void* p;
    uint64_t n;
  } in[] = {{dz, ss}, {dh, 2 * n}, {z, ss}, {y, 2 * n}, {gate, gs}},
    out[] = {{dx, ss}, {dy, 2 * n}, {dgate, gs}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(o.p, o.n, i.p, i.n)) return EP_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return EP_ERR_INVALID_ARG;
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  const Shape s = backward_shape(a.nvec);
  const int blocks = backward_blocks(num_tokens, s.threads, props.sm_count);
  if (columns) {
    if (!workspace || workspace_bytes < (size_t)blocks * 2 * hidden * sizeof(float))
      return EP_ERR_CAPACITY;
    a.part = static_cast<float*>(workspace);
  }
  const auto go = [&](auto kernel) {
    launch_pdl(kernel, (unsigned)blocks, s.threads, 0, st, a);
  };
  if (stream_f32)
    s.nv == 1 ? go(norm_grad_kernel<1, true>) : s.nv == 2 ? go(norm_grad_kernel<2, true>)
                                                          : go(norm_grad_kernel<4, true>);
  else
    s.nv == 1 ? go(norm_grad_kernel<1, false>) : s.nv == 2 ? go(norm_grad_kernel<2, false>)
                                                           : go(norm_grad_kernel<4, false>);
  if (columns)
    launch_pdl(norm_columns_kernel, (unsigned)((hidden + 31) / 32), 256, 0, st, a, blocks);
  return launch_status();
}

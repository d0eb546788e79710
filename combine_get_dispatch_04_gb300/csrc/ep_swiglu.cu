// ep_swiglu.cu -- the experts' gated activation on the rows of the
// expert-major layout, and its gradient, with the input kept in 8 bits.
//
// Forward: h = w * silu(g) * u from rows of [g | u]; the same pass leaves g and
// u as E4M3 codes with one scale per 128 channels, so keeping them costs only
// the bytes written.  Backward: with s = sigmoid(g),
//   dg = w dh u s (1 + g (1 - s)),  du = w dh g s,  dw = sum_n dh g s u.
// The rows are found through the slots, so the weight of a row is the slot's,
// and rows that no slot names are neither read nor written.
#include <cuda_bf16.h>

#include "ep_experts_w4.cuh"
#include "ep_scatter.cuh"

namespace ep {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

struct SwigluArgs {
  const uint8_t* gate_up;  // bf16 [rows, 2 N] (NULL in a backward pass from codes)
  const uint8_t* codes;    // E4M3 [rows, 2 N]
  const float* scales;     // [rows, 2 N / 128]
  const uint8_t* dh;       // bf16 [rows, N]
  int N;
  int64_t rows, slots;
  const int32_t* slot;
  const float* w;  // NULL: 1
  uint8_t* out;    // h [rows, N] or dgate_up [rows, 2 N]
  uint8_t* out_codes;
  float* out_scales;
  float* dw;
  int32_t* err;
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

// The row of slot i (-1: none, or one beyond the buffer, which is reported).
__device__ __forceinline__ int slot_row(const SwigluArgs& a, int64_t i, bool tell) {
  const int r = a.slot[i];
  if (r >= a.rows) {
    if (tell && a.err) atomicOr(a.err, EP_ERRBIT_CAPACITY);
    return -1;
  }
  return r;
}

// Codes and scale of the 16 channels in v, whose block of 128 is held by 8
// neighbouring lanes.  Every step is rounded as the FP8 dispatch rounds it.  A block
// with an infinity or a NaN has codes that read back as NaN throughout.
__device__ __forceinline__ uint4 quantise16(const int4 (&v)[2], float* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // |x| of finite bf16 is ordered as the low 15 bits, and NaN is above all
    m = __vmaxu2(m, __vmaxu2(__vmaxu2((uint32_t)v[i].x & 0x7FFF7FFFu, (uint32_t)v[i].y & 0x7FFF7FFFu),
                             __vmaxu2((uint32_t)v[i].z & 0x7FFF7FFFu, (uint32_t)v[i].w & 0x7FFF7FFFu)));
  }
  m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  const float top = __uint_as_float(m << 16);
  const float am = top < 1e-4f ? 1e-4f : top;  // keeps NaN
  const float inv = __fdiv_rn(448.0f, am);
  *scale = __fdiv_rn(am, 448.0f);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[8];
    unpack_bf16x8(v[i], f);
    q[2 * i] = cvt_e4m3x4(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv), __fmul_rn(f[2], inv),
                          __fmul_rn(f[3], inv));
    q[2 * i + 1] = cvt_e4m3x4(__fmul_rn(f[4], inv), __fmul_rn(f[5], inv), __fmul_rn(f[6], inv),
                              __fmul_rn(f[7], inv));
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

__device__ __forceinline__ void dequantise16(const int4& codes, float scale, float (&f)[16]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&codes);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1)) & 0xFFFFu), __NV_E4M3);
    const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = two.x * scale;
    f[2 * i + 1] = two.y * scale;
  }
}

constexpr int kThreads = 128;
constexpr int kUnroll = 2;  // pieces a lane holds at once

// A warp takes 32 * kUnroll pieces of one slot's row, a piece being kV vectors
// of 8 channels of g and the same of u.
template <bool kKeep>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluArgs a, int parts) {
  constexpr int kV = kKeep ? 2 : 1;
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t i = unit / parts;
  if (i >= a.slots) return;
  const int part = (int)(unit - i * parts);
  const int64_t row = slot_row(a, i, lane == 0 && part == 0);
  if (row < 0) return;
  const float w = a.w ? a.w[i] : 1.0f;
  const int nvec = a.N / 8, p0 = part * 32 * kUnroll + lane;
  const int4* g = reinterpret_cast<const int4*>(a.gate_up) + row * 2 * nvec;
  int4* out = reinterpret_cast<int4*>(a.out) + row * nvec;

  int4 gv[kUnroll][kV], uv[kUnroll][kV];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int v = (p0 + 32 * j) * kV;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      gv[j][k] = uv[j][k] = make_int4(0, 0, 0, 0);
      if (v < nvec) {
        gv[j][k] = ld_stream_v4(g + v + k);
        uv[j][k] = ld_stream_v4(g + nvec + v + k);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int v = (p0 + 32 * j) * kV;
    if (kKeep) {
      float gs, us;
      const uint4 gq = quantise16(reinterpret_cast<const int4(&)[2]>(gv[j]), &gs);
      const uint4 uq = quantise16(reinterpret_cast<const int4(&)[2]>(uv[j]), &us);
      if (v < nvec) {
        int4* q = reinterpret_cast<int4*>(a.out_codes + row * 2 * a.N) + v / 2;
        st_stream_v4(q, *reinterpret_cast<const int4*>(&gq));
        st_stream_v4(q + nvec / 2, *reinterpret_cast<const int4*>(&uq));
        if ((lane & 7) == 0) {
          float* s = a.out_scales + row * (2 * a.N / 128) + v / 16;
          s[0] = gs;
          s[a.N / 128] = us;
        }
      }
    }
    if (v < nvec) {
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        float f[8], u[8];
        unpack_bf16x8(gv[j][k], f);
        unpack_bf16x8(uv[j][k], u);
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = w * silu_times(f[c], u[c]);
        st_stream_v4(out + v + k, pack8(f));
      }
    }
  }
}

// A block takes one slot's row, so that dw is summed in a fixed order.
template <bool kCodes>
__global__ void __launch_bounds__(256) swiglu_grad_kernel(SwigluArgs a) {
  constexpr int kV = kCodes ? 2 : 1;
  pdl_wait_then_release();
  __shared__ float sums[8];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t i = blockIdx.x;
  const int64_t row = slot_row(a, i, tid == 0);
  if (row < 0) {
    if (a.dw && tid == 0) a.dw[i] = 0.0f;
    return;
  }
  const float w = a.w ? a.w[i] : 1.0f;
  const int nvec = a.N / 8, pieces = nvec / kV;
  const int4* dh = reinterpret_cast<const int4*>(a.dh) + row * nvec;
  const int4* src = reinterpret_cast<const int4*>(kCodes ? a.codes + row * 2 * a.N
                                                         : a.gate_up + row * 4 * a.N);
  const float* scale = kCodes ? a.scales + row * (2 * a.N / 128) : nullptr;
  int4* out = reinterpret_cast<int4*>(a.out) + row * 2 * nvec;
  float dot = 0.0f;
  for (int p = tid; p < pieces; p += blockDim.x) {
    int4 dv[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) dv[k] = ld_stream_v4(dh + p * kV + k);
    const int4 gv = ld_stream_v4(src + p), uv = ld_stream_v4(src + pieces + p);
    float g[8 * kV], u[8 * kV];
    if constexpr (kCodes) {
      dequantise16(gv, scale[p >> 3], g);
      dequantise16(uv, scale[a.N / 128 + (p >> 3)], u);
    } else {
      unpack_bf16x8(gv, g);
      unpack_bf16x8(uv, u);
    }
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float d[8], dg[8], du[8];
      unpack_bf16x8(dv[k], d);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x = g[8 * k + c], y = u[8 * k + c];
        // e = exp(-|g|) cannot overflow: s = 1 / (1 + e) or e / (1 + e), and
        // 1 - s is the other of the two, without cancellation
        const float e = expf(-fabsf(x));
        const float r = __fdividef(1.0f, 1.0f + e);
        const float s = x < 0.0f ? e * r : r, o = x < 0.0f ? r : e * r;
        const float silu = x * s;
        dot = fmaf(d[c], silu * y, dot);
        const float wd = w * d[c];
        dg[c] = wd * y * fmaf(silu, o, s);
        du[c] = wd * silu;
      }
      st_stream_v4(out + p * kV + k, pack8(dg));
      st_stream_v4(out + nvec + p * kV + k, pack8(du));
    }
  }
  if (!a.dw) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
  if (lane == 0) sums[tid >> 5] = dot;
  __syncthreads();
  if (tid == 0) {
    for (int j = 1; j < (int)blockDim.x / 32; ++j) dot += sums[j];
    a.dw[i] = dot;
  }
}

// What both directions ask of their sizes and slots.
bool sizes_ok(int inter, int64_t rows, int64_t T, int K, bool codes) {
  if (inter < 8 || inter % (codes ? 128 : 8) || inter > (1 << 24)) return false;
  if (rows < 0 || rows >= (int64_t(1) << 31)) return false;
  return T >= 0 && K >= 1 && K <= EP_MAX_TOPK && T * K < (int64_t(1) << 31);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" ep_status_t ep_ll_swiglu(const void* gate_up, int inter, int64_t num_rows,
                                    const float* topk_weights, int64_t num_tokens, int num_topk,
                                    const int32_t* ll_slot, void* h, uint8_t* codes, float* scales,
                                    int32_t* err_word, ep_stream_t stream) {
  if (!codes != !scales || !sizes_ok(inter, num_rows, num_tokens, num_topk, codes != nullptr))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!ll_slot || (num_rows > 0 && (!gate_up || !h))) return EP_ERR_INVALID_ARG;
  if (!aligned16(gate_up) || !aligned16(h) || !aligned16(codes) || !aligned16(scales))
    return EP_ERR_INVALID_ARG;
  // no output may overlap the input or another output
  const uint64_t n = (uint64_t)num_rows * inter, in = 4 * n, hn = 2 * n, cn = 2 * n, sn = n / 16;
  if (overlap(gate_up, in, h, hn) || overlap(gate_up, in, codes, cn) ||
      overlap(gate_up, in, scales, sn) || overlap(h, hn, codes, cn) || overlap(h, hn, scales, sn) ||
      overlap(codes, cn, scales, sn))
    return EP_ERR_INVALID_ARG;
  SwigluArgs a = {};
  a.gate_up = static_cast<const uint8_t*>(gate_up);
  a.N = inter;
  a.rows = num_rows;
  a.slots = num_tokens * num_topk;
  a.slot = ll_slot;
  a.w = topk_weights;
  a.out = static_cast<uint8_t*>(h);
  a.out_codes = codes;
  a.out_scales = scales;
  a.err = err_word;
  const int per = 32 * kUnroll * 8 * (codes ? 2 : 1);  // channels of a warp
  const int parts = (inter + per - 1) / per;
  const int64_t blocks = (a.slots * parts + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks >= (int64_t(1) << 31)) return EP_ERR_INVALID_ARG;
  if (codes)
    launch_pdl(swiglu_kernel<true>, (unsigned)blocks, kThreads, 0, to_cuda(stream), a, parts);
  else
    launch_pdl(swiglu_kernel<false>, (unsigned)blocks, kThreads, 0, to_cuda(stream), a, parts);
  return launch_status();
}

extern "C" ep_status_t ep_ll_swiglu_backward(const void* dh, const void* gate_up,
                                             const uint8_t* codes, const float* scales, int inter,
                                             int64_t num_rows, const float* topk_weights,
                                             int64_t num_tokens, int num_topk,
                                             const int32_t* ll_slot, void* dgate_up,
                                             float* dweights, int32_t* err_word,
                                             ep_stream_t stream) {
  if (!codes != !scales || (gate_up && codes) ||
      !sizes_ok(inter, num_rows, num_tokens, num_topk, codes != nullptr))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!ll_slot || (num_rows > 0 && (!dh || !dgate_up || (!gate_up && !codes))))
    return EP_ERR_INVALID_ARG;
  if (!aligned16(gate_up) || !aligned16(dh) || !aligned16(codes) || !aligned16(scales) ||
      !aligned16(dgate_up))
    return EP_ERR_INVALID_ARG;
  const uint64_t n = (uint64_t)num_rows * inter;
  if (overlap(dgate_up, 4 * n, dh, 2 * n) || overlap(dgate_up, 4 * n, gate_up, 4 * n) ||
      overlap(dgate_up, 4 * n, codes, 2 * n) || overlap(dgate_up, 4 * n, scales, n / 16))
    return EP_ERR_INVALID_ARG;
  SwigluArgs a = {};
  a.gate_up = static_cast<const uint8_t*>(gate_up);
  a.codes = codes;
  a.scales = scales;
  a.dh = static_cast<const uint8_t*>(dh);
  a.N = inter;
  a.rows = num_rows;
  a.slots = num_tokens * num_topk;
  a.slot = ll_slot;
  a.w = topk_weights;
  a.out = static_cast<uint8_t*>(dgate_up);
  a.dw = dweights;
  a.err = err_word;
  // a thread for each piece of the row, at least a warp and at most 256
  const int pieces = inter / (codes ? 16 : 8);
  const unsigned threads = (unsigned)min(256, (pieces + 31) / 32 * 32);
  if (codes)
    launch_pdl(swiglu_grad_kernel<true>, (unsigned)a.slots, threads, 0, to_cuda(stream), a);
  else
    launch_pdl(swiglu_grad_kernel<false>, (unsigned)a.slots, threads, 0, to_cuda(stream), a);
  return launch_status();
}

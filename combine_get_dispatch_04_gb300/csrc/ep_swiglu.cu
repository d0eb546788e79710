// ep_swiglu.cu -- the experts' gated activation on the rows of the
// expert-major layout, and its gradient, with the input kept in 8 bits.
//
// Forward: h = w * silu(g) * u from rows of [g | u]; the same pass leaves g and
// u as E4M3 codes with one scale per 128 channels, so keeping them costs only
// the bytes written.  Backward: with s = sigmoid(g),
//   dg = w dh u s (1 + g (1 - s)),  du = w dh g s,  dw = sum_n dh g s u.
// The rows are found through the slots, so the weight of a row is the slot's,
// and rows that no slot names are neither read nor written.
//
// Bound by DRAM, with the instructions close behind (some 30 a channel of the gradient).
// Measured: 32768 rows of 2 x 4096 channels with checkpoint, 168 us (its bytes take 162);
// gradient of 262144 rows of 2 x 2048 from codes, 741 us (646), of 131072 from bf16, 420 (401).
#include <cuda_bf16.h>

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

// e = exp(-x) for x = |g|, which cannot overflow, and r = 1 / (1 + e).  With t = -x / ln 2 rounded,
// exp(-x) = 2^t exp(d) for d = -x - t ln 2, what the rounding left (ln 2 in two parts; |d| < 2^-18,
// so exp(d) is 1 + d).  Off by 4 units of 2^-24 at most: 2^-22.5 of the power and the last
// multiply-add's rounding; without d it would be some 1.4 |g| more, which the gradient of the
// weights, a float32 output, shows (55 units at g = -80).  A result below 2^-126 counts as 0.  The
// reciprocal, of a number in [1, 2], is off by 2 units.  (16384 tokens, 2 of 8 experts, 2 x 4096,
// with checkpoint: 168 us, with expf 172, with the power alone 167; gradient of 262144 rows of
// 2 x 2048: 741, 746 and 737 us.)
__device__ __forceinline__ void decay(float g, float& e, float& r) {
  const float x = fminf(fabsf(g), 128.0f);  // an infinity would make d NaN
  const float t = x * -1.44269504f;
  const float d = fmaf(t, 1.90465421e-9f, fmaf(t, -0.693147182f, -x));
  float p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
  e = fmaf(p, d, p);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
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

// The largest magnitude of a block of 128 channels, 8 in each of 16 neighbouring lanes.
__device__ __forceinline__ float block_top(const int4& v) {
  // |x| of finite bf16 is ordered as the low 15 bits, and NaN is above all
  uint32_t m = __vmaxu2(__vmaxu2((uint32_t)v.x & 0x7FFF7FFFu, (uint32_t)v.y & 0x7FFF7FFFu),
                        __vmaxu2((uint32_t)v.z & 0x7FFF7FFFu, (uint32_t)v.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = 8; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(kFull, m, o));
  const float top = __uint_as_float(max(m & 0xFFFFu, m >> 16) << 16);
  return top < 1e-4f ? 1e-4f : top;  // keeps NaN
}
// Codes of 8 channels; inv = 448 / the block's largest magnitude.  Every step is
// rounded as the FP8 dispatch rounds it.  A block with an infinity or a NaN has
// codes that read back as NaN throughout.
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float inv) {
  return make_uint2(cvt_e4m3x4(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv), __fmul_rn(f[2], inv),
                               __fmul_rn(f[3], inv)),
                    cvt_e4m3x4(__fmul_rn(f[4], inv), __fmul_rn(f[5], inv), __fmul_rn(f[6], inv),
                               __fmul_rn(f[7], inv)));
}
__device__ __forceinline__ void dequantise8(const uint2& codes, float scale, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = (i < 2 ? codes.x : codes.y) >> (16 * (i & 1)) & 0xFFFFu;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = v.x * scale;
    f[2 * i + 1] = v.y * scale;
  }
}
__device__ __forceinline__ uint2 ld_stream_v2(const uint2* p) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];"
      : "=r"(v.x), "=r"(v.y)
      : "l"(p));
  return v;
}

// Neighbouring lanes take neighbouring vectors of 8 channels, so that every
// access of a warp fills whole sectors.  (With 16 channels a lane, in two 16-byte
// accesses 32 bytes apart, L2 saw every sector twice: 801 against 753 us for the
// gradient of 262144 rows of 2 x 2048, a warp a row.)
constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // vectors a lane holds at once

// A warp takes 32 * kUnroll vectors of g, and the same of u, of one slot's row.
template <bool kKeep>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluArgs a, int parts) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t i = unit / parts;
  if (i >= a.slots) return;
  const int part = (int)(unit - i * parts);
  const int64_t row = slot_row(a, i, lane == 0 && part == 0);
  if (row < 0) return;
  const float w = a.w ? a.w[i] : 1.0f;
  const int nvec = a.N / 8, v0 = part * 32 * kUnroll + lane;
  const int4* g = reinterpret_cast<const int4*>(a.gate_up) + row * 2 * nvec;
  int4* out = reinterpret_cast<int4*>(a.out) + row * nvec;

  int4 gv[kUnroll], uv[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int v = v0 + 32 * j;
    gv[j] = uv[j] = make_int4(0, 0, 0, 0);
    if (v < nvec) {
      gv[j] = ld_stream_v4(g + v);
      uv[j] = ld_stream_v4(g + nvec + v);
    }
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int v = v0 + 32 * j;
    if (v - lane >= nvec) break;  // the whole warp
    float f[8], u[8];
    unpack_bf16x8(gv[j], f);
    unpack_bf16x8(uv[j], u);
    if (kKeep) {
      // the two blocks' quotients both ways, one division a lane
      const float gt = block_top(gv[j]), ut = block_top(uv[j]);
      const float t = lane & 1 ? ut : gt;
      const bool back = lane & 2;
      const float quotient = __fdiv_rn(back ? t : 448.0f, back ? 448.0f : t);
      const int lane0 = lane & ~3;
      const uint2 gq = quantise8(f, __shfl_sync(kFull, quotient, lane0));
      const uint2 uq = quantise8(u, __shfl_sync(kFull, quotient, lane0 + 1));
      if (v < nvec) {
        uint2* q = reinterpret_cast<uint2*>(a.out_codes + row * 2 * a.N) + v;
        st_stream_v2(q, gq);
        st_stream_v2(q + nvec, uq);
        if ((lane & 14) == 2) {  // lanes 2 and 3 of 16 have the scales of g and u
          float* s = a.out_scales + row * (2 * a.N / 128) + v / 16;
          s[lane & 1 ? a.N / 128 : 0] = quotient;
        }
      }
    }
    if (v < nvec) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float e, r;
        decay(f[c], e, r);
        f[c] = w * (f[c] < 0.0f ? f[c] * e : f[c]) * r * u[c];
      }
      st_stream_v4(out + v, pack8(f));
    }
  }
}

// A warp (kWarpRow) or a block takes one slot's row, so that dw is summed in a
// fixed order.
template <bool kCodes, bool kWarpRow>
__global__ void __launch_bounds__(256) swiglu_grad_kernel(SwigluArgs a) {
  pdl_wait_then_release();
  __shared__ float sums[8];
  const int lane = threadIdx.x & 31;
  const int tid = kWarpRow ? lane : threadIdx.x, threads = kWarpRow ? 32 : blockDim.x;
  const int64_t i = kWarpRow ? (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarpRow && i >= a.slots) return;
  const int64_t row = slot_row(a, i, tid == 0);
  if (row < 0) {
    if (a.dw && tid == 0) a.dw[i] = 0.0f;
    return;
  }
  const float w = a.w ? a.w[i] : 1.0f;
  const int nvec = a.N / 8;
  const int4* dh = reinterpret_cast<const int4*>(a.dh) + row * nvec;
  const uint2* codes = reinterpret_cast<const uint2*>(a.codes) + row * 2 * nvec;
  const int4* gu = reinterpret_cast<const int4*>(a.gate_up) + row * 2 * nvec;
  const float* scale = kCodes ? a.scales + row * (2 * a.N / 128) : nullptr;
  int4* out = reinterpret_cast<int4*>(a.out) + row * 2 * nvec;
  float dot = 0.0f;
#pragma unroll kWarpRow ? 4 : 1
  for (int v = tid; v < nvec; v += threads) {
    const int4 dv = ld_stream_v4(dh + v);
    float g[8], u[8], d[8], dg[8], du[8];
    if constexpr (kCodes) {
      const uint2 gv = ld_stream_v2(codes + v), uv = ld_stream_v2(codes + nvec + v);
      dequantise8(gv, scale[v >> 4], g);
      dequantise8(uv, scale[a.N / 128 + (v >> 4)], u);
    } else {
      const int4 gv = ld_stream_v4(gu + v), uv = ld_stream_v4(gu + nvec + v);
      unpack_bf16x8(gv, g);
      unpack_bf16x8(uv, u);
    }
    unpack_bf16x8(dv, d);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      // s = 1 / (1 + e) or e / (1 + e), and 1 - s is the other of the two,
      // without cancellation
      float e, r;
      decay(g[c], e, r);
      const float s = g[c] < 0.0f ? e * r : r, o = g[c] < 0.0f ? r : e * r;
      const float silu = g[c] * s;
      dot = fmaf(d[c], silu * u[c], dot);
      const float wd = w * d[c];
      dg[c] = wd * u[c] * fmaf(silu, o, s);
      du[c] = wd * silu;
    }
    st_stream_v4(out + v, pack8(dg));
    st_stream_v4(out + nvec + v, pack8(du));
  }
  if (!a.dw) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
  if (!kWarpRow) {
    if (lane == 0) sums[tid >> 5] = dot;
    __syncthreads();
    if (tid == 0)
      for (int j = 1; j < threads / 32; ++j) dot += sums[j];
  }
  if (tid == 0) a.dw[i] = dot;
}

// The gradient gives a row a warp where there are this many slots an SM, or where a row
// has at most this many vectors, else a block.  Warp against block: 4864 rows of 2 x 2048
// channels 16.5 and 18.7 us, 1216 rows 8.6 and 5.7; 1216 rows of 2 x 256, 2.2 and 2.4.
constexpr int kManyRows = 32, kShortRow = 64;

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
  if (!aligned16(gate_up) || !aligned16(h) || !aligned16(codes) || !aligned16(scales) ||
      !aligned4(ll_slot) || !aligned4(topk_weights) || !aligned4(err_word))
    return EP_ERR_INVALID_ARG;
  // no output may overlap an input or another output
  const uint64_t n = (uint64_t)num_rows * inter, in = 4 * n, hn = 2 * n, cn = 2 * n, sn = n / 16;
  const uint64_t slots = (uint64_t)num_tokens * num_topk * 4;
  if (overlap(gate_up, in, h, hn) || overlap(gate_up, in, codes, cn) ||
      overlap(gate_up, in, scales, sn) || overlap(h, hn, codes, cn) || overlap(h, hn, scales, sn) ||
      overlap(codes, cn, scales, sn))
    return EP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(topk_weights), static_cast<const void*>(ll_slot)})
    if (overlap(p, slots, h, hn) || overlap(p, slots, codes, cn) || overlap(p, slots, scales, sn))
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
  const int per = 32 * kUnroll * 8;  // channels of a warp
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
      !aligned16(dgate_up) || !aligned4(ll_slot) || !aligned4(topk_weights) ||
      !aligned4(dweights) || !aligned4(err_word))
    return EP_ERR_INVALID_ARG;
  const uint64_t n = (uint64_t)num_rows * inter, slots = (uint64_t)num_tokens * num_topk * 4;
  const struct {
    const void* p;
    uint64_t n;
  } in[] = {{dh, 2 * n},    {gate_up, 4 * n},        {codes, 2 * n},
            {scales, n / 16}, {topk_weights, slots}, {ll_slot, slots}};
  for (const auto& b : in)
    if (overlap(dgate_up, 4 * n, b.p, b.n) || overlap(dweights, slots, b.p, b.n))
      return EP_ERR_INVALID_ARG;
  if (overlap(dgate_up, 4 * n, dweights, slots)) return EP_ERR_INVALID_ARG;
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
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  cudaStream_t st = to_cuda(stream);
  if (a.slots >= kManyRows * (int64_t)props.sm_count || inter / 8 <= kShortRow) {
    const unsigned blocks = (unsigned)((a.slots + kThreads / 32 - 1) / (kThreads / 32));
    if (codes)
      launch_pdl(swiglu_grad_kernel<true, true>, blocks, kThreads, 0, st, a);
    else
      launch_pdl(swiglu_grad_kernel<false, true>, blocks, kThreads, 0, st, a);
  } else {
    // a thread for each vector of the row, at least a warp and at most 256
    const unsigned threads = (unsigned)min(256, (inter / 8 + 31) / 32 * 32);
    if (codes)
      launch_pdl(swiglu_grad_kernel<true, false>, (unsigned)a.slots, threads, 0, st, a);
    else
      launch_pdl(swiglu_grad_kernel<false, false>, (unsigned)a.slots, threads, 0, st, a);
  }
  return launch_status();
}

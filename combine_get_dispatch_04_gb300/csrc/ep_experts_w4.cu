// ep_experts_w4.cu -- the experts' products with 4-bit weights on the rows of
// the expert-major layout, for few rows per expert.
//
// A warp multiplies 16-row tiles of the weights by up to 8 * NT of the
// expert's rows with mma.sync m16n8k16 (weights as A, rows as B, float32
// accumulators).  The dot product may run over the channels in any order, as
// long as both operands use the same one, and that order is chosen so that
// the stored weights are the A fragment: of 128 channels, thread t of a quad
// takes channels [32 t, 32 t + 32) of its two weight rows, one 16-byte load
// each, and unpacks them in registers.  Nothing passes through shared memory
// but the final sum.  A step of the product is 128 channels, which the warps
// of a block divide among themselves.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ep_experts_w4.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMT = 2;  // 16-row weight tiles per warp (swiglu: one of the gate, one of up)
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes i and i + 4 of the 8 in `w`, as bf16 (128 + q): the bits of q are the
// low mantissa bits of 128.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}

// E4M3 codes c0, c1 (the low halves of `two`) as bf16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// B fragments of 32 channels of one row, in the order of the weights' codes:
// word w of 8 channels gives the pairs (0,4) (1,5) (2,6) (3,7).
template <bool kFP8>
__device__ __forceinline__ void load_row(const uint8_t* p, bool live, uint32_t (&b)[16]) {
  uint32_t x[16];
  if (kFP8) {
    int4 v[2] = {};
    if (live) {
      v[0] = __ldg(reinterpret_cast<const int4*>(p));
      v[1] = __ldg(reinterpret_cast<const int4*>(p) + 1);
    }
    const uint32_t c[8] = {(uint32_t)v[0].x, (uint32_t)v[0].y, (uint32_t)v[0].z, (uint32_t)v[0].w,
                           (uint32_t)v[1].x, (uint32_t)v[1].y, (uint32_t)v[1].z, (uint32_t)v[1].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      // bytes 0..3 of both words: pair (j, j + 4)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[4 * w + j] = e4m3x2_to_bf16x2(
            __byte_perm(c[2 * w], c[2 * w + 1], (uint32_t)(j | ((4 + j) << 4))) & 0xFFFFu);
    }
  } else {
    int4 v[4] = {};
    if (live) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const int4*>(p) + i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = (uint32_t)v[i].x;
      x[4 * i + 1] = (uint32_t)v[i].y;
      x[4 * i + 2] = (uint32_t)v[i].z;
      x[4 * i + 3] = (uint32_t)v[i].w;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      b[4 * w] = __byte_perm(x[4 * w], x[4 * w + 2], 0x5410);
      b[4 * w + 1] = __byte_perm(x[4 * w], x[4 * w + 2], 0x7632);
      b[4 * w + 2] = __byte_perm(x[4 * w + 1], x[4 * w + 3], 0x5410);
      b[4 * w + 3] = __byte_perm(x[4 * w + 1], x[4 * w + 3], 0x7632);
    }
  }
}

// kGroup: 128 (a scale spans a step: it multiplies the float32 sum of the
// step), else 64 or 32 (it multiplies the weights, rounded to bf16 once).
template <int NT, bool kFP8, bool kSwiglu, int kGroup>
__global__ void __launch_bounds__(kThreads) experts_kernel(ExpertsArgs a, int ks) {
  pdl_wait_then_release();
  extern __shared__ float red[];  // [warp][16 * kMT][kPitch], then the live experts
  __shared__ int warp_total[kWarps];
  __shared__ int live_total;
  constexpr int kPitch = 8 * NT + 1;
  uint16_t* live = reinterpret_cast<uint16_t*>(red + kWarps * 16 * kMT * kPitch);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;

  // the experts that have rows, in order
  if (tid == 0) live_total = 0;
  __syncthreads();
  for (int e0 = 0; e0 < a.E; e0 += kThreads) {
    const int e = e0 + tid;
    const int64_t n = e < a.E ? min((int64_t)a.count[e], a.cap) : 0;
    const bool busy = n > 0 && n <= kFewRows;
    const unsigned bal = __ballot_sync(kFull, busy);
    if (lane == 0) warp_total[warp] = __popc(bal);
    __syncthreads();
    int before = live_total;
    for (int w = 0; w < warp; ++w) before += warp_total[w];
    if (busy) live[before + __popc(bal & ((1u << lane) - 1u))] = (uint16_t)e;
    __syncthreads();
    if (tid == kThreads - 1) live_total = before + __popc(bal);
    __syncthreads();
  }
  const int64_t items = (int64_t)live_total * a.tiles;
  const int kw = warp % ks, mw = warp / ks;
  const int steps = (a.I + 127) / 128;
  const int mrows = kSwiglu ? 16 : 16 * kMT;  // output channels per warp
  constexpr int kBytes = kFP8 ? 1 : 2;

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int e = live[item / a.tiles];
    const int tile = (int)(item % a.tiles);
    const int n0 = (tile * (kWarps / ks) + mw) * mrows;
    const int have = (int)min((int64_t)a.count[e], a.cap);

    for (int r0 = 0; r0 < have; r0 += 8 * NT) {
      const int nrows = min(have - r0, 8 * NT);
      float acc[kMT][NT][4] = {};
      const uint8_t* xrow[NT];
      const float* xsc[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int64_t r = (int64_t)e * a.cap + r0 + min(nt * 8 + g, nrows - 1);
        xrow[nt] = a.x + r * a.I * kBytes;
        if (kFP8) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            xsc[nt][c] = a.x_scales + ((int64_t)e * a.cap + r0 + min(nt * 8 + 2 * t4 + c, nrows - 1)) *
                                          (a.I / 128);
        }
      }
      for (int s = kw; s < steps; s += ks) {
        const int k0 = s * 128 + t4 * 32;  // this thread's 32 channels
        const bool kin = k0 < a.I;
        uint4 wv[kMT][2];
        float ws[kMT][2];
        uint32_t zp[kMT][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            int n = n0 + (kSwiglu ? 0 : mt * 16) + h * 8 + g;
            n = min(n, a.N - 1) + (kSwiglu && mt ? a.N : 0);
            const int64_t wrow = (int64_t)e * a.rows + n;
            wv[mt][h] = make_uint4(0, 0, 0, 0);
            ws[mt][h] = 0.0f;
            zp[mt][h] = 0x43084308u;
            if (kin) {
              wv[mt][h] = *reinterpret_cast<const uint4*>(a.q + wrow * (a.I / 2) + k0 / 2);
              const int64_t gi = wrow * (a.I / kGroup) + k0 / kGroup;
              ws[mt][h] = __bfloat162float(a.scales[gi]);
              if (a.zeros) zp[mt][h] = 0x43004300u | (uint32_t)a.zeros[gi] * 0x00010001u;
            }
          }
        }
        uint32_t b[NT][16];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (nt == 0 || nt * 8 < nrows)
            load_row<kFP8>(xrow[nt] + (int64_t)k0 * kBytes, kin && nt * 8 + g < nrows, b[nt]);
        float part[kMT][NT][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const uint32_t w0 = (&wv[mt][0].x)[j], w1 = (&wv[mt][1].x)[j];
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              lo[i] = bf16x2_sub(code_pair(w0, i), zp[mt][0]);
              hi[i] = bf16x2_sub(code_pair(w1, i), zp[mt][1]);
              if (kGroup != 128) {
                const __nv_bfloat162 s0 = __float2bfloat162_rn(ws[mt][0]);
                const __nv_bfloat162 s1 = __float2bfloat162_rn(ws[mt][1]);
                lo[i] = bf16x2_mul(lo[i], *reinterpret_cast<const uint32_t*>(&s0));
                hi[i] = bf16x2_mul(hi[i], *reinterpret_cast<const uint32_t*>(&s1));
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (nt == 0 || nt * 8 < nrows) {
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
                mma_bf16(part[mt][nt], a0, b[nt][4 * j], b[nt][4 * j + 1]);
                mma_bf16(part[mt][nt], a1, b[nt][4 * j + 2], b[nt][4 * j + 3]);
              }
            }
          }
        }
        // the step's sums, scaled in float32: per weight row (a group of 128
        // channels is the step) and per row of x (FP8)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x0 = 1.0f, x1 = 1.0f;
          if (kFP8) {
            x0 = __ldg(xsc[nt][0] + s);
            x1 = __ldg(xsc[nt][1] + s);
          }
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const float s0 = kGroup == 128 ? __shfl_sync(kFull, ws[mt][0], lane & ~3) : 1.0f;
            const float s1 = kGroup == 128 ? __shfl_sync(kFull, ws[mt][1], lane & ~3) : 1.0f;
            acc[mt][nt][0] = fmaf(part[mt][nt][0], s0 * x0, acc[mt][nt][0]);
            acc[mt][nt][1] = fmaf(part[mt][nt][1], s0 * x1, acc[mt][nt][1]);
            acc[mt][nt][2] = fmaf(part[mt][nt][2], s1 * x0, acc[mt][nt][2]);
            acc[mt][nt][3] = fmaf(part[mt][nt][3], s1 * x1, acc[mt][nt][3]);
          }
        }
      }

      // sum over the warps that share the tile, then the epilogue
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            red[(warp * 16 * kMT + mt * 16 + (c >> 1) * 8 + g) * kPitch + nt * 8 + 2 * t4 + (c & 1)] =
                acc[mt][nt][c];
      __syncthreads();
      const int outs = (kWarps / ks) * mrows;  // output channels of the block
      for (int i = tid; i < outs * nrows; i += kThreads) {
        const int ch = i % outs, r = i / outs;
        const int m = ch / mrows, c = ch % mrows;
        const int n = tile * outs + ch;
        float v0 = 0.0f, v1 = 0.0f;
        for (int k = 0; k < ks; ++k) {
          const float* p = red + (m * ks + k) * 16 * kMT * kPitch;
          v0 += p[c * kPitch + r];
          if (kSwiglu) v1 += p[(16 + c) * kPitch + r];
        }
        if (kSwiglu) v0 = v0 / (1.0f + expf(-v0)) * v1;
        if (n < a.N)
          a.y[((int64_t)e * a.cap + r0 + r) * a.N + n] = __float2bfloat16_rn(v0);
      }
      __syncthreads();
    }
  }
}

template <int NT, bool kFP8, bool kSwiglu, int kGroup>
ep_status_t launch_small(ExpertsArgs a, cudaStream_t st) {
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  const int steps = (a.I + 127) / 128;
  int ks = kWarps;  // warps that share one tile
  while (ks > 1 && ks > steps) ks /= 2;
  const int outs = (kWarps / ks) * (kSwiglu ? 16 : 16 * kMT);
  a.tiles = (a.N + outs - 1) / outs;
  const size_t smem = (size_t)kWarps * 16 * kMT * (8 * NT + 1) * 4 + (size_t)a.E * 2;
  static_assert(kWarps * 16 * kMT * 33 * 4 + EP_MAX_EXPERTS * 2 <= 48 * 1024, "shared memory");
  const int64_t most = (int64_t)a.E * a.tiles;
  const unsigned grid = (unsigned)(most < 2 * props.sm_count ? most : 2 * props.sm_count);
  launch_pdl(experts_kernel<NT, kFP8, kSwiglu, kGroup>, grid, kThreads, smem, st, a, ks);
  return launch_status();
}

template <bool kFP8, bool kSwiglu, int kGroup>
ep_status_t launch_rows(const ExpertsArgs& a, cudaStream_t st) {
  if (a.cap <= 8) return launch_small<1, kFP8, kSwiglu, kGroup>(a, st);
  if (a.cap <= 16) return launch_small<2, kFP8, kSwiglu, kGroup>(a, st);
  return launch_small<4, kFP8, kSwiglu, kGroup>(a, st);
}

template <bool kFP8, bool kSwiglu>
ep_status_t launch_group(const ExpertsArgs& a, int group, cudaStream_t st) {
  if (group == 32) return launch_rows<kFP8, kSwiglu, 32>(a, st);
  if (group == 64) return launch_rows<kFP8, kSwiglu, 64>(a, st);
  return launch_rows<kFP8, kSwiglu, 128>(a, st);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" ep_status_t ep_ll_experts_w4(const void* x, int x_fp8, const float* x_scales,
                                        int in_channels, const int32_t* ll_count, int num_experts,
                                        int64_t expert_capacity, const uint8_t* q,
                                        const void* scales, const uint8_t* zeros, int group_size,
                                        int out_channels, int act, void* y, int32_t* err_word,
                                        ep_stream_t stream) {
  if (num_experts < 1 || num_experts > EP_MAX_EXPERTS || expert_capacity < 0 ||
      expert_capacity * (int64_t)num_experts >= (int64_t(1) << 31))
    return EP_ERR_INVALID_ARG;
  if (group_size != 32 && group_size != 64 && group_size != 128) return EP_ERR_INVALID_ARG;
  if (in_channels < group_size || in_channels % group_size || (x_fp8 && in_channels % 128))
    return EP_ERR_INVALID_ARG;
  if (out_channels < 8 || out_channels % 8 || out_channels > (1 << 28)) return EP_ERR_INVALID_ARG;
  if (act != EP_ACT_NONE && act != EP_ACT_SWIGLU) return EP_ERR_INVALID_ARG;
  const bool swiglu = act == EP_ACT_SWIGLU;
  if ((int64_t)num_experts * out_channels * (swiglu ? 2 : 1) >= (int64_t(1) << 31))
    return EP_ERR_INVALID_ARG;
  if (expert_capacity == 0) return EP_OK;
  if (!x || !ll_count || !q || !scales || !y || (x_fp8 && !x_scales)) return EP_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(q) || !aligned16(scales) ||
      !aligned16(zeros) || !aligned16(y) || !aligned16(ll_count))
    return EP_ERR_INVALID_ARG;
  ExpertsArgs a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.x_scales = x_scales;
  a.I = in_channels;
  a.count = ll_count;
  a.E = num_experts;
  a.cap = expert_capacity;
  a.q = q;
  a.scales = static_cast<const __nv_bfloat16*>(scales);
  a.zeros = zeros;
  a.N = out_channels;
  a.rows = swiglu ? 2 * out_channels : out_channels;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.err = err_word;
  cudaStream_t st = to_cuda(stream);
  ep_status_t s;
  if (x_fp8)
    s = swiglu ? launch_group<true, true>(a, group_size, st)
               : launch_group<true, false>(a, group_size, st);
  else
    s = swiglu ? launch_group<false, true>(a, group_size, st)
               : launch_group<false, false>(a, group_size, st);
  return s == EP_OK ? launch_experts_many(a, x_fp8 != 0, swiglu, group_size, st) : s;
}

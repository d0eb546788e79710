// ep_combine_grad.cu -- the gradient of the combine, for the rank-major and
// the expert-major layout.
//
// For every row that a token's slots name: dy = W * dout, one multiply and
// one rounding to bf16, and dweights = <dout, y> in float32.  A block takes
// one token: dout is read once, each of the token's rows of y is read once
// and its row of dy written once, which is all the traffic there is, so the
// kernel is bound by DRAM.  Measured: 131072 tokens of 4096 channels, 64
// experts on 16 ranks, 9.5 GB: 1406 us, 6.8 TB/s (the copy rate); 4096 tokens of
// 7168 channels, eight expert-major rows each, 1.0 GB: 153 us.  512 tokens of
// 256 channels: 3.3 us, the launch.
#include <cuda_bf16.h>

#include "ep_common.cuh"

namespace ep {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xFFFFFFFFu;

struct Args {
  const int4* dout;
  const int4* y;
  int64_t T, rows;
  int nvec;  // 16-byte vectors per row
  const int64_t* topk_idx;  // NULL: expert-major (slot is [T, K])
  const float* w;
  int K, E, El, R;
  const int32_t* slot;
  int4* dy;
  float* dw;
  int32_t* err;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ int4 scale_bf16x8(const float (&f)[8], float w) {
  int4 v;
  v.x = (int)pack_bf16(w * f[0], w * f[1]);
  v.y = (int)pack_bf16(w * f[2], w * f[3]);
  v.z = (int)pack_bf16(w * f[4], w * f[5]);
  v.w = (int)pack_bf16(w * f[6], w * f[7]);
  return v;
}

// The token's distinct rows, their weights (k ascending) and, for every slot,
// which of the rows it names (-1: none).  Run by one warp.
__device__ __forceinline__ int token_rows(const Args& a, int64_t t, int lane, int32_t* row,
                                          float* weight, int32_t* which) {
  const bool in = lane < a.K;
  int32_t r = -1;
  bool bad = false;
  if (in) {
    if (a.topk_idx) {
      const int64_t e = a.topk_idx[t * a.K + lane];
      bad = e < -1 || e >= a.E;
      if (e >= 0 && !bad) r = a.slot[t * a.R + (int)(e / a.El)];
    } else {
      r = a.slot[t * a.K + lane];
    }
  }
  const bool over = r >= a.rows;
  if (r < 0 || over) r = -1;
  if (a.err && (bad || over))
    atomicOr(a.err, (bad ? EP_ERRBIT_BAD_EXPERT : 0) | (over ? EP_ERRBIT_CAPACITY : 0));
  const float w = (in && a.w) ? a.w[t * a.K + lane] : 0.0f;
  const unsigned same = __match_any_sync(kFull, r >= 0 ? r : -1 - lane);
  const bool first = r >= 0 && lane == __ffs(same) - 1;
  const unsigned firsts = __ballot_sync(kFull, first);
  const int mine = __popc(firsts & ((1u << (__ffs(same) - 1)) - 1u));
  float sum = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    const float wk = __shfl_sync(kFull, w, k);
    if (same >> k & 1) sum += wk;
  }
  if (first) {
    row[mine] = r;
    weight[mine] = sum;
  }
  which[lane] = r >= 0 ? mine : -1;
  return __popc(firsts);
}

// NV > 0: the row of dout stays in registers (at most NV vectors a thread);
// NV = 0: it is read again for every row (from L1 or L2).
template <int NV>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(Args a) {
  pdl_wait_then_release();
  __shared__ int32_t row[32], which[32];
  __shared__ float weight[32], part[32][kWarps];
  __shared__ int nrows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  const int4* d = a.dout + t * a.nvec;

  int4 dv[NV > 0 ? NV : 1];
  if (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * kThreads;
      dv[i] = c < a.nvec ? ld_stream_v4(d + c) : make_int4(0, 0, 0, 0);
    }
  }
  if (warp == 0) {
    const int n = token_rows(a, t, lane, row, weight, which);
    if (lane == 0) nrows = n;
  }
  __syncthreads();
  const int n = nrows;
  for (int j = 0; j < n; ++j) {
    const int64_t base = (int64_t)row[j] * a.nvec;
    const float w = weight[j];
    float dot = 0.0f;
    if (NV > 0) {
      int4 yv[NV > 0 ? NV : 1];
      if (a.dw) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = tid + i * kThreads;
          if (c < a.nvec) yv[i] = ld_stream_v4(a.y + base + c);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * kThreads;
        if (c < a.nvec) {
          float f[8], g[8];
          unpack_bf16x8(dv[i], f);
          if (a.dw) {
            unpack_bf16x8(yv[i], g);
#pragma unroll
            for (int h = 0; h < 8; ++h) dot = fmaf(f[h], g[h], dot);
          }
          if (a.dy) st_stream_v4(a.dy + base + c, scale_bf16x8(f, w));
        }
      }
    } else {
      for (int c = tid; c < a.nvec; c += kThreads) {
        float f[8], g[8];
        unpack_bf16x8(d[c], f);
        if (a.dw) {
          unpack_bf16x8(ld_stream_v4(a.y + base + c), g);
#pragma unroll
          for (int h = 0; h < 8; ++h) dot = fmaf(f[h], g[h], dot);
        }
        if (a.dy) st_stream_v4(a.dy + base + c, scale_bf16x8(f, w));
      }
    }
    if (a.dw) {
#pragma unroll
      for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
      if (lane == 0) part[j][warp] = dot;
    }
  }
  if (!a.dw) return;
  __syncthreads();
  if (tid < a.K) {
    const int j = which[tid];
    float sum = 0.0f;
    if (j >= 0) {
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += part[j][i];
    }
    a.dw[t * a.K + tid] = sum;
  }
}

ep_status_t launch(const Args& a, ep_stream_t stream) {
  const unsigned blocks = (unsigned)a.T;
  cudaStream_t st = to_cuda(stream);
  const int nv = (a.nvec + kThreads - 1) / kThreads;
  if (nv <= 1)
    launch_pdl(combine_grad_kernel<1>, blocks, kThreads, 0, st, a);
  else if (nv <= 2)
    launch_pdl(combine_grad_kernel<2>, blocks, kThreads, 0, st, a);
  else if (nv <= 4)
    launch_pdl(combine_grad_kernel<4>, blocks, kThreads, 0, st, a);
  else if (nv <= 8)
    launch_pdl(combine_grad_kernel<8>, blocks, kThreads, 0, st, a);
  else
    launch_pdl(combine_grad_kernel<0>, blocks, kThreads, 0, st, a);
  return launch_status();
}

// The checks both layouts share.
bool grad_ok(const void* dout, const void* y, int hidden, int64_t rows, const float* w, int64_t T,
             const int32_t* slot, const void* dy, const float* dw) {
  if (hidden < 8 || hidden % 8 || rows < 0 || rows >= (int64_t(1) << 31)) return false;
  if (T == 0) return true;
  if (!dout || !slot || !w || !aligned16(dout) || !aligned16(y) || !aligned16(dy)) return false;
  if (dw && !y && rows > 0) return false;
  // a row of dy is written while other tokens still read dout and y
  const uint64_t row = 2 * (uint64_t)hidden;
  return !overlap(dy, rows * row, dout, T * row) && !overlap(dy, rows * row, y, rows * row);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" ep_status_t ep_combine_backward(const void* dout, const void* y, int hidden,
                                           int64_t num_rows, const int64_t* topk_idx,
                                           const float* topk_weights, int64_t num_tokens,
                                           int num_topk, int num_experts, int num_ranks,
                                           const int32_t* slot, void* dy, float* dweights,
                                           int32_t* err_word, ep_stream_t stream) {
  if (!routing_ok_any_t(num_tokens, num_topk, num_experts, num_ranks)) return EP_ERR_INVALID_ARG;
  if (!grad_ok(dout, y, hidden, num_rows, topk_weights, num_tokens, slot, dy, dweights))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0 || (!dy && !dweights)) return EP_OK;
  if (!topk_idx) return EP_ERR_INVALID_ARG;
  Args a = {};
  a.dout = static_cast<const int4*>(dout);
  a.y = static_cast<const int4*>(y);
  a.T = num_tokens;
  a.rows = num_rows;
  a.nvec = hidden / 8;
  a.topk_idx = topk_idx;
  a.w = topk_weights;
  a.K = num_topk;
  a.E = num_experts;
  a.El = num_experts / num_ranks;
  a.R = num_ranks;
  a.slot = slot;
  a.dy = static_cast<int4*>(dy);
  a.dw = dweights;
  a.err = err_word;
  return launch(a, stream);
}

extern "C" ep_status_t ep_ll_combine_backward(const void* dout, const void* y, int hidden,
                                              int64_t num_rows, const float* topk_weights,
                                              int64_t num_tokens, int num_topk,
                                              const int32_t* ll_slot, void* dy, float* dweights,
                                              int32_t* err_word, ep_stream_t stream) {
  if (num_tokens < 0 || num_tokens >= (int64_t(1) << 31) || num_topk < 1 ||
      num_topk > EP_MAX_TOPK)
    return EP_ERR_INVALID_ARG;
  if (!grad_ok(dout, y, hidden, num_rows, topk_weights, num_tokens, ll_slot, dy, dweights))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0 || (!dy && !dweights)) return EP_OK;
  Args a = {};
  a.dout = static_cast<const int4*>(dout);
  a.y = static_cast<const int4*>(y);
  a.T = num_tokens;
  a.rows = num_rows;
  a.nvec = hidden / 8;
  a.w = topk_weights;
  a.K = num_topk;
  a.slot = ll_slot;
  a.dy = static_cast<int4*>(dy);
  a.dw = dweights;
  a.err = err_word;
  return launch(a, stream);
}

// ep_block_norm.cu -- what stands between two blocks: the norm after a block,
// its gate and residual scale, the addition to the residual stream and the norm
// before the next block, in one pass over the row; with the combine of the
// experts' rows in front of it, and its gradient.
//
//   n = y / rms(y) * post,  z = x + scale * gate * n,  h = z / rms(z) * pre
//
// Forward: a block (for short rows a warp) takes one token and keeps its row in
// registers, in 32 bits, between the two sums of squares.  Bound by DRAM: 32768 tokens of
// 7168 channels, bf16, 281 us (its bytes take 281); out of eight expert rows each, 4096
// tokens, 110 us (96); one token 4.8 us, the launch and three passes through the block.
//
// Backward: with d = dh * pre, q = y * post * gate, r = 1 / rms and c = r_z^3
// mean(z d),
//   dx = dz + r_z d - c z                    =: t
//   dy = scale (r_y post gate t - r_y^3 mean(q t) y)
// The sum of q t needs t, and so the sum of z d first; but it is sum(q dz) + r_z sum(q d)
// - c sum(q z), so one reduction of six sums serves both norms.  (r^3 mean(z d) is taken as
// r^2 (r mean(z d)): the cube alone would leave 32 bits at an rms of 1e13 or 1e-13.)  The sums over
// the tokens (of dh z r_z and of t y r_y) stay in the registers of a persistent
// block and are joined by a second kernel in a fixed order.  Bound by DRAM and the
// instructions (some 340 for a vector of 8 channels): 32768 tokens of 7168 channels 478 us
// (421); 997 tokens of 2056, float32, a gate for every channel and token, 18.6 us (8), of which the
// second kernel takes 2 to 4.
#include <cuda_bf16.h>

#include <type_traits>

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
// Asks for 8 values that will be read once, later, and passes them on to L2.
__device__ __forceinline__ void prefetch8(const void* p, bool bf16, int64_t v) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(p) + v * (bf16 ? 16 : 32)));
}
__device__ __forceinline__ float weight1(const void* p, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}

// 32 bytes at once, on a 32-byte boundary.
__device__ __forceinline__ void ld_stream_32(const void* p, int4 (&v)[2]) {
  asm("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y),
        "=r"(v[1].z), "=r"(v[1].w)
      : "l"(p));
}
__device__ __forceinline__ void st_stream_32(void* p, const float (&f)[8]) {
  asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
               "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

// The same of memory that this kernel may write later: not through the read-only path.
__device__ __forceinline__ void ld_written_32(const void* p, int4 (&v)[2]) {
  asm volatile(
      "ld.global.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y),
        "=r"(v[1].z), "=r"(v[1].w)
      : "l"(p));
}
__device__ __forceinline__ int4 ld_written_16(const int4* p) {
  int4 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight values of the stream, read once.  Float32 ones are two 16-byte pieces, or one of 32 where
// the buffer allows it: L2 sees every sector twice otherwise.  kWritten: the kernel may write
// them in place, each thread its own after it has read them.
template <bool kF32>
struct Stream8 {
  int4 v[kF32 ? 2 : 1];
  template <bool kWritten>
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const int4* q = static_cast<const int4*>(p) + at * (kF32 ? 2 : 1);
    if constexpr (kF32) {
      if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {  // the same for all threads
        if (kWritten)
          ld_written_32(q, v);
        else
          ld_stream_32(q, v);
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < (kF32 ? 2 : 1); ++i) v[i] = kWritten ? ld_written_16(q + i) : ld_stream_v4(q + i);
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
      if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        st_stream_32(q, f);
        return;
      }
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
__device__ __forceinline__ void block_sums(float (&v)[kN], float (*part)[kN], int warps) {
  const int lane = threadIdx.x & 31;
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

// z and h of token t from its block output y (in 32 bits; of each of `threads` threads
// NV vectors) and its stream.
template <int NV, bool kF32>
__device__ __forceinline__ void finish_row(const NormArgs& a, int64_t t, int tid, int threads,
                                           float (&y)[NV][8], const Stream8<kF32> (&xv)[NV],
                                           float (*part)[kMaxWarps][1]) {
  const int64_t base = t * a.nvec;
  if (a.z) {
    float f = a.scale;
    if (a.gate_kind == kGateToken) f *= weight1(a.gate, a.bf16, t);
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) s[0] = fmaf(y[i][c], y[i][c], s[0]);
      block_sums<1>(s, part[0], threads >> 5);
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
  block_sums<1>(s, part[1], threads >> 5);
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

// The block's output given per token: a block a token, or (kWarpRow) a warp,
// NV vectors of 8 channels a thread.
constexpr int kRowWarps = 4;  // of a block whose warps have a token each
template <int NV, bool kF32, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? kRowWarps * 32 : 512) norm_kernel(NormArgs a) {
  pdl_wait_then_release();
  __shared__ float part[2][kMaxWarps][1];
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x, threads = kWarpRow ? 32 : blockDim.x;
  const int64_t t =
      kWarpRow ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (kWarpRow && t >= a.T) return;
  const int64_t base = t * a.nvec;
  Stream8<kF32> xv[NV];
  int4 yv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * threads;
    xv[i].zero();
    yv[i] = make_int4(0, 0, 0, 0);
    if (v < a.nvec) {
      xv[i].template load<true>(a.x, base + v);  // z may be x
      if (a.y) yv[i] = ld_stream_v4(reinterpret_cast<const int4*>(a.y) + base + v);
    }
  }
  if (a.gate_kind == kGateFull) {
    for (int v = tid; v < a.nvec; v += threads) prefetch8(a.gate, a.bf16, base + v);
  }
  float y[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) unpack_bf16x8(yv[i], y[i]);
  finish_row<NV, kF32>(a, t, tid, threads, y, xv, part);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ int4 lds128(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// The experts' rows combined first.  A block stays and takes every
// gridDim-th token; what it reads is one sequence of rows (a token's live rows, then its
// row of the stream), of which several are on their way with asynchronous
// copies, each thread's vectors into a place of its own.  The rows of
// the tokens ahead come from lists that the first warp makes before they are read.
// (4096 tokens of 7168 channels, eight rows each: 109 us with 3 or 4 ahead, 116 with 2, 113 with 5.)
constexpr int kRowsAhead = 3;
constexpr int kLists = 8;

struct RowList {
  int n;                            // live rows
  float weight[EP_MAX_TOPK];
  const int4* row[EP_MAX_TOPK + 2]; // and the stream's: its row, or (float32) the two
                                    // 16-byte halves of its vectors
};

// Slot `lane` of token t: its row and weight (-1: none).
__device__ __forceinline__ void load_slot(const NormArgs& a, int64_t t, int lane, int32_t& row,
                                          float& weight) {
  row = -1;
  weight = 1.0f;
  if (t < a.T && lane < a.K) {
    row = __ldg(a.slot + t * a.K + lane);
    if (a.w) weight = __ldg(a.w + t * a.K + lane);
  }
}
// What token t reads, by one warp that holds its slots.
template <int kS>
__device__ __forceinline__ void make_list(const NormArgs& a, int64_t t, int lane, int32_t row,
                                          float weight, RowList& l) {
  const bool over = row >= a.rows;
  if (over && a.err) atomicOr(a.err, EP_ERRBIT_CAPACITY);
  const bool live = row >= 0 && !over;
  const unsigned all = __ballot_sync(kFull, live);
  const int n = __popc(all);
  if (live) {
    const int at = __popc(all & ((1u << lane) - 1u));
    l.row[at] = reinterpret_cast<const int4*>(a.y) + (int64_t)row * a.nvec;
    l.weight[at] = weight;
  }
  if (lane < kS) l.row[n + lane] = static_cast<const int4*>(a.x) + t * a.nvec * kS + lane;
  if (lane == 0) l.n = n;
}

template <int NV, bool kF32>
__global__ void __launch_bounds__(512) norm_rows_kernel(NormArgs a) {
  // every token has a row of the sequence at least, so while a token's rows are taken
  // those of at most kAhead tokens after it are on their way
  constexpr int kAhead = kRowsAhead, kS = kF32 ? 2 : 1;
  static_assert(kAhead + 2 <= kLists, "a list is written while kAhead + 1 others are read");
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[2][kMaxWarps][1];
  __shared__ RowList lists[kLists];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  const int64_t stride = gridDim.x;
  const auto token = [&](int j) { return blockIdx.x + j * stride; };  // of this block
  const int mine = (int)((a.T - blockIdx.x + stride - 1) / stride);

  for (int j = tid >> 5; j < kAhead + 1; j += threads >> 5) {
    int32_t row;
    float weight;
    load_slot(a, token(j), lane, row, weight);
    make_list<kS>(a, token(j), lane, row, weight, lists[j]);
  }
  int32_t next_row = -1;
  float next_weight = 1.0f;
  if (tid < 32) load_slot(a, token(kAhead + 1), lane, next_row, next_weight);
  __syncthreads();

  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = tid + i * threads < a.nvec;
  const uint32_t piece = threads * 16, first = smem_addr(ring) + tid * 16;
  const uint32_t end = first + (kAhead + 1) * NV * piece;  // of this thread's places
  int load_j = 0, load_k = 0;
  uint32_t load_at = first, take_at = first;
  const auto issue = [&]() {
    if (load_j < mine) {
      const RowList& l = lists[load_j % kLists];
      const int n = l.n;
      const int4* p = l.row[load_k];
      const int64_t step = load_k < n ? 1 : kS;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) copy16(load_at + i * piece, p + (tid + i * threads) * step);
      if (++load_k == n + kS) {
        load_k = 0;
        ++load_j;
      }
    }
    load_at += NV * piece;
    if (load_at == end) load_at = first;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) issue();

  const auto take = [&](int4 (&v)[NV]) {  // the next row of the sequence
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = in[i] ? lds128(take_at + i * piece) : make_int4(0, 0, 0, 0);
    take_at += NV * piece;
    if (take_at == end) take_at = first;
    issue();  // into the place that the row before left
  };
  for (int j = 0; j < mine; ++j) {
    __syncthreads();  // the lists and `part` of the token before are no longer read
    if (tid < 32) {
      make_list<kS>(a, token(j + kAhead + 1), lane, next_row, next_weight,
                    lists[(j + kAhead + 1) % kLists]);
      load_slot(a, token(j + kAhead + 2), lane, next_row, next_weight);
    }
    float y[NV][8] = {};
    const RowList& l = lists[j % kLists];
    const int n = l.n;
    for (int k = 0; k < n; ++k) {
      const float w = l.weight[k];
      int4 v[NV];
      take(v);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        unpack_bf16x8(v[i], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) y[i][c] = fmaf(w, f[c], y[i][c]);
      }
    }
    Stream8<kF32> xv[NV];
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      int4 v[NV];
      take(v);
#pragma unroll
      for (int i = 0; i < NV; ++i) xv[i].v[k] = v[i];
    }
    if (a.comb) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * threads;
        if (v < a.nvec)
          st_stream_v4(reinterpret_cast<int4*>(a.comb) + token(j) * a.nvec + v, pack8(y[i]));
      }
    }
    finish_row<NV, kF32>(a, token(j), tid, threads, y, xv, part);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Rows of at most 8 * kRowThreads channels: a thread has one vector of 8, whose weights
// and sums over the tokens stay in registers.  A block takes every gridDim-th
// token and keeps the next ones' vectors on their way with asynchronous copies
// into places of the thread's own.  A row has two halves, the sums and what is
// made of them, with a barrier between; where three rows fit into shared memory, the
// barrier of one row is hidden behind the second half of the row before.
constexpr int kRowThreads = 896;

// The six sums of a row: z z, y y, z d, q dz, q d, q z.
constexpr int kSums = 6;

// Two channels.
using Pair = float2;
__device__ __forceinline__ Pair make_pair(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ Pair mul2(Pair a, float b) { return make_float2(a.x * b, a.y * b); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ Pair fma2(Pair a, float b, Pair c) {
  return make_float2(fmaf(a.x, b, c.x), fmaf(a.y, b, c.y));
}
__device__ __forceinline__ float dot2(Pair a, Pair b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, c));
}
// Channels 2 i and 2 i + 1 of a vector.
__device__ __forceinline__ Pair pair_of(const int4& v, int i) {
  const uint32_t w = (uint32_t)(&v.x)[i];
  return make_pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool kF32>
__device__ __forceinline__ Pair pair_of(const Stream8<kF32>& v, int i) {
  if constexpr (kF32)
    return make_pair(__int_as_float((&v.v[i >> 1].x)[2 * (i & 1)]),
                     __int_as_float((&v.v[i >> 1].x)[2 * (i & 1) + 1]));
  else
    return pair_of(v.v[0], i);
}
__device__ __forceinline__ uint32_t pack2(Pair p) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(p.x, p.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

constexpr int kMaxRing = 220 << 10;  // bytes of a block's rows in shared memory
template <bool kF32>
constexpr int kGradPieces = kF32 ? 6 : 4;  // 16-byte pieces of a thread's vectors of a row

// kStages: rows in shared memory, 3 (one row's second half with the next one's first) or 2.
// kH: with dh (the norm before the next block), kY: with y (the norm after the block or a gate),
// kPost: with the norm after the block.  Without that y is not part of its own gradient, not even
// as 0 y, which is NaN where y is not finite.  (A branch instead of instances for that: 16384 tokens
// of 7168, float32, 395 against 379 us.  In the sums a branch on the weight is the faster: with
// instances 16384 tokens of 4096, float32, 204 against 188 us, of spills.)
template <bool kF32, bool kFullGate, int kStages, bool kH, bool kY, bool kPost>
__global__ void __launch_bounds__(kRowThreads, 1) norm_grad_row_kernel(NormArgs a) {
  constexpr int kPieces = kGradPieces<kF32>, kS = kF32 ? 2 : 1;
  constexpr bool kOverlap = kStages == 3;
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[2][32][8];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int warps = threads >> 5;
  const bool in = tid < a.nvec;
  const int v = in ? tid : a.nvec - 1;
  Pair pre[4], q[4];  // the channels' weights; q: post * gate
  {
    float p[8], w[8], g[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) p[c] = 0.0f, w[c] = g[c] = 1.0f;
    if (kH) weight8(a.pre, a.bf16, v, p);
    if (a.post) weight8(a.post, a.bf16, v, w);
    if (a.gate_kind == kGateChannel) weight8(a.gate, a.bf16, v, g);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      pre[k] = make_pair(p[2 * k], p[2 * k + 1]);
      q[k] = make_pair(w[2 * k] * g[2 * k], w[2 * k + 1] * g[2 * k + 1]);
    }
  }
  Pair cpre[4] = {}, cpost[4] = {};  // sums over this block's tokens

  // A row in shared memory: z, dz, y and dh, each in the threads' order.  Of float32 inputs
  // a warp's 32 lanes copy neighbouring 16-byte pieces, not each its own two (L2
  // would see every sector twice).
  const uint32_t base = smem_addr(ring), piece = threads * 16;
  const auto place = [&](int stage, int array) {  // array 0..3, of this thread
    const uint32_t from = base + stage * kPieces * piece;
    return array < 2 ? from + (array * piece + tid * 16) * kS
                     : from + (2 * kS + array - 2) * piece + tid * 16;
  };
  // what is never copied (no such input, no such channel) is 0 throughout
#pragma unroll 1
  for (int i = 0; i < kStages * 4; ++i) {
    const int k = i & 3;
    if (in && (k == 1 ? a.dz != nullptr : k == 2 ? kY && a.y : kH)) continue;
    for (int j = 0; j < (k < 2 ? kS : 1); ++j)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(place(i >> 2, k) + j * 16),
                   "r"(0)
                   : "memory");
  }
  const auto copy = [&](int stage, int64_t t) {
    if (t < a.T) {
      const int64_t i = t * a.nvec + tid;
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        // piece k * 32 + lane of the warp's
        const int at = kS == 1 ? tid : warp * 64 + k * 32 + lane;
        if (at < a.nvec * kS) {
          const int64_t from = t * a.nvec * kS + at;
          const uint32_t to = (at - tid * kS) * 16;
          if (kH) copy16(place(stage, 0) + to, static_cast<const int4*>(a.x) + from);
          if (a.dz) copy16(place(stage, 1) + to, static_cast<const int4*>(a.dz) + from);
        }
      }
      if (kY && in && a.y) copy16(place(stage, 2), reinterpret_cast<const int4*>(a.y) + i);
      if (kFullGate && in) prefetch8(a.gate, a.bf16, i);
      if (kH && in) copy16(place(stage, 3), reinterpret_cast<const int4*>(a.dh) + i);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  struct Vectors {
    Stream8<kF32> z, dz;
    int4 y, dh;
  };
  const auto take = [&](int stage, Vectors& r) {
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      r.z.v[k] = lds128(place(stage, 0) + k * 16);
      r.dz.v[k] = lds128(place(stage, 1) + k * 16);
    }
    r.y = lds128(place(stage, 2));
    r.dh = lds128(place(stage, 3));
  };
  const auto arrived = [&](auto pending) {  // all but the last `pending` rows
    asm volatile("cp.async.wait_group %0;" ::"n"(decltype(pending)::value) : "memory");
    if (kF32) __syncwarp();  // other lanes' copies too
  };
  const auto again = [&](int stage, int64_t t) {  // a row into the place of one that was read
    if (kF32) __syncwarp();
    copy(stage, t);
  };
  const auto full_gate = [&](int64_t t, Pair (&g)[4]) {
    float f[8];
    weight8(a.gate, a.bf16, t * a.nvec + v, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) g[k] = make_pair(f[2 * k], f[2 * k + 1]);
  };

  // The row's sums, this warp's part.  A warp folds the six values into each other:
  // after the steps over 16, 8 and 4 lanes a lane holds one of eight (the last two are nothing).
  const auto first_half = [&](int64_t t, int stage, int turn) {
    float s[8] = {};
    Vectors r;
    take(stage, r);
    Pair g[4];
    if (kFullGate) full_gate(t, g);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Pair z = pair_of(r.z, k), y = pair_of(r.y, k), d = mul2(pair_of(r.dh, k), pre[k]);
      if (kH) {
        s[0] = dot2(z, z, s[0]);
        s[2] = dot2(z, d, s[2]);
      }
      if (kY) {
        Pair p = mul2(y, q[k]);
        if (kFullGate) p = mul2(p, g[k]);
        s[1] = dot2(y, y, s[1]);
        s[3] = dot2(p, pair_of(r.dz, k), s[3]);
        if (kH) {
          s[4] = dot2(p, d, s[4]);
          s[5] = dot2(p, z, s[5]);
        }
      }
    }
#pragma unroll
    for (int h = 4; h; h >>= 1) {
      const bool upper = lane & (4 * h);
#pragma unroll
      for (int k = 0; k < h; ++k) {
        const float give = upper ? s[k] : s[k + h], keep = upper ? s[k + h] : s[k];
        s[k] = keep + __shfl_xor_sync(kFull, give, 4 * h);
      }
    }
    s[0] += __shfl_xor_sync(kFull, s[0], 2);
    s[0] += __shfl_xor_sync(kFull, s[0], 1);
    if ((lane & 3) == 0) part[turn][warp][lane >> 2] = s[0];
  };
  // After the barrier: lane l adds up value l % 8 of the warps.
  float rz, cz, fr, cy;
  const auto join = [&](int64_t t, int turn) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; i += 4)
      if (i + (lane >> 3) < warps) u += part[turn][i + (lane >> 3)][lane & 7];
    u += __shfl_xor_sync(kFull, u, 8);
    u += __shfl_xor_sync(kFull, u, 16);
    float s[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) s[i] = __shfl_sync(kFull, u, i);
    const float inv_h = 1.0f / (float)a.H;
    rz = kH ? rsqrtf(s[0] * inv_h + a.eps) : 0.0f;
    cz = rz * rz * (rz * (s[2] * inv_h));
    const float ry = a.post ? rsqrtf(s[1] * inv_h + a.eps) : 1.0f;
    const float qt = s[3] + rz * s[4] - cz * s[5];  // sum of q t
    const float f = a.scale * (a.gate_kind == kGateToken ? weight1(a.gate, a.bf16, t) : 1.0f);
    fr = f * ry;
    cy = a.post ? f * (ry * ry) * (ry * (qt * inv_h)) : 0.0f;
    if (a.gate_kind == kGateToken && tid == 0 && a.dgate)
      static_cast<float*>(a.dgate)[t] = a.scale * ry * qt;
  };
  // The row's outputs and its share of the sums over the tokens.
  const auto second_half = [&](int64_t t, int stage) {
    if (!in) return;
    Vectors r;
    take(stage, r);
    const int64_t i = t * a.nvec + tid;
    Pair g[4], tt[kF32 ? 4 : 1], dg[kFullGate ? 4 : 1];
    if (kFullGate) full_gate(t, g);
    int4 dx4, dy4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      Pair tk = pair_of(r.dz, k);  // the gradient of x
      if (kH) {
        const Pair z = pair_of(r.z, k), hr = mul2(pair_of(r.dh, k), rz);
        tk = fma2(hr, pre[k], fma2(z, -cz, tk));
        cpre[k] = fma2(hr, z, cpre[k]);
      }
      Pair u = mul2(tk, fr);
      if (kY) {
        const Pair y = pair_of(r.y, k);
        if constexpr (kFullGate) {
          dg[k] = mul2(mul2(u, y), q[k]);
          u = mul2(u, g[k]);
        }
        cpost[k] = fma2(u, y, cpost[k]);  // without the channel's gate, which the second kernel knows
        u = kPost ? fma2(u, q[k], mul2(y, -cy)) : mul2(u, q[k]);
      }
      (&dy4.x)[k] = (int)pack2(u);
      if (kF32)
        tt[kF32 ? k : 0] = tk;
      else
        (&dx4.x)[k] = (int)pack2(tk);
    }
    const auto store8 = [&](void* p, const Pair* w) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[2 * k] = w[k].x, f[2 * k + 1] = w[k].y;
      Stream8<true>::store(p, i, f);
    };
    if constexpr (kF32)
      store8(a.dx, tt);
    else
      st_stream_v4(static_cast<int4*>(a.dx) + i, dx4);
    if (a.dy) st_stream_v4(reinterpret_cast<int4*>(a.dy) + i, dy4);
    if constexpr (kFullGate) {
      if (a.dgate && a.bf16)
        st_stream_v4(static_cast<int4*>(a.dgate) + i,
                     make_int4((int)pack2(dg[0]), (int)pack2(dg[1]), (int)pack2(dg[2]),
                               (int)pack2(dg[3])));
      else if (a.dgate)
        store8(a.dgate, dg);
    }
  };
  const int64_t step = gridDim.x;
  int64_t t = blockIdx.x;
  copy(0, t);
  copy(1, t + step);
  if (kOverlap) {
    copy(2, t + 2 * step);
    arrived(std::integral_constant<int, 2>());
    first_half(t, 0, 0);
    __syncthreads();
    join(t, 0);
    int turn = 1, stage = 0;  // of row t
    while (true) {
      const int next = stage == 2 ? 0 : stage + 1;
      const bool more = t + step < a.T;
      if (more) {
        arrived(std::integral_constant<int, 1>());
        first_half(t + step, next, turn);
      }
      second_half(t, stage);
      if (!more) break;
      again(stage, t + 3 * step);
      t += step;
      stage = next;
      __syncthreads();
      join(t, turn);
      turn ^= 1;
    }
  } else {
    for (int turn = 0; t < a.T; t += step, turn ^= 1) {
      arrived(std::integral_constant<int, 1>());
      first_half(t, turn, turn);
      __syncthreads();
      join(t, turn);
      second_half(t, turn);
      again(turn, t + 2 * step);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!a.part || !in) return;
  float4* p = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * 2 * a.H) + 2 * tid;
  p[0] = make_float4(cpre[0].x, cpre[0].y, cpre[1].x, cpre[1].y);
  p[1] = make_float4(cpre[2].x, cpre[2].y, cpre[3].x, cpre[3].y);
  p += a.H / 4;
  p[0] = make_float4(cpost[0].x, cpost[0].y, cpost[1].x, cpost[1].y);
  p[1] = make_float4(cpost[2].x, cpost[2].y, cpost[3].x, cpost[3].y);
}

// Longer rows: NV vectors a thread, loaded when their token's turn comes.  Bound by that wait and by
// spills (the values of four vectors take more than the 128 registers, some 650 bytes): 8192 tokens of
// 8192 channels 408 us (their bytes 120), float32 464 (180), of 16384 channels 681 (240).
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
        if (a.dh) zv[i].template load<false>(a.x, base + v);
        if (a.dz) dzv[i].template load<false>(a.dz, base + v);
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
    block_sums<6>(s, part[turn], threads >> 5);
    const float rz = a.dh ? rsqrtf(s[0] * inv_h + a.eps) : 0.0f;
    const float cz = rz * rz * (rz * (s[2] * inv_h));
    const float ry = a.post ? rsqrtf(s[1] * inv_h + a.eps) : 1.0f;
    const float qt = s[3] + rz * s[4] - cz * s[5];  // sum of q t
    const float f = a.scale * gt;
    const float cy = a.post ? f * (ry * ry) * (ry * (qt * inv_h)) : 0.0f;
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

// The blocks' sums, added up channel by channel: kChannels channels of one of the two a
// block, its warps over the blocks of the first kernel, a batch of loads at once.
constexpr int kColumnWarps = 16, kColumnBatch = 16;
template <int kChannels>
__global__ void __launch_bounds__(kColumnWarps * 32) norm_columns_kernel(NormArgs a, int blocks) {
  constexpr int kRows = 32 / kChannels;  // that a warp reads at once
  pdl_wait_then_release();
  __shared__ float sum[kColumnWarps][kChannels];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x * kChannels + lane % kChannels, which = blockIdx.y;
  float s = 0.0f;
  if (h < a.H) {
    const float* p = a.part + which * a.H + h;
    constexpr int kStep = kColumnWarps * kRows;
    for (int b0 = warp * kRows + lane / kChannels; b0 < blocks; b0 += kStep * kColumnBatch) {
      float v[kColumnBatch];
#pragma unroll
      for (int i = 0; i < kColumnBatch; ++i) {
        const int b = b0 + i * kStep;
        v[i] = b < blocks ? p[(int64_t)b * 2 * a.H] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kColumnBatch; ++i) s += v[i];
    }
  }
#pragma unroll
  for (int o = kChannels; o < 32; o <<= 1) s += __shfl_xor_sync(kFull, s, o);
  if (lane < kChannels) sum[warp][lane] = s;
  __syncthreads();
  if (warp || lane >= kChannels || h >= a.H) return;
#pragma unroll
  for (int i = 1; i < kColumnWarps; ++i) s += sum[i][lane];
  if (which == 0) {
    if (a.dpre) a.dpre[h] = s;
    return;
  }
  const bool channel = a.gate_kind == kGateChannel;
  if (a.dpost) a.dpost[h] = channel ? s * weight1(a.gate, a.bf16, h) : s;
  if (channel && a.dgate)
    static_cast<float*>(a.dgate)[h] = a.post ? s * weight1(a.post, a.bf16, h) : s;
}

// Rows from here on take 32 channels a block, shorter ones 8, whose first kernel has more
// blocks to add up (8 against 32, both kernels: 23887 tokens of 480 channels 38.0 and 42.7 us, 4096 of
// 1024 18.7 and 20.0, 997 of 2056 19.7 and 18.8, 1024 of 7168 31.3 and 27.6).
constexpr int kWideColumns = 2048;

// Vectors a thread and threads a row for rows of nvec vectors.
struct Shape {
  int nv, threads;
};
// A warp for rows of up to 128 vectors, else a block (16266 tokens of 360 channels: 8.9 and
// 17.2 us).
Shape forward_shape(int nvec) {
  if (nvec <= 128) return {nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4, 32};
  const int nv = nvec <= 256 ? 2 : 4;
  return {nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}
Shape rows_shape(int nvec) {
  const int nv = nvec <= 128 ? 1 : nvec <= 1024 ? 2 : 4;
  return {nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}
// One vector a thread, or four for rows beyond that.
Shape backward_shape(int nvec) {
  const int nv = nvec <= kRowThreads ? 1 : 4;
  return {nv, ((nvec + nv - 1) / nv + 31) / 32 * 32};
}
// Blocks that stay for the whole of the work, the same number on every SM: as many
// threads as registers allow, and three tokens a block at least (997 tokens of 2056 channels: 20.4 us with
// two on an SM, 23.6 with one, 25.9 with three).
int backward_blocks(int64_t T, int threads, int sm_count) {
  const int most = kRowThreads / threads < 1 ? 1 : kRowThreads / threads < 16 ? kRowThreads / threads : 16;
  const int64_t want = T / (3 * sm_count);
  const int64_t blocks = (int64_t)sm_count * (want < 1 ? 1 : want < most ? want : most);
  return (int)(T < blocks ? T : blocks);
}

template <bool kF32, bool kFullGate, int kStages, bool kH, bool kY, bool kPost>
bool launch_backward_parts(const NormArgs& a, int blocks, int threads, cudaStream_t st) {
  constexpr int kThreadBytes = kStages * kGradPieces<kF32> * 16;
  const auto kernel = norm_grad_row_kernel<kF32, kFullGate, kStages, kH, kY, kPost>;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev] &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxRing) != cudaSuccess)
      return false;
    done[dev] = true;
  }
  return launch_pdl(kernel, (unsigned)blocks, threads, (size_t)threads * kThreadBytes, st, a) ==
         cudaSuccess;
}
// A full gate comes with y.  Without dh and without y (which then counts as 0) the
// gradient of the block's output is a product.
template <bool kF32, bool kFullGate, int kStages>
bool launch_backward_stages(const NormArgs& a, int blocks, int threads, cudaStream_t st) {
  if constexpr (!kFullGate) {
    if (a.dh && !a.post && a.gate_kind == kGateNone)
      return launch_backward_parts<kF32, false, kStages, true, false, false>(a, blocks, threads, st);
  }
  if (a.post)
    return a.dh ? launch_backward_parts<kF32, kFullGate, kStages, true, true, true>(a, blocks, threads, st)
                : launch_backward_parts<kF32, kFullGate, kStages, false, true, true>(a, blocks, threads, st);
  return a.dh ? launch_backward_parts<kF32, kFullGate, kStages, true, true, false>(a, blocks, threads, st)
              : launch_backward_parts<kF32, kFullGate, kStages, false, true, false>(a, blocks, threads, st);
}
template <bool kF32, bool kFullGate>
bool launch_backward_rows(const NormArgs& a, int blocks, int threads, cudaStream_t st) {
  if constexpr (3 * kGradPieces<kF32> * 16 * kRowThreads > kMaxRing) {
    if (3 * kGradPieces<kF32> * 16 * threads > kMaxRing)
      return launch_backward_stages<kF32, kFullGate, 2>(a, blocks, threads, st);
  }
  return launch_backward_stages<kF32, kFullGate, 3>(a, blocks, threads, st);
}

template <int NV, bool kF32>
bool launch_rows(const NormArgs& a, int threads, const DeviceProps& props, cudaStream_t st) {
  const auto kernel = norm_rows_kernel<NV, kF32>;
  const size_t smem = (size_t)(kRowsAhead + 1) * NV * threads * 16;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev] && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (kRowsAhead + 1) * NV * 512 * 16) != cudaSuccess)
      return false;
    done[dev] = true;
  }
  // blocks that fit an SM by shared memory (and 6 KB for each block's own) and threads
  int per = (int)(props.smem_per_sm / (smem + 6144));
  per = per < 1024 / threads ? per : 1024 / threads;
  per = per < 1 ? 1 : per > 32 ? 32 : per;
  const int64_t blocks = (int64_t)per * props.sm_count;
  return launch_pdl(kernel, (unsigned)(a.T < blocks ? a.T : blocks), threads, smem, st, a) ==
         cudaSuccess;
}
template <int NV, bool kF32>
bool launch_forward(const NormArgs& a, int threads, const DeviceProps& props, cudaStream_t st) {
  if (a.slot) return launch_rows<NV, kF32>(a, threads, props, st);
  if (threads == 32)
    return launch_pdl(norm_kernel<NV, kF32, true>, (unsigned)((a.T + kRowWarps - 1) / kRowWarps),
                      kRowWarps * 32, 0, st, a) == cudaSuccess;
  if constexpr (NV > 1)
    return launch_pdl(norm_kernel<NV, kF32, false>, (unsigned)a.T, threads, 0, st, a) == cudaSuccess;
  return false;
}

struct Buffer {
  const void* p;
  uint64_t n;
};
// Whether an output overlaps an input or another output.
template <int kIn, int kOut>
bool any_overlap(const Buffer (&in)[kIn], const Buffer (&out)[kOut]) {
  for (int i = 0; i < kOut; ++i) {
    for (const Buffer& b : in)
      if (overlap(out[i].p, out[i].n, b.p, b.n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
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
  if (!aligned16(x) || !aligned16(y) || !aligned16(z) || !aligned16(h) || !aligned16(combined) ||
      !aligned4(ll_slot) || !aligned4(topk_weights) || !aligned4(err_word))
    return EP_ERR_INVALID_ARG;
  // a token's outputs are written while others still read: nothing may overlap,
  // but z may be x itself, which each token reads before it writes
  const uint64_t n = (uint64_t)num_tokens * hidden, xs = n * (stream_f32 ? 4 : 2);
  const uint64_t each = weights_bf16 ? 2 : 4;
  const uint64_t gate_size = gate_kind == kGateFull      ? n
                             : gate_kind == kGateChannel ? hidden
                             : gate_kind == kGateToken   ? num_tokens
                                                         : 0;
  const Buffer in[] = {{z == x ? nullptr : x, xs},
                       {y, (uint64_t)a.rows * hidden * 2},
                       {gate, gate_size * each},
                       {post_weight, hidden * each},
                       {pre_weight, hidden * each},
                       {topk_weights, ll_slot ? (uint64_t)num_tokens * num_topk * 4 : 0},
                       {ll_slot, ll_slot ? (uint64_t)num_tokens * num_topk * 4 : 0}};
  const Buffer out[] = {{z, xs}, {h, 2 * n}, {combined, 2 * n}};
  if (any_overlap(in, out) || overlap(h, 2 * n, x, xs) || overlap(combined, 2 * n, x, xs))
    return EP_ERR_INVALID_ARG;
  const Shape s = ll_slot ? rows_shape(a.nvec) : forward_shape(a.nvec);
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  cudaStream_t st = to_cuda(stream);
  const bool ok =
      stream_f32 ? (s.nv == 1   ? launch_forward<1, true>(a, s.threads, props, st)
                    : s.nv == 2 ? launch_forward<2, true>(a, s.threads, props, st)
                                : launch_forward<4, true>(a, s.threads, props, st))
                 : (s.nv == 1   ? launch_forward<1, false>(a, s.threads, props, st)
                    : s.nv == 2 ? launch_forward<2, false>(a, s.threads, props, st)
                                : launch_forward<4, false>(a, s.threads, props, st));
  if (!ok) {
    cudaGetLastError();
    return EP_ERR_CUDA;
  }
  return EP_OK;
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
  const uint64_t each = weights_bf16 ? 2 : 4;
  const uint64_t gate_size = gate_kind == kGateFull      ? n
                             : gate_kind == kGateChannel ? hidden
                             : gate_kind == kGateToken   ? num_tokens
                                                         : 0;
  const Buffer in[] = {{dz, ss},
                       {dh, 2 * n},
                       {z, ss},
                       {y, 2 * n},
                       {gate, gate_size * each},
                       {post_weight, hidden * each},
                       {pre_weight, hidden * each}};
  const Buffer out[] = {{dx, ss},
                        {dy, 2 * n},
                        {dgate, gate_size * (gate_kind == kGateFull ? each : 4)},
                        {dpost_weight, hidden * 4ull},
                        {dpre_weight, hidden * 4ull},
                        {columns ? workspace : nullptr, workspace_bytes}};
  if (any_overlap(in, out)) return EP_ERR_INVALID_ARG;
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  const Shape s = backward_shape(a.nvec);
  const int blocks = backward_blocks(num_tokens, s.threads, props.sm_count);
  if (columns) {
    if (!workspace || workspace_bytes < (size_t)blocks * 2 * hidden * sizeof(float))
      return EP_ERR_CAPACITY;
    a.part = static_cast<float*>(workspace);
  }
  bool ok;
  if (s.nv == 1) {
    const bool full = gate_kind == kGateFull;
    ok = stream_f32 ? (full ? launch_backward_rows<true, true>(a, blocks, s.threads, st)
                            : launch_backward_rows<true, false>(a, blocks, s.threads, st))
                    : (full ? launch_backward_rows<false, true>(a, blocks, s.threads, st)
                            : launch_backward_rows<false, false>(a, blocks, s.threads, st));
  } else {
    ok = (stream_f32 ? launch_pdl(norm_grad_kernel<4, true>, (unsigned)blocks, s.threads, 0, st, a)
                     : launch_pdl(norm_grad_kernel<4, false>, (unsigned)blocks, s.threads, 0, st,
                                  a)) == cudaSuccess;
  }
  if (ok && columns)
    ok = (hidden < kWideColumns
              ? launch_pdl(norm_columns_kernel<8>, dim3((unsigned)(hidden / 8), 2),
                           kColumnWarps * 32, 0, st, a, blocks)
              : launch_pdl(norm_columns_kernel<32>, dim3((unsigned)((hidden + 31) / 32), 2),
                           kColumnWarps * 32, 0, st, a, blocks)) == cudaSuccess;
  if (!ok) {
    cudaGetLastError();
    return EP_ERR_CUDA;
  }
  return EP_OK;
}

// ep_experts_w4.cu -- the experts' products with 4-bit weights on the rows of
// the expert-major layout, for few rows per expert.
//
// A warp multiplies a tile of 64 weight rows (swiglu: 32 of the gate and the
// same 32 of the up projection) by up to 8 rows of x with mma.sync m16n8k16
// (weights as A, rows as B, float32 accumulators): at a few rows the tensor
// rate is not what counts, and A can come from registers.  The dot product may
// run over the channels in any order, as long as both operands use the same
// one.  A step is 128 channels; thread t of a quad takes the t-th quarter of
// every 64 channels (32 where those have a scale of their own), so that one
// matrix step never mixes groups, and unpacks the codes of its bytes without
// moving them to another thread.  The sums of a group are scaled in float32;
// no weight is rounded.
//
// Codes become integers less their zero point before they are multiplied: in
// bf16 from 128 + q (the bits of q are the low mantissa bits of 128), in f16
// beside E4M3 rows, both exact.  (Multiplying 128 + q and taking (128 + zero)
// * sum(x) off afterwards takes 7 instructions for 8 bf16 codes instead of 11
// and 509 us instead of 531 below, but its sums round at some 30 times the
// size of the products, and overflow before them.)
//
// The floor is the stream of the codes, which the copies alone reach (306 us
// for 256 experts of 7168 x 2048); what bounds it is the warps' own time: about
// 670 instructions a step, two cycles each for those of the integer pipe, and the
// latencies that four warps a scheduler leave open (the register file holds
// no more).  So every warp keeps two steps on their way with asynchronous
// copies, across the ends of its tiles, pointers advance instead of being
// computed, and lanes without a row of x read the last one instead of zeros
// (their columns are not stored).  The warps of a block share a tile by its
// channels when there are too few tiles for all warps.
//
// Measured at 256 experts of 2048 -> 7168 channels (1.9 GB of codes), about two
// rows each: 531 us with groups of 128 (3.5 TB/s), 566-595 us with groups of 64
// and zero points; 7168 -> 2048 channels, 457 us, E4M3 rows 409 us.  One token,
// 8 experts, gate and up of 2048 x 7168: 40.3 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ep_experts_w4.cuh"

namespace ep {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xFFFFFFFFu;

constexpr int kMT = 4;                     // 16-row weight tiles per warp
constexpr int kTileRows = kMT * 16;
constexpr int kStages = 3;                 // of a warp's codes
constexpr int kStage = kTileRows * 64;     // bytes of codes of a step
constexpr int kScales = kTileRows * 12;    // of a warp: scales and zero points of four groups
constexpr int kSmem = kWarps * (kStages * kStage + kScales);

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// (a & b) | c in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Codes i and i + 4 of the 8 in w (i = 0..3) less their zero point, as bf16:
// 0x4300 | q is 128 + q; zp = 128 + zero, both exact, and so is the difference.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t zp, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(v), "r"(zp));
  }
}
// The same as f16: 0x6400 | q is 1024 + q, and with q in
// the next four bits 1024 + 16 q, so two of four need no shift.
// low = -(1024 + zero), high = -(64 + zero), as f16 pairs.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t low, uint32_t high,
                                          uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i ? w >> 8 : w;
    const uint32_t a = and_or(v, 0x000F000Fu, 0x64006400u), b = and_or(v, 0x00F000F0u, 0x64006400u);
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * i]) : "r"(a), "r"(low));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[2 * i + 1]) : "r"(b), "r"(0x2C002C00u), "r"(high));
  }
}

// The B fragments of 8 channels: the pairs (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ void pairs_bf16(const uint4& x, uint32_t (&b)[4]) {
  b[0] = __byte_perm(x.x, x.z, 0x5410);
  b[1] = __byte_perm(x.x, x.z, 0x7632);
  b[2] = __byte_perm(x.y, x.w, 0x5410);
  b[3] = __byte_perm(x.y, x.w, 0x7632);
}
__device__ __forceinline__ void pairs_e4m3(const uint2& x, uint32_t (&b)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = __byte_perm(x.x, x.y, (uint32_t)(j | (4 + j) << 4));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFF), __NV_E4M3);
    b[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// First channel, within a step, of word j (8 channels) of thread t of a quad:
// the t-th quarter of every 64 channels, or of every 32 where those have
// scales of their own.
template <int kGroup>
__device__ __forceinline__ int word_channel(int t, int j) {
  return kGroup == 32 ? j * 32 + t * 8 : (j >> 1) * 64 + t * 16 + (j & 1) * 8;
}

// The 16-byte chunks of a staged weight row are permuted by its place among
// eight rows, so that the loads of fragments meet no bank twice.
__device__ __forceinline__ int chunk_swizzle(int g) { return (g & 2) | (g >> 2 & 1); }

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Row i * 8 + g of a tile of weight rows, relative to the tile's
// first: rows beyond the last channel read the last one (32-bit indices and
// one multiply-add an address, instead of a pointer for each row).
template <bool kSwiglu>
__device__ __forceinline__ uint32_t tile_row(int i, int g, int last, int N) {
  if (!kSwiglu) return (uint32_t)min(g + 8 * i, last);
  return i < kMT ? (uint32_t)min(g + 8 * i, last) : (uint32_t)(min(g + 8 * (i - kMT), last) + N);
}

// What a warp reads with its own lanes for the products of a tile; pointers
// to x and its scales advance from step to step.
struct Sources {
  const uint8_t* x;             // the row of x: this lane's channels
  const float* xs;              // scales of the expert's E4M3 rows, and which two
  uint32_t xrow[2];
  const __nv_bfloat16* scale;   // scales and zero points of the tile's first row
  const uint8_t* zero;
  int last;                     // last row of the tile that is a channel
};

// Scales and zero points of four groups of a tile's rows.  A lane loads those
// of rows lane and lane + 32 while a step is multiplied, and puts them
// into shared memory after it: 64 rows of 4 scales, then 64 of 4 zero points.
// Where every thread loads what it needs itself, each step, 16 loads and their
// addresses (677 us, with groups of 64 and zero points, against 610).
struct Scales {
  uint2 s[2];
  uint32_t z[2];
};
// Where the row's groups come in fours they are aligned to be read at once;
// else one by one, groups beyond the row's end as any.
template <bool kSwiglu, bool kZeros>
__device__ __forceinline__ void load_scales(const Sources& src, int g0, int lane, int N,
                                            uint32_t groups, Scales& v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t at =
        (uint64_t)tile_row<kSwiglu>((lane >> 3) + 4 * i, lane & 7, src.last, N) * groups + g0;
    const uint16_t* u = reinterpret_cast<const uint16_t*>(src.scale) + at;
    const uint8_t* z = src.zero + at;
    if (groups % 4 == 0) {
      v.s[i] = __ldg(reinterpret_cast<const uint2*>(u));
      if (kZeros) v.z[i] = __ldg(reinterpret_cast<const uint32_t*>(z)) & 0x0F0F0F0Fu;
    } else {
      uint32_t f[4], w = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = g0 + q < (int)groups ? q : 0;
        f[q] = __ldg(u + k);
        if (kZeros) w |= (uint32_t)__ldg(z + k) << (8 * q);
      }
      v.s[i] = make_uint2(f[0] | f[1] << 16, f[2] | f[3] << 16);
      if (kZeros) v.z[i] = w & 0x0F0F0F0Fu;
    }
  }
}
template <bool kZeros>
__device__ __forceinline__ void store_scales(uint32_t at, int lane, const Scales& v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = lane + 32 * i;
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + row * 8), "r"(v.s[i].x),
                 "r"(v.s[i].y) : "memory");
    if (kZeros)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + kTileRows * 8 + row * 4), "r"(v.z[i])
                   : "memory");
  }
}

// The products of step s of a tile.  ragged: channels end within the step.
template <bool kFP8, bool kSwiglu, int kGroup, bool kZeros>
__device__ __forceinline__ void step_products(const ExpertsArgs& a, const Sources& src,
                                              int s, bool ragged, uint32_t stage,
                                              uint32_t scales, int lane, float (&acc)[kMT][4]) {
  constexpr int kPer = 128 / kGroup;
  const int g = lane >> 2, t = lane & 3;
  // everything that comes from global memory goes out before the wait for
  // the codes
  uint4 xv[kFP8 ? 2 : 4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // word_channel less this thread's own offset, which the pointer holds
    const int k = word_channel<kGroup>(0, j);
    if (kFP8) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src.x + k));
      (&xv[j >> 1].x)[(j & 1) * 2] = v.x;
      (&xv[j >> 1].x)[(j & 1) * 2 + 1] = v.y;
    } else if (!ragged) {
      xv[kFP8 ? 0 : j] = __ldg(reinterpret_cast<const uint4*>(src.x + 2 * k));
    } else {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (s * 128 + word_channel<kGroup>(t, j) < a.I)
        v = __ldg(reinterpret_cast<const uint4*>(src.x + 2 * k));
      xv[kFP8 ? 0 : j] = v;
    }
  }
  float xs[2] = {1.0f, 1.0f};
  if (kFP8) {
    xs[0] = __ldg(src.xs + src.xrow[0]);
    xs[1] = __ldg(src.xs + src.xrow[1]);
  }
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
  __syncwarp();

  // this thread's first row, this step's first group of the four
  const int in = kPer == 4 ? 0 : s * kPer & (4 - kPer);
  const uint32_t scale0 = scales + g * 8 + in * 2;
  const uint32_t zero0 = scales + kTileRows * 8 + g * 4 + in;
  float part[kMT][4] = {};
  uint32_t z[kMT][2];
  uint2 w[kMT][2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int q = j / (4 / kPer);  // the word's group
    if (j % (4 / kPer) == 0) {
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          z[mt][h] = kZeros ? lds8(zero0 + mt * 64 + h * 32 + q) : 8;
    }
    uint32_t b[4];
    if (kFP8) {
      const uint4 v = xv[j >> 1];
      pairs_e4m3(j & 1 ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y), b);
    } else {
      pairs_bf16(xv[kFP8 ? 0 : j], b);
    }
    const int byte = word_channel<kGroup>(t, j) / 2;
    const uint32_t at = stage + ((byte >> 4 ^ chunk_swizzle(g)) << 4) + (byte & 15) + g * 64;
    if (kGroup == 32 || j % 2 == 0) {  // else the words lie side by side
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kGroup == 32)
            w[mt][h].x = lds32(at + mt * 1024 + h * 512);
          else
            w[mt][h] = lds64(at + mt * 1024 + h * 512);
        }
    }
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      const bool second = kGroup != 32 && j % 2;
      const uint32_t w0 = second ? w[mt][0].y : w[mt][0].x, w1 = second ? w[mt][1].y : w[mt][1].x;
      const uint32_t z0 = z[mt][0], z1 = z[mt][1];
      uint32_t lo[4], hi[4];
      if (kFP8) {
        // -(1024 + z) and -(64 + z) as f16: 0xE400 | z, 0xD400 | z << 4
        codes_f16(w0, 0xE400E400u | z0 * 0x00010001u, 0xD400D400u | z0 * 0x00100010u, lo);
        codes_f16(w1, 0xE400E400u | z1 * 0x00010001u, 0xD400D400u | z1 * 0x00100010u, hi);
        mma_f16(part[mt], lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
        mma_f16(part[mt], lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
      } else {
        codes_bf16(w0, 0x43004300u | z0 * 0x00010001u, lo);
        codes_bf16(w1, 0x43004300u | z1 * 0x00010001u, hi);
        mma_bf16(part[mt], lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
        mma_bf16(part[mt], lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
      }
    }
    if ((j + 1) % (4 / kPer) == 0) {  // the end of a group
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const float s0 = __uint_as_float(lds16(scale0 + mt * 128 + q * 2) << 16);
        const float s1 = __uint_as_float(lds16(scale0 + mt * 128 + 64 + q * 2) << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = kFP8 ? part[mt][i] * xs[i & 1] : part[mt][i];
          acc[mt][i] = fmaf(v, i < 2 ? s0 : s1, acc[mt][i]);
          part[mt][i] = 0.0f;
        }
      }
    }
  }
}

// A warp's place in its sequence of tiles and steps; one for the copies and,
// some steps behind, one for the products.
struct Cursor {
  int item, s, e, n0;  // tile and step; the tile's expert and first output channel
};

template <bool kFP8, bool kSwiglu, int kGroup, bool kZeros>
__global__ void __launch_bounds__(kThreads, 2) experts_kernel(ExpertsArgs a) {
  constexpr int kChannels = kSwiglu ? kTileRows / 2 : kTileRows;  // output channels of a tile
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t smem[];  // stages, then the live experts
  __shared__ int warp_total[kWarps];
  __shared__ int live_total;
  __shared__ int used_slot[kWarps];  // the stage of a warp's last step
  uint16_t* live = reinterpret_cast<uint16_t*>(smem + kSmem);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;

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
  const int steps = (a.I + 127) / 128, groups = a.I / kGroup;
  const int items = live_total * a.tiles;
  // warps per tile: what leaves the busiest warp the fewest steps
  int ks = 1;
  {
    const int warps = (int)gridDim.x * kWarps;
    int64_t best = (int64_t)((items + warps - 1) / warps) * steps;
    for (int k = 2; k <= kWarps && k <= steps; k *= 2) {
      const int64_t most = (int64_t)((items * (int64_t)k + warps - 1) / warps) * ((steps + k - 1) / k);
      if (most < best) {
        best = most;
        ks = k;
      }
    }
  }
  const int kw = warp % ks, team = warp / ks, teams = kWarps / ks;
  const int first = blockIdx.x * teams + team, stride = gridDim.x * teams;
  const uint32_t stage0 = smem_addr(smem) + warp * kStages * kStage;
  const uint32_t scales = smem_addr(smem) + kWarps * kStages * kStage + warp * kScales;

  const auto enter = [&](Cursor& c) {
    if (c.item < items) {
      c.e = live[c.item / a.tiles];
      c.n0 = c.item % a.tiles * kChannels;
    }
    c.s = kw;
  };
  Cursor load, use;
  load.item = use.item = first;
  enter(load);
  enter(use);
  const uint8_t* codes;  // this lane's chunk of the tile's first row at load.s
  int last = 0;
  const auto point = [&]() {
    codes = a.q + ((int64_t)load.e * a.rows + load.n0) * (a.I / 2) + load.s * 64 + t * 16;
    last = min(kChannels, a.N - load.n0) - 1;
  };
  if (load.item < items) point();
  const uint32_t chunk = (uint32_t)(g * 64 + ((t ^ chunk_swizzle(g)) << 4));
  const auto issue = [&](uint32_t stage) {
    if (load.item < items) {
      // beyond the last channel: any bytes of the row, x is zero there
      const uint8_t* p = load.s * 128 + t * 32 < a.I ? codes : codes - load.s * 64 - t * 16;
#pragma unroll
      for (int i = 0; i < 2 * kMT; ++i)
        copy16(stage + chunk + i * 512,
               p + (uint64_t)tile_row<kSwiglu>(i, g, last, a.N) * (uint32_t)(a.I / 2));
      codes += ks * 64;
      load.s += ks;
      if (load.s >= steps) {
        load.item += stride;
        enter(load);
        if (load.item < items) point();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(stage0 + i * kStage);
  int slot = 0;

  while (use.item < items) {
    const int nrows = (int)min((int64_t)a.count[use.e], a.cap);
    Sources src;
    {
      const int64_t row = (int64_t)use.e * a.cap;
      const int64_t at = ((int64_t)use.e * a.rows + use.n0) * groups;
      src.x = a.x + ((row + min(g, nrows - 1)) * a.I + use.s * 128 + word_channel<kGroup>(t, 0)) *
                        (kFP8 ? 1 : 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) src.xrow[i] = (uint32_t)(min(2 * t + i, nrows - 1) * steps);
      src.xs = kFP8 ? a.x_scales + row * steps + use.s : nullptr;
      src.scale = a.scales + at;
      src.zero = a.zeros + at;
      src.last = min(kChannels, a.N - use.n0) - 1;
    }
    float acc[kMT][4] = {};
    constexpr int kPer = 128 / kGroup;
    Scales sc;
    if (use.s < steps) {
      load_scales<kSwiglu, kZeros>(src, use.s * kPer & ~3, lane, a.N, groups, sc);
      __syncwarp();
      store_scales<kZeros>(scales, lane, sc);
    }
    for (; use.s < steps; use.s += ks) {
      const int next = (use.s + ks) * kPer & ~3;
      const bool fresh = next != (use.s * kPer & ~3) && use.s + ks < steps;
      if (fresh) load_scales<kSwiglu, kZeros>(src, next, lane, a.N, groups, sc);
      step_products<kFP8, kSwiglu, kGroup, kZeros>(a, src, use.s, !kFP8 && use.s * 128 + 128 > a.I,
                                                   stage0 + slot * kStage, scales, lane, acc);
      src.x += ks * 128 * (kFP8 ? 1 : 2);
      src.xs += ks;
      __syncwarp();
      if (fresh) store_scales<kZeros>(scales, lane, sc);
      issue(stage0 + (slot == 0 ? kStages - 1 : slot - 1) * kStage);
      slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    __nv_bfloat16* y = a.y + (int64_t)use.e * a.cap * a.N;
    if (ks > 1) {
      // the team's sums meet in shared memory: each warp's in the stage that
      // its last step used (the next copy into it is a step away)
      if (lane == 0) used_slot[warp] = slot == 0 ? kStages - 1 : slot - 1;
      __syncwarp();
      const auto sums = [&](int w) {
        return reinterpret_cast<float*>(smem + (w * kStages + used_slot[w]) * kStage);
      };
      float* mine = sums(warp);
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(mine + (mt * 16 + h * 8 + g) * 8 + 2 * t) =
              make_float2(acc[mt][2 * h], acc[mt][2 * h + 1]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(ks * 32) : "memory");
      for (int i = kw * 32 + lane; i < kChannels * nrows; i += ks * 32) {
        const int ch = i % kChannels, r = i / kChannels;
        float v0 = 0.0f, v1 = 0.0f;
        for (int k = 0; k < ks; ++k) {
          const float* p = sums(team * ks + k);
          v0 += p[ch * 8 + r];
          if (kSwiglu) v1 += p[(kChannels + ch) * 8 + r];
        }
        if (kSwiglu) v0 = silu_times(v0, v1);
        if (use.n0 + ch < a.N) y[(int64_t)r * a.N + use.n0 + ch] = __float2bfloat16_rn(v0);
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(ks * 32) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1), ch = use.n0 + (i >> 1) * 8 + g;
        if (r >= nrows) continue;
#pragma unroll
        for (int mt = 0; mt < (kSwiglu ? kMT / 2 : kMT); ++mt) {
          float v = acc[mt][i];
          if (kSwiglu) v = silu_times(v, acc[mt + kMT / 2][i]);
          if (ch + mt * 16 < a.N) y[(int64_t)r * a.N + ch + mt * 16] = __float2bfloat16_rn(v);
        }
      }
    }
    use.item += stride;
    enter(use);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <bool kFP8, bool kSwiglu, int kGroup, bool kZeros>
ep_status_t launch_small(ExpertsArgs a, cudaStream_t st) {
  const auto kernel = experts_kernel<kFP8, kSwiglu, kGroup, kZeros>;
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  static std::mutex mu;
  static int resident[64] = {};  // blocks per SM, at a few hundred experts
  int dev = -1, blocks = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EP_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (resident[dev] == 0) {
      int n = 0;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmem + EP_MAX_EXPERTS * 2) != cudaSuccess ||
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, kSmem + 1024) !=
              cudaSuccess ||
          n < 1)
        return EP_ERR_CUDA;
      resident[dev] = n;
    }
    blocks = resident[dev];
  }
  constexpr int kChannels = kTileRows / (kSwiglu ? 2 : 1);
  a.tiles = (a.N + kChannels - 1) / kChannels;
  launch_pdl(kernel, (unsigned)(blocks * props.sm_count), kThreads, kSmem + (size_t)a.E * 2, st, a);
  return launch_status();
}

template <bool kFP8, bool kSwiglu, int kGroup>
ep_status_t launch_zeros(const ExpertsArgs& a, cudaStream_t st) {
  return a.zeros ? launch_small<kFP8, kSwiglu, kGroup, true>(a, st)
                 : launch_small<kFP8, kSwiglu, kGroup, false>(a, st);
}

template <bool kFP8, bool kSwiglu>
ep_status_t launch_group(const ExpertsArgs& a, int group, cudaStream_t st) {
  if (group == 32) return launch_zeros<kFP8, kSwiglu, 32>(a, st);
  if (group == 64) return launch_zeros<kFP8, kSwiglu, 64>(a, st);
  return launch_zeros<kFP8, kSwiglu, 128>(a, st);
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
  // rows of y are written while other tiles still read x
  const uint64_t all = (uint64_t)num_experts * expert_capacity;
  if (overlap(y, all * out_channels * 2, x, all * in_channels * (x_fp8 ? 1 : 2)))
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

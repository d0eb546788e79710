// ep_experts_w4_tc.cu -- the experts' products with 4-bit weights for experts
// with many rows: tcgen05 with the weights as operand A in tensor memory.
//
// D[channel][row] = sum over one group of (q - zero) * x: the codes less
// their zero point are small integers, exact in bf16 and in E4M3, so A holds
// them unscaled and the tensor cores add exact products in float32.  A
// group's sums are then read from tensor memory, multiplied by the group's
// scale (and, for E4M3 rows, the scale of the row's 128 channels) and added
// to float32 accumulators in registers: no weight is ever rounded, and E4M3
// rows are multiplied as they are, at the 8-bit rate.
//
// A block takes 128 weight rows (swiglu: 64 of the gate and the same 64 of
// the up projection) times up to 256 rows of x, as two halves of up to 128
// rows, so that one half's sums are read while the other's are computed:
//   warp 0      TMA of the x tiles (128 channels x the rows, swizzled 128 B)
//   warp 1      tensor memory, and the tcgen05.mma of both halves
//   warp 2      TMA of the weight codes (128 rows x 64 bytes)
//   warp 3      the scales of E4M3 rows, into shared memory
//   warps 4-7   codes -> integers -> operand A in tensor memory
//   warps 8-15  sums of a half -> scaled -> registers; the epilogue
// Every wait is bounded; a block whose wait runs out reports
// EP_ERRBIT_TIMEOUT and leaves.
#include <cuda.h>

#include "ep_experts_w4.cuh"

namespace ep {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256;      // rows of x per block, two halves
constexpr int kHalf = 128;
constexpr int kBoxRows = 32;    // rows per TMA box of x
constexpr int kSlotsA = 4;      // operand A slots of 128 channels in tensor memory
constexpr int kSlotsS = 8;      // slots of row scales
constexpr int kWBytes = 8192;   // 128 weight rows x 64 bytes
constexpr unsigned kFull = 0xFFFFFFFFu;

template <bool kFP8>
struct Cfg {
  static constexpr int kXBytes = kRows * (kFP8 ? 128 : 256);  // a stage of 128 channels
  static constexpr int kStagesX = kFP8 ? 4 : 3;
  static constexpr int kStagesW = kFP8 ? 10 : 3;
  static constexpr int kColsA = kFP8 ? 32 : 64;  // tensor-memory columns per slot of A
  static constexpr int kSmem =
      1024 + kStagesX * kXBytes + kStagesW * kWBytes + (kFP8 ? kSlotsS * kRows * 4 : 0);
};

struct Barriers {
  uint64_t xfull[4], xempty[4], wfull[10], wempty[10], afull[kSlotsA], aempty[kSlotsA], pfull[2],
      pempty[2], sfull[kSlotsS], sempty[kSlotsS];
};

// --- the items of a block ----------------------------------------------------
struct Item {
  int e, tile, r0, rows, nh;  // nh: rows of a half, a multiple of 16
};

// Walks the experts with more than kFewRows rows; item numbers run over the
// experts, their chunks of rows, and the tiles of channels, tiles innermost.
struct Walk {
  const int32_t* count;
  int64_t cap;
  int E, tiles;
  int e = -1, n = 0, chunks = 0;
  int64_t base = 0, items = 0;

  __device__ Walk(const ExpertsArgs& a) : count(a.count), cap(a.cap), E(a.E), tiles(a.tiles) {}

  __device__ bool at(int64_t item, Item* it) {
    while (item >= base + items) {
      base += items;
      if (++e >= E) return false;
      n = (int)min((int64_t)__ldg(count + e), cap);
      chunks = n > kFewRows ? (n + kRows - 1) / kRows : 0;
      items = (int64_t)chunks * tiles;
    }
    const int local = (int)(item - base);
    const int chunk = local / tiles, size = (n + chunks - 1) / chunks;
    it->e = e;
    it->tile = local - chunk * tiles;
    it->r0 = chunk * size;
    it->rows = min(size, n - it->r0);
    it->nh = max(16, ((it->rows + 1) / 2 + 15) / 16 * 16);
    return true;
  }
};

// --- PTX ----------------------------------------------------------------------
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

// D (+)= A (tensor memory) * B (shared memory, K-major, 128-byte swizzle)
template <bool kFP8>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                    bool accumulate) {
  if (kFP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// Shared-memory descriptor of a K-major tile with 128-byte swizzle: 8-row
// groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)64 << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}

// two float32 at once
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}

// --- codes -> operand A ---------------------------------------------------------
// Eight codes as four bf16 pairs in channel order: byte j of the word holds
// the pair (2j, 2j + 1); 0x4300 | q is 128 + q, less 128 + zero.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t zp, uint32_t* out) {
  const uint32_t odd = w >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = __byte_perm(w, odd, (uint32_t)(j | j << 4 | (4 + j) << 8 | (4 + j) << 12));
    const uint32_t v = (two & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(out[j]) : "r"(v), "r"(zp));
  }
}

// Eight codes as E4M3 bytes, looked up in the 16 bytes of (q - zero).
__device__ __forceinline__ void codes_e4m3(uint32_t w, const uint4& t, uint32_t* out) {
  const uint32_t idx = w & 0x77777777u, high = (w >> 3) & 0x11111111u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t i = h ? idx >> 16 : idx, m = h ? high >> 16 : high;
    const uint32_t lo = __byte_perm(t.x, t.y, i), hi = __byte_perm(t.z, t.w, i);
    const uint32_t mask = __byte_perm(0x0000FF00u, 0, m);
    out[h] = (lo & ~mask) | (hi & mask);
  }
}

// The E4M3 code of an integer of at most 15 in magnitude.
__device__ __forceinline__ uint32_t e4m3_of_int(int v) {
  const int m = v < 0 ? -v : v;
  if (m == 0) return 0;
  const int p = 31 - __clz(m);  // m = 2^p * (1 + frac), three fraction bits hold it
  return (uint32_t)((v < 0 ? 0x80 : 0) | (7 + p) << 3 | ((m << 3 >> p) & 7));
}

template <bool kFP8, bool kSwiglu, int kGroup>
__global__ void __launch_bounds__(kThreads, 1)
    experts_tc_kernel(ExpertsArgs a, const __grid_constant__ CUtensorMap xmap,
                      const __grid_constant__ CUtensorMap wmap) {
  using C = Cfg<kFP8>;
  constexpr int kPerBlock = 128 / kGroup;  // groups in a step of 128 channels
  constexpr int kMmaPerGroup = kGroup / (kFP8 ? 32 : 16);
  extern __shared__ uint8_t raw[];
  __shared__ Barriers bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ uint4 tables[16];  // E4M3 of (q - zero), one 16-byte table per zero point

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = base;
  uint8_t* sw = sx + C::kStagesX * C::kXBytes;
  float* ss = reinterpret_cast<float*>(sw + C::kStagesW * kWBytes);

  if (tid == 0) {
    for (int i = 0; i < C::kStagesX; ++i) mbar_init(&bar.xfull[i], 1), mbar_init(&bar.xempty[i], 1);
    for (int i = 0; i < C::kStagesW; ++i) mbar_init(&bar.wfull[i], 1), mbar_init(&bar.wempty[i], 4);
    for (int i = 0; i < kSlotsA; ++i) mbar_init(&bar.afull[i], 4), mbar_init(&bar.aempty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.pfull[i], 1), mbar_init(&bar.pempty[i], 4);
    for (int i = 0; i < kSlotsS; ++i) mbar_init(&bar.sfull[i], 1), mbar_init(&bar.sempty[i], 8);
    fence_barrier_init();
    abort_flag = 0;
  }
  if (kFP8 && tid < 16) {
    uint32_t w[4];
    for (int i = 0; i < 4; ++i) {
      w[i] = 0;
      for (int b = 0; b < 4; ++b) w[i] |= e4m3_of_int(4 * i + b - tid) << (8 * b);
    }
    tables[tid] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t tmem_a = tmem + 2 * kHalf;
  volatile int* abort = &abort_flag;

  pdl_wait_then_release();

  const int blocks = (a.I + 127) / 128;  // steps of 128 channels
  const int groups = a.I / kGroup;
  const auto give_up = [&]() {
    abort_flag = 1;
    if (a.err) atomicOr(a.err, EP_ERRBIT_TIMEOUT);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    Walk walk(a);
    Item it;
    if (warp == 0 && lane == 0) {  // x tiles
      uint32_t n = 0;
      for (int64_t item = blockIdx.x; walk.at(item, &it) && !*abort; item += gridDim.x) {
        const int row = (int)(it.e * a.cap) + it.r0, boxes = 2 * it.nh / kBoxRows;
        const uint32_t bytes = (uint32_t)(2 * it.nh) * (kFP8 ? 128 : 256);
        for (int b = 0; b < blocks; ++b, ++n) {
          const int s = n % C::kStagesX;
          if (!mbar_wait_bounded(&bar.xempty[s], (n / C::kStagesX & 1) ^ 1, abort)) {
            give_up();
            break;
          }
          mbar_arrive_expect_tx(&bar.xfull[s], bytes);
          uint8_t* dst = sx + s * C::kXBytes;
          for (int i = 0; i < boxes; ++i) {
            if (kFP8) {
              tma_2d(dst + i * kBoxRows * 128, &xmap, b * 128, row + i * kBoxRows, &bar.xfull[s]);
            } else {
              tma_2d(dst + i * kBoxRows * 128, &xmap, b * 128, row + i * kBoxRows, &bar.xfull[s]);
              tma_2d(dst + kRows * 128 + i * kBoxRows * 128, &xmap, b * 128 + 64,
                     row + i * kBoxRows, &bar.xfull[s]);
            }
          }
        }
      }
    } else if (warp == 1 && lane == 0) {  // products
      const uint32_t idesc0 = 1u << 4 | (kFP8 ? 0u : (1u << 7 | 1u << 10)) | (128u >> 4) << 24;
      uint32_t n = 0, p = 0;  // steps, groups
      bool ok = true;
      for (int64_t item = blockIdx.x; ok && walk.at(item, &it) && !*abort; item += gridDim.x) {
        const uint32_t idesc = idesc0 | (uint32_t)(it.nh >> 3) << 17;
        for (int b = 0; ok && b < blocks; ++b, ++n) {
          const int s = n % C::kStagesX, sa = n % kSlotsA;
          ok = mbar_wait_bounded(&bar.xfull[s], n / C::kStagesX & 1, abort) &&
               mbar_wait_bounded(&bar.afull[sa], n / kSlotsA & 1, abort);
          const int here = min(kPerBlock, groups - b * kPerBlock);
          for (int g = 0; ok && g < here; ++g, ++p) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              ok = ok && mbar_wait_bounded(&bar.pempty[h], (p & 1) ^ 1, abort);
              if (!ok) break;
              fence_after();
#pragma unroll
              for (int j = 0; j < kMmaPerGroup; ++j) {
                const int k = g * kMmaPerGroup + j;  // matrix step within the block
                const uint32_t xa = smem_addr(sx + s * C::kXBytes) + (uint32_t)(h * it.nh) * 128 +
                                    (kFP8 ? k * 32 : (k >> 2) * kRows * 128 + (k & 3) * 32);
                mma<kFP8>(tmem + h * kHalf, tmem_a + sa * C::kColsA + k * 8, smem_desc(xa), idesc,
                          j > 0);
              }
              commit(&bar.pfull[h]);
            }
          }
          if (!ok) break;
          commit(&bar.xempty[s]);
          commit(&bar.aempty[sa]);
        }
      }
      // the last arrivals land before the block may leave
      if (ok && n > 0)
        ok = mbar_wait_bounded(&bar.aempty[(n - 1) % kSlotsA], (n - 1) / kSlotsA & 1, abort);
      if (!ok) give_up();
    } else if (warp == 2 && lane == 0) {  // weight codes
      uint32_t n = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; ok && walk.at(item, &it) && !*abort; item += gridDim.x) {
        const int row0 = it.e * a.rows + it.tile * (kSwiglu ? 64 : 128);
        const int row1 = row0 + (kSwiglu ? a.N : 64);
        for (int b = 0; b < blocks; ++b, ++n) {
          const int s = n % C::kStagesW;
          ok = mbar_wait_bounded(&bar.wempty[s], (n / C::kStagesW & 1) ^ 1, abort);
          if (!ok) break;
          mbar_arrive_expect_tx(&bar.wfull[s], kWBytes);
          tma_2d(sw + s * kWBytes, &wmap, b * 64, row0, &bar.wfull[s]);
          tma_2d(sw + s * kWBytes + 4096, &wmap, b * 64, row1, &bar.wfull[s]);
        }
      }
      if (!ok) give_up();
    } else if (kFP8 && warp == 3) {  // row scales
      uint32_t n = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; ok && walk.at(item, &it) && !*abort; item += gridDim.x) {
        const float* src = a.x_scales + ((int64_t)it.e * a.cap + it.r0) * blocks;
        int off[8];
        float now[8], next[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          off[i] = min(lane + 32 * i, it.rows - 1) * blocks;
          now[i] = __ldg(src + off[i]);
          next[i] = __ldg(src + off[i] + min(1, blocks - 1));
        }
        for (int b = 0; b < blocks; ++b, ++n) {
          const int s = n % kSlotsS;
          float later[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) later[i] = __ldg(src + off[i] + min(b + 2, blocks - 1));
          ok = mbar_wait_bounded(&bar.sempty[s], (n / kSlotsS & 1) ^ 1, abort);
          if (!__all_sync(kFull, ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss[s * kRows + lane + 32 * i] = now[i];
            now[i] = next[i];
            next[i] = later[i];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sfull[s]);
        }
      }
      if (!ok) give_up();
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // codes -> operand A; this thread's weight row is tensor-memory lane
    // 32 * (warp % 4) + lane
    const int quad = warp & 3;
    const int ch = kSwiglu ? quad * 16 + (lane & 15) : quad * 32 + lane;
    const int srow = kSwiglu ? ch + (lane >= 16 ? 64 : 0) : ch;
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    Walk walk(a);
    Item it;
    uint32_t n = 0;
    bool ok = true;
    for (int64_t item = blockIdx.x; ok && walk.at(item, &it) && !*abort; item += gridDim.x) {
      const int c = min(it.tile * (kSwiglu ? 64 : 128) + ch, a.N - 1);
      const int64_t wrow = (int64_t)it.e * a.rows + c + (kSwiglu && lane >= 16 ? a.N : 0);
      const uint8_t* zrow = a.zeros ? a.zeros + wrow * groups : nullptr;
      for (int b = 0; b < blocks; ++b, ++n) {
        uint32_t z[kPerBlock];
#pragma unroll
        for (int g = 0; g < kPerBlock; ++g)
          z[g] = zrow ? (uint32_t)__ldg(zrow + min(b * kPerBlock + g, groups - 1)) : 8u;
        const int s = n % C::kStagesW, sa = n % kSlotsA;
        ok = mbar_wait_bounded(&bar.wfull[s], n / C::kStagesW & 1, abort);
        ok = ok && mbar_wait_bounded(&bar.aempty[sa], (n / kSlotsA & 1) ^ 1, abort);
        if (!__all_sync(kFull, ok)) {
          ok = false;
          break;
        }
        fence_after();
        const uint4* src = reinterpret_cast<const uint4*>(sw + s * kWBytes + srow * 64);
        const int swz = (srow >> 1) & 3;
        if (kFP8) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w = src[i ^ swz];
            const uint4 t = tables[z[i * kPerBlock / 4] & 15];
            codes_e4m3(w.x, t, r + 8 * i);
            codes_e4m3(w.y, t, r + 8 * i + 2);
            codes_e4m3(w.z, t, r + 8 * i + 4);
            codes_e4m3(w.w, t, r + 8 * i + 6);
          }
          tmem_st32(tmem_a + sa * C::kColsA + lane_addr, r);
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int chunk = half * 2 + i;
              const uint4 w = src[chunk ^ swz];
              const uint32_t zp = 0x43004300u | z[chunk * kPerBlock / 4] * 0x00010001u;
              codes_bf16(w.x, zp, r + 16 * i);
              codes_bf16(w.y, zp, r + 16 * i + 4);
              codes_bf16(w.z, zp, r + 16 * i + 8);
              codes_bf16(w.w, zp, r + 16 * i + 12);
            }
            tmem_st32(tmem_a + sa * C::kColsA + half * 32 + lane_addr, r);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.wempty[s]);
          mbar_arrive(&bar.afull[sa]);
        }
      }
    }
    if (!ok) give_up();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int h = (warp - 8) >> 2, quad = warp & 3;
    const int ch = kSwiglu ? quad * 16 + (lane & 15) : quad * 32 + lane;
    const uint32_t part = tmem + h * kHalf + ((uint32_t)(quad * 32) << 16);
    Walk walk(a);
    Item it;
    uint32_t n = 0, p = 0;
    bool ok = true;
    for (int64_t item = blockIdx.x; ok && walk.at(item, &it) && !*abort; item += gridDim.x) {
      const int n0 = it.tile * (kSwiglu ? 64 : 128) + ch;
      const int64_t wrow =
          (int64_t)it.e * a.rows + min(n0, a.N - 1) + (kSwiglu && lane >= 16 ? a.N : 0);
      const __nv_bfloat16* srow = a.scales + wrow * groups;
      uint64_t acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = 0;
      __nv_bfloat16 s0 = srow[0], s1 = srow[min(1, groups - 1)];
      for (int g = 0; g < groups; ++g, ++p) {
        const __nv_bfloat16 s2 = srow[min(g + 2, groups - 1)];
        const uint32_t sv = __float_as_uint(__bfloat162float(s0));
        const uint64_t scale = pack2(sv, sv);
        const int slot = n % kSlotsS;
        ok = mbar_wait_bounded(&bar.pfull[h], p & 1, abort);
        if (kFP8 && g % kPerBlock == 0)
          ok = ok && mbar_wait_bounded(&bar.sfull[slot], n / kSlotsS & 1, abort);
        if (!__all_sync(kFull, ok)) {
          ok = false;
          break;
        }
        fence_after();
        const float* xs = ss + slot * kRows + h * it.nh;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c * 32 < it.nh) {
            uint32_t r[32];
            tmem_ld32(part + c * 32, r);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint64_t v = pack2(r[2 * i], r[2 * i + 1]);
              if (kFP8) v = mul2(v, *reinterpret_cast<const uint64_t*>(xs + c * 32 + 2 * i));
              fma2(acc[c * 16 + i], v, scale);
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.pempty[h]);
        if (g % kPerBlock == kPerBlock - 1 || g == groups - 1) {
          if (kFP8 && lane == 0) mbar_arrive(&bar.sempty[slot]);
          ++n;
        }
        s0 = s1;
        s1 = s2;
      }
      if (!ok) break;
      const int left = it.rows - h * it.nh;  // live rows of this half
      __nv_bfloat16* y = a.y + ((int64_t)it.e * a.cap + it.r0 + h * it.nh) * a.N + n0;
      if (kSwiglu) {
        // lanes 0-15 hold the gate, 16-31 the up projection of the same
        // channels: the lower lanes finish the first row of each pair, the
        // upper ones the second
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) {
          const float2 v = unpack2(acc[i]);
          const float other = __shfl_xor_sync(kFull, lane < 16 ? v.y : v.x, 16);
          const float gate = lane < 16 ? v.x : other, up = lane < 16 ? other : v.y;
          const int r = 2 * i + (lane >> 4);
          if (r < left && r < it.nh && n0 < a.N)
            y[(int64_t)r * a.N] = __float2bfloat16_rn(gate / (1.0f + expf(-gate)) * up);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) {
          const float2 v = unpack2(acc[i]);
          if (n0 < a.N) {
            if (2 * i < left && 2 * i < it.nh) y[(int64_t)(2 * i) * a.N] = __float2bfloat16_rn(v.x);
            if (2 * i + 1 < left && 2 * i + 1 < it.nh)
              y[(int64_t)(2 * i + 1) * a.N] = __float2bfloat16_rn(v.y);
          }
        }
      }
    }
    if (!ok) give_up();
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (abort_flag) {  // let the copies and products in flight land (at most 20 ms)
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 20000000ull) {
    }
    __syncthreads();
  }
  __syncwarp();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// --- host ------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* ptr, uint64_t inner,
               uint64_t outer, uint64_t stride, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {inner, outer}, strides[1] = {stride};
  const cuuint32_t box[2] = {box_inner, box_outer}, step[2] = {1, 1};
  const EncodeTiled fn = encode_tiled();
  return fn && fn(map, type, 2, const_cast<void*>(ptr), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFP8, bool kSwiglu, int kGroup>
ep_status_t launch(ExpertsArgs a, cudaStream_t st) {
  using C = Cfg<kFP8>;
  const auto kernel = experts_tc_kernel<kFP8, kSwiglu, kGroup>;
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return EP_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      // the register split draws on what the block was launched with
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs * kThreads < 65536 ||
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
              cudaSuccess)
        return EP_ERR_CUDA;
      ready[dev] = true;
    }
  }
  CUtensorMap xmap, wmap;
  if (!encode_2d(&xmap, kFP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                 a.x, a.I, (uint64_t)a.E * a.cap, (uint64_t)a.I * (kFP8 ? 1 : 2), kFP8 ? 128 : 64,
                 kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q, a.I / 2, (uint64_t)a.E * a.rows,
                 a.I / 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B))
    return EP_ERR_CUDA;
  const int width = kSwiglu ? 64 : 128;
  a.tiles = (a.N + width - 1) / width;
  launch_pdl(kernel, props.sm_count, kThreads, C::kSmem, st, a, xmap, wmap);
  return launch_status();
}

template <bool kFP8, bool kSwiglu>
ep_status_t launch_group(const ExpertsArgs& a, int group, cudaStream_t st) {
  if (group == 32) return launch<kFP8, kSwiglu, 32>(a, st);
  if (group == 64) return launch<kFP8, kSwiglu, 64>(a, st);
  return launch<kFP8, kSwiglu, 128>(a, st);
}

}  // namespace

ep_status_t launch_experts_many(const ExpertsArgs& a, bool fp8, bool swiglu, int group,
                                cudaStream_t st) {
  if (a.cap <= kFewRows) return EP_OK;
  if (fp8)
    return swiglu ? launch_group<true, true>(a, group, st) : launch_group<true, false>(a, group, st);
  return swiglu ? launch_group<false, true>(a, group, st) : launch_group<false, false>(a, group, st);
}

}  // namespace ep

// ep_experts_w4_tc.cu -- the experts' products with 4-bit weights for experts
// with many rows: tcgen05 with the weights as operand A in tensor memory.
//
// D[channel][row] = sum over one group of (q - zero) * x: the codes less
// their zero point are small integers, exact in bf16, and codes and zero
// points are exact in E4M3 (as two operands: q and -zero), so A holds them
// unscaled and the tensor cores add exact products in float32.  A group's
// sums are then read from tensor memory, multiplied by the group's
// scale (and, for E4M3 rows, the scale of the row's 128 channels) and added
// to float32 accumulators in registers: no weight is ever rounded, and E4M3
// rows are multiplied as they are, at the 8-bit rate.
//
// A block takes 128 weight rows (swiglu: 64 of the gate and the same 64 of
// the up projection) times up to 192 (E4M3: 160) rows of x, with two buffers of
// sums in tensor memory (the columns behind them hold A), so that one group's
// sums are read while the next group is multiplied:
//   warp 0       TMA of the x tiles (128 channels x the rows, swizzled 128 B)
//   warp 1       tensor memory, and the tcgen05.mma
//   warp 2       TMA of the weight codes (128 rows x 64 bytes)
//   warp 3       group scales, zero points and scales of E4M3 rows, by
//                4-byte asynchronous copies into shared memory
//   4 to 7       codes -> integers -> operand A
//   8 to 15      sums -> scaled -> registers, each four of them for half of
//                the rows; the epilogue
// Every wait is bounded; a block whose wait runs out reports
// EP_ERRBIT_TIMEOUT and leaves.
//
// What bounds it is the scaling beside the products: every group's sums are
// read from tensor memory and multiplied into the accumulators (E4M3 rows:
// after a product with the row's scale), two to an instruction, by the summing
// warps; without that work the same launch took 712 instead of 779 us (bf16)
// and 1.50 instead of 1.84 ms (E4M3).  Measured in long runs (960 W): 8 experts
// of 4096 x 4096, 16384 tokens of two experts, bf16 rows: 820-840 us, 1.31-1.34
// PFLOP/s; 256 experts, gate and up of 2048 x 7168, 4096 tokens of eight experts,
// E4M3 rows: 1.89-1.95 ms, 0.99-1.02 PFLOP/s (short runs 780 us and 1.84 ms);
// about 28 rows an expert, 7168 -> 2048 channels: bf16 874 us, E4M3 696 us.
#include <cuda.h>

#include "ep_experts_w4.cuh"

namespace ep {
namespace {

constexpr int kParts = 2;  // teams of four warps that add up sums, a part of the rows each
constexpr int kBoxes = 6;  // x is loaded in boxes of 32, 64, ... 192 rows
constexpr int kWBytes = 8192;   // 128 weight rows x 64 bytes
constexpr unsigned kFull = 0xFFFFFFFFu;

// A step is 128 channels: one stage of x, one of codes, one slot of A, and
// one slot of scales.
template <bool kFP8, int kGroup>
struct Cfg {
  static constexpr int kThreads = 128 * (2 + kParts);
  // registers per thread: at launch, then for the copying, unpacking and
  // summing warps; the split draws on what the launch gave
  static constexpr int kLaunchRegs = 128;
  static constexpr int kRegsCopy = 56, kRegsUnpack = 104, kRegsSum = 176;
  static_assert(128 * (kRegsCopy + kRegsUnpack + kParts * kRegsSum) <= kThreads * kLaunchRegs,
                "the split would wait for ever");
  // rows of x per block: what the accumulators of two teams hold in registers
  // without moves (E4M3 rows need registers for their scales as well)
  static constexpr int kRows = kFP8 ? 160 : 192;
  static constexpr int kPart = kRows / kParts;
  static constexpr int kXBytes = kRows * (kFP8 ? 128 : 256);
  static constexpr int kStagesX = kFP8 ? 4 : 3;  // at least kSlotsA
  static constexpr int kStagesW = !kFP8 && kGroup == 32 ? 6 : 8;  // what fits
  static constexpr int kPerStep = 128 / kGroup;  // groups in a step
  // tensor-memory columns of a slot of A (E4M3: and of each group's zero points)
  static constexpr int kColsA = kFP8 ? 32 + 8 * kPerStep : 64;
  static constexpr int kSlotsA = (512 - 2 * kRows) / kColsA < 4 ? (512 - 2 * kRows) / kColsA : 4;
  static constexpr int kSlotsS = 8;
  // words of a slot of scales: per group 128 scale words and 128 zero-point words
  static constexpr int kSWords = kPerStep * 256;
  // slots for the rows' scales, four steps of all rows each
  static constexpr int kSlotsXs = kStagesX + 2;
  static constexpr int kXsBytes = kFP8 ? kRows * 16 : 0;
  static constexpr int kSmem = 1024 + kStagesX * kXBytes + kStagesW * kWBytes +
                               kSlotsS * kSWords * 4 + kSlotsXs * kXsBytes;
};

// One tensor map per height of a box, so that a step of x is one copy (two
// for bf16) whatever the number of rows.
struct XMaps {
  CUtensorMap rows[kBoxes];  // [i]: 32 * (i + 1) rows
};

template <typename C>
struct Barriers {
  // full: a step's x (one arrival), A (four) and scales (32) are in place;
  // done: its products are finished; sfull: its zero points are in place
  uint64_t full[C::kStagesX], done[C::kStagesX], wfull[C::kStagesW], wempty[C::kStagesW];
  uint64_t sfull[C::kSlotsS], pfull[2], pempty[2];
};

// --- the items of a block ----------------------------------------------------
struct Item {
  int e, tile, r0, rows, np;  // np: rows of a part, a multiple of 16
};

// Walks the experts with more than kFewRows rows; item numbers run over the
// experts, their chunks of rows, and the tiles of channels, tiles innermost.
// 32 bits hold them: an item is at least 64 channels of 2-byte results for
// more than kFewRows rows, so 2^31 of them would not fit the GPU's memory.
struct Walk {
  int e = -1, n = 0, chunks = 0, base = 0, items = 0;

  template <int kRows>
  __device__ bool at(const ExpertsArgs& a, int item, Item* it) {
    while (item >= base + items) {
      base += items;
      if (++e >= a.E) {
        --e;
        items = 0;
        return false;
      }
      n = min(__ldg(a.count + e), (int)a.cap);
      chunks = n > kFewRows ? (n + kRows - 1) / kRows : 0;
      items = chunks * a.tiles;
    }
    const int local = item - base, chunk = local / a.tiles, size = (n + chunks - 1) / chunks;
    it->e = e;
    it->tile = local - chunk * a.tiles;
    it->r0 = chunk * size;
    it->rows = min(size, n - it->r0);
    it->np = (it->rows + 31) / 32 * (32 / kParts);
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

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
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

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 columns of the thread's own lane.  The load and its wait are one statement,
// so that no use moves between them.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// 16 columns of the warp's 32 lanes, in the layout of a matrix fragment: thread
// 4g + q gets, of columns 2q, 2q + 1 (v[0..7]) and 8 + 2q, 8 + 2q + 1, the
// lanes g, g + 8, g + 16, g + 24: v[8 * half + 2 * j + i], j the lane's eighth.
__device__ __forceinline__ void tmem_ld_fragment(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%8,%9,%10,%11}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%4,%5,%6,%7,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr), "r"(addr + (16u << 16))
      : "memory");
}

// Waits for the phase of the barrier at `bar` (a shared address) with the
// given parity; false if it has not completed after kTries tries.  The hardware
// suspends a try for 3.7 us (measured: 2^20 tries took 3.9 s): about 1 s in all.
// (Four instructions a try: the warps that wait share their schedulers with
// those that work, and a limit by the clock after the tries took 2% longer.)
constexpr uint32_t kTries = 1u << 18;
#define EP_WAIT(kPause)                                                       \
  uint32_t left;                                                              \
  asm volatile(                                                               \
      "{\n\t.reg .pred P;\n\t"                                                \
      "mov.u32 %0, %3;\n"                                                     \
      "TRY:\n\t"                                                              \
      "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %4;\n\t"         \
      "@P bra DONE;\n\t" kPause                                               \
      "sub.u32 %0, %0, 1;\n\t"                                                \
      "setp.ne.u32 P, %0, 0;\n\t"                                             \
      "@P bra TRY;\n"                                                         \
      "DONE:\n\t}"                                                            \
      : "=&r"(left)                                                           \
      : "r"(bar), "r"(parity), "r"(kTries), "r"(1000u)                        \
      : "memory");                                                            \
  return left != 0;
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) { EP_WAIT("") }
// For warps that run ahead of the others: their tries leave the schedulers to
// those that are waited for.
__device__ __forceinline__ bool wait_idle(uint32_t bar, uint32_t parity) {
  EP_WAIT("nanosleep.u32 64;\n\t")
}
#undef EP_WAIT
__device__ __forceinline__ bool wait_idle(uint64_t* bar, uint32_t parity) {
  return wait_idle(smem_addr(bar), parity);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  return wait(smem_addr(bar), parity);
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint64_t lds64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// 4-byte asynchronous copy; the barrier counts one arrival per thread when
// its copies so far have landed.
__device__ __forceinline__ void copy_word(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
// The word that holds the element at p.
__device__ __forceinline__ const void* word_of(const void* p) {
  return reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
}

// A ring of slots: the slot and the parity of its current round.
template <int kSlots>
struct Ring {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) {
      slot = 0;
      round ^= 1;
    }
  }
};

// --- sums -> accumulators ---------------------------------------------------------
// Two float32 at once: half the instructions of fmaf.
__device__ __forceinline__ uint64_t mul2(uint32_t v0, uint32_t v1, uint64_t x) {
  uint64_t t;
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tmul.rn.f32x2 %0, v, %3;\n\t}"
      : "=l"(t)
      : "r"(v0), "r"(v1), "l"(x));
  return t;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t v0, uint32_t v1, uint64_t scale) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(v0), "r"(v1), "l"(scale));
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t t, uint64_t scale) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(t), "l"(scale));
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// What the loop over the groups of an item needs.
struct SumArgs {
  uint32_t pfull, pempty;  // barriers (shared addresses)
  uint32_t scale, xs;      // this thread's first scale word, its part's row scales
  uint32_t src;            // this part's columns of sums
  uint32_t odd;            // bit j: whether row j's first group is a word's high half
  int groups;
};

// Adds up all groups of an item for 16 * kChunks rows; n and p count steps
// and groups over the items, q the slots of the rows' scales.  With bf16 rows a thread holds one weight row
// times all rows of x; with E4M3 rows four weight rows (j) times a quarter of
// the rows of x, since the rows' scales, which every thread needs in
// registers, would else take 640 of the cycles of shared memory for a step,
// instead of 160 (FP8 decode step 1942 us -> 1842; bf16 rows have none to
// save, and four scales to read instead of one cost them 779 -> 832 us).  One
// instance per number of chunks: a branch in the inner loop costs as much as
// a chunk.
template <bool kFP8, int kGroup, int kChunks>
__device__ __forceinline__ bool add_groups(const SumArgs& s, int lane, uint32_t& n, uint32_t& p,
                                           uint32_t& q,
                                           uint64_t (&acc)[Cfg<kFP8, kGroup>::kPart / 2]) {
  using C = Cfg<kFP8, kGroup>;
#pragma unroll 1
  for (int g = 0; g < s.groups; ++g) {
    const uint32_t slot = n % C::kSlotsS, buf = p & 1;
    const uint32_t in = C::kPerStep == 1 ? 0 : g % C::kPerStep;
    // (the scales are there too: their copies arrive where the products wait)
    const bool fine = wait(s.pfull + buf * 8, p >> 1 & 1);
    fence_after();
    const uint32_t at = slot * C::kSWords * 4 + in * 1024;
    uint64_t scale[kFP8 ? 4 : 1];
#pragma unroll
    for (int j = 0; j < (kFP8 ? 4 : 1); ++j) {
      // bf16 -> float32 is a shift; the word holds groups 2i and 2i + 1
      const uint32_t word = lds32(s.scale + at + j * 32);
      const uint32_t sv = (s.odd >> j ^ g) & 1 ? word & 0xFFFF0000u : word << 16;
      // E4M3 codes are products of 2^-9
      const float f = kFP8 ? __uint_as_float(sv) * 512.0f : __uint_as_float(sv);
      asm("mov.b64 %0, {%1, %1};" : "=l"(scale[j]) : "f"(f));
    }
    const uint32_t src = s.src + buf * C::kRows, b = g / C::kPerStep;
    const uint32_t xs = s.xs + q % C::kSlotsXs * C::kXsBytes + (b & 3) * C::kRows * 4;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      // the loads of a chunk together, then all products, then all sums:
      // neighbours that wait for one another cost a latency each
      uint32_t v[16];
      if (kFP8) {
        const uint64_t x[2] = {lds64(xs + c * 64), lds64(xs + c * 64 + 32)};
        tmem_ld_fragment(src + c * 16, v);
        uint64_t t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = mul2(v[2 * i], v[2 * i + 1], x[i >> 2]);
#pragma unroll
        for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], t[i], scale[i & 3]);
      } else {
        tmem_ld16(src + c * 16, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], v[2 * i], v[2 * i + 1], scale[0]);
      }
    }
    fence_before();
    if (__any_sync(kFull, !fine)) return false;
    ++p;
    const bool last = C::kPerStep == 1 || in == C::kPerStep - 1 || g == s.groups - 1;
    if (lane == 0) arrive(s.pempty + buf * 8);
    if (last) ++n;
    if (kFP8 && last && ((b & 3) == 3 || g == s.groups - 1)) ++q;
  }
  return true;
}

// --- codes -> operand A ---------------------------------------------------------
// Eight codes as four bf16 pairs in channel order: byte j of the word holds
// the pair (2j, 2j + 1); 0x4300 | q is 128 + q, less 128 + zero.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t zp, uint32_t* out) {
  const uint32_t odd = w >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = __byte_perm(w, odd, (uint32_t)(j | j << 4 | (4 + j) << 8 | (4 + j) << 12));
    uint32_t v;  // (two & 0x000F000F) | 0x43004300
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(two), "r"(0x000F000Fu), "r"(0x43004300u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(out[j]) : "r"(v), "r"(zp));
  }
}

// Eight codes as E4M3 bytes in channel order: the codes themselves.  E4M3's
// subnormals and first normal numbers are k * 2^-9 for k = 0..15, so a 4-bit
// code is the E4M3 number q * 2^-9 as it stands: 5 instructions for 8 codes
// instead of 13 that subtract the zero point by looking q - zero up.
__device__ __forceinline__ void codes_e4m3(uint32_t w, uint32_t* out) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = w >> 4 & 0x0F0F0F0Fu;
  out[0] = __byte_perm(even, odd, 0x5140);
  out[1] = __byte_perm(even, odd, 0x7362);
}

// Lane r of tensor memory (0..127) holds the weight row of this channel of the
// tile; with swiglu, lanes 16..31 of each 32 hold the up projection's.  With
// E4M3 rows a thread of the summing warps gets lanes g, g + 8, g + 16 and
// g + 24: four neighbouring channels, or two of the gate and the same two of
// up, which it stores at once.  Within the four they are rotated, so that the
// eight lanes that read their codes together do not meet a bank of shared
// memory twice.
template <bool kFP8, bool kSwiglu>
__device__ __forceinline__ int lane_channel(int r) {
  const int g = r & 7, j = r >> 3 & 3;
  if (!kFP8) return kSwiglu ? (r >> 5) * 16 + (r & 15) : r;
  return kSwiglu ? (r >> 5) * 16 + 2 * g + ((j ^ g >> 2) & 1)
                 : (r >> 5) * 32 + 4 * g + ((j + (g >> 1)) & 3);
}
template <bool kSwiglu>
__device__ __forceinline__ bool lane_is_up(int r) {
  return kSwiglu && (r & 16);
}
template <bool kFP8, bool kSwiglu>
__device__ __forceinline__ int64_t lane_row(const ExpertsArgs& a, const Item& it, int r) {
  const int c = min(it.tile * (kSwiglu ? 64 : 128) + lane_channel<kFP8, kSwiglu>(r), a.N - 1);
  return (int64_t)it.e * a.rows + c + (lane_is_up<kSwiglu>(r) ? a.N : 0);
}

// Writes one part of an item's rows, bf16 rows of x: acc[i] holds rows 2i and
// 2i + 1 of the thread's own channel.
template <bool kSwiglu, int kPart>
__device__ __forceinline__ void store_rows(const ExpertsArgs& a, const Item& it, int h, int quad,
                                           int lane, const uint64_t (&acc)[kPart / 2]) {
  const int n0 = it.tile * (kSwiglu ? 64 : 128) + lane_channel<false, kSwiglu>(quad * 32 + lane);
  const int left = min(it.rows - h * it.np, it.np);  // live rows of this part
  __nv_bfloat16* dst =
      a.y + ((int64_t)it.e * a.cap + it.r0 + h * it.np + (kSwiglu ? lane >> 4 : 0)) * a.N + n0;
  // the lanes that stay (a lane and the one 16 further have the same channel)
  const unsigned in = __ballot_sync(kFull, n0 < a.N);
  if (n0 >= a.N) {
    // a channel beyond the last tile's end
  } else if (kSwiglu) {
    // lanes 0-15 hold the gate, 16-31 the up projection of the same
    // channels: the lower lanes finish the first row of each pair, the
    // upper ones the second
#pragma unroll
    for (int i = 0; i < kPart / 2; ++i) {
      if (2 * i >= left) break;
      const float2 v = unpack2(acc[i]);
      const float other = __shfl_xor_sync(in, lane < 16 ? v.y : v.x, 16);
      const float gate = lane < 16 ? v.x : other, up = lane < 16 ? other : v.y;
      const float out = silu_times(gate, up);
      if (2 * i + (lane >> 4) < left) *dst = __float2bfloat16_rn(out);
      dst += 2 * a.N;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPart / 2; ++i) {
      if (2 * i >= left) break;
      const float2 v = unpack2(acc[i]);
      dst[0] = __float2bfloat16_rn(v.x);
      if (2 * i + 1 < left) dst[a.N] = __float2bfloat16_rn(v.y);
      dst += 2 * a.N;
    }
  }
}

// The same for E4M3 rows, in the layout of a matrix fragment.
template <bool kSwiglu, int kPart>
__device__ __forceinline__ void store_fragment(const ExpertsArgs& a, const Item& it, int h, int quad,
                                               int lane, const uint64_t (&acc)[kPart / 2]) {
  const int g = lane >> 2, q = lane & 3;
  // acc[8c + 4b + j]: rows 16c + 8b + 2q and the next, weight row j
  const int n0 = it.tile * (kSwiglu ? 64 : 128) + (kSwiglu ? quad * 16 + 2 * g : quad * 32 + 4 * g);
  const int left = min(it.rows - h * it.np, it.np);  // live rows of this part
  __nv_bfloat16* dst = a.y + ((int64_t)it.e * a.cap + it.r0 + h * it.np + 2 * q) * a.N + n0;
  if (n0 < a.N) {  // else beyond the last tile's end
#pragma unroll
    for (int i = 0; i < kPart / 8; ++i) {
      if (8 * i >= left) break;
      const float2 v[4] = {unpack2(acc[4 * i]), unpack2(acc[4 * i + 1]), unpack2(acc[4 * i + 2]),
                           unpack2(acc[4 * i + 3])};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float f[4] = {k ? v[0].y : v[0].x, k ? v[1].y : v[1].x, k ? v[2].y : v[2].x,
                            k ? v[3].y : v[3].x};
        if (8 * i + 2 * q + k < left) {
          if (kSwiglu) {
            const float o0 = silu_times(f[0], f[2]), o1 = silu_times(f[1], f[3]);
            *reinterpret_cast<__nv_bfloat162*>(dst + k * a.N) =
                g < 4 ? __floats2bfloat162_rn(o0, o1) : __floats2bfloat162_rn(o1, o0);
          } else {
            // back by g / 2 places: one, then two
            const bool one = g & 2, two = g & 4;
            const float r0 = one ? f[3] : f[0], r1 = one ? f[0] : f[1];
            const float r2 = one ? f[1] : f[2], r3 = one ? f[2] : f[3];
            __nv_bfloat162 o[2] = {__floats2bfloat162_rn(two ? r2 : r0, two ? r3 : r1),
                                   __floats2bfloat162_rn(two ? r0 : r2, two ? r1 : r3)};
            *reinterpret_cast<uint2*>(dst + k * a.N) = *reinterpret_cast<const uint2*>(o);
          }
        }
      }
      dst += 8 * (int64_t)a.N;
    }
  }
}

template <bool kFP8, bool kSwiglu, int kGroup>
__global__ void __launch_bounds__(Cfg<kFP8, kGroup>::kThreads, 1)
    experts_tc_kernel(ExpertsArgs a, const __grid_constant__ XMaps xmaps,
                      const __grid_constant__ CUtensorMap wmap) {
  using C = Cfg<kFP8, kGroup>;
  constexpr int kPerStep = C::kPerStep;
  constexpr int kMmaPerGroup = kGroup / (kFP8 ? 32 : 16);
  extern __shared__ uint8_t raw[];
  __shared__ Barriers<C> bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = base;
  uint8_t* sw = sx + C::kStagesX * C::kXBytes;
  uint32_t* ss = reinterpret_cast<uint32_t*>(sw + C::kStagesW * kWBytes);
  uint8_t* sxs = reinterpret_cast<uint8_t*>(ss + C::kSlotsS * C::kSWords);

  if (tid == 0) {
    for (int i = 0; i < C::kStagesX; ++i) mbar_init(&bar.full[i], 37), mbar_init(&bar.done[i], 1);
    for (int i = 0; i < C::kStagesW; ++i) mbar_init(&bar.wfull[i], 1), mbar_init(&bar.wempty[i], 4);
    for (int i = 0; i < C::kSlotsS; ++i) mbar_init(&bar.sfull[i], 32);
    for (int i = 0; i < 2; ++i) mbar_init(&bar.pfull[i], 2), mbar_init(&bar.pempty[i], 4 * kParts);
    fence_barrier_init();
    abort_flag = 0;
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
  const uint32_t tmem_a = tmem + 2 * C::kRows;
  const volatile int* abort = &abort_flag;

  pdl_wait_then_release();

  const auto free_tmem = [&]() {
    if (warp == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  };
  // Where every expert is the other kernel's, the block leaves: the walk below
  // would read the counts one after another (256 experts of two rows each, both
  // launches: 607 us without this, 585 with it).
  bool busy = false;
  for (int e = tid; e < a.E; e += C::kThreads) busy |= min((int64_t)a.count[e], a.cap) > kFewRows;
  if (!__syncthreads_or(busy)) {
    free_tmem();
    return;
  }

  const int steps = (a.I + 127) / 128;
  const int groups = a.I / kGroup;
  const auto give_up = [&]() {
    abort_flag = 1;
    if (a.err) atomicOr(a.err, EP_ERRBIT_TIMEOUT);
  };
  Walk walk;
  Item it;
  bool ok = true;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsCopy));
    if (warp == 0 && lane == 0) {  // x tiles
      Ring<C::kStagesX> rx;
      int unarmed = blockIdx.x == 0 ? a.stall : -1;  // test hook: steps until one is left out
      for (int item = blockIdx.x; ok && walk.at<C::kRows>(a, item, &it) && !*abort; item += gridDim.x) {
        const int row = (int)(it.e * a.cap) + it.r0;
        const CUtensorMap* map = &xmaps.rows[it.np / (32 / kParts) - 1];
        const uint32_t bytes = (uint32_t)(kParts * it.np) * (kFP8 ? 128 : 256);
        for (int b = 0; b < steps; ++b) {
          ok = wait_idle(&bar.done[rx.slot], rx.round ^ 1);
          if (!ok) break;
          if (unarmed-- != 0) {
            uint8_t* dst = sx + rx.slot * C::kXBytes;
            mbar_arrive_expect_tx(&bar.full[rx.slot], bytes);
            tma_2d(dst, map, b * 128, row, &bar.full[rx.slot]);
            if (!kFP8) tma_2d(dst + C::kRows * 128, map, b * 128 + 64, row, &bar.full[rx.slot]);
          }
          rx.next();
        }
      }
      if (!ok) give_up();
    } else if (warp == 1) {  // products: the whole warp waits, one lane issues
      const uint32_t idesc0 = 1u << 4 | (kFP8 ? 0u : (1u << 7 | 1u << 10)) | (128u >> 4) << 24;
      const uint64_t desc0 = smem_desc(0);
      Ring<C::kStagesX> rx;
      Ring<C::kSlotsA> ra;
      Ring<2> rp;
      bool any = false;
      for (int item = blockIdx.x; ok && walk.at<C::kRows>(a, item, &it) && !*abort; item += gridDim.x) {
        const uint32_t idesc = idesc0 | (uint32_t)(kParts * it.np >> 3) << 17;
        for (int b = 0; ok && b < steps; ++b) {
          ok = wait(&bar.full[rx.slot], rx.round);
          const uint32_t x0 = smem_addr(sx + rx.slot * C::kXBytes);
          const uint32_t a0 = tmem_a + ra.slot * C::kColsA;
          const int here = kPerStep == 1 ? 1 : min(kPerStep, groups - b * kPerStep);
          for (int g = 0; g < here; ++g) {
            ok = ok && wait(&bar.pempty[rp.slot], rp.round ^ 1);
            if (!__all_sync(kFull, ok)) {
              ok = false;
              break;
            }
            fence_after();
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < kMmaPerGroup; ++j) {
                const int k = g * kMmaPerGroup + j;  // matrix step within the step
                const uint32_t off = kFP8 ? k * 32 : (k >> 2) * C::kRows * 128 + (k & 3) * 32;
                const uint64_t xd = desc0 | (uint64_t)((x0 + off) >> 4);
                mma<kFP8>(tmem + rp.slot * C::kRows, a0 + k * 8, xd, idesc, j > 0);
                // less zero * x: the same rows of x with the group's zero points
                if (kFP8) mma<kFP8>(tmem + rp.slot * C::kRows, a0 + 32 + g * 8, xd, idesc, true);
              }
              commit(&bar.pfull[rp.slot]);
              mbar_arrive(&bar.pfull[rp.slot]);  // releases what this warp has waited for
              if (g == here - 1) commit(&bar.done[rx.slot]);
            }
            __syncwarp();
            rp.next();
          }
          any = ok;
          rx.next();
          ra.next();
        }
      }
      // the last arrivals land before the block may leave
      if (ok && any) {
        const int last = (rx.slot + C::kStagesX - 1) % C::kStagesX;
        ok = wait(&bar.done[last], rx.slot == 0 ? rx.round ^ 1 : rx.round);
      }
      if (!ok) give_up();
    } else if (warp == 2 && lane == 0) {  // weight codes
      Ring<C::kStagesW> rw;
      for (int item = blockIdx.x; ok && walk.at<C::kRows>(a, item, &it) && !*abort; item += gridDim.x) {
        const int row0 = it.e * a.rows + it.tile * (kSwiglu ? 64 : 128);
        for (int b = 0; b < steps; ++b) {
          ok = wait_idle(&bar.wempty[rw.slot], rw.round ^ 1);
          if (!ok) break;
          uint8_t* dst = sw + rw.slot * kWBytes;
          mbar_arrive_expect_tx(&bar.wfull[rw.slot], kWBytes);
          tma_2d(dst, &wmap, b * 64, row0, &bar.wfull[rw.slot]);
          tma_2d(dst + 4096, &wmap, b * 64, row0 + (kSwiglu ? a.N : 64), &bar.wfull[rw.slot]);
          rw.next();
        }
      }
      if (!ok) give_up();
    } else if (warp == 3) {  // scales and zero points
      // A slot is free once the products of two steps later are done: they went
      // into the buffer whose sums it scaled.  The stages of x are fewer than
      // the slots by more than that, so the x stage's barrier says it.
      static_assert(C::kSlotsS >= C::kStagesX + 2, "a slot would be in use");
      // The same holds for the slots of the rows' scales, a step at least each.
      Ring<C::kSlotsS> rs;
      Ring<C::kSlotsXs> rq;
      Ring<C::kStagesX> rx;
      for (int item = blockIdx.x; ok && walk.at<C::kRows>(a, item, &it) && !*abort; item += gridDim.x) {
        const float* xs = kFP8 ? a.x_scales + ((int64_t)it.e * a.cap + it.r0) * steps : nullptr;
        int64_t at[4];  // this lane's four weight rows: their first group
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = lane_row<kFP8, kSwiglu>(a, it, lane + 32 * i) * groups;
        for (int b = 0; b < steps; ++b) {
          ok = wait_idle(&bar.done[rx.slot], rx.round ^ 1);
          if (!__all_sync(kFull, ok)) {
            ok = false;
            break;
          }
          uint32_t* dst = ss + rs.slot * C::kSWords;
#pragma unroll
          for (int g = 0; g < kPerStep; ++g) {
            const int gi = kPerStep == 1 ? b : min(b * kPerStep + g, groups - 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              copy_word(dst + g * 256 + lane + 32 * i, word_of(a.scales + at[i] + gi));
              if (a.zeros)
                copy_word(dst + g * 256 + 128 + lane + 32 * i, word_of(a.zeros + at[i] + gi));
            }
          }
          if (kFP8 && b % 4 == 0) {
            // a row's scales of four steps lie in one line: at once they look
            // it up while it is there (256 experts of 7168 x 2048, 28 rows
            // each: 742 us; a scale a row each step, 818 us)
            uint8_t* to = sxs + rq.slot * C::kXsBytes;
#pragma unroll
            for (int i = 0; i < C::kRows / 32; ++i) {
              const int r = lane + 32 * i;
              if (r >= kParts * it.np) break;
              const float* from = xs + min(r, it.rows - 1) * steps + b;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (b + j < steps) copy_word(to + (j * C::kRows + r) * 4, from + j);
            }
            rq.next();
          }
          if (a.zeros) copies_arrive(&bar.sfull[rs.slot]);
          copies_arrive(&bar.full[rx.slot]);
          rs.next();
          rx.next();
        }
      }
      if (!ok) give_up();
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsUnpack));
    // codes -> operand A: this thread's weight row is lane 32 * quad + lane of
    // tensor memory
    const int quad = warp & 3, r = quad * 32 + lane;
    const int srow = lane_channel<kFP8, kSwiglu>(r) + (lane_is_up<kSwiglu>(r) ? 64 : 0);
    const uint32_t swz = (uint32_t)((srow >> 1) & 3) << 4;
    const uint32_t row_addr = smem_addr(sw) + srow * 64;
    const uint32_t zero_addr = smem_addr(ss) + (128 + r) * 4;
    const uint32_t a_addr = tmem_a + ((uint32_t)(quad * 32) << 16);
    const uint32_t wfull0 = smem_addr(bar.wfull), sfull0 = smem_addr(bar.sfull);
    const uint32_t done0 = smem_addr(bar.done);
    uint32_t base = 0;  // steps of the items before
    for (int item = blockIdx.x; ok && walk.at<C::kRows>(a, item, &it) && !*abort; item += gridDim.x) {
      const int at4 = (int)(lane_row<kFP8, kSwiglu>(a, it, r) * groups & 3);
      for (int b = 0; b < steps; ++b) {
        const uint32_t n = base + b, was = n - C::kSlotsA;  // the step that had the slot of A
        const uint32_t w_slot = n % C::kStagesW, s_slot = n % C::kSlotsS;
        bool fine = wait_idle(wfull0 + w_slot * 8, n / C::kStagesW & 1);
        if (a.zeros) fine &= wait_idle(sfull0 + s_slot * 8, n / C::kSlotsS & 1);
        if (n >= C::kSlotsA)
          fine &= wait_idle(done0 + was % C::kStagesX * 8, was / C::kStagesX & 1);
        if (__any_sync(kFull, !fine)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t src = row_addr + w_slot * kWBytes;
        const uint32_t dst = a_addr + n % C::kSlotsA * C::kColsA;
        uint32_t zero = 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 32 channels
          const uint4 w = lds128(src + (i << 4 ^ swz));
          if (i % (4 / kPerStep) == 0) {  // the next group's zero point
            if (a.zeros) {
              const int g = i * kPerStep / 4;
              const int gi = at4 + min(b * kPerStep + g, groups - 1);
              zero = lds32(zero_addr + s_slot * C::kSWords * 4 + g * 1024) >> (8 * (gi & 3)) & 15;
            }
            if (kFP8) {  // -zero * 2^-9, for every channel of a matrix step
              const uint32_t z4 = (zero | 0x80u) * 0x01010101u;
              const uint32_t v[8] = {z4, z4, z4, z4, z4, z4, z4, z4};
              tmem_st8(dst + 32 + i * kPerStep / 4 * 8, v);
            }
          }
          if (kFP8) {
            uint32_t v[8];
            codes_e4m3(w.x, v);
            codes_e4m3(w.y, v + 2);
            codes_e4m3(w.z, v + 4);
            codes_e4m3(w.w, v + 6);
            tmem_st8(dst + i * 8, v);
          } else {
            const uint32_t zp = 0x43004300u | zero * 0x00010001u;
            uint32_t v[16];
            codes_bf16(w.x, zp, v);
            codes_bf16(w.y, zp, v + 4);
            codes_bf16(w.z, zp, v + 8);
            codes_bf16(w.w, zp, v + 12);
            tmem_st16(dst + i * 16, v);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.full[n % C::kStagesX]);
          mbar_arrive(&bar.wempty[w_slot]);
        }
      }
      base += steps;
    }
    if (!ok) give_up();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSum));
    const int h = (warp - 8) >> 2, quad = warp & 3;
    // E4M3 rows: this thread's lanes 8j + g, columns 2q and 2q + 1 of eight
    const int g = kFP8 ? lane >> 2 : lane, q = kFP8 ? lane & 3 : 0;
    SumArgs sum;
    sum.pfull = smem_addr(bar.pfull);
    sum.pempty = smem_addr(bar.pempty);
    sum.scale = smem_addr(ss) + (quad * 32 + g) * 4;
    sum.groups = groups;
    uint32_t n = 0, p = 0, c = 0;  // steps, groups, slots of the rows' scales
    for (int item = blockIdx.x; ok && walk.at<C::kRows>(a, item, &it) && !*abort; item += gridDim.x) {
      sum.odd = 0;
#pragma unroll
      for (int j = 0; j < (kFP8 ? 4 : 1); ++j)
        sum.odd |= (uint32_t)(lane_row<kFP8, kSwiglu>(a, it, quad * 32 + j * 8 + g) * groups & 1) << j;
      sum.src = tmem + ((uint32_t)(quad * 32) << 16) + h * it.np;
      sum.xs = smem_addr(sxs) + (h * it.np + 2 * q) * 4;
      uint64_t acc[C::kPart / 2];
#pragma unroll
      for (int i = 0; i < C::kPart / 2; ++i) acc[i] = 0;
      switch (it.np / 16) {
        case 1: ok = add_groups<kFP8, kGroup, 1>(sum, lane, n, p, c, acc); break;
        case 2: ok = add_groups<kFP8, kGroup, 2>(sum, lane, n, p, c, acc); break;
        case 3: ok = add_groups<kFP8, kGroup, 3>(sum, lane, n, p, c, acc); break;
        case 4: ok = add_groups<kFP8, kGroup, 4>(sum, lane, n, p, c, acc); break;
        case 5: ok = add_groups<kFP8, kGroup, 5>(sum, lane, n, p, c, acc); break;
        default: ok = add_groups<kFP8, kGroup, C::kPart / 16>(sum, lane, n, p, c, acc); break;
      }
      if (!ok) break;
      if constexpr (kFP8)
        store_fragment<kSwiglu, C::kPart>(a, it, h, quad, lane, acc);
      else
        store_rows<kSwiglu, C::kPart>(a, it, h, quad, lane, acc);
      __syncwarp();
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
  free_tmem();
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

thread_local int g_stall_step = -1;  // set by ep_debug_set_experts_stall, used once

template <bool kFP8, bool kSwiglu, int kGroup>
ep_status_t launch(ExpertsArgs a, cudaStream_t st) {
  using C = Cfg<kFP8, kGroup>;
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
      if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs < C::kLaunchRegs ||
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
              cudaSuccess)
        return EP_ERR_CUDA;
      ready[dev] = true;
    }
  }
  XMaps xmaps;
  CUtensorMap wmap;
  for (int i = 0; i < kBoxes; ++i)
    if (!encode_2d(&xmaps.rows[i],
                   kFP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x,
                   a.I, (uint64_t)a.E * a.cap, (uint64_t)a.I * (kFP8 ? 1 : 2), kFP8 ? 128 : 64,
                   32 * (i + 1), CU_TENSOR_MAP_SWIZZLE_128B))
      return EP_ERR_CUDA;
  if (!encode_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q, a.I / 2, (uint64_t)a.E * a.rows,
                 a.I / 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B))
    return EP_ERR_CUDA;
  const int width = kSwiglu ? 64 : 128;
  a.tiles = (a.N + width - 1) / width;
  a.stall = g_stall_step;
  g_stall_step = -1;
  launch_pdl(kernel, props.sm_count, C::kThreads, C::kSmem, st, a, xmaps, wmap);
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

extern "C" void ep_debug_set_experts_stall(int step) { ep::g_stall_step = step < 0 ? -1 : step; }

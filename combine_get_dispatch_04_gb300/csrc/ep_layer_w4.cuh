// ep_layer_w4.cuh -- a whole mixture-of-experts layer for a few tokens: the
// choice of experts, both products with 4-bit weights, the gated activation and
// the weighted sum over the experts, in two launches.
//
//   h[t,k] = w[t,k] * silu(G_e x[t]) * U_e x[t],  out[t] = sum_k D_e h[t,k],  e = e_k
//
// First launch: every block routes all tokens (a warp each) and lists the experts
// that were chosen, each with the tokens that chose it; its warps then multiply
// tiles of 16 gate and 16 up channels by an entry's tokens (columns of the matrix
// instruction; an expert with more than 8 tokens has several entries).  Second
// launch: tiles of 16 output channels, each summed over all chosen experts in
// shared memory, so that no expert's output is ever stored; an entry is 4 tokens, as h
// comes in two bf16 (its rounding, and what that leaves), in columns of their own, and
// only the layer's result is rounded noticeably.
//
// A block takes whole tiles, the same number on every SM but for one, and its 16
// warps share the tiles' steps (4096 codes) evenly: each takes one run of
// consecutive steps, keeps two steps on their way with asynchronous copies, and where a
// tile lies in several warps' runs, its parts are added in the order of the channels
// through shared memory.  The order of every sum depends on the sizes and the choice
// alone, so results repeat bit for bit.
//
// Codes become operands with few instructions: the four bits of a code,
// placed in the low bits of a bf16, are the number q 2^-133 (a subnormal, or
// in the next four bits the first normal numbers, which continue the same
// scale), and one fused multiply-add makes (q - zero) / 64 of it, exactly.
//
// What bounds it: with many experts the latencies of a step (some 300 instructions a lane) at
// four warps a scheduler: 61 to 64% of the issue slots, no pipe above 62%, 4.7 TB/s in the first
// launch and 3.7 in the second; with one token also what comes before and between (routing and
// lists 4.5 us, a launch and the way to the first product 5 us).  Measured on 256 experts
// of 7168 -> 2 x 2048 -> 7168, 8 chosen by a router with a bias that all tokens share: 16
// tokens 354 us (they choose 70 experts, whose bytes take 237), 8 tokens 232 (46, 156), 4
// tokens 142 (27, 93), 1 token 53 (27 us); 5 tokens on 64 experts of 4096 -> 2 x 1024, groups of 64 and zero
// points, 56 us (26).  A further entry of an expert reads its codes again (8 experts of
// 4096 -> 2 x 4096, 2 chosen, 16 tokens: 70 us for 31).  More stages (4: 55 us for one
// token) or more warps (20: 58 us, registers) did not help.
#pragma once

#include <cuda_bf16.h>

#include "ep_experts_w4.cuh"
#include "ep_route.cuh"
#include "ep_w4.cuh"

namespace ep {

struct LayerArgs;
// The launches (false: CUDA refused one).
bool launch_layer_up(const LayerArgs& a, int group, int blocks, cudaStream_t st);
bool launch_layer_down(const LayerArgs& a, int group, int blocks, cudaStream_t st);

constexpr int kWarps = 16;  // of a block, one block an SM
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTokens = EP_LAYER_MAX_TOKENS;
constexpr int kMaxExperts = EP_LAYER_MAX_EXPERTS;
constexpr int kMaxSlots = kMaxTokens * EP_MAX_TOPK;

// A chosen expert with the tokens that chose it, or some of them where they are
// more than the matrix instruction has columns for.
struct Entry {
  int expert;
  int n;            // tokens
  uint8_t tok[8];
  uint16_t row[8];  // of h: token * K + slot
};
struct Lists {
  int count;
  int pad[3];
  Entry entry[kMaxSlots];
};

struct Weights {
  const uint8_t* q;
  const uint16_t* scales;
  const uint8_t* zeros;
  int rows;    // of an expert
  int pitch;   // bytes of a row
  int groups;  // of a row
};

struct LayerArgs {
  RouteArgs route;
  int route_run;  // of choose_in_shared: the router's own
  bool logits_bf16;
  const uint8_t* x;
  int T, H, N;
  Weights up, down;
  // h [T * K, 2 * pitch]: of every 128 channels the operand's words (place_of), each
  // 32 channels' upper parts before their lower ones; pitch: N in whole blocks of 128
  __nv_bfloat16* h;
  int h_pitch, down_group;
  bool codes_first;  // out of L2, see copy16_first
  Lists* lists;            // of the down projection
  __nv_bfloat16* out;
};

// Sizes of a launch.  A step is 4096 codes: 128 channels of 32 rows (16 of the
// gate, 16 of the up projection), or 256 channels of 16 rows.
template <bool kDown, int kGroup, bool kZeros>
struct Sizes {
  static constexpr int kRows = kDown ? 16 : 32;
  static constexpr int kChannels = kDown ? 256 : 128;
  static constexpr int kColumns = kDown ? 4 : 8;           // tokens of an entry
  static constexpr int kPer = 128 / kGroup;                // groups of 128 channels
  static constexpr int kGroups = kChannels / kGroup;       // of a step
  static constexpr int kScaleRow = kGroups < 2 ? 4 : 2 * kGroups;  // bytes: whole words
  static constexpr int kZeroRow = kGroups < 4 ? 4 : kGroups;
  static constexpr int kCodes = 2048;
  static constexpr int kStage = kCodes + kRows * (kScaleRow + (kZeros ? kZeroRow : 0));
  static constexpr int kStages = 3;
  // a warp's part of a tile whose first step is another warp's; of the down
  // projection also its current tile, both [token][channel]
  static constexpr int kParts = kDown ? 2 * 1024 : 1024;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kBytes = kRing + kWarps * kParts + (int)sizeof(Lists);
};

// Codes i and i + 4 (i = 0..3) of the 8 in w less their zero point, over 64:
// pairs of bf16.  nz: minus the zero point over 64.
__device__ __forceinline__ void codes_over_64(uint32_t w, uint32_t nz, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i ? w >> 8 : w;
    const uint32_t a = v & 0x000F000Fu, b = v & 0x00F000F0u;  // q 2^-133, 16 q 2^-133
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[2 * i]) : "r"(a), "r"(0x7F007F00u), "r"(nz));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[2 * i + 1]) : "r"(b), "r"(0x7D007D00u), "r"(nz));
  }
}
// A pair of -z / 64 from byte k of the zero points in w: z 2^-133 times -2^127.
__device__ __forceinline__ uint32_t minus_zero(uint32_t w, int k) {
  uint32_t o;
  asm("mul.rn.bf16x2 %0, %1, %2;"
      : "=r"(o)
      : "r"(__byte_perm(w, 0, k | 4 << 4 | k << 8 | 4 << 12)), "r"(0xFF00FF00u));
  return o;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
// The first product of a sum.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// The codes pass through L2 as the first to be replaced: otherwise they
// displace what every launch needs again, the kernels' own instructions among it.  That
// pays for calls of few codes (one token 53.1 against 55.2 us, 5 tokens of 4096 x 1024 56.3
// against 59.5); with many, reading ahead is faster (4 tokens 155 against 150 us, 16: 395
// against 372).
__device__ __forceinline__ void copy16_first(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy16_ahead(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_few(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    copy16(dst, src);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes)
                 : "memory");
}

// First of the 8 channels of word j of thread t of a quad, within 128 channels.
template <int kGroup>
__device__ __forceinline__ int channel_of(int t, int j) {
  return kGroup == 128 ? t * 32 + j * 8 : word_channel<kGroup>(t, j);
}

// Where channel c of h is kept within its row: the 8 channels of word j of thread t lie beside
// those of the quad's other threads, so that a warp loads them from one line, and
// within the 8 channel i pairs with i + 4.
__device__ __forceinline__ int place_of(int c, int group) {
  const int t = group == 128 ? c >> 5 & 3 : group == 64 ? c >> 4 & 3 : c >> 3 & 3;
  const int j = group == 128 ? c >> 3 & 3 : group == 64 ? (c >> 5 & 2) | (c >> 3 & 1) : c >> 5 & 3;
  return (c & ~127) * 2 + j * 64 + t * 8 + (c & 3) * 2 + (c >> 2 & 1);
}

// The products of one launch.
template <bool kDown, int kGroup, bool kZeros>
__device__ __forceinline__ void products(const LayerArgs& a, const Lists& l, const float* weight,
                                         uint8_t* smem) {
  using S = Sizes<kDown, kGroup, kZeros>;
  constexpr int kStages = S::kStages, kPer = S::kPer, kRowBytes = S::kChannels / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Weights& W = kDown ? a.down : a.up;
  // channels come in whole groups of at least 32, so tiles of 16 are whole
  const int in = 2 * W.pitch, channels = kDown ? a.H : a.N, tiles = channels / 16;
  const int steps = (in + S::kChannels - 1) / S::kChannels, count = l.count;
  const int items = kDown ? tiles : tiles * count;
  const int item_steps = kDown ? steps * count : steps;
  const int mine = items > (int)blockIdx.x ? (items - (int)blockIdx.x - 1) / (int)gridDim.x + 1 : 0;
  const auto start = [&](int w) { return (int)((int64_t)mine * item_steps * w / kWarps); };
  const int p0 = start(warp), p1 = start(warp + 1);
  const uint64_t policy = l2_policy_evict_first();
  // Scales and zero points of a step can be copied in words; the row is then
  // a whole number of steps.  Else lanes load them one by one.
  const bool words = W.groups % (S::kGroups < 4 ? 4 : S::kGroups) == 0;
  const bool ragged = in % S::kChannels != 0;

  const uint32_t ring = smem_addr(smem) + warp * kStages * S::kStage;
  float* parts = reinterpret_cast<float*>(smem + S::kRing);

  // --- copies: this lane's 16 bytes of each of four rows of a step ---
  constexpr int kLanesRow = kRowBytes / 16;  // lanes a row
  const int lrow = lane / kLanesRow, lcol = lane % kLanesRow * 16;
  const uint8_t* codes = nullptr;
  const uint16_t* scales = nullptr;
  const uint8_t* zeros = nullptr;
  uint32_t row_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    row_at[i] = (uint32_t)(kDown ? 4 * i : 8 * (i & 1) + (i >> 1) * channels) * (uint32_t)W.pitch;
  const auto swizzle = [](int r) {  // of the 16-byte pieces of row r: no bank twice
    return kDown ? (r & 1) << 2 | (r & 2) | (r >> 2 & 1) : chunk_swizzle(r);
  };
  const auto write_at = [&](int i) {
    const int r = kDown ? 4 * i + lrow : 8 * i + lrow;
    return (uint32_t)(r * kRowBytes + ((lcol >> 4 ^ swizzle(r & 7)) << 4));
  };

  struct Cursor {
    int j, e, s;  // tile of the block, entry, step
  };
  const auto tile_of = [&](Cursor& c) {  // the tile's first channel; up: sets its entry
    const int id = (int)blockIdx.x + c.j * (int)gridDim.x;
    if (kDown) return id * 16;
    c.e = id / tiles;
    return (id - c.e * tiles) * 16;
  };
  Cursor load = {0, 0, 0};
  if (p0 < p1) {
    load.j = p0 / item_steps;
    const int rest = p0 - load.j * item_steps;
    if (kDown) load.e = rest / steps;
    load.s = kDown ? rest - load.e * steps : rest;
  }
  Cursor use = load;
  int to_load = p1 - p0, load_n0 = tile_of(load);
  const auto point = [&]() {  // the pointers for `load`
    const int64_t row0 = (int64_t)l.entry[load.e].expert * W.rows + load_n0;
    codes = W.q + (row0 + lrow) * W.pitch + load.s * kRowBytes + lcol;
    const int r = kDown ? lane & 15 : (lane & 15) + (lane >> 4) * channels;
    scales = W.scales + (row0 + r) * W.groups;
    if (kZeros) zeros = W.zeros + (row0 + r) * W.groups;
  };
  if (to_load > 0) point();

  const auto issue = [&](uint32_t stage) {
    if (to_load > 0) {
      --to_load;
      // beyond a row's last channel: any of its bytes, they meet zeros
      const uint8_t* p = codes;
      if (ragged && load.s * kRowBytes + lcol >= W.pitch) p -= load.s * kRowBytes + lcol;
      if (a.codes_first) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy16_first(stage + write_at(i), p + row_at[i], policy);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy16_ahead(stage + write_at(i), p + row_at[i]);
      }
      codes += kRowBytes;
      // of the step's groups; with fewer than a word's, of the whole word
      const int sg = S::kGroups < 2 ? load.s & ~1 : load.s * S::kGroups;
      const int zg = load.s * S::kGroups & ~(S::kZeroRow - 1);
      if (!kDown || lane < 16) {
        const uint32_t dst = stage + S::kCodes + lane * S::kScaleRow;
        if (words) {
          copy_few<S::kScaleRow>(dst, scales + sg);
        } else {
#pragma unroll
          for (int k = 0; k < S::kScaleRow / 2; ++k)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + 2 * k),
                         "h"(__ldg(scales + min(sg + k, W.groups - 1)))
                         : "memory");
        }
      }
      if (kZeros && (!kDown || lane >= 16)) {
        const uint32_t dst = stage + S::kCodes + S::kRows * S::kScaleRow +
                             (kDown ? lane & 15 : lane) * S::kZeroRow;
        if (words) {
          copy_few<S::kZeroRow>(dst, zeros + zg);
        } else {
#pragma unroll
          for (int k = 0; k < S::kZeroRow; ++k)
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(dst + k),
                         "r"((uint32_t)__ldg(zeros + min(zg + k, W.groups - 1)))
                         : "memory");
        }
      }
      if (++load.s == steps) {
        load.s = 0;
        if (!kDown || ++load.e == count) {
          load.e = 0;
          ++load.j;
          load_n0 = tile_of(load);
        }
        if (to_load > 0) point();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) issue(ring + i * S::kStage);

  // --- products ---
  constexpr int kM = kDown ? 1 : 2;  // tiles of sums: gate and up projection
  float acc[kM][4] = {};
  // every step has two tiles of operand A: rows (up) or halves of the channels (down)
  // The columns' words of a step; each is loaded for the next step as soon as it has been
  // multiplied, so that its latency passes behind the products of the others.
  uint4 xv[kDown ? 2 : 1][4];
  const auto column = [&](const uint8_t* xp, int s, int h, int j) {
    const int ch = h * 128 + channel_of<kGroup>(0, j);  // and this thread's, which xp has
    const int at = kDown ? h * 256 + j * 64 : ch;
    if (!ragged || s + 1 < steps || s * S::kChannels + channel_of<kGroup>(t, 0) + ch < in)
      xv[h][j] = __ldg(reinterpret_cast<const uint4*>(xp + 2 * at));
    else
      xv[h][j] = make_uint4(0, 0, 0, 0);
  };
  constexpr int kColumnBytes = S::kChannels * (kDown ? 4 : 2);  // of a step
  const auto step = [&](const uint8_t* xp, int s, uint32_t stage, bool more) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    uint32_t w[2][2][4];  // [tile][row g, row g + 8][word]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t row = stage + (kDown ? r * 8 + g : m * 16 + r * 8 + g) * kRowBytes;
        uint32_t(&o)[4] = w[m][r];
#pragma unroll
        for (int j = 0; j < 4; j += kGroup == 128 ? 4 : kGroup == 64 ? 2 : 1) {
          const int byte = (kDown ? m * 64 : 0) + channel_of<kGroup>(t, j) / 2;
          const uint32_t at = row + ((byte >> 4 ^ swizzle(g)) << 4) + (byte & 15);
          if (kGroup == 128) {
            const uint4 v = lds128(at);
            o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
          } else if (kGroup == 64) {
            const uint2 v = lds64(at);
            o[j] = v.x, o[(j + 1) & 3] = v.y;
          } else {
            o[j] = lds32(at);
          }
        }
      }
    // scales and zero points of rows g and g + 8 (of both tiles: up), packed
    constexpr int kRowSets = kDown ? 1 : 2, kWords = (S::kGroups + 1) / 2;
    uint32_t sw[kRowSets][2][kWords], zw[kRowSets][2][S::kGroups > 4 ? 2 : 1];
#pragma unroll
    for (int m = 0; m < kRowSets; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = m * 16 + r * 8 + g;
        const uint32_t sc = stage + S::kCodes + row * S::kScaleRow;
        uint32_t(&o)[kWords] = sw[m][r];
        if constexpr (S::kGroups == 1) {
          o[0] = lds16(sc + (s & 1) * 2);
        } else if constexpr (kWords == 1) {
          o[0] = lds32(sc);
        } else if constexpr (kWords == 2) {
          const uint2 v = lds64(sc);
          o[0] = v.x, o[1] = v.y;
        } else {
          const uint4 v = lds128(sc);
          o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
        }
        if constexpr (kZeros) {
          const uint32_t zr = stage + S::kCodes + S::kRows * S::kScaleRow + row * S::kZeroRow +
                              (s * S::kGroups & (S::kZeroRow - 1));
          if constexpr (S::kGroups > 4) {
            const uint2 v = lds64(zr);
            zw[m][r][0] = v.x & 0x0F0F0F0Fu, zw[m][r][1] = v.y & 0x0F0F0F0Fu;
          } else {
            zw[m][r][0] = (S::kGroups == 4   ? lds32(zr)
                           : S::kGroups == 2 ? lds16(zr)
                                             : lds8(zr)) & 0x0F0F0F0Fu;
          }
        }
      }
    float part[2][4];
    uint32_t nz[2][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = j / (4 / kPer);  // the word's group
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int group = kDown ? m * kPer + q : q, set = kDown ? 0 : m;
        if (j % (4 / kPer) == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            nz[m][r] = kZeros ? minus_zero(zw[set][r][group >> 2], group & 3) : 0xBE00BE00u;
        }
        uint32_t lo[4], hi[4], b[4];
        codes_over_64(w[m][0][j], nz[m][0], lo);
        codes_over_64(w[m][1][j], nz[m][1], hi);
        if (kDown) {
          const uint4& v = xv[kDown ? m : 0][j];
          b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
        } else {
          pairs_bf16(xv[0][j], b);
        }
        if (j % (4 / kPer) == 0)
          mma_bf16_first(part[m], lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
        else
          mma_bf16(part[m], lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
        mma_bf16(part[m], lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
        if (more && (kDown || m == 1)) column(xp + kColumnBytes, s + 1, kDown ? m : 0, j);
        if ((j + 1) % (4 / kPer) == 0) {  // the end of a group
          float sf[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t word = sw[set][r][group >> 1];
            sf[r] = __uint_as_float(group & 1 ? word & 0xFFFF0000u : word << 16);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& v = acc[kDown ? 0 : m][i];
            v = fmaf(part[m][i], sf[i >> 1], v);
          }
        }
      }
    }
  };

  // Up: the tile's h.  Operands are 1/64 of the weights.
  const auto finish_up = [&](const Entry& e, int n0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 2 * t + (i & 1);
      if (c >= e.n) continue;
      const int row = e.row[c];
      const float v = weight[row] * silu_times(64.0f * acc[0][i], 64.0f * acc[kM - 1][i]);
      const __nv_bfloat16 hi = __float2bfloat16_rn(v);
      const float rest = v - __bfloat162float(hi);
      __nv_bfloat16* to = a.h + (int64_t)row * 2 * a.h_pitch +
                          place_of(n0 + (i >> 1) * 8 + g, a.down_group);
      to[0] = hi;
      // an infinite h leaves nothing
      to[32] = __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.0f);
    }
  };
  // Down: adds the entry's sums to the tile's, and writes a tile.
  const auto add_entry = [&](const Entry& e, float* tile) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = acc[0][i] + __shfl_xor_sync(kFull, acc[0][i], 2);  // h in two parts
      const int c = 2 * t + (i & 1);
      if (t < 2 && c < e.n) tile[e.tok[c] * 16 + (i >> 1) * 8 + g] += v;
    }
    __syncwarp();
  };
  const auto clear_tile = [&](float* tile) {
    for (int i = lane; i < a.T * 16; i += 32) tile[i] = 0.0f;
    __syncwarp();
  };
  const auto finish_down = [&](const float* tile, int n0) {
    for (int i = lane; i < a.T * 16; i += 32)
      a.out[(int64_t)(i >> 4) * a.H + n0 + (i & 15)] = __float2bfloat16_rn(64.0f * tile[i]);
    __syncwarp();
  };
  const auto clear = [&]() {
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
  };

  // a run that begins inside a tile leaves that tile's sums in its first part
  bool head = p0 < p1 && (use.s != 0 || (kDown && use.e != 0));
  float* const first = parts + warp * (S::kParts / 4);
  float* tile = kDown && !head ? first + 256 : first;
  if (kDown) clear_tile(tile);
  int slot = 0, n0 = tile_of(use);
  for (int p = p0; p < p1;) {
    const Entry& e = l.entry[use.e];
    const int n = min(steps - use.s, p1 - p);
    // columns without a token repeat the first: their sums are not used
    const uint8_t* xp;
    if (kDown) {
      const int c = (g & 3) < e.n ? g & 3 : 0;
      xp = reinterpret_cast<const uint8_t*>(a.h + (int64_t)e.row[c] * 2 * a.h_pitch +
                                            (g < 4 ? 0 : 32) + t * 8);
    } else {
      xp = a.x + ((int64_t)e.tok[g < e.n ? g : 0] * a.H + channel_of<kGroup>(t, 0)) * 2;
    }
    xp += use.s * kColumnBytes;
#pragma unroll
    for (int h = 0; h < (kDown ? 2 : 1); ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) column(xp, use.s, h, j);
    for (int i = 0; i < n; ++i) {
      step(xp, use.s + i, ring + slot * S::kStage, i + 1 < n);
      xp += kColumnBytes;
      __syncwarp();
      issue(ring + (slot == 0 ? kStages - 1 : slot - 1) * S::kStage);
      slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    p += n;
    use.s += n;
    if (kDown) {
      add_entry(e, tile);
      clear();
    }
    if (use.s < steps) break;  // the end of the run
    use.s = 0;
    if (kDown && ++use.e < count) continue;
    if (head) {
      if (!kDown) {
#pragma unroll
        for (int m = 0; m < kM; ++m)
          reinterpret_cast<float4*>(first)[m * 32 + lane] =
              make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
      }
      tile = first + 256;
      head = false;
    } else if (kDown) {
      finish_down(tile, n0);
    } else {
      finish_up(e, n0);
    }
    if (kDown) clear_tile(tile);
    clear();
    use.e = 0;
    ++use.j;
    n0 = tile_of(use);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // The end of the run, inside a tile: the warp that has the tile's first step
  // adds the parts of those after it, in order.
  const bool open = p0 < p1 && (use.s != 0 || (kDown && use.e != 0));
  if (!kDown && open && head) {
#pragma unroll
    for (int m = 0; m < kM; ++m)
      reinterpret_cast<float4*>(first)[m * 32 + lane] =
          make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  }
  __syncthreads();
  if (!open || head) return;
  const int end = (use.j + 1) * item_steps;
  for (int v = warp + 1; v < kWarps && start(v) < end; ++v) {
    if (start(v) == start(v + 1)) continue;
    const float* other = parts + v * (S::kParts / 4);
    if (kDown) {
      for (int i = lane; i < a.T * 16; i += 32) tile[i] += other[i];
      __syncwarp();
    } else {
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const float4 f = reinterpret_cast<const float4*>(other)[m * 32 + lane];
        acc[m][0] += f.x, acc[m][1] += f.y, acc[m][2] += f.z, acc[m][3] += f.w;
      }
    }
  }
  if (kDown)
    finish_down(tile, n0);
  else
    finish_up(l.entry[use.e], n0);
}

// Raises the kernel's shared memory, once per device, and launches it.
template <typename Kernel>
bool launch_layer(Kernel kernel, int bytes, bool (&done)[64], std::mutex& mu, const LayerArgs& a,
                  int blocks, cudaStream_t st) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev] && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           bytes) != cudaSuccess)
      return false;
    done[dev] = true;
  }
  return launch_pdl(kernel, (unsigned)blocks, kThreads, bytes, st, a) == cudaSuccess;
}

// The instance for a group size, with zero points or without.
#define EP_LAYER_INSTANCE(KERNEL, DOWN, GROUP, ZEROS)                                            \
  {                                                                                              \
    static std::mutex mu;                                                                        \
    static bool done[64] = {};                                                                   \
    return launch_layer(KERNEL<GROUP, ZEROS>, Sizes<DOWN, GROUP, ZEROS>::kBytes, done, mu, a,    \
                        blocks, st);                                                             \
  }
#define EP_LAYER_INSTANCES(KERNEL, DOWN, WEIGHTS)                     \
  if (WEIGHTS.zeros) {                                                \
    if (group == 32) EP_LAYER_INSTANCE(KERNEL, DOWN, 32, true)        \
    if (group == 64) EP_LAYER_INSTANCE(KERNEL, DOWN, 64, true)        \
    EP_LAYER_INSTANCE(KERNEL, DOWN, 128, true)                        \
  }                                                                   \
  if (group == 32) EP_LAYER_INSTANCE(KERNEL, DOWN, 32, false)         \
  if (group == 64) EP_LAYER_INSTANCE(KERNEL, DOWN, 64, false)         \
  EP_LAYER_INSTANCE(KERNEL, DOWN, 128, false)

}  // namespace ep

// ep_layer_w4.cuh -- a whole mixture-of-experts layer for a few tokens: the
// choice of experts, both products with 4-bit weights, the gated activation and
// the weighted sum over the experts, in two launches.
//
//   h[t,k] = w[t,k] * silu(G_e x[t]) * U_e x[t],  out[t] = sum_k D_e h[t,k],  e = e_k
//
// First launch: every block routes all tokens (a warp each) and makes the list
// of the experts that were chosen; its warps then multiply tiles of 16 gate and
// 16 up channels by the tokens.  Second launch: tiles of 16 output channels,
// each summed over all chosen experts in registers, so that no expert's
// output is ever stored.  The columns of the matrix instruction are the
// tokens themselves: a token that did not choose an expert has zeros there.
//
// What bounds it is the stream of the codes.  A block takes whole tiles, and
// its 16 warps share the tiles' steps (128 channels) evenly: each takes one
// run of consecutive steps, keeps several steps on their way with asynchronous
// copies, and where a tile lies in several warps' runs, its parts are added in the
// order of the channels through shared memory.  The order of every sum depends on the sizes
// and the choice alone, so results repeat bit for bit.
//
// Codes become operands with few instructions: the four bits of a code,
// placed in the low bits of a bf16, are the number q 2^-133 (a subnormal, or
// in the next four bits the first normal numbers, which continue the same
// scale), and one fused multiply-add makes (q - zero) / 64 of it, exactly.  h
// is kept as two bf16 (its rounding, and what that leaves), in columns of
// their own, so the layer's result is rounded once.
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
constexpr int kMaxTokens = 16;
constexpr int kMaxExperts = 1024;
constexpr int kMaxSlots = kMaxTokens * EP_MAX_TOPK;

// The experts that some token chose, in order, and who chose them.
struct Lists {
  int count;
  int pad[3];
  int mask[kMaxSlots];                      // a bit for each token
  uint16_t expert[kMaxSlots];
  uint8_t slot[kMaxSlots * kMaxTokens];     // the token's slot + 1, 0: not chosen
};
static_assert(sizeof(Lists) % 16 == 0, "copied in vectors");

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
  bool logits_bf16, vec;
  int group_lanes;  // of the choice in registers; 0: in shared memory
  const uint8_t* x;
  int T, H, N;
  Weights up, down;
  __nv_bfloat16 *hi, *lo;  // [T * K, N]
  Lists* lists;
  __nv_bfloat16* out;
};

// Shared memory of a launch: the warps' stages, then the parts of tiles that
// lie in several warps' runs, then the lists.
template <bool kDown, int NT>
struct Shared {
  static constexpr int kMT = kDown ? 1 : 2;  // tiles of 16 weight rows
  static constexpr int kRows = 16 * kMT;
  static constexpr int kStages = kDown ? 6 : 4;
  static constexpr int kCodes = kRows * 64;                // of a step
  static constexpr int kStage = kCodes + kRows * (8 + 4);  // and scales and zero points
  static constexpr int kParts = kMT * NT * 512;            // of a warp
  static constexpr int kBytes = kWarps * (kStages * kStage + kParts) + (int)sizeof(Lists);
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
// A pair of -z / 64, z < 16.
__device__ __forceinline__ uint32_t minus_zero(uint32_t z) {
  const uint32_t f = __float_as_uint((float)z * -0.015625f);
  return __byte_perm(f, f, 0x3232);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
template <int kBytes>
__device__ __forceinline__ void copy_few(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes)
               : "memory");
}

// First channel, within a step, of word j of thread t of a quad.
template <int kGroup>
__device__ __forceinline__ int channel_of(int t, int j) {
  return kGroup == 128 ? t * 32 + j * 8 : word_channel<kGroup>(t, j);
}

// A warp's place in its run: tile `j` of the block, chosen expert `e`, step `s`.
struct Cursor {
  int j, e, s, n0;  // n0: the tile's first channel
};

// The products of one launch.
template <bool kDown, int NT, int kGroup, bool kZeros>
__device__ __forceinline__ void products(const LayerArgs& a, const Lists& l, const float* weight,
                                         uint8_t* smem) {
  using S = Shared<kDown, NT>;
  constexpr int kMT = S::kMT, kStages = S::kStages, kPer = 128 / kGroup;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Weights& W = kDown ? a.down : a.up;
  const int in = 2 * W.pitch, channels = kDown ? a.H : a.N, K = a.route.K;
  // channels come in whole groups of at least 32, so tiles are whole
  const int steps = (in + 127) / 128, tiles = channels / 16, count = l.count;
  const int items = kDown ? tiles : tiles * count;
  const int item_steps = kDown ? steps * count : steps;
  const int mine = items > (int)blockIdx.x ? (items - (int)blockIdx.x - 1) / (int)gridDim.x + 1 : 0;
  const auto start = [&](int w) { return (int)((int64_t)mine * item_steps * w / kWarps); };
  const int p0 = start(warp), p1 = start(warp + 1);
  const bool aligned = W.groups % 4 == 0;  // scales and zero points can be copied in words

  const uint32_t ring = smem_addr(smem) + warp * kStages * S::kStage;
  float4* parts = reinterpret_cast<float4*>(smem + kWarps * kStages * S::kStage);

  const auto enter = [&](Cursor& c) {
    const int id = (int)blockIdx.x + c.j * (int)gridDim.x;
    if (kDown) {
      c.n0 = id * 16;
    } else {
      c.e = id / tiles;
      c.n0 = (id - c.e * tiles) * 16;
    }
  };
  const auto advance = [&](Cursor& c) {
    if (++c.s < steps) return;
    c.s = 0;
    if (kDown) {
      if (++c.e < count) return;
      c.e = 0;
    }
    ++c.j;
    enter(c);
  };
  Cursor load = {}, use;
  if (p0 < p1) {
    load.j = p0 / item_steps;
    const int rest = p0 - load.j * item_steps;
    enter(load);
    if (kDown) load.e = rest / steps;
    load.s = kDown ? rest - load.e * steps : rest;
  }
  use = load;
  int to_load = p1 - p0;

  const auto issue = [&](int slot) {
    if (to_load > 0) {
      --to_load;
      const uint32_t stage = ring + slot * S::kStage;
      const int64_t row0 = (int64_t)l.expert[load.e] * W.rows + load.n0;
      // beyond a row's last channel: any of its bytes, they meet zeros
      const int col = load.s * 64 + t * 16;
      const uint8_t* base = W.q + row0 * W.pitch + (col < W.pitch ? col : 0);
      const uint32_t chunk = stage + g * 64 + ((t ^ chunk_swizzle(g)) << 4);
#pragma unroll
      for (int i = 0; i < 2 * kMT; ++i) {
        const int r = g + 8 * (i & 1) + (i >> 1) * channels;
        copy16(chunk + i * 512, base + (uint32_t)r * (uint32_t)W.pitch);
      }
      // scales (8 bytes a row) and zero points (4): of the step's groups, from the
      // last multiple of 2 and of 4 on
      const int half = lane >> 4, r = lane & 15;
      const int sg = kGroup == 128 ? load.s & ~1 : load.s * kPer, zg = load.s * kPer & ~3;
      if (!kDown || half == 0) {
        const uint16_t* p = W.scales + (row0 + r + half * channels) * W.groups;
        const uint32_t dst = stage + S::kCodes + lane * 8;
        if (aligned) {
          copy_few<kGroup == 32 ? 8 : 4>(dst, p + sg);
        } else {
          uint32_t v[2] = {};
#pragma unroll
          for (int k = 0; k < (kGroup == 32 ? 4 : 2); ++k)
            v[k >> 1] |= (uint32_t)__ldg(p + min(sg + k, W.groups - 1)) << (16 * (k & 1));
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(v[0]), "r"(v[1])
                       : "memory");
        }
      }
      if (kZeros && (!kDown || half == 1)) {
        const uint8_t* p = W.zeros + (row0 + r + (kDown ? 0 : half * channels)) * W.groups;
        const uint32_t dst = stage + S::kCodes + S::kRows * 8 + (kDown ? lane & 15 : lane) * 4;
        if (aligned) {
          copy_few<4>(dst, p + zg);
        } else {
          uint32_t v = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v |= (uint32_t)__ldg(p + min(zg + k, W.groups - 1)) << (8 * k);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
        }
      }
      advance(load);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float acc[kMT][NT][4];
  const auto clear = [&]() {
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.0f;
  };
  // The tile's results; operands are 1/64 of the weights.
  const auto finish = [&](const Cursor& c) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ch = c.n0 + g + 8 * (i >> 1);
        if (kDown) {
          float v = acc[0][nt][i];
          v += __shfl_xor_sync(kFull, v, 2);  // what the rounding of h left
          const int tok = nt * 4 + 2 * t + (i & 1);
          if (t < 2 && tok < a.T)
            a.out[(int64_t)tok * a.H + ch] = __float2bfloat16_rn(64.0f * v);
        } else {
          const int tok = nt * 8 + 2 * t + (i & 1);
          const int k = tok < a.T ? l.slot[c.e * kMaxTokens + tok] : 0;
          if (k) {
            const int row = tok * K + k - 1;
            const float v = weight[row] * silu_times(64.0f * acc[0][nt][i],
                                                     64.0f * acc[kMT - 1][nt][i]);
            const __nv_bfloat16 hi = __float2bfloat16_rn(v);
            const float rest = v - __bfloat162float(hi);
            a.hi[(int64_t)row * a.N + ch] = hi;
            // an infinite h leaves nothing
            a.lo[(int64_t)row * a.N + ch] =
                __float2bfloat16_rn(fabsf(v) < INFINITY && fabsf(rest) < INFINITY ? rest : 0.0f);
          }
        }
      }
  };

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  clear();
  bool head = p0 < p1 && (use.s != 0 || (kDown && use.e != 0));
  int slot = 0, expert = -1;
  int mask = 0;
  const uint8_t* xp[NT];

  for (int p = p0; p < p1; ++p) {
    if (use.e != expert || use.s == 0) {
      expert = use.e;
      mask = l.mask[expert];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int tok = kDown ? nt * 4 + (g & 3) : nt * 8 + g;
        const bool in_it = mask >> tok & 1;
        if (kDown) {
          const __nv_bfloat16* base = g < 4 ? a.hi : a.lo;
          const int row = tok * K + l.slot[expert * kMaxTokens + tok] - 1;
          xp[nt] = in_it ? reinterpret_cast<const uint8_t*>(base + (int64_t)row * a.N) : nullptr;
        } else {
          xp[nt] = in_it ? a.x + (int64_t)tok * a.H * 2 : nullptr;
        }
      }
    }
    const auto column = [&](int nt, int j) {
      const int ch = use.s * 128 + channel_of<kGroup>(t, j);
      return xp[nt] && ch < in ? __ldg(reinterpret_cast<const uint4*>(xp[nt] + 2 * ch))
                               : make_uint4(0, 0, 0, 0);
    };
    const auto busy = [&](int nt) {
      return NT == 1 || (mask >> (kDown ? nt * 4 : nt * 8) & (kDown ? 15 : 255));
    };
    constexpr int kAhead = NT > 2 ? 2 : 4;  // words of the columns loaded at once
    uint4 xv[NT][kAhead];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (busy(nt)) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) xv[nt][j] = column(nt, j);
      }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();

    const uint32_t stage = ring + slot * S::kStage;
    uint32_t w[kMT][2][4];
#pragma unroll
    for (int i = 0; i < 2 * kMT; ++i) {
      const uint32_t row = stage + i * 512 + g * 64;
      uint32_t(&o)[4] = w[i >> 1][i & 1];
      if (kGroup == 128) {
        const uint4 v = lds128(row + ((t ^ chunk_swizzle(g)) << 4));
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; j += kGroup == 32 ? 1 : 2) {
          const int byte = word_channel<kGroup>(t, j) / 2;
          const uint32_t at = row + ((byte >> 4 ^ chunk_swizzle(g)) << 4) + (byte & 15);
          if (kGroup == 32) {
            o[j] = lds32(at);
          } else {
            const uint2 v = lds64(at);
            o[j] = v.x, o[j + 1 & 3] = v.y;
          }
        }
      }
    }
    const uint32_t scales = stage + S::kCodes + g * 8 + (kGroup == 128 ? (use.s & 1) * 2 : 0);
    const uint32_t zeros = stage + S::kCodes + S::kRows * 8 + g * 4 + (use.s * kPer & 3);
    float part[kMT][NT][4] = {};
    uint32_t nz[kMT][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = j / (4 / kPer);  // the word's group
      if (j == kAhead) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (busy(nt)) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) xv[nt][k] = column(nt, (kAhead + k) & 3);
          }
      }
      if (j % (4 / kPer) == 0) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            nz[mt][h] =
                kZeros ? minus_zero(lds8(zeros + mt * 64 + h * 32 + q) & 15) : 0xBE00BE00u;
      }
      uint32_t lo[kMT][4], hi[kMT][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        codes_over_64(w[mt][0][j], nz[mt][0], lo[mt]);
        codes_over_64(w[mt][1][j], nz[mt][1], hi[mt]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (busy(nt)) {
          uint32_t b[4];
          pairs_bf16(xv[nt][j % kAhead], b);
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            mma_bf16(part[mt][nt], lo[mt][0], hi[mt][0], lo[mt][1], hi[mt][1], b[0], b[1]);
            mma_bf16(part[mt][nt], lo[mt][2], hi[mt][2], lo[mt][3], hi[mt][3], b[2], b[3]);
          }
        }
      if ((j + 1) % (4 / kPer) == 0) {  // the end of a group
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          const float s0 = __uint_as_float(lds16(scales + mt * 128 + q * 2) << 16);
          const float s1 = __uint_as_float(lds16(scales + mt * 128 + 64 + q * 2) << 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (busy(nt)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                acc[mt][nt][i] = fmaf(part[mt][nt][i], i < 2 ? s0 : s1, acc[mt][nt][i]);
                part[mt][nt][i] = 0.0f;
              }
            }
        }
      }
    }
    const Cursor at = use;
    advance(use);
    if (use.j != at.j) {  // the tile's last step
      if (head) {
#pragma unroll
        for (int i = 0; i < kMT * NT; ++i)
          parts[(warp * kMT * NT + i) * 32 + lane] =
              *reinterpret_cast<const float4*>(acc[i / NT][i % NT]);
        head = false;
      } else {
        finish(at);
      }
      clear();
    }
    __syncwarp();
    issue(slot == 0 ? kStages - 1 : slot - 1);
    slot = slot == kStages - 1 ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // the end of the run, inside a tile: the warp that has the tile's first step
  // adds the parts of those after it
  const bool open = p0 < p1 && (use.s != 0 || (kDown && use.e != 0));
  if (open && head) {
#pragma unroll
    for (int i = 0; i < kMT * NT; ++i)
      parts[(warp * kMT * NT + i) * 32 + lane] =
          *reinterpret_cast<const float4*>(acc[i / NT][i % NT]);
  }
  __syncthreads();
  if (open && !head) {
    const int end = (use.j + 1) * item_steps;
    for (int v = warp + 1; v < kWarps && start(v) < end; ++v) {
      if (start(v) == start(v + 1)) continue;
#pragma unroll
      for (int i = 0; i < kMT * NT; ++i) {
        const float4 f = parts[(v * kMT * NT + i) * 32 + lane];
        float(&c)[4] = acc[i / NT][i % NT];
        c[0] += f.x, c[1] += f.y, c[2] += f.z, c[3] += f.w;
      }
    }
    finish(use);
  }
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
#define EP_LAYER_INSTANCE(KERNEL, DOWN, NT, GROUP, ZEROS)                                          \
  {                                                                                                \
    static std::mutex mu;                                                                          \
    static bool done[64] = {};                                                                     \
    return launch_layer(KERNEL<NT, GROUP, ZEROS>, Shared<DOWN, NT>::kBytes, done, mu, a, blocks, st); \
  }
#define EP_LAYER_GROUPS(KERNEL, DOWN, NT, WEIGHTS)                               \
  if (WEIGHTS.zeros) {                                                           \
    if (group == 32) EP_LAYER_INSTANCE(KERNEL, DOWN, NT, 32, true)               \
    if (group == 64) EP_LAYER_INSTANCE(KERNEL, DOWN, NT, 64, true)               \
    EP_LAYER_INSTANCE(KERNEL, DOWN, NT, 128, true)                               \
  }                                                                              \
  if (group == 32) EP_LAYER_INSTANCE(KERNEL, DOWN, NT, 32, false)                \
  if (group == 64) EP_LAYER_INSTANCE(KERNEL, DOWN, NT, 64, false)                \
  EP_LAYER_INSTANCE(KERNEL, DOWN, NT, 128, false)

}  // namespace ep

// ep_layer_w4.cu -- the entry point of the layer for a few tokens and its first
// launch: routing, gate and up projections, activation (ep_layer_w4.cuh).
#include "ep_layer_w4.cuh"

namespace ep {
namespace {

// What the lists are made of, in shared memory: the experts that some token
// chose, in order, and who chose them.
struct Chosen {
  uint32_t words[kMaxExperts / 32];       // a bit for each expert
  int mask[kMaxSlots];                    // a bit for each token
  uint16_t expert[kMaxSlots];
  uint8_t slot[kMaxSlots][kMaxTokens];    // the token's slot + 1, 0: not chosen
  int sums[kWarps];
};

// The tokens' choices, a warp each; every block computes them alike.
__device__ void route_all(const LayerArgs& a, uint8_t* scratch, int64_t* idx, float* w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= a.T) return;
  uint32_t* key = reinterpret_cast<uint32_t*>(scratch) +
                  warp * (a.route.E + kMaxGroups + 2 * EP_MAX_TOPK);
  float* gscore = reinterpret_cast<float*>(key + a.route.E);
  int* slot = reinterpret_cast<int*>(gscore + kMaxGroups);
  float* score = reinterpret_cast<float*>(slot + EP_MAX_TOPK);
  RouteArgs r = a.route;
  r.idx = idx;
  r.w = w;
  float m, z;
  if (a.logits_bf16) {
    if (a.group_lanes)
      choose_in_registers<32, 8, true>(r, warp, lane, a.group_lanes, a.vec, slot, m, z);
    else
      choose_in_shared<true>(r, warp, lane, key, gscore, slot, m, z);
    __syncwarp();
    write_slots<32, true>(r, warp, true, lane, slot, score, m, z);
  } else {
    if (a.group_lanes)
      choose_in_registers<32, 8, false>(r, warp, lane, a.group_lanes, a.vec, slot, m, z);
    else
      choose_in_shared<false>(r, warp, lane, key, gscore, slot, m, z);
    __syncwarp();
    write_slots<32, false>(r, warp, true, lane, slot, score, m, z);
  }
}

// Which experts the slots name, and for each the tokens; returns their number.
__device__ int gather_chosen(const LayerArgs& a, const int64_t* idx, Chosen& c) {
  const int tid = threadIdx.x, K = a.route.K, slots = a.T * K;
  if (tid < kMaxExperts / 32) c.words[tid] = 0;
  for (int i = tid; i < slots; i += kThreads) {
    c.mask[i] = 0;
    *reinterpret_cast<int4*>(c.slot[i]) = make_int4(0, 0, 0, 0);
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kThreads)
    if (idx[i] >= 0) atomicOr(&c.words[idx[i] >> 5], 1u << (idx[i] & 31));
  __syncthreads();
  int total = 0;
  for (int j = 0; j < (a.route.E + 31) / 32; ++j) total += __popc(c.words[j]);
  for (int i = tid; i < slots; i += kThreads) {
    if (idx[i] < 0) continue;
    const int e = (int)idx[i], t = i / K;
    int at = __popc(c.words[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int j = 0; j < (e >> 5); ++j) at += __popc(c.words[j]);
    c.expert[at] = (uint16_t)e;  // by every slot that names it, alike
    c.slot[at][t] = (uint8_t)(i - t * K + 1);
    atomicOr(&c.mask[at], 1 << t);
  }
  __syncthreads();
  return total;
}

// The entries of `total` experts, each of at most `most` tokens.
__device__ void make_lists(const LayerArgs& a, Chosen& c, int total, int most, Lists& l) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kMaxSlots <= kThreads, "a thread for every chosen expert");
  const int mask = tid < total ? c.mask[tid] : 0;
  const int own = (__popc(mask) + most - 1) / most;
  int at = own;  // sums up to and with this thread
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) c.sums[warp] = at;
  __syncthreads();
  for (int i = 0; i < warp; ++i) at += c.sums[i];
  if (tid == kThreads - 1) l.count = at;
  int k = (at - own) * most;  // entry and column of the next token
  for (int rest = mask; rest; rest &= rest - 1, ++k) {
    const int t = __ffs(rest) - 1;
    Entry& e = l.entry[k / most];
    e.expert = c.expert[tid];
    e.n = min(__popc(rest) + k % most, most);
    e.tok[k % most] = (uint8_t)t;
    e.row[k % most] = (uint16_t)(t * a.route.K + c.slot[tid][t] - 1);
  }
  __syncthreads();
}

template <int kGroup, bool kZeros>
__global__ void __launch_bounds__(kThreads, 1) layer_up_kernel(LayerArgs a) {
  using S = Sizes<false, kGroup, kZeros>;
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t idx[kMaxSlots];
  __shared__ float weight[kMaxSlots];
  // before the products the ring is free
  static_assert(kWarps * (kMaxExperts + kMaxGroups + 2 * EP_MAX_TOPK) * 4 <= S::kRing &&
                    sizeof(Chosen) <= S::kRing,
                "the choice fits into the ring");
  Chosen& c = *reinterpret_cast<Chosen*>(smem);
  Lists& l = *reinterpret_cast<Lists*>(smem + S::kBytes - sizeof(Lists));
  route_all(a, smem, idx, weight);
  __syncthreads();
  const int total = gather_chosen(a, idx, c);
  if (blockIdx.x == gridDim.x - 1) {  // the block with the fewest tiles
    make_lists(a, c, total, Sizes<true, 128, false>::kColumns, l);
    for (int i = threadIdx.x; i < a.T * a.route.K; i += kThreads) {
      a.route.idx[i] = idx[i];
      a.route.w[i] = weight[i];
    }
    for (int i = threadIdx.x; i < 1 + l.count * (int)(sizeof(Entry) / 16); i += kThreads)
      reinterpret_cast<int4*>(a.lists)[i] = reinterpret_cast<const int4*>(&l)[i];
    __syncthreads();
  }
  make_lists(a, c, total, S::kColumns, l);
  products<false, kGroup, kZeros>(a, l, weight, smem);
}

}  // namespace

bool launch_layer_up(const LayerArgs& a, int group, int blocks, cudaStream_t st) {
  EP_LAYER_INSTANCES(layer_up_kernel, false, a.up)
}

namespace {

bool sizes_ok(int64_t T, int H, int N, int E, int K) {
  return T >= 0 && T <= kMaxTokens && H >= 32 && N >= 32 && E >= 1 &&
         E <= kMaxExperts && K >= 1 && K <= EP_MAX_TOPK && K <= E && H <= (1 << 20) &&
         N <= (1 << 20) && (int64_t)H * N < (int64_t(1) << 31);
}
bool weights_ok(const uint8_t* q, const void* scales, const uint8_t* zeros, int group, int in) {
  return (group == 32 || group == 64 || group == 128) && in % group == 0 && q && scales &&
         aligned16(q) && aligned16(scales) && aligned16(zeros);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_layer_w4_workspace_bytes(int64_t num_tokens, int inter, int num_topk) {
  if (num_tokens < 1 || num_tokens > kMaxTokens || inter < 1 || num_topk < 1 ||
      num_topk > EP_MAX_TOPK)
    return 0;
  return sizeof(Lists) + 2 * align_up((size_t)num_tokens * num_topk * inter * 2, 16);
}

extern "C" ep_status_t ep_layer_w4(const void* x, int hidden, int inter, int64_t num_tokens,
                                   const void* logits, int logits_bf16, int64_t row_stride,
                                   const float* bias, int num_experts, int num_topk, int score,
                                   int num_groups, int topk_groups, int renormalize, float scale,
                                   const uint8_t* gate_up_q, const void* gate_up_scales,
                                   const uint8_t* gate_up_zeros, int gate_up_group,
                                   const uint8_t* down_q, const void* down_scales,
                                   const uint8_t* down_zeros, int down_group, int64_t* topk_idx,
                                   float* topk_weights, void* out, void* workspace,
                                   size_t workspace_bytes, ep_stream_t stream) {
  if (!sizes_ok(num_tokens, hidden, inter, num_experts, num_topk) || row_stride < num_experts)
    return EP_ERR_INVALID_ARG;
  if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
  if (num_groups < 1 || num_groups > kMaxGroups || num_experts % num_groups || topk_groups < 1 ||
      topk_groups > num_groups)
    return EP_ERR_INVALID_ARG;
  if (!weights_ok(gate_up_q, gate_up_scales, gate_up_zeros, gate_up_group, hidden) ||
      !weights_ok(down_q, down_scales, down_zeros, down_group, inter))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!x || !logits || !topk_idx || !topk_weights || !out || !workspace) return EP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (logits_bf16 ? 2 : 4) || !aligned16(x) ||
      !aligned16(bias) || !aligned16(topk_idx) || !aligned16(topk_weights) || !aligned16(out) ||
      !aligned16(workspace))
    return EP_ERR_INVALID_ARG;
  if (workspace_bytes < ep_layer_w4_workspace_bytes(num_tokens, inter, num_topk))
    return EP_ERR_CAPACITY;
  // The first launch still reads x and the logits while it writes, and the
  // second writes `out` only after it: out may be x.
  const uint64_t slots = (uint64_t)num_tokens * num_topk, size = logits_bf16 ? 2 : 4;
  const uint64_t lbytes = ((num_tokens - 1) * row_stride + num_experts) * size;
  const uint64_t xbytes = (uint64_t)num_tokens * hidden * 2;
  const struct {
    const void* p;
    uint64_t n;
  } outs[] = {{topk_idx, slots * 8}, {topk_weights, slots * 4}, {workspace, workspace_bytes},
              {out, xbytes}};
  for (int i = 0; i < 4; ++i) {
    if (overlap(outs[i].p, outs[i].n, logits, lbytes)) return EP_ERR_INVALID_ARG;
    if (i < 3 && overlap(outs[i].p, outs[i].n, x, xbytes)) return EP_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return EP_ERR_INVALID_ARG;
  }
  LayerArgs a = {};
  a.route = {logits,      row_stride,  bias, num_tokens, num_experts, num_topk, num_groups,
             topk_groups, score == EP_SCORE_SIGMOID, renormalize != 0, scale, topk_idx,
             topk_weights};
  if (a.route.keep == a.route.G) a.route.G = a.route.keep = 1;  // every group is kept
  a.logits_bf16 = logits_bf16 != 0;
  a.vec = num_experts % 8 == 0 && aligned16(logits) && row_stride * size % 16 == 0;
  const int group = num_experts / a.route.G, lanes = group / 8;
  // eight experts a lane, groups of a power of two of whole lanes: in registers
  a.group_lanes = num_experts > 256 ? 0
                  : a.route.G == 1  ? 32
                  : group % 8 == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  a.x = static_cast<const uint8_t*>(x);
  a.T = (int)num_tokens;
  a.H = hidden;
  a.N = inter;
  a.up = {gate_up_q, static_cast<const uint16_t*>(gate_up_scales), gate_up_zeros, 2 * inter,
          hidden / 2, hidden / gate_up_group};
  a.down = {down_q, static_cast<const uint16_t*>(down_scales), down_zeros, hidden, inter / 2,
            inter / down_group};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.lists = reinterpret_cast<Lists*>(ws);
  a.hi = reinterpret_cast<__nv_bfloat16*>(ws + sizeof(Lists));
  a.lo = reinterpret_cast<__nv_bfloat16*>(ws + sizeof(Lists) + align_up(slots * inter * 2, 16));
  a.out = static_cast<__nv_bfloat16*>(out);
  DeviceProps props;
  if (!device_props(&props)) return EP_ERR_CUDA;
  cudaStream_t st = to_cuda(stream);
  if (!launch_layer_up(a, gate_up_group, props.sm_count, st) ||
      !launch_layer_down(a, down_group, props.sm_count, st)) {
    cudaGetLastError();
    return EP_ERR_CUDA;
  }
  return EP_OK;
}

// ep_layer_w4.cu -- the entry point of the layer for a few tokens and its first
// launch: routing, gate and up projections, activation (ep_layer_w4.cuh).
#include "ep_layer_w4.cuh"

namespace ep {
namespace {

// The tokens' choices, a warp each; every block computes them alike.  A launch
// finds none of its instructions in the SM's caches and fetches each line of them from L2,
// so up to the products the code is kept short: one float32 copy of the logits and the bias in
// shared memory serves all types and strides, and loops are not unrolled.
__device__ void route_all(const LayerArgs& a, float* scratch, int64_t* idx, float* w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.route.E;
  float* logits = scratch;
  float* bias = logits + a.T * E;
#pragma unroll 1
  for (int i = tid; i < (a.route.bias ? a.T + 1 : a.T) * E; i += kThreads) {
    const int t = i / E, e = i - t * E;
    const int64_t at = t * a.route.stride + e;
    float v;
    if (t == a.T)
      v = a.route.bias[e];
    else if (a.logits_bf16)
      v = load_logit<true>(a.route.logits, at);
    else
      v = load_logit<false>(a.route.logits, at);
    logits[i] = v;
  }
  __syncthreads();
  if (warp >= a.T) return;
  uint32_t* key = reinterpret_cast<uint32_t*>(bias + E) + warp * (E + kMaxGroups + 2 * EP_MAX_TOPK);
  float* gscore = reinterpret_cast<float*>(key + E);
  int* slot = reinterpret_cast<int*>(gscore + kMaxGroups);
  float* score = reinterpret_cast<float*>(slot + EP_MAX_TOPK);
  RouteArgs r = a.route;
  r.logits = logits;
  r.stride = E;
  if (r.bias) r.bias = bias;
  r.idx = idx;
  r.w = w;
  float m, z;
  choose_in_shared<false, 1>(r, warp, lane, a.route_run, key, gscore, slot, m, z);
  __syncwarp();
  write_slots<32, false>(r, warp, true, lane, slot, score, m, z);
}

// The entries, each of at most `most` tokens, of the experts in the order of
// their first slots.  A thread looks through all slots for those that name its slot's
// expert; the code is short on purpose, as route_all's is.
__device__ void make_lists(const LayerArgs& a, const int* idx, int* sums, int most, Lists& l) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.route.K;
  static_assert(kMaxSlots <= kThreads, "a thread for every slot");
  const int expert = tid < a.T * K ? idx[tid] : -1;
  int n = 0, before = 0;
  if (expert >= 0) {
#pragma unroll 1
    for (int i = 0; i < a.T * K; ++i) {
      const bool same = idx[i] == expert;
      n += same;
      before += same && i < tid;
    }
  }
  const int own = before ? 0 : (n + most - 1) / most;
  int at = own;  // sums up to and with this thread
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) sums[warp] = at;
  __syncthreads();
  for (int i = 0; i < warp; ++i) at += sums[i];
  if (tid == kThreads - 1) l.count = at;
  if (own) {
    int k = 0;  // of its tokens
    for (int i = tid; k < n; ++i) {
      if (idx[i] != expert) continue;
      Entry& e = l.entry[at - own + k / most];
      e.expert = expert;
      e.n = min(n - k / most * most, most);
      e.tok[k % most] = (uint8_t)(i / K);
      e.row[k % most] = (uint16_t)i;
      ++k;
    }
  }
  __syncthreads();
}

template <int kGroup, bool kZeros>
__global__ void __launch_bounds__(kThreads, 1) layer_up_kernel(LayerArgs a) {
  using S = Sizes<false, kGroup, kZeros>;
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t chosen[kMaxSlots];
  __shared__ float weight[kMaxSlots];
  __shared__ int idx[kMaxSlots], sums[kWarps];
  // before the products the ring is free
  static_assert((kMaxExperts * (2 * kMaxTokens + 1) + kMaxTokens * (kMaxGroups + 2 * EP_MAX_TOPK)) *
                        4 <= S::kRing,
                "the choice fits into the ring");
  Lists& l = *reinterpret_cast<Lists*>(smem + S::kBytes - sizeof(Lists));
  const int tid = threadIdx.x;
  route_all(a, reinterpret_cast<float*>(smem), chosen, weight);
  __syncthreads();
  if (tid < a.T * a.route.K) idx[tid] = (int)chosen[tid];
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1) {  // the block with the fewest tiles
    make_lists(a, idx, sums, Sizes<true, 128, false>::kColumns, l);
    if (tid < a.T * a.route.K) {
      a.route.idx[tid] = chosen[tid];
      a.route.w[tid] = weight[tid];
    }
    for (int i = tid; i < 1 + l.count * (int)(sizeof(Entry) / 16); i += kThreads)
      reinterpret_cast<int4*>(a.lists)[i] = reinterpret_cast<const int4*>(&l)[i];
    __syncthreads();
  }
  make_lists(a, idx, sums, S::kColumns, l);
  products<false, kGroup, kZeros>(a, l, weight, smem);
}

}  // namespace

bool launch_layer_up(const LayerArgs& a, int group, int blocks, cudaStream_t st) {
  EP_LAYER_INSTANCES(layer_up_kernel, false, a.up)
}

namespace {

// Bytes of codes of a call, at most, below which they leave L2 first (copy16_first).
constexpr uint64_t kCodesFirst = 400 << 20;

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
  return sizeof(Lists) + (size_t)num_tokens * num_topk * align_up(inter, 128) * 4;
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
  // Nothing that is written may overlap anything, but for out and x: the second launch,
  // which writes out, does not read x.
  const uint64_t slots = (uint64_t)num_tokens * num_topk, size = logits_bf16 ? 2 : 4;
  const uint64_t xbytes = (uint64_t)num_tokens * hidden * 2;
  const uint64_t all = (uint64_t)num_experts * hidden * inter;  // weights of the down projection
  struct Buffer {
    const void* p;
    uint64_t n;
  };
  const Buffer outs[] = {{topk_idx, slots * 8}, {topk_weights, slots * 4},
                         {workspace, workspace_bytes}, {out, xbytes}};
  const Buffer ins[] = {{logits, ((num_tokens - 1) * row_stride + num_experts) * size},
                        {bias, (uint64_t)num_experts * 4},
                        {gate_up_q, all},
                        {gate_up_scales, 4 * all / gate_up_group},
                        {gate_up_zeros, 2 * all / gate_up_group},
                        {down_q, all / 2},
                        {down_scales, 2 * all / down_group},
                        {down_zeros, all / down_group}};
  for (int i = 0; i < 4; ++i) {
    for (const Buffer& b : ins)
      if (overlap(outs[i].p, outs[i].n, b.p, b.n)) return EP_ERR_INVALID_ARG;
    if (i < 3 && overlap(outs[i].p, outs[i].n, x, xbytes)) return EP_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return EP_ERR_INVALID_ARG;
  }
  LayerArgs a = {};
  a.route = {logits,      row_stride,  bias, num_tokens, num_experts, num_topk, num_groups,
             topk_groups, score == EP_SCORE_SIGMOID, renormalize != 0, scale, topk_idx,
             topk_weights};
  if (a.route.keep == a.route.G) a.route.G = a.route.keep = 1;  // every group is kept
  a.route_run = route_tile(num_experts, a.route.G).vpl;
  a.logits_bf16 = logits_bf16 != 0;
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
  a.h = reinterpret_cast<__nv_bfloat16*>(ws + sizeof(Lists));
  a.h_pitch = (int)align_up(inter, 128);
  a.down_group = down_group;
  a.codes_first = slots * 3 * hidden * inter / 2 < kCodesFirst;
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

// ep_layer_w4_down.cu -- the second launch of the layer for a few tokens: the
// down projection, summed over the experts (ep_layer_w4.cuh).
#include "ep_layer_w4.cuh"

namespace ep {
namespace {

template <int NT, int kGroup, bool kZeros>
__global__ void __launch_bounds__(kThreads, 1) layer_down_kernel(LayerArgs a) {
  using S = Shared<true, NT>;
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t smem[];
  Lists& l = *reinterpret_cast<Lists*>(smem + S::kBytes - sizeof(Lists));
  for (int i = threadIdx.x; i < (int)(sizeof(Lists) / 16); i += kThreads)
    reinterpret_cast<int4*>(&l)[i] = reinterpret_cast<const int4*>(a.lists)[i];
  __syncthreads();
  if (l.count == 0) {  // no token chose any expert
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)a.T * a.H;
         i += (int64_t)gridDim.x * kThreads)
      a.out[i] = __float2bfloat16_rn(0.0f);
    return;
  }
  products<true, NT, kGroup, kZeros>(a, l, nullptr, smem);
}

}  // namespace

bool launch_layer_down(const LayerArgs& a, int group, int blocks, cudaStream_t st) {
  if (a.T <= 4) {
    EP_LAYER_GROUPS(layer_down_kernel, true, 1, a.down)
  }
  if (a.T <= 8) {
    EP_LAYER_GROUPS(layer_down_kernel, true, 2, a.down)
  }
  EP_LAYER_GROUPS(layer_down_kernel, true, 4, a.down)
}

}  // namespace ep

// ep_layer_w4_down.cu -- the second launch of the layer for a few tokens: the
// down projection, summed over the experts (ep_layer_w4.cuh).
#include "ep_layer_w4.cuh"

namespace ep {
namespace {

template <int kGroup, bool kZeros>
__global__ void __launch_bounds__(kThreads, 1) layer_down_kernel(LayerArgs a) {
  using S = Sizes<true, kGroup, kZeros>;
  pdl_wait_then_release();
  extern __shared__ __align__(16) uint8_t smem[];
  Lists& l = *reinterpret_cast<Lists*>(smem + S::kBytes - sizeof(Lists));
  const int count = a.lists->count;
  for (int i = threadIdx.x; i < count * (int)(sizeof(Entry) / 16); i += kThreads)
    reinterpret_cast<int4*>(l.entry)[i] = reinterpret_cast<const int4*>(a.lists->entry)[i];
  if (threadIdx.x == 0) l.count = count;
  __syncthreads();
  if (count == 0) {  // no token chose any expert
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)a.T * a.H;
         i += (int64_t)gridDim.x * kThreads)
      a.out[i] = __float2bfloat16_rn(0.0f);
    return;
  }
  products<true, kGroup, kZeros>(a, l, nullptr, smem);
}

}  // namespace

bool launch_layer_down(const LayerArgs& a, int group, int blocks, cudaStream_t st) {
  EP_LAYER_INSTANCES(layer_down_kernel, true, a.down)
}

}  // namespace ep

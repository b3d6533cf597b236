// The few-token experts' kernels for bf16 weights.
#include "ep_moe.cuh"

namespace ep {

template int launch<0>(const UpArgs &, const DownArgs &, cudaStream_t);

}  // namespace ep

// The few-token experts' kernels for 4-bit weights in groups of 64.
#include "ep_moe.cuh"

namespace ep {

template int launch<64>(const UpArgs &, const DownArgs &, cudaStream_t);

}  // namespace ep

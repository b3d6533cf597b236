// The few-token experts' kernels for 4-bit weights in groups of 32.
#include "ep_moe.cuh"

namespace ep {

template int launch<32>(const UpArgs &, const DownArgs &, cudaStream_t);

}  // namespace ep

// heads_bf16.cu -- the instances of heads.cuh for one storage type.
#include "heads.cuh"

namespace ls {
template cudaError_t launch_heads<bf16>(const HeadsCall&, cudaStream_t);
}  // namespace ls

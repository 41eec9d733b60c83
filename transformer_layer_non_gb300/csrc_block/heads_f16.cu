// heads_f16.cu -- the instances of heads.cuh for one storage type.
#include "heads.cuh"

namespace ls {
template cudaError_t launch_heads<__half>(const HeadsCall&, cudaStream_t);
}  // namespace ls

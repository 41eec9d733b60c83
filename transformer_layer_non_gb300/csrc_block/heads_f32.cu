// heads_f32.cu -- the instances of heads.cuh for one storage type.
#include "heads.cuh"

namespace ls {
template cudaError_t launch_heads<float>(const HeadsCall&, cudaStream_t);
}  // namespace ls

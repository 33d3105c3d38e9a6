// One instantiation unit of the linear-attention walk (linattn_kernels.h): bf16 I/O, q and k
// of at most 256 channels.  Units compile in parallel.
#include "linattn_kernels.h"

namespace selscan {

hipError_t launch_lin_bf16_256(LinWalk walk, const LinParams* p, hipStream_t stream) {
  return lin_choose<uint16_t, 256>(walk, p, stream);
}

}  // namespace selscan

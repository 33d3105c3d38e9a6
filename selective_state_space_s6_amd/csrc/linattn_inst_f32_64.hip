// One instantiation unit of the linear-attention walk (linattn_kernels.h): fp32 I/O, q and k
// of at most 64 channels.  Units compile in parallel.
#include "linattn_kernels.h"

namespace selscan {

hipError_t launch_lin_f32_64(LinWalk walk, const LinParams* p, hipStream_t stream) {
  return lin_choose<float, 64>(walk, p, stream);
}

}  // namespace selscan

// One instantiation unit of the linear-attention walk (linattn_kernels.h): bf16 I/O, q and k
// of at most 256 channels.  Units compile in parallel.
#include "linattn_kernels.h"

namespace selscan {

hipError_t launch_lin_bf16_256(bool rev, bool state, const LinParams& p, hipStream_t stream) {
  return lin_choose<uint16_t, 256>(rev, state, p, stream);
}

}  // namespace selscan

// One instantiation unit of the linear-attention walk (linattn_kernels.h): bf16 I/O, q and k
// of at most 256 channels.  Units compile in parallel.
#include "linattn_kernels.h"

namespace selscan {

hipError_t launch_lin_bf16_256(bool rev, bool state, const LinParams& p, hipStream_t stream) {
  if (p.vd <= 64)
    return p.parts == 3 ? lin_dispatch<uint16_t, 256, 4, 3>(rev, state, p, stream) : lin_dispatch<uint16_t, 256, 4, 2>(rev, state, p, stream);
  return p.parts == 3 ? lin_dispatch<uint16_t, 256, 8, 3>(rev, state, p, stream) : lin_dispatch<uint16_t, 256, 8, 2>(rev, state, p, stream);
}

}  // namespace selscan

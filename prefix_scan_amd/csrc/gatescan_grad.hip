// gatescan_grad.hip -- the gradient of the gated recurrence (gatescan.hpp,
// gatescan_tile.hpp).
#include "gatescan_tile.hpp"

namespace libscan {

hipError_t launch_gatescan_grad(const GateArgs &a, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: return launch_gate_tiles<float, true>(a, stream);
    case LIBSCAN_BF16: return launch_gate_tiles<__bf16, true>(a, stream);
    default: return launch_gate_tiles<_Float16, true>(a, stream);
    }
}

}  // namespace libscan

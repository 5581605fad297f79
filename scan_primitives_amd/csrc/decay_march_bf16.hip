// decay_march_bf16.hip: the marches of decay attention for bf16 operands, rows of whole 16-byte pieces.
#include "decay_march.hpp"

namespace sx {

hipError_t launch_marches_bf16(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  return launch_marches<true, Rows::Whole>(p, first, count, local, stream);
}

}  // namespace sx

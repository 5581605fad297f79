// decay_march_f32.hip: the marches of decay attention for f32 operands, rows of whole 16-byte pieces.
#include "decay_march.hpp"

namespace sx {

hipError_t launch_marches_f32(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  return launch_marches<false, Rows::Whole>(p, first, count, local, stream);
}

}  // namespace sx

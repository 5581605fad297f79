// decay_march_f32_any.hip: the marches of decay attention for f32 operands, rows of any stride, by elements.
#include "decay_march.hpp"

namespace sx {

hipError_t launch_marches_f32_any(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  return launch_marches<false, Rows::Elements>(p, first, count, local, stream);
}

}  // namespace sx

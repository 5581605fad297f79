// decay_march_bf16_any.hip: the marches of decay attention for bf16 operands, rows of any stride, by elements.
#include "decay_march.hpp"

namespace sx {

hipError_t launch_marches_bf16_any(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  return launch_marches<true, Rows::Elements>(p, first, count, local, stream);
}

}  // namespace sx

// decay_march_f32_cut.hip: the marches of decay attention for f32 operands, rows that end in part of a piece.
#include "decay_march.hpp"

namespace sx {

hipError_t launch_marches_f32_cut(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  return launch_marches<false, Rows::Cut>(p, first, count, local, stream);
}

}  // namespace sx

// decay_march_bf16_cut.hip: the marches of decay attention for bf16 operands, rows that end in part of a piece.
#include "decay_march.hpp"

namespace sx {

hipError_t launch_marches_bf16_cut(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  return launch_marches<true, Rows::Cut>(p, first, count, local, stream);
}

}  // namespace sx

// The kernels of gsample_draw.cuh for f16 logits.
#include "gsample_draw.cuh"

namespace gsample {

void* draw_kernel_f16(bool vec, bool verify) {
  return draw_kernel_of<2>(vec, verify);
}

void* verify_draw_kernel_f16(bool vec) { return verify_draw_kernel_of<2>(vec); }

}  // namespace gsample

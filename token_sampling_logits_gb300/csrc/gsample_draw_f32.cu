// The kernels of gsample_draw.cuh for f32 logits.
#include "gsample_draw.cuh"

namespace gsample {

void* draw_kernel_f32(bool vec, bool verify) {
  return draw_kernel_of<0>(vec, verify);
}

void* verify_draw_kernel_f32(bool vec) { return verify_draw_kernel_of<0>(vec); }

}  // namespace gsample

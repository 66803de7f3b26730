// The kernels of gsample_draw.cuh for bf16 logits.
#include "gsample_draw.cuh"

namespace gsample {

void* draw_kernel_bf16(bool vec, bool verify) {
  return draw_kernel_of<1>(vec, verify);
}

void* verify_draw_kernel_bf16(bool vec) { return verify_draw_kernel_of<1>(vec); }

}  // namespace gsample

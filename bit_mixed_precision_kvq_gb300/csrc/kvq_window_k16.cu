// kvq_window_k16.cu -- the windowed decode kernels with bf16 K.
#include "kvq_window.cuh"

namespace kvq {
namespace win {
Kernel window_kernel_k16(int vb, int G, Form f) { return kernel_of<16>(vb, G, f); }
}  // namespace win
}  // namespace kvq

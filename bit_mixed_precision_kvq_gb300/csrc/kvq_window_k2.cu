// kvq_window_k2.cu -- the windowed decode kernels with 2-bit K.
#include "kvq_window.cuh"

namespace kvq {
namespace win {
Kernel window_kernel_k2(int vb, int G, Form f) { return kernel_of<2>(vb, G, f); }
}  // namespace win
}  // namespace kvq

// kvq_window_k4.cu -- the windowed decode kernels with 4-bit K.
#include "kvq_window.cuh"

namespace kvq {
namespace win {
Kernel window_kernel_k4(int vb, int G, Form f) { return kernel_of<4>(vb, G, f); }
}  // namespace win
}  // namespace kvq

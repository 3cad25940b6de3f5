// kvq_window_k8.cu -- the windowed decode kernels with 8-bit K.
#include "kvq_window.cuh"

namespace kvq {
namespace win {
Kernel window_kernel_k8(int vb, int G, Form f) { return kernel_of<8>(vb, G, f); }
}  // namespace win
}  // namespace kvq

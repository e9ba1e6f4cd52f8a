// kernels_window.hip -- attention with a sliding window and a few first tokens
// that stay visible, over a paged cache (attn_kernels.hpp).
#include "attn_kernels.hpp"

namespace lg {

hipError_t launch_window(const WindowArgs& a, int D, int shape, bool f16, bool kv8, hipStream_t s) {
  return launch_any(a, D, shape, f16, kv8, s);
}

}  // namespace lg

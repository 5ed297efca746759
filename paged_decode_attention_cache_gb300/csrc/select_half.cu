// select_half.cu -- page selection over fp16 bounds (fp16 and K8/V4 caches).
#include "select_pages.cuh"

namespace pkv {

cudaError_t launch_select_half(const SelectParams& p, cudaStream_t stream) { return launch_select_t<__half>(p, stream); }

}  // namespace pkv

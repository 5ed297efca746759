// select_e4m3.cu -- page selection over e4m3 bounds.
#include "select_pages.cuh"

namespace pkv {

cudaError_t launch_select_e4m3(const SelectParams& p, cudaStream_t stream) { return launch_select_t<E4M3>(p, stream); }

}  // namespace pkv

// select_i8.cu -- page selection over int8 bounds.
#include "select_pages.cuh"

namespace pkv {

cudaError_t launch_select_i8(const SelectParams& p, cudaStream_t stream) { return launch_select_t<I8>(p, stream); }

}  // namespace pkv

// Attention of drafted trees over float16 pages (one translation unit a cache type
// keeps the build parallel).
#include "tree_attend.cuh"

namespace lc {

int launch_tree_f16(const TreeArgs &a, cudaStream_t cs) { return launch_tree_type<LC_CACHE_F16>(a, cs); }
cudaError_t take_error_tree_f16(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

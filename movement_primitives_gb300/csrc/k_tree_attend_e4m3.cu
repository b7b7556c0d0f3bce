// Attention of drafted trees over E4M3 pages (one translation unit a cache type
// keeps the build parallel).
#include "tree_attend.cuh"

namespace lc {

int launch_tree_e4m3(const TreeArgs &a, cudaStream_t cs) { return launch_tree_type<LC_CACHE_E4M3>(a, cs); }
cudaError_t take_error_tree_e4m3(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

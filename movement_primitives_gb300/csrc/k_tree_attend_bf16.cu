// Attention of drafted trees over bfloat16 pages (one translation unit a cache type
// keeps the build parallel).
#include "tree_attend.cuh"

namespace lc {

int launch_tree_bf16(const TreeArgs &a, cudaStream_t cs) { return launch_tree_type<LC_CACHE_BF16>(a, cs); }
cudaError_t take_error_tree_bf16(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

// Cache attention over E4M3 pages (one translation unit a cache type keeps the
// build parallel).
#include "cache_attend.cuh"

namespace lc {

int launch_attend_e4m3(const AttendArgs &a, int unit_blocks, bool vec, int *runs, cudaStream_t cs) {
    return launch_attend_type<LC_CACHE_E4M3>(a, unit_blocks, vec, runs, cs);
}
cudaError_t take_error_attend_e4m3(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

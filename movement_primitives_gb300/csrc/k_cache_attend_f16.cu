// Cache attention over float16 pages (one translation unit a cache type keeps
// the build parallel).
#include "cache_attend.cuh"

namespace lc {

int launch_attend_f16(const AttendArgs &a, int unit_blocks, bool vec, int *runs, cudaStream_t cs) {
    return launch_attend_type<LC_CACHE_F16>(a, unit_blocks, vec, runs, cs);
}
cudaError_t take_error_attend_f16(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

// Prompt attention of float16 rows (one translation unit a type keeps the build
// parallel).
#include "prompt_attend.cuh"

namespace lc {

int launch_prompt_f16(const PromptArgs &a, int64_t items, cudaStream_t cs) {
    return launch_prompt_type<true>(a, items, cs);
}
cudaError_t take_error_prompt_f16(unsigned long long *v) { return take_module_error(v); }

}  // namespace lc

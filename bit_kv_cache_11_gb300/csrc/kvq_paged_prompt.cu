// Instantiations of the paged prompt kernel.
#include "kvq_paged_prompt.cuh"

namespace kvq {
cudaError_t launch_paged_prompt(const PagedAttnParams& a, int items_max, const CUtensorMap& km,
                                const CUtensorMap& vm, int D, bool bf16, cudaStream_t st) {
  PagedPromptParams p;
  p.a = a;
  p.items_max = items_max;
  if (D == 128)
    return bf16 ? launch_paged_prompt_t<128, true>(p, km, vm, st)
                : launch_paged_prompt_t<128, false>(p, km, vm, st);
  return bf16 ? launch_paged_prompt_t<64, true>(p, km, vm, st)
              : launch_paged_prompt_t<64, false>(p, km, vm, st);
}
}  // namespace kvq

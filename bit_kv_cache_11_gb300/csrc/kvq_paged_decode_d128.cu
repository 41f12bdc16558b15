// Instantiations of the paged decode kernel: head_dim 128.
#include "kvq_paged_decode.cuh"

namespace kvq {
cudaError_t paged_decode_d128(const PagedAttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                            bool bf16, int nt, cudaStream_t st) {
  if (nt == 1)
    return bf16 ? launch_paged_decode_t<128, 1, true, false>(p, km, vm, st)
                : launch_paged_decode_t<128, 1, false, false>(p, km, vm, st);
  return bf16 ? launch_paged_decode_t<128, 2, true, false>(p, km, vm, st)
              : launch_paged_decode_t<128, 2, false, false>(p, km, vm, st);
}
}  // namespace kvq

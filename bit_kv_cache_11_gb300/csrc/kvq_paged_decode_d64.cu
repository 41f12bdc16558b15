// Instantiations of the paged decode kernel: head_dim 64.
#include "kvq_paged_decode.cuh"

namespace kvq {
cudaError_t paged_decode_d64(const PagedAttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                            bool bf16, int nt, cudaStream_t st) {
  if (nt == 1)
    return bf16 ? launch_paged_decode_t<64, 1, true>(p, km, vm, st)
                : launch_paged_decode_t<64, 1, false>(p, km, vm, st);
  return bf16 ? launch_paged_decode_t<64, 2, true>(p, km, vm, st)
              : launch_paged_decode_t<64, 2, false>(p, km, vm, st);
}
}  // namespace kvq

// attn_paged_f16.cu -- the paged attention kernels of one cache type (see attn_paged.cuh)
#include "attn_paged.cuh"

namespace qw {
cudaError_t launch_attn_paged_f16(const PagedArgs &a, int d, int cols, int sms, cudaStream_t st) {
  return paged_launch<kPagedF16>(a, d, cols, sms, st);
}
}  // namespace qw

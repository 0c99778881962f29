// fr_paged_attn_f16.cu -- the paged attention kernels over f16 pages.
#include "fr_paged_attn.cuh"

namespace fr {
namespace paged {

fr_status launch_attn_f16(const KvDesc& kv, const AttnArgs& a, int nt, int ctas, cudaStream_t st) {
    return launch_type<FR_KV_F16>(kv, a, nt, ctas, st);
}

}  // namespace paged
}  // namespace fr

// fr_paged_attn_e4m3.cu -- the paged attention kernels over e4m3 pages.
#include "fr_paged_attn.cuh"

namespace fr {
namespace paged {

fr_status launch_attn_e4m3(const KvDesc& kv, const AttnArgs& a, int nt, int ctas, cudaStream_t st) {
    return launch_type<FR_KV_E4M3>(kv, a, nt, ctas, st);
}

}  // namespace paged
}  // namespace fr

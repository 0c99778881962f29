// fr_paged_qkv_bf16.cu -- the kernels of fr_qkv_post_paged over bf16 rows.
#include "fr_paged_qkv.cuh"

namespace fr {
namespace paged {

fr_status launch_qkv_bf16(const QkvArgs& g, const RopeTable& tb, int hd, bool e4, cudaStream_t st) {
    return launch_qkv<__nv_bfloat16>(g, tb, hd, e4, st);
}

}  // namespace paged
}  // namespace fr

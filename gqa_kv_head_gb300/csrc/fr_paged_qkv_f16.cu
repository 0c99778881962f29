// fr_paged_qkv_f16.cu -- the kernels of fr_qkv_post_paged over f16 rows.
#include "fr_paged_qkv.cuh"

namespace fr {
namespace paged {

fr_status launch_qkv_f16(const QkvArgs& g, const RopeTable& tb, int hd, bool e4, cudaStream_t st) {
    return launch_qkv<__half>(g, tb, hd, e4, st);
}

}  // namespace paged
}  // namespace fr

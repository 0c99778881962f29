// fr_paged_qkv.cu -- fr_qkv_post_paged: checks of its arguments.
#include "fr_paged_qkv.cuh"

using namespace fr;
using namespace fr::paged;

extern "C" fr_status fr_qkv_post_paged(const fr_paged_kv* kv_, const fr_paged_batch* batch_, int row_type, const void* q,
                                       int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                                       int64_t v_stride, const int32_t* pos, int n_head, const float* q_norm,
                                       const float* k_norm, float eps, const fr_rope_params* rp, int interleaved,
                                       float q_scale, uint16_t* q16_out, void* workspace, cudaStream_t stream) {
    const KvDesc* kv = kv_desc(kv_);
    const BatchDesc* bt = batch_desc(batch_);
    if (!kv || !bt || !q || !k_new || !v_new || !pos || !rp || !q16_out) return FR_ERR_INVALID_ARG;
    if (row_type != FR_ROWS_F32 && row_type != FR_ROWS_F16 && row_type != FR_ROWS_BF16) return FR_ERR_INVALID_ARG;
    if (n_head < 1 || (interleaved != 0 && interleaved != 1)) return FR_ERR_INVALID_ARG;
    if (n_head > (1 << 16)) return FR_ERR_UNSUPPORTED;
    if ((q_norm || k_norm) && !(eps >= 0.f && isfinite(eps))) return FR_ERR_INVALID_ARG;
    const int elem = row_type == FR_ROWS_F32 ? 4 : 2;
    QkvArgs g;
    memset(&g, 0, sizeof(g));
    const fr_status bad = append_args(kv_, batch_, elem, k_new, k_stride, v_new, v_stride, pos, workspace, &g.kv);
    if (bad != FR_OK) return bad;
    if (q_stride < (int64_t)n_head * kv->hd || (q_stride & (16 / elem - 1))) return FR_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(q16_out) || !aligned16(q_norm) || !aligned16(k_norm)) return FR_ERR_INVALID_ARG;
    RopeTable tb;
    if (!build_rope_table(rp, resolve_q_scale(q_scale, kv->hd), kv->hd, &tb)) return FR_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FR_ERR_CUDA;
    if (dev != kv->dev || dev != bt->dev) return FR_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k_new, v_new, pos, q16_out, q_norm, k_norm, workspace};
    for (const void* p : ptrs)
        if (p && !device_ptr_ok(p, dev)) return FR_ERR_INVALID_ARG;
    g.q = q;
    g.q_stride = q_stride;
    g.q16 = reinterpret_cast<__half*>(q16_out);
    g.q_norm = Norm{q_norm, eps, interleaved};
    g.k_norm = Norm{k_norm, eps, interleaved};
    g.n_head = n_head;
    const bool e4 = kv->type == FR_KV_E4M3;
    return row_type == FR_ROWS_F32   ? launch_qkv_f32(g, tb, kv->hd, e4, stream)
           : row_type == FR_ROWS_F16 ? launch_qkv_f16(g, tb, kv->hd, e4, stream)
                                     : launch_qkv_bf16(g, tb, kv->hd, e4, stream);
}

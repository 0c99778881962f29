// fr_paged_append.cu -- fr_kv_append_paged: a step's new K and V rows into the
// pages of their sequences (the arithmetic and its layout: fr_paged_rows.cuh).
#include "fr_paged_rows.cuh"

namespace fr {
namespace paged {

// K and V are neighbours, so that K's arithmetic overlaps V's loads.
template <typename T, int HD, bool E4, int KEEP>
__global__ void __launch_bounds__(256)
kv_append_paged_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RopeTable tb) {
    append_piece<T, HD, E4, KEEP, false>(a, tb, Norm{nullptr, 0.f, 0}, blockIdx.x & 1, (int)(blockIdx.x >> 1), blockIdx.y);
}
template <typename T, int HD, bool E4>
__global__ void __launch_bounds__((Prompt<T, E4>::THREADS), (E4 ? 2 : 3))
kv_append_prompt_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RopeTable tb, int shift, int heads) {
    append_prompt<T, HD, E4, false, Prompt<T, E4>::KR, Prompt<T, E4>::HC>(a, tb, Norm{nullptr, 0.f, 0}, shift, heads, blockIdx.x & 1, (int)(blockIdx.x >> 1),
                                    blockIdx.y * heads);
}

template <typename T, int HD, bool E4>
static cudaError_t launch_append(const AppendArgs& a, const RopeTable& tb, cudaStream_t st) {
    // decode: few rows a piece, small blocks
    if (a.n_tok <= 2 * a.n_seq)
        return launch(kv_append_paged_kernel<T, HD, E4, 1>, 2 * most_pieces(a, a.page_shift), a.n_kv_head, 64, st, a, tb);
    const PromptPlan p = plan_prompt<T, HD, E4>(a, tb.n_dims);
    if (!p.heads)
        return launch(kv_append_paged_kernel<T, HD, E4, 4>, 2 * most_pieces(a, a.page_shift), a.n_kv_head, 256, st, a, tb);
    return launch(kv_append_prompt_kernel<T, HD, E4>, 2 * most_pieces(a, p.shift), p.groups, Prompt<T, E4>::THREADS, st, a, tb,
                  p.shift, p.heads);
}
template <typename T, int HD>
static cudaError_t launch_append(const AppendArgs& a, const RopeTable& tb, bool e4, cudaStream_t st) {
    return e4 ? launch_append<T, HD, true>(a, tb, st) : launch_append<T, HD, false>(a, tb, st);
}
template <typename T>
static cudaError_t launch_append(const AppendArgs& a, const RopeTable& tb, int hd, bool e4, cudaStream_t st) {
    return hd == 64 ? launch_append<T, 64>(a, tb, e4, st) : hd == 128 ? launch_append<T, 128>(a, tb, e4, st)
                                                                      : launch_append<T, 256>(a, tb, e4, st);
}

fr_status append_args(const fr_paged_kv* kv_, const fr_paged_batch* batch_, int elem, const void* k_new, int64_t k_stride,
                      const void* v_new, int64_t v_stride, const int32_t* pos, void* workspace, AppendArgs* a) {
    const KvDesc* kv = kv_desc(kv_);
    const BatchDesc* bt = batch_desc(batch_);
    const int64_t least = (int64_t)kv->n_kv_head * kv->hd, step = 16 / elem - 1;
    if (k_stride < least || (k_stride & step) || v_stride < least || (v_stride & step)) return FR_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || ((uintptr_t)pos & 3) || !aligned16(workspace)) return FR_ERR_INVALID_ARG;
    memset(a, 0, sizeof(*a));
    a->k_new = k_new;
    a->v_new = v_new;
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->pos = pos;
    a->tok_start = bt->tok_start;
    a->kv_len = bt->kv_len;
    a->table = bt->table;
    a->table_stride = bt->table_stride;
    a->k = kv->k;
    a->v = kv->v;
    a->k_scale = kv->k_scale;
    a->v_scale = kv->v_scale;
    a->k_page = kv->k_page;
    a->k_head = kv->k_head;
    a->k_row = kv->k_row;
    a->v_page = kv->v_page;
    a->v_head = kv->v_head;
    a->v_row = kv->v_row;
    a->status = reinterpret_cast<unsigned*>(workspace);
    a->n_seq = bt->n_seq;
    a->n_tok = bt->n_tok;
    a->max_pages = bt->max_pages;
    a->n_pages = kv->n_pages;
    a->page_shift = kv->page_shift;
    a->n_kv_head = kv->n_kv_head;
    return FR_OK;
}

}  // namespace paged
}  // namespace fr

using namespace fr;
using namespace fr::paged;

extern "C" fr_status fr_kv_append_paged(const fr_paged_kv* kv_, const fr_paged_batch* batch_, int row_type,
                                        const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                                        const int32_t* pos, const fr_rope_params* rp, void* workspace,
                                        cudaStream_t stream) {
    const KvDesc* kv = kv_desc(kv_);
    const BatchDesc* bt = batch_desc(batch_);
    if (!kv || !bt || !k_new || !v_new || !pos || !rp) return FR_ERR_INVALID_ARG;
    if (row_type != FR_ROWS_F32 && row_type != FR_ROWS_F16) return FR_ERR_INVALID_ARG;
    AppendArgs a;
    const fr_status bad = append_args(kv_, batch_, row_type == FR_ROWS_F32 ? 4 : 2, k_new, k_stride, v_new, v_stride, pos,
                                      workspace, &a);
    if (bad != FR_OK) return bad;
    RopeTable tb;
    if (!build_rope_table(rp, 1.0f, kv->hd, &tb)) return FR_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FR_ERR_CUDA;
    if (dev != kv->dev || dev != bt->dev) return FR_ERR_INVALID_ARG;
    if (!device_ptr_ok(k_new, dev) || !device_ptr_ok(v_new, dev) || !device_ptr_ok(pos, dev) ||
        (workspace && !device_ptr_ok(workspace, dev)))
        return FR_ERR_INVALID_ARG;
    const bool e4 = kv->type == FR_KV_E4M3;
    const cudaError_t e = row_type == FR_ROWS_F32 ? launch_append<float>(a, tb, kv->hd, e4, stream)
                                                  : launch_append<__half>(a, tb, kv->hd, e4, stream);
    return e == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}

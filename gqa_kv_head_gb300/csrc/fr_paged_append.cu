// fr_paged_append.cu -- a step's new K and V rows into the pages of their
// sequences: K rotated as in fr_kv_append, both rounded once to f16, or stored
// as e4m3 codes with one power-of-two scale for each page and head.
//
// Bound by the bytes of the rows read and written; a decode step (one row for
// each sequence) is bound by latency. One block takes one piece (a sequence's
// new rows inside one page) of kHeads heads, K or V: an e4m3 page has its
// scale from every row in it, so one block must see all of a page's new rows.
// A work item is 8 elements of a row: four rotated pairs (or 8 contiguous
// elements), loaded as two vectors and kept in registers between the maximum
// and the rounding, so the rows are read once.
//
// e4m3: s = the smallest power of two with amax <= 448 s over the page. New
// rows may make it grow; the page's earlier codes are then stored again at the
// new scale. The ratio is a power of two, so that moves e4m3 exponents and
// loses nothing but what falls below e4m3's smallest step.
#include <math.h>
#include <string.h>

#include "fr_paged.h"

namespace fr {
namespace paged {

struct AppendArgs {
    const void *k_new, *v_new;
    int64_t k_stride, v_stride;           // elements between tokens
    const int32_t *pos, *tok_start, *kv_len, *table;
    int64_t table_stride;
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t k_page, k_head, k_row, v_page, v_head, v_row;
    unsigned* status;                     // nullable
    int n_seq, n_tok, max_pages, n_pages, page_shift, n_kv_head;
};

constexpr int kKeep = 8;                  // items of a thread held in registers
constexpr int kMinScaleExp = -100;        // smallest scale 2^-100: its reciprocal stays normal

// Smallest power of two s with amax <= 448 s, amax finite and >= 0.
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    // amax = 1.f * 2^e: 448 = 1.75 * 2^8, so s = 2^(e - 8), or twice that above 1.75
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < kMinScaleExp) e = kMinScaleExp;        // zeros and subnormals too
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{ .reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1; cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3; "
        "mov.b32 %0, {lo, hi}; }" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t x) {
    uint32_t h;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, a; }" : "=r"(h) : "r"(x));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x)),
                 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load1<__half>(const __half* p) { return __half2float(__ldg(p)); }

// The 8 elements of item c (slots 4c .. 4c + 3 of a K row, or elements 8c ..
// 8c + 7 of a V row): vectors at d0 and d1, or (single) one dim for each.
struct Item {
    int d[8];
    bool vec;
};

// T: type of the new rows; E4: e4m3 pages; HEADS: heads of one block.
template <typename T, int HD, bool E4, int HEADS>
__global__ void __launch_bounds__(256)
kv_append_paged_kernel(const AppendArgs a, const __grid_constant__ RopeTable tb) {
    constexpr int ITEMS = HD / 8;                 // items of a row
    constexpr int KEEP = kKeep / HEADS;
    __shared__ int sc[16];
    __shared__ float red[8][HEADS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, warps = nthr >> 5;
    const bool is_v = blockIdx.z != 0;
    const int ps = 1 << a.page_shift;

    // ---- which piece: the sequences' pieces in order, counted from kv_len -----
    const int64_t want = blockIdx.x;
    int64_t base = 0;
    bool found = false;
    for (int b0 = 0; b0 < a.n_seq && !found; b0 += nthr) {
        const int b = b0 + tid;
        int n = 0, first = 0, tok0 = 0, n_q = 0;
        bool bad = false;
        if (b < a.n_seq) {
            const SeqInfo s = seq_info(a.tok_start, a.kv_len, b, a.n_tok, a.max_pages, a.page_shift);
            bad = s.bad || s.n_q > s.n_kv;
            if (!bad && s.n_q > 0) {
                tok0 = s.tok0;
                n_q = s.n_q;
                first = s.n_kv - s.n_q;
                n = ((s.n_kv - 1) >> a.page_shift) - (first >> a.page_shift) + 1;
            }
        }
        if (bad && a.status && want == 0 && blockIdx.y == 0 && !is_v) atomicOr(a.status, kStatusInput);
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) sc[warp] = inc;
        if (tid == 0) sc[8] = -1;
        __syncthreads();
        int64_t off = base;
        for (int w = 0; w < warp; ++w) off += sc[w];
        const int64_t end = off + inc;
        if (n > 0 && want >= end - n && want < end) {
            sc[8] = b;
            sc[9] = (int)(want - (end - n));
            sc[10] = first;
            sc[11] = tok0;
            sc[12] = n_q;
        }
        int64_t all = 0;
        for (int w = 0; w < warps; ++w) all += sc[w];
        base += all;
        __syncthreads();
        found = sc[8] >= 0;
        if (!found) __syncthreads();
    }
    if (!found) return;
    const int b = sc[8], first = sc[10], last = first + sc[12];          // cache rows [first, last) are new
    const int pi = (first >> a.page_shift) + sc[9];                      // page of the sequence
    const int page = __ldcg(a.table + b * a.table_stride + pi);
    if (page < 0 || page >= a.n_pages) {
        if (tid == 0 && a.status) atomicOr(a.status, kStatusInput);
        return;
    }
    const int r0 = max(first - (pi << a.page_shift), 0), r1 = min(last - (pi << a.page_shift), ps);
    const int tok = sc[11] + (pi << a.page_shift) + r0 - first;          // token of row r0
    const int h0 = blockIdx.y * HEADS, nh = min(HEADS, a.n_kv_head - h0);
    const T* src = reinterpret_cast<const T*>(is_v ? a.v_new : a.k_new);
    const int64_t s_tok = is_v ? a.v_stride : a.k_stride;
    const int64_t p_page = is_v ? a.v_page : a.k_page, p_head = is_v ? a.v_head : a.k_head, p_row = is_v ? a.v_row : a.k_row;
    const int n_items = (r1 - r0) * ITEMS;
    const bool vec = is_v || (tb.n_dims & 7) == 0;

    auto item_dims = [&](int c) {
        Item it;
        it.vec = vec;
        if (is_v) {
#pragma unroll
            for (int u = 0; u < 8; ++u) it.d[u] = c * 8 + u;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                int x, y;
                rope_slot_dims(c * 4 + u, tb, x, y);
                it.d[2 * u] = x;
                it.d[2 * u + 1] = y;
            }
        }
        return it;
    };
    // Elements in slot order: x[2u], x[2u + 1] are slot u's two dims. A rotated
    // vector item has its first dims at d[0] .. d[0] + 3 and its second ones at
    // d[1] .. d[1] + 3; the others are 8 contiguous elements from d[0].
    auto rotated = [&](int c) { return !is_v && c * 4 < tb.half; };
    auto load = [&](const Item& it, int c, const T* row, float* x) {
        if (it.vec) {
            const bool rot = rotated(c);
            const float4 p = load4<T>(row + it.d[0]), q = load4<T>(row + (rot ? it.d[1] : it.d[0] + 4));
            if (rot) {
                x[0] = p.x; x[2] = p.y; x[4] = p.z; x[6] = p.w;
                x[1] = q.x; x[3] = q.y; x[5] = q.z; x[7] = q.w;
            } else {
                x[0] = p.x; x[1] = p.y; x[2] = p.z; x[3] = p.w;
                x[4] = q.x; x[5] = q.y; x[6] = q.z; x[7] = q.w;
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = load1<T>(row + it.d[u]);
        }
    };
    auto angles = [&](int c, int t, float* cs, float* sn) {
        if (is_v) return;
        const int p = __ldg(a.pos + t);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c * 4 + u < tb.half) rope_cs_tab(p, c * 4 + u, tb, cs[u], sn[u]);
    };
    auto rotate = [&](int c, const float* cs, const float* sn, float* x) {
        if (is_v) return;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c * 4 + u < tb.half) {
                const float x0 = x[2 * u], x1 = x[2 * u + 1];
                x[2 * u] = rope_lo(x0, x1, cs[u], sn[u], 1.f);
                x[2 * u + 1] = rope_hi(x0, x1, cs[u], sn[u], 1.f);
            }
    };
    auto store = [&](const Item& it, int c, int64_t at, const float* x, float inv) {
        const bool rot = rotated(c);
        if (E4) {
            unsigned char* dst = reinterpret_cast<unsigned char*>(is_v ? a.v : a.k) + at;
            if (it.vec) {
                const uint32_t p = rot ? to_e4m3x4(x[0] * inv, x[2] * inv, x[4] * inv, x[6] * inv)
                                       : to_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                const uint32_t q = rot ? to_e4m3x4(x[1] * inv, x[3] * inv, x[5] * inv, x[7] * inv)
                                       : to_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
                if (rot) {
                    *reinterpret_cast<uint32_t*>(dst + it.d[0]) = p;
                    *reinterpret_cast<uint32_t*>(dst + it.d[1]) = q;
                } else {
                    *reinterpret_cast<uint2*>(dst + it.d[0]) = make_uint2(p, q);
                }
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) dst[it.d[u]] = (unsigned char)to_e4m3x4(x[u] * inv, 0.f, 0.f, 0.f);
            }
        } else {
            __half* dst = reinterpret_cast<__half*>(is_v ? a.v : a.k) + at;
            if (it.vec) {
                const uint2 p = rot ? make_uint2(pack_half2(x[0], x[2]), pack_half2(x[4], x[6]))
                                    : make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
                const uint2 q = rot ? make_uint2(pack_half2(x[1], x[3]), pack_half2(x[5], x[7]))
                                    : make_uint2(pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
                if (rot) {
                    *reinterpret_cast<uint2*>(dst + it.d[0]) = p;
                    *reinterpret_cast<uint2*>(dst + it.d[1]) = q;
                } else {
                    *reinterpret_cast<uint4*>(dst + it.d[0]) = make_uint4(p.x, p.y, q.x, q.y);
                }
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) dst[it.d[u]] = __float2half_rn(x[u]);
            }
        }
    };
    auto at_row = [&](int r, int h) { return page * p_page + (int64_t)h * p_head + (int64_t)r * p_row; };

    if (!E4) {
        for (int w = tid; w < n_items; w += nthr) {
            const int i = w / ITEMS, c = w - i * ITEMS;
            const T* row = src + (int64_t)(tok + i) * s_tok + (int64_t)h0 * HD;
            const Item it = item_dims(c);
            float x[HEADS][8], cs[4], sn[4];
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h < nh) load(it, c, row + h * HD, x[h]);
            angles(c, tok + i, cs, sn);
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h < nh) {
                    rotate(c, cs, sn, x[h]);
                    store(it, c, at_row(r0 + i, h0 + h), x[h], 1.f);
                }
        }
        return;
    }

    // ---- e4m3: the largest finite value first ------------------------------
    float* scale = (is_v ? a.v_scale : a.k_scale) + (int64_t)page * a.n_kv_head + h0;
    float kept[KEEP][HEADS][8], amax[HEADS], old[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        amax[h] = 0.f;
        old[h] = r0 > 0 && h < nh ? scale[h] : 0.f;           // a page's first rows start it anew
    }
    auto fetch = [&](int w, float (*x)[8]) {
        const int i = w / ITEMS, c = w - i * ITEMS;
        const T* row = src + (int64_t)(tok + i) * s_tok + (int64_t)h0 * HD;
        const Item it = item_dims(c);
        float cs[4], sn[4];
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
            if (h < nh) load(it, c, row + h * HD, x[h]);
        angles(c, tok + i, cs, sn);
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
            if (h < nh) rotate(c, cs, sn, x[h]);
    };
    auto widen = [&](float (*x)[8]) {
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
            if (h < nh)
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float v = fabsf(x[h][u]);
                    if (v <= 3.402823466e38f) amax[h] = fmaxf(amax[h], v);    // inf and NaN set no scale
                }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (tid + k * nthr < n_items) {
            fetch(tid + k * nthr, kept[k]);
            widen(kept[k]);
        }
    for (int w = tid + KEEP * nthr; w < n_items; w += nthr) {
        float x[HEADS][8];
        fetch(w, x);
        widen(x);
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
#pragma unroll
        for (int o = 16; o; o >>= 1) amax[h] = fmaxf(amax[h], __shfl_xor_sync(~0u, amax[h], o));
        if (lane == 0) red[warp][h] = amax[h];
    }
    __syncthreads();
    float inv[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        float m = red[0][h];
        for (int w = 1; w < warps; ++w) m = fmaxf(m, red[w][h]);
        const float s = fmaxf(pow2_scale(m), old[h]);
        inv[h] = 1.f / s;
        if (h < nh) {
            if (tid == 0) scale[h] = s;
            if (r0 > 0 && s > old[h]) {                       // the page's earlier rows at the grown scale
                const float ratio = old[h] / s;
                for (int w = tid; w < r0 * (HD / 8); w += nthr) {
                    const int r = w / (HD / 8), c = w - r * (HD / 8);
                    uint2* p = reinterpret_cast<uint2*>(reinterpret_cast<unsigned char*>(is_v ? a.v : a.k) +
                                                        at_row(r, h0 + h) + c * 8);
                    uint2 x = *p;
                    const float2 a0 = from_e4m3x2(x.x & 0xffffu), a1 = from_e4m3x2(x.x >> 16),
                                 a2 = from_e4m3x2(x.y & 0xffffu), a3 = from_e4m3x2(x.y >> 16);
                    x.x = to_e4m3x4(a0.x * ratio, a0.y * ratio, a1.x * ratio, a1.y * ratio);
                    x.y = to_e4m3x4(a2.x * ratio, a2.y * ratio, a3.x * ratio, a3.y * ratio);
                    *p = x;
                }
            }
        }
    }
    auto put = [&](int w, float (*x)[8]) {
        const int i = w / ITEMS, c = w - i * ITEMS;
        const Item it = item_dims(c);
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
            if (h < nh) store(it, c, at_row(r0 + i, h0 + h), x[h], inv[h]);
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (tid + k * nthr < n_items) put(tid + k * nthr, kept[k]);
    for (int w = tid + KEEP * nthr; w < n_items; w += nthr) {
        float x[HEADS][8];
        fetch(w, x);
        put(w, x);
    }
}

template <typename T, int HD, bool E4>
static cudaError_t launch_append(const AppendArgs& a, const RopeTable& tb, cudaStream_t st) {
    // at most one piece a token, and for each sequence its whole pages and two partly new ones
    const int64_t by_page = 2 * (int64_t)a.n_seq + (a.n_tok >> a.page_shift);
    const int64_t pieces = a.n_tok < by_page ? a.n_tok : by_page;
    // two heads share a block's angles once there are blocks enough without
    const bool two = a.n_kv_head > 1 && pieces * a.n_kv_head >= 608;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)pieces, (unsigned)(two ? (a.n_kv_head + 1) / 2 : a.n_kv_head), 2);
    cfg.blockDim = dim3(a.n_tok <= 2 * a.n_seq ? 64 : 256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return two ? cudaLaunchKernelEx(&cfg, kv_append_paged_kernel<T, HD, E4, 2>, a, tb)
               : cudaLaunchKernelEx(&cfg, kv_append_paged_kernel<T, HD, E4, 1>, a, tb);
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
    const int64_t least = (int64_t)kv->n_kv_head * kv->hd, step = row_type == FR_ROWS_F32 ? 3 : 7;
    if (k_stride < least || (k_stride & step) || v_stride < least || (v_stride & step)) return FR_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || ((uintptr_t)pos & 3) || !aligned16(workspace)) return FR_ERR_INVALID_ARG;
    RopeTable tb;
    if (!build_rope_table(rp, 1.0f, kv->hd, &tb)) return FR_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FR_ERR_CUDA;
    if (dev != kv->dev || dev != bt->dev) return FR_ERR_INVALID_ARG;
    if (!device_ptr_ok(k_new, dev) || !device_ptr_ok(v_new, dev) || !device_ptr_ok(pos, dev) ||
        (workspace && !device_ptr_ok(workspace, dev)))
        return FR_ERR_INVALID_ARG;
    AppendArgs a;
    memset(&a, 0, sizeof(a));
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.pos = pos;
    a.tok_start = bt->tok_start;
    a.kv_len = bt->kv_len;
    a.table = bt->table;
    a.table_stride = bt->table_stride;
    a.k = kv->k;
    a.v = kv->v;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
    a.k_page = kv->k_page;
    a.k_head = kv->k_head;
    a.k_row = kv->k_row;
    a.v_page = kv->v_page;
    a.v_head = kv->v_head;
    a.v_row = kv->v_row;
    a.status = reinterpret_cast<unsigned*>(workspace);
    a.n_seq = bt->n_seq;
    a.n_tok = bt->n_tok;
    a.max_pages = bt->max_pages;
    a.n_pages = kv->n_pages;
    a.page_shift = kv->page_shift;
    a.n_kv_head = kv->n_kv_head;
    const bool e4 = kv->type == FR_KV_E4M3;
    const cudaError_t e = row_type == FR_ROWS_F32 ? launch_append<float>(a, tb, kv->hd, e4, stream)
                                                  : launch_append<__half>(a, tb, kv->hd, e4, stream);
    return e == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}

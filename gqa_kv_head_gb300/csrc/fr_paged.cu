// fr_paged.cu -- the paged-cache entry points: descriptors of a cache and of a
// step's batch, argument checks, the attention's launch choices and the kernel
// that merges the states of split segments.
#include <math.h>
#include <string.h>

#include "fr_paged.h"
#include "fr_sm100.cuh"

namespace fr {
namespace paged {

using sm100::ex2;

// The states (m, l, O) of one split segment's row become its output row:
//   out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p,
// in the order of the pieces, whatever order they were computed in. One block
// per (segment, row, 4 * cols dims): thread = (4 dims, group of states). Bound by
// latency, and by how slowly one SM reads lines that others have just written,
// so a row is spread over blocks and the first kAhead states of each group are
// asked for before the weights are known. Blocks of unsplit segments leave at
// once.
constexpr int kAhead = 4, kMergeThreads = 512;

__global__ void __launch_bounds__(kMergeThreads)
paged_merge_kernel(const Split* __restrict__ split, const int* __restrict__ n_split, const float* __restrict__ part_o,
                   const float2* __restrict__ part_ml, float* __restrict__ out, int row_tile, int hd, int group,
                   int n_kv_head, int cols) {
    __shared__ float red_l[kMergeThreads / 32], red_m[kMergeThreads / 32];
    extern __shared__ float4 red[];                 // [threads], then the states' weights
    float* wt = reinterpret_cast<float*>(red + blockDim.x);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int n_entries = __ldcg(n_split);
    const int4 s0 = __ldcg(reinterpret_cast<const int4*>(split + blockIdx.x));
    const int2 s1 = __ldcg(reinterpret_cast<const int2*>(split + blockIdx.x) + 2);
    const int first = s0.x, n = s0.y - first + 1, tok0 = s0.z, row0 = s0.w, rows = s1.x, head = s1.y;
    if ((int)blockIdx.x >= n_entries || n < 1) return;
    const int groups = blockDim.x / cols, c = blockIdx.z * cols + tid % cols, gi = tid / cols;
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        auto slot = [&](int p) { return (int64_t)(2 * (first + p) + (p == 0 ? 1 : 0)) * row_tile + row; };
        float4 ahead[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int p = gi + i * groups;
            ahead[i] = p < n ? __ldcg(reinterpret_cast<const float4*>(part_o + slot(p) * hd) + c) : make_float4(0, 0, 0, 0);
        }
        const float2 mine = tid < n ? __ldcg(part_ml + slot(tid)) : make_float2(-INFINITY, 0.f);
        float m = mine.x;
        for (int p = tid + blockDim.x; p < n; p += blockDim.x) m = fmaxf(m, __ldcg(part_ml + slot(p)).x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (lane == 0) red_m[warp] = m;
        __syncthreads();
        m = red_m[0];
        for (int w = 1; w < warps; ++w) m = fmaxf(m, red_m[w]);
        float l = 0.f;
        for (int p = tid; p < n; p += blockDim.x) {
            const float2 ml = p == tid ? mine : __ldcg(part_ml + slot(p));
            const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
            wt[p] = w;
            l += w == 0.f ? 0.f : w * ml.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
        if (lane == 0) red_l[warp] = l;
        __syncthreads();
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](int p, const float4& y) {
            const float w = wt[p];
            if (w == 0.f) return;                   // an empty state may hold anything
            x.x += w * y.x;
            x.y += w * y.y;
            x.z += w * y.z;
            x.w += w * y.w;
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (gi + i * groups < n) add(gi + i * groups, ahead[i]);
#pragma unroll 8
        for (int p = gi + kAhead * groups; p < n; p += groups)
            add(p, __ldcg(reinterpret_cast<const float4*>(part_o + slot(p) * hd) + c));
        red[tid] = x;
        __syncthreads();
        if (gi == 0) {
            l = 0.f;
            for (int w = 0; w < warps; ++w) l += red_l[w];
            for (int i = 1; i < groups; ++i) {
                const float4 y = red[i * cols + tid];
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
            const float inv = m == -INFINITY ? 0.f : 1.f / l;
            const int i = (row0 + row) / group, hh = row0 + row - i * group;
            float* dst = out + ((int64_t)(tok0 + i) * n_kv_head * group + head * group + hh) * hd + c * 4;
            *reinterpret_cast<float4*>(dst) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        }
        if (row + (int)gridDim.y < rows) __syncthreads();   // the shared arrays are read
    }
    // The next kernel on the stream may start now, and not before: attention
    // CTAs that find merge blocks in their SM's shared memory may not fit beside
    // them and would start only when another one ends.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- descriptors ---------------------------------------------------------------

// Strides of a [n_pages][n_kv_head][page_size][hd] view: 16-byte multiples, and
// no two elements at one address (an expanded view would be written twice).
static bool strides_ok(const int64_t* st, int n_pages, int n_head, int page_size, int hd, int elem) {
    struct D { int64_t stride; int n; } d[3] = {{st[0], n_pages}, {st[1], n_head}, {st[2], page_size}};
    for (int i = 0; i < 3; ++i) {
        if (d[i].n == 1) continue;                 // the stride of a size-1 dimension is never used
        if (d[i].stride <= 0 || (d[i].stride * elem) % 16 != 0 || d[i].stride > (int64_t{1} << 40) / elem - 1) return false;
    }
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if ((d[j].n == 1 ? 0 : d[j].stride) < (d[i].n == 1 ? 0 : d[i].stride)) {
                const D t = d[i];
                d[i] = d[j];
                d[j] = t;
            }
    int64_t extent = hd;
    for (int i = 0; i < 3; ++i) {
        if (d[i].n == 1) continue;
        if (d[i].stride < extent) return false;
        if (d[i].stride > (int64_t{1} << 62) / d[i].n - extent / d[i].n - 1) return false;   // (no memory is that large)
        extent += d[i].stride * (d[i].n - 1);
    }
    return true;
}

static bool encode_pages(unsigned char* dst, const KvDesc& d, const void* base, int64_t page, int64_t head, int64_t row,
                         int box_rows, bool tc) {
    auto enc = get_encoder();
    if (!enc) return false;
    const bool e4 = d.type == FR_KV_E4M3;
    const int elem = e4 ? 1 : 2, row_bytes = d.hd * elem, box_bytes = row_bytes < 128 ? row_bytes : 128;
    const cuuint32_t in_box = box_bytes / elem;
    cuuint64_t dims[5] = {in_box, (cuuint64_t)d.page_size, (cuuint64_t)(row_bytes / box_bytes), (cuuint64_t)d.n_kv_head,
                          (cuuint64_t)d.n_pages};
    // the stride of a size-1 dimension is never used, but has to be valid
    cuuint64_t strides[4] = {(cuuint64_t)row * elem, (cuuint64_t)box_bytes, (cuuint64_t)(d.n_kv_head > 1 ? head * elem : 16),
                             (cuuint64_t)(d.n_pages > 1 ? page * elem : 16)};
    cuuint32_t box[5] = {in_box, (cuuint32_t)box_rows, tc ? 1u : (cuuint32_t)(row_bytes / box_bytes), 1, 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    CUtensorMap m;
    if (enc(&m, e4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(base), dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            tc && e4 ? CU_TENSOR_MAP_SWIZZLE_NONE : box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    memcpy(dst, &m, sizeof(m));
    return true;
}

// Average query rows of a sequence and KV head from which the 128-row kernel is
// taken: where the small tiles would read the keys twice, at hd 256 in e4m3 four
// times. Small tiles and one of 128, us, 64 sequences of 1..8000 keys, 4 KV heads:
//   f16   hd 64, 32 rows 85 and 115, 36 rows 135 and 133, 64 rows 148 and 135; hd 128, 32
//         rows 125 and 130, 36 rows 196 and 148; hd 256, 16 rows 174 and 202, 20 rows 327
//         and 203, 36 rows 480 and 207
//   e4m3  hd 64, 32 rows 104 and 172, 36 rows 168 and 169, 64 rows 183 and 171; hd 128, 36
//         rows 247 and 240, 64 rows 279 and 242; hd 256, 36 rows 294 and 326, 52 rows 382
//         and 329, 64 rows 393 and 331
// and 65536 keys, 8 KV heads, hd 128, 32 rows: f16 62 and 71, e4m3 68 and 102. Two
// tiles of 16 rows over few long segments run side by side and meet in L2: hd 256,
// 32 rows, 65536 keys of 1, 2, 4 heads 27 and 30, 37 and 43, 59 and 64; 16 x 8000
// keys 29 and 32; 64 x 2000 keys 39 and 37.
// Those calls keep their choice, and with it their sums' order. With sinks, and the 128-row
// kernel since faster: window 2048, small tiles and one of 128, us, 64 sequences of 4 heads,
// 16 of 2, 2 of 8:
//   f16   hd 128, 16 rows 52 and 67, 19 and 21.5, 13.5 and 16; 20 rows 82 and 67, 22.9 and 21.6,
//         18.8 and 16.2; 32 rows 87 and 69; hd 64, 20 rows 61 and 61, 36 rows 100 and 63; hd 256,
//         20 rows 162 and 108, 27.4 and 26.6, 19.5 and 19.8; 36 rows 238 and 113, 34 and 27
//   e4m3  hd 64, 32 rows 76 and 108, 36 rows 115 and 111; hd 128, 32 rows 111 and 140, 36 rows
//         166 and 142; hd 256, 36 rows 189 and 182, 37 and 39; 64 rows 246 and 185, 45 and 41
static int many_rows(int hd, int type, int64_t segs, bool sinks) {
    if (sinks && hd == 128 && type == FR_KV_F16) return 17;
    return hd < 256 ? 33 : type == FR_KV_E4M3 ? 49 : segs >= 32 ? 17 : 33;
}
static int max_nt(int hd) { return hd == 256 ? 2 : 4; }
// Attention CTAs for row tiles of 8*nt rows on a GPU of sms SMs (the workspace is sized for the most)
static int ctas_for(int hd, int nt, int sms) {
    const int per = ctas_per_sm(hd, nt), most = kMaxCtas * per / 4;
    return per * sms < most ? per * sms : most;
}
static size_t ws_rows(int hd) {        // rows of split states, two states for each CTA
    size_t n = 0;
    for (int nt = 1; nt <= max_nt(hd); nt *= 2) {
        const size_t r = (size_t)2 * ctas_for(hd, nt, kMaxCtas) * 8 * nt;
        if (r > n) n = r;
    }
    return n < (size_t)2 * kTcCtas * kTcRows ? (size_t)2 * kTcCtas * kTcRows : n;
}
static size_t ws_bytes(int hd) {
    return kWsHeader + sizeof(Split) * kMaxCtas + ws_rows(hd) * (sizeof(float2) + 4 * (size_t)hd);
}

}  // namespace paged
}  // namespace fr

using namespace fr;
using namespace fr::paged;

extern "C" fr_status fr_paged_kv_init(fr_paged_kv* kv, int type, void* k, const int64_t* k_strides, void* v,
                                      const int64_t* v_strides, float* k_scale, float* v_scale, int n_pages,
                                      int page_size, int n_kv_head, int hd) {
    if (!kv || !k || !v || !k_strides || !v_strides) return FR_ERR_INVALID_ARG;
    memset(kv, 0, sizeof(*kv));
    if (type != FR_KV_F16 && type != FR_KV_E4M3) return FR_ERR_INVALID_ARG;
    if (n_pages < 1 || n_kv_head < 1 || page_size < 1 || hd < 1) return FR_ERR_INVALID_ARG;
    if (hd != 64 && hd != 128 && hd != 256) return FR_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return FR_ERR_UNSUPPORTED;
    if (n_kv_head > 65535) return FR_ERR_UNSUPPORTED;
    const bool e4 = type == FR_KV_E4M3;
    if (e4 ? !k_scale || !v_scale : k_scale || v_scale) return FR_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || (((uintptr_t)k_scale | (uintptr_t)v_scale) & 3)) return FR_ERR_INVALID_ARG;
    const int elem = e4 ? 1 : 2;
    if (!strides_ok(k_strides, n_pages, n_kv_head, page_size, hd, elem) ||
        !strides_ok(v_strides, n_pages, n_kv_head, page_size, hd, elem))
        return FR_ERR_INVALID_ARG;
    KvDesc d;
    memset(&d, 0, sizeof(d));
    if (cudaGetDevice(&d.dev) != cudaSuccess) return FR_ERR_CUDA;
    if (!device_ptr_ok(k, d.dev) || !device_ptr_ok(v, d.dev) || (e4 && (!device_ptr_ok(k_scale, d.dev) ||
                                                                       !device_ptr_ok(v_scale, d.dev))))
        return FR_ERR_INVALID_ARG;
    d.k = k;
    d.v = v;
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.k_page = k_strides[0];
    d.k_head = k_strides[1];
    d.k_row = k_strides[2];
    d.v_page = v_strides[0];
    d.v_head = v_strides[1];
    d.v_row = v_strides[2];
    d.n_pages = n_pages;
    d.page_size = page_size;
    d.page_shift = __builtin_ctz((unsigned)page_size);
    d.n_kv_head = n_kv_head;
    d.hd = hd;
    d.type = type;
    d.magic = kKvMagic;
    if (!encode_pages(d.k_map, d, k, d.k_page, d.k_head, d.k_row, kTile, false) ||
        !encode_pages(d.v_map, d, v, d.v_page, d.v_head, d.v_row, kTile, false))
        return FR_ERR_CUDA;
    const int rows = tc_box_rows(page_size, hd, e4);
    if (!encode_pages(d.k_map_tc, d, k, d.k_page, d.k_head, d.k_row, rows, true) ||
        !encode_pages(d.v_map_tc, d, v, d.v_page, d.v_head, d.v_row, rows, true))
        return FR_ERR_CUDA;
    memcpy(kv, &d, sizeof(d));
    return FR_OK;
}

extern "C" fr_status fr_paged_batch_init(fr_paged_batch* batch, const int32_t* tok_start, const int32_t* kv_len,
                                         const int32_t* page_table, int64_t page_table_stride, int n_seq, int n_tok,
                                         int max_pages) {
    if (!batch || !tok_start || !kv_len || !page_table) return FR_ERR_INVALID_ARG;
    memset(batch, 0, sizeof(*batch));
    if (n_seq < 1 || n_tok < 1 || max_pages < 1 || page_table_stride < max_pages) return FR_ERR_INVALID_ARG;
    if (n_seq > kMaxSeq || n_tok > (1 << 20) || max_pages > (1 << 22)) return FR_ERR_UNSUPPORTED;
    if (((uintptr_t)tok_start | (uintptr_t)kv_len | (uintptr_t)page_table) & 3) return FR_ERR_INVALID_ARG;
    BatchDesc d;
    memset(&d, 0, sizeof(d));
    if (cudaGetDevice(&d.dev) != cudaSuccess) return FR_ERR_CUDA;
    if (!device_ptr_ok(tok_start, d.dev) || !device_ptr_ok(kv_len, d.dev) || !device_ptr_ok(page_table, d.dev))
        return FR_ERR_INVALID_ARG;
    d.tok_start = tok_start;
    d.kv_len = kv_len;
    d.table = page_table;
    d.table_stride = page_table_stride;
    d.n_seq = n_seq;
    d.n_tok = n_tok;
    d.max_pages = max_pages;
    d.magic = kBatchMagic;
    memcpy(batch, &d, sizeof(d));
    return FR_OK;
}

extern "C" size_t fr_paged_attn_workspace_size(int n_head, int n_kv_head, int hd) {
    if (n_head < 1 || n_kv_head < 1 || n_head % n_kv_head) return 0;
    if (hd != 64 && hd != 128 && hd != 256) return 0;
    return ws_bytes(hd);
}

extern "C" fr_status fr_paged_attn(const fr_paged_kv* kv, const fr_paged_batch* batch, const uint16_t* q16,
                                   int64_t q_tok_stride, int n_head, int causal, int window, float kq_scale, float* out,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return fr_paged_attn_sinks(kv, batch, q16, q_tok_stride, n_head, causal, window, 0, kq_scale, out, workspace,
                               workspace_bytes, stream);
}

extern "C" fr_status fr_paged_attn_sinks(const fr_paged_kv* kv_, const fr_paged_batch* batch_, const uint16_t* q16,
                                         int64_t q_tok_stride, int n_head, int causal, int window, int n_sink,
                                         float kq_scale, float* out, void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream) {
    const KvDesc* kv = kv_desc(kv_);
    const BatchDesc* bt = batch_desc(batch_);
    if (!kv || !bt || !q16 || !out || !workspace) return FR_ERR_INVALID_ARG;
    if (n_head < 1 || n_head % kv->n_kv_head) return FR_ERR_INVALID_ARG;
    if (n_head > (1 << 16)) return FR_ERR_UNSUPPORTED;
    if (q_tok_stride < (int64_t)n_head * kv->hd || (q_tok_stride & 7)) return FR_ERR_INVALID_ARG;
    const float scale_log2 = (float)((double)kq_scale * 1.4426950408889634);
    if (window < 0 || (window > 0 && !causal) || !isfinite(scale_log2)) return FR_ERR_INVALID_ARG;
    if (n_sink < 0 || (n_sink > 0 && window == 0)) return FR_ERR_INVALID_ARG;
    if (!aligned16(q16) || !aligned16(out) || !aligned16(workspace)) return FR_ERR_INVALID_ARG;
    if (((int64_t)bt->max_pages << kv->page_shift) > 0x7fff0000) return FR_ERR_UNSUPPORTED;
    if (workspace_bytes < ws_bytes(kv->hd)) return FR_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FR_ERR_CUDA;
    if (dev != kv->dev || dev != bt->dev) return FR_ERR_INVALID_ARG;
    if (!device_ptr_ok(q16, dev) || !device_ptr_ok(out, dev) || !device_ptr_ok(workspace, dev)) return FR_ERR_INVALID_ARG;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return FR_ERR_CUDA;

    const int G = n_head / kv->n_kv_head;
    // Row tile: 8 rows for each MMA column block, as many blocks as an average
    // sequence of the batch fills (a longer one takes several row tiles)
    const int64_t most_keys = (int64_t)bt->max_pages << kv->page_shift;
    // a window that no sequence outgrows is none (and positions less it stay in 32 bits)
    const bool windowed = window > 0 && window < most_keys, sinks = windowed && n_sink > 0;
    const int64_t avg = (int64_t)G * ((bt->n_tok + bt->n_seq - 1) / bt->n_seq);
    const int nt = avg <= 8 ? 1 : avg <= 16 ? 2 : max_nt(kv->hd);
    const bool many = avg >= many_rows(kv->hd, kv->type, (int64_t)bt->n_seq * kv->n_kv_head, sinks) && G <= kTcRows;
    const int rt = many ? kTcRows / G * G : 8 * nt;
    const int part_rows = many ? kTcRows : rt;        // rows of a state in the workspace
    // at most this many segments, and units of work, whatever the lengths say
    const int64_t per_tok = (int64_t)bt->n_tok * ((G + rt - 1) / rt), per_seq = bt->n_seq + (int64_t)bt->n_tok * G / rt;
    const int64_t segs = (per_tok < per_seq ? per_tok : per_seq) * kv->n_kv_head;
    const int64_t cap_units = (((int64_t)bt->max_pages << kv->page_shift) + kUnit - 1) / kUnit;
    int64_t ctas = !many ? ctas_for(kv->hd, nt, sms) : sms < kTcCtas ? sms : kTcCtas;
    const int64_t cap = segs * (cap_units + (many ? kTcSegCost : kSegCost));
    if (cap > 0x7fffffff) return FR_ERR_UNSUPPORTED;
    if (cap < ctas) ctas = cap;

    char* w = reinterpret_cast<char*>(workspace);
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.q16 = reinterpret_cast<const __half*>(q16);
    a.q_stride = q_tok_stride;
    a.out = out;
    a.tok_start = bt->tok_start;
    a.kv_len = bt->kv_len;
    a.table = bt->table;
    a.table_stride = bt->table_stride;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
    a.status = reinterpret_cast<unsigned*>(w);
    a.n_split = reinterpret_cast<int*>(w + 64);
    a.split = reinterpret_cast<Split*>(w + kWsHeader);
    a.part_ml = reinterpret_cast<float2*>(w + kWsHeader + sizeof(Split) * kMaxCtas);
    a.part_o = reinterpret_cast<float*>(a.part_ml + ws_rows(kv->hd));
    a.n_seq = bt->n_seq;
    a.n_tok = bt->n_tok;
    a.max_pages = bt->max_pages;
    a.n_pages = kv->n_pages;
    a.page_shift = kv->page_shift;
    a.n_kv_head = kv->n_kv_head;
    a.group = G;
    // r * ceil(2^32 / G) / 2^32 = r / G + r e / (2^32 G) with e < G: exact below r e < 2^32
    if (G > 1 && (int64_t)bt->n_tok * G * G < (int64_t{1} << 32)) a.group_magic = (unsigned)(((uint64_t{1} << 32) + G - 1) / G);
    a.row_tile = rt;
    a.causal = causal ? 1 : 0;
    a.window = windowed ? window : 0;
    a.sink = !sinks ? 0 : n_sink < most_keys ? n_sink : (int)most_keys;
    a.split_by_segment = segs <= ctas ? 1 : 0;
    a.scale_log2 = scale_log2;
    const fr_status st = many                     ? launch_attn_tc(*kv, a, (int)ctas, stream)
                         : kv->type == FR_KV_E4M3 ? launch_attn_e4m3(*kv, a, nt, (int)ctas, stream)
                                                : launch_attn_f16(*kv, a, nt, (int)ctas, stream);
    if (st != FR_OK) return st;

    const int64_t rows = a.split_by_segment ? ((int64_t)G * bt->n_tok < rt ? (int64_t)G * bt->n_tok : rt)
                                            : (avg < rt ? avg : rt);      // (a block goes on to the rows behind)
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    // threads for the states that a segment has when all are as long: kAhead for each group
    const int64_t usual = bt->n_tok < bt->n_seq ? bt->n_tok : bt->n_seq * ((avg + rt - 1) / rt);
    const int64_t groups = (ctas / (usual * kv->n_kv_head) + 2 + kAhead - 1) / kAhead;
    const int64_t entries = a.split_by_segment ? segs : ctas;
    // few rows in all: 64 dims to a block, so that more SMs read the fresh states; many: fewer blocks
    const int cols = kv->hd > 64 && entries * rows > 608 ? 32 : 16;
    int64_t threads = (groups * cols + 31) / 32 * 32;
    // no more blocks than run at a time: prompts have many states of many rows, and
    // most entries nothing to join (2048 tokens: 23 -> 13 us)
    const int64_t z = kv->hd / (4 * cols), wave = (int64_t)sms * 32 / (entries * z);
    cfg.gridDim = dim3((unsigned)entries, (unsigned)(rows <= wave ? rows : wave < 1 ? 1 : wave), (unsigned)z);
    cfg.blockDim = dim3((unsigned)(threads > kMergeThreads ? kMergeThreads : threads));
    cfg.dynamicSmemBytes = cfg.blockDim.x * sizeof(float4) + kMaxCtas * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_merge_kernel, (const Split*)a.split, (const int*)a.n_split,
                                             (const float*)a.part_o, (const float2*)a.part_ml, out, part_rows, kv->hd, G,
                                             kv->n_kv_head, cols);
    return e == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}

// fr_paged_append.cu -- a step's new K and V rows into the pages of their
// sequences: K rotated as in fr_kv_append, both rounded once to f16, or stored
// as e4m3 codes with one power-of-two scale for each page and head.
//
// Bound by the bytes of the rows read and written; a decode step (one row for
// each sequence) is bound by latency. A block takes one piece (a sequence's new
// rows inside one page, or for f16 pages inside a part of one), K or V:
//   * one head, small blocks (kv_append_paged_kernel): decode steps, and the
//     shapes that the other kernel leaves out;
//   * several heads one after the other (kv_append_prompt_kernel): prompts. The
//     angles of a row are the same for every head, and at about 100 instructions
//     an angle, computed for each head again, they took longer than the bytes.
//     So a thread keeps the cosines and sines of its few row places in
//     registers and takes head after head through them. (Shared over a cluster
//     through its distributed memory instead, they took as long as before.)
// An e4m3 page has its scale from every row in it, so one block sees all of a
// page's new rows of a head; rows are read once and stay in registers between
// the maximum and the rounding.
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

// Scaled cosines and sines of a thread's four slots. One copy of the code: inlined
// for every element, the slow reduction of sincosf alone would outgrow the
// instruction cache.
__device__ __noinline__ float2 rope_cs_fixed(int pos, uint64_t turns, float mscale) {
    float2 r;
    rope_cs(pos, turns, mscale, r.x, r.y);
    return r;
}
__device__ __noinline__ float2 rope_cs_f32(int pos, int i, const RopeTable* tb) {
    float2 r;
    rope_cs_tab(pos, i, *tb, r.x, r.y);
    return r;
}
struct Angles {
    uint64_t turns[4];                            // of slots 4c .. 4c + 3 (exact mode)
    // The constants are asked for at once, ahead of everything: read where they
    // are used they cost a fresh block two trips to memory in a row.
    __device__ __forceinline__ void get(const RopeTable& tb, int c) {
#pragma unroll
        for (int u = 0; u < 4; ++u) turns[u] = tb.turns[min(c * 4 + u, kMaxPairs - 1)];
    }
    __device__ __forceinline__ float2 at(int pos, int c, int u, const RopeTable& tb) const {
        return tb.mode == FR_ROPE_GGML_F32 ? rope_cs_f32(pos, c * 4 + u, &tb) : rope_cs_fixed(pos, turns[u], tb.mscale);
    }
};

// Four elements of a row as they come, and as floats.
template <typename T> struct Raw;
template <> struct Raw<float> {
    using V = float4;
    __device__ static __forceinline__ float4 floats(const V& v) { return v; }
    __device__ static __forceinline__ float one(const float* p) { return *p; }
};
template <> struct Raw<__half> {
    using V = uint2;
    __device__ static __forceinline__ float4 floats(const V& v) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)),
                     b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    __device__ static __forceinline__ float one(const __half* p) { return __half2float(*p); }
};

// The nth piece: the sequences' pieces (of 2^shift rows at most, aligned) in
// order, counted from their lengths. Every warp finds it alone, with no barrier
// ahead of the loads, 128 sequences at a time so that their numbers arrive together.
struct Piece {
    int b, first, last, tok, row0, row1;      // sequence; its new cache rows; token of row0; the piece's cache rows
    bool found;
};
__device__ __forceinline__ Piece find_piece(const AppendArgs& a, int shift, int nth) {
    const int lane = threadIdx.x & 31;
    Piece p;
    p.found = false;
    for (int b0 = 0; b0 < a.n_seq && !p.found; b0 += 128) {
        int f[4], t[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = t[i] = q[i] = 0;
            if (b0 + i * 32 + lane < a.n_seq) {
                const SeqInfo s = seq_info(a.tok_start, a.kv_len, b0 + i * 32 + lane, a.n_tok, a.max_pages, a.page_shift);
                if (!s.bad && s.n_q <= s.n_kv) {
                    f[i] = s.n_kv - s.n_q;
                    t[i] = s.tok0;
                    q[i] = s.n_q;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p.found) continue;
            const int n = q[i] > 0 ? ((f[i] + q[i] - 1) >> shift) - (f[i] >> shift) + 1 : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += x;
            }
            const unsigned hit = __ballot_sync(~0u, nth < inc);        // the first of these lanes has it
            if (hit) {
                const int at = __ffs(hit) - 1;
                p.found = true;
                p.b = b0 + i * 32 + at;
                p.first = __shfl_sync(~0u, f[i], at);
                p.last = p.first + __shfl_sync(~0u, q[i], at);
                const int unit = (p.first >> shift) + nth - __shfl_sync(~0u, inc - n, at);
                p.row0 = max(p.first, unit << shift);
                p.row1 = min(p.last, (unit + 1) << shift);
                p.tok = __shfl_sync(~0u, t[i], at) + p.row0 - p.first;
            } else {
                nth -= __shfl_sync(~0u, inc, 31);
            }
        }
    }
    return p;
}
// One warp of the grid looks at every sequence's numbers.
__device__ __forceinline__ void report_bad(const AppendArgs& a) {
    if (!a.status || blockIdx.x || blockIdx.y || threadIdx.x >= 32) return;
    bool bad = false;
    for (int i = threadIdx.x; i < a.n_seq; i += 32) {
        const SeqInfo s = seq_info(a.tok_start, a.kv_len, i, a.n_tok, a.max_pages, a.page_shift);
        bad |= s.bad || s.n_q > s.n_kv;
    }
    if (bad) atomicOr(a.status, kStatusInput);
}
// An e4m3 page's rows 0 .. rows - 1, hd of them a row, at a scale grown by 1 / ratio.
__device__ __forceinline__ void restore_rows(unsigned char* page, int rows, int items, int64_t row_stride, float ratio) {
    for (int w = threadIdx.x; w < rows * items; w += blockDim.x) {
        uint2* p = reinterpret_cast<uint2*>(page + w / items * row_stride + w % items * 8);
        uint2 y = *p;
        const float2 a0 = from_e4m3x2(y.x & 0xffffu), a1 = from_e4m3x2(y.x >> 16), a2 = from_e4m3x2(y.y & 0xffffu),
                     a3 = from_e4m3x2(y.y >> 16);
        y.x = to_e4m3x4(a0.x * ratio, a0.y * ratio, a1.x * ratio, a1.y * ratio);
        y.y = to_e4m3x4(a2.x * ratio, a2.y * ratio, a3.x * ratio, a3.y * ratio);
        *p = y;
    }
}
// The larger of m and the finite magnitudes of y (infinities and NaN set no scale).
__device__ __forceinline__ float widen(float m0, const float* y) {
    float m = m0;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = fmaxf(m, fabsf(y[u]));                // (NaN leaves it)
    if (m > 3.402823466e38f) {
        m = m0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (fabsf(y[u]) <= 3.402823466e38f) m = fmaxf(m, fabsf(y[u]));
    }
    return m;
}
// rope_lo and rope_hi at scale 1.
__device__ __forceinline__ void rotate(float& lo, float& hi, const float2& cs) {
    const float x = lo, y = hi;
    lo = __fmaf_rn(x, cs.x, -__fmul_rn(y, cs.y));
    hi = __fmaf_rn(x, cs.y, __fmul_rn(y, cs.x));
}

// T: type of the new rows; E4: e4m3 pages; KEEP: items of a thread held in registers.
template <typename T, int HD, bool E4, int KEEP>
__global__ void __launch_bounds__(256)
kv_append_paged_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RopeTable tb) {
    constexpr int ITEMS = HD / 8;                 // items of a row
    using V = typename Raw<T>::V;
    __shared__ float red[8];
    const bool is_v = blockIdx.x & 1;             // neighbours, so that K's arithmetic overlaps V's loads
    Angles angles;
    if (!is_v) angles.get(tb, threadIdx.x % ITEMS);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, warps = nthr >> 5;
    const Piece pc = find_piece(a, a.page_shift, (int)(blockIdx.x >> 1));
    report_bad(a);
    if (!pc.found) return;                                               // fewer pieces than blocks
    const int pi = pc.row0 >> a.page_shift;                              // page of the sequence
    const int page = a.table[pc.b * a.table_stride + pi];
    const int r0 = pc.row0 - (pi << a.page_shift), tok = pc.tok;
    const int h = blockIdx.y;
    const T* src = reinterpret_cast<const T*>(is_v ? a.v_new : a.k_new) + (int64_t)tok * (is_v ? a.v_stride : a.k_stride) + h * HD;
    const int64_t s_tok = is_v ? a.v_stride : a.k_stride;
    const int64_t p_row = is_v ? a.v_row : a.k_row;
    const int64_t p_base = page * (is_v ? a.v_page : a.k_page) + h * (is_v ? a.v_head : a.k_head);

    // This thread's items: rows r, r + rstep, ... of the piece, all at place c of
    // their row (a block's threads are a multiple of a row's items). x[u] and
    // x[4 + u] are the two dims of slot 4c + u: where rotated dims come as
    // vectors, at d0 .. d0 + 3 and d1 .. d1 + 3; other vectors are 8 contiguous
    // elements, which no rotation touches.
    const int c = tid % ITEMS, r = tid / ITEMS, rstep = nthr / ITEMS, n_rows = pc.row1 - pc.row0;
    const bool vec = is_v || (tb.n_dims & 7) == 0, rot = !is_v && c * 4 < tb.half;
    const int d0 = rot ? c * 4 : c * 8, d1 = rot ? c * 4 + tb.half : c * 8 + 4;
    V raw[KEEP][2];
    float x[E4 ? KEEP : 1][8];
    auto load = [&](int i, V* v) {
        if (i < n_rows && vec) {
            const T* row = src + i * s_tok;
            v[0] = *reinterpret_cast<const V*>(row + d0);
            v[1] = *reinterpret_cast<const V*>(row + d1);
        }
    };
    // item (row i, place c) as rotated floats, from its vectors or (n_dims no multiple of 8) element by element
    auto values = [&](int i, const V* v, float* y) {
        if (vec) {
            const float4 p = Raw<T>::floats(v[0]), q = Raw<T>::floats(v[1]);
            y[0] = p.x; y[1] = p.y; y[2] = p.z; y[3] = p.w;
            y[4] = q.x; y[5] = q.y; y[6] = q.z; y[7] = q.w;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                int p, q;
                rope_slot_dims(c * 4 + u, tb, p, q);
                y[u] = Raw<T>::one(src + i * s_tok + p);
                y[4 + u] = Raw<T>::one(src + i * s_tok + q);
            }
        }
        if (!rot) return;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c * 4 + u < tb.half) rotate(y[u], y[4 + u], angles.at(a.pos[tok + i], c, u, tb));
    };
    auto store = [&](int i, const float* y, float inv) {
        const int64_t at = p_base + (r0 + i) * p_row;
        if (E4) {
            unsigned char* dst = reinterpret_cast<unsigned char*>(is_v ? a.v : a.k) + at;
            if (vec) {
                *reinterpret_cast<uint32_t*>(dst + d0) = to_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                *reinterpret_cast<uint32_t*>(dst + d1) = to_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    int p, q;
                    rope_slot_dims(c * 4 + u, tb, p, q);
                    dst[p] = (unsigned char)to_e4m3x4(y[u] * inv, 0.f, 0.f, 0.f);
                    dst[q] = (unsigned char)to_e4m3x4(y[4 + u] * inv, 0.f, 0.f, 0.f);
                }
            }
        } else {
            __half* dst = reinterpret_cast<__half*>(is_v ? a.v : a.k) + at;
            if (vec) {
                *reinterpret_cast<uint2*>(dst + d0) = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
                *reinterpret_cast<uint2*>(dst + d1) = make_uint2(pack_half2(y[4], y[5]), pack_half2(y[6], y[7]));
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    int p, q;
                    rope_slot_dims(c * 4 + u, tb, p, q);
                    dst[p] = __float2half_rn(y[u]);
                    dst[q] = __float2half_rn(y[4 + u]);
                }
            }
        }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k) load(r + k * rstep, raw[k]);
    const bool bad_page = page < 0 || page >= a.n_pages;
    if (bad_page && tid == 0 && a.status) atomicOr(a.status, kStatusInput);
    if (bad_page) return;
    const int behind = r + KEEP * rstep;          // rows that registers do not hold
    if (!E4) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const int i = r + k * rstep;
            if (i >= n_rows) break;
            values(i, raw[k], x[0]);
            store(i, x[0], 1.f);
        }
        for (int i = behind; i < n_rows; i += rstep) {
            V v[2];
            load(i, v);
            values(i, v, x[0]);
            store(i, x[0], 1.f);
        }
        return;
    }
    // ---- e4m3: the page's scale from the largest finite value ----------------
    float* scale = (is_v ? a.v_scale : a.k_scale) + (int64_t)page * a.n_kv_head + h;
    const float old = r0 > 0 ? *scale : 0.f;                              // a page's first rows start it anew
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        const int i = r + k * rstep;
        if (i >= n_rows) break;
        values(i, raw[k], x[k]);
        amax = widen(amax, x[k]);
    }
    for (int i = behind; i < n_rows; i += rstep) {
        V v[2];
        float y[8];
        load(i, v);
        values(i, v, y);
        amax = widen(amax, y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    if (lane == 0) red[warp] = amax;
    __syncthreads();
    float m = red[0];
    for (int w = 1; w < warps; ++w) m = fmaxf(m, red[w]);
    const float s = fmaxf(pow2_scale(m), old), inv = 1.f / s;
    if (tid == 0) *scale = s;
    if (r0 > 0 && s > old)                                    // the page's earlier rows at the grown scale
        restore_rows(reinterpret_cast<unsigned char*>(is_v ? a.v : a.k) + p_base, r0, ITEMS, p_row, old / s);
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        const int i = r + k * rstep;
        if (i >= n_rows) break;
        store(i, x[k], inv);
    }
    for (int i = behind; i < n_rows; i += rstep) {
        V v[2];
        float y[8];
        load(i, v);
        values(i, v, y);
        store(i, y, inv);
    }
}

// Prompts, n_dims a multiple of 8. A thread has place c of KR rows and takes the
// block's heads through them, HC heads' loads at a time; the angles are computed
// while the first of these are on their way. e4m3: KR = 4 rows, so a page has at
// most 1024 items (64 rows at hd 128). Measured on 5000 tokens of 8 heads of hd
// 128 in 64-row pages, f16 rows: 15.7 us with 256 threads of 4 rows, two heads at
// a time; 17.7 with 512 threads of 2 rows and 4 heads, 22 with 1024 of one row.
template <typename T, bool E4>
struct Prompt {
    static constexpr int THREADS = 256, KR = E4 ? 4 : 1;
    static constexpr int HC = (E4 ? 2 : 8) / (sizeof(T) == 4 ? 2 : 1);
};
template <typename T, int HD, bool E4>
__global__ void __launch_bounds__((Prompt<T, E4>::THREADS), (E4 ? 2 : 3))
kv_append_prompt_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RopeTable tb, int shift, int heads) {
    constexpr int ITEMS = HD / 8, NTH = Prompt<T, E4>::THREADS, KR = Prompt<T, E4>::KR, HC = Prompt<T, E4>::HC;
    using V = typename Raw<T>::V;
    __shared__ float red[2][HC][NTH / 32];
    const bool is_v = blockIdx.x & 1;
    Angles angles;
    if (!is_v) angles.get(tb, threadIdx.x % ITEMS);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Piece pc = find_piece(a, shift, (int)(blockIdx.x >> 1));
    report_bad(a);
    if (!pc.found) return;                                               // fewer pieces than blocks
    const int pi = pc.row0 >> a.page_shift;                              // page of the sequence
    const int page = a.table[pc.b * a.table_stride + pi];
    const int r0 = pc.row0 - (pi << a.page_shift), n_rows = pc.row1 - pc.row0;
    const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, a.n_kv_head);
    const int64_t s_tok = is_v ? a.v_stride : a.k_stride, p_row = is_v ? a.v_row : a.k_row, p_head = is_v ? a.v_head : a.k_head;
    const T* src = reinterpret_cast<const T*>(is_v ? a.v_new : a.k_new) + pc.tok * s_tok;
    // (places as in the other kernel)
    const int c = tid % ITEMS, r = tid / ITEMS;
    constexpr int RSTEP = NTH / ITEMS;
    const bool rot = !is_v && c * 4 < tb.half;
    const int d0 = rot ? c * 4 : c * 8, d1 = rot ? c * 4 + tb.half : c * 8 + 4;
    int pos[KR];
#pragma unroll
    for (int k = 0; k < KR; ++k) pos[k] = rot && r + k * RSTEP < n_rows ? a.pos[pc.tok + r + k * RSTEP] : 0;
    V raw[HC][KR][2];
    auto load = [&](int h) {
#pragma unroll
        for (int j = 0; j < HC; ++j)
#pragma unroll
            for (int k = 0; k < KR; ++k)
                if (h + j < h1 && r + k * RSTEP < n_rows) {
                    const T* row = src + (r + k * RSTEP) * s_tok + (h + j) * HD;
                    raw[j][k][0] = *reinterpret_cast<const V*>(row + d0);
                    raw[j][k][1] = *reinterpret_cast<const V*>(row + d1);
                }
    };
    load(h0);
    const bool bad_page = page < 0 || page >= a.n_pages;
    if (bad_page && tid == 0 && a.status) atomicOr(a.status, kStatusInput);
    if (bad_page) return;
    float2 cs[KR][4];
    if (rot)
#pragma unroll
        for (int k = 0; k < KR; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) cs[k][u] = angles.at(pos[k], c, u, tb);
    auto values = [&](int j, int k, float* y) {
        const float4 p = Raw<T>::floats(raw[j][k][0]), q = Raw<T>::floats(raw[j][k][1]);
        y[0] = p.x; y[1] = p.y; y[2] = p.z; y[3] = p.w;
        y[4] = q.x; y[5] = q.y; y[6] = q.z; y[7] = q.w;
        if (rot)
#pragma unroll
            for (int u = 0; u < 4; ++u) rotate(y[u], y[4 + u], cs[k][u]);
    };
    const int64_t p_base = page * (is_v ? a.v_page : a.k_page);
    for (int h = h0; h < h1; h += HC) {
        if (h > h0) load(h);
        if (!E4) {
            __half* dst = reinterpret_cast<__half*>(is_v ? a.v : a.k) + p_base + (r0 + r) * p_row;
#pragma unroll
            for (int j = 0; j < HC; ++j)
                if (h + j < h1 && r < n_rows) {
                    float y[8];
                    values(j, 0, y);
                    __half* at = dst + (h + j) * p_head;
                    *reinterpret_cast<uint2*>(at + d0) = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
                    *reinterpret_cast<uint2*>(at + d1) = make_uint2(pack_half2(y[4], y[5]), pack_half2(y[6], y[7]));
                }
            continue;
        }
        const int par = (h - h0) / HC & 1;                               // two sets of maxima: one barrier for each HC heads
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < KR; ++k)
                if (h + j < h1 && r + k * RSTEP < n_rows) {
                    float y[8];
                    values(j, k, y);
                    m = widen(m, y);
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            if (lane == 0) red[par][j][warp] = m;
        }
        float old[HC];
        float* scale = (is_v ? a.v_scale : a.k_scale) + (int64_t)page * a.n_kv_head + h;
#pragma unroll
        for (int j = 0; j < HC; ++j) old[j] = r0 > 0 && h + j < h1 ? scale[j] : 0.f;   // a page's first rows start it anew
        __syncthreads();
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            if (h + j >= h1) break;
            float m = red[par][j][lane & (NTH / 32 - 1)];
#pragma unroll
            for (int o = NTH / 64; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            const float s = fmaxf(pow2_scale(m), old[j]), inv = 1.f / s;
            unsigned char* dst = reinterpret_cast<unsigned char*>(is_v ? a.v : a.k) + p_base + (h + j) * p_head;
            if (tid == 0) scale[j] = s;
            if (r0 > 0 && s > old[j]) restore_rows(dst, r0, ITEMS, p_row, old[j] / s);   // the page's earlier rows
#pragma unroll
            for (int k = 0; k < KR; ++k)
                if (r + k * RSTEP < n_rows) {
                    float y[8];
                    values(j, k, y);
                    unsigned char* at = dst + (r0 + r + k * RSTEP) * p_row;
                    *reinterpret_cast<uint32_t*>(at + d0) = to_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                    *reinterpret_cast<uint32_t*>(at + d1) = to_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
                }
        }
    }
}

// Programmatic launch: set-up overlaps the kernel before it on the stream.
template <typename K, typename... A>
static cudaError_t launch(K kernel, int64_t x, int y, int threads, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)x, (unsigned)y);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// At most this many pieces of 2^shift rows: one a token, and for each sequence
// its whole ones and two that its rows fill in part.
static int64_t most_pieces(const AppendArgs& a, int shift) {
    const int64_t n = 2 * (int64_t)a.n_seq + (a.n_tok >> shift);
    return a.n_tok < n ? a.n_tok : n;
}
template <typename T, int HD, bool E4>
static cudaError_t launch_append(const AppendArgs& a, const RopeTable& tb, cudaStream_t st) {
    // decode: few rows a piece, small blocks
    if (a.n_tok <= 2 * a.n_seq)
        return launch(kv_append_paged_kernel<T, HD, E4, 1>, 2 * most_pieces(a, a.page_shift), a.n_kv_head, 64, st, a, tb);
    using P = Prompt<T, E4>;
    constexpr int kRows = P::THREADS * P::KR / (HD / 8);                 // rows of a prompt block
    int shift = a.page_shift;
    if (!E4)
        while ((1 << shift) > kRows) --shift;                            // an f16 piece may be a part of a page
    if ((1 << shift) > kRows || (tb.n_dims & 7))
        return launch(kv_append_paged_kernel<T, HD, E4, 4>, 2 * most_pieces(a, a.page_shift), a.n_kv_head, 256, st, a, tb);
    // all heads to a block, or as few as leave kBlocks blocks
    constexpr int64_t kBlocks = E4 ? 456 : 608;
    const int64_t n = 2 * most_pieces(a, shift);
    int64_t heads = n * a.n_kv_head / kBlocks;
    heads = heads < P::HC ? P::HC : heads;
    const int groups = (int)((a.n_kv_head + heads - 1) / heads);
    heads = (a.n_kv_head + groups - 1) / groups;
    return launch(kv_append_prompt_kernel<T, HD, E4>, n, groups, P::THREADS, st, a, tb, shift, (int)heads);
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

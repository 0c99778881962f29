// fr_paged_qkv.cuh -- the rows of a step's projection in one launch: query heads
// normed, rotated, scaled and rounded to f16 rows; key heads normed, rotated and
// written with the values into the pages of their sequences.
//
//   n(x) = w x / sqrt(mean(x^2) + eps)  for each head (or x, without weights)
//   Q16 = q_scale * R(pos) n(q),  K = R(pos) n(k),  V = v
//
// Bound by the bytes of the rows read and written, a decode step by latency. The
// norm is taken in the pass that rotates: the 8 to 32 threads that hold a row
// (8 elements each) join their sums of squares by shuffles, so a row is read
// once, stays in registers, and is written once. Blocks of two kinds share the
// launch: the first ones take pieces of pages as the append does
// (fr_paged_rows.cuh), the others tiles of tokens, one head after another of the
// queries, whose angles a thread keeps in registers.
#pragma once

#include "fr_paged_rows.cuh"

namespace fr {
namespace paged {

struct QkvArgs {
    AppendArgs kv;
    const void* q;
    int64_t q_stride;
    __half* q16;
    Norm q_norm, k_norm;
    int n_head;
    int kv_blocks;                        // blocks that take pieces
    int kv_heads, kv_groups, kv_shift;    // heads of such a block, groups of heads, rows of its piece
    int q_heads, q_groups;                // query heads of a block, and groups
};

// Query heads h0 .. h1 - 1 of the block's tile of tokens, HC heads' loads at a time.
template <typename T, int HD, int HC>
__device__ __forceinline__ void query_rows(const QkvArgs& g, const RopeTable& tb, int tile, int h0) {
    constexpr int ITEMS = HD / 8;
    using V = typename Raw<T>::V;
    const Norm& nm = g.q_norm;
    const int c = threadIdx.x % ITEMS, t = tile * (int)(blockDim.x / ITEMS) + threadIdx.x / ITEMS;
    Angles angles;
    angles.get(tb, c);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (t >= g.kv.n_tok) return;
    const int h1 = min(h0 + g.q_heads, g.n_head);
    // (places as in append_piece)
    const bool together = nm.interleaved, vec = together || (tb.n_dims & 7) == 0, rot = c * 4 < tb.half;
    const int d0 = rot && !together ? c * 4 : c * 8, d1 = rot && !together ? c * 4 + tb.half : c * 8 + 4;
    const T* src = reinterpret_cast<const T*>(g.q) + t * g.q_stride;
    const int n_real = g.kv.tok_start[g.kv.n_seq], pos = g.kv.pos[t];
    V raw[HC][2];
    auto load = [&](int h) {
#pragma unroll
        for (int j = 0; j < HC; ++j)
            if (h + j < h1 && vec) {
                raw[j][0] = *reinterpret_cast<const V*>(src + (int64_t)(h + j) * HD + d0);
                raw[j][1] = *reinterpret_cast<const V*>(src + (int64_t)(h + j) * HD + d1);
            }
    };
    if (t >= n_real) return;                          // behind the last sequence
    load(h0);
    int p[4], q[4];                                   // dims of the slots, where they are no vectors
    float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0;
    if (!vec) {
#pragma unroll
        for (int u = 0; u < 4; ++u) rope_slot_dims(c * 4 + u, tb, p[u], q[u]);
    }
    if (nm.w) {
        if (vec) {
            w0 = *reinterpret_cast<const float4*>(nm.w + d0);
            w1 = *reinterpret_cast<const float4*>(nm.w + d1);
        } else {
            w0 = make_float4(nm.w[p[0]], nm.w[p[1]], nm.w[p[2]], nm.w[p[3]]);
            w1 = make_float4(nm.w[q[0]], nm.w[q[1]], nm.w[q[2]], nm.w[q[3]]);
        }
    }
    float2 cs[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) cs[u] = c * 4 + u < tb.half ? angles.at(pos, c, u, tb) : make_float2(1.f, 0.f);
    __half* dst = g.q16 + (int64_t)t * g.n_head * HD;
    for (int h = h0; h < h1; h += HC) {
        if (h > h0) load(h);
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            if (h + j >= h1) break;
            float y[8];
            if (vec) {
                const float4 a = Raw<T>::floats(raw[j][0]), b = Raw<T>::floats(raw[j][1]);
                y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w;
                y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    y[u] = Raw<T>::one(src + (int64_t)(h + j) * HD + p[u]);
                    y[4 + u] = Raw<T>::one(src + (int64_t)(h + j) * HD + q[u]);
                }
            }
            if (nm.w) {
                bool small;
                const float inv = row_rms<ITEMS>(y, nm.eps, small);
                scale_row(y, inv, small, w0, w1);
            }
            auto turn = [&](float& lo, float& hi, int u) {
                const float x0 = lo, x1 = hi;
                if (c * 4 + u < tb.half) {
                    lo = rope_lo(x0, x1, cs[u].x, cs[u].y, tb.q_scale);
                    hi = rope_hi(x0, x1, cs[u].x, cs[u].y, tb.q_scale);
                } else {
                    lo = __fmul_rn(x0, tb.q_scale);
                    hi = __fmul_rn(x1, tb.q_scale);
                }
            };
            if (together) {
#pragma unroll
                for (int u = 0; u < 4; ++u) turn(y[2 * u], y[2 * u + 1], u);
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) turn(y[u], y[4 + u], u);
            }
            __half* at = dst + (int64_t)(h + j) * HD;
            if (vec) {
                *reinterpret_cast<uint2*>(at + d0) = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
                *reinterpret_cast<uint2*>(at + d1) = make_uint2(pack_half2(y[4], y[5]), pack_half2(y[6], y[7]));
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    at[p[u]] = __float2half_rn(y[u]);
                    at[q[u]] = __float2half_rn(y[4 + u]);
                }
            }
        }
    }
}

// Decode steps, and the shapes that the prompt form leaves out (KEEP as in append_piece).
template <typename T, int HD, bool E4, int KEEP>
__global__ void __launch_bounds__(KEEP == 1 ? 64 : 256)
qkv_post_paged_kernel(const __grid_constant__ QkvArgs g, const __grid_constant__ RopeTable tb) {
    const int b = blockIdx.x;
    if (b < g.kv_blocks) {
        const int i = b >> 1, nth = i / g.kv.n_kv_head;
        append_piece<T, HD, E4, KEEP, true>(g.kv, tb, g.k_norm, b & 1, nth, i - nth * g.kv.n_kv_head);
    } else {
        const int i = b - g.kv_blocks, tile = i / g.q_groups;
        query_rows<T, HD, KEEP == 1 ? 4 : sizeof(T) == 4 ? 4 : 8>(g, tb, tile, (i - tile * g.q_groups) * g.q_heads);
    }
}
template <typename T, int HD, bool E4>
__global__ void __launch_bounds__((Prompt<T, E4>::THREADS), (E4 ? 2 : 3))
qkv_post_prompt_kernel(const __grid_constant__ QkvArgs g, const __grid_constant__ RopeTable tb) {
    const int b = blockIdx.x;
    if (b < g.kv_blocks) {
        const int i = b >> 1, nth = i / g.kv_groups;
        append_prompt<T, HD, E4, true>(g.kv, tb, g.k_norm, g.kv_shift, g.kv_heads, b & 1, nth, (i - nth * g.kv_groups) * g.kv_heads);
    } else {
        const int i = b - g.kv_blocks, tile = i / g.q_groups;
        query_rows<T, HD, sizeof(T) == 4 ? 4 : 8>(g, tb, tile, (i - tile * g.q_groups) * g.q_heads);
    }
}

template <typename T, int HD, bool E4>
static fr_status launch_qkv(QkvArgs g, const RopeTable& tb, cudaStream_t st) {
    const AppendArgs& a = g.kv;
    const bool decode = a.n_tok <= 2 * a.n_seq;
    const PromptPlan p = plan_prompt<T, HD, E4>(a, tb.n_dims);
    const bool prompt = !decode && p.heads;
    const int threads = decode ? 64 : 256;
    int64_t kv_blocks;
    if (prompt) {
        g.kv_shift = p.shift;
        g.kv_heads = p.heads;
        g.kv_groups = p.groups;
        kv_blocks = 2 * most_pieces(a, p.shift) * p.groups;
    } else {
        kv_blocks = 2 * most_pieces(a, a.page_shift) * a.n_kv_head;
    }
    // query heads of a block: as many as leave enough blocks
    const int per = threads / (HD / 8);
    const int64_t tiles = (a.n_tok + per - 1) / per;
    int64_t heads = tiles * g.n_head / 608;
    const int least = decode ? 1 : 4;
    heads = heads < least ? least : heads > g.n_head ? g.n_head : heads;
    g.q_groups = (int)((g.n_head + heads - 1) / heads);
    g.q_heads = (g.n_head + g.q_groups - 1) / g.q_groups;
    const int64_t blocks = kv_blocks + tiles * g.q_groups;
    if (blocks > 0x7fffffff) return FR_ERR_UNSUPPORTED;
    g.kv_blocks = (int)kv_blocks;
    const cudaError_t e = prompt   ? launch(qkv_post_prompt_kernel<T, HD, E4>, blocks, 1, Prompt<T, E4>::THREADS, st, g, tb)
                          : decode ? launch(qkv_post_paged_kernel<T, HD, E4, 1>, blocks, 1, threads, st, g, tb)
                                   : launch(qkv_post_paged_kernel<T, HD, E4, 4>, blocks, 1, threads, st, g, tb);
    return e == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}
template <typename T, int HD>
static fr_status launch_qkv(const QkvArgs& g, const RopeTable& tb, bool e4, cudaStream_t st) {
    return e4 ? launch_qkv<T, HD, true>(g, tb, st) : launch_qkv<T, HD, false>(g, tb, st);
}
template <typename T>
static fr_status launch_qkv(const QkvArgs& g, const RopeTable& tb, int hd, bool e4, cudaStream_t st) {
    return hd == 64 ? launch_qkv<T, 64>(g, tb, e4, st) : hd == 128 ? launch_qkv<T, 128>(g, tb, e4, st)
                                                                   : launch_qkv<T, 256>(g, tb, e4, st);
}
fr_status launch_qkv_f32(const QkvArgs& g, const RopeTable& tb, int hd, bool e4, cudaStream_t st);
fr_status launch_qkv_f16(const QkvArgs& g, const RopeTable& tb, int hd, bool e4, cudaStream_t st);
fr_status launch_qkv_bf16(const QkvArgs& g, const RopeTable& tb, int hd, bool e4, cudaStream_t st);

}  // namespace paged
}  // namespace fr

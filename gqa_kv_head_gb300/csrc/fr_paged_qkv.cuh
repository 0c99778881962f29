// fr_paged_qkv.cuh -- the rows of a step's projection in one launch: query heads
// normed, rotated, scaled and rounded to f16 rows; key heads normed, rotated and
// written with the values into the pages of their sequences.
//
//   n(x) = w x / sqrt(mean(x^2) + eps)  for each head (or x, without weights)
//   Q16 = q_scale * R(pos) n(q),  K = R(pos) n(k),  V = v
//
// Bound by the bytes of the rows read and written, a decode step by latency. The
// norm is taken in the pass that rotates: the 4 to 32 threads that hold a row
// (8 or 16 elements each) join their sums of squares by shuffles, so a row is read
// once, stays in registers, and is written once. The angles of a token are the
// same for all its heads, and at about 100 instructions an angle they are what is
// left to save: a thread keeps the cosines and sines of its place in registers
// and takes head after head through them.
//   * Prompts into f16 pages (qkv_post_tokens_kernel): blocks of 64 threads take a
//     tile of tokens and a part of the list of all heads, queries, keys and values;
//     the pages of the tokens are looked up by their warps. A thread asks for its part
//     of the next four heads by cp.async, into places of its own, so that the bytes on
//     their way need no registers and nobody waits for anybody. 6005 bf16 tokens of 32
//     query and 8 KV heads of 128 (148 MB): 30.1 us, 4.9 TB/s. On the way there: heads
//     through registers, keys and values by pieces beside them 36.7; one list through
//     registers 37 to 46 (too little on its way); the ring in blocks of 256 threads 33
//     to 34, of 64 threads 31.8, and with registers for ten of them on an SM 29.7 (6
//     places; 4 places 30.8, 10 places 35.6). Reading and writing the query rows alone
//     takes 17.4, with norms and rotation 24, of which the angles are 4.2.
//   * e4m3 pages (qkv_post_prompt_kernel): a page has its scale from all its rows, so
//     keys and values go by pieces of pages as in the append (fr_paged_rows.cuh), with
//     as few rows of a thread, and as many heads at a time, as the page allows; query
//     heads through the ring by tiles of tokens, a warp to a token, whose lanes share
//     the angles out and hand them around. The two kinds of blocks take turns.
//     4980 f32 tokens of 15 query and 5 KV heads of 64, 32-row pages (45 MB): 18.0 us
//     (four rows of a thread, kinds one after the other: 24); queries alone 11.7, keys
//     and values alone 12 to 13: instructions and the latency of a piece bound it.
//     The case of 6005 bf16 tokens above in 64-row e4m3 pages 37.4 (each lane with all
//     its angles 39.8). 8 or 16 rows of a page to each of 256 threads are blocks of 512
//     instead, 16 with the angles in shared memory: 128-row pages 48.0 (by pieces of a
//     head 68.1), and f32, hd 256, 16 query and 2 KV heads 43.7 (50.6).
//   * Decode steps: the same two kinds of blocks, of 64 threads, one head each.
//   * Prompts with n_dims no multiple of 8: the same, of 256 threads. The dims of a thread's pairs
//     are no vectors there (interleaved: they are, but a pair that turns may be beside one that does
//     not), so that elements come and go one by one, and angles are worked out for each head again: the
//     bf16 prompts above with n_dims 100 90 us (interleaved 51; n_dims 96 31 and 38), f32 to e4m3 with
//     28 37 (25). Heads rotate multiples of 8 dims as a rule, and the vector forms keep their registers.
#pragma once

#include <type_traits>

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
    int kv_heads, kv_groups;              // heads of such a block, groups of heads
    int heads, groups;                    // of the others: heads of a block, groups of heads
    int wide;                             // 16 elements of a row to a thread
};

// E / 2 elements of a row as they come, and as floats.
template <typename T, int N> struct alignas(16) Part {
    typename Raw<T>::V v[N / 4];
    __device__ __forceinline__ void load(const T* p) {
        constexpr int W = N / 4 * (int)sizeof(typename Raw<T>::V) / 16;      // 16-byte words
        if (W == 0) {
            v[0] = *reinterpret_cast<const typename Raw<T>::V*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(p)[i];
        }
    }
    // from a thread's place in the ring: 16-byte words NT places apart
    template <int NT>
    __device__ __forceinline__ void shared(const unsigned char* p) {
        constexpr int W = N / 4 * (int)sizeof(typename Raw<T>::V) / 16;
        if (W == 0) {
            v[0] = *reinterpret_cast<const typename Raw<T>::V*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(v)[i] = *reinterpret_cast<const uint4*>(p + i * 16 * NT);
        }
    }
    __device__ __forceinline__ void floats(float* y) const {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) *reinterpret_cast<float4*>(y + 4 * i) = Raw<T>::floats(v[i]);
    }
};
template <int N>
__device__ __forceinline__ void store_halves(__half* at, const float* y) {
    uint32_t h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) h[i] = pack_half2(y[2 * i], y[2 * i + 1]);
    if (N == 8) *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2 % (N / 2)], h[3 % (N / 2)]);
    else *reinterpret_cast<uint2*>(at) = make_uint2(h[0], h[1]);
}

constexpr int kTokenThreads = 64, kTokenBlocks = 10;      // of a block of tokens; such blocks on an SM
constexpr int64_t kBlocks = 608;                          // blocks that a launch is to have, where heads can be cut

// Some heads of a token: where element 0 of head 0 comes from, and results go to dst[h * dst_head + d].
struct HeadRows {
    const void* src;
    __half* dst;
    int64_t dst_head;
    const float* w;                       // null: no norm
    float eps, scale;
    int half;                             // pairs that turn
    bool together;                        // interleaved pairs
};
// A thread's E elements of a head, in two halves of E / 2 pairs' elements: at d0 and d1
// (interleaved, or not turned: E neighbours), as in append_piece.
template <int E>
struct Dims {
    int d0, d1;
    __device__ __forceinline__ Dims(int c, int half, bool together) {
        constexpr int P = E / 2;
        const bool halves = c * P < half && !together;
        d0 = halves ? c * P : c * E;
        d1 = halves ? c * P + half : c * E + P;
    }
};
// What turns and scales a thread's elements. Normed rows are a R(w x) with a = scale /
// rms: the weights go into the rotation's factors, four of a pair, which all heads
// share. Without a norm the products are those of fr_qkv_post, in its order.
template <int HD, int E, bool NORMED>
struct Turner {
    static constexpr int ITEMS = HD / E, P = E / 2;
    float4 f[NORMED ? P : 1];             // of a pair: w0 cos, w1 sin, w0 sin, w1 cos
    float2 cs[NORMED ? 1 : P];
    __device__ __forceinline__ Turner(const HeadRows& r, int c, const Dims<E>& d, const float2* angles) {
        const bool every = c * P + P <= r.half;
        if (NORMED) {
            alignas(16) float w[E];
#pragma unroll
            for (int i = 0; i < P; i += 4) {
                *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(r.w + d.d0 + i);
                *reinterpret_cast<float4*>(w + P + i) = *reinterpret_cast<const float4*>(r.w + d.d1 + i);
            }
#pragma unroll
            for (int u = 0; u < P; ++u) {
                const float w0 = r.together ? w[2 * u] : w[u], w1 = r.together ? w[2 * u + 1] : w[P + u];
                const float2 a = angles[u];
                f[u] = make_float4(w0 * a.x, w1 * a.y, w0 * a.y, w1 * a.x);
                if (!every && c * P + u >= r.half) f[u] = make_float4(w0, 0.f, 0.f, w1);
            }
        } else {
#pragma unroll
            for (int u = 0; u < P; ++u) cs[u] = angles[u];
        }
    }
    __device__ __forceinline__ void operator()(const HeadRows& r, int c, float* y) const {
        float a = r.scale;
        if (NORMED) {
            int scaled;
            const float inv = row_rms<ITEMS, E>(y, r.eps, scaled);
            if (__builtin_expect(scaled != 0, 0)) {
#pragma unroll
                for (int u = 0; u < E; ++u) y[u] *= resize(scaled);
            }
            a *= inv;
        }
        auto turn = [&](float& lo, float& hi, int u) {
            const float x0 = lo, x1 = hi;
            if (NORMED) {
                lo = fmaf(x0, f[u].x, -(x1 * f[u].y)) * a;
                hi = fmaf(x0, f[u].z, x1 * f[u].w) * a;
            } else {
                lo = rope_lo(x0, x1, cs[u].x, cs[u].y, a);
                hi = rope_hi(x0, x1, cs[u].x, cs[u].y, a);
            }
        };
        auto pass = [&](float& lo, float& hi, int u) {
            lo = NORMED ? lo * f[u].x * a : __fmul_rn(lo, a);
            hi = NORMED ? hi * f[u].w * a : __fmul_rn(hi, a);
        };
        if (r.together) {
            if (c * P + P <= r.half) {
#pragma unroll
                for (int u = 0; u < P; ++u) turn(y[2 * u], y[2 * u + 1], u);
            } else {
#pragma unroll
                for (int u = 0; u < P; ++u) {
                    if (c * P + u < r.half) turn(y[2 * u], y[2 * u + 1], u);
                    else pass(y[2 * u], y[2 * u + 1], u);
                }
            }
        } else if (c * P < r.half) {      // (all of a thread's pairs turn, or none)
#pragma unroll
            for (int u = 0; u < P; ++u) turn(y[u], y[P + u], u);
        } else {
#pragma unroll
            for (int u = 0; u < P; ++u) pass(y[u], y[P + u], u);
        }
    }
};
// Decode: heads h0 .. h1 - 1 through registers, the next two on their way.
template <typename T, int HD, int E, bool NORMED>
__device__ __forceinline__ void head_rows(const HeadRows& r, int h0, int h1, const float2* angles) {
    constexpr int P = E / 2, HC = 2;
    const int c = threadIdx.x % (HD / E);
    const Dims<E> d(c, r.half, r.together);
    const T* src = reinterpret_cast<const T*>(r.src);
    Part<T, P> raw[HC][2];
    auto load = [&](int h) {
#pragma unroll
        for (int j = 0; j < HC; ++j)
            if (h + j < h1) {
                raw[j][0].load(src + (int64_t)(h + j) * HD + d.d0);
                raw[j][1].load(src + (int64_t)(h + j) * HD + d.d1);
            }
    };
    load(h0);
    const Turner<HD, E, NORMED> turner(r, c, d, angles);
    for (int h = h0; h < h1; h += HC) {
        if (h > h0) load(h);
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            if (h + j >= h1) break;
            alignas(16) float y[E];
            raw[j][0].floats(y);
            raw[j][1].floats(y + P);
            turner(r, c, y);
            store_halves<P>(r.dst + (h + j) * r.dst_head + d.d0, y);
            store_halves<P>(r.dst + (h + j) * r.dst_head + d.d1, y + P);
        }
    }
}
// Prompts: a thread's elements of the next STAGES - 1 heads are on their way into
// places of its own in shared memory (no barrier: nobody else looks at them).
constexpr int kStages = 5;
template <typename T, int E, int NT>
__host__ __device__ constexpr int ring_bytes() { return NT * (kStages * E * (int)sizeof(T) + E / 2 * 8); }
template <int BYTES, int NT>
__device__ __forceinline__ void ring_copy(uint32_t dst, const void* src) {
#pragma unroll
    for (int i = 0; i < BYTES; i += 16) {
        if (BYTES >= 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst + i * NT), "l"((const char*)src + i) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(dst), "l"(src) : "memory");
    }
}

// Query heads element by element: pairs of halves with a number of pairs that vectors do not divide.
template <typename T, int HD>
__device__ __noinline__ void query_heads_odd(const QkvArgs* g, const RopeTable* tb, int t, int h0, int h1, const float2* cs) {
    constexpr int ITEMS = HD / 8;
    const Norm nm = g->q_norm;
    const int c = threadIdx.x % ITEMS;
    for (int h = h0; h < h1; ++h) {
        const T* src = reinterpret_cast<const T*>(g->q) + t * g->q_stride + (int64_t)h * HD;
        __half* dst = g->q16 + ((int64_t)t * g->n_head + h) * HD;
        float y[8];
        int p[4], q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            rope_slot_dims(c * 4 + u, *tb, p[u], q[u]);
            y[u] = Raw<T>::one(src + p[u]);
            y[4 + u] = Raw<T>::one(src + q[u]);
        }
        if (nm.w) {
            int scaled;
            const float inv = row_rms<ITEMS>(y, nm.eps, scaled);
            scale_row(y, inv, scaled, make_float4(nm.w[p[0]], nm.w[p[1]], nm.w[p[2]], nm.w[p[3]]),
                      make_float4(nm.w[q[0]], nm.w[q[1]], nm.w[q[2]], nm.w[q[3]]));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool turns = c * 4 + u < tb->half;
            dst[p[u]] = __float2half_rn(turns ? rope_lo(y[u], y[4 + u], cs[u].x, cs[u].y, tb->q_scale) : __fmul_rn(y[u], tb->q_scale));
            dst[q[u]] = __float2half_rn(turns ? rope_hi(y[u], y[4 + u], cs[u].x, cs[u].y, tb->q_scale) : __fmul_rn(y[4 + u], tb->q_scale));
        }
    }
}

// Sequence and cache row of each of a warp's tokens t (ITEMS lanes have the same one); -1:
// of none that fits. 128 sequences at a time, whose numbers arrive together.
struct Place {
    int b, row;
};
template <int ITEMS>
__device__ __forceinline__ Place find_tokens(const AppendArgs& a, int t, bool wanted) {
    const int lane = threadIdx.x & 31;
    Place p{-1, 0};
    for (int b0 = 0; b0 < a.n_seq && __any_sync(~0u, wanted && p.b < 0); b0 += 128) {
        int t0[4], t1[4], base[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t0[i] = t1[i] = base[i] = 0;
            if (b0 + i * 32 + lane < a.n_seq) {
                const SeqInfo s = seq_info(a.tok_start, a.kv_len, b0 + i * 32 + lane, a.n_tok, a.max_pages, a.page_shift);
                if (!s.bad && s.n_q <= s.n_kv) {
                    t0[i] = s.tok0;
                    t1[i] = s.tok0 + s.n_q;
                    base[i] = s.n_kv - s.n_q - s.tok0;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 32 / ITEMS; ++k) {
                const int token = __shfl_sync(~0u, t, k * ITEMS);
                const unsigned hit = __ballot_sync(~0u, token >= t0[i] && token < t1[i]);
                const int at = hit ? __ffs(hit) - 1 : 0, first = __shfl_sync(~0u, base[i], at);
                if (hit && lane / ITEMS == k && p.b < 0) p = Place{b0 + i * 32 + at, first + token};
            }
    }
    return p;
}

// A tile of tokens and heads h0 .. of the list: queries, and where PAGES (f16) keys and
// values behind them. NT: threads of a ring in shared memory (0: none).
// SHARE: the lanes of a warp hold one token, 32 / ITEMS heads at a time, work out its
// angles together and hand them around (PAGES: not so).
template <typename T, int HD, int E, bool PAGES, int NT, bool SHARE = false>
__device__ __forceinline__ void token_rows(const QkvArgs& g, const RopeTable& tb, int tile, int h0) {
    constexpr int ITEMS = HD / E, P = E / 2;
    constexpr bool RING = NT > 0;
    constexpr int EACH = SHARE ? 32 / ITEMS : 1, LANES = ITEMS * EACH;      // heads at a time, lanes of a token
    static_assert(!SHARE || (RING && !PAGES && P % EACH == 0), "");
    const AppendArgs& a = g.kv;
    const int c = threadIdx.x % ITEMS, nth = threadIdx.x % LANES / ITEMS;
    const int t_ = tile * (int)(blockDim.x / LANES) + threadIdx.x / LANES, t = min(t_, a.n_tok - 1);
    Angles angles[P / 4];
    uint64_t turns[P / EACH];
    if (SHARE) {
#pragma unroll
        for (int i = 0; i < P / EACH; ++i) turns[i] = tb.turns[min(c * P + nth + i * EACH, kMaxPairs - 1)];
    } else {
#pragma unroll
        for (int i = 0; i < P / 4; ++i) angles[i].get(tb, c * (P / 4) + i);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int n_real = a.tok_start[a.n_seq], pos = a.pos[t];
    const bool here = t_ < a.n_tok && t_ < n_real;        // (else behind the last sequence)
    const int h1 = min(h0 + g.heads, g.n_head + (PAGES ? 2 * a.n_kv_head : 0));
    // kind 0: queries, 1: keys, 2: values; their heads are numbered from `behind` in the list
    auto source = [&](int kind) {
        return kind == 0 ? reinterpret_cast<const T*>(g.q) + t * g.q_stride
               : kind == 1 ? reinterpret_cast<const T*>(a.k_new) + t * a.k_stride : reinterpret_cast<const T*>(a.v_new) + t * a.v_stride;
    };
    auto behind = [&](int kind) { return kind == 0 ? 0 : g.n_head + (kind - 1) * a.n_kv_head; };
    HeadRows r{source(0), g.q16 + (int64_t)t * g.n_head * HD, HD, g.q_norm.w, g.q_norm.eps, tb.q_scale, tb.half,
               g.q_norm.interleaved != 0};
    extern __shared__ __align__(16) unsigned char ring[];
    // (stage, half, 16-byte word, thread)
    constexpr int PART = P * (int)sizeof(T), STAGE = 2 * PART * NT;
    unsigned char* const mine = ring + threadIdx.x * (PART < 16 ? PART : 16);
    const uint32_t ring_u = RING ? smem_u32(mine) : 0u;
    int ask_left = here ? (h1 - h0 - nth + EACH - 1) / EACH : 0, ask_kind = -1, ask_kind_left = 0, ask_d = 0;   // heads to ask for, in all and of their kind
    const T* ask_at = nullptr;
    uint32_t ask_to = 0;
    auto ask = [&]() {
        if (ask_left > 0) {
            if (ask_kind_left == 0 && SHARE) {
                const Dims<E> d(c, r.half, r.together);
                ask_at = source(0) + (int64_t)(h0 + nth) * HD + d.d0;
                ask_d = d.d1 - d.d0;
                ask_kind_left = ask_left;
            }
            if (ask_kind_left == 0) {
                int head;                                 // the next kind that has some of the heads
                do {
                    ++ask_kind;
                    head = max(h1 - ask_left - behind(ask_kind), 0);
                    ask_kind_left = min(h1 - behind(ask_kind), ask_kind == 0 ? g.n_head : a.n_kv_head) - head;
                } while (ask_kind_left <= 0);
                const Dims<E> d(c, ask_kind == 2 ? 0 : r.half, r.together);
                ask_at = source(ask_kind) + (int64_t)head * HD + d.d0;
                ask_d = d.d1 - d.d0;
            }
            ring_copy<PART, NT>(ring_u + ask_to, ask_at);
            ring_copy<PART, NT>(ring_u + ask_to + PART * NT, ask_at + ask_d);
            ask_at += EACH * HD;
            ask_to = ask_to == (kStages - 1) * STAGE ? 0 : ask_to + STAGE;
            --ask_left;
            --ask_kind_left;
        }
        cp_async_commit();
    };
    if (RING)
        for (int i = 0; i < kStages - 1; ++i) ask();
    int page = -1, row = 0;
    if (PAGES) {
        report_bad(a);
        if (h1 > g.n_head) {
            const Place p = find_tokens<ITEMS>(a, t, here);
            if (p.b >= 0) {
                page = a.table[p.b * a.table_stride + (p.row >> a.page_shift)];
                row = p.row & ((1 << a.page_shift) - 1);
                if (page < 0 || page >= a.n_pages) {
                    if (a.status) atomicOr(a.status, kStatusInput);
                    page = -1;
                }
            }
        }
    }
    if (!here) return;
    float2 cs[RING ? 1 : P];
    float2* angle = RING ? reinterpret_cast<float2*>(ring + kStages * STAGE) + threadIdx.x : cs;      // a place of its own too
    if (SHARE) {
#pragma unroll
        for (int i = 0; i < P / EACH; ++i) {
            const int pair = c * P + nth + i * EACH;
            float2 x = make_float2(1.f, 0.f);
            if (pair < tb.half) x = tb.mode == FR_ROPE_GGML_F32 ? rope_cs_f32(pos, pair, &tb) : rope_cs_fixed(pos, turns[i], tb.mscale);
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                angle[(i * EACH + k) * NT] = make_float2(__shfl_sync(~0u, x.x, k * ITEMS + c), __shfl_sync(~0u, x.y, k * ITEMS + c));
        }
    } else
#pragma unroll
    for (int u = 0; u < P; ++u)
        angle[u * (RING ? NT : 1)] = c * P + u < tb.half ? angles[u / 4].at(pos, c * (P / 4) + u / 4, u % 4, tb) : make_float2(1.f, 0.f);
    if (!RING) {
        if (!g.q_norm.interleaved && (tb.n_dims & 7)) query_heads_odd<T, HD>(&g, &tb, t, h0, h1, cs);
        else if (r.w) head_rows<T, HD, E, true>(r, h0, h1, cs);
        else head_rows<T, HD, E, false>(r, h0, h1, cs);
        return;
    }
    int slot = 0;
    auto through = [&](auto normed, int from, int to) {
        float2 own[P];
#pragma unroll
        for (int u = 0; u < P; ++u) own[u] = angle[u * NT];
        const Dims<E> d(c, r.half, r.together);
        const Turner<HD, E, decltype(normed)::value> turner(r, c, d, own);
        __half* dst = r.dst + (from + nth) * r.dst_head + d.d0;
        const int dd = d.d1 - d.d0;
#pragma unroll 1
        for (int n = to - from - nth; n > 0; n -= EACH) {
            cp_async_wait<kStages - 2>();
            Part<T, P> raw[2];
            raw[0].template shared<NT>(mine + slot);
            raw[1].template shared<NT>(mine + slot + PART * NT);
            slot = slot == (kStages - 1) * STAGE ? 0 : slot + STAGE;
            ask();
            alignas(16) float y[E];
            raw[0].floats(y);
            raw[1].floats(y + P);
            turner(r, c, y);
            store_halves<P>(dst, y);
            store_halves<P>(dst + dd, y + P);
            dst += EACH * r.dst_head;
        }
    };
#pragma unroll 1
    for (int kind = 0;; ++kind) {
        const int from = max(h0 - behind(kind), 0), to = min(h1 - behind(kind), kind == 0 ? g.n_head : a.n_kv_head);
        if (from < to) {
            if (r.w) through(std::true_type(), from, to);
            else through(std::false_type(), from, to);
        }
        if (!PAGES || kind == 2 || page < 0) break;
        if (kind == 0) {
            r.dst = reinterpret_cast<__half*>(a.k) + page * a.k_page + row * a.k_row;
            r.dst_head = a.k_head;
            r.w = g.k_norm.w;
            r.eps = g.k_norm.eps;
            r.scale = 1.f;
        } else {
            r.dst = reinterpret_cast<__half*>(a.v) + page * a.v_page + row * a.v_row;
            r.dst_head = a.v_head;
            r.w = nullptr;
            r.half = 0;
            r.together = false;
        }
    }
    cp_async_wait<0>();                                   // (rows of a token without a page are not looked at)
}

// Decode steps, and the shapes that the prompt forms leave out (KEEP as in append_piece).
template <typename T, int HD, bool E4, int KEEP>
__global__ void __launch_bounds__(KEEP == 1 ? 64 : 256)
qkv_post_paged_kernel(const __grid_constant__ QkvArgs g, const __grid_constant__ RopeTable tb) {
    const int b = blockIdx.x;
    if (b < g.kv_blocks) {
        const int i = b >> 1, nth = i / g.kv.n_kv_head;
        append_piece<T, HD, E4, KEEP, true>(g.kv, tb, g.k_norm, b & 1, nth, i - nth * g.kv.n_kv_head);
    } else {
        const int i = b - g.kv_blocks, tile = i / g.groups;
        token_rows<T, HD, 8, false, 0>(g, tb, tile, (i - tile * g.groups) * g.heads);
    }
}
// Prompts into f16 pages.
template <typename T, int HD>
__global__ void __launch_bounds__(kTokenThreads, kTokenBlocks)
qkv_post_tokens_kernel(const __grid_constant__ QkvArgs g, const __grid_constant__ RopeTable tb) {
    const int tile = blockIdx.x / g.groups, h0 = (blockIdx.x - tile * g.groups) * g.heads;
    if (sizeof(T) == 2 && g.wide) token_rows<T, HD, 16, true, kTokenThreads>(g, tb, tile, h0);
    else token_rows<T, HD, 8, true, kTokenThreads>(g, tb, tile, h0);
}
// Prompts into e4m3 pages: pieces of a page, KR rows of it to a thread (0: page too large,
// its heads one at a time).
template <typename T, int HD, int KR, int NT>
__global__ void __launch_bounds__(NT, NT > 256 ? 1 : KR == 1 && sizeof(T) == 4 ? 3 : 2)
qkv_post_prompt_kernel(const __grid_constant__ QkvArgs g, const __grid_constant__ RopeTable tb) {
    // the two kinds of blocks take turns while there are both: pieces wait, tiles stream
    const int b = blockIdx.x, both = 2 * min(g.kv_blocks, (int)gridDim.x - g.kv_blocks);
    const bool piece = b < both ? !(b & 1) : g.kv_blocks > both / 2;
    const int nth_block = b < both ? b >> 1 : b - both / 2;
    if (piece) {
        const int i = nth_block >> 1, nth = i / g.kv_groups;
        const int h0 = (i - nth * g.kv_groups) * g.kv_heads;
        if (KR > 0)
            append_prompt<T, HD, true, true, KR ? KR : 1, KR < 8 ? (sizeof(T) == 4 ? 4 : 8) / (KR ? KR : 1) : 1, NT>(
                g.kv, tb, g.k_norm, g.kv.page_shift, g.kv_heads, nth_block & 1, nth, h0);
        else
            append_piece<T, HD, true, 4, true>(g.kv, tb, g.k_norm, nth_block & 1, nth, h0);
    } else {
        const int i = nth_block, tile = i / g.groups, h0 = (i - tile * g.groups) * g.heads;
        if (sizeof(T) == 2 && g.wide) token_rows<T, HD, 16, false, NT, true>(g, tb, tile, h0);
        else token_rows<T, HD, 8, false, NT, true>(g, tb, tile, h0);
    }
}

// A launch with the ring's shared memory (which: the kernel, for its own record of
// the devices whose limit is raised).
template <typename T, int HD, int which, int NT, typename K>
static fr_status launch_ring(K kernel, int64_t blocks, cudaStream_t st, const QkvArgs& g, const RopeTable& tb) {
    static unsigned long long done = 0ull;
    constexpr int ring = ring_bytes<T, sizeof(T) == 2 ? 16 : 8, NT>(), kept = which == 16 ? 8 * 4 * 8 * NT : 0;      // (angles of eight rows)
    constexpr int wide = ring > kept ? ring : kept, narrow = ring_bytes<T, 8, NT>() > kept ? ring_bytes<T, 8, NT>() : kept;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FR_ERR_CUDA;
    if (dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> dev & 1ull)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, wide) != cudaSuccess) return FR_ERR_CUDA;
        if (dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELEASE);
    }
    const cudaError_t e = launch_smem(kernel, blocks, 1, NT, g.wide || sizeof(T) == 4 ? wide : narrow, st, g, tb);
    return e == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}
template <typename T, int HD, bool E4>
static fr_status launch_qkv(QkvArgs g, const RopeTable& tb, cudaStream_t st) {
    const AppendArgs& a = g.kv;
    const bool decode = a.n_tok <= 2 * a.n_seq, together = g.q_norm.interleaved != 0;
    // rows of a page that each of an e4m3 block's 256 threads has
    const int kr = ((HD / 8) << a.page_shift) / 256, rows = kr < 2 ? 1 : kr;
    const bool prompt = !decode && tb.n_dims % 8 == 0;
    const int threads = decode ? 64 : prompt && !E4 ? kTokenThreads : prompt && (rows == 8 || rows == 16) ? 512 : 256;
    // (16 elements to a thread take fewer shuffles and addresses; a decode step would wait for twice the angles)
    g.wide = prompt && sizeof(T) == 2 && (together || tb.n_dims % 16 == 0);
    const int lanes = HD / (g.wide ? 16 : 8), each = prompt && E4 ? 32 / lanes : 1;     // of a token's head; heads at a time
    const int per = threads / (lanes * each);
    const int64_t tiles = (a.n_tok + per - 1) / per;
    // a block has as many heads as leave enough blocks
    auto cut = [](int64_t pieces, int heads, int64_t blocks, int least, int* of_block, int* groups) {
        int64_t n = pieces * heads / blocks;
        n = n < least ? least : n;
        n = n > heads ? heads : n;
        *groups = (int)((heads + n - 1) / n);
        *of_block = (heads + *groups - 1) / *groups;
    };
    const int all = g.n_head + (prompt && !E4 ? 2 * a.n_kv_head : 0);
    cut(tiles, all, kBlocks, decode ? 1 : 4 * each, &g.heads, &g.groups);
    int64_t kv_blocks = 0;
    if (!prompt) {
        kv_blocks = 2 * most_pieces(a, a.page_shift) * a.n_kv_head;
    } else if (E4) {
        const int64_t pieces = 2 * most_pieces(a, a.page_shift);
        const int least = rows == 16 ? 1 : (sizeof(T) == 4 ? 4 : 8) / (rows < 4 ? rows : 4);      // heads at a time
        if (rows <= 16) cut(pieces, a.n_kv_head, kBlocks / 2, least, &g.kv_heads, &g.kv_groups);
        else g.kv_heads = 1, g.kv_groups = a.n_kv_head;
        kv_blocks = pieces * g.kv_groups;
    }
    const int64_t blocks = kv_blocks + tiles * g.groups;
    if (blocks > 0x7fffffff) return FR_ERR_UNSUPPORTED;
    g.kv_blocks = (int)kv_blocks;
    cudaError_t e;
    if (decode) e = launch(qkv_post_paged_kernel<T, HD, E4, 1>, blocks, 1, threads, st, g, tb);
    else if (!prompt) e = launch(qkv_post_paged_kernel<T, HD, E4, 4>, blocks, 1, threads, st, g, tb);
    else if (!E4) return launch_ring<T, HD, 0, kTokenThreads>(qkv_post_tokens_kernel<T, HD>, blocks, st, g, tb);
    else if (rows == 1) return launch_ring<T, HD, 1, 256>(qkv_post_prompt_kernel<T, HD, 1, 256>, blocks, st, g, tb);
    else if (rows == 2) return launch_ring<T, HD, 2, 256>(qkv_post_prompt_kernel<T, HD, 2, 256>, blocks, st, g, tb);
    else if (rows == 4) return launch_ring<T, HD, 4, 256>(qkv_post_prompt_kernel<T, HD, 4, 256>, blocks, st, g, tb);
    else if (rows == 8) return launch_ring<T, HD, 8, 512>(qkv_post_prompt_kernel<T, HD, 4, 512>, blocks, st, g, tb);
    else {                                // (pages of at most 256 rows)
        if constexpr (HD >= 128)
            if (rows == 16) return launch_ring<T, HD, 16, 512>(qkv_post_prompt_kernel<T, HD, 8, 512>, blocks, st, g, tb);
        if constexpr (HD >= 256)
            return launch_ring<T, HD, 32, 256>(qkv_post_prompt_kernel<T, HD, 0, 256>, blocks, st, g, tb);
        return FR_ERR_UNSUPPORTED;
    }
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

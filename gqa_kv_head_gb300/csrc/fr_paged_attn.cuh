// fr_paged_attn.cuh -- attention of a step's query rows over a paged K/V cache
// (f16 pages, or e4m3 pages with a scale for each page and head).
//
// For a sequence's KV head, the G query heads that share it and the sequence's
// n_q new tokens give rows r = i*G + g. With x_rj = scale * <q_r, k_j> in log2
// units, masked keys at -inf,
//   out_r = sum_j 2^(x_rj - m_r) v_j / sum_j 2^(x_rj - m_r)
// in one pass over the keys with a running reference m_r.
//
// Few rows and many keys (many rows: fr_paged_tc.cu): bound by the bytes of K and V. Keys are the MMA's M
// and query rows its N (S^T = K Q^T, O^T = V^T P^T by mma.sync m16n8k16), so a
// K or V element enters one MMA for up to 8 rows, and every warp works alone
// on 16-key tiles: its own ring of TMA-filled slots, its own running state, no
// block barrier until a piece of a sequence ends. mma.sync and not tcgen05:
// the rows of a decode step fill N = 8..32, the tensor time is a fraction of
// the load time either way, and S^T and P^T stay in the registers of one warp
// where a tcgen05 kernel passes them through TMEM and shared memory and
// synchronises the CTA on every tile.
//
// Work split: the keys of all (sequence, KV head, row tile) segments form one
// list of units (a tile for each warp of a CTA, 64 to 256 keys); each CTA (one to
// three per SM) takes an equal contiguous share of it, read from kv_len on the
// device, so uneven lengths balance and a captured graph follows the lengths. A
// segment inside one CTA is normalised
// and written there; one cut by a share's end leaves (m, l, O) states in the
// workspace for the merge kernel (fr_paged.cu).
//
// P enters the PV product as two f16 terms P_hi + P_lo (22 bits), held between
// 2^7 and 2^15 at the maximum to keep P_lo off f16's subnormals: the result
// carries fp32 accuracy like fr_decode_attn's. e4m3 codes become f16 in registers, which is exact; K's
// scale joins the score's factor, V's scale the weights, relative to the
// largest V scale that the row has met in its view (a running reference beside
// m). It is one number a warp where the rows have met about the same; tiles at
// the ends of the views may set rows apart, since a scale that only other rows
// see may be any number of times larger, and then each has its own. (One for
// every row throughout: 63.4 us at 131072 keys of e4m3 and 54.2 at 32 sequences of
// ..4096 keys with 16 rows, in place of 60.3 and 49.8.)
#pragma once

#include <cuda_fp16.h>
#include <string.h>

#include <type_traits>

#include "fr_paged_work.cuh"

namespace fr {
namespace paged {

using namespace sm100;

// Weights are 2^(x - mref): a row's reference mref is 7 below its maximum when
// set, and moves when a score exceeds it by 15, so weights reach 2^15 at most in
// f16 and P_lo stays off f16's subnormals for all weights that matter. x is the
// rounded product of score and factor wherever it is used: in one FMA with the
// subtraction it would be off the maximum's x by up to half its last place,
// more than 15 from 2^28 on, and equal scores would differ.
constexpr float kBelow = 7.0f, kAbove = 15.0f;
constexpr float kNoRef = -3.402823466e38f;           // a row without a key so far
constexpr float kVMin = 0x1p-120f;                   // a V reference at least: its reciprocal stays finite
// Rows whose V references differ by no more share the largest of them. That costs the
// weights of the others 4 bits at either end of their views: f16's fixed step is then
// 2^-24 of the row's largest weight at most, beside 2^-22 of each.
constexpr float kVSlack = 16.0f;
constexpr uint64_t kWaitNs = 2000000000ull;
// An MMA drops bits of the sum that it adds to, always towards zero: with values of one
// sign, rows were too small by 2.5e-6 of themselves where a warp had 512 keys of a piece and
// by 4.8e-5 where it had 8192 (hd 256 and 32 rows 3.0e-5, e4m3 2.1e-5 and 1.0e-5). A warp with more than
// so many therefore takes the products of each tile by themselves and adds them to O in
// fp32 (2e-7 at any length): 64 sequences of ..8192 keys 163.8 and 164.7 us, e4m3 93.4 and
// 93.3. For all pieces it would cost the short ones (1 x 968 keys of hd 256 8.3 and 8.6 us, 65536
// 26.5 and 28.3, e4m3 131072 61.3 and 64.4; from 512 keys on 64.9 there).
constexpr int kChainKeys = 1024;

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int row, int head, int page,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
        "[%7];"
        :: "r"(dst), "l"((uint64_t)map), "r"(0), "r"(row), "r"(0), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// D (16x8 f32) += A (16x16 f16, row) * B (16x8 f16, col); free to be scheduled
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int HD, int TYPE, int NT>
struct Cfg {
    static constexpr bool E4 = TYPE == FR_KV_E4M3;
    static constexpr int RT = 8 * NT;                       // query rows of a row tile
    static constexpr int ROWB = HD * (E4 ? 1 : 2);          // bytes of a K or V row
    static constexpr int PITCH = ROWB < 128 ? ROWB : 128;   // bytes of a row in one box
    static constexpr int MT = HD / 16;                      // 16-dim blocks of O^T, and k steps of S^T
    static constexpr int W = cta_warps(HD, NT);
    static constexpr int LIMIT = cta_smem(HD, NT);          // shared memory of one CTA
    // Q rows lie in shared memory; the fragments stay in registers for a piece
    // where these allow (hd 128 with 16 rows reads them again for each tile: 63 ->
    // 59 us at 131072 keys of e4m3, the registers went to a third CTA)
    static constexpr bool QREG = many_warps(HD, NT) ? HD * NT <= 128 : HD * NT <= 256;
    static constexpr int QPITCH = HD * 2 + 16;              // bytes: rows on different banks
    static constexpr int QBYTES = RT * QPITCH;
    static constexpr int STATE = W * RT * 8;
    static constexpr int ENTRIES = 8;                       // tiles requested and not used up, at most
    static constexpr int META = W * ENTRIES * 32;
    static constexpr int VIEWS = 2 * RT * 8;
    // alignment slack, buffers above, then barriers, walks and scan words
    static constexpr int FIXED = 1024 + QBYTES + STATE + META + VIEWS + W * 64 + (W + 2) * 64 + 128;
    // 32 keys a slot where three slots of them fit (K, V and the next K), else 16
    static constexpr int SUB = 3 * W * 32 * ROWB <= LIMIT - FIXED ? 2 : 1;
    static constexpr int KT = kTile * SUB;                  // keys of a warp's tile
    static constexpr int SUBB = kTile * ROWB, SLOT = SUB * SUBB;
    static constexpr int NS_ = (LIMIT - FIXED) / (W * SLOT);
    static constexpr int NS = NS_ > 8 ? 8 : NS_;            // slots of a warp's ring
    static constexpr int SMEM = FIXED + NS * W * SLOT;
    static_assert(NS >= 3 && SMEM <= 232448, "ring");
    // what the kernel lays out behind the alignment slack
    static_assert(NS * W * SLOT + QBYTES + STATE + META + VIEWS + W * 64 + (W + 2) * 64 + 128 <= SMEM - 1024,
                  "shared memory layout");
    // rows of a warp's O^T that one slot holds in fp32: the epilogue's chunk
    static constexpr int CNT = SLOT / (HD * 32) < NT ? SLOT / (HD * 32) : NT;
    static_assert(CNT >= 1 && NT % CNT == 0, "epilogue chunk");
};

// Waits for a slot of a warp's ring of n, in its phase. One that gives up waits, again with
// a limit, for the copies that are in flight behind it: the warp asks for no more, and the CTA
// must not end before they have landed.
static __device__ __noinline__ bool wait_long(uint32_t bars, int slot, uint32_t phase, int n) {
    if (mbar_wait(bars + 8 * slot, phase, kWaitNs)) return true;
    uint64_t limit = kWaitNs;
    for (int i = 0; i < n; ++i) {
        if (!mbar_wait(bars + 8 * slot, phase, limit)) limit = 20000ull;
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
    return false;
}

// A lane for a row: the row's V reference, raised to the largest scale of the steps of
// a tile (first key key0, U steps) that it sees, and what its O is to be scaled by.
template <int U, bool SINK>
static __device__ __noinline__ float2 raise_v(int2 see, int sink, float old, float2* ref, int key0, uint32_t bad, float v0,
                                              float v1) {
    float v = old, f = 1.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int j = key0 + u * kTile;
        if (!(bad >> u & 1u) && j < see.x && (j + kTile > see.y || (SINK && j < sink))) v = fmaxf(v, fabsf(u ? v1 : v0));
    }
    if (v > old) f = old / v;
    *ref = make_float2(1.f / v, v);
    return make_float2(v, f);
}

template <int HD, int TYPE, int NT, bool SINK>
__global__ void __launch_bounds__(cta_warps(HD, NT) * 32, ctas_per_sm(HD, NT))
paged_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using C = Cfg<HD, TYPE, NT>;
    constexpr int W = C::W, RT = C::RT, MT = C::MT, NS = C::NS, KT = C::KT, SUB = C::SUB;
    constexpr bool E4 = C::E4;
    constexpr int MV = E4 ? 2 : 1;                          // 16-dim blocks of one load of V
    using P = Units<RT, KT, W, kSegCost, SINK>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    unsigned char* ring = base + warp * NS * C::SLOT;
    unsigned char* after = base + W * NS * C::SLOT;
    unsigned char* q_sm = after;                                                         // [RT][QPITCH]
    // [warp][RT]: at a piece's end (reference, sum of weights); before it (1 / v, v), v the V references of rows set apart
    float2* state = reinterpret_cast<float2*>(q_sm + C::QBYTES);
    struct Entry { float ks[2], vs[2]; uint32_t bad, pad[3]; };                          // of a tile's 16-key halves
    unsigned char* misc = q_sm + C::QBYTES + C::STATE;
    Entry* meta = reinterpret_cast<Entry*>(misc) + warp * C::ENTRIES;
    int2* views = reinterpret_cast<int2*>(misc + C::META);                               // [2][RT]
    misc += C::META + C::VIEWS;
    uint64_t* bars = reinterpret_cast<uint64_t*>(misc) + warp * 8;
    Walk* cws = reinterpret_cast<Walk*>(misc + W * 64);                             // [2]
    Walk* pw = cws + 2 + warp;
    int* scan = reinterpret_cast<int*>(cws + 2 + W);                                // [32]
    const uint32_t ring_u = smem_addr(ring), bars_u = smem_addr(bars);

    if (lane == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(bars_u + 8 * i, 1);
        mbar_fence_init();
        if (warp == 0) {
            prefetch_tmap(&k_map);
            prefetch_tmap(&v_map);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this CTA's share of the units ------------------------------------
    const int cta = blockIdx.x;
    const Share share = first_walk<P, W * 32>(a, cta, scan, cws);
    if (share.units == 0) return;
    // For a piece's rows: the keys each sees, [y, x), and copies of its Q rows to
    // shared memory (a 16-dim group in the order the MMA takes its dims).
    constexpr int QN = (RT * HD / 8 + W * 32 - 1) / (W * 32);      // 16-byte chunks of a thread
    uint4 qx[QN];                // (e4m3: on their way)
    auto open_piece = [&](int which) {
        const Walk& w = cws[which];
        if (!w.more) return;
        const int row0 = w.s.rt * RT, rows = min(RT, w.s.n_q * a.group - row0);
        if (tid < RT) {
            int hi = w.s.n_kv, lo = 0;
            if (a.causal) {
                const int p = w.s.n_kv - w.s.n_q + token_of(row0 + min(tid, rows - 1), a);
                hi = min(hi, p + 1);
                if (a.window > 0) lo = max(0, p + 1 - a.window);
            }
            views[which * RT + tid] = make_int2(hi, lo);
        }
        const uint32_t q_u = smem_addr(q_sm);
#pragma unroll
        for (int k = 0; k < QN; ++k) {
            const int r = (k * W * 32 + tid) / (HD / 8), c = tid % (HD / 8);
            if (r >= RT) break;
            const int i = token_of(row0 + min(r, rows - 1), a), hh = row0 + min(r, rows - 1) - i * a.group;
            const __half* src = a.q16 + (int64_t)(w.s.tok0 + i) * a.q_stride + (int64_t)(w.s.h * a.group + hh) * HD + c * 8;
            // rows behind the last are zeros
            if (E4)
                qx[k] = r < rows ? __ldcg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            else
                cp_async16(q_u + r * C::QPITCH + c * 16, src, r < rows ? 16 : 0);
        }
        if (!E4) cp_async_commit();
    };
    // The copies have arrived; e4m3's MMA takes dims 4i .. 4i + 3 as two pairs 8 places apart.
    auto close_open = [&](int which) {
        if (!E4) {
            cp_async_wait<0>();
        } else if (cws[which].more) {
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const int r = (k * W * 32 + tid) / (HD / 8), c = tid % (HD / 8);
                if (r >= RT) break;
                unsigned char* dst = q_sm + r * C::QPITCH + (c >> 1) * 32 + (c & 1) * 8;
                *reinterpret_cast<uint2*>(dst) = make_uint2(qx[k].x, qx[k].z);
                *reinterpret_cast<uint2*>(dst + 16) = make_uint2(qx[k].y, qx[k].w);
            }
        }
    };
    __syncthreads();
    if (!cws[0].more) return;    // (only if the lengths change during the call)
    if (lane < 16) reinterpret_cast<int*>(pw)[lane] = reinterpret_cast<const int*>(cws)[lane];
    open_piece(0);               // ahead of the ring's requests, which fill the memory system's queues
    __syncwarp();

    // ---- the warp's ring: slots q = 0, 1, ... hold K, V, K, V, ... of its tiles ----
    int2 pt = walk_tiles<P>(*pw, warp);   // the next tile to request of the piece, and its end
    if (pt.x >= pt.y) pt = request_next<P>(pw, &a, warp);
    constexpr int BLK = 32 / SUB;  // tiles of a page block: a lane for each 16 keys
    int blk = 0;                 // tiles of the page block used up
    int b_page = -1, p_page[SUB] = {};
    float b_ks = 0.f, b_vs = 0.f;
    int i_slot = 0, i_tile = 0;  // ring slot of the next request; its tile's number mod ENTRIES
    bool i_v = false, fresh = false, b_has = false, timeout = false;
    // Page numbers of the warp's next 32 16-key steps, one a lane; -1: none. Asked
    // for one request ahead of their use.
    auto load_pages = [&]() {
        blk = 0;
        const int tl = pt.x + lane / SUB * W, key = tile_key<P>(pw->s, tl, sink_tiles<P>(pw->s, a)) + lane % SUB * kTile;
        // (16 keys that no row sees: their page may be gone)
        b_has = tl < pt.y && key < pw->s.n_kv && (key + kTile > pw->s.lo || P::is_sink(key, a));
        b_page = -1;
        if (b_has) b_page = __ldcg(a.table + pw->s.b * a.table_stride + (key >> a.page_shift));
        fresh = true;
    };
    load_pages();
    auto request = [&]() {
        if (pt.x >= pt.y) return;                      // the share's end
        if (!i_v) {              // a new tile: its pages
            if (fresh && b_has && (b_page < 0 || b_page >= a.n_pages)) {
                atomicOr(a.status, kStatusInput);
                b_page = -1;
            }
            uint32_t bad = 0u;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                p_page[u] = __shfl_sync(~0u, b_page, blk * SUB + u);
                // no such page: page 0, which exists, is read in its place and its keys are masked
                if (p_page[u] < 0) bad |= 1u << u;
                p_page[u] = max(p_page[u], 0);
            }
            if (lane == 0) meta[i_tile].bad = bad;
        }
        if (lane == 0 && !timeout) {
            const uint32_t bar = bars_u + 8 * i_slot;
            const int key = tile_key<P>(pw->s, pt.x, sink_tiles<P>(pw->s, a)), in_page = (1 << a.page_shift) - 1, head = pw->s.h;
            mbar_expect_tx(bar, C::SLOT);
#pragma unroll
            for (int u = 0; u < SUB; ++u)
                tma_load_5d(ring_u + i_slot * C::SLOT + u * C::SUBB, i_v ? &v_map : &k_map, (key + u * kTile) & in_page,
                            head, p_page[u], bar);
        }
        if (++i_slot == NS) i_slot = 0;
        if (!i_v) {
            if (E4 && fresh) {   // the block's scales, awaited with the V request
                b_ks = b_vs = 0.f;
                if (b_page >= 0) {
                    b_ks = __ldcg(a.k_scale + (int64_t)b_page * a.n_kv_head + pw->s.h);
                    b_vs = __ldcg(a.v_scale + (int64_t)b_page * a.n_kv_head + pw->s.h);
                }
            }
            fresh = false;
        } else {
            if (E4) {            // the tile's scales, for the consumer
                float ks[SUB], vs[SUB];
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    ks[u] = __shfl_sync(~0u, b_ks, blk * SUB + u);
                    vs[u] = __shfl_sync(~0u, b_vs, blk * SUB + u);
                }
                if (lane == 0) {
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        meta[i_tile].ks[u] = ks[u];
                        meta[i_tile].vs[u] = vs[u];
                    }
                }
            }
            i_tile = (i_tile + 1) % C::ENTRIES;
            ++blk;
            if ((pt.x += W) >= pt.y) {
                pt = request_next<P>(pw, &a, warp);
                blk = BLK;
            }
            if (blk == BLK) load_pages();
        }
        i_v = !i_v;
    };
    __syncwarp();
    for (int i = 0; i < NS; ++i) request();
    __syncwarp();                // the tile entries above are read by the whole warp

    int c_slot = 0, c_tile = 0;
    uint32_t c_phase = 0;
    auto wait_slot = [&]() {
        if (mbar_test(bars_u + 8 * c_slot, c_phase)) return;
        // after one wait that gave up there is nothing to wait for: the kernel ends
        if (!timeout && !wait_long(bars_u, c_slot, c_phase, NS)) timeout = true;
    };
    auto pass_slot = [&](bool hold) {    // this slot is used up: request what comes NS slots later, unless it is held
        __syncwarp();
        if (!hold) request();
        if (++c_slot == NS) {
            c_slot = 0;
            c_phase ^= 1;
        }
    };

    // Addresses of this lane's 16-byte chunks for ldmatrix, in the TMA's swizzle:
    // row r of a 16-row box, chunk c + h with h this lane's bit and c even, is at
    // (base + lane part) ^ (c << 4), the slots being aligned beyond those bits.
    auto swz = [](int r) { return C::PITCH == 128 ? r & 7 : (r >> 1) & 3; };
    constexpr int CPB = C::PITCH / 16;               // chunks of a row in a box
    const int k_r = (lane & 7) + ((lane >> 3) & 1) * 8, k_h = lane >> 4;
    const int v_r = E4 ? k_r : (lane & 7) + (lane >> 4) * 8, v_h = E4 ? k_h : (lane >> 3) & 1;
    const uint32_t k_lane = ring_u + k_r * C::PITCH + ((k_h ^ swz(k_r)) << 4);
    const uint32_t v_lane = ring_u + v_r * C::PITCH + ((v_h ^ swz(v_r)) << 4);
    auto at_chunk = [](uint32_t base, int sub, int c) {
        return (base ^ ((c % CPB) << 4)) + sub * C::SUBB + c / CPB * (kTile * C::PITCH);
    };

    close_open(0);
    __syncthreads();
    for (int which = 0;; which ^= 1) {
        // ---- a piece: its rows and their Q fragments --------------------------
        const Walk& cw = cws[which];
        const int2* view = views + which * RT;
        const bool whole = cw.ua == 0 && cw.ub == cw.s.n_units;
        // state slot: 2*cta + 1 for a segment that goes on in the next CTA from its start here, else 2*cta
        const int part = 2 * cta + (cw.ua == 0 && !whole ? 1 : 0);
        const int row0 = cw.s.rt * RT, tok0 = cw.s.tok0, head0 = cw.s.h * a.group;
        const int rows = min(RT, cw.s.n_q * a.group - row0);
        if (tid == (W - 1) * 32) {         // (the last warp has no more tiles than the others)
            put_split(a, share, cta, cw, row0, rows);
            walk_next<P>(&cw, &cws[which ^ 1], &a);
        }
        const int min_lim = view[0].x, max_low = view[RT - 1].y;       // (rows behind the last see what it sees)
        const uint32_t q_lane = smem_addr(q_sm) + ((lane & 7) + (NT > 1 ? lane >> 4 : 0) * 8) * C::QPITCH +
                                (NT > 1 ? (lane >> 3) & 1 : lane >> 3) * 16;
        uint32_t qf[C::QREG ? MT : 1][NT][2];
        if (C::QREG) {
            if (NT == 1) {                           // four matrices: two k steps of one row block
#pragma unroll
                for (int kk = 0; kk < MT; kk += 2)
                    ldsm_x4(q_lane + kk * 32, qf[kk][0][0], qf[kk][0][1], qf[kk + 1][0][0], qf[kk + 1][0][1]);
            } else {
#pragma unroll
                for (int kk = 0; kk < MT; ++kk)
#pragma unroll
                    for (int n = 0; n < NT; n += 2)
                        ldsm_x4(q_lane + n * 8 * C::QPITCH + kk * 32, qf[kk][n][0], qf[kk][n][1], qf[kk][(n + 1) % NT][0],
                                qf[kk][(n + 1) % NT][1]);
            }
        }
        // B fragments of step kk for all row blocks
        auto q_frags = [&](int kk, uint32_t (*b)[2]) {
            if (C::QREG) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    b[n][0] = qf[kk][n][0];
                    b[n][1] = qf[kk][n][1];
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; n += 2)
                    ldsm_x4(q_lane + n * 8 * C::QPITCH + kk * 32, b[n][0], b[n][1], b[(n + 1) % NT][0], b[(n + 1) % NT][1]);
            }
        };

        float o[MT][NT][4];
        float mref[NT][2], l[NT][2];
        // 1 / largest V scale in the rows' views so far; of rows set apart (their own are in state[]), the largest of them
        float vinv = 1.f / kVMin;
        bool apart = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mref[n][0] = mref[n][1] = kNoRef;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) o[m][n][0] = o[m][n][1] = o[m][n][2] = o[m][n][3] = 0.f;
        }

        const int2 tiles = walk_tiles<P>(cw, warp);
        const int first_tiles = sink_tiles<P>(cw.s, a), tile0 = cw.s.tile0 - first_tiles;
        const bool tile_sums = (tiles.y - tiles.x) * KT > kChainKeys * W;
        for (int t = tiles.x; t < tiles.y; t += W) {
            // ---- S^T = K Q^T ------------------------------------------------
            wait_slot();
            const Entry& en = meta[c_tile];
            const uint32_t bad = en.bad;
            const uint32_t k_base = k_lane + c_slot * C::SLOT;
            float s[SUB][NT][4], s2[SUB][NT][4];     // s2: a second chain of MMAs where there is one tile
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][n][e] = s2[u][n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < MT; kk += E4 ? 2 : 1) {
                uint32_t qa[NT][2], qb[NT][2];
                q_frags(kk, qa);
                if (E4) q_frags(kk + 1, qb);
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t r[4];
                    ldsm_x4(at_chunk(k_base, u, E4 ? kk : 2 * kk), r[0], r[1], r[2], r[3]);
                    if (E4) {
                        const uint32_t a0[4] = {e4m3_lo(r[0]), e4m3_lo(r[1]), e4m3_hi(r[0]), e4m3_hi(r[1])};
                        const uint32_t a1[4] = {e4m3_lo(r[2]), e4m3_lo(r[3]), e4m3_hi(r[2]), e4m3_hi(r[3])};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma(s[u][n], a0, qa[n][0], qa[n][1]);
                            mma(SUB == 1 ? s2[u][n] : s[u][n], a1, qb[n][0], qb[n][1]);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma(SUB == 1 && (kk & 1) ? s2[u][n] : s[u][n], r, qa[n][0], qa[n][1]);
                    }
                }
            }
            if (SUB == 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[0][n][e] += s2[0][n][e];
            }
            float sc[SUB], vs[SUB], vmax = 0.f;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                sc[u] = E4 ? a.scale_log2 * en.ks[u] : a.scale_log2;
                vs[u] = E4 ? en.vs[u] : 1.f;
                vmax = fmaxf(vmax, fabsf(vs[u]));
            }
            pass_slot(false);

            // ---- softmax weights: exponents x - mref first -------------------
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][n][e] = __fmul_rn(s[u][n][e], sc[u]);
            const int key0 = SINK && t < first_tiles ? t * KT : (tile0 + t) * KT;
            const bool edge = bad != 0u || key0 + KT > min_lim || (key0 < max_low && P::hidden(key0 + KT - 1, a));
            bool up = false;
            float y[SUB][NT][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[u][n][e] = __fsub_rn(s[u][n][e], mref[n][e & 1]);
                        up |= y[u][n][e] > kAbove;
                    }
            if (__builtin_expect(edge, 0)) {
                up = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int2 see = view[n * 8 + 2 * t4 + c];
#pragma unroll
                        for (int u = 0; u < SUB; ++u)
#pragma unroll
                            for (int e = c; e < 4; e += 2) {
                                const int j = key0 + u * kTile + g + (e >> 1) * 8;
                                if ((bad >> u & 1u) || j >= see.x || (j < see.y && P::hidden(j, a))) y[u][n][e] = -INFINITY;
                                up |= y[u][n][e] > kAbove;
                            }
                    }
            }
            // (somewhat above 1: a scale times its own rounded reciprocal)
            const bool vup = E4 && vmax * vinv > 1.0001f;
            if (__any_sync(~0u, up) || vup) {
                float va = 1.f;
                if (vup) {
                    // One reference for all rows: where all see every key that is looked up (of a tile ahead of
                    // all windows those before the sinks' end), or where those that do not see the step are at
                    // their end, and see none whose scale is far smaller
                    const bool one_view = !edge || (min_lim == cw.s.n_kv && view[0].y == max_low) ||
                                          (SINK && key0 + KT <= view[0].y);
                    const bool at_end = max_low <= key0 &&
                                        (SUB == 1 || key0 + kTile < min_lim || fabsf(vs[SUB - 1]) <= kVSlack * fabsf(vs[0])) &&
                                        (vinv == 1.f / kVMin || vmax * vinv < 0x1p60f);
                    if (__builtin_expect(!apart && (one_view || at_end), 1)) {
                        const float inv = 1.f / vmax;
                        va = inv / vinv;
                        vinv = inv;
                    } else {
                        // a lane for a row: the largest scale of the steps that it sees
                        // (lanes behind the last row do a row's work again)
                        const int row = lane % RT;
                        float2* ref = state + warp * RT + row;
                        const float old = apart ? ref->y : 1.f / vinv;
                        __syncwarp();
                        const float2 raised = raise_v<SUB, SINK>(view[row], a.sink, old, ref, key0, bad, vs[0], vs[SUB - 1]);
                        // (not negative: ordered as their bits)
                        const float v = raised.x, most = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(v))),
                                    least = __uint_as_float(__reduce_min_sync(~0u, __float_as_uint(v)));
                        apart = most > kVSlack * least;
                        vinv = 1.f / (apart ? least : most);
                        const float vr = apart ? raised.y : raised.y * (v / most);
#pragma unroll
                        for (int u = 0; u < SUB; ++u)
                            if (fabsf(vs[u]) > most) vs[u] = 0.f;        // nobody sees this step
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float f = __shfl_sync(~0u, vr, n * 8 + 2 * t4 + c);
#pragma unroll
                                for (int m = 0; m < MT; ++m) {
                                    o[m][n][c] *= f;
                                    o[m][n][2 + c] *= f;
                                }
                            }
                        __syncwarp();                // (the references are read by all lanes)
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float al[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float m = -INFINITY;
#pragma unroll
                        for (int u = 0; u < SUB; ++u)
#pragma unroll
                            for (int e = c; e < 4; e += 2)
                                m = fmaxf(m, y[u][n][e] == -INFINITY ? -INFINITY : s[u][n][e]);
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, w));
                        m = fmaxf(m - kBelow, mref[n][c]);
                        al[c] = ex2(mref[n][c] - m);
                        mref[n][c] = m;
                        l[n][c] *= al[c];
                        if (E4) al[c] *= va;
#pragma unroll
                        for (int u = 0; u < SUB; ++u)
#pragma unroll
                            for (int e = c; e < 4; e += 2)
                                y[u][n][e] = y[u][n][e] == -INFINITY ? -INFINITY : __fsub_rn(s[u][n][e], m);
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        o[m][n][0] *= al[0];
                        o[m][n][1] *= al[1];
                        o[m][n][2] *= al[0];
                        o[m][n][3] *= al[1];
                    }
                }
            }
            if (E4 && !apart) {
#pragma unroll
                for (int u = 0; u < SUB; ++u) vs[u] *= vinv;
            }
            // Of rows set apart, step u's V scale over the row's reference: at most 1 in size where
            // the row sees the step, and held to 1 where it does not, so that its zero weights stay zeros
            auto v_share = [&](int u, int n, int c) {
                return copysignf(__saturatef(fabsf(vs[u]) * state[warp * RT + n * 8 + 2 * t4 + c].x), vs[u]);
            };
            uint32_t ph[SUB][NT][2], pl[SUB][NT][2];
            auto weigh = [&](auto rows_apart) {
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float f0 = vs[u], f1 = vs[u];
                        if (decltype(rows_apart)::value) {
                            f0 = v_share(u, n, 0);
                            f1 = v_share(u, n, 1);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float w0 = ex2(y[u][n][2 * e]), w1 = ex2(y[u][n][2 * e + 1]);
                            l[n][0] += w0;
                            l[n][1] += w1;
                            if (E4) {
                                w0 *= f0;
                                w1 *= f1;
                            }
                            const __half2 h = __floats2half2_rn(w0, w1);
                            const float2 hf = __half22float2(h);
                            ph[u][n][e] = movm(*reinterpret_cast<const uint32_t*>(&h));
                            pl[u][n][e] = movm(pack_half2(w0 - hf.x, w1 - hf.y));
                        }
                    }
            };
            if (E4 && __builtin_expect(apart, 0)) weigh(std::true_type());
            else weigh(std::false_type());

            // ---- O^T += V^T P^T ------------------------------------------------
            wait_slot();
            if (__builtin_expect(edge, 0)) {
                // A masked key has weight 0, but 0 * inf and 0 * NaN are NaN: rows
                // of V that no query row sees are cleared (they may lie behind the
                // sequence's end), and non-finite rows seen by some rows only are
                // added here for those rows and then cleared.
                for (int u = 0; u < SUB; ++u) {
                    unsigned char* sp = ring + c_slot * C::SLOT + u * C::SUBB;
                    const bool no_page = bad >> u & 1u;
                    for (int e = 0; e < 2; ++e) {
                        const int j0 = key0 + u * kTile + e * 8;
                        bool vis = false, msk = false;
                        for (int r = 2 * t4; r < rows; r += (r & 1) ? 7 : 1) {
                            const int2 see = view[r];
                            const bool m = no_page || j0 + g >= see.x || (j0 + g < see.y && P::hidden(j0 + g, a));
                            vis |= !m;
                            msk |= m;
                        }
                        unsigned v = __ballot_sync(~0u, vis), m = __ballot_sync(~0u, msk);
                        v |= v >> 2;
                        v |= v >> 1;
                        m |= m >> 2;
                        m |= m >> 1;
                        unsigned dead = ~v & 0x11111111u, part = v & m & 0x11111111u;    // bit 4i: key j0 + i
                        for (; part; part &= part - 1) {
                            const int j = (__ffs(part) - 1) >> 2;
                            const unsigned char* row = sp + (j + e * 8) * C::PITCH;
                            bool weird = false;
                            for (int c = lane; c < C::ROWB / 4; c += 32) {
                                const uint32_t x = *reinterpret_cast<const uint32_t*>(
                                    row + c * 4 / C::PITCH * (kTile * C::PITCH) + c * 4 % C::PITCH);
                                if (E4) {
                                    const uint32_t z = x & 0x7f7f7f7fu;
                                    weird |= (z & 0xffu) == 0x7fu || (z >> 8 & 0xffu) == 0x7fu ||
                                             (z >> 16 & 0xffu) == 0x7fu || z >> 24 == 0x7fu;
                                } else {
                                    weird |= (x & 0x7c00u) == 0x7c00u || (x & 0x7c000000u) == 0x7c000000u;
                                }
                            }
                            if (!__any_sync(~0u, weird)) continue;
                            dead |= 1u << (4 * j);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    float x = e ? y[0][n][2 + c] : y[0][n][c], vsc = vs[0];
                                    if (SUB == 2 && u) {
                                        x = e ? y[SUB - 1][n][2 + c] : y[SUB - 1][n][c];
                                        vsc = vs[SUB - 1];
                                    }
                                    if (E4 && apart) vsc = SUB == 2 && u ? v_share(SUB - 1, n, c) : v_share(0, n, c);
                                    x = __shfl_sync(~0u, x, j * 4 + t4);
                                    if (x == -INFINITY) continue;
                                    const float w = ex2(x) * vsc;
#pragma unroll
                                    for (int m = 0; m < MT; ++m)
#pragma unroll
                                        for (int i = 0; i < 2; ++i) {
                                            const int d = m * 16 + (E4 ? 2 * g + i : g + 8 * i), by = d * (E4 ? 1 : 2);
                                            const unsigned char* at = row + by / C::PITCH * (kTile * C::PITCH) +
                                                                      ((by % C::PITCH >> 4 ^ swz(j)) << 4) + (by & 15);
                                            float v;
                                            if (E4) {
                                                const uint32_t hv = e4m3_lo(*at);
                                                v = __half2float(__ushort_as_half((unsigned short)hv));
                                            } else {
                                                v = __half2float(*reinterpret_cast<const __half*>(at));
                                            }
                                            o[m][n][2 * i + c] += w * v;
                                        }
                                }
                        }
                        __syncwarp();
                        if (dead)
                            for (int c = lane; c < C::SUBB / 32; c += 32) {    // the 8 rows of this half, box by box
                                const int box = c / (C::PITCH / 2), at = c % (C::PITCH / 2) * 16;
                                if (dead >> (4 * (at / C::PITCH)) & 1u)
                                    *reinterpret_cast<uint4*>(sp + box * (kTile * C::PITCH) + e * 8 * C::PITCH + at) =
                                        make_uint4(0, 0, 0, 0);
                            }
                    }
                }
                fence_proxy_async_cta();             // the slot's next fill comes by TMA
                __syncwarp();
            }
            const uint32_t v_base = v_lane + c_slot * C::SLOT;
            // V^T of step u: dims m * 16 .. (e4m3: two blocks of 16)
            auto v_frags = [&](int m, int u, uint32_t (*r)[4]) {
                uint32_t x[4];
                ldsm_x4_t(at_chunk(v_base, u, E4 ? m : 2 * m), x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (E4) {
                        x[i] = __byte_perm(x[i], 0, 0x3120);
                        r[E4 ? i >> 1 : 0][2 * (i & 1)] = e4m3_lo(x[i]);
                        r[E4 ? i >> 1 : 0][2 * (i & 1) + 1] = e4m3_hi(x[i]);
                    } else {
                        r[0][i] = x[i];
                    }
                }
            };
            if (!tile_sums) {
#pragma unroll
                for (int m = 0; m < MT; m += MV)
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        uint32_t r[MV][4];
                        v_frags(m, u, r);
                        if (E4) {
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 2 * MV; ++i)
                                    mma(o[m + i % MV][n], r[i % MV], i < MV ? ph[u][n][0] : pl[u][n][0],
                                        i < MV ? ph[u][n][1] : pl[u][n][1]);
                        } else {
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma(o[m][n], r[0], ph[u][n][0], ph[u][n][1]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma(o[m][n], r[0], pl[u][n][0], pl[u][n][1]);
                        }
                    }
            } else {
#pragma unroll
                for (int m = 0; m < MT; m += MV) {
                    uint32_t r[SUB][MV][4];
#pragma unroll
                    for (int u = 0; u < SUB; ++u) v_frags(m, u, r[u]);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < MV; ++i) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int u = 0; u < SUB; ++u) {
                                mma(d, r[u][i], ph[u][n][0], ph[u][n][1]);
                                mma(d, r[u][i], pl[u][n][0], pl[u][n][1]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[m + i][n][e] += d[e];
                        }
                }
            }
            pass_slot(t + W >= tiles.y);        // the piece's last slot takes O first
            c_tile = (c_tile + 1) % C::ENTRIES;
        }

        // ---- the piece's end: the warps' states become one --------------------
        const bool had = tiles.x < tiles.y;          // a warp without a tile has no state, and holds no slot
        const int held = c_slot == 0 ? NS - 1 : c_slot - 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], w);
                // no weight: no key seen. Only NaN scores: a state all the same, so that they reach the result
                if (l[n][e] == 0.f) mref[n][e] = -INFINITY;
                else if (mref[n][e] == kNoRef) mref[n][e] = 0.f;
                float2* st = state + warp * RT + n * 8 + 2 * t4 + e;
                if (E4) {                            // O without its V reference
                    const float v = apart ? st->y : 1.f / vinv;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        o[m][n][e] *= v;
                        o[m][n][2 + e] *= v;
                    }
                    if (apart) __syncwarp();
                }
                if (g == 0) *st = make_float2(mref[n][e], l[n][e]);
            }
        // O^T as fp32 rows in the slot that the warp held back, in chunks of CNT
        // row blocks; dims of a row are moved by its number against bank conflicts
        auto o_at = [](int r, int d) { return r * HD + (d ^ ((r >> 1 & 3) << 3)); };
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += C::CNT) {
            if (n0) __syncthreads();
            if (had) {
                float* dst = reinterpret_cast<float*>(ring + held * C::SLOT);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < C::CNT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[o_at(n * 8 + 2 * t4 + (e & 1), m * 16 + (E4 ? 2 * g + (e >> 1) : g + 8 * (e >> 1)))] =
                                o[m][n0 + n][e];
                if (lane == 0) reinterpret_cast<const float**>(scan)[warp] = dst;
            }
            __syncthreads();
            if (n0 == 0) open_piece(which ^ 1);      // the next piece's Q rows come while this one is written
            const int chunk_rows = min(C::CNT * 8, rows - n0 * 8);
            for (int w = tid; w < chunk_rows * (HD / 4); w += W * 32) {
                const int rr = w / (HD / 4), r = n0 * 8 + rr, d = (w - rr * (HD / 4)) * 4;
                float m = -INFINITY, lsum = 0.f;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int v = 0; v < W; ++v) m = fmaxf(m, state[v * RT + r].x);
#pragma unroll
                for (int v = 0; v < W; ++v) {
                    const float2 st = state[v * RT + r];
                    if (st.x == -INFINITY) continue;             // no key seen, or no tile
                    const float f = ex2(st.x - m);
                    lsum += st.y * f;
                    const float* src = reinterpret_cast<const float* const*>(scan)[v];
                    const float4 y = *reinterpret_cast<const float4*>(src + o_at(rr, d));
                    x.x += f * y.x;
                    x.y += f * y.y;
                    x.z += f * y.z;
                    x.w += f * y.w;
                }
                if (whole) {
                    const float inv = m == -INFINITY ? 0.f : 1.f / lsum;
                    x.x *= inv;
                    x.y *= inv;
                    x.z *= inv;
                    x.w *= inv;
                    const int i = token_of(row0 + r, a), hh = (row0 + r) - i * a.group;
                    float* dst = a.out + ((int64_t)(tok0 + i) * a.n_kv_head * a.group + head0 + hh) * HD;
                    *reinterpret_cast<float4*>(dst + d) = x;
                } else {
                    *reinterpret_cast<float4*>(a.part_o + ((int64_t)part * RT + r) * HD + d) = x;
                    if (d == 0) a.part_ml[part * RT + r] = make_float2(m, lsum);
                }
            }
        }
        close_open(which ^ 1);
        fence_proxy_async_cta();                     // the held slot's next fill comes by TMA
        __syncthreads();
        if (had) request();
        if (!cws[which ^ 1].more) break;
    }
    if (timeout) atomicOr(a.status, kStatusTimeout);
}

// Programmatic launch: set-up overlaps the kernel before it on the stream.
template <int HD, int TYPE, int NT, bool SINK>
static fr_status launch_one(const KvDesc& kv, const AttnArgs& a, int ctas, cudaStream_t st) {
    using C = Cfg<HD, TYPE, NT>;
    static unsigned long long done = 0ull;           // devices whose shared-memory limit is raised
    if (kv.dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> kv.dev & 1ull)) {
        if (cudaFuncSetAttribute(paged_attn_kernel<HD, TYPE, NT, SINK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::SMEM) != cudaSuccess)
            return FR_ERR_CUDA;
        if (kv.dev < 64) __atomic_fetch_or(&done, 1ull << kv.dev, __ATOMIC_RELEASE);
    }
    CUtensorMap km, vm;
    memcpy(&km, kv.k_map, sizeof(km));
    memcpy(&vm, kv.v_map, sizeof(vm));
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(C::W * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attn_kernel<HD, TYPE, NT, SINK>, a, km, vm) == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}

template <int TYPE, bool SINK>
static fr_status launch_hd(const KvDesc& kv, const AttnArgs& a, int nt, int ctas, cudaStream_t st) {
    switch (kv.hd) {
        case 64: return nt == 1 ? launch_one<64, TYPE, 1, SINK>(kv, a, ctas, st)
                      : nt == 2 ? launch_one<64, TYPE, 2, SINK>(kv, a, ctas, st) : launch_one<64, TYPE, 4, SINK>(kv, a, ctas, st);
        case 128: return nt == 1 ? launch_one<128, TYPE, 1, SINK>(kv, a, ctas, st)
                       : nt == 2 ? launch_one<128, TYPE, 2, SINK>(kv, a, ctas, st) : launch_one<128, TYPE, 4, SINK>(kv, a, ctas, st);
        default: return nt == 1 ? launch_one<256, TYPE, 1, SINK>(kv, a, ctas, st) : launch_one<256, TYPE, 2, SINK>(kv, a, ctas, st);
    }
}
template <int TYPE>
static fr_status launch_type(const KvDesc& kv, const AttnArgs& a, int nt, int ctas, cudaStream_t st) {
    return a.sink ? launch_hd<TYPE, true>(kv, a, nt, ctas, st) : launch_hd<TYPE, false>(kv, a, nt, ctas, st);
}

}  // namespace paged
}  // namespace fr

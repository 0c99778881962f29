// fr_paged_tc.cu -- attention over pages for many query rows of a sequence and KV
// head (prompts, wide speculative windows): row tiles of up to 128 rows
// on tcgen05.
//
// Beyond a few tens of rows the bound is no longer the bytes of K and V but the
// matrix work: an mma.sync kernel of small row tiles reads the keys again for
// each tile and ends at about 190 TFLOP/s. Here a row tile holds whole tokens
// (128 / G tokens of G heads, so one TMA box is the tile) as the M of
// S = Q K^T and O += P V; S, P and O live in TMEM. One CTA an SM works through
// its share of the list of units (fr_paged_work.cuh) piece by piece:
//   warps 0-7  softmax: a thread owns a row's half of the tile's 64 columns;
//              masks from the row's view, running reference and sum, P as two
//              f16 terms (P_hi + P_lo, 22 bits) back into TMEM. Where a tile
//              holds keys that some row does not see, rows of V that nobody
//              sees, or that hold infinities or NaN, are cleared; the latter are
//              added at the piece's end for the rows that see them.
//   warp 8     producer: page numbers and TMA, K and V in rings of their own; it
//              runs on into the next piece.
//   warp 9     MMA issuer: S of the next tile ahead of PV of this one.
//   10-13      e4m3 only: codes to f16, from the slots that the TMA fills into the
//              MMA's. K's scale joins the score's factor, V's the weights,
//              relative to the largest in the row's view so far (another running
//              reference beside the maximum).
// The roles follow the list each with its own walk and meet only at mbarriers.
// Waits are bounded; one that gives up sets the status word, and the CTA still
// drains its copies and MMAs and frees its TMEM.
//
// Measured: 2048 new tokens at the end of 32768 keys, 32 heads on 8, hd 128, f16: 1.97 ms,
// 540 TFLOP/s (P_lo counted: 810). Four prompts of 2048: 350 us in f16 and 629 us
// in e4m3 (1344 and 1619 us in tiles of 32 rows). A tile takes 1.1 us in f16, a
// chain of S, softmax and PV in which none of the units is busy for more than a
// third; three S tiles in TMEM in place of two were 3-6 % slower up to hd 128.
// e4m3 is bound by the conversion: two warps took 752 us for the four prompts,
// one load at a time 875; the same four with the registers split by warpgroup
// (144 and 112) spilled more and took 657.
#include <string.h>

#include "fr_paged_work.cuh"

namespace fr {
namespace paged {
namespace tc {

using namespace sm100;

constexpr int kBN = 64;                      // keys of a tile
constexpr int kSmax = 256, kProd = 8, kMma = 9, kConv = 10, kConvThreads = 128;   // softmax threads; warps
// Weights are 2^(x - reference): a row's reference is 7 below its maximum when set,
// and moves when a score exceeds it by 15 (P_lo off f16's subnormals, P_hi within f16).
constexpr float kBelow = 7.0f, kAbove = 15.0f;
constexpr uint64_t kLimit = 2000000000ull;

template <int HD, bool E4>
struct Cfg {
    static constexpr int THREADS = E4 ? 448 : 320;
    static constexpr int NB = HD / 64;                        // 128-byte column boxes of f16
    static constexpr int KS = HD == 64 ? 6 : HD == 128 ? 4 : 2;   // K slots, and V slots
    // e4m3: slots of codes, K and V in turn, of RAWR rows each
    static constexpr int RAWR = raw_rows(HD), BOXB = HD < 128 ? HD : 128, RAW_BYTES = RAWR * HD, PARTS = kBN / RAWR;
    static constexpr int RS = !E4 ? 0 : HD == 64 ? 8 : HD == 128 ? 6 : 3;
    static constexpr int Q_BOX = 128 * 128, KV_BOX = kBN * 128, TILE = kBN * HD * 2;
    static constexpr int Q = 0, K = 128 * HD * 2, V = K + KS * TILE, RAW = V + KS * TILE,
                         AUX = RAW + RS * RAW_BYTES;
    // auxiliary area: half-row maxima and sums, walks, scan, tiles' pages, odd rows of V, barriers
    static constexpr int A_MAX = 0, A_L = 2048, A_WALK = A_L + 1024, A_SCAN = A_WALK + 64 * 17, A_META = A_SCAN + 256,
                         A_ODD = A_META + 16 * 64, A_BAR = A_ODD + 528, AUX_BYTES = A_BAR + 512;
    static constexpr int SMEM = AUX + AUX_BYTES + 1024;
    static_assert(SMEM <= 232448, "shared memory");
    // barriers
    static constexpr int B_KF = 0, B_KE = KS, B_VF = 2 * KS, B_VE = 3 * KS, B_SF = 4 * KS, B_PF = B_SF + 2, B_OD = B_SF + 4,
                         B_OF = B_SF + 6, B_QF = B_SF + 7, B_QE = B_SF + 8, B_OE = B_SF + 9, B_END = B_SF + 10,
                         B_RF = B_SF + 11, B_RE = B_RF + RS, N_BAR = B_RE + RS;
    static_assert(N_BAR <= 60, "barriers");
    // TMEM columns: O, two S tiles, two tiles of P_hi and of P_lo words (two keys a column)
    static constexpr int T_O = 0, T_S = HD, T_P = HD + 2 * kBN, T_PL = T_P + kBN;
    static_assert(T_PL + kBN <= 512, "TMEM");
};

struct TcMaps {
    CUtensorMap q, k, v;
};
struct Meta {                                                // a tile's 16-key steps
    float ks[4], vs[4];                                      // e4m3: scales
    int page[4];                                             // -1: none
    uint32_t none;                                           // bit i: step i has none
    int pad[3];
};
struct Pages {                                               // the cache as plain memory (rare rows are read there)
    const void *k, *v;
    int64_t k_page, k_head, k_row, v_page, v_head, v_row;
    int box_rows;                                            // rows of a K or V box (tc_box_rows)
    int tok_tile;                                            // tokens of a row tile
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int row, int chunk, int head, int page,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
        "[%7];"
        :: "r"(dst), "l"((uint64_t)map), "r"(0), "r"(row), "r"(chunk), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ void load_q(uint32_t dst, const CUtensorMap* map, int dim, int head, int tok, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"((uint64_t)map), "r"(dim), "r"(head), "r"(tok), "r"(bar) : "memory");
}
// Does a pair of f16 hold an infinity or NaN?
__device__ __forceinline__ bool odd_half2(uint32_t x) { return (x & 0x7c00u) == 0x7c00u || (x & 0x7c000000u) == 0x7c000000u; }

// Element i of a page.
template <bool E4>
__device__ __forceinline__ float page_value(const void* p, int64_t i) {
    if (!E4) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return __half2float(__ushort_as_half((unsigned short)e4m3_lo(reinterpret_cast<const unsigned char*>(p)[i])));
}

// Keys that a row sees: [lo, hi).
__device__ __forceinline__ int2 row_view(const Seg& s, int row, const AttnArgs& a) {
    int hi = s.n_kv, lo = 0;
    if (a.causal) {
        const int p = s.n_kv - s.n_q + token_of(row, a);
        hi = min(hi, p + 1);
        if (a.window > 0) lo = max(0, p + 1 - a.window);
    }
    return make_int2(lo, hi);
}

template <int HD, bool E4>
__global__ void __launch_bounds__((Cfg<HD, E4>::THREADS), 1)
paged_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ TcMaps mp, const __grid_constant__ Pages pg) {
    using C = Cfg<HD, E4>;
    using P = Units<0, kBN, 1, kTcSegCost>;
    constexpr int KS = C::KS, RS = E4 ? C::RS : 1, HB = kBN / 2, OH = HD / 2;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    unsigned char* aux = sm + C::AUX;
    float* s_max = reinterpret_cast<float*>(aux + C::A_MAX);             // [2][2][128]
    float* s_l = reinterpret_cast<float*>(aux + C::A_L);                 // [2][128]
    Walk* walks = reinterpret_cast<Walk*>(aux + C::A_WALK);              // the share's start, then one for each warp
    int* scan = reinterpret_cast<int*>(aux + C::A_SCAN);
    Meta* s_meta = reinterpret_cast<Meta*>(aux + C::A_META);             // [16]
    // Odd rows of V, two deep: one warp may be a tile, or a piece, ahead of another
    volatile int* s_odd = reinterpret_cast<volatile int*>(aux + C::A_ODD);             // [2][64] tile (+ 1) with an odd row here
    volatile int* s_piece = s_odd + 2 * kBN;                             // [2] piece (+ 1) that met odd rows
    uint64_t* bars = reinterpret_cast<uint64_t*>(aux + C::A_BAR);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 62);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    bool failed = false;                 // after a first wait that gave up, the others do so at once
    auto wait = [&](int b, uint32_t parity) {
        if (mbar_wait(bar(b), parity, failed ? 0ull : kLimit)) return;
        failed = true;
        atomicOr(a.status, kStatusTimeout);
    };

    if (tid == 0) {
        for (int i = 0; i < C::N_BAR; ++i) {
            const bool full = (i >= C::B_KF && i < C::B_KF + KS) || (i >= C::B_VF && i < C::B_VF + KS);
            mbar_init(bar(i), i == C::B_PF || i == C::B_PF + 1 || i == C::B_OE ? kSmax / 32 : (E4 && full) || i >= C::B_RE ? kConvThreads / 32 : 1);
        }
        mbar_fence_init();
        prefetch_tmap(&mp.k);
        prefetch_tmap(&mp.v);
        s_piece[0] = s_piece[1] = 0;
    }
    if (tid < 2 * kBN) s_odd[tid] = 0;
    if (warp == kMma) tmem_alloc(smem_addr(s_tmem), 512);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Share share = first_walk<P, C::THREADS>(a, cta, scan, walks);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *s_tmem;
    const bool work = share.units > 0 && walks[0].more;
    if (work && lane < 16) reinterpret_cast<int*>(walks + 1 + warp)[lane] = reinterpret_cast<const int*>(walks)[lane];
    __syncwarp();
    Walk* w = walks + 1 + warp;
    const int G = a.group;

    if (!work) {
        // nothing of the list
    } else if (warp == kProd) {
        int n = 0, piece = 0, blk = 0, nk = 0, nv = 0, nq = 0, item = 0;     // tiles; pieces; loads
        auto free_slot = [&](int b, uint32_t parity) {
            if (lane == 0) wait(b, parity);
            failed = __shfl_sync(~0u, (int)failed, 0);
        };
        for (;;) {
            const int2 t = walk_tiles<P>(*w, 0);
            const Seg& s = w->s;
            int page = -1;
            bool has = false;
            float ks = 0.f, vs = 0.f;
            auto look_up = [&](int tile) {       // pages of the next 32 16-key steps, one a lane
                const int key = (s.tile0 + tile) * kBN + lane * kTile;
                // (a box is looked up for its first key, also where only its last ones are in view)
                has = key < s.n_kv && (key | (pg.box_rows - 1)) >= s.lo && tile + lane / 4 < t.y;
                page = has ? a.table[s.b * a.table_stride + (key >> a.page_shift)] : -1;
                if (has && (page < 0 || page >= a.n_pages)) {
                    atomicOr(a.status, kStatusInput);
                    page = -1;
                }
                if (E4) {
                    ks = page >= 0 ? a.k_scale[(int64_t)page * a.n_kv_head + s.h] : 0.f;
                    vs = page >= 0 ? a.v_scale[(int64_t)page * a.n_kv_head + s.h] : 0.f;
                }
                blk = 0;
            };
            if (t.x < t.y) look_up(t.x);
            for (int tile = t.x; tile < t.y; ++tile, ++n) {
                if (blk == 8) look_up(tile);
                const int st = n % KS, key = (s.tile0 + tile) * kBN, in_page = (1 << a.page_shift) - 1;
                // (this wait also keeps the tile within 16 of the softmax's)
                if (!E4 && n >= KS) free_slot(C::B_KE + st, ((n / KS) - 1) & 1);
                if (E4 && item >= C::RS) free_slot(C::B_RE + item % RS, ((item / RS) - 1) & 1);
                Meta& m = s_meta[n & 15];
                const unsigned gone = __ballot_sync(~0u, page < 0) >> (blk * 4) & 15u;
                if (lane == 0) m.none = gone;
                if (lane >> 2 == blk) {
                    m.page[lane & 3] = page;
                    if (E4) {
                        m.ks[lane & 3] = ks;
                        m.vs[lane & 3] = vs;
                    }
                }
                ++blk;
                __syncwarp();
                // rows r0 .. r0 + n_rows - 1 of the tile, a box to a lane (page 0 in place of none: masked)
                auto tile_loads = [&](const CUtensorMap* map, uint32_t dst, int b, int r0, int n_rows) {
                    constexpr int PITCH = E4 ? C::BOXB : 128, CH = HD * (E4 ? 1 : 2) / PITCH;
                    if (lane == 0) mbar_expect_tx(bar(b), n_rows * PITCH * CH);
                    __syncwarp();
                    const int c = lane % CH, r = lane / CH * pg.box_rows;
                    if (r < n_rows)
                        load_box(dst + (c * n_rows + r) * PITCH, map, (key + r0 + r) & in_page, c, s.h,
                                 max(m.page[(r0 + r) >> 4], 0), bar(b));
                };
                auto code_loads = [&](const CUtensorMap* map, bool waited) {
#pragma unroll 1
                    for (int part = 0; part < C::PARTS; ++part) {
                        const int rs = item % RS;
                        if (item >= C::RS && !(waited && part == 0)) free_slot(C::B_RE + rs, ((item / RS) - 1) & 1);
                        if (failed) return;
                        tile_loads(map, smem_addr(sm + C::RAW + rs * C::RAW_BYTES), C::B_RF + rs, part * C::RAWR, C::RAWR);
                        ++item;
                    }
                };
                // (after a wait that gave up nothing more is loaded)
                if (E4) {
                    if (!failed) code_loads(&mp.k, true);
                } else if (!failed) {
                    tile_loads(&mp.k, smem_addr(sm + C::K + st * C::TILE), C::B_KF + st, 0, kBN);
                    ++nk;
                }
                if (tile == t.x) {
                    if (piece > 0) free_slot(C::B_QE, (piece - 1) & 1);
                    if (!failed) {
                        if (lane == 0) mbar_expect_tx(bar(C::B_QF), C::NB * 128 * G * pg.tok_tile);
                        __syncwarp();
                        if (lane < C::NB)
                            load_q(smem_addr(sm + C::Q + lane * C::Q_BOX), &mp.q, lane * 64, s.h * G,
                                   s.tok0 + s.rt * pg.tok_tile, bar(C::B_QF));
                        ++nq;
                    }
                }
                if (!E4 && n >= KS) free_slot(C::B_VE + st, ((n / KS) - 1) & 1);
                if (E4) {
                    if (!failed) code_loads(&mp.v, false);
                } else if (!failed) {
                    tile_loads(&mp.v, smem_addr(sm + C::V + st * C::TILE), C::B_VF + st, 0, kBN);
                    ++nv;
                }
            }
            if (t.x < t.y) ++piece;
            __syncwarp();
            if (lane == 0) walk_on<P>(w, w, &a);
            __syncwarp();
            if (!w->more) break;
        }
        if (lane == 0) {                         // every load has landed before the CTA ends
            for (int i = max(0, item - C::RS); i < item; ++i)
                if (!mbar_wait(bar(C::B_RF + i % RS), (i / RS) & 1, kLimit))
                    atomicOr(a.status, kStatusTimeout);
            for (int i = max(0, nk - KS); i < nk; ++i)
                if (!mbar_wait(bar(C::B_KF + i % KS), (i / KS) & 1, kLimit)) atomicOr(a.status, kStatusTimeout);
            for (int i = max(0, nv - KS); i < nv; ++i)
                if (!mbar_wait(bar(C::B_VF + i % KS), (i / KS) & 1, kLimit)) atomicOr(a.status, kStatusTimeout);
            if (nq > 0 && !mbar_wait(bar(C::B_QF), (nq - 1) & 1, kLimit)) atomicOr(a.status, kStatusTimeout);
        }
    } else if (warp == kMma) {
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_f16_f32(128, kBN, 0, 0), id_o = idesc_f16_f32(128, HD, 0, 1);
            const uint32_t q_base = smem_addr(sm + C::Q);
            auto issue_s = [&](int n) {
                const int st = n % KS;
                wait(C::B_KF + st, (n / KS) & 1);
                tc_fence_after();
                const uint32_t k_base = smem_addr(sm + C::K + st * C::TILE), d = tbase + C::T_S + (n & 1) * kBN;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    mma_ss(d, sdesc_sw128(q_base + (kk >> 2) * C::Q_BOX + (kk & 3) * 32, 16, 1024),
                           sdesc_sw128(k_base + (kk >> 2) * C::KV_BOX + (kk & 3) * 32, 16, 1024), id_s, kk > 0);
                mma_commit(bar(C::B_SF + (n & 1)));
                mma_commit(bar(C::B_KE + st));
            };
            int n = 0, piece = 0;
            for (;;) {
                const int2 t = walk_tiles<P>(*w, 0);
                const int cnt = t.y - t.x;
                if (cnt > 0) {
                    wait(C::B_QF, piece & 1);
                    tc_fence_after();
                    issue_s(n);
                    if (cnt == 1) mma_commit(bar(C::B_QE));
                    for (int i = 0; i < cnt; ++i) {
                        if (i + 1 < cnt) {
                            issue_s(n + i + 1);
                            if (i + 2 == cnt) mma_commit(bar(C::B_QE));      // Q may be overwritten
                        }
                        if (i == 0 && piece > 0) wait(C::B_OE, (piece - 1) & 1);   // the last piece's O is read
                        const int m = n + i, st = m % KS;
                        wait(C::B_PF + (m & 1), (m >> 1) & 1);
                        wait(C::B_VF + st, (m / KS) & 1);
                        tc_fence_after();
                        const uint32_t v_base = smem_addr(sm + C::V + st * C::TILE);
#pragma unroll
                        for (int ks = 0; ks < kBN / 16; ++ks) {
                            // P words: [buffer][half of the keys][16 columns]
                            const uint32_t col = (m & 1) * HB + ks * 8;
                            const uint64_t vd = sdesc_sw128(v_base + ks * 2048, C::KV_BOX, 1024);
                            mma_ts(tbase + C::T_O, tbase + C::T_P + col, vd, id_o, i > 0 || ks > 0 ? 1u : 0u);
                            mma_ts(tbase + C::T_O, tbase + C::T_PL + col, vd, id_o, 1u);
                        }
                        mma_commit(bar(C::B_OD + (m & 1)));
                        mma_commit(bar(C::B_VE + st));
                    }
                    mma_commit(bar(C::B_OF));
                    n += cnt;
                    ++piece;
                }
                walk_on<P>(w, w, &a);
                if (!w->more) break;
            }
            mma_commit(bar(C::B_END));
            if (!mbar_wait(bar(C::B_END), 0, kLimit)) atomicOr(a.status, kStatusTimeout);
        }
    } else if (E4 && warp >= kConv) {
        // codes to f16, which is exact: 16 of a row at a time, into the 128-byte swizzle of the MMA's operands
        const int ct = tid - kConv * 32;
        int n = 0, item = 0;
        auto convert = [&](unsigned char* ring, int b_full, int b_empty) {
            const int st = n % KS;
            if (n >= KS) wait(b_empty + st, ((n / KS) - 1) & 1);
            unsigned char* dst = ring + st * C::TILE;
#pragma unroll 1
            for (int part = 0; part < C::PARTS; ++part, ++item) {
                constexpr int PER_ROW = C::BOXB / 16;
                const int rs = item % RS;
                wait(C::B_RF + rs, (item / RS) & 1);
                const unsigned char* src = sm + C::RAW + rs * C::RAW_BYTES;
                constexpr int N = C::RAW_BYTES / 16 / kConvThreads;
                uint4 zs[N];                          // (all loads ahead of the stores)
#pragma unroll
                for (int u = 0; u < N; ++u) zs[u] = *reinterpret_cast<const uint4*>(src + (ct + u * kConvThreads) * 16);
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    const uint4 z = zs[u];
                    const int i = ct + u * kConvThreads;
                    const int row = part * C::RAWR + i / PER_ROW % C::RAWR;
                    const int d = i / (PER_ROW * C::RAWR) * C::BOXB + i % PER_ROW * 16;
                    const uint4 lo = make_uint4(e4m3_lo(z.x), e4m3_hi(z.x), e4m3_lo(z.y), e4m3_hi(z.y));
                    const uint4 hi = make_uint4(e4m3_lo(z.z), e4m3_hi(z.z), e4m3_lo(z.w), e4m3_hi(z.w));
                    unsigned char* to = dst + (d >> 6) * C::KV_BOX + row * 128;
                    const int c = d >> 3 & 7, odd = d >> 6 & 1;      // (of a row's two boxes one starts with its odd chunks: other banks)
                    *reinterpret_cast<uint4*>(to + (((c + odd) ^ (row & 7)) << 4)) = odd ? hi : lo;
                    *reinterpret_cast<uint4*>(to + (((c + 1 - odd) ^ (row & 7)) << 4)) = odd ? lo : hi;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_RE + rs));
            }
            fence_proxy_async_cta();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b_full + st));
        };
        for (;;) {
            const int2 t = walk_tiles<P>(*w, 0);
            for (int tile = t.x; tile < t.y; ++tile, ++n) {
                convert(sm + C::K, C::B_KF, C::B_KE);
                convert(sm + C::V, C::B_VF, C::B_VE);
            }
            __syncwarp();
            if (lane == 0) walk_on<P>(w, w, &a);
            __syncwarp();
            if (!w->more) break;
        }
    } else {
        const int qd = warp & 3, half = warp >> 2, r = qd * 32 + lane, c_base = half * HB;
        const uint32_t lanes = (uint32_t)(qd * 32) << 16;
        int n = 0, piece = 0;
        for (;;) {
            const int2 t = walk_tiles<P>(*w, 0);
            const Seg& s = w->s;
            const int row0 = s.rt * a.row_tile, rows = min(a.row_tile, s.n_q * G - row0);
            const int2 first = row_view(s, row0, a), end = row_view(s, row0 + rows - 1, a);
            const int2 view = r < rows ? row_view(s, row0 + r, a) : make_int2(0, 0);
            const bool active = qd * 32 < rows;
            if (tid == 0) put_split(a, share, cta, *w, row0, rows);
            float m_ref = -INFINITY, l = 0.f, v_ref = 0.f;
            for (int tile = t.x; tile < t.y; ++tile, ++n) {
                wait(C::B_SF + (n & 1), (n >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                const int key0 = (s.tile0 + tile) * kBN;
                const Meta& m = s_meta[n & 15];
                const uint32_t none = m.none;
                const bool edge = none || key0 + kBN > first.y || key0 < end.x;
                float v_max = 0.f, v_step[2] = {1.f, 1.f};        // e4m3: V's scales, of the steps that the row sees
                if (E4) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = key0 + i * kTile;
                        const float v = edge && (j >= view.y || j + kTile <= view.x || (none >> i & 1u)) ? 0.f : m.vs[i];
                        v_max = fmaxf(v_max, fabsf(v));
                        if (i >> 1 == half) v_step[i & 1] = v;
                    }
                }
                float x[HB], pm = -INFINITY;
                if (active) {
                    tmem_ld_x32(tbase + lanes + C::T_S + (n & 1) * kBN + c_base, reinterpret_cast<uint32_t*>(x));
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < HB; ++c) x[c] = __fmul_rn(x[c], E4 ? a.scale_log2 * m.ks[half * 2 + c / 16] : a.scale_log2);
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < HB; ++c) {
                            const int j = key0 + c_base + c;
                            if (j < view.x || j >= view.y || (none >> ((c_base + c) >> 4) & 1u)) x[c] = -INFINITY;
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < HB; ++c) m4[c & 3] = fmaxf(m4[c & 3], x[c]);
                    // (rows behind the tile's last hold anything and are not read: only their reference stays still)
                    if (r < rows) pm = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                }
                s_max[((n & 1) * 2 + half) * 128 + r] = pm;
                asm volatile("bar.sync %0, 64;" :: "r"(qd + 1) : "memory");          // the row's two halves
                const float mx = fmaxf(pm, s_max[((n & 1) * 2 + (half ^ 1)) * 128 + r]);
                float m_new = m_ref;
                if (mx - m_ref > kAbove) m_new = fmaxf(mx - kBelow, m_ref);              // (m_ref = -inf: any score)
                const bool grown = m_ref != -INFINITY && m_new != m_ref;
                const float alpha = grown ? ex2(m_ref - m_new) : 1.f;
                // V's scales join the weights relative to the largest that the row has met
                float o_scale = alpha;
                const bool v_up = E4 && v_max > v_ref;
                if (v_up) {
                    const float v = fmaxf(v_max, 0x1p-120f);         // its reciprocal stays finite
                    o_scale *= v_ref / v;
                    v_ref = v;
                }
                if (E4) {
                    const float v_inv = v_ref > 0.f ? 1.f / v_ref : 0.f;
                    v_step[0] *= v_inv;
                    v_step[1] *= v_inv;
                }
                if (active) {
                    if (__any_sync(~0u, grown || v_up) && tile > t.x) {
                        wait(C::B_OD + ((n - 1) & 1), ((n - 1) >> 1) & 1);           // O holds PV up to the tile before
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < OH; c += 32) {
                            uint32_t o[32];
                            tmem_ld_x32(tbase + lanes + C::T_O + half * OH + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * o_scale);
                            tmem_st_x32(tbase + lanes + C::T_O + half * OH + c, o);
                        }
                        tmem_wait_st();
                    }
                    const float sub = m_new == -INFINITY ? 0.f : m_new;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int c = 0; c < HB; c += 2) {
                        float p0 = ex2(__fsub_rn(x[c], sub)), p1 = ex2(__fsub_rn(x[c + 1], sub));
                        s4[(c >> 1) & 3] += p0 + p1;
                        if (E4) {
                            p0 *= v_step[c / 16];
                            p1 *= v_step[c / 16];
                        }
                        hi[c / 2] = pack_half2(p0, p1);
                        const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi[c / 2]));
                        lo[c / 2] = pack_half2(p0 - hf.x, p1 - hf.y);
                    }
                    tmem_st_x16(tbase + lanes + C::T_P + (n & 1) * HB + half * 16, hi);
                    tmem_st_x16(tbase + lanes + C::T_PL + (n & 1) * HB + half * 16, lo);
                    l = fmaf(l, alpha, (s4[0] + s4[1]) + (s4[2] + s4[3]));
                    tmem_wait_st();
                }
                m_ref = m_new;
                if (edge) {
                    // V's rows that nobody sees, and odd ones seen by some only (0 * inf and 0 * NaN are NaN)
                    wait(C::B_VF + n % KS, (n / KS) & 1);
                    unsigned char* v = sm + C::V + n % KS * C::TILE;
                    auto at = [&](int i) { return reinterpret_cast<uint4*>(v + (i >> 9) * C::KV_BOX + (i & 511) * 16); };
                    auto dead = [&](int j) { return key0 + j >= end.y || key0 + j < first.x || (none >> (j >> 4) & 1u); };
                    for (int i = tid; i < kBN * HD / 8; i += kSmax) {
                        const int j = (i & 511) >> 3;
                        if (dead(j) || (key0 + j < first.y && key0 + j >= end.x)) continue;
                        const uint4 z = *at(i);
                        if (odd_half2(z.x) || odd_half2(z.y) || odd_half2(z.z) || odd_half2(z.w)) {
                            s_odd[(n & 1) * kBN + j] = n + 1;
                            s_piece[piece & 1] = piece + 1;
                        }
                    }
                    asm volatile("bar.sync 5, 256;" ::: "memory");
                    for (int i = tid; i < kBN * HD / 8; i += kSmax) {
                        const int j = (i & 511) >> 3;
                        if (dead(j) || s_odd[(n & 1) * kBN + j] == n + 1) *at(i) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_cta();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_PF + (n & 1)));     // (256 arrivals on one barrier would queue)
            }
            // ---- the piece's end ------------------------------------------------
            const bool any = t.x < t.y;
            if (any) {
                wait(C::B_OF, piece & 1);
                __syncwarp();
                tc_fence_after();
            }
            s_l[half * 128 + r] = l;
            asm volatile("bar.sync %0, 64;" :: "r"(qd + 1) : "memory");
            l += s_l[(half ^ 1) * 128 + r];
            asm volatile("bar.sync %0, 64;" :: "r"(qd + 1) : "memory");              // (read before the next piece writes it)
            const bool whole = w->ua == 0 && w->ub == s.n_units;
            const int part = 2 * cta + (w->ua == 0 && !whole ? 1 : 0);
            const float m_out = l == 0.f ? -INFINITY : m_ref == -INFINITY ? 0.f : m_ref;
            const float f = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f, f_v = E4 ? v_ref : 1.f;
            const int tok = token_of(row0 + min(r, rows - 1), a), hh = row0 + min(r, rows - 1) - tok * G;
            float* dst = whole ? a.out + ((int64_t)(s.tok0 + tok) * a.n_kv_head * G + s.h * G + hh) * HD
                               : a.part_o + ((int64_t)part * 128 + r) * HD;
            const bool odd = any && s_piece[piece & 1] == piece + 1;
            if (active) {
#pragma unroll 1
                for (int c = 0; c < OH; c += 32) {
                    float o[32];
                    if (any) {
                        tmem_ld_x32(tbase + lanes + C::T_O + half * OH + c, reinterpret_cast<uint32_t*>(o));
                        tmem_wait_ld();
                    }
                    if (r < rows) {
                        if (!any || l == 0.f) {
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] = 0.f;
                        } else if (odd) {
                            // the cleared rows that this row sees: one by one, from memory
                            const __half* q = a.q16 + (int64_t)(s.tok0 + tok) * a.q_stride + (int64_t)(s.h * G + hh) * HD;
                            const int from = max(view.x, (s.tile0 + t.x) * kBN), to = min(view.y, (s.tile0 + t.y) * kBN);
                            for (int j = from; j < to; ++j) {
                                const int j0 = j / kBN * kBN;              // (only tiles with keys that some row does not see were cleared)
                                if (!(j0 + kBN > first.y || j0 < end.x) || (j >= end.x && j < first.y)) continue;
                                const int page = a.table[s.b * a.table_stride + (j >> a.page_shift)];
                                if (page < 0 || page >= a.n_pages) continue;
                                const int in = j & ((1 << a.page_shift) - 1);
                                const int64_t k = page * pg.k_page + s.h * pg.k_head + in * pg.k_row;
                                const int64_t v = page * pg.v_page + s.h * pg.v_head + in * pg.v_row;
                                bool bad = false;
                                for (int d = 0; d < HD; ++d) bad |= !isfinite(page_value<E4>(pg.v, v + d));
                                if (!bad) continue;
                                float x = 0.f;
                                for (int d = 0; d < HD; ++d) x = fmaf(__half2float(q[d]), page_value<E4>(pg.k, k + d), x);
                                const int64_t sc = (int64_t)page * a.n_kv_head + s.h;
                                const float x_log2 = __fmul_rn(x, E4 ? a.scale_log2 * a.k_scale[sc] : a.scale_log2);
                                const float p = ex2(__fsub_rn(x_log2, m_out)) *
                                                (E4 ? (v_ref > 0.f ? a.v_scale[sc] * (1.f / v_ref) : 0.f) : 1.f);
#pragma unroll
                                for (int u = 0; u < 32; ++u) o[u] = fmaf(p, page_value<E4>(pg.v, v + half * OH + c + u), o[u]);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 32; u += 4)
                            *reinterpret_cast<float4*>(dst + half * OH + c + u) =
                                make_float4(o[u] * f_v * f, o[u + 1] * f_v * f, o[u + 2] * f_v * f, o[u + 3] * f_v * f);
                    }
                    __syncwarp();
                }
                if (!whole && half == 0 && r < rows) a.part_ml[part * 128 + r] = make_float2(m_out, l);
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_OE));
                ++piece;
            }
            __syncwarp();
            if (lane == 0) walk_on<P>(w, w, &a);
            __syncwarp();
            if (!w->more) break;
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == kMma) tmem_dealloc(tbase, 512);
}

template <int HD, bool E4>
static fr_status launch(const KvDesc& kv, const AttnArgs& a, int ctas, cudaStream_t st) {
    using C = Cfg<HD, E4>;
    static unsigned long long done = 0ull;           // devices whose shared-memory limit is raised
    if (kv.dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> kv.dev & 1ull)) {
        if (cudaFuncSetAttribute(paged_tc_kernel<HD, E4>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
            cudaSuccess)
            return FR_ERR_CUDA;
        if (kv.dev < 64) __atomic_fetch_or(&done, 1ull << kv.dev, __ATOMIC_RELEASE);
    }
    auto enc = get_encoder();
    if (!enc) return FR_ERR_CUDA;
    TcMaps mp;
    memset(&mp, 0, sizeof(mp));
    memcpy(&mp.k, kv.k_map_tc, sizeof(mp.k));
    memcpy(&mp.v, kv.v_map_tc, sizeof(mp.v));
    // Q rows of whole tokens, in the order of a row tile: 64 dims x G heads x tokens
    const int tok_tile = a.row_tile / a.group;
    cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)a.n_kv_head * a.group, (cuuint64_t)a.n_tok};
    // (the stride of a size-1 dimension is never used, but has to be valid)
    cuuint64_t strides[2] = {(cuuint64_t)HD * 2, a.n_tok > 1 ? (cuuint64_t)a.q_stride * 2 : dims[1] * HD * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)tok_tile}, es[3] = {1, 1, 1};
    if (enc(&mp.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(a.q16), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return FR_ERR_CUDA;
    const Pages pg{kv.k, kv.v, kv.k_page, kv.k_head, kv.k_row, kv.v_page, kv.v_head, kv.v_row,
                   tc_box_rows(kv.page_size, HD, E4), tok_tile};
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_tc_kernel<HD, E4>, a, mp, pg) == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}

}  // namespace tc

fr_status launch_attn_tc(const KvDesc& kv, const AttnArgs& a, int ctas, cudaStream_t st) {
    if (kv.type == FR_KV_E4M3)
        return kv.hd == 64    ? tc::launch<64, true>(kv, a, ctas, st)
               : kv.hd == 128 ? tc::launch<128, true>(kv, a, ctas, st)
                              : tc::launch<256, true>(kv, a, ctas, st);
    return kv.hd == 64    ? tc::launch<64, false>(kv, a, ctas, st)
           : kv.hd == 128 ? tc::launch<128, false>(kv, a, ctas, st)
                          : tc::launch<256, false>(kv, a, ctas, st);
}

}  // namespace paged
}  // namespace fr

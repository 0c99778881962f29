// fr_paged_work.cuh -- the list of work that the paged attention kernels share
// out: the keys of all (sequence, KV head, row tile) segments as units, counted
// from the lengths on the device, and a CTA's walk over its part of them.
#pragma once

#include "fr_paged.h"
#include "fr_sm100.cuh"

namespace fr {
namespace paged {

// Two e4m3 codes (the low or the high half of x) as f16x2, exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
    uint32_t y;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, a; }" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
    uint32_t y;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, b; }" : "=r"(y) : "r"(x));
    return y;
}

// Row r's token: r / group, by a multiplication where the host found it exact.
__device__ __forceinline__ int token_of(int r, const AttnArgs& a) {
    return a.group_magic ? (int)__umulhi((unsigned)r, a.group_magic) : r / a.group;
}

// A kernel's units: RT rows of a row tile (0: as the launch says), tiles of KT
// keys, W of them (one for each warp) a unit, SEG more units for a segment.
template <int RT_, int KT_, int W_, int SEG_>
struct Units {
    static constexpr int KT = KT_, W = W_, SEG = SEG_;
    __device__ static __forceinline__ int rows(const AttnArgs& a) { return RT_ ? RT_ : a.row_tile; }
};

// One (sequence, KV head, row tile): its rows, and its keys as tiles.
struct Seg {
    int b, h, rt, n_rt;
    int tok0, n_q, n_kv;
    int tile0, n_tiles, n_units;
    int lo;             // first key in some row's view
};

template <class P>
__device__ __forceinline__ void seg_keys(Seg& s, const AttnArgs& a) {
    int hi = s.n_kv, lo = 0;
    if (a.causal) {
        // the tile's first and last token; one row tile holds all of most sequences
        const int i0 = s.rt == 0 ? 0 : token_of(s.rt * P::rows(a), a);
        const int i1 = s.rt == s.n_rt - 1 ? s.n_q - 1 : token_of((s.rt + 1) * P::rows(a) - 1, a);
        const int first = s.n_kv - s.n_q;
        hi = min(hi, first + i1 + 1);
        if (a.window > 0) lo = max(0, first + i0 - a.window + 1);
    }
    s.lo = lo;
    s.tile0 = lo / P::KT;
    s.n_tiles = hi > lo ? (hi + P::KT - 1) / P::KT - s.tile0 : 0;
    // a segment's start and end cost a CTA as much as some units of its keys: it
    // counts those ahead of them (rows without keys still get their zeros)
    s.n_units = P::SEG + (s.n_tiles + P::W - 1) / P::W;
}
template <class P>
__device__ __forceinline__ bool seg_seq(Seg& s, const AttnArgs& a, int b) {
    const SeqInfo q = seq_info(a.tok_start, a.kv_len, b, a.n_tok, a.max_pages, a.page_shift);
    s.b = b;
    s.tok0 = q.tok0;
    s.n_q = q.n_q;
    s.n_kv = q.n_kv;
    s.n_rt = (q.n_q * a.group + P::rows(a) - 1) / P::rows(a);
    return q.bad;
}
// The next segment in order (row tile fastest, then KV head, then sequence).
template <class P>
__device__ __forceinline__ void seg_next(Seg& s, const AttnArgs& a) {
    if (++s.rt == s.n_rt) {
        s.rt = 0;
        if (++s.h == a.n_kv_head) {
            s.h = 0;
            int b = s.b;
            do {
                if (++b >= a.n_seq) return;
                seg_seq<P>(s, a, b);
            } while (s.n_rt == 0);
        }
    }
    seg_keys<P>(s, a);
}
// Units of all segments of one KV head of each lane's sequence (0 without rows).
// Called by whole warps: a sequence of many row tiles is counted by all lanes.
constexpr int kSerialTiles = 4;
template <class P>
__device__ __forceinline__ int seq_units(const AttnArgs& a, const Seg& s) {
    int u = 0;
    Seg x = s;
    if (s.n_rt <= kSerialTiles)
        for (x.rt = 0; x.rt < s.n_rt; ++x.rt) {
            seg_keys<P>(x, a);
            u += x.n_units;
        }
    for (unsigned big = __ballot_sync(~0u, s.n_rt > kSerialTiles); big; big &= big - 1) {
        const int from = __ffs(big) - 1, lane = threadIdx.x & 31;
        x.n_q = __shfl_sync(~0u, s.n_q, from);
        x.n_kv = __shfl_sync(~0u, s.n_kv, from);
        x.n_rt = __shfl_sync(~0u, s.n_rt, from);
        int sum = 0;
        for (x.rt = lane; x.rt < x.n_rt; x.rt += 32) {
            seg_keys<P>(x, a);
            sum += x.n_units;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == from) u = sum;
    }
    return u;
}
// Called by a whole warp with one sequence's numbers: the row tile that holds unit
// rem of its list, and rem within it.
template <class P>
__device__ __noinline__ int2 find_row_tile(Seg x, int rem, const AttnArgs* a) {
    const int lane = threadIdx.x & 31;
    for (int rt0 = 0;; rt0 += 32) {
        x.rt = rt0 + lane;
        if (x.rt < x.n_rt) seg_keys<P>(x, *a);
        const int own = x.rt < x.n_rt ? x.n_units : 0;
        int inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(~0u, rem < inc);
        if (hit || rt0 + 32 >= x.n_rt) {
            const int at = hit ? __ffs(hit) - 1 : 0;
            return make_int2(rt0 + at, rem - __shfl_sync(~0u, inc - own, at));
        }
        rem -= __shfl_sync(~0u, inc, 31);
    }
}

// A walk over a CTA's share of the units: the piece of a segment it is at. In
// shared memory: one for the CTA, two pieces deep, and one for each warp's
// requests, which run ahead.
struct Walk {
    Seg s;
    int left;           // units of the share from this piece on
    int ua, ub;         // this piece's units within the segment
    int more;           // 0: the share has ended
    int seg_no;         // the segment's number in the whole list
};
static_assert(sizeof(Walk) == 64, "walk");
template <class P>
__device__ __forceinline__ int2 walk_tiles(const Walk& w, int warp) {
    return make_int2(max(w.ua - P::SEG, 0) * P::W + warp, min(max(w.ub - P::SEG, 0) * P::W, w.s.n_tiles));
}
template <class P>
__device__ __forceinline__ void walk_on(const Walk* from, Walk* to, const AttnArgs* a) {
    Walk v = *from;
    v.left -= v.ub - v.ua;
    v.more = v.left > 0;
    if (v.more) {
        seg_next<P>(v.s, *a);
        ++v.seg_no;
        v.ua = 0;
        v.ub = min(v.s.n_units, v.left);
    }
    *to = v;
}
// What happens once a piece stays out of line: the loop over tiles is what the
// instruction cache has to hold.
template <class P>
__device__ __noinline__ void walk_next(const Walk* from, Walk* to, const AttnArgs* a) {
    walk_on<P>(from, to, a);
}
// The warp's requests go on to its next piece with tiles: {next tile, end}, {0, 0} at the share's end.
template <class P>
__device__ __noinline__ int2 request_next(Walk* w, const AttnArgs* a, int warp) {
    for (;;) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) walk_next<P>(w, w, a);
        __syncwarp();
        if (!w->more) return make_int2(0, 0);
        const int2 t = walk_tiles<P>(*w, warp);
        if (t.x < t.y) return t;
    }
}
// A CTA's share of the list: its first unit, units (0: none), and the totals.
struct Share {
    int u0, units, total, n_cta;
};
// Do the sequences have more tokens than the step has rows? (Only ranges that are not in
// order can: the backward ones among them are skipped, the others overlap.) Called by
// the whole block. Their units may then be more than an int counts.
template <int NTH>
__device__ __noinline__ bool ranges_overlap(const AttnArgs* a, int* scan) {
    const int tid = threadIdx.x, most = a->n_tok + 1;              // (enough to tell, and 1024 of them fit)
    int n = 0;
    for (int b = tid; b < a->n_seq; b += NTH)
        n = min(n + seq_info(a->tok_start, a->kv_len, b, a->n_tok, a->max_pages, a->page_shift).n_q, most);
    n = __reduce_add_sync(~0u, n);
    __syncthreads();                                               // (scan[] has been read)
    if ((tid & 31) == 0) scan[tid >> 5] = n;
    __syncthreads();
    int64_t sum = 0;
    for (int w = 0; w < NTH / 32; ++w) sum += scan[w];
    return sum > a->n_tok;
}
// The share of CTA `cta`, and the walk's first piece in cws[0] (more = 0: none),
// which a barrier of the block has yet to publish. scan: 4 * NTH / 32 words.
template <class P, int NTH>
__device__ __forceinline__ Share first_walk(const AttnArgs& a, int cta, int* scan, Walk* cws) {
    // (a thread for each of the first NTH sequences keeps what it reads)
    constexpr int NW = NTH / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Share sh{0, 0, 0, 0};
    Seg seq;
    int per_head = 0, u_b = 0, s_b = 0, more_u = 0, more_s = 0;   // of this thread's sequence; of those behind
    bool bad_any = false;
    {
        seq.n_rt = 0;
        if (tid < a.n_seq) bad_any = seg_seq<P>(seq, a, tid);
        per_head = seq_units<P>(a, seq);
        u_b = per_head * a.n_kv_head;
        s_b = seq.n_rt * a.n_kv_head;
        for (int b0 = NTH; b0 < a.n_seq; b0 += NTH) {
            Seg s;
            s.n_rt = 0;
            if (b0 + tid < a.n_seq) bad_any |= seg_seq<P>(s, a, b0 + tid);
            more_u += seq_units<P>(a, s) * a.n_kv_head;
            more_s += s.n_rt * a.n_kv_head;
        }
        if (bad_any && cta == 0) atomicOr(a.status, kStatusInput);
    }
    auto scan_warp = [&](int& u, int& n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, u, o), y = __shfl_up_sync(~0u, n, o);
            if (lane >= o) {
                u += x;
                n += y;
            }
        }
    };
    int inc = u_b, inc_s = s_b;
    scan_warp(inc, inc_s);
    if (a.n_seq > NTH) scan_warp(more_u, more_s);
    // (segments have two units and more each, so that their counts leave a bit for bad input)
    const int bad_bit = __any_sync(~0u, bad_any) ? 1 << 30 : 0;
    if (lane == 31) {
        scan[warp] = inc;
        scan[NW + warp] = (inc_s & ((1 << 30) - 1)) | bad_bit;
        scan[2 * NW + warp] = more_u;
        scan[3 * NW + warp] = more_s;
    }
    if (tid == 0) cws[0].more = 0;
    __syncthreads();
    int base_u = 0, base_s = 0, total = 0, segs = 0, some_bad = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int n = scan[NW + w] & ((1 << 30) - 1);
        some_bad |= scan[NW + w];
        if (w < warp) {
            inc += scan[w];
            inc_s += n;
        }
        base_u += scan[w];
        base_s += n;
        total += scan[2 * NW + w];
        segs += scan[3 * NW + w];
    }
    total += base_u;             // (the host refuses batches whose ranges in order could pass 31 bits)
    segs += base_s;
    if (__builtin_expect(some_bad >> 30, 0) && ranges_overlap<NTH>(&a, scan)) {
        if (cta == 0 && tid == 0) *a.n_split = 0;
        return sh;
    }
    const int n_cta = min((int)gridDim.x, total);
    if (cta == 0 && tid == 0)    // entries of split[] that this call writes
        *a.n_split = a.split_by_segment ? min(kMaxCtas, segs) : n_cta;
    if (cta >= n_cta) return sh;
    // shares [floor(total i / n_cta), floor(total (i + 1) / n_cta)): segments of one
    // length are cut alike, at their ends where the numbers allow
    const int per_cta = total / n_cta, extra = total - per_cta * n_cta;
    auto share = [&](int i) { return per_cta * i + extra * i / n_cta; };
    const int u0 = share(cta), my_units = share(cta + 1) - u0;
    sh = Share{u0, my_units, total, n_cta};
    {
        int b = tid;
        for (;;) {
            const bool hit = u_b > 0 && u0 >= inc - u_b && u0 < inc;   // one thread of the block: the share starts in its sequence
            int rem = u0 - (inc - u_b), head = 0, tile = 0;
            if (hit) {
                head = a.n_kv_head == 1 ? 0 : rem / per_head;
                rem -= head * per_head;
            }
            if (const unsigned many = __ballot_sync(~0u, hit && seq.n_rt > kSerialTiles)) {
                const int from = __ffs(many) - 1;
                Seg x;
                x.n_q = __shfl_sync(~0u, seq.n_q, from);
                x.n_kv = __shfl_sync(~0u, seq.n_kv, from);
                x.n_rt = __shfl_sync(~0u, seq.n_rt, from);
                const int2 at = find_row_tile<P>(x, __shfl_sync(~0u, rem, from), &a);
                if (lane == from) {
                    tile = at.x;
                    rem = at.y;
                }
            }
            if (hit) {
                Walk w;
                w.s = seq;
                w.s.h = head;
                for (w.s.rt = tile;; ++w.s.rt) {
                    seg_keys<P>(w.s, a);
                    if (rem < w.s.n_units || w.s.rt + 1 >= w.s.n_rt) break;
                    rem -= w.s.n_units;
                }
                w.seg_no = inc_s - s_b + w.s.h * w.s.n_rt + w.s.rt;
                w.ua = rem;
                w.left = my_units;
                w.ub = min(w.s.n_units, w.ua + w.left);
                w.more = w.s.n_rt > 0;
                cws[0] = w;
            }
            if (u0 < base_u || b - tid >= a.n_seq) break;
            // the next NTH sequences
            b += NTH;
            seq.n_rt = 0;
            if (b < a.n_seq) seg_seq<P>(seq, a, b);
            per_head = seq_units<P>(a, seq);
            u_b = per_head * a.n_kv_head;
            s_b = seq.n_rt * a.n_kv_head;
            inc = u_b;
            inc_s = s_b;
            scan_warp(inc, inc_s);
            __syncthreads();
            if (lane == 31) {
                scan[warp] = inc;
                scan[NW + warp] = inc_s;
            }
            __syncthreads();
            inc += base_u;
            inc_s += base_s;
            for (int w = 0; w < NW; ++w) {
                if (w < warp) {
                    inc += scan[w];
                    inc_s += scan[NW + w];
                }
                base_u += scan[w];
                base_s += scan[NW + w];
            }
        }
    }
    return sh;
}
// The merge kernel's entry for the piece that w is at: who holds states of its
// segment. Written by one thread a piece.
__device__ __forceinline__ void put_split(const AttnArgs& a, const Share& sh, int cta, const Walk& w, int row0, int rows) {
    const bool starts = w.ua == 0, whole = starts && w.ub == w.s.n_units, last_piece = w.left <= w.ub - w.ua;
    Split sp{cta, -1, w.s.tok0, row0, rows, w.s.h, {0, 0}};
    if (starts && !whole) {
        // the CTA whose share holds its last unit x: the largest c whose first unit is <= x
        const int x = sh.u0 + sh.units - w.left + w.s.n_units - 1;
        sp.last = min(sh.n_cta - 1, (int)((((int64_t)x + 1) * sh.n_cta - 1) / sh.total));
    }
    const int at = a.split_by_segment ? w.seg_no : cta;
    if ((a.split_by_segment ? starts : last_piece) && at < kMaxCtas) a.split[at] = sp;
}

}  // namespace paged
}  // namespace fr

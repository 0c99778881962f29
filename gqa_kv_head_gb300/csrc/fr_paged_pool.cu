// fr_paged_pool.cu -- the bookkeeping of a paged cache's pages on the device: sequences
// that share the pages of a prefix (fork), pages for a step's new rows (reserve),
// pages given back (free, trim), a pool moved together (compact), and the copies
// that reserve and compact ask for (copy).
//
// State: refs[p], how many table entries hold page p (0: free), the tables and the
// lengths. Nothing else is kept from call to call, no list of free pages either:
// a call that needs pages counts refs == 0 from the front, so that it always takes
// the lowest ones, whatever the order in which others came back.
//
// The calls on tables are integer work of a few thousand words, bound by the
// latency of the dependent trips to memory between their phases. Those with
// phases that every sequence has to finish (reserve, compact, fork) run as one
// cluster of 1 to 8 CTAs of 1024 threads: its hardware barrier is the cheapest
// meeting of more than one SM's threads, and the counts that a prefix sum needs
// pass through distributed shared memory. Free and trim need no meeting.
// Copies are bound by bytes: one 16-byte word after another, four of a thread in
// flight, any strides. Four blocks of 256 threads an SM: with nothing to copy 2.1 us
// (eight 2.7); a compaction's 176 MB take 29 (26 on cold caches: 88 MB read from DRAM; of the
// 88 written 40 arrive there meanwhile, the rest stays in L2).
//
// In a captured graph, one call among others: reserve 2.4 us for 80 slots without new
// rows, about 6 in a pool of 32885 pages; fork of 64 children of 63 pages about 5.
// What a step of serving takes (free, fork, lengths, reserve, copy for 64 children of
// one prompt): 18.9 us; with CTAs of 1024 threads for all sizes it took 24.3.
//
// Results do not depend on timing: where several callers meet (a page that all
// its holders go on in, a child named twice) the order of the sequences decides.
#include <string.h>

#include "fr_paged.h"
#include "fr_sm100.cuh"

namespace fr {
namespace paged {
namespace pool {

using sm100::cluster_nrank;
using sm100::cluster_rank;
using sm100::cluster_sync;
using sm100::smem_addr;

// Threads of a CTA: many for large pools and batches; a few sequences are done sooner by
// few warps, whose instructions one SM has to issue (80 slots, 634 pages, no new rows:
// 2.4 us by 256 threads, 3.3 by 1024).
constexpr int kFewThreads = 256, kThreads = 1024, kMaxCluster = 8;
constexpr int kOwn = kMaxSeq / (kThreads * kMaxCluster);      // sequences of a thread at most
constexpr unsigned kStatusNoPages = 0x200u;
static_assert(((kStatusInput | kStatusNoPages) & ~0xff00u) == 0, "fr_pages_check sets them by their byte");
constexpr int kMaxPages = 1 << 28;

struct Move {                             // rows 0 .. rows - 1 of page `from` belong into page `to`
    int from, to, rows, pad;
};
struct Job {                              // a sequence's new entries, or a fork
    int x, y, z, w;
};

struct PoolDesc {
    int32_t *refs, *kv_len, *table;
    int64_t table_stride;
    char* ws;
    int n_seq, max_pages, n_pages, page_shift, dev;
    uint32_t magic;
};
constexpr uint32_t kPoolMagic = 0x46525047u;
static_assert(sizeof(PoolDesc) <= sizeof(fr_page_pool), "fr_page_pool is too small");

// Workspace: [0, 4) status word, [64, 68) number of moves, then from kWsHeader on
// the moves, the map of compact, the list of reserve's pages, jobs.
static size_t n_moves_most(int n_pages, int n_seq) { return (size_t)(n_pages / 2 + 1 > n_seq ? n_pages / 2 + 1 : n_seq); }
static size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }
static size_t pool_ws_bytes(int n_pages, int n_seq) {
    return kWsHeader + sizeof(Move) * n_moves_most(n_pages, n_seq) + 2 * align16(4 * (size_t)n_pages) + sizeof(Job) * (size_t)n_seq;
}

struct PoolArgs {
    int32_t *refs, *kv_len, *table;
    int64_t table_stride;
    unsigned* status;
    int* n_moves;
    Move* moves;
    int *map, *list;
    Job* jobs;
    int n_seq, max_pages, n_pages, page_shift;
};

__device__ __forceinline__ void launch_begins() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Word at the same shared-memory place in CTA `rank`.
template <typename T>
__device__ __forceinline__ T peer(const T* p, int rank) {
    const uint32_t at = sm100::map_rank(smem_addr(p), rank);
    if (sizeof(T) == 8) {
        unsigned long long v;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
        return (T)v;
    }
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return (T)v;
}
// Pages 32 at a time, in order: this warp's share of the pool, counted with f.
struct PageShare {
    int first, end;
};
template <int NT>
__device__ __forceinline__ PageShare page_share(const PoolArgs& a) {
    const int warps = NT / 32 * (int)cluster_nrank(), w = (int)cluster_rank() * (NT / 32) + (threadIdx.x >> 5);
    const int per = (int)((((int64_t)a.n_pages + warps - 1) / warps + 127) / 128 * 128);
    const int64_t first = (int64_t)per * w;
    PageShare s;
    s.first = first < a.n_pages ? (int)first : a.n_pages;
    s.end = s.first + per < a.n_pages ? s.first + per : a.n_pages;
    return s;
}
// refs of pages p, p + 32, p + 64, p + 96 (own behind the end).
__device__ __forceinline__ void load_refs(const PoolArgs& a, int p, int end, int own, int* r) {
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u] = p + u * 32 < end ? __ldcg(a.refs + p + u * 32) : own;
}
// A count of each warp of the cluster, in order: those before this warp, and all.
template <int NT>
__device__ __forceinline__ int2 warp_counts(const int* counts) {
    const int lane = threadIdx.x & 31, me = threadIdx.x >> 5, rank = (int)cluster_rank();
    int before = 0, all = 0;
    for (int r = 0; r < (int)cluster_nrank(); ++r) {
        const int v = lane < NT / 32 ? peer(counts + lane, r) : 0;
        all += v;
        if (r < rank || (r == rank && lane < me)) before += v;
    }
    return make_int2(__reduce_add_sync(~0u, before), __reduce_add_sync(~0u, all));
}

// Numbers of sequence b for a step: keys before it and after it. False: they do not fit.
__device__ __forceinline__ bool step_of(const PoolArgs& a, const int32_t* tok_start, int b, int& first, int& n) {
    n = a.kv_len[b];
    first = n;
    if (n < 0 || n > ((int64_t)a.max_pages << a.page_shift)) return false;
    if (!tok_start) return true;
    const int t0 = tok_start[b], t1 = tok_start[b + 1];
    if (t0 < 0 || t1 < t0 || t1 - t0 > n) return false;
    first = n - (t1 - t0);
    return true;
}

// All threads of the cluster meet; a cluster of one CTA by the cheaper barrier.
__device__ __forceinline__ void meet() {
    if (cluster_nrank() == 1) __syncthreads();
    else cluster_sync();
}
// The same, and whether x held anywhere (flag: a word of shared memory for this one
// call, which the others look at until they meet again).
__device__ __forceinline__ bool meet_any(bool x, int* flag) {
    int any = __syncthreads_or(x);
    if (cluster_nrank() == 1) return any != 0;
    if (threadIdx.x == 0) *flag = any;
    cluster_sync();
    any = 0;
    for (int r = 0; r < (int)cluster_nrank(); ++r) any |= peer(flag, r);
    return any != 0;
}

// ---- reserve ------------------------------------------------------------------
// Phases: (1) what the sequences need, from their numbers, and the free pages
// counted meanwhile; where some go on in a page that others hold too, all of those
// take their count off it, and a page that nobody holds any more goes to the last of
// them (marked in refs as a negative number); (2) prefix sums of the needs; (3) the
// lowest free pages listed; (4) tables filled: single entries by the thread that asked,
// several of a sequence by a warp.
constexpr int kListHere = 2048;           // pages that a single CTA lists in shared memory
template <int NT>
__global__ void __launch_bounds__(NT, 1)
pages_reserve_kernel(const __grid_constant__ PoolArgs a, const int32_t* tok_start) {
    constexpr int WARPS = NT / 32;
    __shared__ unsigned long long s_scan[WARPS], s_tot[kOwn];        // needs (low 40 bits) and copies
    __shared__ int s_free[WARPS], s_any, s_list[kListHere];
    launch_begins();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cluster_rank(), ranks = (int)cluster_nrank();
    const int total_thr = NT * ranks, gtid = rank * NT + tid;
    // (a thread's k-th sequence; most calls have none behind the first)
    auto none = [&](int k) { return k > 0 && k * total_thr >= a.n_seq; };
    int first[kOwn], end[kOwn], part[kOwn];          // keys before and after; the page that earlier rows share
    bool bad = false, shared = false;
    int t0[kOwn], t1[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        end[k] = t0[k] = t1[k] = 0;
        if (none(k)) continue;
        const int b = k * total_thr + gtid;
        const bool is = b < a.n_seq;
        end[k] = is ? a.kv_len[b] : 0;
        t0[k] = is ? tok_start[b] : 0;
        t1[k] = is ? tok_start[b + 1] : 0;
    }
    // free pages of this warp's share, as bits for the first eight steps
    const PageShare sh = page_share<NT>(a);
    int n_free = 0;
    unsigned bits = 0u;
    for (int p = sh.first + lane, step = 0; p - lane < sh.end; p += 128, ++step) {
        int r[4];
        load_refs(a, p, sh.end, 1, r);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            n_free += r[u] == 0;
            if (step < 8 && r[u] == 0) bits |= 1u << (step * 4 + u);
        }
    }
    n_free = __reduce_add_sync(~0u, n_free);
    if (lane == 0) s_free[warp] = n_free;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int b = k * total_thr + gtid;
        part[k] = -1;
        first[k] = 0;
        if (none(k)) continue;
        if (end[k] < 0 || end[k] > ((int64_t)a.max_pages << a.page_shift) || t0[k] < 0 || t1[k] < t0[k] || t1[k] - t0[k] > end[k]) {
            bad = true;
            end[k] = t1[k] = t0[k] = 0;
        }
        first[k] = end[k] - (t1[k] - t0[k]);
        if (first[k] == end[k] || !(first[k] & ((1 << a.page_shift) - 1))) continue;
        const int p = a.table[b * a.table_stride + (first[k] >> a.page_shift)];
        const int holders = p >= 0 && p < a.n_pages ? __ldcg(a.refs + p) : 0;
        if (holders == 1) {
            first[k] = min(end[k], (first[k] | ((1 << a.page_shift) - 1)) + 1);       // it goes on in its page
        } else if (holders > 1) {
            part[k] = p;
            shared = true;
        } else {
            bad = true;                               // no such page, or one that counts no holder: the entry is filled anew
        }
    }
    if (meet_any(shared, &s_any)) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (!none(k) && part[k] >= 0) atomicSub(a.refs + part[k], 1);
        meet();
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (!none(k) && part[k] >= 0 && __ldcg(a.refs + part[k]) <= 0) atomicMin(a.refs + part[k], -(k * total_thr + gtid + 1));
        meet();
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (!none(k) && part[k] >= 0 && __ldcg(a.refs + part[k]) == -(k * total_thr + gtid + 1)) {
                a.refs[part[k]] = 1;                  // it keeps its page
                part[k] = -1;
                first[k] = min(end[k], (first[k] | ((1 << a.page_shift) - 1)) + 1);
            }
    }
    // entries that each needs: of the pages from that of key `first` on
    auto entry = [&](int k) { return first[k] >> a.page_shift; };
    auto count = [&](int k) { return first[k] < end[k] ? ((end[k] - 1) >> a.page_shift) - entry(k) + 1 : 0; };
    unsigned long long before[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        if (none(k)) continue;
        const unsigned long long own = (unsigned long long)count(k) | (unsigned long long)(part[k] >= 0) << 40;
        unsigned long long inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += x;
        }
        if (k) __syncthreads();                       // (s_scan has been read)
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        unsigned long long mine = lane < WARPS ? s_scan[lane] : 0, sum = mine;       // of the warps
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += x;
        }
        before[k] = __shfl_sync(~0u, sum - mine, warp) + inc - own;
        if (tid == 31) s_tot[k] = sum;
    }
    meet();
    const int2 free_of = warp_counts<NT>(s_free);
    unsigned long long need = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        if (none(k)) continue;
        unsigned long long base = need;
        for (int r = 0; r < ranks; ++r) {
            const unsigned long long v = peer(s_tot + k, r);
            if (r < rank) base += v;
            need += v;
        }
        before[k] += base;
    }
    const long long wanted = (long long)(need & ((1ull << 40) - 1));
    if (gtid == 0) *a.n_moves = (int)(need >> 40);
    const bool any_bad = __any_sync(~0u, bad), short_of = gtid == 0 && wanted > free_of.y;
    if (lane == 0 && (any_bad || short_of)) atomicOr(a.status, (any_bad ? kStatusInput : 0u) | (short_of ? kStatusNoPages : 0u));
    if (wanted == 0) {
        meet();                                       // (the others have read this CTA's counts)
        return;
    }
    // the lowest free pages, as many as are wanted
    int* const list = ranks == 1 && wanted <= kListHere ? s_list : a.list;
    int at = free_of.x;
    for (int p = sh.first + lane, step = 0; p - lane < sh.end && at < wanted; p += 128, ++step) {
        int r[4] = {1, 1, 1, 1};
        if (step >= 8) load_refs(a, p, sh.end, 1, r);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool is = step < 8 ? bits >> (step * 4 + u) & 1u : r[u] == 0;
            const unsigned m = __ballot_sync(~0u, is);
            const int place = at + __popc(m & ((1u << lane) - 1u));
            if (is && place < wanted) list[place] = p + u * 32;
            at += __popc(m);
        }
    }
    bool many = false;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int b = k * total_thr + gtid;
        if (none(k) || b >= a.n_seq) continue;
        const unsigned long long at_page = before[k] & ((1ull << 40) - 1);
        const int from = at_page < (unsigned long long)a.n_pages ? (int)at_page : a.n_pages, n = count(k);
        const int copy = part[k] >= 0 ? (int)(before[k] >> 40) : -1;
        if (copy >= 0) a.moves[copy] = Move{part[k], -1, first[k] & ((1 << a.page_shift) - 1), 0};
        a.jobs[b] = Job{from, entry(k), n > 1 ? n : 0, copy};
        many |= n > 1;
        t0[k] = from;
        t1[k] = copy;
    }
    if (ranks == 1) {
        many = __syncthreads_or(many);
    } else {                                          // (no CTA looks into another's memory from here on)
        cluster_sync();
        many = true;
    }
    auto page_at = [&](int i) { return i >= free_of.y ? -1 : list == s_list ? s_list[i] : __ldcg(a.list + i); };
    auto put = [&](int seq, int from, int row, int e, int copy) {
        const int page = page_at(from + e);
        a.table[seq * a.table_stride + row + e] = page;
        if (page >= 0) a.refs[page] = 1;
        if (e == 0 && copy >= 0) a.moves[copy].to = page;
    };
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
        if (!none(k) && count(k) == 1) put(k * total_thr + gtid, t0[k], entry(k), 0, t1[k]);
    if (!many) return;
    const int warps = WARPS * ranks, per = min(32, (a.n_seq + warps - 1) / warps);      // sequences of a warp
    for (int b0 = (rank * WARPS + warp) * per; b0 < a.n_seq; b0 += warps * per) {
        int4 j = make_int4(0, 0, 0, -1);
        if (lane < per && b0 + lane < a.n_seq) j = __ldcg(reinterpret_cast<const int4*>(a.jobs + b0 + lane));
        for (unsigned left = __ballot_sync(~0u, j.z > 0); left; left &= left - 1) {
            const int from = __ffs(left) - 1;
            const int x = __shfl_sync(~0u, j.x, from), y = __shfl_sync(~0u, j.y, from), z = __shfl_sync(~0u, j.z, from),
                      w = __shfl_sync(~0u, j.w, from);
#pragma unroll 4
            for (int e = lane; e < z; e += 32) put(b0 + from, x, y, e, w);
        }
    }
}

// ---- fork ---------------------------------------------------------------------
// Of several pairs with one child the first counts. Few pairs: every thread looks
// through the children before its own; many: a child is claimed in its length, 0 so
// far, which becomes the smallest of the pairs' negative marks.
constexpr int kFewPairs = kFewThreads;
template <int NT>
__global__ void __launch_bounds__(NT, 1)
pages_fork_kernel(const __grid_constant__ PoolArgs a, const int32_t* parent, const int32_t* child, const int32_t* length, int n) {
    __shared__ int s_child[kFewPairs];
    __shared__ Job s_jobs[kFewPairs];
    launch_begins();
    const int tid = threadIdx.x, rank = (int)cluster_rank(), ranks = (int)cluster_nrank();
    const int total_thr = NT * ranks, gtid = rank * NT + tid, lane = tid & 31;
    const bool few = n <= kFewPairs;                   // (each CTA works them out for itself)
    int len[kOwn], to[kOwn], from[kOwn];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        len[k] = to[k] = -1;
        const int i = k * total_thr + (few ? tid : gtid);
        if (i >= n || (few && k)) continue;
        const int p = parent[i], c = child[i], l = length ? length[i] : 0;
        if (p == -1 || c == -1) continue;              // no pair
        if (p < 0 || p >= a.n_seq || c < 0 || c >= a.n_seq || p == c) {
            bad = true;
            continue;
        }
        const int have = a.kv_len[p], was = a.kv_len[c], m = length ? l : have;
        if (have < 0 || have > ((int64_t)a.max_pages << a.page_shift) || m < 0 || m > have || was != 0) {
            bad = true;
            continue;
        }
        len[k] = m;
        to[k] = c;
        from[k] = p;
    }
    auto pages = [&](int k) { return (int)(((int64_t)len[k] + (1 << a.page_shift) - 1) >> a.page_shift); };
    if (few) {
        if (tid < n) s_child[tid] = to[0];
        meet();                                        // (lengths have been read by all CTAs)
        if (tid < n) {
            bool mine = to[0] >= 0;
            for (int i = 0; i < tid && mine; ++i) mine = s_child[i] != to[0];
            bad |= to[0] >= 0 && !mine;
            if (mine && rank == 0) a.kv_len[to[0]] = len[0];
            s_jobs[tid] = mine ? Job{from[0], to[0], pages(0), 0} : Job{0, 0, 0, 0};
        }
        __syncthreads();
    } else {
        meet();                                        // lengths have been read
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (to[k] >= 0) atomicMin(a.kv_len + to[k], k * total_thr + gtid - n);
        meet();
        bool mine[kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            mine[k] = to[k] >= 0 && __ldcg(a.kv_len + to[k]) == k * total_thr + gtid - n;
            bad |= to[k] >= 0 && !mine[k];
        }
        meet();                                        // marks have been read
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int i = k * total_thr + gtid;
            if (i >= n) continue;
            if (mine[k]) a.kv_len[to[k]] = len[k];
            a.jobs[i] = mine[k] ? Job{from[k], to[k], pages(k), 0} : Job{0, 0, 0, 0};
        }
        meet();
    }
    if (__any_sync(~0u, bad) && lane == 0) atomicOr(a.status, kStatusInput);
    // pieces of 128 entries of a pair's tables to a warp
    const int chunks = (a.max_pages + 127) / 128, warps = (NT / 32) * ranks;
    bool odd = false;
    for (int64_t it = rank * (NT / 32) + (tid >> 5); it < (int64_t)n * chunks; it += warps) {
        const int i = (int)(it / chunks), e0 = (int)(it - (int64_t)i * chunks) * 128 + lane;
        Job j;
        if (few) {
            j = s_jobs[i];
        } else {
            const int4 v = __ldcg(reinterpret_cast<const int4*>(a.jobs + i));
            j = Job{v.x, v.y, v.z, v.w};
        }
        const int32_t* src = a.table + j.x * a.table_stride;
        int32_t* dst = a.table + j.y * a.table_stride;
        int p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = e0 + u * 32 < j.z ? src[e0 + u * 32] : -1;
        // (counts only grow here, and only those above 0: what is read here decides the same for every child)
        int held[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) held[u] = p[u] >= 0 && p[u] < a.n_pages ? __ldcg(a.refs + p[u]) : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (e0 + u * 32 >= j.z) continue;
            odd |= held[u] <= 0 && p[u] != -1;         // no page, or one that counts no holder (-1: trimmed)
            dst[e0 + u * 32] = held[u] > 0 ? p[u] : -1;
            if (held[u] > 0) atomicAdd(a.refs + p[u], 1);
        }
    }
    if (__any_sync(~0u, odd) && lane == 0) atomicOr(a.status, kStatusInput);
}

// ---- free and trim ------------------------------------------------------------
// An entry is given back; true: it held what it should not.
__device__ __forceinline__ bool drop(const PoolArgs& a, int32_t* entry, int p) {
    if (p == -1) return false;
    *entry = -1;
    if (p < 0 || p >= a.n_pages) return true;
    if (atomicSub(a.refs + p, 1) > 0) return false;
    atomicAdd(a.refs + p, 1);
    return true;
}
// A block for a sequence of the list. Named twice, a sequence gives every page back
// once: each block drops what its own shortening of the length laid free.
__global__ void __launch_bounds__(256)
pages_free_kernel(const __grid_constant__ PoolArgs a, const int32_t* seq, const int32_t* keep) {
    __shared__ int s_from, s_to;
    launch_begins();
    if (threadIdx.x == 0) {
        const int b = seq[blockIdx.x], k = keep ? keep[blockIdx.x] : 0;
        int from = 0, to = 0;
        if (b != -1) {
            const int most = (int)min((int64_t)a.max_pages << a.page_shift, (int64_t)0x7fffffff);
            if (b < 0 || b >= a.n_seq || k < 0) {
                atomicOr(a.status, kStatusInput);
            } else {
                const int old = atomicMin(a.kv_len + b, k), up = (1 << a.page_shift) - 1;
                if (old < 0 || old > most) {
                    atomicOr(a.status, kStatusInput);  // (a length that does not fit stays, and so do the entries)
                    if (old > most) atomicMax(a.kv_len + b, old);
                } else if (old > k) {
                    from = (int)(((int64_t)k + up) >> a.page_shift);
                    to = (int)(((int64_t)old + up) >> a.page_shift);
                }
            }
        }
        s_from = from;
        s_to = to;
    }
    __syncthreads();
    const int from = s_from, to = s_to;
    if (from >= to) return;
    int32_t* row = a.table + seq[blockIdx.x] * a.table_stride;
    bool odd = false;
    for (int e = from + threadIdx.x; e < to; e += 4 * blockDim.x) {
        int p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = e + u * (int)blockDim.x < to ? row[e + u * blockDim.x] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) odd |= drop(a, row + e + u * blockDim.x, p[u]);
    }
    if (odd) atomicOr(a.status, kStatusInput);
}
// Entries [from, to) of every sequence: behind the sinks' pages and before the first
// key that the step's first row sees. Blocks of 1024 entries.
__global__ void __launch_bounds__(256)
pages_trim_kernel(const __grid_constant__ PoolArgs a, const int32_t* tok_start, int window, int sinks, int chunks) {
    launch_begins();
    bool odd = false;
    for (int64_t it = blockIdx.x; it < (int64_t)a.n_seq * chunks; it += gridDim.x) {
        const int b = (int)(it / chunks), e0 = (int)(it - (int64_t)b * chunks) * 1024;
        int first, n;
        if (!step_of(a, tok_start, b, first, n)) {
            odd = true;
            continue;
        }
        const int64_t low = (int64_t)first - window + 1;       // the first key of the window
        const int from = max(e0, (int)(((int64_t)sinks + (1 << a.page_shift) - 1) >> a.page_shift));
        const int to = low <= 0 ? 0 : (int)min((int64_t)e0 + 1024, low >> a.page_shift);
        int32_t* row = a.table + b * a.table_stride;
        int p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = from + (int)threadIdx.x + u * 256 < to ? row[from + threadIdx.x + u * 256] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) odd |= drop(a, row + from + threadIdx.x + u * 256, p[u]);
    }
    if (odd) atomicOr(a.status, kStatusInput);
}

// ---- compact ------------------------------------------------------------------
// U pages are held. The k-th highest of those at U and behind goes into the k-th
// lowest hole before U: their numbers are page - used_before and U - 1 - used_before.
__global__ void __launch_bounds__(kThreads, 1)
pages_compact_kernel(const __grid_constant__ PoolArgs a) {
    __shared__ int s_used[kThreads / 32];
    launch_begins();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gtid = (int)cluster_rank() * kThreads + tid, total_thr = kThreads * (int)cluster_nrank();
    if (gtid == 0) *a.n_moves = 0;
    const PageShare sh = page_share<kThreads>(a);
    int used = 0;
    for (int p = sh.first + lane; p - lane < sh.end; p += 128) {
        int r[4];
        load_refs(a, p, sh.end, 0, r);
#pragma unroll
        for (int u = 0; u < 4; ++u) used += r[u] != 0;
    }
    used = __reduce_add_sync(~0u, used);
    if (lane == 0) s_used[warp] = used;
    cluster_sync();
    const int2 count = warp_counts<kThreads>(s_used);
    const int U = count.y;
    int at = count.x, holes = 0;
    for (int p = sh.first + lane; p - lane < sh.end; p += 128) {
        int r[4];
        load_refs(a, p, sh.end, 0, r);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int page = p + u * 32;
            const unsigned m = __ballot_sync(~0u, r[u] != 0);
            const int before = at + __popc(m & ((1u << lane) - 1u));
            at += __popc(m);
            if (page >= sh.end) continue;
            if (r[u] == 0) {
                a.map[page] = -1;
                if (page < U) {
                    a.moves[page - before].to = page;
                    ++holes;
                }
            } else if (page < U) {
                a.map[page] = page;
            } else {
                a.moves[U - 1 - before].from = page;
            }
        }
    }
    holes = __reduce_add_sync(~0u, holes);
    if (lane == 0 && holes) atomicAdd(a.n_moves, holes);
    cluster_sync();
    const int n = __ldcg(a.n_moves);
    for (int k = gtid; k < n; k += total_thr) {
        const int4 v = __ldcg(reinterpret_cast<const int4*>(a.moves + k));
        a.map[v.x] = v.y;
        a.refs[v.y] = __ldcg(a.refs + v.x);
        a.refs[v.x] = 0;
        a.moves[k].rows = 1 << a.page_shift;
    }
}
// The tables' entries go along.
__global__ void __launch_bounds__(256)
pages_remap_kernel(const __grid_constant__ PoolArgs a, int chunks) {
    launch_begins();
    if (__ldcg(a.n_moves) == 0) return;
    bool odd = false;
    for (int64_t it = blockIdx.x; it < (int64_t)a.n_seq * chunks; it += gridDim.x) {
        const int b = (int)(it / chunks), e0 = (int)(it - (int64_t)b * chunks) * 1024 + threadIdx.x;
        int first, n;
        if (!step_of(a, nullptr, b, first, n)) {
            odd = true;
            continue;
        }
        const int to = (int)(((int64_t)n + (1 << a.page_shift) - 1) >> a.page_shift);
        int32_t* row = a.table + b * a.table_stride;
        int p[4], q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = e0 + u * 256 < to ? row[e0 + u * 256] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = p[u] >= 0 && p[u] < a.n_pages ? __ldcg(a.map + p[u]) : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (p[u] == -1) continue;
            odd |= q[u] < 0;                           // no such page, or one that counts no holder
            if (q[u] >= 0 && q[u] != p[u]) row[e0 + u * 256] = q[u];
        }
    }
    if (odd) atomicOr(a.status, kStatusInput);
}

// ---- copy ---------------------------------------------------------------------
struct CopyArgs {
    char *k, *v;
    int64_t k_page, k_head, k_row, v_page, v_head, v_row;     // bytes
    float *k_scale, *v_scale;
    const int* n_moves;
    const Move* moves;
    int n_pages, page_shift, n_kv_head, row_shift;            // 2^row_shift 16-byte words in a row
    int tiles;                                                // of kCopyTile words of K, or V, of a page
};
constexpr int kCopyTile = 1024;

__global__ void __launch_bounds__(256)
pages_copy_kernel(const __grid_constant__ CopyArgs a) {
    launch_begins();
    const int n = __ldcg(a.n_moves), words = a.n_kv_head << (a.page_shift + a.row_shift);
    for (int64_t it = blockIdx.x; it < (int64_t)n * 2 * a.tiles; it += gridDim.x) {
        const int64_t mk = it / a.tiles;
        const int tile = (int)(it - mk * a.tiles), is_v = (int)(mk & 1);
        const int4 m = __ldcg(reinterpret_cast<const int4*>(a.moves + (mk >> 1)));
        if (m.x < 0 || m.x >= a.n_pages || m.y < 0 || m.y >= a.n_pages) continue;      // (-1: there was no page)
        const char* src = (is_v ? a.v + m.x * a.v_page : a.k + m.x * a.k_page);
        char* dst = (is_v ? a.v + m.y * a.v_page : a.k + m.y * a.k_page);
        const int64_t head = is_v ? a.v_head : a.k_head, row = is_v ? a.v_row : a.k_row;
        uint4 x[4];
        int64_t at[4];
        bool have[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int w = tile * kCopyTile + u * 256 + threadIdx.x;
            const int r = w >> a.row_shift & ((1 << a.page_shift) - 1);
            have[u] = w < words && r < m.z;
            at[u] = (int64_t)(w >> (a.row_shift + a.page_shift)) * head + r * row + (int64_t)(w & ((1 << a.row_shift) - 1)) * 16;
            if (have[u]) x[u] = __ldcg(reinterpret_cast<const uint4*>(src + at[u]));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (have[u]) *reinterpret_cast<uint4*>(dst + at[u]) = x[u];
        if (a.k_scale && tile == 0 && m.z > 0) {
            float* s = is_v ? a.v_scale : a.k_scale;
            for (int h = threadIdx.x; h < a.n_kv_head; h += 256)
                s[(int64_t)m.y * a.n_kv_head + h] = s[(int64_t)m.x * a.n_kv_head + h];
        }
    }
}

// ---- host ---------------------------------------------------------------------
static const PoolDesc* pool_desc(const fr_page_pool* p) {
    const PoolDesc* d = reinterpret_cast<const PoolDesc*>(p);
    return p && d->magic == kPoolMagic ? d : nullptr;
}
static PoolArgs pool_args(const PoolDesc& d) {
    PoolArgs a;
    a.refs = d.refs;
    a.kv_len = d.kv_len;
    a.table = d.table;
    a.table_stride = d.table_stride;
    a.status = reinterpret_cast<unsigned*>(d.ws);
    a.n_moves = reinterpret_cast<int*>(d.ws + 64);
    a.moves = reinterpret_cast<Move*>(d.ws + kWsHeader);
    char* after = reinterpret_cast<char*>(a.moves + n_moves_most(d.n_pages, d.n_seq));
    a.map = reinterpret_cast<int*>(after);
    a.list = reinterpret_cast<int*>(after + align16(4 * (size_t)d.n_pages));
    a.jobs = reinterpret_cast<Job*>(after + 2 * align16(4 * (size_t)d.n_pages));
    a.n_seq = d.n_seq;
    a.max_pages = d.max_pages;
    a.n_pages = d.n_pages;
    a.page_shift = d.page_shift;
    return a;
}
// The pool's GPU has to be the current one.
static fr_status on_device(int dev) {
    int now = 0;
    if (cudaGetDevice(&now) != cudaSuccess) return FR_ERR_CUDA;
    return now == dev ? FR_OK : FR_ERR_INVALID_ARG;
}
template <typename K, typename... A>
static fr_status launch(K kernel, int64_t blocks, int threads, int cluster, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FR_OK : FR_ERR_CUDA;
}
constexpr int kWordsEach = 32768;         // (16384 or 65536 for 32885 pages: the same)
// CTAs of the cluster for so many sequences (kOwn to a thread) and words of refs or tables.
static int cluster_for(int64_t seqs, int64_t words) {
    int c = 1;
    while (c < kMaxCluster && ((int64_t)c * kThreads * kOwn < seqs || (int64_t)c * kWordsEach < words)) c *= 2;
    return c;
}
static int chunks_of(const PoolDesc& d) { return (d.max_pages + 1023) / 1024; }

}  // namespace pool
}  // namespace paged
}  // namespace fr

using namespace fr;
using namespace fr::paged;
using namespace fr::paged::pool;

extern "C" size_t fr_pages_workspace_size(int n_pages, int n_seq) {
    if (n_pages < 1 || n_seq < 1 || n_pages > kMaxPages || n_seq > kMaxSeq) return 0;
    return pool_ws_bytes(n_pages, n_seq);
}

extern "C" fr_status fr_page_pool_init(fr_page_pool* pool, int32_t* refs, int n_pages, int page_size, int32_t* kv_len,
                                       int32_t* page_table, int64_t page_table_stride, int n_seq, int max_pages,
                                       void* workspace, size_t workspace_bytes) {
    if (!pool || !refs || !kv_len || !page_table || !workspace) return FR_ERR_INVALID_ARG;
    memset(pool, 0, sizeof(*pool));
    if (n_pages < 1 || page_size < 1 || n_seq < 1 || max_pages < 1 || page_table_stride < max_pages) return FR_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return FR_ERR_UNSUPPORTED;
    if (n_pages > kMaxPages || n_seq > kMaxSeq || max_pages > (1 << 22)) return FR_ERR_UNSUPPORTED;
    if (((uintptr_t)refs | (uintptr_t)kv_len | (uintptr_t)page_table) & 3 || !aligned16(workspace)) return FR_ERR_INVALID_ARG;
    if (workspace_bytes < pool_ws_bytes(n_pages, n_seq)) return FR_ERR_WORKSPACE;
    PoolDesc d;
    memset(&d, 0, sizeof(d));
    if (cudaGetDevice(&d.dev) != cudaSuccess) return FR_ERR_CUDA;
    const void* ptrs[] = {refs, kv_len, page_table, workspace};
    for (const void* p : ptrs)
        if (!device_ptr_ok(p, d.dev)) return FR_ERR_INVALID_ARG;
    d.refs = refs;
    d.kv_len = kv_len;
    d.table = page_table;
    d.table_stride = page_table_stride;
    d.ws = reinterpret_cast<char*>(workspace);
    d.n_seq = n_seq;
    d.max_pages = max_pages;
    d.n_pages = n_pages;
    d.page_shift = __builtin_ctz((unsigned)page_size);
    d.magic = kPoolMagic;
    memcpy(pool, &d, sizeof(d));
    return FR_OK;
}

extern "C" fr_status fr_pages_check(const fr_page_pool* pool, cudaStream_t stream) {
    const PoolDesc* d = pool_desc(pool);
    if (!d) return FR_ERR_INVALID_ARG;
    unsigned word = 0;
    if (cudaMemcpyAsync(&word, d->ws, sizeof(word), cudaMemcpyDeviceToHost, stream) != cudaSuccess) return FR_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return FR_ERR_CUDA;
    if (word == 0) return FR_OK;
    // One state a call, and only that is cleared: pages that ran out first, then the numbers
    // that did not fit (byte 1 of the word holds both bits)
    const bool pages = (word & kStatusNoPages) != 0;
    const int left = pages ? (int)((word & kStatusInput) >> 8) : 0;
    if (cudaMemsetAsync(d->ws, 0, sizeof(word), stream) != cudaSuccess) return FR_ERR_CUDA;
    if (left && cudaMemsetAsync(d->ws + 1, left, 1, stream) != cudaSuccess) return FR_ERR_CUDA;
    return pages ? FR_ERR_DEVICE_PAGES : FR_ERR_DEVICE_INPUT;
}

extern "C" fr_status fr_pages_reserve(const fr_page_pool* pool, const int32_t* tok_start, cudaStream_t stream) {
    const PoolDesc* d = pool_desc(pool);
    if (!d || !tok_start || ((uintptr_t)tok_start & 3)) return FR_ERR_INVALID_ARG;
    const fr_status s = on_device(d->dev);
    if (s != FR_OK) return s;
    if (!device_ptr_ok(tok_start, d->dev)) return FR_ERR_INVALID_ARG;
    if (d->n_seq <= 2 * kFewThreads && d->n_pages <= 16384)
        return launch(pages_reserve_kernel<kFewThreads>, 1, kFewThreads, 1, stream, pool_args(*d), tok_start);
    const int c = cluster_for(d->n_seq, d->n_pages);
    return launch(pages_reserve_kernel<kThreads>, c, kThreads, c, stream, pool_args(*d), tok_start);
}

extern "C" fr_status fr_pages_fork(const fr_page_pool* pool, const int32_t* parent, const int32_t* child,
                                   const int32_t* length, int n, cudaStream_t stream) {
    const PoolDesc* d = pool_desc(pool);
    if (!d || !parent || !child || n < 1 || n > d->n_seq) return FR_ERR_INVALID_ARG;
    if (((uintptr_t)parent | (uintptr_t)child | (uintptr_t)length) & 3) return FR_ERR_INVALID_ARG;
    const fr_status s = on_device(d->dev);
    if (s != FR_OK) return s;
    if (!device_ptr_ok(parent, d->dev) || !device_ptr_ok(child, d->dev) || (length && !device_ptr_ok(length, d->dev)))
        return FR_ERR_INVALID_ARG;
    const int64_t entries = (int64_t)n * d->max_pages;
    if (n <= kFewPairs && entries <= 2048)
        return launch(pages_fork_kernel<kFewThreads>, 1, kFewThreads, 1, stream, pool_args(*d), parent, child, length, n);
    const int c = cluster_for(n, 4 * entries);
    return launch(pages_fork_kernel<kThreads>, c, kThreads, c, stream, pool_args(*d), parent, child, length, n);
}

extern "C" fr_status fr_pages_free(const fr_page_pool* pool, const int32_t* seq, const int32_t* keep, int n, cudaStream_t stream) {
    const PoolDesc* d = pool_desc(pool);
    if (!d || !seq || n < 1 || (((uintptr_t)seq | (uintptr_t)keep) & 3)) return FR_ERR_INVALID_ARG;
    const fr_status s = on_device(d->dev);
    if (s != FR_OK) return s;
    if (!device_ptr_ok(seq, d->dev) || (keep && !device_ptr_ok(keep, d->dev))) return FR_ERR_INVALID_ARG;
    return launch(pages_free_kernel, n, 256, 0, stream, pool_args(*d), seq, keep);
}

extern "C" fr_status fr_pages_trim(const fr_page_pool* pool, const int32_t* tok_start, int window, int n_sink, cudaStream_t stream) {
    const PoolDesc* d = pool_desc(pool);
    if (!d || window < 1 || n_sink < 0 || ((uintptr_t)tok_start & 3)) return FR_ERR_INVALID_ARG;
    const fr_status s = on_device(d->dev);
    if (s != FR_OK) return s;
    if (tok_start && !device_ptr_ok(tok_start, d->dev)) return FR_ERR_INVALID_ARG;
    const int chunks = chunks_of(*d);
    const int64_t items = (int64_t)d->n_seq * chunks;
    return launch(pages_trim_kernel, items < 4096 ? items : 4096, 256, 0, stream, pool_args(*d), tok_start, window, n_sink, chunks);
}

extern "C" fr_status fr_pages_compact(const fr_page_pool* pool, cudaStream_t stream) {
    const PoolDesc* d = pool_desc(pool);
    if (!d) return FR_ERR_INVALID_ARG;
    fr_status s = on_device(d->dev);
    if (s != FR_OK) return s;
    const PoolArgs a = pool_args(*d);
    const int c = cluster_for(1, d->n_pages), chunks = chunks_of(*d);
    s = launch(pages_compact_kernel, c, kThreads, c, stream, a);
    if (s != FR_OK) return s;
    const int64_t items = (int64_t)d->n_seq * chunks;
    return launch(pages_remap_kernel, items < 4096 ? items : 4096, 256, 0, stream, a, chunks);
}

extern "C" fr_status fr_pages_copy(const fr_paged_kv* kv_, const fr_page_pool* pool, cudaStream_t stream) {
    const KvDesc* kv = kv_desc(kv_);
    const PoolDesc* d = pool_desc(pool);
    if (!kv || !d || kv->n_pages != d->n_pages || kv->page_shift != d->page_shift || kv->dev != d->dev) return FR_ERR_INVALID_ARG;
    const fr_status s = on_device(d->dev);
    if (s != FR_OK) return s;
    const PoolArgs p = pool_args(*d);
    const int elem = kv->type == FR_KV_E4M3 ? 1 : 2;
    CopyArgs a;
    memset(&a, 0, sizeof(a));
    a.k = reinterpret_cast<char*>(kv->k);
    a.v = reinterpret_cast<char*>(kv->v);
    a.k_page = kv->k_page * elem;
    a.k_head = kv->k_head * elem;
    a.k_row = kv->k_row * elem;
    a.v_page = kv->v_page * elem;
    a.v_head = kv->v_head * elem;
    a.v_row = kv->v_row * elem;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
    a.n_moves = p.n_moves;
    a.moves = p.moves;
    a.n_pages = d->n_pages;
    a.page_shift = d->page_shift;
    a.n_kv_head = kv->n_kv_head;
    a.row_shift = __builtin_ctz((unsigned)(kv->hd * elem / 16));
    const int64_t words = (int64_t)kv->n_kv_head << (a.page_shift + a.row_shift);
    if (words > 0x7fffffff - kCopyTile) return FR_ERR_UNSUPPORTED;
    a.tiles = (int)((words + kCopyTile - 1) / kCopyTile);
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d->dev) != cudaSuccess) return FR_ERR_CUDA;
    const int64_t most = (int64_t)n_moves_most(d->n_pages, d->n_seq) * 2 * a.tiles, wave = (int64_t)sms * 4;
    return launch(pages_copy_kernel, most < wave ? most : wave, 256, 0, stream, a);
}

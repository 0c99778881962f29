// fr_paged.h -- host-side pieces shared by the paged-cache entry points
// (fr_paged.cu: descriptors, checks and the merge kernel; fr_paged_append.cu:
// the append; fr_paged_attn_*.cu: the attention kernels).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fr_common.cuh"

namespace fr {
namespace paged {

constexpr int kTile = 16;            // keys of an MMA step (its M)
constexpr int kUnit = 64;            // keys of one unit of work at least: a tile for each warp of a CTA
// Warps of an attention CTA, CTAs per SM and shared memory of each, for nt blocks
// of 8 query rows. Up to 16 rows at hd <= 128 the accumulators leave room for
// many warps of small CTAs, which share out many short sequences well; else
// eight warps are all that the registers hold, and one CTA of them writes half
// the split states of two. The shares of an SM's shared memory leave room for a
// few small blocks of the kernel before: where they lie in the way of a CTA, it
// starts only when another one ends.
__host__ __device__ constexpr bool many_warps(int hd, int nt) { return nt <= 2 && hd <= 128; }
__host__ __device__ constexpr int cta_warps(int hd, int nt) { return many_warps(hd, nt) ? 4 : 8; }
__host__ __device__ constexpr int ctas_per_sm(int hd, int nt) { return many_warps(hd, nt) ? 3 : 1; }
__host__ __device__ constexpr int cta_smem(int hd, int nt) { return many_warps(hd, nt) ? 65536 : 212992; }
constexpr int kMaxCtas = 640;        // entries of split[], and more than the attention CTAs of any launch (two split states each)
constexpr int kMaxSeq = 65536;
constexpr int kSegCost = 2;          // units that a segment's start and end count for in the work split
constexpr int kTcSegCost = 4;        // the same for the 128-row kernel (four prompts of 2048, 2 / 4 / 6 / 9: 368 / 347 / 356 / 375 us)
constexpr int kTcRows = 128;         // its row tile at most
constexpr int kTcCtas = 160;         // its CTAs at most, one per SM
// its loads: rows of a slot of e4m3 codes (what fits beside the f16 tiles), and of a TMA box
__host__ __device__ constexpr int raw_rows(int hd) { return hd == 256 ? 32 : 64; }
inline int tc_box_rows(int page_size, int hd, bool e4) {
    const int most = e4 ? raw_rows(hd) : 64;
    return page_size < most ? page_size : most;
}
constexpr size_t kWsHeader = 1024;   // [0, 4): status word, as in the other workspaces

// What fr_paged_kv holds, in the library's own terms.
struct KvDesc {
    // 5-D CUtensorMap bytes (dim in box, row, box, head, page) of the attention's
    // tile loads; copied to an aligned place at the launch
    unsigned char k_map[sizeof(CUtensorMap)], v_map[sizeof(CUtensorMap)];
    unsigned char k_map_tc[sizeof(CUtensorMap)], v_map_tc[sizeof(CUtensorMap)];   // of the 128-row kernel's: boxes of up to 64 rows
    void *k, *v;
    float *k_scale, *v_scale;        // e4m3: [n_pages][n_kv_head]
    int64_t k_page, k_head, k_row;   // strides in elements
    int64_t v_page, v_head, v_row;
    int n_pages, page_size, page_shift, n_kv_head, hd, type, dev;
    uint32_t magic;
};
struct BatchDesc {
    const int32_t *tok_start, *kv_len, *table;
    int64_t table_stride;
    int n_seq, n_tok, max_pages, dev;
    uint32_t magic;
};
constexpr uint32_t kKvMagic = 0x46525056u, kBatchMagic = 0x46525042u;
static_assert(sizeof(KvDesc) <= sizeof(fr_paged_kv), "fr_paged_kv is too small");
static_assert(sizeof(BatchDesc) <= sizeof(fr_paged_batch), "fr_paged_batch is too small");

// One segment whose keys went to several CTAs: the merge kernel's work item.
struct alignas(16) Split {
    int first, last;                 // CTAs with a state of it (last < first: nothing to merge)
    int tok0, row0, rows, head;      // query rows row0 .. row0 + rows - 1 of KV head `head`, first token tok0
    int pad[2];
};

struct AttnArgs {
    const __half* q16;
    int64_t q_stride;
    float* out;
    const int32_t *tok_start, *kv_len, *table;
    int64_t table_stride;
    const float *k_scale, *v_scale;
    float* part_o;                   // [2 * CTAs][row tile][hd]: unnormalised sums
    float2* part_ml;                 // [2 * CTAs][row tile]: reference maximum (log2 units), sum of weights
    Split* split;                    // [kMaxCtas]
    int* n_split;                    // entries of it that the call wrote
    unsigned* status;
    int n_seq, n_tok, max_pages, n_pages, page_shift, n_kv_head, group, causal, window;
    int row_tile;                    // rows of a row tile where the kernel does not fix them
    unsigned group_magic;            // ceil(2^32 / group) where a multiplication by it divides rows exactly, else 0
    int split_by_segment;            // split[] is indexed by the segment's number, else by its first CTA
    float scale_log2;                // kq_scale * log2(e)
};

// Sizes of one sequence, bad input cut to what memory holds.
struct SeqInfo {
    int tok0, n_q, n_kv;
    bool bad;
};
__device__ __forceinline__ SeqInfo seq_info(const int32_t* tok_start, const int32_t* kv_len, int b, int n_tok,
                                            int max_pages, int page_shift) {
    SeqInfo s;
    // (plain loads: the kernel before may have written these while this one was
    // starting, which the read-only path does not cover)
    const int t0 = tok_start[b], t1 = tok_start[b + 1], n = kv_len[b];
    const int64_t most = (int64_t)max_pages << page_shift;
    s.bad = t0 < 0 || t1 < t0 || t1 > n_tok || n < 0 || n > most;
    s.tok0 = t0;
    s.n_q = s.bad ? 0 : t1 - t0;
    s.n_kv = s.bad ? 0 : n;
    return s;
}

// bits of a workspace's status word (1, 2 and 4 are waits that gave up)
constexpr unsigned kStatusTimeout = 1u, kStatusInput = 0x100u;

fr_status launch_attn_f16(const KvDesc& kv, const AttnArgs& a, int row_tiles8, int ctas, cudaStream_t st);
// either type, row tiles of up to 128 rows (a.row_tile: whole tokens)
fr_status launch_attn_tc(const KvDesc& kv, const AttnArgs& a, int ctas, cudaStream_t st);
fr_status launch_attn_e4m3(const KvDesc& kv, const AttnArgs& a, int row_tiles8, int ctas, cudaStream_t st);
// The driver's encoder of TMA descriptors (null: not found). Any thread may come first.
inline PFN_cuTensorMapEncodeTiled_v12000 get_encoder() {
    static void* fn = nullptr;
    void* p = __atomic_load_n(&fn, __ATOMIC_ACQUIRE);
    if (!p) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        __atomic_store_n(&fn, p, __ATOMIC_RELEASE);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}
// Pointer checks shared by the entry points.
inline const KvDesc* kv_desc(const fr_paged_kv* p) {
    const KvDesc* d = reinterpret_cast<const KvDesc*>(p);
    return p && d->magic == kKvMagic ? d : nullptr;
}
inline const BatchDesc* batch_desc(const fr_paged_batch* p) {
    const BatchDesc* d = reinterpret_cast<const BatchDesc*>(p);
    return p && d->magic == kBatchMagic ? d : nullptr;
}

}  // namespace paged
}  // namespace fr

// Block tables and slot maps of a step, and the append of its keys and
// values to the paged cache.
#include "mnb_attn.h"
#include "mnb_device.h"

namespace mnb {

// ---------------------------------------------------------------------------
// Tables. With have = ceil(cached / P) and need = the blocks a request takes
// now, everything a request or a token needs is a prefix sum over the
// requests before it: of need (its place in the free list) and of added (its
// first row). Every workgroup scans all requests itself, kScan at a time
// (8 bytes per request out of cache: cheaper than a second launch), then
// resolves its own share of the tokens and of the new table entries by
// binary search in the scanned sums. A token's block is worked out from the
// request's sums, never read back from an entry this launch writes, so
// nothing orders the workgroups.
// Bound: latency (a launch, two dependent loads, a scan, up to eleven steps of
// a search). On the device 8 decoding requests 4.3 us, 1000 5.5, 64 prompts of
// 26240 tokens 4.9, where an empty launch is 2.4; with a token's four searches
// one after another (1024 tokens for 256 threads) and 64-bit divisions by the
// page it was 4.8, 9.6 and 8.1. Many requests cost their passes: 65536 105 us, 173
// with 1024 a pass and none requested ahead.
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 512;
constexpr int kTabPer = 4;                         // requests per thread and pass
constexpr int kScan = kTabThreads * kTabPer;       // requests per pass
constexpr int kTabTokens = 512;                    // tokens per workgroup: one search per thread

// x / page for 0 <= x < 2^30, page = 16 m, magic = ceil(2^32 / m): the error of
// the product is below x / 16 * m / 2^32 < 1 / m, so the floor is exact.
__device__ __forceinline__ int32_t blocks_in(int32_t x, uint64_t magic) {
    return (int32_t)(((uint32_t)x >> 4) * magic >> 32);
}
__device__ __forceinline__ int32_t blocks_for(int32_t x, uint64_t magic) {
    return x > 0 ? blocks_in(x - 1, magic) + 1 : 0;
}

// Largest i < n with first[i] <= x (first[0] <= x; ascending).
__device__ __forceinline__ int last_not_above(const int64_t *first, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kTabThreads) void kv_tables_kernel(KvTablesArgs a) {
    __shared__ int64_t s_start[kScan];   // first new row of each request of the pass
    __shared__ int64_t s_off[kScan];     // its place in the free list
    __shared__ int32_t s_cached[kScan];
    __shared__ int64_t s_wave[2][kTabThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t limit = a.width * a.page;        // <= 2^30
    const int64_t t0 = (int64_t)blockIdx.x * kTabTokens;
    const int64_t t1 = t0 + kTabTokens < a.tokens ? t0 + kTabTokens : a.tokens;
    int64_t rows_before = 0, blocks_before = 0;    // over the passes so far
    int32_t next_cached[kTabPer], next_added[kTabPer];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < kTabPer; ++i) {
            const int b = base + tid * kTabPer + i;
            next_cached[i] = b < a.batch ? a.cached[b] : 0;
            next_added[i] = b < a.batch ? a.added[b] : 0;
        }
    };
    fetch(0);
    for (int base = 0; base < a.batch; base += kScan) {
        const int n = a.batch - base < kScan ? a.batch - base : kScan;
        int32_t cached[kTabPer];
        int32_t added[kTabPer], need[kTabPer], len[kTabPer];
        int64_t sum_rows = 0, sum_blocks = 0;
#pragma unroll
        for (int i = 0; i < kTabPer; ++i) {
            const int b = tid * kTabPer + i;
            cached[i] = 0;
            added[i] = need[i] = len[i] = 0;
            if (b < n) {
                const int32_t c = next_cached[i], d = next_added[i];
                // (past the limit nothing has a place, wherever it starts)
                cached[i] = c < 0 ? 0 : c < limit ? c : limit;
                added[i] = d > 0 ? d : 0;
                len[i] = added[i] < limit - cached[i] ? cached[i] + added[i] : limit;
                need[i] = blocks_for(len[i], a.page_magic) - blocks_for(cached[i], a.page_magic);
            }
            sum_rows += added[i];
            sum_blocks += need[i];
        }
        fetch(base + kScan);
        // exclusive prefix over the workgroup's threads
        int64_t in_rows = sum_rows, in_blocks = sum_blocks;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t r = __shfl_up(in_rows, d), k = __shfl_up(in_blocks, d);
            if (lane >= d) {
                in_rows += r;
                in_blocks += k;
            }
        }
        if (lane == 63) {
            s_wave[0][wave] = in_rows;
            s_wave[1][wave] = in_blocks;
        }
        __syncthreads();
        int64_t rows = rows_before + in_rows - sum_rows, blocks = blocks_before + in_blocks - sum_blocks;
        int64_t all_rows = rows_before, all_blocks = blocks_before;
#pragma unroll
        for (int w = 0; w < kTabThreads / 64; ++w) {
            if (w < wave) {
                rows += s_wave[0][w];
                blocks += s_wave[1][w];
            }
            all_rows += s_wave[0][w];
            all_blocks += s_wave[1][w];
        }
#pragma unroll
        for (int i = 0; i < kTabPer; ++i) {
            const int b = tid * kTabPer + i;
            if (b < n) {
                s_start[b] = rows;
                s_off[b] = blocks;
                s_cached[b] = cached[i];
                if (blockIdx.x == 0) {
                    a.lens[base + b] = (int32_t)len[i];
                    a.starts[base + b] = (int32_t)(rows < a.tokens ? rows : a.tokens);
                }
                rows += added[i];
                blocks += need[i];
            }
        }
        __syncthreads();
        // new table entries, dealt over all threads of the launch
        for (int64_t e = blocks_before + (int64_t)blockIdx.x * kTabThreads + tid; e < all_blocks;
             e += (int64_t)gridDim.x * kTabThreads) {
            const int b = last_not_above(s_off, n, e);
            const int64_t have = blocks_for(s_cached[b], a.page_magic);
            a.table[(int64_t)(base + b) * a.width + have + (e - s_off[b])] = e < a.n_free ? a.free_blocks[e] : -1;
        }
        // this workgroup's tokens that belong to requests of this pass
        const int64_t u0 = t0 > rows_before ? t0 : rows_before, u1 = t1 < all_rows ? t1 : all_rows;
        for (int64_t t = u0 + tid; t < u1; t += kTabThreads) {
            const int b = last_not_above(s_start, n, t);
            const int32_t c = s_cached[b];
            const int64_t past = t - s_start[b];
            int64_t slot = -1;
            if (past < limit - c) {
                const int32_t pos = c + (int32_t)past;
                const int32_t have = blocks_for(c, a.page_magic), place = blocks_in(pos, a.page_magic);
                const int64_t fresh = s_off[b] + place - have;   // in the free list
                int64_t id = -1;
                if (place < have) id = a.table[(int64_t)(base + b) * a.width + place];
                else if (fresh < a.n_free) id = a.free_blocks[fresh];
                if (id >= 0) slot = id * a.page + (pos - place * a.page);
            }
            a.slots[t] = slot;
        }
        rows_before = all_rows;
        blocks_before = all_blocks;
        __syncthreads();
    }
    for (int64_t t = (t0 > rows_before ? t0 : rows_before) + tid; t < t1; t += kTabThreads) a.slots[t] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.batch] = (int32_t)(rows_before < a.tokens ? rows_before : a.tokens);
        a.taken[0] = (int32_t)blocks_before;
    }
}

hipError_t launch_kv_tables(const KvTablesArgs &a, hipStream_t st) {
    const int64_t wgs = (a.tokens + kTabTokens - 1) / kTabTokens;
    KvTablesArgs c = a;
    c.page_magic = ((1ull << 32) + a.page / 16 - 1) / (a.page / 16);
    kv_tables_kernel<<<(unsigned)(wgs < 1 ? 1 : wgs), kTabThreads, 0, st>>>(c);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Append: a copy of 16-byte pieces, token rows in, page rows out. A workgroup
// takes `per` tokens, as many as its threads have pieces for (or one), and
// neighbouring tokens of a page meet in the L2. Bound: memory (26240 tokens of 2
// x 2 KB read and written: 44.7 us, 4.8 TB/s, what a large copy reaches), and
// the launch for a decoding step (8 tokens: 2.5 us). With one token a workgroup
// 26240 of one head of 64 took 14.9 us instead of 5.0, 100000 of two heads of 128
// 50 instead of 30.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

// (SHARED: per > 1; otherwise a token's place is worked out in scalar registers)
template <bool SHARED> __global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendArgs a, int per) {
    const int row_pieces = a.row_bytes / 16, pieces = a.heads * row_pieces, both = 2 * pieces;
    const int which = SHARED ? threadIdx.x / both : 0, first = threadIdx.x - which * both;
    if (SHARED && which >= per) return;
    if (!SHARED) per = 1;
    const uint32_t parts = a.page / 16;   // of 16 tokens
    for (int64_t t = (int64_t)blockIdx.x * per + which; t < a.tokens; t += (int64_t)gridDim.x * per) {
        const int64_t slot = a.slots[t];
        if (slot < 0) continue;
        const uint64_t part = (uint64_t)slot >> 4;
        uint64_t block;
        if constexpr (!SHARED) block = (uint64_t)slot / (uint32_t)a.page;
        else block = part >> 32 ? part / parts : (uint32_t)part / parts;   // (a lane's own: 64 bits are slow)
        if (block >= (uint64_t)a.num_blocks) continue;
        const int64_t at = (int64_t)block * a.block_stride + (slot - (int64_t)block * a.page) * a.token_stride;
        for (int p = first; p < both; p += kAppendThreads) {
            const bool second = p >= pieces;
            const int i = second ? p - pieces : p, h = i / row_pieces;
            const int64_t to = at + h * a.head_stride + (i - h * row_pieces) * 16;
            const uint8_t *from = second ? a.v + t * a.v_stride : a.k + t * a.k_stride;
            *reinterpret_cast<u32x4 *>((second ? a.v_cache : a.k_cache) + to) =
                *reinterpret_cast<const u32x4 *>(from + (int64_t)i * 16);
        }
    }
}

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t st) {
    const int64_t both = 2 * ((int64_t)a.heads * (a.row_bytes / 16));
    const int per = both < kAppendThreads ? (int)(kAppendThreads / both) : 1;
    const int64_t wgs = (a.tokens + per - 1) / per;
    const unsigned grid = (unsigned)(wgs < 65536 ? wgs : 65536);
    if (per > 1) kv_append_kernel<true><<<grid, kAppendThreads, 0, st>>>(a, per);
    else kv_append_kernel<false><<<grid, kAppendThreads, 0, st>>>(a, 1);
    return hipGetLastError();
}

}  // namespace mnb

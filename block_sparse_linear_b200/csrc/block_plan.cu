// Block tables and slot maps from request lengths: the paged cache's block allocator
// on the device, so that a serving step (or a captured graph of one) needs no host
// round trip to grow its sequences. With B tokens a block, len_b tokens held and n_b
// new ones,
//   have_b  = ceil(len_b / B),   need_b = ceil((len_b + n_b) / B) - have_b
//   upto_b  = need_0 + ... + need_b                             (inclusive scan)
//   granted = need_b == 0 or upto_b <= free                     (in line: no overtaking)
//   table[b][have_b + j] = free_list[free - 1 - (upto_b - need_b) - j],  0 <= j < need_b
//   position(b, t) = len_b + t,   slot(b, t) = table[b][position / B] * B + position % B
// The free list is a stack; a release pushes a sequence's blocks back in table order.
//
// Everything is a few integers per sequence and 12 bytes per padded token, so a decode
// step is bound by its dependent round trips (lengths and counts; free-list entries;
// table entries), and one CTA that keeps the scan in shared memory is the fewest of
// them. The row outputs of a prefill wave (12 bytes a token, megabytes) go to a second
// launch over the whole GPU once they pass kPlanRowsInline entries: below that the one
// CTA writes them itself, which saves the launch.
#include "common.cuh"

namespace spla {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int64_t kPlanRowsInline = 4096;       // four per thread of the one CTA
constexpr int kRowsThreads = 256;
constexpr int kRowsPerCta = 4 * kRowsThreads;

struct BlockPoolView {
    int32_t* table;          // [batch][mbp]
    int32_t* free_list;      // [num_phys], a stack of *free_count entries
    int32_t* free_count;     // [1]
    int32_t batch, mbp, num_phys, bs;
};

// Inclusive scan of `x` over the CTA (x >= 0); *total gets the sum. One barrier before
// the shared partials are reused is the caller's.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_tot, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    int64_t below = 0, all = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        const int64_t t = warp_tot[w];
        if (w < warp) below += t;
        all += t;
    }
    *total = all;
    return v + below;
}

// Position and slot of new token t of sequence b; reads the (just written) table.
__device__ __forceinline__ void plan_row(const BlockPoolView& p, int64_t i, int b, int t, int n,
                                         int len, int32_t* positions, int64_t* slots,
                                         int32_t* status) {
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < n) {
        pos = len + t;
        if (slots) {
            const int lb = pos / p.bs;
            const int32_t phys = p.table[(int64_t)b * p.mbp + lb];
            if (phys >= 0 && phys < p.num_phys)
                slot = (int64_t)phys * p.bs + (pos - lb * p.bs);
            else
                set_status(status, SPLA_DEV_BAD_BLOCK_TABLE);
        }
    }
    if (positions) positions[i] = pos;
    if (slots) slots[i] = slot;
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(BlockPoolView p, const int32_t* lens, const int32_t* n_new, int32_t max_new,
            int32_t* n_granted, int32_t* lens_after, int32_t* positions, int64_t* slots,
            int32_t* free_out, int rows_inline, int32_t* status) {
    __shared__ int64_t warp_tot[kPlanWarps];
    __shared__ int32_t s_taken, s_base, s_end[kPlanThreads], s_dst[kPlanThreads];
    const int tid = threadIdx.x;
    if (tid == 0) {
        s_taken = 0;
        s_base = 0;
    }
    pdl_wait();
    pdl_trigger();
    const int64_t cap = (int64_t)p.mbp * p.bs;
    int32_t nfree = *p.free_count;
    if (nfree < 0 || nfree > p.num_phys) {
        if (tid == 0) set_status(status, SPLA_DEV_CAPACITY);
        nfree = 0;
    }
    int64_t carry = 0;                          // blocks asked for by earlier rounds
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int32_t len = 0, n = 0, have = 0, need = 0;
        if (b < p.batch) {
            len = lens[b];
            n = n_new[b];
            int32_t bad = 0;
            if (n < 0 || n > max_new) bad = SPLA_DEV_BAD_COUNT;
            else if (len < 0 || (int64_t)len + n > cap) bad = SPLA_DEV_CAPACITY;
            if (bad) {
                set_status(status, bad);
                n = 0;
            } else {
                have = (int)(((int64_t)len + p.bs - 1) / p.bs);
                need = (int)(((int64_t)len + n + p.bs - 1) / p.bs) - have;
            }
        }
        int64_t asked;
        const int64_t upto = carry + block_scan(need, warp_tot, &asked);
        carry += asked;
        if (need && upto > nfree) {
            set_status(status, SPLA_DEV_NO_BLOCKS);
            n = 0;
            need = 0;
        }
        if (need) atomicMax(&s_taken, (int32_t)upto);
        if (b < p.batch) {
            n_granted[b] = n;
            if (lens_after) lens_after[b] = len + n;
        }
        // The round's new blocks in a row, entry i from the stack's place free - 1 - i: the
        // threads take consecutive entries (coalesced) and find each one's sequence by its
        // end in the scan. s_dst + i is the entry's place in its table row.
        const int32_t before = s_base;
        __syncthreads();                        // s_taken is final, s_base read
        s_end[tid] = (int32_t)min(upto, (int64_t)s_taken);
        s_dst[tid] = have - (int32_t)(upto - need);
        if (tid == 0) s_base = s_taken;
        __syncthreads();
        for (int32_t i0 = before + tid; i0 < s_taken; i0 += 4 * kPlanThreads) {
            int32_t blk[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t i = i0 + u * kPlanThreads;
                blk[u] = i < s_taken ? p.free_list[nfree - 1 - i] : 0;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t i = i0 + u * kPlanThreads;
                if (i >= s_taken) break;
                int lo = 0;                     // the first sequence whose end is past i
#pragma unroll
                for (int w = kPlanThreads / 2; w; w >>= 1)
                    if (s_end[lo + w - 1] <= i) lo += w;
                p.table[(int64_t)(b0 + lo) * p.mbp + s_dst[lo] + i] = blk[u];
            }
        }
        __syncthreads();                        // warp_tot is free again; table rows visible
    }
    if (tid == 0) *free_out = nfree - s_taken;
    if (!rows_inline) return;
    const int64_t rows = (int64_t)p.batch * max_new;
    for (int64_t i = tid; i < rows; i += kPlanThreads) {
        const int b = (int)(i / max_new), t = (int)(i - (int64_t)b * max_new);
        const int32_t n = n_granted[b];
        plan_row(p, i, b, t, n, n > 0 ? lens[b] : 0, positions, slots, status);
    }
}

// Row outputs over the whole GPU: grid (token tiles, batch).
__global__ void __launch_bounds__(kRowsThreads)
plan_rows_kernel(BlockPoolView p, const int32_t* lens, const int32_t* n_granted, int32_t max_new,
                 int32_t* positions, int64_t* slots, int32_t* status) {
    pdl_trigger();
    pdl_wait();
    for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const int32_t n = n_granted[b];
        const int32_t len = n > 0 ? lens[b] : 0;
        const int64_t t0 = (int64_t)blockIdx.x * kRowsPerCta + threadIdx.x;
#pragma unroll
        for (int u = 0; u < kRowsPerCta / kRowsThreads; ++u) {
            const int64_t t = t0 + u * kRowsThreads;
            if (t < max_new)
                plan_row(p, (int64_t)b * max_new + t, b, (int)t, n, len, positions, slots, status);
        }
    }
}

// Blocks past keep_lens[b] tokens go back to the stack; one CTA, a thread per sequence
// for the scan, a warp per 32 sequences for their entries, one sequence after another (a look
// over the entries, then the push). Bound by those rounds of loads in a row: a sequence of
// 16384 blocks takes 109 us, 256 of 64 blocks 25 us, drafts given back about 10 us.
__global__ void __launch_bounds__(kPlanThreads)
release_kernel(BlockPoolView p, const int32_t* keep_lens, int32_t* lens, int32_t* status) {
    __shared__ int64_t warp_tot[kPlanWarps];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    const int64_t cap = (int64_t)p.mbp * p.bs;
    const int32_t nfree = *p.free_count;
    if (nfree < 0 || nfree > p.num_phys) {
        if (tid == 0) set_status(status, SPLA_DEV_CAPACITY);
        return;
    }
    int64_t pushed = nfree;                     // stack height reached by earlier rounds
    int64_t offered = nfree;                    // what it would be with the refused ones too
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int32_t first = 0, gone = 0, keep = -1;
        if (b < p.batch) {
            const int32_t len = lens[b];
            keep = keep_lens[b];
            if (keep < 0) set_status(status, SPLA_DEV_BAD_COUNT);
            else if (len < 0 || len > cap) { set_status(status, SPLA_DEV_CAPACITY); keep = -1; }
            else if (keep >= len) keep = -1;    // nothing to give back
            if (keep >= 0) {
                first = (int)(((int64_t)keep + p.bs - 1) / p.bs);
                gone = (int)(((int64_t)len + p.bs - 1) / p.bs) - first;
            }
        }
        // a sequence with an entry outside the pool keeps its blocks
        bool good = true;
        for (int s = 0; s < 32; ++s) {
            const int sn = __shfl_sync(0xffffffffu, gone, s);
            const int sf = __shfl_sync(0xffffffffu, first, s);
            const int32_t* row = p.table + (int64_t)(b - lane + s) * p.mbp + sf;
            bool ok = true;
            for (int j = lane; j < sn; j += 32) ok = ok && row[j] >= 0 && row[j] < p.num_phys;
            ok = __all_sync(0xffffffffu, ok);
            if (lane == s) good = ok;
        }
        if (!good) {
            set_status(status, SPLA_DEV_BAD_BLOCK_TABLE);
            gone = 0;
            keep = -1;
        }
        int64_t total;
        const int64_t end = offered + block_scan(gone, warp_tot, &total);
        offered += total;
        // more blocks than the pool has: something was given back twice; this sequence
        // and the ones after it are left as they are
        if (gone && end > p.num_phys) {
            set_status(status, SPLA_DEV_CAPACITY);
            gone = 0;
            keep = -1;
        }
        const int32_t at = (int32_t)(end - gone);
        for (int s = 0; s < 32; ++s) {
            const int sn = __shfl_sync(0xffffffffu, gone, s);
            const int sf = __shfl_sync(0xffffffffu, first, s);
            const int sa = __shfl_sync(0xffffffffu, at, s);
            int32_t* row = p.table + (int64_t)(b - lane + s) * p.mbp + sf;
            for (int j = lane; j < sn; j += 32) {
                p.free_list[sa + j] = row[j];
                row[j] = -1;
            }
        }
        if (keep >= 0) lens[b] = keep;
        __syncthreads();
        // height after this round: the largest end that was pushed
        int64_t* top = warp_tot;
        const unsigned hi = __reduce_max_sync(0xffffffffu, gone ? (unsigned)(end) : (unsigned)pushed);
        if (lane == 0) top[tid >> 5] = hi;
        __syncthreads();
        for (int w = 0; w < kPlanWarps; ++w) pushed = pushed > top[w] ? pushed : top[w];
        __syncthreads();
    }
    if (tid == 0) *p.free_count = (int32_t)pushed;
}

// ------------------------------------------------------------------ host launchers
static BlockPoolView pool_view(const spla_block_pool* q) {
    BlockPoolView p;
    p.table = q->block_table;
    p.free_list = q->free_list;
    p.free_count = q->free_count;
    p.batch = q->batch;
    p.mbp = q->max_blocks_per_seq;
    p.num_phys = q->num_phys_blocks;
    p.bs = q->block_size;
    return p;
}

cudaError_t launch_block_plan(const spla_block_pool* pool, const int32_t* lens,
                              const int32_t* n_new, int32_t max_new, int32_t* n_granted,
                              int32_t* lens_after, int32_t* positions, int64_t* slots,
                              int32_t* free_out, int32_t* status, cudaStream_t s) {
    const BlockPoolView p = pool_view(pool);
    const int64_t rows = positions || slots ? (int64_t)p.batch * max_new : 0;
    const int rows_inline = rows > 0 && rows <= kPlanRowsInline;
    cudaError_t e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, lens, n_new,
                               max_new, n_granted, lens_after, positions, slots, free_out,
                               rows_inline, status);
    if (e != cudaSuccess || rows == 0 || rows_inline) return e;
    const int tiles = (int)(((int64_t)max_new + kRowsPerCta - 1) / kRowsPerCta);
    return launch_pdl(plan_rows_kernel, dim3(tiles, p.batch < 65535 ? p.batch : 65535),
                      dim3(kRowsThreads), 0, s, p, lens, n_granted, max_new, positions, slots,
                      status);
}

cudaError_t launch_block_release(const spla_block_pool* pool, const int32_t* keep_lens,
                                 int32_t* lens, int32_t* status, cudaStream_t s) {
    return launch_pdl(release_kernel, dim3(1), dim3(kPlanThreads), 0, s, pool_view(pool),
                      keep_lens, lens, status);
}

}  // namespace spla

// Block tables, slot maps, positions and per-token adapter ids of a step from
// its requests' lengths.
//
// With before_r = ceil(past_r / b) and after_r = ceil((past_r + new_r) / b), a
// request takes after_r - before_r pages (less those that its row holds beyond
// before_r, where the caller says how many it holds); rows and pages are handed out by two
// prefix sums over the requests.  Row t belongs to the request whose row range
// holds it (a binary search in the sums), its token to block pos / b of that
// request: a page of the free list if that block is new, else an entry of the
// block table that was there before the call.
//
// A few hundred KB at most move, so latency bounds it.  One launch: every CTA
// forms both sums itself (R <= 4096 lengths from L2, 16 per thread) and then
// takes its share of the rows and new blocks, which needs no exchange between
// CTAs: new blocks are read from the free list, never from the table entry
// that another CTA may still be writing.  64 requests take 3.7 us, 1024 take 5.7 us.
#include "lora_internal.cuh"
#include "lora_kv.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;

struct Sums {
    long long rows, pages;
};

struct Need {
    int rows, pages;   // rows the request brings, pages it takes
    int after;         // blocks it has afterwards
    bool bad;          // its lengths are refused
};

// Blocks of a request that are there before the call; the next one takes the first of its pages.
__device__ __forceinline__ int blocks_before(const LayoutArgs &a, int past, int held) {
    return max((past + a.block - 1) / a.block, held);
}

__device__ __forceinline__ Need need_of(const LayoutArgs &a, int past, int fresh, int held) {
    Need n;
    n.rows = fresh < 0 ? 0 : fresh;
    n.bad = past < 0 || fresh < 0 || (long long)past + fresh > (long long)a.max_blocks * a.block || held < 0 || held > a.max_blocks;
    n.pages = n.after = 0;
    if (n.bad) return n;
    const int before = blocks_before(a, past, held);
    n.after = max(before, (past + fresh + a.block - 1) / a.block);
    if (a.free_pages) n.pages = n.after - before;
    return n;
}

// First request whose running sum exceeds x.
__device__ __forceinline__ int owner(const int *ends, int R, int x) {
    int lo = 0, hi = R;
    while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (ends[m] > x) hi = m;
        else lo = m + 1;
    }
    return lo;
}

template <bool HELD>
__global__ void __launch_bounds__(kThreads) kv_layout_kernel(LayoutArgs a) {
    const auto held_of = [&](int r) { return HELD ? a.held[r] : 0; };
    extern __shared__ int sm[];
    int *row_end = sm, *page_end = sm + a.R;                                   // running sums
    unsigned char *failed = reinterpret_cast<unsigned char *>(sm + 2 * a.R);   // per request
    __shared__ Sums warp_sum[kThreads / 32];
    __shared__ int last_page;                                                  // pages handed out
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.R + kThreads - 1) / kThreads, r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
    if (tid == 0) last_page = 0;

    Sums mine{0, 0};
    for (int r = r0; r < r1; ++r) {
        const Need n = need_of(a, a.past[r], a.fresh_len[r], held_of(r));
        mine.rows += n.rows;
        mine.pages += n.pages;
    }
    Sums run = mine;   // inclusive over the warp, then exclusive over the block
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(~0u, run.rows, d), y = __shfl_up_sync(~0u, run.pages, d);
        if (lane >= d) {
            run.rows += x;
            run.pages += y;
        }
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    run.rows -= mine.rows;
    run.pages -= mine.pages;
    for (int w = 0; w < warp; ++w) {
        run.rows += warp_sum[w].rows;
        run.pages += warp_sum[w].pages;
    }
    const int head = a.free_head ? *a.free_head : 0;
    const int avail = head < 0 || head > a.num_free ? 0 : a.num_free - head;
    int flags = head < 0 || head > a.num_free ? LORA_DEV_ERR_NO_PAGES : 0;
    for (int r = r0; r < r1; ++r) {
        const int past = a.past[r], fresh = a.fresh_len[r], held = held_of(r);
        const Need n = need_of(a, past, fresh, held);
        run.rows += n.rows;
        run.pages += n.pages;
        bool f = n.bad || (n.rows > 0 && run.rows > a.T);
        if (f) flags |= LORA_DEV_ERR_BAD_LENGTH;
        if (n.pages > 0 && run.pages > avail) {
            if (!f) flags |= LORA_DEV_ERR_NO_PAGES;
            f = true;
        }
        row_end[r] = (int)min(run.rows, (long long)a.T);
        page_end[r] = (int)min(run.pages, (long long)INT32_MAX);
        failed[r] = f;
        if (!f && n.pages > 0) atomicMax(&last_page, (int)run.pages);
        if (blockIdx.x == 0) {
            if (r == 0) a.cu[0] = 0;
            a.cu[r + 1] = row_end[r];
            a.kv_len[r] = f ? 0 : past + fresh;
            if (HELD) a.held_out[r] = f ? held : n.after;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (flags && a.err) atomicOr(a.err, flags);
        if (tid == 0 && a.head_out) *a.head_out = head + last_page;
    }

    // 32 bits without a sign: a last step beyond 2^31 rows does not turn back
    const unsigned me = blockIdx.x * kThreads + tid, all = gridDim.x * kThreads;
    for (unsigned j = me; j < (unsigned)last_page; j += all) {
        const int r = owner(page_end, a.R, (int)j);
        if (failed[r]) continue;
        const int start = r ? page_end[r - 1] : 0;
        a.table[(size_t)r * a.max_blocks + blocks_before(a, a.past[r], held_of(r)) + j - start] = a.free_pages[head + j];
    }
    const unsigned used = row_end[a.R - 1];
    for (unsigned t = me; t < (unsigned)a.T; t += all) {
        int pos = -1, slot = -1, id = -1;
        const int r = t < used ? owner(row_end, a.R, (int)t) : 0;
        if (t < used && !failed[r]) {
            const int past = a.past[r], before = blocks_before(a, past, held_of(r));
            pos = past + (int)t - (r ? row_end[r - 1] : 0);
            const int blk = pos / a.block;
            const int page = a.free_pages && blk >= before ? a.free_pages[head + (r ? page_end[r - 1] : 0) + blk - before]
                                                           : a.table[(size_t)r * a.max_blocks + blk];
            // a page whose slots would pass 31 bits cannot be in any cache
            if (page < 0 || (long long)(page + 1LL) * a.block > INT32_MAX) {
                if (a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_PAGE);
            } else {
                slot = page * a.block + pos % a.block;
            }
            if (a.req_ids) id = a.req_ids[r];
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
        if (a.ids) a.ids[t] = id;
    }
}

}  // namespace

int launch_kv_layout(const LayoutArgs &a, cudaStream_t st) {
    const int work = a.T > a.R ? a.T : a.R;
    int grid = (work - 1) / kThreads + 1;   // R is at least 1
    if (grid > 592) grid = 592;
    const size_t smem = (size_t)a.R * 9;
    if (a.held) kv_layout_kernel<true><<<grid, kThreads, smem, st>>>(a);
    else kv_layout_kernel<false><<<grid, kThreads, smem, st>>>(a);
    count_launch();
    return cuda_check(cudaGetLastError());
}

}  // namespace lora

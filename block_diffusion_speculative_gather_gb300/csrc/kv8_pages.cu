// Page plans of the 8-bit paged KV cache: block tables, row maps and slot
// maps built on the device from the sequences' lengths, and the way back.
//
// The work is a few kilobytes of integers; the calls are bound by launch and
// memory latency.  One CTA scans the sequences (two exclusive sums at once:
// pages and rows), so admission "in order while it fits" needs no exchange
// between CTAs; the row maps, which can be long, are filled by the same CTA
// while they are short and by a second launch over all SMs otherwise.
// 32 sequences, 316 rows: 3.6 us; 2048 sequences, 82582 rows: 8.3 us in
// two launches.

#include "gemm.cuh"
#include "kv8.cuh"

namespace dfl {
namespace {

constexpr int PT = 1024;           // threads of the scan
constexpr int PLAN_SMEM_SEQS = 4096;   // row starts kept in shared memory up to here
// Rows that the scanning CTA fills itself: a second launch costs about 2 us,
// one pass of 1024 threads over their rows (three dependent loads) about 1.
constexpr int PLAN_INLINE_ROWS = 4096;

struct Two {
    long long pages, rows;
};

__device__ __forceinline__ Two shfl_up2(Two v, int o) {
    return {__shfl_up_sync(0xffffffffu, v.pages, o), __shfl_up_sync(0xffffffffu, v.rows, o)};
}

// Exclusive sums over the CTA's PT threads, and the totals.
__device__ Two block_scan(Two v, Two* total, Two* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Two inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two u = shfl_up2(inc, o);
        if (lane >= o) {
            inc.pages += u.pages;
            inc.rows += u.rows;
        }
    }
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        Two w = sm[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Two u = shfl_up2(w, o);
            if (lane >= o) {
                w.pages += u.pages;
                w.rows += u.rows;
            }
        }
        sm[lane] = w;
    }
    __syncthreads();
    const Two before = warp ? sm[warp - 1] : Two{0, 0};
    *total = sm[31];
    __syncthreads();
    return {before.pages + inc.pages - v.pages, before.rows + inc.rows - v.rows};
}

__device__ __forceinline__ int pages_of(int len) { return (int)(((long long)len + KV8_PAGE - 1) / KV8_PAGE); }

// Row r's sequence: the last s with start[s] <= r.
__device__ __forceinline__ int find_seq(const int* start, int S, int r) {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void fill_row(const PagesPlanArgs& a, const int* start, int total, int r) {
    int pos = -1, slot = -1;
    if (r < total) {
        const int s = find_seq(start, a.S, r);
        const int r0 = start[s], n = start[s + 1] - r0;
        pos = a.kv_after[s] - n + (r - r0);
        const int page = a.table[(size_t)s * a.max_pages + pos / KV8_PAGE];
        if (page >= 0 && page < (1 << 25)) slot = page * KV8_PAGE + pos % KV8_PAGE;
    }
    a.positions[r] = pos;
    a.slots[r] = slot;
}

__global__ void __launch_bounds__(PT) pages_plan_kernel(PagesPlanArgs a, int inline_rows) {
    __shared__ Two sm[32];
    __shared__ int s_start[PLAN_SMEM_SEQS + 1];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    int n_free = a.n_free[0];
    n_free = n_free < 0 ? 0 : (n_free > a.free_cap ? a.free_cap : n_free);
    Two carry{0, 0}, granted{0, 0};
    for (int base = 0; base < a.S; base += PT) {
        const int s = base + tid;
        int kv = 0, q = 0, old = 0, need = 0;
        bool fine = false;
        if (s < a.S) {
            kv = a.kv_len[s];
            q = a.q_len[s];
            // lengths that are negative, or a table row that cannot hold them, get nothing
            fine = kv >= 0 && q >= 0 && (long long)kv + q <= (long long)a.max_pages * KV8_PAGE;
            if (fine) {
                old = pages_of(kv);
                need = pages_of(kv + q) - old;
            }
        }
        Two total;
        const Two before = block_scan(Two{need, fine ? q : 0}, &total, sm);
        const long long p0 = carry.pages + before.pages, r0 = carry.rows + before.rows;
        // the sums only grow, so the sequences that fit are a prefix of the valid ones
        const bool ok = fine && p0 + need <= n_free && r0 + q <= a.rows;
        if (!ok) need = q = 0;
        // pages handed out and rows given before this sequence: the same sums,
        // since everything valid before an admitted sequence was admitted
        Two got;
        const Two given = block_scan(Two{need, q}, &got, sm);
        const long long pg = granted.pages + given.pages, rg = granted.rows + given.rows;
        if (s < a.S) {
            a.row_start[s] = (int)rg;
            if (s < PLAN_SMEM_SEQS) s_start[s] = (int)rg;
            a.kv_after[s] = kv + q;
        }
        // new entries: a lane its own sequence's while they are few (their loads
        // are in flight together), else a warp's lanes share each sequence's
        int most = need;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const int other = __shfl_xor_sync(0xffffffffu, most, o);
            most = most > other ? most : other;
        }
        if (most <= 8) {
            for (int i = 0; i < need; ++i)
                a.table[(size_t)s * a.max_pages + old + i] = a.free_pages[n_free - 1 - pg - i];
        }
        unsigned todo = __ballot_sync(0xffffffffu, most > 8 && need > 0);
        while (todo) {
            const int l = __ffs(todo) - 1;
            todo &= todo - 1;
            const int n = __shfl_sync(0xffffffffu, need, l), o = __shfl_sync(0xffffffffu, old, l);
            const int ss = __shfl_sync(0xffffffffu, s, l);
            const long long p = __shfl_sync(0xffffffffu, pg, l);
            for (int i = lane; i < n; i += 32)
                a.table[(size_t)ss * a.max_pages + o + i] = a.free_pages[n_free - 1 - p - i];
        }
        carry = {carry.pages + total.pages, carry.rows + total.rows};
        granted = {granted.pages + got.pages, granted.rows + got.rows};
    }
    const int total = (int)granted.rows;
    if (tid == 0) {
        a.row_start[a.S] = total;
        if (a.S <= PLAN_SMEM_SEQS) s_start[a.S] = total;
        a.n_free_out[0] = n_free - (int)granted.pages;
    }
    if (!inline_rows) return;
    __syncthreads();   // row starts, lengths and table entries of this CTA
    const int* start = a.S <= PLAN_SMEM_SEQS ? s_start : a.row_start;
    for (int r = tid; r < a.rows; r += PT) fill_row(a, start, total, r);
}

// Row maps of one sequence a CTA column (blockIdx.x, its rows dealt over
// blockIdx.y), then this CTA's share of the rows behind the last.
__global__ void pages_rows_kernel(PagesPlanArgs a) {
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, step = gridDim.y * blockDim.x;
    const int r0 = a.row_start[s], n = a.row_start[s + 1] - r0, total = a.row_start[a.S];
    const int p0 = a.kv_after[s] - n;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < n; i += step) {
        const int pos = p0 + i, page = a.table[(size_t)s * a.max_pages + pos / KV8_PAGE];
        a.positions[r0 + i] = pos;
        a.slots[r0 + i] = page >= 0 && page < (1 << 25) ? page * KV8_PAGE + pos % KV8_PAGE : -1;
    }
    const long long all = (long long)gridDim.x * step;
    for (long long r = total + ((long long)blockIdx.y * gridDim.x + s) * blockDim.x + threadIdx.x; r < a.rows; r += all) {
        a.positions[r] = -1;
        a.slots[r] = -1;
    }
}

__global__ void __launch_bounds__(PT) pages_trim_kernel(PagesTrimArgs a) {
    __shared__ Two sm[32];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    long long n_free = a.n_free[0];
    if (n_free < 0) n_free = 0;
    for (int base = 0; base < a.S; base += PT) {
        const int s = base + tid;
        int first = 0, back = 0;
        if (s < a.S) {
            int kv = a.kv_len[s], to = a.new_len[s];
            if (to < 0) to = 0;
            if (kv > to && kv <= (long long)a.max_pages * KV8_PAGE) {
                first = pages_of(to);
                back = pages_of(kv) - first;
                a.kv_len[s] = to;
            }
        }
        Two total;
        const Two before = block_scan(Two{back, 0}, &total, sm);
        unsigned todo = __ballot_sync(0xffffffffu, back > 0);
        while (todo) {
            const int l = __ffs(todo) - 1;
            todo &= todo - 1;
            const int n = __shfl_sync(0xffffffffu, back, l), f = __shfl_sync(0xffffffffu, first, l);
            const int ss = __shfl_sync(0xffffffffu, s, l);
            const long long p = n_free + __shfl_sync(0xffffffffu, before.pages, l);
            for (int i = lane; i < n; i += 32) {
                int* e = a.table + (size_t)ss * a.max_pages + f + i;
                // the last page goes back first: it is the first handed out again
                const long long at = p + n - 1 - i;
                if (at < a.free_cap) a.free_pages[at] = *e;
                *e = -1;
            }
        }
        n_free += total.pages;
    }
    __syncthreads();
    if (tid == 0) a.n_free[0] = (int)(n_free > a.free_cap ? a.free_cap : n_free);
}

}  // namespace

int launch_pages_plan(const PagesPlanArgs& a, cudaStream_t s) {
    const int inl = a.rows <= PLAN_INLINE_ROWS;
    cudaError_t e = launch_k(pages_plan_kernel, dim3(1), dim3(PT), 0, s, a, inl);
    if (e == cudaSuccess && !inl) {
        // a CTA of 64 threads a sequence, more where they have many rows
        const int each = (a.rows + a.S - 1) / a.S, tpb = each > 128 ? 256 : 64;
        int y = (each + tpb - 1) / tpb;
        y = y > 64 ? 64 : y;
        e = launch_k(pages_rows_kernel, dim3(a.S, y), dim3(tpb), 0, s, a);
    }
    return (int)e;
}

int launch_pages_trim(const PagesTrimArgs& a, cudaStream_t s) {
    return (int)launch_k(pages_trim_kernel, dim3(1), dim3(PT), 0, s, a);
}

}  // namespace dfl

// Page tables, slots and positions of a paged KV cache, built on the device from the requests'
// lengths (the host counterpart is model.KvPagePool: the same pages in the same order).
//
// The free pages are a stack.  Finished requests (n_new = -1) push theirs, a request's last page
// first; then every other request b pops the pages its ctx_len[b] + n_new[b] positions need beyond
// the held[b] it has, in request order.  With R pages pushed and F free before, the k-th page
// popped is stack entry F + R - 1 - k, so two exclusive sums over the requests (pages pushed, pages
// popped) tell every request its pages, and a third one (rows) tells every new row its request.
//
// Up to PG_SMALL requests, one kernel: every CTA forms the three sums for itself in shared memory (a few
// KB from L2) and takes its share of the requests' page moves and of the rows, a warp's worth at a time.
// An entry it pops is read from the stack below F or, at F and above, from the table row of the request
// that pushed it, and nothing it reads is written by another CTA: the stack is written at F and above, a
// table row past its request's held pages, a finished request's row not at all; new counters that take the
// old ones' place are written by the CTA that is the last to have read those, as an atomic with acquire and
// release tells (in place 3.5 us for 8 requests without rows and 4.0 for 500, apart 2.9 and 3.5).
// More requests: a first kernel (one CTA) leaves the sums in the workspace for the second; 1025 requests with a
// row each 7.8 us, 8000 21, 65535 149, where the one CTA's 64 turns of sums are nearly all of it.
// All of it is latency, a chain of dependent reads: 8 requests 4.8 us as two kernels and 3.6 as one, 500
// requests with 14,371 rows 6.8 and 4.5, 1024 requests with 71,545 rows 7.6 and 7.4.
#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

constexpr int PG_THREADS = 1024;   // kernel 1
constexpr int PG_WORK = 256;       // kernel 2
constexpr int PG_SMALL = 1024;     // requests the single kernel takes

struct PagesArgs {
    int32_t* table;
    int page, max_pages, n_pages;
    int32_t* free_pages;
    const int32_t* n_free_in;
    int32_t* n_free_out;
    const int32_t* held_in;
    int32_t* held_out;
    const int32_t* ctx_len;
    const int32_t* n_new;
    int B;
    int32_t* row_start;
    int32_t* pos;
    long long* slots;
    int max_rows;
    bool in_place;   // new counters in the old ones' place
    // workspace: [0] CTAs that have read those (zero between calls); for more than PG_SMALL requests
    // [1] free pages before, [2] pages pushed, [3] bit 0 pages may be pushed, bit 1 popped, then the sums
    int32_t* ws;
    unsigned* err;
};

// The sums over the requests, in the workspace or in shared memory, and what follows from them.
struct PagesSums {
    int32_t *held, *need, *push, *pop;   // pages held before; needed (-1: finished); first push; first pop
    const int32_t* start;                // [B + 1] first rows
    int F, R;                            // free pages before, pages pushed
    bool push_ok, pop_ok;
};
__device__ __forceinline__ PagesSums ws_sums(const PagesArgs& A) {
    int32_t* w = A.ws + 4;
    const long long B = A.B;
    return PagesSums{w, w + B, w + 2 * B, w + 3 * B, A.row_start, A.ws[1], A.ws[2], (A.ws[3] & 1) != 0, (A.ws[3] & 2) != 0};
}

// Exclusive sums of three values over the CTA's threads; tot receives the CTA's totals.  Every
// request's values are at most 2^30, so the sums are formed in 64 bits.
__device__ __forceinline__ void block_scan3(long long v[3], long long tot[3], long long (*sm)[33]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long inc[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        inc[q] = v[q];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc[q], off);
            if (lane >= off) inc[q] += o;
        }
        if (lane == 31) sm[q][w] = inc[q];
    }
    __syncthreads();
    if (w < 3) {
        long long x = lane < PG_THREADS / 32 ? sm[w][lane] : 0, s = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += o;
        }
        sm[w][lane] = s - x;
        if (lane == 31) sm[w][32] = s;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        v[q] = sm[q][w] + inc[q] - v[q];
        tot[q] = sm[q][32];
    }
    __syncthreads();
}

// The sums of all requests by one CTA of PG_THREADS, into P's arrays and `start` [B + 1]; rows are
// clamped to max_rows.  report: record what is out of range, and *popped = the pages popped.
__device__ __forceinline__ void pages_scan(const PagesArgs& A, PagesSums& P, int32_t* start, bool report, int* popped) {
    __shared__ long long sm[3][33];
    const int tid = threadIdx.x;
    const int F0 = *A.n_free_in;
    const bool sane = F0 >= 0 && F0 <= A.n_pages;
    P.F = sane ? F0 : 0;
    const long long cap = static_cast<long long>(A.page) * A.max_pages;
    long long carry[3] = {0, 0, 0};   // pushed, popped, rows
    unsigned bad = sane ? 0u : ERR_BAD_COUNT;
    for (int b0 = 0; b0 < A.B; b0 += PG_THREADS) {
        const int b = b0 + tid;
        long long v[3] = {0, 0, 0};
        int held = 0, need = 0;
        if (b < A.B) {
            held = A.held_in[b];
            int n = A.n_new[b];
            const int ctx = A.ctx_len[b];
            if (held < 0 || held > A.max_pages) {
                bad |= ERR_BAD_COUNT;
                held = held < 0 ? 0 : A.max_pages;
            }
            if (n == -1) {
                v[0] = held;
                need = -1;
            } else {
                if (n < -1 || ctx < 0 || static_cast<long long>(ctx) + n > cap) {
                    bad |= n < -1 ? ERR_BAD_COUNT : ERR_BAD_LENGTH;
                    n = 0;
                } else {
                    need = static_cast<int>((static_cast<long long>(ctx) + n + A.page - 1) / A.page);
                }
                v[1] = need > held ? need - held : 0;
                v[2] = n;
            }
        }
        long long tot[3];
        block_scan3(v, tot, sm);
        if (b < A.B) {
            P.held[b] = held;
            P.need[b] = need;
            // sums past the pool or past int are refused below; clamp what is stored
            P.push[b] = static_cast<int32_t>(min(carry[0] + v[0], 1ll << 30));
            P.pop[b] = static_cast<int32_t>(min(carry[1] + v[1], 1ll << 30));
            start[b] = static_cast<int32_t>(min(carry[2] + v[2], static_cast<long long>(A.max_rows)));
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) carry[q] += tot[q];
    }
    P.push_ok = sane && P.F + carry[0] <= A.n_pages;
    P.R = P.push_ok ? static_cast<int>(carry[0]) : 0;
    P.pop_ok = P.push_ok && carry[1] <= P.F + P.R;
    *popped = P.pop_ok ? static_cast<int>(carry[1]) : 0;
    if (!P.push_ok) bad |= ERR_BAD_COUNT;
    if (P.push_ok && !P.pop_ok) bad |= ERR_NO_PAGES;
    if (carry[2] > A.max_rows) bad |= ERR_BAD_COUNT;
    if (report && bad) atomicOr(A.err, bad);
    if (tid == 0) start[A.B] = static_cast<int32_t>(min(carry[2], static_cast<long long>(A.max_rows)));
    if (!sane) P.F = F0;   // handed back as it is (nothing is popped)
}

// held and n_free after the call; they may be the arrays the scan has read.
__device__ __forceinline__ void pages_finish(const PagesArgs& A, const PagesSums& P, int popped) {
    for (int b = threadIdx.x; b < A.B; b += PG_THREADS) {
        const int held = P.held[b], need = P.need[b];
        A.held_out[b] = need < 0 ? (P.push_ok ? 0 : held) : (P.pop_ok && need > held ? need : held);
    }
    if (threadIdx.x == 0) *A.n_free_out = P.F + P.R - popped;
}

// The last request b in [0, B) with start[b] <= x, by a 32-way search of the whole warp (start is
// nondecreasing, start[0] <= x).
__device__ __forceinline__ int warp_find(const int32_t* start, int B, int x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;   // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && start[i] <= x);
        const int k = 31 - __clz(m);   // lane 0 always holds
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}
// The same by one thread.
__device__ __forceinline__ int thread_find(const int32_t* start, int B, int x) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}
// The same from request b on (start[b] <= x), in steps that double: rows of a warp mostly belong to the same
// request or the next, but any number of requests without rows may lie between two of them (1024 requests,
// rows in the first and the last: 40.5 us by single steps, 4.8 so; 65535: 3900 and 151).
__device__ __forceinline__ int thread_find_on(const int32_t* start, int B, int b, int x) {
    int hi = b + 1;
    for (int step = 1; hi < B && start[hi] <= x; step *= 2) {
        b = hi;
        hi += step;
    }
    return b + thread_find(start + b, min(hi, B) - b, x);
}

// Page j of request b after this call, -1 where it has none.
__device__ __forceinline__ int page_of(const PagesArgs& A, const PagesSums& P, int b, int j) {
    const int held = P.held[b];
    if (j < held) return A.table[static_cast<long long>(b) * A.max_pages + j];
    if (!P.pop_ok) return -1;
    const int i = P.F + P.R - 1 - (P.pop[b] + j - held);   // entry of the stack after the pushes
    if (i < P.F) return A.free_pages[i];
    // pushed in this call: the last request that starts at or before it (requests that push
    // nothing share their successor's start, so the last one is the pusher)
    const int x = i - P.F, p = thread_find(P.push, A.B, x);
    return A.table[static_cast<long long>(p) * A.max_pages + P.held[p] - 1 - (x - P.push[p])];
}

// One warp: the pages request b pushes or pops.
__device__ __forceinline__ void move_pages(const PagesArgs& A, const PagesSums& P, int b) {
    const int lane = threadIdx.x & 31, held = P.held[b], need = P.need[b];
    int32_t* row = A.table + static_cast<long long>(b) * A.max_pages;
    if (need < 0) {
        if (!P.push_ok) return;
        const int top = P.F + P.push[b] + held - 1;
        for (int j = lane; j < held; j += 32) {
            const int pg = row[j];
            if (pg < 0 || pg >= A.n_pages) atomicOr(A.err, ERR_BAD_PAGE);
            A.free_pages[top - j] = pg;
        }
    } else if (P.pop_ok) {
        for (int j = held + lane; j < need; j += 32) {
            const int pg = page_of(A, P, b, j);
            if (pg < 0 || pg >= A.n_pages) atomicOr(A.err, ERR_BAD_PAGE);
            row[j] = pg;
        }
    }
}

// One warp: position and slot of rows t0 .. t0 + 31.
__device__ __forceinline__ void write_rows(const PagesArgs& A, const PagesSums& P, int t0, int total) {
    const int first = warp_find(P.start, A.B, t0), t = t0 + (threadIdx.x & 31);
    if (t < total) {
        const int b = thread_find_on(P.start, A.B, first, t);
        const int p = A.ctx_len[b] + t - P.start[b], j = p / A.page;
        int pg = page_of(A, P, b, j);
        if (pg < -1 || pg >= A.n_pages || (pg < 0 && P.pop_ok)) {
            atomicOr(A.err, ERR_BAD_PAGE);
            pg = -1;
        }
        A.pos[t] = p;
        A.slots[t] = pg < 0 ? -1 : static_cast<long long>(pg) * A.page + (p - j * A.page);
    }
    __syncwarp();
}

__global__ void __launch_bounds__(PG_THREADS) kv_pages_kernel(const __grid_constant__ PagesArgs A) {
    griddep_launch();
    __shared__ int32_t held[PG_SMALL], need[PG_SMALL], push[PG_SMALL], pop[PG_SMALL], start[PG_SMALL + 1];
    __shared__ bool last;
    griddep_wait();
    PagesSums P{held, need, push, pop, start, 0, 0, false, false};
    int popped;
    pages_scan(A, P, start, blockIdx.x == 0, &popped);
    __syncthreads();
    if (threadIdx.x == 0) {
        last = blockIdx.x == 0;
        if (A.in_place) {   // this CTA has read held and n_free: its reads come before the last one's writes
            unsigned n;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(A.ws) : "memory");
            last = n + 1 == gridDim.x;
            if (last) *A.ws = 0;
        }
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b <= A.B; b += PG_THREADS) A.row_start[b] = start[b];
    const int total = start[A.B], W = gridDim.x * (PG_THREADS / 32);
    const long long tasks = A.B + (total + 31ll) / 32;
    for (long long t = blockIdx.x * (PG_THREADS / 32) + (threadIdx.x >> 5); t < tasks; t += W) {
        if (t < A.B) move_pages(A, P, static_cast<int>(t));
        else write_rows(A, P, static_cast<int>(t - A.B) * 32, total);
    }
    __syncthreads();
    if (last) pages_finish(A, P, popped);
}

__global__ void __launch_bounds__(PG_THREADS) kv_pages_scan_kernel(const __grid_constant__ PagesArgs A) {
    griddep_launch();
    griddep_wait();
    int32_t* w = A.ws + 4;
    const long long B = A.B;
    PagesSums P{w, w + B, w + 2 * B, w + 3 * B, A.row_start, 0, 0, false, false};
    int popped;
    pages_scan(A, P, A.row_start, true, &popped);
    pages_finish(A, P, popped);   // a thread reads the entries it wrote itself
    if (threadIdx.x == 0) {
        A.ws[1] = P.F;
        A.ws[2] = P.R;
        A.ws[3] = (P.push_ok ? 1 : 0) | (P.pop_ok ? 2 : 0);
    }
}

// CTAs [0, seq_ctas): a warp per request.  The others: a warp per 32 new rows.
__global__ void __launch_bounds__(PG_WORK) kv_pages_write_kernel(const __grid_constant__ PagesArgs A, int seq_ctas) {
    griddep_launch();
    griddep_wait();
    const int w = threadIdx.x >> 5;
    const PagesSums P = ws_sums(A);
    if (static_cast<int>(blockIdx.x) < seq_ctas) {
        const int b = blockIdx.x * (PG_WORK / 32) + w;
        if (b < A.B) move_pages(A, P, b);
        return;
    }
    const int total = A.row_start[A.B];
    const int t0 = ((static_cast<int>(blockIdx.x) - seq_ctas) * (PG_WORK / 32) + w) * 32;
    if (t0 < total) write_rows(A, P, t0, total);
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

size_t xv_kv_pages_workspace_size(int B) { return B < 1 ? 0 : (16ull + 16ull * B + 255) / 256 * 256; }

xv_status xv_kv_pages_update(int32_t* page_table, int page_size, int max_pages, int n_pages, int32_t* free_pages,
                             const int32_t* n_free, int32_t* n_free_out, const int32_t* held, int32_t* held_out,
                             const int32_t* ctx_len, const int32_t* n_new, int B, int32_t* row_start, int32_t* pos,
                             long long* slots, int max_rows, void* ws, size_t ws_bytes, xv_stream s) {
    if (!free_pages || !n_free || !n_free_out || !held || !held_out || !ctx_len || !n_new || !row_start || !pos || !slots)
        return fail(XV_ERR_ARG, "kv_pages_update: null pointer");
    if (B < 1 || max_rows < 1) return fail(XV_ERR_ARG, "kv_pages_update: need B >= 1 and max_rows >= 1");
    if (B > 65535 || max_rows > (1 << 30)) return fail(XV_ERR_UNSUPPORTED, "kv_pages_update: B above 65535 or max_rows above 2^30");
    KvPages kv{};
    int Lmax = 0;
    const xv_kv_pages pages{page_table, page_size, max_pages, n_pages};
    if (xv_status st = kv_pages_check(&pages, 1, 1, &kv, &Lmax)) return st;
    const size_t need = xv_kv_pages_workspace_size(B);
    if (!ws || ws_bytes < need) return fail(XV_ERR_WORKSPACE, "kv_pages_update: workspace of %zu bytes needed", need);
    if (!aligned16(ws)) return fail(XV_ERR_UNSUPPORTED, "kv_pages_update: workspace must be 16-byte aligned");
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "kv_pages_update: device error word unavailable");
    PagesArgs a{page_table, kv.page, kv.max_pages, kv.n_pages, free_pages, n_free, n_free_out, held, held_out, ctx_len,
                n_new, B, row_start, pos, slots, max_rows, false, static_cast<int32_t*>(ws), err};
    auto overlap = [](const int32_t* x, const int32_t* y, int n) { return x < y + n && y < x + n; };
    a.in_place = overlap(n_free, n_free_out, 1) || overlap(held, held_out, B);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
    if (B <= PG_SMALL) {
        // a warp task per request and per 32 rows, 32 to a CTA, up to an SM's worth of CTAs each
        int sms = 0;
        if (xv_status e = device_sm_count(&sms)) return e;
        const int ctas = ceil_div(B + (max_rows + 31ll) / 32, PG_THREADS / 32);
        trace_pre(st);
        launch_k(kv_pages_kernel, dim3(ctas < sms ? ctas : sms), dim3(PG_THREADS), 0, st, a);
        return launched("kv_pages_kernel", st, K_PAGES, 12ll * max_rows + 48ll * B);
    }
    trace_pre(st);
    launch_k(kv_pages_scan_kernel, dim3(1), dim3(PG_THREADS), 0, st, a);
    if (xv_status e = launched("kv_pages_scan_kernel", st, K_PAGES, 32ll * B)) return e;
    const int seq_ctas = ceil_div(B, PG_WORK / 32);
    trace_pre(st);
    launch_k(kv_pages_write_kernel, dim3(seq_ctas + ceil_div(max_rows, PG_WORK)), dim3(PG_WORK), 0, st, a, seq_ctas);
    return launched("kv_pages_write_kernel", st, K_PAGES, 12ll * max_rows + 16ll * B);
}

}  // extern "C"

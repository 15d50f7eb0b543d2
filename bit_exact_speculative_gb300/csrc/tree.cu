// A tree of drafted tokens: positions of its nodes, the greedy walk along it, and the kept
// path's K/V rows into the cache.
//
// A tree of up to XV_KMAX nodes per sequence is an array of parents with parent[i] < i; node 0 is
// the last committed token, every other node a draft that continues its parent.  Node i at depth d
// stands at position ctx_len + d of the sequence its path spells.
//
// Each of these is a few hundred bytes to a few megabytes of work: launch and round-trip latency
// bound them, so a sequence is one warp (walk) or a few CTAs (append), each value is read once and
// the loads a step needs are requested together.  Walk and append together: one tree of 16 nodes 3.3 us,
// 256 trees of 61 nodes with 4 heads of 256 7.2 us.
#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

// Nodes of sequence b: n_nodes[b] clamped to [0, N] (recorded when it was outside), or N.
__device__ __forceinline__ int tree_nodes(const int32_t* n_nodes, int b, int N, unsigned* err, bool report) {
    if (!n_nodes) return N;
    const int n = n_nodes[b];
    if (n < 0 || n > N) {
        if (report) atomicOr(err, ERR_BAD_COUNT);
        return n < 0 ? 0 : N;
    }
    return n;
}

// One warp per sequence: pos = ctx + depth.  Depths by pointer doubling: after r rounds jump[i] is
// the 2^r-th ancestor and dep[i] the number of steps taken.
__global__ void __launch_bounds__(128) tree_positions_kernel(const int32_t* __restrict__ parent, const int32_t* __restrict__ n_nodes,
                                                             const int32_t* __restrict__ ctx_len, int B, int N,
                                                             int32_t* __restrict__ pos, unsigned* err) {
    griddep_launch();
    griddep_wait();
    __shared__ int8_t jump[4][XV_KMAX];
    __shared__ int8_t dep[4][XV_KMAX];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x * 4 + w;
    if (b >= B) return;
    const int n = tree_nodes(n_nodes, b, N, err, lane == 0), ctx = ctx_len[b];
    for (int i = lane; i < n; i += 32) {
        int p = parent[static_cast<long long>(b) * N + i];
        if (p < -1 || p >= i) {
            atomicOr(err, ERR_BAD_TREE);
            p = -1;
        }
        jump[w][i] = static_cast<int8_t>(p);
        dep[w][i] = p >= 0;
    }
    __syncwarp();
    for (int span = 1; span < n; span <<= 1) {
        int8_t j[2], d[2];
        for (int u = 0; u < 2; ++u) {
            const int i = lane + 32 * u;
            if (i >= n) continue;
            const int p = jump[w][i];
            j[u] = p >= 0 ? jump[w][p] : -1;
            d[u] = static_cast<int8_t>(dep[w][i] + (p >= 0 ? dep[w][p] : 0));
        }
        __syncwarp();
        for (int u = 0; u < 2; ++u) {
            const int i = lane + 32 * u;
            if (i >= n) continue;
            jump[w][i] = j[u];
            dep[w][i] = d[u];
        }
        __syncwarp();
    }
    for (int i = lane; i < n; i += 32) pos[static_cast<long long>(b) * N + i] = ctx + dep[w][i];
}

// One warp per sequence, nodes lane and lane + 32 in a lane's registers.  A node can be walked to
// when its token is its parent's argmax; each step takes the lowest such child of the current node
// (two ballots), so the walk is as long as the kept path.
__global__ void __launch_bounds__(128) tree_accept_kernel(const int32_t* __restrict__ tokens, const int32_t* __restrict__ parent,
                                                          const int32_t* __restrict__ n_nodes, const int32_t* __restrict__ argmax,
                                                          int B, int N, int32_t* __restrict__ path, int32_t* __restrict__ n_keep,
                                                          int32_t* __restrict__ next, unsigned* err) {
    griddep_launch();
    griddep_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (b >= B) return;
    const long long at = static_cast<long long>(b) * N;
    const int n = tree_nodes(n_nodes, b, N, err, lane == 0);
    int par[2], tok[2], am[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        const bool in = i < n;
        par[u] = in ? parent[at + i] : -1;
        tok[u] = in ? tokens[at + i] : 0;
        am[u] = in ? argmax[at + i] : -1;
        if (in && (par[u] < -1 || par[u] >= i)) {
            atomicOr(err, ERR_BAD_TREE);
            par[u] = -1;
        }
    }
    bool hit[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int p = par[u] < 0 ? 0 : par[u];
        const int lo = __shfl_sync(0xffffffffu, am[0], p & 31), hi = __shfl_sync(0xffffffffu, am[1], p & 31);
        hit[u] = par[u] >= 0 && tok[u] == (p < 32 ? lo : hi);
    }
    int keep = 0, cur = -1, mine[2] = {-1, -1};   // mine[u]: node kept at step lane + 32 u
    if (n > 0) {
        cur = 0;
        for (;;) {
            if (lane == (keep & 31)) {
                if (keep < 32) mine[0] = cur;
                else mine[1] = cur;
            }
            ++keep;
            const unsigned lo = __ballot_sync(0xffffffffu, hit[0] && par[0] == cur);
            const unsigned hi = __ballot_sync(0xffffffffu, hit[1] && par[1] == cur);
            if (!(lo | hi)) break;
            cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
        }
    }
    const int lo = __shfl_sync(0xffffffffu, am[0], cur & 31), hi = __shfl_sync(0xffffffffu, am[1], cur & 31);
    if (lane == 0) {
        n_keep[b] = keep;
        next[b] = n > 0 ? (cur < 32 ? lo : hi) : -1;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (lane + 32 * u < N) path[at + lane + 32 * u] = mine[u];
}

// CTA (b, y): kept rows y, y + gridDim.y, ... of sequence b; 16 bytes per thread and access.
__global__ void __launch_bounds__(256) kv_append_path_kernel(const uint16_t* __restrict__ src, long long src_stride,
                                                             const int32_t* __restrict__ path, const int32_t* __restrict__ n_keep,
                                                             const int32_t* __restrict__ ctx_len, int N, int Hkv, int hd,
                                                             KvPages kv, uint16_t* __restrict__ kc, uint16_t* __restrict__ vc,
                                                             unsigned* err) {
    griddep_launch();
    griddep_wait();
    const int b = blockIdx.x;
    int n = n_keep[b];
    const int ctx = ctx_len[b];
    const bool first = blockIdx.y == 0 && threadIdx.x == 0;
    if (n < 0 || n > N) {
        if (first) atomicOr(err, ERR_BAD_COUNT);
        n = n < 0 ? 0 : N;
    }
    const int chunks = Hkv * hd / 8;
    for (int t = blockIdx.y; t < n; t += gridDim.y) {
        const int node = path[static_cast<long long>(b) * N + t];
        const long long pos = static_cast<long long>(ctx) + t;
        if (node < 0 || node >= N || pos < 0 || pos >= static_cast<long long>(kv.page) * kv.max_pages) {
            if (threadIdx.x == 0) atomicOr(err, node < 0 || node >= N ? ERR_BAD_COUNT : ERR_BAD_LENGTH);
            continue;
        }
        int pg = b, at = static_cast<int>(pos);
        if (kv.table) {
            const int j = at / kv.page;
            at -= j * kv.page;
            pg = kv.table[static_cast<long long>(b) * kv.max_pages + j];
            if (pg < 0 || pg >= kv.n_pages) {
                if (threadIdx.x == 0) atomicOr(err, ERR_BAD_PAGE);
                continue;
            }
        }
        const uint16_t* row = src + (static_cast<long long>(b) * N + node) * src_stride;
        for (int c = threadIdx.x; c < 2 * chunks; c += blockDim.x) {
            const bool is_v = c >= chunks;
            const int cc = is_v ? c - chunks : c;
            const int h = cc / (hd / 8), d = (cc % (hd / 8)) * 8;
            const uint4 v = *reinterpret_cast<const uint4*>(row + static_cast<long long>(c) * 8);
            *reinterpret_cast<uint4*>((is_v ? vc : kc) + ((static_cast<long long>(pg) * Hkv + h) * kv.page + at) * hd + d) = v;
        }
    }
}

xv_status tree_sizes(const char* what, int B, int N) {
    if (B < 1 || N < 1) return fail(XV_ERR_ARG, "%s: need B >= 1 and N >= 1", what);
    if (N > XV_KMAX) return fail(XV_ERR_UNSUPPORTED, "%s: N = %d exceeds %d", what, N, XV_KMAX);
    if (B > 65535) return fail(XV_ERR_UNSUPPORTED, "%s: B must be below 65536", what);
    return XV_OK;
}

xv_status append_path(const uint16_t* kv_src, long long src_stride, const int32_t* path, const int32_t* n_keep,
                      const int32_t* ctx_len, int N, int B, int Hkv, int hd, const KvPages& kv, uint16_t* kc, uint16_t* vc,
                      cudaStream_t s) {
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "kv_append_path: device error word unavailable");
    // few sequences: a CTA per kept row up to 8; many: their CTAs fill the device anyway
    const int y = B <= 64 ? (N < 8 ? N : 8) : (N < 2 ? N : 2);
    trace_pre(s);
    launch_k(kv_append_path_kernel, dim3(B, y), dim3(256), 0, s, kv_src, src_stride, path, n_keep, ctx_len, N, Hkv, hd, kv,
             kc, vc, err);
    return launched("kv_append_path_kernel", s, K_KV_APPEND_PATH, 8ll * B * N * Hkv * hd);
}

xv_status append_path_checks(const uint16_t* kv_src, long long src_stride, const int32_t* path, const int32_t* n_keep,
                             const int32_t* ctx_len, int N, int B, int Hkv, int hd, const uint16_t* kc, const uint16_t* vc) {
    if (!kv_src || !path || !n_keep || !ctx_len || !kc || !vc) return fail(XV_ERR_ARG, "kv_append_path: null pointer");
    if (xv_status st = tree_sizes("kv_append_path", B, N)) return st;
    if (Hkv < 1 || hd < 8 || hd % 8) return fail(XV_ERR_ARG, "kv_append_path: need Hkv >= 1 and hd a positive multiple of 8");
    if (static_cast<long long>(Hkv) * hd > (1 << 30)) return fail(XV_ERR_UNSUPPORTED, "kv_append_path: Hkv*hd too large");
    if (src_stride < 2ll * Hkv * hd) return fail(XV_ERR_ARG, "kv_append_path: src_stride below 2*Hkv*hd");
    if (!aligned16(kv_src) || (src_stride % 8) || !aligned16(kc) || !aligned16(vc))
        return fail(XV_ERR_UNSUPPORTED, "kv_append_path: 16-byte alignment required");
    return XV_OK;
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

xv_status xv_tree_positions(const int32_t* parent, const int32_t* n_nodes, const int32_t* ctx_len, int N, int B,
                            int32_t* pos, xv_stream s) {
    if (!parent || !ctx_len || !pos) return fail(XV_ERR_ARG, "tree_positions: null pointer");
    if (xv_status st = tree_sizes("tree_positions", B, N)) return st;
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "tree_positions: device error word unavailable");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
    trace_pre(st);
    launch_k(tree_positions_kernel, dim3(ceil_div(B, 4)), dim3(128), 0, st, parent, n_nodes, ctx_len, B, N, pos, err);
    return launched("tree_positions_kernel", st, K_TREE_POS, 8ll * B * N + 8ll * B);
}

xv_status xv_tree_accept(const int32_t* tokens, const int32_t* parent, const int32_t* n_nodes, const int32_t* argmax, int N,
                         int B, int32_t* path, int32_t* n_keep, int32_t* next_token, xv_stream s) {
    if (!tokens || !parent || !argmax || !path || !n_keep || !next_token) return fail(XV_ERR_ARG, "tree_accept: null pointer");
    if (xv_status st = tree_sizes("tree_accept", B, N)) return st;
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "tree_accept: device error word unavailable");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
    trace_pre(st);
    launch_k(tree_accept_kernel, dim3(ceil_div(B, 4)), dim3(128), 0, st, tokens, parent, n_nodes, argmax, B, N, path, n_keep,
             next_token, err);
    return launched("tree_accept_kernel", st, K_TREE_ACCEPT, 16ll * B * N + 12ll * B);
}

xv_status xv_kv_append_path(const uint16_t* kv_src, long long src_stride, const int32_t* path, const int32_t* n_keep,
                            const int32_t* ctx_len, int N, int B, int Hkv, int hd, int Lmax, uint16_t* kc, uint16_t* vc,
                            xv_stream s) {
    if (xv_status st = append_path_checks(kv_src, src_stride, path, n_keep, ctx_len, N, B, Hkv, hd, kc, vc)) return st;
    if (Lmax < 1) return fail(XV_ERR_ARG, "kv_append_path: Lmax must be positive");
    return append_path(kv_src, src_stride, path, n_keep, ctx_len, N, B, Hkv, hd, kv_contiguous(B, Lmax), kc, vc,
                       reinterpret_cast<cudaStream_t>(s));
}

xv_status xv_kv_append_path_paged(const uint16_t* kv_src, long long src_stride, const int32_t* path, const int32_t* n_keep,
                                  const int32_t* ctx_len, int N, int B, int Hkv, int hd, const xv_kv_pages* pages,
                                  uint16_t* kpool, uint16_t* vpool, xv_stream s) {
    if (xv_status st = append_path_checks(kv_src, src_stride, path, n_keep, ctx_len, N, B, Hkv, hd, kpool, vpool)) return st;
    KvPages kv{};
    int Lmax = 0;
    if (xv_status st = kv_pages_check(pages, Hkv, hd, &kv, &Lmax)) return st;
    return append_path(kv_src, src_stride, path, n_keep, ctx_len, N, B, Hkv, hd, kv, kpool, vpool,
                       reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

// Log probabilities of given tokens, entropies and top alternatives of rows of logits.
//
// For a row x of V logits:
//     m = max x,  S = sum exp(x_i - m),  D = sum exp(x_i - m) (x_i - m),
//     logprob(t) = (x_t - m) - log S,   entropy = log S - D / S,
// and the n largest x_i, the lowest index first among equals (a NaN below every number).
//
// A row is cut into chunks of SC_CHUNK logits, one CTA each, every logit read once into a register.
// A chunk's (m, S, D) and its n best go to the workspace; the CTA that finishes a row last (an
// atomic counter) joins the chunks in order.  Chunks, threads' shares of them and the order of every
// sum are fixed by V and the logits' type, so a row has the same bits in a call of any number of
// rows, at any position and alignment.
//
// A chunk's n best: SC_GROUPS groups of threads give their largest values; the n-th largest of those
// bounds the n-th largest logit from below, and the few logits (usually 1 to 2 n) at or above the
// bound are ranked by comparing each with each.  Groups that tie at the bound are told apart by
// their lowest index there, so a chunk of one value (a masked one, all -inf) has few candidates too.
#include <cmath>

#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

constexpr int SC_THREADS = 256;
constexpr int SC_PER = 32;                          // logits per thread
constexpr int SC_CHUNK = SC_THREADS * SC_PER;
constexpr int SC_GROUPS = 64;                       // groups of 4 neighbouring threads, 128 logits each
constexpr int SC_CAND = XV_TOP_MAX * SC_CHUNK / SC_GROUPS;   // logits of the XV_TOP_MAX best groups
constexpr int SC_V_MAX = 1 << 19;
constexpr int SC_C_MAX = SC_V_MAX / SC_CHUNK;
static_assert(SC_C_MAX * XV_TOP_MAX <= SC_CAND, "the join's keys share the candidates' buffer");
static_assert(XV_TOP_MAX <= SC_GROUPS, "");

using Key = unsigned long long;   // (order of the value) << 32 | ~index: larger is better, 0 is none

struct ScoreArgs {
    const void* logits;
    long long ld;
    const int32_t* tokens;
    const int32_t* n_rows;
    int M, V, C, top;
    float* logprob;
    float* entropy;
    int32_t* ids;
    float* lps;
    unsigned* cnt;     // [M], zero between calls
    float4* part;      // [M][C] (m, S, D, -)
    Key* keys;         // [M][C][top]
    unsigned* err;
};

// Unsigned order of a float: NaN 0, then -inf .. +inf, -0 as +0.
__device__ __forceinline__ unsigned order_of(float x) {
    const unsigned u = __float_as_uint(__fadd_rn(x, 0.f));
    return x != x ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o) {
    return o == 0 ? __uint_as_float(0x7fc00000u) : __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

template <typename T>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int W = 4;   // logits per 16 bytes
    static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
    static __device__ __forceinline__ void wide(const float* p, float* v) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p));
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
};
template <>
struct Logits<uint16_t> {
    static constexpr int W = 8;
    static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(__ldg(p)); }
    static __device__ __forceinline__ void wide(const uint16_t* p, float* v) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

// Index, within its chunk, of a thread's i-th logit: runs of W neighbours, SC_THREADS * W apart.
template <int W>
__device__ __forceinline__ int chunk_index(int t, int i) {
    return (i / W) * (SC_THREADS * W) + t * W + i % W;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(SC_THREADS) logprobs_kernel(const __grid_constant__ ScoreArgs A) {
    griddep_launch();
    griddep_wait();
    using L = Logits<T>;
    constexpr int W = L::W;
    __shared__ __align__(16) Key cand[TOP ? SC_CAND : 1];
    __shared__ unsigned gmax[SC_GROUPS], gidx[SC_GROUPS];
    __shared__ float wm[8], ws_[8], wd[8];
    __shared__ float4 parts[SC_C_MAX];
    __shared__ Key s_bound;
    __shared__ unsigned s_tau, s_more, s_n;
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / A.C, chunk = blockIdx.x - row * A.C;
    if (A.n_rows && row >= *A.n_rows) return;
    const T* x = static_cast<const T*>(A.logits) + row * A.ld;
    const int base = chunk * SC_CHUNK, left = A.V - base;   // logits from the chunk's first on

    float v[SC_PER];
    if (left >= SC_CHUNK && (reinterpret_cast<uintptr_t>(x) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < SC_PER; i += W) L::wide(x + base + chunk_index<W>(tid, i), v + i);
    } else {
#pragma unroll
        for (int i = 0; i < SC_PER; ++i) {
            const int at = chunk_index<W>(tid, i);
            v[i] = at < left ? L::one(x + base + at) : -INFINITY;
        }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < SC_PER; ++i) mx = fmaxf(mx, v[i]);
    // a thread without a number (all NaN, or behind the row) stays below every number
    unsigned best = 0;
    if (TOP) {
        best = order_of(mx);
        if (mx == -INFINITY) {
            best = 0;
#pragma unroll
            for (int i = 0; i < SC_PER; ++i)
                if (v[i] == -INFINITY && chunk_index<W>(tid, i) < left) best = order_of(-INFINITY);
        }
        unsigned g = best;
        g = max(g, __shfl_xor_sync(0xffffffffu, g, 1));
        g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if ((tid & 3) == 0) gmax[tid >> 2] = g;
        if (tid == 0) s_n = 0;
    }
    float m = mx;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) wm[warp] = m;
    __syncthreads();
    m = wm[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = fmaxf(m, wm[w]);
    if (TOP && tid < SC_GROUPS) {
        // tau: the top-th largest of the groups' values
        const unsigned mine = gmax[tid];
        int gt = 0, ge = 0;
#pragma unroll 8
        for (int g = 0; g < SC_GROUPS; ++g) {
            const unsigned o = gmax[g];
            gt += o > mine;
            ge += o >= mine;
        }
        if (gt < A.top && ge >= A.top) {   // the same values by every thread of this value
            s_tau = mine;
            s_more = ge > A.top ? A.top - gt : 0;   // ties at tau: this many of its groups are in
        }
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float s = 0.f, d = 0.f;
#pragma unroll
    for (int i = 0; i < SC_PER; ++i) {
        const float c = __fsub_rn(v[i], ref);
        const float e = ex2_approx(__fmul_rn(c, 1.4426950408889634f));
        s = __fadd_rn(s, e);
        d = __fmaf_rn(e, fmaxf(c, -3e38f), d);   // exp(-inf) (-inf) is 0 here
    }
    s = warp_sum(s);
    d = warp_sum(d);
    if (lane == 0) ws_[warp] = s, wd[warp] = d;
    __syncthreads();
    const long long slot = static_cast<long long>(row) * A.C + chunk;
    if (tid == 0) {
        s = ws_[0], d = wd[0];
#pragma unroll
        for (int w = 1; w < 8; ++w) s = __fadd_rn(s, ws_[w]), d = __fadd_rn(d, wd[w]);
        __stcg(A.part + slot, make_float4(ref, s, d, 0.f));
    }
    if (TOP) {
        const unsigned tau = s_tau;
        unsigned lim = 0xffffffffu;   // of the logits equal to tau, those up to this index
        if (s_more) {
            unsigned lo = 0xffffffffu;
            if (best == tau)
#pragma unroll
                for (int i = SC_PER - 1; i >= 0; --i)
                    if (order_of(v[i]) == tau && chunk_index<W>(tid, i) < left) lo = chunk_index<W>(tid, i);
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, 2));
            if ((tid & 3) == 0) gidx[tid >> 2] = gmax[tid >> 2] == tau ? lo : 0xffffffffu;
            __syncthreads();
            if (tid < SC_GROUPS) {
                const unsigned mine = gidx[tid];
                int lt = 0;
#pragma unroll 8
                for (int g = 0; g < SC_GROUPS; ++g) lt += gidx[g] < mine || (gidx[g] == mine && g < tid);
                if (lt == static_cast<int>(s_more) - 1) s_bound = mine;   // 0xffffffff: fewer logits than top
            }
            __syncthreads();
            lim = static_cast<unsigned>(s_bound);
        }
        if (best >= tau) {
#pragma unroll
            for (int i = 0; i < SC_PER; ++i) {
                const unsigned o = order_of(v[i]), at = chunk_index<W>(tid, i);
                if ((o > tau || (o == tau && at <= lim)) && static_cast<int>(at) < left) {
                    const unsigned k = atomicAdd(&s_n, 1u);
                    if (k < SC_CAND) cand[k] = static_cast<Key>(o) << 32 | static_cast<unsigned>(~(base + at));
                }
            }
        }
        __syncthreads();
        const int n = min(static_cast<int>(s_n), SC_CAND);
        Key* out = A.keys + slot * A.top;
        for (int i = tid; i < n; i += SC_THREADS) {
            const Key mine = cand[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += cand[j] > mine;
            if (rank < A.top) __stcg(out + rank, mine);
        }
        for (int i = n + tid; i < A.top; i += SC_THREADS) __stcg(out + i, Key(0));
    }
    // the row's last CTA joins its chunks
    __syncthreads();
    if (tid == 0) {
        s_last = 1;
        if (A.C > 1) {
            __threadfence();
            s_last = atomicAdd(A.cnt + row, 1u) == static_cast<unsigned>(A.C - 1);
            if (s_last) A.cnt[row] = 0;
        }
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    for (int c = tid; c < A.C; c += SC_THREADS) parts[c] = __ldcg(A.part + static_cast<long long>(row) * A.C + c);
    const int nk = TOP ? A.C * A.top : 0;
    if (TOP) {
        const Key* in = A.keys + static_cast<long long>(row) * nk;
        for (int i = tid; i < nk; i += SC_THREADS) cand[i] = __ldcg(in + i);
        if (tid == 0) s_n = 0, s_bound = 0;
    }
    __syncthreads();
    float mrow = -INFINITY, srow = 0.f, drow = 0.f;
    for (int c = 0; c < A.C; ++c)
        if (parts[c].y != 0.f) mrow = fmaxf(mrow, parts[c].x);
    for (int c = 0; c < A.C; ++c) {
        const float4 p = parts[c];
        if (p.y == 0.f) continue;   // nothing but -inf
        const float off = __fsub_rn(p.x, mrow), w = expf(off);
        srow = __fmaf_rn(w, p.y, srow);
        drow = __fmaf_rn(w, __fmaf_rn(fmaxf(off, -3e38f), p.y, p.z), drow);
    }
    const bool empty = srow == 0.f;   // every logit -inf
    const float logs = logf(srow);
    auto score = [&](float xv) { return empty ? -INFINITY : __fsub_rn(__fsub_rn(xv, mrow), logs); };
    if (tid == 0) {
        if (A.entropy) A.entropy[row] = empty ? 0.f : __fsub_rn(logs, __fdiv_rn(drow, srow));
        const int t = A.tokens[row];
        float lp = 0.f;   // -1: no token
        if (t >= 0 && t < A.V) {
            lp = score(L::one(x + t));
        } else if (t != -1) {
            atomicOr(A.err, ERR_BAD_TOKEN);
            lp = __uint_as_float(0x7fc00000u);
        }
        A.logprob[row] = lp;
    }
    if (TOP) {
        // a lower bound of the top-th largest key: of the chunks' p-th keys the k-th largest, p k >= top
        const int p = max(A.top > 1 ? 2 : 1, (A.top + A.C - 1) / A.C), k = (A.top + p - 1) / p;
        if (tid < A.C) {
            const Key mine = cand[tid * A.top + p - 1];
            int gt = 0, ge = 0;
            for (int c = 0; c < A.C; ++c) {
                const Key o = cand[c * A.top + p - 1];
                gt += o > mine;
                ge += o >= mine;
            }
            if (gt < k && ge >= k) s_bound = mine;
        }
        __syncthreads();
        const Key bound = s_bound;
        for (int i = tid; i < nk; i += SC_THREADS) {
            const Key mine = cand[i];
            if (mine < bound || mine == 0) continue;
            int rank = 0;   // keys above this one; a chunk's stand in order, so its first smaller one ends it
            for (int c = 0; c < A.C && rank < A.top; ++c)
                for (int j = 0; j < A.top && cand[c * A.top + j] > mine; ++j) ++rank;
            if (rank >= A.top) continue;
            const long long o = static_cast<long long>(row) * A.top + rank;
            A.ids[o] = static_cast<int32_t>(~static_cast<unsigned>(mine));
            A.lps[o] = score(value_of(static_cast<unsigned>(mine >> 32)));
        }
    }
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool sizes_ok(int M, int V, int top) {
    return M >= 1 && V >= 1 && V <= SC_V_MAX && top >= 0 && top <= XV_TOP_MAX && top <= V &&
           static_cast<long long>(M) * ceil_div(V, SC_CHUNK) < (1ll << 31);
}

xv_status logprobs(const void* logits, bool f32, long long ld, const int32_t* tokens, const int32_t* n_rows, int M, int V,
                   float* logprob, float* entropy, int top, int32_t* ids, float* lps, void* ws, size_t ws_bytes,
                   cudaStream_t s) {
    if (!logits || !tokens || !logprob) return fail(XV_ERR_ARG, "logprobs: null logits, tokens or logprob");
    if (M < 1 || V < 1) return fail(XV_ERR_ARG, "logprobs: need M and V >= 1");
    if (ld < V) return fail(XV_ERR_ARG, "logprobs: row stride %lld below V = %d", ld, V);
    if (top < 0 || top > V) return fail(XV_ERR_ARG, "logprobs: top = %d outside [0, V = %d]", top, V);
    if (top && (!ids || !lps)) return fail(XV_ERR_ARG, "logprobs: top alternatives need top_ids and top_logprobs");
    if (top > XV_TOP_MAX) return fail(XV_ERR_UNSUPPORTED, "logprobs: top = %d above %d", top, XV_TOP_MAX);
    if (!sizes_ok(M, V, top)) return fail(XV_ERR_UNSUPPORTED, "logprobs: V = %d above %d, or too many rows (%d)", V, SC_V_MAX, M);
    if (reinterpret_cast<uintptr_t>(logits) % (f32 ? 4 : 2)) return fail(XV_ERR_UNSUPPORTED, "logprobs: unaligned logits");
    if (!ws || ws_bytes < xv_logprobs_workspace_size(M, V, top))
        return fail(XV_ERR_WORKSPACE, "logprobs: workspace of %zu bytes needed", xv_logprobs_workspace_size(M, V, top));
    if (!aligned16(ws)) return fail(XV_ERR_UNSUPPORTED, "logprobs: workspace must be 16-byte aligned");
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "logprobs: device error word unavailable");
    const int C = ceil_div(V, SC_CHUNK);
    uint8_t* w = static_cast<uint8_t*>(ws);
    ScoreArgs a{logits, ld, tokens, n_rows, M, V, C, top, logprob, entropy, ids, lps, reinterpret_cast<unsigned*>(w), nullptr,
                nullptr, err};
    w += round256(static_cast<size_t>(M) * 4);
    a.part = reinterpret_cast<float4*>(w);
    w += round256(static_cast<size_t>(M) * C * sizeof(float4));
    a.keys = reinterpret_cast<Key*>(w);
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(M) * C));
    trace_pre(s);
    auto go = [&](auto kern) { launch_k(kern, grid, dim3(SC_THREADS), 0, s, a); };
    if (f32) top ? go(logprobs_kernel<float, true>) : go(logprobs_kernel<float, false>);
    else top ? go(logprobs_kernel<uint16_t, true>) : go(logprobs_kernel<uint16_t, false>);
    return launched("logprobs_kernel", s, K_LOGPROBS, (f32 ? 4ll : 2ll) * M * V + M * (12ll + 8 * top));
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

size_t xv_logprobs_workspace_size(int M, int V, int top) {
    if (!sizes_ok(M, V, top)) return 0;
    const size_t n = static_cast<size_t>(M) * ceil_div(V, SC_CHUNK);
    return round256(static_cast<size_t>(M) * 4) + round256(n * sizeof(float4)) + round256(n * top * sizeof(Key));
}

xv_status xv_logprobs(const float* logits, long long ld, const int32_t* tokens, const int32_t* n_rows, int M, int V,
                      float* logprob, float* entropy, int top, int32_t* top_ids, float* top_logprobs, void* ws,
                      size_t ws_bytes, xv_stream s) {
    return logprobs(logits, true, ld, tokens, n_rows, M, V, logprob, entropy, top, top_ids, top_logprobs, ws, ws_bytes,
                    reinterpret_cast<cudaStream_t>(s));
}

xv_status xv_logprobs_bf16(const uint16_t* logits, long long ld, const int32_t* tokens, const int32_t* n_rows, int M, int V,
                           float* logprob, float* entropy, int top, int32_t* top_ids, float* top_logprobs, void* ws,
                           size_t ws_bytes, xv_stream s) {
    return logprobs(logits, false, ld, tokens, n_rows, M, V, logprob, entropy, top, top_ids, top_logprobs, ws, ws_bytes,
                    reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

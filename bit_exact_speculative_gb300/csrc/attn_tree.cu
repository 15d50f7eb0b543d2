// Attention of a tree of drafted tokens over a bf16 KV cache.
#include <cmath>

#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

struct TreeArgs {
    const uint16_t* q;
    long long q_stride;
    const uint16_t* kc;
    const uint16_t* vc;
    KvPages kv;
    const int32_t* ctx_len;
    const uint16_t* src;
    long long src_stride;
    const int32_t* parent;
    const int32_t* n_nodes;
    int N, B, Hq, Hkv, max_ctx;
    float sl2;
    const uint16_t* gate;
    long long gate_stride;
    uint16_t* out;
    long long out_stride;
    unsigned* err;
};

// One CTA per (node, q head): warp w takes visible positions w, w + 8, ...; an online softmax per
// warp, merged at the end.
template <int HD>
__global__ void __launch_bounds__(256) attn_tree_kernel(TreeArgs A) {
    griddep_launch();
    griddep_wait();
    constexpr int E = HD / 32;
    __shared__ float sm_m[8], sm_l[8], sm_o[8][HD];
    __shared__ int chain[XV_KMAX];
    const int h = blockIdx.x % A.Hq, row = blockIdx.x / A.Hq, b = row / A.N, i = row % A.N, g = h / (A.Hq / A.Hkv);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int n = A.n_nodes ? A.n_nodes[b] : A.N, ctx = A.ctx_len[b];
    const bool short_ctx = ctx < 0 || ctx > A.max_ctx;
    if (threadIdx.x == 0 && (n < 0 || n > A.N)) atomicOr(A.err, ERR_BAD_COUNT);
    if (threadIdx.x == 0 && short_ctx) atomicOr(A.err, ERR_BAD_LENGTH);
    if (short_ctx || i >= n) return;     // i < N: a count above N is clamped by it
    int depth = 0;
    for (int a = i; a >= 0;) {
        if (threadIdx.x == 0) chain[depth] = a;
        ++depth;
        int p = A.parent[static_cast<long long>(b) * A.N + a];
        if (p < -1 || p >= a) {
            if (threadIdx.x == 0) atomicOr(A.err, ERR_BAD_TREE);
            p = -1;
        }
        a = p;
    }
    __syncthreads();
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_to_f32(A.q[row * A.q_stride + h * HD + e * 32 + lane]);
        o[e] = 0.f;
    }
    for (int p = w; p < ctx + depth; p += 8) {
        const uint16_t *kp, *vp;
        if (p < ctx) {
            int at = p, pg = b;
            if (A.kv.table) {
                pg = A.kv.table[static_cast<long long>(b) * A.kv.max_pages + p / A.kv.page];
                at = p % A.kv.page;
                if (pg < 0 || pg >= A.kv.n_pages) {
                    if (lane == 0) atomicOr(A.err, ERR_BAD_PAGE);
                    pg = 0;
                }
            }
            const long long off = ((static_cast<long long>(pg) * A.Hkv + g) * A.kv.page + at) * HD;
            kp = A.kc + off;
            vp = A.vc + off;
        } else {
            kp = A.src + (static_cast<long long>(b) * A.N + chain[depth - 1 - (p - ctx)]) * A.src_stride + g * HD;
            vp = kp + A.Hkv * HD;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * bf16_to_f32(kp[e * 32 + lane]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= A.sl2;
        const float mn = fmaxf(m, s), al = m == -INFINITY ? 0.f : exp2f(m - mn), pr = exp2f(s - mn);
        l = l * al + pr;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * al + pr * bf16_to_f32(vp[e * 32 + lane]);
        m = mn;
    }
    if (lane == 0) {
        sm_m[w] = m;
        sm_l[w] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[w][e * 32 + lane] = o[e];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int j = 0; j < 8; ++j) M = fmaxf(M, sm_m[j]);
    for (int j = 0; j < 8; ++j) L += sm_l[j] > 0.f ? sm_l[j] * exp2f(sm_m[j] - M) : 0.f;
    for (int d = threadIdx.x; d < HD; d += 256) {
        float acc = 0.f;
        for (int j = 0; j < 8; ++j) acc += sm_l[j] > 0.f ? sm_o[j][d] * exp2f(sm_m[j] - M) : 0.f;
        float y = acc / L;
        if (A.gate) {
            const float gt = bf16_to_f32(A.gate[row * A.gate_stride + h * HD + d]);
            y = bf16_to_f32(f32_to_bf16(y)) / (1.f + expf(-gt));
        }
        A.out[row * A.out_stride + h * HD + d] = f32_to_bf16(y);
    }
}

size_t tree_workspace(int B, int N, int Hq, int hd, int max_ctx) {
    (void)B, (void)N, (void)Hq, (void)hd, (void)max_ctx;
    return 256;
}

xv_status tree_launch(TreeArgs a, int hd, cudaStream_t s) {
    a.err = device_error_word();
    if (!a.err) return fail(XV_ERR_CUDA, "attn_tree: device error word unavailable");
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.N * a.Hq));
    trace_pre(s);
    if (hd == 256) launch_k(attn_tree_kernel<256>, grid, dim3(256), 0, s, a);
    else if (hd == 128) launch_k(attn_tree_kernel<128>, grid, dim3(256), 0, s, a);
    else launch_k(attn_tree_kernel<64>, grid, dim3(256), 0, s, a);
    return launched("attn_tree_kernel", s, K_ATTN_TREE, 4ll * a.B * a.Hkv * a.max_ctx * hd);
}

xv_status tree_checks(const TreeArgs& a, int hd, int Lmax, const void* ws, size_t ws_bytes) {
    if (!a.q || !a.kc || !a.vc || !a.ctx_len || !a.src || !a.parent || !a.out) return fail(XV_ERR_ARG, "attn_tree: null pointer");
    if (a.B < 1 || a.N < 1 || a.Hq < 1 || a.Hkv < 1 || Lmax < 1) return fail(XV_ERR_ARG, "attn_tree: sizes must be positive");
    if (a.N > XV_KMAX) return fail(XV_ERR_UNSUPPORTED, "attn_tree: N = %d exceeds %d", a.N, XV_KMAX);
    if (a.Hq % a.Hkv) return fail(XV_ERR_ARG, "attn_tree: Hq must be a multiple of Hkv");
    if (hd != 64 && hd != 128 && hd != 256) return fail(XV_ERR_UNSUPPORTED, "attn_tree: hd must be 64, 128 or 256 (got %d)", hd);
    if (a.Hq / a.Hkv > 128) return fail(XV_ERR_UNSUPPORTED, "attn_tree: more than 128 q heads per kv head");
    if (a.max_ctx < 0 || a.max_ctx > Lmax) return fail(XV_ERR_ARG, "attn_tree: need 0 <= max_ctx <= Lmax");
    if (a.B > 65535 || a.Hkv > 65535) return fail(XV_ERR_UNSUPPORTED, "attn_tree: B and Hkv must be below 65536");
    if (static_cast<long long>(a.B) * a.N * a.Hq > (1ll << 30)) return fail(XV_ERR_UNSUPPORTED, "attn_tree: more than 2^30 rows");
    const long long w = static_cast<long long>(a.Hq) * hd, kw = 2ll * a.Hkv * hd;
    if (a.q_stride < w || a.out_stride < w || a.src_stride < kw) return fail(XV_ERR_ARG, "attn_tree: a row stride is below its row");
    if (a.gate && a.gate_stride < w) return fail(XV_ERR_ARG, "attn_tree: gate_stride below Hq*hd");
    if (!aligned16(a.q) || !aligned16(a.src) || a.q_stride % 8 || a.src_stride % 8 || !aligned16(a.kc) || !aligned16(a.vc))
        return fail(XV_ERR_UNSUPPORTED, "attn_tree: q rows, kv_src rows and caches must be 16-byte aligned");
    const size_t need = tree_workspace(a.B, a.N, a.Hq, hd, a.max_ctx);
    if (!ws || ws_bytes < need) return fail(XV_ERR_WORKSPACE, "attn_tree: workspace of %zu bytes needed", need);
    if (!aligned16(ws)) return fail(XV_ERR_UNSUPPORTED, "attn_tree: workspace must be 16-byte aligned");
    return XV_OK;
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

size_t xv_attn_tree_workspace_size(int B, int N, int Hq, int hd, int max_ctx) {
    if (B < 1 || N < 1 || N > XV_KMAX || Hq < 1 || hd < 1 || max_ctx < 0) return 0;
    return tree_workspace(B, N, Hq, hd, max_ctx);
}

xv_status xv_attn_tree(const uint16_t* q, long long q_stride, const uint16_t* kc, const uint16_t* vc,
                       const int32_t* ctx_len, const uint16_t* kv_src, long long src_stride, const int32_t* parent,
                       const int32_t* n_nodes, int N, int B, int Hq, int Hkv, int hd, int Lmax, int max_ctx, float scale,
                       const uint16_t* gate, long long gate_stride, uint16_t* out, long long out_stride, void* ws,
                       size_t ws_bytes, xv_stream s) {
    TreeArgs a{q, q_stride, kc, vc, kv_contiguous(B, Lmax), ctx_len, kv_src, src_stride, parent, n_nodes, N, B, Hq, Hkv,
               max_ctx, scale * 1.4426950408889634f, gate, gate_stride, out, out_stride, nullptr};
    if (xv_status st = tree_checks(a, hd, Lmax, ws, ws_bytes)) return st;
    if (static_cast<long long>(B) * Hkv > (1ll << 31)) return fail(XV_ERR_UNSUPPORTED, "attn_tree: cache too large");
    return tree_launch(a, hd, reinterpret_cast<cudaStream_t>(s));
}

xv_status xv_attn_tree_paged(const uint16_t* q, long long q_stride, const uint16_t* kpool, const uint16_t* vpool,
                             const xv_kv_pages* pages, const int32_t* ctx_len, const uint16_t* kv_src, long long src_stride,
                             const int32_t* parent, const int32_t* n_nodes, int N, int B, int Hq, int Hkv, int hd,
                             int max_ctx, float scale, const uint16_t* gate, long long gate_stride, uint16_t* out,
                             long long out_stride, void* ws, size_t ws_bytes, xv_stream s) {
    KvPages kv{};
    int Lmax = 0;
    if (xv_status st = kv_pages_check(pages, Hkv, hd, &kv, &Lmax)) return st;
    TreeArgs a{q, q_stride, kpool, vpool, kv, ctx_len, kv_src, src_stride, parent, n_nodes, N, B, Hq, Hkv,
               max_ctx, scale * 1.4426950408889634f, gate, gate_stride, out, out_stride, nullptr};
    if (xv_status st = tree_checks(a, hd, Lmax, ws, ws_bytes)) return st;
    return tree_launch(a, hd, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

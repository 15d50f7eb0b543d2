// Appending K and V rows to a cache held in 8 bits.
//
// A head of a token is hd e4m3 codes and one fp32 scale, for K and for V:
//     den = min(max(max |x_i|, 448 2^-40), 448 2^60),  scale = den / 448,  code_i = e4m3(448 x_i / den)
// (448 is e4m3's largest value; 448 x_i is exact in fp32, so the quotient is rounded once before the
// code's own rounding, and one that lies on the border of two codes in exact arithmetic lies there
// here).  The bounds on den keep every ratio of two scales within 2^100, which the attention's fp32
// exponents carry; 448 2^60 is past any activation.  A head with a non-finite value gets the scale
// NaN and codes 0: whoever sees it reads NaN, whoever does not is not touched by it.
//
// One scale per token and head, not per block of tokens: a block's shared scale would change the
// codes of committed tokens with every token that joins the block (a draft that is rejected later,
// too), and a verify would no longer give the bits of decoding its tokens one at a time.
//
// What bounds it: 2 bytes read and 1 written per value.  A head takes hd / 8 lanes of 16 bytes in and
// 8 out, its maximum a shuffle tree inside them.
#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

struct AppendQ8Args {
    const uint16_t* src;
    long long src_stride;
    const int32_t* ctx_len;
    const int32_t* n_rows;
    int R, Hkv, units;   // units: heads of all rows, K and V
    KvPages kv;
    uint8_t* code[2];
    float* scale[2];
    unsigned* err;
};

constexpr int AQ_THREADS = 256;

// Two fp32 values as e4m3, the first in the low byte; past 448 they become 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A unit, one head of K or V of one row, takes HD / 8 lanes; a CTA does U passes of them, all their
// loads issued first.
template <int HD, int U>
__global__ void __launch_bounds__(AQ_THREADS) kv_append_q8_kernel(const __grid_constant__ AppendQ8Args A) {
    griddep_launch();
    constexpr int LPH = HD / 8, HPP = AQ_THREADS / LPH;
    const int tid = threadIdx.x, c = tid % LPH, hs = tid / LPH, H2 = 2 * A.Hkv;
    griddep_wait();
    uint4 raw[U];
    long long at[U];   // head of the pools that the unit goes to, times page, plus its row; -1: nowhere
    bool isv[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int u = (blockIdx.x * U + k) * HPP + hs;
        at[k] = -1;
        raw[k] = make_uint4(0, 0, 0, 0);
        isv[k] = false;
        if (u >= A.units) continue;
        const int row = u / H2, h2 = u - row * H2, b = row / A.R, r = row - b * A.R;
        isv[k] = h2 >= A.Hkv;
        const int h = h2 - (isv[k] ? A.Hkv : 0);
        int n = A.R;
        if (A.n_rows) {
            n = A.n_rows[b];
            if ((n < 0 || n > A.R) && r == 0 && h2 == 0 && c == 0) atomicOr(A.err, ERR_BAD_COUNT);
        }
        if (r >= n) continue;
        raw[k] = *(reinterpret_cast<const uint4*>(A.src + row * A.src_stride + static_cast<long long>(h2) * HD) + c);
        const int len = A.ctx_len[b];
        const long long pos = static_cast<long long>(len) - 1 + r;
        if (pos < 0 || pos >= static_cast<long long>(A.kv.page) * A.kv.max_pages) {
            if (c == 0) atomicOr(A.err, ERR_BAD_LENGTH);
            continue;
        }
        int pg = b, prow = static_cast<int>(pos);
        if (A.kv.table) {
            const int j = prow / A.kv.page;
            prow -= j * A.kv.page;
            pg = A.kv.table[static_cast<long long>(b) * A.kv.max_pages + j];
            if (pg < 0 || pg >= A.kv.n_pages) {
                if (c == 0) atomicOr(A.err, ERR_BAD_PAGE);
                continue;
            }
        }
        at[k] = (static_cast<long long>(pg) * A.Hkv + h) * A.kv.page + prow;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        unsigned big = 0;   // the largest magnitude's bits (NaN above infinity above every number)
#pragma unroll
        for (int i = 0; i < 4; ++i) big = max(big, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
        for (int off = LPH / 2; off > 0; off >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
        if (at[k] < 0) continue;
        const bool bad = big >= 0x7f80u;
        const float den = fminf(fmaxf(__uint_as_float(big << 16), 448.f * 0x1p-40f), 448.f * 0x1p60f);
        uint32_t q[2] = {0, 0};
        if (!bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
                q[i >> 1] |= e4m3x2(__fdiv_rn(__fmul_rn(lo, 448.f), den), __fdiv_rn(__fmul_rn(hi, 448.f), den)) << (16 * (i & 1));
            }
        }
        *reinterpret_cast<uint2*>(A.code[isv[k]] + at[k] * HD + c * 8) = make_uint2(q[0], q[1]);
        if (c == 0) A.scale[isv[k]][at[k]] = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(den, 448.f);
    }
}

xv_status append_q8(const uint16_t* src, long long src_stride, const int32_t* ctx_len, const int32_t* n_rows, int R, int B,
                    int Hkv, int hd, const KvPages& kv, const xv_kv_q8* cache, cudaStream_t s) {
    if (!src || !ctx_len) return fail(XV_ERR_ARG, "kv_append_q8: null kv_src or ctx_len");
    if (R < 1 || B < 1 || Hkv < 1) return fail(XV_ERR_ARG, "kv_append_q8: need R, B and Hkv >= 1");
    if (hd != 64 && hd != 128 && hd != 256) return fail(XV_ERR_UNSUPPORTED, "kv_append_q8: hd must be 64, 128 or 256 (got %d)", hd);
    if (src_stride < 2ll * Hkv * hd) return fail(XV_ERR_ARG, "kv_append_q8: row stride %lld below its row", src_stride);
    if (!aligned16(src) || src_stride % 8) return fail(XV_ERR_UNSUPPORTED, "kv_append_q8: rows must be 16-byte aligned");
    const long long units = 2ll * B * R * Hkv;
    if (units > (1ll << 30)) return fail(XV_ERR_UNSUPPORTED, "kv_append_q8: more than 2^29 rows times heads");
    AppendQ8Args a{src, src_stride, ctx_len, n_rows, R, Hkv, static_cast<int>(units), kv, {cache->k, cache->v},
                   {cache->k_scale, cache->v_scale}, device_error_word()};
    if (!a.err) return fail(XV_ERR_CUDA, "kv_append_q8: device error word unavailable");
    const int hpp = AQ_THREADS * 8 / hd;
    trace_pre(s);
    auto go = [&](auto kern, int u) { launch_k(kern, dim3(ceil_div(units, static_cast<long long>(u) * hpp)), dim3(AQ_THREADS), 0, s, a); };
    hd == 256 ? go(kv_append_q8_kernel<256, 1>, 1) : hd == 128 ? go(kv_append_q8_kernel<128, 1>, 1) : go(kv_append_q8_kernel<64, 1>, 1);
    return launched("kv_append_q8_kernel", s, K_KV_APPEND_Q8, units * (3ll * hd + 4));
}

}  // namespace

xv_status kv_q8_check(const xv_kv_q8* c, const char* what) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return fail(XV_ERR_ARG, "%s: null cache", what);
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
        return fail(XV_ERR_UNSUPPORTED, "%s: codes and scales must be 16-byte aligned", what);
    return XV_OK;
}

xv_status kv_contiguous_check(int B, int Hkv, int hd, int Lmax, const char* what) {
    if (B < 1 || Hkv < 1 || Lmax < 1) return fail(XV_ERR_ARG, "%s: need B, Hkv and Lmax >= 1", what);
    if (Lmax > (1 << 30)) return fail(XV_ERR_UNSUPPORTED, "%s: more than 2^30 positions", what);
    if (static_cast<long long>(B) * Hkv > (1ll << 31) - 1 || static_cast<double>(B) * Hkv * Lmax * hd > 1.1e12)
        return fail(XV_ERR_UNSUPPORTED, "%s: cache too large", what);
    return XV_OK;
}

}  // namespace xv

using namespace xv;

extern "C" {

xv_status xv_kv_append_q8(const uint16_t* kv_src, long long src_stride, const int32_t* ctx_len, const int32_t* n_rows, int R,
                          int B, int Hkv, int hd, int Lmax, const xv_kv_q8* cache, xv_stream s) {
    if (xv_status st = kv_q8_check(cache, "kv_append_q8")) return st;
    if (xv_status st = kv_contiguous_check(B, Hkv, hd, Lmax, "kv_append_q8")) return st;
    return append_q8(kv_src, src_stride, ctx_len, n_rows, R, B, Hkv, hd, kv_contiguous(B, Lmax), cache,
                     reinterpret_cast<cudaStream_t>(s));
}

xv_status xv_kv_append_q8_paged(const uint16_t* kv_src, long long src_stride, const int32_t* ctx_len, const int32_t* n_rows,
                                int R, int B, int Hkv, int hd, const xv_kv_pages* pages, const xv_kv_q8* cache, xv_stream s) {
    if (xv_status st = kv_q8_check(cache, "kv_append_q8")) return st;
    if (B < 1 || Hkv < 1 || hd < 1) return fail(XV_ERR_ARG, "kv_append_q8: need B, Hkv and hd >= 1");
    KvPages kv;
    int Lmax;
    if (xv_status st = kv_pages_check(pages, Hkv, hd, &kv, &Lmax)) return st;
    return append_q8(kv_src, src_stride, ctx_len, n_rows, R, B, Hkv, hd, kv, cache, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

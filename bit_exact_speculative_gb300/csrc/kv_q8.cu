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
// What bounds it: 2 bytes read and 1 written per value.  A head takes hd / 32 lanes of four pieces of 16
// bytes in and 8 out, its maximum a shuffle tree inside them (8192 rows of 8 heads of 128: 8.3 us, 7.5 at
// the memory's rate; with two pieces a lane 9.7, with one 14.7 us).  Its codes come from one quotient
// f = 448 / den: x f rounded to 16 bits of significand is 448 x / den on the right side of every border
// of two codes, and on it where the exact quotient is.  For 448 x = X 2^a with X < 2^11 and a border times
// den = Y 2^c with Y < 2^13 (5 bits times 8); where they differ they do so by 2^min(a, c) at least, 2^-13
// of either, and x f is off by 2^-23.  (With a division per value 20.9 us.)
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
    Divisor heads, rows, page;   // by 2 Hkv, R and kv.page
    KvPages kv;
    uint8_t* code[2];
    float* scale[2];
    unsigned* err;
};

constexpr int AQ_THREADS = 128;
constexpr int AQ_VECS = 4;   // pieces of 8 values per thread

// Two fp32 values as e4m3, the first in the low byte; past 448 they become 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// x rounded to 16 bits of significand (the nearest; a carry moves on into the exponent).
__device__ __forceinline__ float round16(float x) { return __uint_as_float((__float_as_uint(x) + 0x80u) & 0xffffff00u); }

// A unit, one head of K or V of one row, takes HD / (8 AQ_VECS) lanes.  (The rows behind a sequence's
// count are there to be read, too.)
template <int HD>
__global__ void __launch_bounds__(AQ_THREADS) kv_append_q8_kernel(const __grid_constant__ AppendQ8Args A) {
    griddep_launch();
    constexpr int V = AQ_VECS, LPH = HD / (8 * V), HPP = AQ_THREADS / LPH;
    const int tid = threadIdx.x, c = tid % LPH, H2 = 2 * A.Hkv;
    const int unit = static_cast<int>(blockIdx.x) * HPP + tid / LPH, u = min(unit, A.units - 1);
    const int row = A.heads.div(u), h2 = u - row * H2, b = A.rows.div(row), r = row - b * A.R;
    const bool isv = h2 >= A.Hkv;
    const uint4* src = reinterpret_cast<const uint4*>(A.src + row * A.src_stride + static_cast<long long>(h2) * HD) + c;
    griddep_wait();
    uint4 raw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) raw[j] = src[j * LPH];
    const int n = A.n_rows ? __ldg(A.n_rows + b) : A.R, len = __ldg(A.ctx_len + b);
    // where the unit goes: head of the pools times page, plus its row
    auto place = [&]() -> long long {
        if (unit >= A.units) return -1;
        if ((n < 0 || n > A.R) && r == 0 && h2 == 0 && c == 0) atomicOr(A.err, ERR_BAD_COUNT);
        if (r >= n) return -1;
        const long long pos = static_cast<long long>(len) - 1 + r;
        if (pos < 0 || pos >= static_cast<long long>(A.kv.page) * A.kv.max_pages) {
            if (c == 0) atomicOr(A.err, ERR_BAD_LENGTH);
            return -1;
        }
        int pg = b, prow = static_cast<int>(pos);
        if (A.kv.table) {
            const int j = A.page.div(prow);
            prow -= j * A.kv.page;
            pg = __ldg(A.kv.table + static_cast<long long>(b) * A.kv.max_pages + j);
            if (pg < 0 || pg >= A.kv.n_pages) {
                if (c == 0) atomicOr(A.err, ERR_BAD_PAGE);
                return -1;
            }
        }
        return (static_cast<long long>(pg) * A.Hkv + (isv ? h2 - A.Hkv : h2)) * A.kv.page + prow;
    };
    const long long at = place();
    uint32_t w[4 * V];
    unsigned big = 0;   // the largest magnitude's bits (NaN above infinity above every number)
#pragma unroll
    for (int j = 0; j < V; ++j) w[4 * j] = raw[j].x, w[4 * j + 1] = raw[j].y, w[4 * j + 2] = raw[j].z, w[4 * j + 3] = raw[j].w;
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) big = __vmaxu2(big, w[i] & 0x7fff7fffu);
    big = max(big & 0xffffu, big >> 16);
#pragma unroll
    for (int off = LPH / 2; off > 0; off >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
    if (at < 0) return;
    const bool bad = big >= 0x7f80u;
    const float den = fminf(fmaxf(__uint_as_float(big << 16), 448.f * 0x1p-40f), 448.f * 0x1p60f), f = __fdiv_rn(448.f, den);
    uint8_t* code = (isv ? A.code[1] : A.code[0]) + at * HD + c * 8;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        uint32_t q[2] = {0, 0};
        if (!bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo = __uint_as_float(w[4 * j + i] << 16), hi = __uint_as_float(w[4 * j + i] & 0xffff0000u);
                mul2(lo, hi, f, f);
                q[i >> 1] |= e4m3x2(round16(lo), round16(hi)) << (16 * (i & 1));
            }
        }
        *reinterpret_cast<uint2*>(code + j * LPH * 8) = make_uint2(q[0], q[1]);
    }
    if (c == 0) (isv ? A.scale[1] : A.scale[0])[at] = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(den, 448.f);
}

xv_status append_q8(const uint16_t* src, long long src_stride, const int32_t* ctx_len, const int32_t* n_rows, int R, int B,
                    int Hkv, int hd, const KvPages& kv, const xv_kv_q8* cache, cudaStream_t s) {
    if (!src || !ctx_len) return fail(XV_ERR_ARG, "kv_append_q8: null kv_src or ctx_len");
    if (R < 1 || B < 1 || Hkv < 1) return fail(XV_ERR_ARG, "kv_append_q8: need R, B and Hkv >= 1");
    if (hd != 64 && hd != 128 && hd != 256) return fail(XV_ERR_UNSUPPORTED, "kv_append_q8: hd must be 64, 128 or 256 (got %d)", hd);
    if (src_stride < 2ll * Hkv * hd) return fail(XV_ERR_ARG, "kv_append_q8: row stride %lld below its row", src_stride);
    if (!aligned16(src) || src_stride % 8) return fail(XV_ERR_UNSUPPORTED, "kv_append_q8: rows must be 16-byte aligned");
    const long long rows = static_cast<long long>(B) * R;   // (times the heads it may pass 2^63)
    if (rows > (1ll << 29) / Hkv) return fail(XV_ERR_UNSUPPORTED, "kv_append_q8: more than 2^29 rows times heads");
    const long long units = 2 * rows * Hkv;
    AppendQ8Args a{src, src_stride, ctx_len, n_rows, R, Hkv, static_cast<int>(units),
                   Divisor(2 * Hkv), Divisor(R), Divisor(kv.page), kv, {cache->k, cache->v},
                   {cache->k_scale, cache->v_scale}, device_error_word()};
    if (!a.err) return fail(XV_ERR_CUDA, "kv_append_q8: device error word unavailable");
    trace_pre(s);
    auto go = [&](auto kern) { launch_k(kern, dim3(ceil_div(units, static_cast<long long>(AQ_THREADS) * 8 * AQ_VECS / hd)), dim3(AQ_THREADS), 0, s, a); };
    if (hd == 256) go(kv_append_q8_kernel<256>);
    else if (hd == 128) go(kv_append_q8_kernel<128>);
    else go(kv_append_q8_kernel<64>);
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

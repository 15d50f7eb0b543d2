// Per-head RMSNorm of queries and keys with the position rotation in the same pass.
//
// For a head x of hd values at position p, in fp32 and rounded to bf16 once at the end:
//     y = x / sqrt(mean(x^2) + eps) * (1 + w)          (y = x without a norm weight)
//     (y_i, y_j) <- (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = p * f_i,
// over the rot/2 pairs of the first rot values: (i, i + rot/2), or (2i, 2i + 1) when interleaved.
//
// The angle: freq[i] holds f_i in turns per position as a 64-bit binary fraction, so p * freq[i]
// modulo 2^64 is the angle modulo one turn to 2^-64 * p of a turn, for any 32-bit p.  An fp32
// angle p * f_i would be off by p * 2^-24 radians (0.008 at 131072 positions, 0.03 at 500000).
//
// What bounds it: every value is read once and written once with ~10 operations between, so HBM
// for long row counts and one load-to-store latency for a verify step's few rows.  A head takes
// hd/8 lanes of 16 bytes each, its sum of squares a fixed shuffle tree inside them, so a head's
// bits depend on that head, its weight and its position alone.  cos and sin are formed once per
// row and shared by the row's heads through shared memory.
#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

struct RopeArgs {
    const uint16_t* q;
    long long q_stride;
    uint16_t* q_out;
    long long qo_stride;
    const uint16_t* kv;      // k heads, then (append) v heads
    long long kv_stride;
    uint16_t* k_out;         // rows, or null when appending
    long long ko_stride;
    const uint16_t* q_norm;
    const uint16_t* k_norm;
    float eps;
    const unsigned long long* freq;
    int rot, inter;
    const int32_t* pos;
    const int32_t* n_rows;   // device count of live rows, or null (all M)
    int M, Hq, Hkv;
    const long long* slots;  // append: slot of each row
    uint16_t* kpool;
    uint16_t* vpool;
    int page;
    long long n_slots;       // n_pages * page
    unsigned* err;
};

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_U = 4;    // heads whose loads a lane group has in flight together

__device__ __forceinline__ void rope_unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 rope_pack(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// CTA (x, y): row x, heads y*HPB .. (HPB = heads per pass * passes); a head per LPH lanes.
template <int HD>
__global__ void __launch_bounds__(ROPE_THREADS) qk_norm_rope_kernel(RopeArgs A, int heads_per_cta) {
    griddep_launch();
    constexpr int LPH = HD / 8, HPP = ROPE_THREADS / LPH;   // lanes per head, heads per pass
    __shared__ float2 cs[HD / 2];
    const long long row = blockIdx.x;
    const int tid = threadIdx.x, c = tid % LPH, hs = tid / LPH;
    griddep_wait();
    if (A.n_rows && row >= *A.n_rows) return;
    const int H = A.Hq + A.Hkv + (A.k_out ? 0 : A.Hkv);
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, H);
    long long slot = 0;
    if (!A.k_out) {
        slot = A.slots[row];
        if (slot >= A.n_slots || slot < -1) {
            if (tid == 0 && blockIdx.y == 0) atomicOr(A.err, ERR_BAD_PAGE);
            slot = -1;
        }
    }
    if (tid < A.rot / 2) {
        const unsigned long long turns = static_cast<unsigned long long>(static_cast<long long>(A.pos[row])) * A.freq[tid];
        float s, co;
        sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f, &s, &co);
        cs[tid] = make_float2(co, s);
    }
    __syncthreads();
    for (int hb = h0; hb < h1; hb += HPP * ROPE_U) {
        uint4 raw[ROPE_U];
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int h = hb + u * HPP + hs;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (h < h1) {
                const uint16_t* src = h < A.Hq ? A.q + row * A.q_stride + static_cast<long long>(h) * HD
                                               : A.kv + row * A.kv_stride + static_cast<long long>(h - A.Hq) * HD;
                raw[u] = *reinterpret_cast<const uint4*>(src + c * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int h = hb + u * HPP + hs;
            if (hb + u * HPP >= h1) break;           // the same for the whole CTA
            const bool isq = h < A.Hq, isv = h >= A.Hq + A.Hkv;
            float x[8];
            rope_unpack(raw[u], x);
            const uint16_t* w = isq ? A.q_norm : A.k_norm;
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __fmaf_rn(x[e], x[e], ss);
#pragma unroll
            for (int off = LPH / 2; off > 0; off >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
            if (w && !isv) {
                const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.f / HD), A.eps)));
                float wf[8];
                rope_unpack(*reinterpret_cast<const uint4*>(w + c * 8), wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], inv), __fadd_rn(1.f, wf[e]));
            }
            const int half = A.rot / 2;
            if (A.inter) {
                if (8 * c < A.rot && !isv) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 t = cs[4 * c + e / 2];
                        const float a = x[e], b = x[e + 1];
                        x[e] = a * t.x - b * t.y;
                        x[e + 1] = b * t.x + a * t.y;
                    }
                }
            } else if (A.rot) {
                // the partner values sit half/8 lanes away in the same head
                const bool lo = 8 * c < half, in = 8 * c < A.rot;
                const int lane = tid & 31, partner = in ? (lo ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float o = __shfl_sync(0xffffffffu, x[e], partner);
                    if (in && !isv) {
                        const float2 t = cs[8 * c + e - (lo ? 0 : half)];
                        x[e] = lo ? x[e] * t.x - o * t.y : x[e] * t.x + o * t.y;
                    }
                }
            }
            if (h >= h1) continue;
            const uint4 y = isv ? raw[u] : rope_pack(x);
            if (isq) {
                *reinterpret_cast<uint4*>(A.q_out + row * A.qo_stride + static_cast<long long>(h) * HD + c * 8) = y;
            } else if (A.k_out) {
                *reinterpret_cast<uint4*>(A.k_out + row * A.ko_stride + static_cast<long long>(h - A.Hq) * HD + c * 8) = y;
            } else if (slot >= 0) {
                const int g = h - A.Hq - (isv ? A.Hkv : 0);
                const long long pg = slot / A.page, at = slot - pg * A.page;
                *reinterpret_cast<uint4*>((isv ? A.vpool : A.kpool) + ((pg * A.Hkv + g) * A.page + at) * HD + c * 8) = y;
            }
        }
    }
}

xv_status rope_checks(const RopeArgs& a, int hd) {
    if (!a.q || !a.q_out || !a.kv) return fail(XV_ERR_ARG, "qk_norm_rope: null q, q_out or kv");
    if (a.M < 1 || a.Hq < 1 || a.Hkv < 1) return fail(XV_ERR_ARG, "qk_norm_rope: need M, Hq and Hkv >= 1");
    if (hd != 64 && hd != 128 && hd != 256) return fail(XV_ERR_UNSUPPORTED, "qk_norm_rope: hd must be 64, 128 or 256 (got %d)", hd);
    if (a.rot < 0 || a.rot > hd) return fail(XV_ERR_ARG, "qk_norm_rope: rot = %d outside [0, hd = %d]", a.rot, hd);
    if (a.rot % 16) return fail(XV_ERR_UNSUPPORTED, "qk_norm_rope: rot must be a multiple of 16 (got %d)", a.rot);
    if (a.rot && (!a.freq || !a.pos)) return fail(XV_ERR_ARG, "qk_norm_rope: a rotation needs freq and pos");
    if (a.Hq > 65535 || a.Hkv > 65535) return fail(XV_ERR_UNSUPPORTED, "qk_norm_rope: Hq and Hkv must be below 65536");
    const long long qw = static_cast<long long>(a.Hq) * hd, kw = static_cast<long long>(a.Hkv) * hd;
    if (a.q_stride < qw || a.qo_stride < qw || a.kv_stride < (a.k_out ? kw : 2 * kw) || (a.k_out && a.ko_stride < kw))
        return fail(XV_ERR_ARG, "qk_norm_rope: a row stride is below its row");
    if (!aligned16(a.q) || !aligned16(a.q_out) || !aligned16(a.kv) || !aligned16(a.k_out) || !aligned16(a.q_norm) ||
        !aligned16(a.k_norm) || a.q_stride % 8 || a.qo_stride % 8 || a.kv_stride % 8 || a.ko_stride % 8)
        return fail(XV_ERR_UNSUPPORTED, "qk_norm_rope: rows and norm weights must be 16-byte aligned");
    return XV_OK;
}

xv_status rope_launch(RopeArgs a, int hd, cudaStream_t s) {
    a.err = device_error_word();
    if (!a.err) return fail(XV_ERR_CUDA, "qk_norm_rope: device error word unavailable");
    const int H = a.Hq + a.Hkv + (a.k_out ? 0 : a.Hkv), hpp = ROPE_THREADS * 8 / hd;
    int per = H;
    if (a.M < 1024) per = hpp;
    const dim3 grid(a.M, ceil_div(H, per));
    trace_pre(s);
    if (hd == 256) launch_k(qk_norm_rope_kernel<256>, grid, dim3(ROPE_THREADS), 0, s, a, per);
    else if (hd == 128) launch_k(qk_norm_rope_kernel<128>, grid, dim3(ROPE_THREADS), 0, s, a, per);
    else launch_k(qk_norm_rope_kernel<64>, grid, dim3(ROPE_THREADS), 0, s, a, per);
    return launched("qk_norm_rope_kernel", s, K_ROPE, 4ll * a.M * H * hd);
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

xv_status xv_qk_norm_rope(const uint16_t* q, long long q_stride, uint16_t* q_out, long long q_out_stride,
                          const uint16_t* k, long long k_stride, uint16_t* k_out, long long k_out_stride,
                          const xv_qk_rope* rope, const int32_t* pos, const int32_t* n_rows, int M, int Hq, int Hkv,
                          int hd, xv_stream s) {
    if (!rope) return fail(XV_ERR_ARG, "qk_norm_rope: null rope");
    if (!k_out) return fail(XV_ERR_ARG, "qk_norm_rope: null k_out");
    RopeArgs a{q, q_stride, q_out, q_out_stride, k, k_stride, k_out, k_out_stride, rope->q_norm, rope->k_norm, rope->eps,
               reinterpret_cast<const unsigned long long*>(rope->freq), rope->rot, rope->interleaved, pos, n_rows, M, Hq,
               Hkv, nullptr, nullptr, nullptr, 1, 0, nullptr};
    if (xv_status st = rope_checks(a, hd)) return st;
    return rope_launch(a, hd, reinterpret_cast<cudaStream_t>(s));
}

xv_status xv_qk_norm_rope_append(const uint16_t* q, long long q_stride, uint16_t* q_out, long long q_out_stride,
                                 const uint16_t* kv, long long kv_stride, const xv_qk_rope* rope, const int32_t* pos,
                                 const long long* slots, const int32_t* n_rows, int M, int Hq, int Hkv, int hd,
                                 int page_size, int n_pages, uint16_t* kpool, uint16_t* vpool, xv_stream s) {
    if (!rope) return fail(XV_ERR_ARG, "qk_norm_rope_append: null rope");
    if (!slots || !kpool || !vpool) return fail(XV_ERR_ARG, "qk_norm_rope_append: null slots or pools");
    if (page_size < 1 || n_pages < 1) return fail(XV_ERR_ARG, "qk_norm_rope_append: page_size and n_pages must be positive");
    if (!aligned16(kpool) || !aligned16(vpool)) return fail(XV_ERR_UNSUPPORTED, "qk_norm_rope_append: pools must be 16-byte aligned");
    RopeArgs a{q, q_stride, q_out, q_out_stride, kv, kv_stride, nullptr, 0, rope->q_norm, rope->k_norm, rope->eps,
               reinterpret_cast<const unsigned long long*>(rope->freq), rope->rot, rope->interleaved, pos, n_rows, M, Hq,
               Hkv, slots, kpool, vpool, page_size, static_cast<long long>(page_size) * n_pages, nullptr};
    if (xv_status st = rope_checks(a, hd)) return st;
    return rope_launch(a, hd, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

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
// What bounds it: every value is read once and written once.  8192 rows of 40 + 8 heads of 128: 43.7 us
// for 201 MB, 4.6 TB/s, 0.69 of the measured copy rate; more or fewer resident CTAs change nothing, the
// ~110 instructions a lane needs per 8 values (V's too, whose result is dropped) share the issue slots with
// the loads.  A verify step's 8 rows: 2.0 us, one load-to-store latency.  A head takes hd/8 lanes of 16
// bytes each, its sum of squares a fixed shuffle tree inside them, so a head's bits depend on that head, its
// weight and its position alone.  fp32 pairs go two to an instruction; cos and sin are formed once per row and
// read as rows of floats (as (cos, sin) pairs, the lanes' reads met in the same banks 16 deep).
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
constexpr int ROPE_U = 4;    // units whose loads a lane group has in flight together
constexpr int ROPE_ROWS = 16;   // rows per CTA, at most

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
// Two fp32 operations in one instruction: (a, b) *= (x, y), and (a, b) * (x, y) + (u, v).
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
__device__ __forceinline__ void fma2(float a, float b, float x, float y, float& u, float& v) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%0, %1};\n\t"
        "fma.rn.f32x2 r, p, q, r;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "+f"(u), "+f"(v) : "f"(a), "f"(b), "f"(x), "f"(y));
}

// CTA (x, y): rows x * rpc .. of `rpc` rows, of each row's heads y * hpc .. of `hpc` (rpc > 1 only
// with every head of a row in the CTA).  A unit, one head of one row, takes LPH lanes; HPP units run at
// a time, and the loads of up to ROPE_U passes go out before what the angles need.  cos, sin and -sin
// of the CTA's rows stand in shared memory as rows of floats, read 16 bytes at a time.
constexpr int ROPE_TAB = 1024;   // floats per table: rpc * rot / 2 of them are used

template <int HD, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, 4) qk_norm_rope_kernel(const __grid_constant__ RopeArgs A, int hpc, int rpc, unsigned inv_h) {
    griddep_launch();
    constexpr int LPH = HD / 8, HPP = ROPE_THREADS / LPH;   // lanes per unit, units per pass
    __shared__ __align__(16) float tab[3][ROPE_TAB];
    __shared__ long long s_at[ROPE_ROWS];   // element of a row's first kv head in the pools, -1: nowhere
    const long long row0 = static_cast<long long>(blockIdx.x) * rpc;
    const int tid = threadIdx.x, c = tid % LPH, hs = tid / LPH;
    const int H = A.Hq + A.Hkv + (A.k_out ? 0 : A.Hkv);
    const int h0 = blockIdx.y * hpc, nh = min(hpc, H - h0);
    griddep_wait();
    const long long M = A.n_rows ? min(A.M, max(*A.n_rows, 0)) : A.M;
    const int nrow = static_cast<int>(min(static_cast<long long>(rpc), M - row0));
    if (nrow <= 0) return;
    const int units = nrow * nh;
    // unit -> (row, head): the product form of the division is exact for unit < 512 (rpc > 1)
    auto split = [&](int u, int* h) {
        const int r = rpc > 1 ? static_cast<int>((u * inv_h) >> 16) : 0;
        *h = h0 + u - r * nh;
        return r;
    };
    uint4 raw[ROPE_U];
    auto load = [&](int u0) {
#pragma unroll
        for (int k = 0; k < ROPE_U; ++k) {
            const int u = u0 + k * HPP + hs;
            raw[k] = make_uint4(0, 0, 0, 0);
            if (u < units) {
                int h;
                const long long row = row0 + split(u, &h);
                raw[k] = *(reinterpret_cast<const uint4*>(h < A.Hq ? A.q + row * A.q_stride + static_cast<long long>(h) * HD
                                                                   : A.kv + row * A.kv_stride + static_cast<long long>(h - A.Hq) * HD) + c);
            }
        }
    };
    load(0);
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if (A.q_norm) wq = __ldg(reinterpret_cast<const uint4*>(A.q_norm) + c);
    if (A.k_norm) wk = __ldg(reinterpret_cast<const uint4*>(A.k_norm) + c);
    const int half = A.rot / 2;
    for (int i = tid; i < nrow * half; i += ROPE_THREADS) {
        const int r = i / half;
        const unsigned long long turns = static_cast<unsigned long long>(static_cast<long long>(A.pos[row0 + r])) * A.freq[i - r * half];
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f, &sn, &cn);
        tab[0][i] = cn;
        tab[1][i] = sn;
        tab[2][i] = -sn;
    }
    if (!A.k_out && tid >= ROPE_THREADS - nrow) {
        const int r = ROPE_THREADS - 1 - tid;
        long long slot = A.slots[row0 + r];
        if (slot >= A.n_slots || slot < -1) {
            if (blockIdx.y == 0) atomicOr(A.err, ERR_BAD_PAGE);
            slot = -1;
        }
        const long long pg = slot / A.page;
        s_at[r] = slot < 0 ? -1 : (pg * A.Hkv * A.page + (slot - pg * A.page)) * HD;
    }
    __syncthreads();
    // this lane's values of a head meet frequencies f0 ..: 8 of them, or 4 when interleaved
    const bool in = 8 * c < A.rot, lo = 8 * c < half;
    const int f0 = INTER ? 4 * c : 8 * c - (lo ? 0 : half);
    const int lane = tid & 31, partner = !INTER && in ? (lo ? lane + half / 8 : lane - half / 8) : lane;
    for (int u0 = 0; u0 < units; u0 += HPP * ROPE_U) {
        if (u0) load(u0);
#pragma unroll
        for (int k = 0; k < ROPE_U; ++k) {
            const int u = u0 + k * HPP + hs;
            if (u0 + k * HPP >= units) break;           // the same for the whole CTA
            int h;
            const int r = split(min(u, units - 1), &h);
            const bool isq = h < A.Hq, isv = h >= A.Hq + A.Hkv;
            float x[8];
            rope_unpack(raw[k], x);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) fma2(x[e], x[e + 1], x[e], x[e + 1], s0, s1);
            float ss = __fadd_rn(s0, s1);
#pragma unroll
            for (int off = LPH / 2; off > 0; off >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
            if (isq ? A.q_norm != nullptr : A.k_norm != nullptr) {
                const float inv = rsqrtf(__fmaf_rn(ss, 1.f / HD, A.eps));
                float wf[8];
                rope_unpack(isq ? wq : wk, wf);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float g0 = inv, g1 = inv;   // inv (1 + w)
                    fma2(wf[e], wf[e + 1], inv, inv, g0, g1);
                    mul2(x[e], x[e + 1], g0, g1);
                }
            }
            if (half) {
                if constexpr (INTER) {
                    if (in) {
                        const float4 cn = *reinterpret_cast<const float4*>(&tab[0][r * half + f0]);
                        const float4 sn = *reinterpret_cast<const float4*>(&tab[1][r * half + f0]);
                        const float cv[4] = {cn.x, cn.y, cn.z, cn.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = x[2 * e], b = x[2 * e + 1];
                            mul2(x[2 * e], x[2 * e + 1], cv[e], cv[e]);
                            fma2(-b, a, sv[e], sv[e], x[2 * e], x[2 * e + 1]);
                        }
                    }
                } else {
                    // the partner values sit half/8 lanes away in the same head
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, x[e], partner);
                    if (in) {
                        const float4* ct = reinterpret_cast<const float4*>(&tab[0][r * half + f0]);
                        const float4* st = reinterpret_cast<const float4*>(&tab[lo ? 2 : 1][r * half + f0]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float4 cn = ct[q], sn = st[q];
                            mul2(x[4 * q], x[4 * q + 1], cn.x, cn.y);
                            mul2(x[4 * q + 2], x[4 * q + 3], cn.z, cn.w);
                            fma2(o[4 * q], o[4 * q + 1], sn.x, sn.y, x[4 * q], x[4 * q + 1]);
                            fma2(o[4 * q + 2], o[4 * q + 3], sn.z, sn.w, x[4 * q + 2], x[4 * q + 3]);
                        }
                    }
                }
            }
            if (u >= units) continue;
            const uint4 y = isv ? raw[k] : rope_pack(x);
            const long long row = row0 + r;
            if (isq) {
                *reinterpret_cast<uint4*>(A.q_out + row * A.qo_stride + static_cast<long long>(h) * HD + c * 8) = y;
            } else if (A.k_out) {
                *reinterpret_cast<uint4*>(A.k_out + row * A.ko_stride + static_cast<long long>(h - A.Hq) * HD + c * 8) = y;
            } else if (s_at[r] >= 0) {
                const int g = h - A.Hq - (isv ? A.Hkv : 0);
                *reinterpret_cast<uint4*>((isv ? A.vpool : A.kpool) + s_at[r] + static_cast<long long>(g) * A.page * HD + c * 8) = y;
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
    // Few rows: one pass of heads per CTA, so that a row's heads spread over the SMs; more: as many
    // passes as keep the CTAs to one wave (8 of 256 threads per SM), up to the ROPE_U whose loads go
    // out together; many rows: several per CTA, up to four passes, so that the loads of a pass are all
    // used and what a CTA does once is done for more.  Measured: 500 rows of 32 heads of 256, one pass
    // 8.7 us, this rule 6.0; 8192 rows of 24 heads of 64, a row per CTA 30.7 us, five 15.0, six 17.1; of
    // 48 heads of 128, a row 47.7, four 43; of 28 heads of 256, a row 60.8, four 54; 4096 rows of 32
    // heads of 256, a row 31.4, three 32.1.
    int sms = 0;
    if (xv_status st = device_sm_count(&sms)) return st;
    int hpc = hpp, rpc = 1;
    while (hpc < ROPE_U * hpp && hpc < H && static_cast<long long>(a.M) * ceil_div(H, hpc) > 8ll * sms) hpc += hpp;
    if (hpc >= H) {
        hpc = H;
        // units of a full pass's loads, of r rows' passes: the r that leaves the least of them empty
        const int pass = ROPE_U * hpp;
        auto room = [&](int r) { return ceil_div(r * H, pass) * pass; };
        for (int r = 2; r <= ROPE_ROWS && r * H <= 4 * pass && r * H < 512 && r * a.rot / 2 <= ROPE_TAB && a.M / r >= 8 * sms; ++r)
            if (static_cast<long long>(r) * room(rpc) >= static_cast<long long>(rpc) * room(r)) rpc = r;
    }
    const dim3 grid(ceil_div(a.M, rpc), ceil_div(H, hpc));
    const unsigned inv_h = (65536u + hpc - 1) / hpc;
    trace_pre(s);
    auto go = [&](auto kern) { launch_k(kern, grid, dim3(ROPE_THREADS), 0, s, a, hpc, rpc, inv_h); };
    if (a.inter) hd == 256 ? go(qk_norm_rope_kernel<256, true>) : hd == 128 ? go(qk_norm_rope_kernel<128, true>) : go(qk_norm_rope_kernel<64, true>);
    else hd == 256 ? go(qk_norm_rope_kernel<256, false>) : hd == 128 ? go(qk_norm_rope_kernel<128, false>) : go(qk_norm_rope_kernel<64, false>);
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

// Decode-row attention over an 8-bit KV cache, whole contexts or a sliding window with sinks.
//
// A row of length len sees the positions below len, or with a window W those of them at or past
// len - W and the first `sinks`.  With codes k_j, v_j (e4m3) and scales ks_j, vs_j per position:
//     s_j = (q . k_j) ks_j scale,  out = sum_j exp(s_j) vs_j v_j / sum_j exp(s_j).
// In log2 units t_j = s_j log2(e) + log2(vs_j): the weight of the code v_j is 2^t_j, that of the
// softmax's sum 2^t_j / vs_j, so one exponential serves both, and the running reference m follows
// the t_j, i.e. what the output's terms weigh:
//     p_j = 2^(t_j - m + P_SHIFT),  O += p_j v_j,  l += p_j / vs_j.
//
// Exactness ("Follow-up to my earlier post on Qwen3.8-27B decode speed", r/LocalLLaMA post: verify
// attention as decode rows): positions are cut into splits at fixed absolute boundaries and tiles of
// 64; a row goes through its tiles in order, a tile without a position it sees leaves its m, l and O
// as they were, and its splits are joined in a fixed order.  A row's bits depend on its own length,
// q and what it sees, not on the rows and sequences beside it.
//
// The products run on tcgen05, accumulators in tensor memory:
//   S = Q K^T   in e4m3, K straight from its TMA stage.  A bf16 q is the sum of two e4m3 values (the
//               nearest, and the nearest to what is left): both go through the tensor core into one
//               accumulator, at fp8's rate as dear as one bf16 product and without a pass that widens
//               K.  A row is scaled by a power of two first, its largest value into [128, 256).
//   O += P V    in fp16: P needs more range than two e4m3 terms have (a weight 2^-17 of the largest
//               would be 0, and a long context can hold half its weight in such), so V is widened
//               (exactly) by warps of their own between its TMA stage and the tensor core's operand.
//               P_SHIFT puts p at up to 2^15: fp16 keeps weights to 2^-21 of the reference at full
//               precision (and to 2^-31 at all), and the reference may stay up to RESCALE_SLACK below
//               the row's largest t_j: with a slack of 2 every fifth tile of a row waited for the
//               P V before it to rescale O.  P is written over S in tensor memory, where the MMA reads it.
//
// Kernel 1 (attn_q8_kernel): work items (slot, 64-row tile, kv head, sequence); a slot is a split,
// or with a window one of the splits that the window and the sinks can touch.  One CTA per item up
// to two waves of them, else persistent CTAs that walk contiguous ranges.  Kernel 2
// (attn_q8_combine_kernel): one CTA per (row, q head) joins the row's splits.
#include <cmath>

#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

constexpr int T = 64;                  // positions per tile
constexpr float NEG_INF = -INFINITY;
constexpr float P_SHIFT = 7.f, RESCALE_SLACK = 8.f;

// Split boundaries: Q8_SHORT positions each below Q8_SWITCH, Q8_LONG beyond.
constexpr int Q8_SHORT = 256, Q8_SWITCH = 4096, Q8_LONG = 1024;
__host__ __device__ inline int q8_split_begin(int s) {
    constexpr int NS = Q8_SWITCH / Q8_SHORT;
    return s < NS ? s * Q8_SHORT : Q8_SWITCH + (s - NS) * Q8_LONG;
}
// The split that position p lies in.
__host__ __device__ inline int q8_split_of(int p) {
    return p < Q8_SWITCH ? p / Q8_SHORT : Q8_SWITCH / Q8_SHORT + (p - Q8_SWITCH) / Q8_LONG;
}

template <int HD>
struct Shape {
    static constexpr int KROW = HD < 128 ? HD : 128;          // bytes of a code row in a swizzled block
    static constexpr int KB = HD / KROW;                      // code blocks [64 positions][KROW] per tile
    static constexpr int KBLK = T * KROW;
    static constexpr int CODE = T * HD;                       // one K or V tile of codes
    static constexpr int VB = HD / 64;                        // fp16 blocks [64 positions][64 dims]
    static constexpr int VBLK = T * 128;
    static constexpr int VWIDE = VB * VBLK;                   // one fp16 V tile
    static constexpr int SK = HD == 128 ? 3 : 4, SV = 3, SW = 2;
    static constexpr int CONV = HD == 256 ? 4 : 2;            // widening warps
    static constexpr int WARPS = 8 + CONV, THREADS = 32 * WARPS;
    static constexpr int Q_THREADS = 32 * (4 + CONV);
    static constexpr int PER_SM = HD == 256 ? 1 : 2;
    static constexpr int SC = 4;                              // slots of prepared scales
    static constexpr int RAW = 8;                             // tiles whose scales are on their way
    // the MMA reads 128 rows of Q: rows 64..127 of a block are what follows it, and end in tensor
    // memory lanes that nobody reads
    static constexpr int Q_OFF = 0;                           // nearest terms, then what is left
    static constexpr int K_OFF = Q_OFF + 2 * CODE;
    static constexpr int V_OFF = K_OFF + SK * CODE;
    static constexpr int W_OFF = V_OFF + SV * CODE;
    static constexpr int BAR_OFF = W_OFF + SW * VWIDE;
    static constexpr int N_BARS = 2 * (SK + SV + SW + SC) + 2 + 2 + 2 + 5;
    static constexpr int SMEM = 1024 + BAR_OFF + 8 * N_BARS;
    static constexpr uint32_t O_COL = 2 * T;
    static constexpr uint32_t TMEM_COLS = HD == 256 ? 512 : 256;
    static_assert(O_COL + HD <= TMEM_COLS, "");
    static_assert(KBLK % 1024 == 0 && VBLK % 1024 == 0 && PER_SM * (SMEM + 9 * 1024 + 256) <= 228 * 1024, "");
};

struct Q8Args {
    const uint16_t* q;
    long long q_stride;
    KvPages kv;
    const float* k_scale;
    const float* v_scale;
    const int32_t* ctx_len;
    const int32_t* n_rows;
    int R, G, Hq, Hkv, B;
    int nslot, nsink;    // slots per row, of which the first nsink are the sinks' splits
    int max_len, window, sinks;
    int shift;           // the window, where the slots past the sinks' begin at it; 0: slots are splits
    float sl2;           // scale * log2(e)
    float* opart;        // [B*R*Hq][nslot][HD]
    float2* ml;          // [B*R*Hq][nslot]
    unsigned* err;
};

// Rows of sequence b.
__device__ __forceinline__ int q8_rows(const int32_t* n_rows, int b, int R) {
    return n_rows ? min(max(__ldg(n_rows + b), 0), R) : R;
}
// First split of the slots past the sinks', for a sequence whose first row has length L0.
__device__ __forceinline__ int q8_first(int L0, int shift, int nsink) {
    return shift && L0 > shift ? max(nsink, q8_split_of(L0 - shift)) : nsink;
}

struct Item {
    int b, g, row_base, slot, L0, rows, maxlen, p_begin;
    int ntiles, head, skip;   // live tiles: the split's first `head`, then from tile head + skip on
    bool live, bad;
    __device__ __forceinline__ int pos(int i) const { return p_begin + (i < head ? i : i + skip) * T; }
};

// (Out of line: in every role's loop the warps' code outgrew the instruction caches.)
__device__ __noinline__ Item q8_item(const Q8Args& A, int it, int nrt) {
    Item I;
    I.slot = it % A.nslot;
    int rest = it / A.nslot;
    I.row_base = (rest % nrt) * 64;
    rest /= nrt;
    I.g = rest % A.Hkv;
    I.b = rest / A.Hkv;
    const int nr = q8_rows(A.n_rows, I.b, A.R);
    I.rows = nr * A.G;
    I.L0 = __ldg(A.ctx_len + I.b);
    I.bad = nr > 0 && (I.L0 < 1 || I.L0 > A.max_len - nr + 1);
    I.live = !I.bad && I.row_base < I.rows;
    I.ntiles = I.head = I.skip = I.maxlen = I.p_begin = 0;
    if (!I.live) return I;
    // the longest and the shortest length among the item's rows; what other rows see beside a row
    // changes nothing of it
    I.maxlen = I.L0 + (min(I.rows, I.row_base + 64) - 1) / A.G;
    const int minlen = I.L0 + I.row_base / A.G;
    const int split = I.slot < A.nsink ? I.slot : q8_first(I.L0, A.shift, A.nsink) + I.slot - A.nsink;
    I.p_begin = q8_split_begin(split);
    const int end = min(q8_split_begin(split + 1), I.maxlen);
    const int nt = max(0, end - I.p_begin + T - 1) / T;
    int lo = 0;   // first tile that a window reaches
    if (A.window && minlen > A.window) {
        lo = min(nt, max(0, minlen - A.window - I.p_begin) / T);
        I.head = min(lo, max(0, A.sinks - I.p_begin + T - 1) / T);
    }
    I.skip = lo - I.head;
    I.ntiles = nt - I.skip;
    I.live = I.ntiles > 0;
    return I;
}

__device__ __forceinline__ int q8_page(const KvPages& kv, int b, int p, int* row, unsigned* err) {
    if (!kv.table) {
        *row = p;
        return b;
    }
    const int j = p / kv.page;
    *row = p - j * kv.page;
    int pg = kv.table[static_cast<long long>(b) * kv.max_pages + j];
    if (pg < 0 || pg >= kv.n_pages) {
        atomicOr(err, ERR_BAD_PAGE);
        pg = 0;
    }
    return pg;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 values as fp16, exactly.
__device__ __forceinline__ uint32_t f16x2_of(uint16_t e) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(e));
    return r;
}
__device__ __forceinline__ float2 floats_of(uint32_t h2) {
    float2 f;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h2));
    return f;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Live Q rows of an item -> tile row, as two e4m3 terms of q 2^e (the row's largest magnitude in
// [128, 256)) in swizzled blocks, and fac[row] = 2^-e.  NT threads (whole warps) from t0.
template <int HD, int NT>
__device__ __forceinline__ void load_q(uint8_t* sq, float* fac, const Q8Args& A, const Item& I, int t0) {
    using S = Shape<HD>;
    constexpr int LPH = HD / 8, RPP = NT / LPH, UN = 4;
    const int n = min(64, I.rows - I.row_base), c = t0 % LPH;
    for (int r0 = 0; r0 < n; r0 += RPP * UN) {
        uint4 v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int row = r0 + k * RPP + t0 / LPH;
            v[k] = make_uint4(0, 0, 0, 0);
            if (row < n) {
                const int r = (I.row_base + row) / A.G, h = I.g * A.G + (I.row_base + row) % A.G;
                v[k] = *reinterpret_cast<const uint4*>(A.q + (static_cast<long long>(I.b) * A.R + r) * A.q_stride +
                                                       static_cast<long long>(h) * HD + c * 8);
            }
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int row = r0 + k * RPP + t0 / LPH;
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            unsigned big = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) big = max(big, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
            for (int off = LPH / 2; off > 0; off >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
            if (row >= n) continue;
            const bool bad = big >= 0x7f80u;
            const int e = 134 - max(static_cast<int>(big >> 7), 8);   // 2^e: the exponent field to 134, e <= 126
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = __fmul_rn(__uint_as_float(w[i] << 16), up), b = __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), up);
                const uint32_t h = bad ? 0x7f7fu : e4m3x2(a, b);
                const float2 f = floats_of(f16x2_of(static_cast<uint16_t>(h)));
                const uint32_t l = bad ? 0u : e4m3x2(__fsub_rn(a, f.x), __fsub_rn(b, f.y));
                hi[i >> 1] |= h << (16 * (i & 1));
                lo[i >> 1] |= l << (16 * (i & 1));
            }
            const int byte = c * 8, blk = byte / S::KROW, chunk = (byte % S::KROW) >> 4;
            const int sw = S::KROW == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
            uint8_t* dst = sq + blk * S::KBLK + row * S::KROW + sw * 16 + (byte & 8);
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(dst + S::CODE) = make_uint2(lo[0], lo[1]);
            if (c == 0) fac[row] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        }
    }
}

// K-major operand in rows of 64 bytes with the 64-byte swizzle (groups of 8 rows 512 bytes apart).
__device__ __forceinline__ uint64_t sw64_kmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(16u >> 4) << 16;
    d |= static_cast<uint64_t>(512u >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(4) << 61;
    return d;
}
template <int ROW>
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t saddr) {
    return ROW == 128 ? sw128_kmajor_desc(saddr) : sw64_kmajor_desc(saddr);
}
// Instruction descriptor: fp32 accumulator; the input formats' fields are 0 for e4m3 (kind::f8f6f4)
// and for fp16 (kind::f16) alike.
constexpr uint32_t idesc0(int M, int N, bool b_mn_major = false) {
    return (1u << 4) | (b_mn_major ? (1u << 16) : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D (+)= A B^T, e4m3 operands in shared memory.
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D (+)= A B^T, fp16, A in tensor memory.
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Two fp32 operations in one instruction: (a, b) *= (x, y); (u, v) = (u, v) (x, y) + (a, b); (a, b) += (x, y).
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
__device__ __forceinline__ void fma2(float& u, float& v, float x, float y, float a, float b) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(u), "+f"(v) : "f"(x), "f"(y), "f"(a), "f"(b));
}
// (u, v) += (x, y) (a, b)
__device__ __forceinline__ void fma2_acc(float& u, float& v, float x, float y, float a, float b) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%0, %1};\n\t"
        "fma.rn.f32x2 r, p, q, r;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "+f"(u), "+f"(v) : "f"(x), "f"(y), "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
// Bounded wait: after one of the CTA's waits has given up, every later one returns at once.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t par, volatile int* aborted, unsigned* err) {
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (mbar_try_wait(bar, par)) return true;
        if (*aborted) return false;
        if (globaltimer() - t0 > WAIT_LIMIT_NS) {
            atomicOr(err, ERR_WAIT_TIMEOUT);
            *aborted = 1;
            return false;
        }
    }
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The tiles of a CTA's items in order.  With PLACE a whole warp steps, and lane i looks up where tile i
// of an item lies, so that a page table's latency is met once per item.
template <bool PLACE>
struct Tiles {
    Item I;
    int it, i;       // item, and the next tile of it
    int z, row;      // lane i: head of the pools and row in it of tile i
    __device__ __forceinline__ void look(const Q8Args& A) {
        if (!PLACE) return;
        const int lane = threadIdx.x & 31;
        if (lane < I.ntiles) z = q8_page(A.kv, I.b, I.pos(lane), &row, A.err) * A.Hkv + I.g;
    }
    __device__ __forceinline__ void start(const Q8Args& A, int first, int nrt) {
        it = first;
        i = z = row = 0;
        I = q8_item(A, it, nrt);
        look(A);
    }
    // steps to the next tile; false past the last
    __device__ __forceinline__ bool step(const Q8Args& A, int it1, int nrt) {
        if (++i < I.ntiles) return true;
        i = 0;
        while (++it < it1) {
            I = q8_item(A, it, nrt);
            if (I.live) {
                look(A);
                return true;
            }
        }
        return false;
    }
    __device__ __forceinline__ int head() const { return __shfl_sync(0xffffffffu, z, i); }
    __device__ __forceinline__ int place() const { return __shfl_sync(0xffffffffu, row, i); }
};
static_assert(Q8_LONG <= 32 * T && Q8_SHORT <= 32 * T, "a lane per tile of an item");

// Warps of a CTA and what they do per tile t (counted over the CTA's items):
//   2, 3   TMA of the K and V codes into their rings
//   7      the tile's scales: ks, log2(vs) and 1 / vs of its positions into a ring of prepared slots
//   8..    widen the V codes to fp16 (positions past every row's length become 0)
//   6      MMAs: S(t + 1) = Q K^T, then O += P(t) V; S(t) and P(t) share buffer t % 2: the S that
//          overwrites a P is issued after the P V that reads it, and MMAs run in order
//   0, 1   softmax, a thread per query row: S out of tensor memory, t_j, mask, reference (moved when
//          the tile's largest t_j passes it by RESCALE_SLACK, and then O and l are rescaled), P back
//   4, 5   an item's O, m and l to the workspace, while the next item's first tiles run
template <int HD, bool MULTI>
__global__ void __launch_bounds__(Shape<HD>::THREADS, Shape<HD>::PER_SM)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Q8Args A) {
    griddep_launch();
    using S = Shape<HD>;
    constexpr int SK = S::SK, SV = S::SV, SW = S::SW, SC = S::SC, RAW = S::RAW, CONV = S::CONV;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int s_abort;
    __shared__ float2 ml_sm[64];                        // (m, l) of the item being written out
    __shared__ float q_fac[2][64];                      // by the count of Q loads
    __shared__ __align__(16) float sc_ks[SC][T], sc_lv[SC][T], sc_iv[SC][T];
    __shared__ float raw_k[RAW][T], raw_v[RAW][T];
    const uint32_t rawb = smem_u32(smem_raw);
    const uint32_t base = (rawb + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - rawb);
    auto sK = [&](int st) { return base + S::K_OFF + st * S::CODE; };
    auto sV = [&](int st) { return base + S::V_OFF + st * S::CODE; };
    auto sW = [&](int st) { return base + S::W_OFF + st * S::VWIDE; };
    const uint32_t bar0 = base + S::BAR_OFF;
    auto fullK = [&](int st) { return bar0 + 8u * st; };
    auto emptyK = [&](int st) { return bar0 + 8u * (SK + st); };
    const uint32_t bar1 = bar0 + 8u * 2 * SK;
    auto fullV = [&](int st) { return bar1 + 8u * st; };
    auto emptyV = [&](int st) { return bar1 + 8u * (SV + st); };
    const uint32_t bar2 = bar1 + 8u * 2 * SV;
    auto fullW = [&](int st) { return bar2 + 8u * st; };
    auto emptyW = [&](int st) { return bar2 + 8u * (SW + st); };
    const uint32_t bar3 = bar2 + 8u * 2 * SW;
    auto fullS = [&](int st) { return bar3 + 8u * st; };
    auto emptyS = [&](int st) { return bar3 + 8u * (SC + st); };
    const uint32_t bx = bar3 + 8u * 2 * SC;
    auto sbar = [&](int j) { return bx + 8u * j; };           // S of a tile is complete
    auto pready = [&](int j) { return bx + 8u * (2 + j); };   // its P is in tensor memory
    auto pfree = [&](int j) { return bx + 8u * (4 + j); };    // its P V is complete
    const uint32_t done = bx + 8u * 6, ofree = bx + 8u * 7, qfull = bx + 8u * 8, mlready = bx + 8u * 9, qfirst = bx + 8u * 10;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nrt = (A.R * A.G + 63) / 64;
    const int n_items = A.nslot * nrt * A.Hkv * A.B;
    const int per_slot = n_items / A.nslot;
    // one item per CTA: slots slowest, so that a row's last splits, often short, come last
    const int it0 = MULTI ? static_cast<int>(static_cast<long long>(blockIdx.x) * n_items / gridDim.x)
                          : (static_cast<int>(blockIdx.x) % per_slot) * A.nslot + static_cast<int>(blockIdx.x) / per_slot;
    const int it1 = MULTI ? static_cast<int>(static_cast<long long>(blockIdx.x + 1) * n_items / gridDim.x) : it0 + 1;
    griddep_wait();
    int first = it0;
    while (first < it1 && !q8_item(A, first, nrt).live) ++first;
    if (tid == 0)
        for (int it = it0; it < it1; ++it) {
            const Item I = q8_item(A, it, nrt);
            if (I.slot || I.row_base || I.g) continue;
            if (I.bad) atomicOr(A.err, ERR_BAD_LENGTH);
            if (A.n_rows && (A.n_rows[I.b] < 0 || A.n_rows[I.b] > A.R)) atomicOr(A.err, ERR_BAD_COUNT);
        }
    if (first >= it1) return;   // nothing live here: no barrier or tensor memory was set up

    if (tid == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        for (int st = 0; st < SK; ++st) mbar_init(fullK(st), 1), mbar_init(emptyK(st), 1);
        for (int st = 0; st < SV; ++st) mbar_init(fullV(st), 1), mbar_init(emptyV(st), CONV);
        for (int st = 0; st < SW; ++st) mbar_init(fullW(st), CONV), mbar_init(emptyW(st), 1);
        for (int st = 0; st < SC; ++st) mbar_init(fullS(st), 1), mbar_init(emptyS(st), 2);
        for (int j = 0; j < 2; ++j) mbar_init(sbar(j), 1), mbar_init(pready(j), 64), mbar_init(pfree(j), 1);
        mbar_init(done, 1);
        mbar_init(ofree, 64);
        mbar_init(qfull, 64);
        mbar_init(mlready, 64);
        mbar_init(qfirst, S::Q_THREADS);
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_slot), S::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = tmem_slot, tO = tS + S::O_COL;
    // the warps that wait for tiles anyway load the first item's Q; the softmax warps reload it when an
    // item's differs
    if (warp < 2 || warp == 4 || warp == 5 || warp >= 8) {
        load_q<HD, S::Q_THREADS>(smem + S::Q_OFF, q_fac[0], A, q8_item(A, first, nrt), tid - (warp < 2 ? 0 : warp < 8 ? 64 : 128));
        fence_proxy_async_smem();
        mbar_arrive(qfirst);
    }

    auto W = [&](uint32_t bar, uint32_t par) -> bool { return mbar_try_wait(bar, par) || wait_slow(bar, par, &s_abort, A.err); };
    // the same verdict for every lane of a warp
    auto WW = [&](uint32_t bar, uint32_t par) -> bool { return __all_sync(0xffffffffu, W(bar, par)); };
    auto same_q = [](const Item& x, int b, int g, int rb) { return x.b == b && x.g == g && x.row_base == rb; };

    if (warp == 2 || warp == 3) {
        // ---- TMA
        const bool isK = warp == 2;
        const int NS = isK ? SK : SV;
        const CUtensorMap* map = isK ? &tmK : &tmV;
        int t = 0;
        Tiles<true> x;
        x.start(A, first, nrt);
        do {
            const int st = t % NS, z = x.head(), row = x.place();
            if (t >= NS && !WW(isK ? emptyK(st) : emptyV(st), ((t / NS) & 1u) ^ 1u)) break;
            if (lane == 0) {
                const uint32_t fb = isK ? fullK(st) : fullV(st), dst = isK ? sK(st) : sV(st);
                mbar_arrive_expect_tx(fb, S::CODE);
#pragma unroll
                for (int cb = 0; cb < S::KB; ++cb) tma_load_3d(dst + cb * S::KBLK, map, cb * S::KROW, row, z, fb);
            }
            ++t;
        } while (x.step(A, it1, nrt));
        // every issued copy lands before the CTA may leave
        for (int j = t > NS ? t - NS : 0; j < t; ++j) mbar_wait(isK ? fullK(j % NS) : fullV(j % NS), (j / NS) & 1u, A.err);
    } else if (warp == 7) {
        // ---- scales: every lane copies those of its two positions RAW - 1 tiles ahead, and reads only
        // what it copied itself
        Tiles<true> x;   // copying
        Tiles<false> y;  // preparing
        x.start(A, first, nrt);
        y.start(A, first, nrt);
        bool more = true;
        int tc = 0;
        auto copy = [&]() {
            if (more) {
                const int p = x.I.pos(x.i);
                const long long at = static_cast<long long>(x.head()) * A.kv.page + x.place();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j = lane + 32 * h;
                    const bool in = p + j < x.I.maxlen;
                    const long long a = in ? at + j : 0;
                    cp_async4(smem_u32(&raw_k[tc % RAW][j]), A.k_scale + a, in);
                    cp_async4(smem_u32(&raw_v[tc % RAW][j]), A.v_scale + a, in);
                }
                ++tc;
                more = x.step(A, it1, nrt);
            }
            cp_async_commit();   // a group per call, an empty one past the last tile
        };
        for (int i = 0; i < RAW - 1; ++i) copy();
        int t = 0;
        do {
            copy();   // into the slot that the last round has read
            cp_async_wait<RAW - 1>();
            const int st = t % SC;
            if (t >= SC && !WW(emptyS(st), ((t / SC) & 1u) ^ 1u)) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = lane + 32 * h;
                const bool in = y.I.pos(y.i) + j < y.I.maxlen;
                const float vs = raw_v[t % RAW][j];
                const float vc = fminf(fmaxf(vs, 0x1p-40f), 0x1p60f);   // a NaN becomes 2^-40
                sc_ks[st][j] = in ? raw_k[t % RAW][j] : 0.f;
                sc_lv[st][j] = !in ? 0.f : vs != vs ? vs : lg2_approx(vc);   // a NaN scale speaks through t_j alone
                sc_iv[st][j] = in ? __frcp_rn(vc) : 1.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fullS(st));
            ++t;
        } while (y.step(A, it1, nrt));
        cp_async_wait_all();
    } else if (warp >= 8) {
        // ---- V codes to fp16.  A lane takes 16 dims of a position: 8 positions x 4 such chunks per
        // pass of a warp, so both sides of the swizzles meet every bank once per 8 lanes
        constexpr int CPR = HD / 64, PASSES = 8 * CPR / CONV;   // column groups of 64 dims; passes per warp
        const int r8 = lane & 7, c4 = lane >> 3;
        int t = 0;
        Tiles<false> x;
        x.start(A, first, nrt);
        do {
            const int sv = t % SV, sw = t % SW;
            if (!WW(fullV(sv), (t / SV) & 1u)) break;
            if (t >= SW && !WW(emptyW(sw), ((t / SW) & 1u) ^ 1u)) break;
            const int left = x.I.maxlen - x.I.pos(x.i);
            const uint8_t* src = smem + (sV(sv) - base);
            uint8_t* dst = smem + (sW(sw) - base);
#pragma unroll 4
            for (int i = 0; i < PASSES; ++i) {
                const int u = (warp - 8) * PASSES + i, row = (u / CPR) * 8 + r8, cg = u % CPR;   // cg: 64 dims
                const int byte = cg * 64 + c4 * 16, blk = byte / S::KROW, ch = (byte % S::KROW) >> 4;
                const int chs = S::KROW == 128 ? ch ^ r8 : ch ^ (r8 >> 1);
                const uint4 e = *reinterpret_cast<const uint4*>(src + blk * S::KBLK + row * S::KROW + chs * 16);
                uint4 a = make_uint4(0, 0, 0, 0), b = a;
                if (row < left) {
                    a = make_uint4(f16x2_of(e.x & 0xffff), f16x2_of(e.x >> 16), f16x2_of(e.y & 0xffff), f16x2_of(e.y >> 16));
                    b = make_uint4(f16x2_of(e.z & 0xffff), f16x2_of(e.z >> 16), f16x2_of(e.w & 0xffff), f16x2_of(e.w >> 16));
                }
                uint8_t* d = dst + cg * S::VBLK + row * 128;
                *reinterpret_cast<uint4*>(d + (((2 * c4) ^ r8) * 16)) = a;
                *reinterpret_cast<uint4*>(d + (((2 * c4 + 1) ^ r8) * 16)) = b;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(emptyV(sv));
                mbar_arrive(fullW(sw));
            }
            ++t;
        } while (x.step(A, it1, nrt));
    } else if (warp == 6) {
        // ---- MMAs
        if (lane == 0) {
            constexpr uint32_t IDS = idesc0(128, T), IDO = idesc0(128, HD, true);
            constexpr uint32_t VBLK = S::VB > 1 ? S::VBLK : 1024;
            constexpr int KS = S::KROW / 32;   // MMAs of 32 codes per block row
            const uint32_t sQ = base + S::Q_OFF;
            auto qk = [&](int tt) -> bool {
                const int st = tt % SK;
                if (!W(fullK(st), (tt / SK) & 1u)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < HD / 32; ++ks) {
                    const uint32_t off = (ks / KS) * S::KBLK + (ks % KS) * 32;
                    const uint64_t bd = kmajor_desc<S::KROW>(sK(st) + off);
                    mma_fp8(tS + (tt & 1) * T, kmajor_desc<S::KROW>(sQ + off), bd, IDS, ks > 0 ? 1u : 0u);
                    mma_fp8(tS + (tt & 1) * T, kmajor_desc<S::KROW>(sQ + S::CODE + off), bd, IDS, 1u);
                }
                tc_commit(sbar(tt & 1));
                tc_commit(emptyK(st));
                return true;
            };
            int t = 0, jl = 0, nq = 0, qb = -1, qg = -1, qrb = -1;
            bool ok = W(qfirst, 0u), pre = false;   // pre: this item's first S went out with the last item
            for (int it = first; ok && it < it1; ++it) {
                const Item I = q8_item(A, it, nrt);
                if (!I.live) continue;
                if (MULTI && jl > 0 && !same_q(I, qb, qg, qrb)) {
                    if (!W(qfull, nq & 1u)) break;
                    ++nq;
                }
                qb = I.b, qg = I.g, qrb = I.row_base;
                if (!pre && !qk(t)) break;
                pre = false;
                bool next_same = false;   // the next live item has this Q: its first S goes out before the last P V
                if (MULTI) {
                    int nx = it + 1;
                    while (nx < it1 && !q8_item(A, nx, nrt).live) ++nx;
                    next_same = nx < it1 && same_q(q8_item(A, nx, nrt), I.b, I.g, I.row_base);
                }
                for (int i = 0; i < I.ntiles; ++i) {
                    const int tt = t + i, sw = tt % SW;
                    if ((i + 1 < I.ntiles || next_same) && !qk(tt + 1)) { ok = false; break; }
                    if (i + 1 == I.ntiles && next_same) pre = true;
                    if (MULTI && i == 0 && jl > 0 && !W(ofree, (jl - 1) & 1u)) { ok = false; break; }
                    if (!W(pready(tt & 1), (tt >> 1) & 1u) || !W(fullW(sw), (tt / SW) & 1u)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < T / 16; ++kk)   // 16 positions: 8 columns of P, two 8-row groups of V
                        mma_f16_ta(tO, tS + (tt & 1) * T + kk * 8, sw128_mnmajor_desc(sW(sw) + kk * 2048, VBLK, 1024), IDO,
                                   (i > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(pfree(tt & 1));
                    tc_commit(emptyW(sw));
                }
                t += I.ntiles;
                ++jl;
            }
            tc_commit(done);   // every MMA issued is complete before the CTA may leave
            mbar_wait(done, 0u, A.err);
        }
    } else if (warp >= 4) {
        // ---- epilogue: thread = tile row rho (tensor memory lane rho)
        const int rho = tid - 128;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        int t = 0, jl = 0;
        for (int it = first; it < it1; ++it) {
            const Item I = q8_item(A, it, nrt);
            if (!I.live) continue;
            const int tl = t + I.ntiles - 1;
            if (!WW(mlready, jl & 1u) || !WW(pfree(tl & 1), (tl >> 1) & 1u)) break;
            tc_fence_after();
            const int grow = I.row_base + rho;
            const bool live = grow < I.rows;
            const int r = grow / A.G, h = I.g * A.G + grow % A.G;
            const long long idx = ((static_cast<long long>(I.b) * A.R + r) * A.Hq + h) * A.nslot + I.slot;
            float* op = A.opart + idx * HD;
            const float2 ml = ml_sm[rho];
            if (__any_sync(0xffffffffu, live)) {
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    float o[32];
#pragma unroll
                    for (int q2 = 0; q2 < 2; ++q2) tmem_ld16(tO + lane_off + c * 32 + q2 * 16, o + q2 * 16);
                    tmem_ld_wait();
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(op + c * 32 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (live) A.ml[idx] = ml;
            }
            tc_fence_before();
            mbar_arrive(ofree);   // O (and ml_sm) may be overwritten by the next item
            t += I.ntiles;
            ++jl;
        }
    } else {
        // ---- softmax: thread = tile row rho (tensor memory lane rho)
        const int rho = tid;
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        int t = 0, jl = 0, nq = 0, qb = -1, qg = -1, qrb = -1;
        const bool q_in = WW(qfirst, 0u);
        for (int it = first; q_in && it < it1; ++it) {
            const Item I = q8_item(A, it, nrt);
            if (!I.live) continue;
            if constexpr (MULTI) {
                if (jl > 0 && !same_q(I, qb, qg, qrb)) {
                    // every S of the old Q is complete (this warp has seen the last), and the MMA warp
                    // issues none of this item until qfull
                    load_q<HD, 64>(smem + S::Q_OFF, q_fac[(nq + 1) & 1], A, I, rho);
                    fence_proxy_async_smem();
                    mbar_arrive(qfull);
                    if (!WW(qfull, nq & 1u)) break;   // the other warp's factors too
                    ++nq;
                }
            }
            qb = I.b, qg = I.g, qrb = I.row_base;
            const int grow = I.row_base + rho;
            const int len = grow < I.rows ? I.L0 + grow / A.G : 0;
            const int from = A.window ? max(0, len - A.window) : 0;   // sees [from, len) and [0, upto)
            const int upto = min(A.sinks, len);
            const bool mine = grow < I.rows, any = I.row_base + 32 * warp < I.rows;   // a row; a row in the warp
            const float c = mine ? __fmul_rn(A.sl2, q_fac[nq & 1][rho]) : 0.f;
            float m = NEG_INF, l = 0.f;
            bool ok = true;
            for (int i = 0; i < I.ntiles; ++i) {
                const int tt = t + i, sc = tt % SC;
                if (!WW(fullS(sc), (tt / SC) & 1u) || !WW(sbar(tt & 1), (tt >> 1) & 1u)) { ok = false; break; }
                tc_fence_after();
                if (!any) {   // the whole warp's rows are behind the item's: their P is whatever S was
                    tc_fence_before();
                    mbar_arrive(pready(tt & 1));
                    if (lane == 0) mbar_arrive(emptyS(sc));
                    continue;
                }
                const int p0 = I.pos(i);
                const bool whole = __all_sync(0xffffffffu, !mine || (p0 >= from && p0 + T <= len));
                // t_j of 32 positions, twice: for their maximum, and again for p (registers for 64 and code
                // unrolled over them cost more than the second read)
                auto scores = [&](int j0, float* s) {
                    tmem_ld16(tS + lane_off + (tt & 1) * T + j0, s);
                    tmem_ld16(tS + lane_off + (tt & 1) * T + j0 + 16, s + 16);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 ks = *reinterpret_cast<const float4*>(&sc_ks[sc][j0 + j]);
                        const float4 lv = *reinterpret_cast<const float4*>(&sc_lv[sc][j0 + j]);
                        mul2(s[j], s[j + 1], c, c);
                        mul2(s[j + 2], s[j + 3], c, c);
                        fma2(s[j], s[j + 1], ks.x, ks.y, lv.x, lv.y);
                        fma2(s[j + 2], s[j + 3], ks.z, ks.w, lv.z, lv.w);
                    }
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int p = p0 + j0 + j;
                            if (!(p < len && (p >= from || p < upto))) s[j] = NEG_INF;
                        }
                    }
                };
                float mx4[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll 1
                for (int j0 = 0; j0 < T; j0 += 32) {
                    float s[32];
                    scores(j0, s);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mx4[(j / 2) & 3] = fmaxf(mx4[(j / 2) & 3], fmaxf(s[j], s[j + 1]));
                }
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                const float mn = (m == NEG_INF || mx > __fadd_rn(m, RESCALE_SLACK)) ? mx : m;
                const bool dead = mn == NEG_INF;
                const float al = (dead || mn == m) ? 1.f : ex2_approx(__fsub_rn(m, mn));
                const float mo = dead ? 0.f : __fsub_rn(mn, P_SHIFT);
                float ts[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int j0 = 0; j0 < T; j0 += 32) {
                    float s[32], pk[16];
                    scores(j0, s);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 iv = *reinterpret_cast<const float4*>(&sc_iv[sc][j0 + j]);
                        float* p = s + j;
                        add2(p[0], p[1], -mo, -mo);
                        add2(p[2], p[3], -mo, -mo);
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = ex2_approx(p[e]);
                        fma2_acc(ts[0], ts[1], p[0], p[1], iv.x, iv.y);
                        fma2_acc(ts[2], ts[3], p[2], p[3], iv.z, iv.w);
                        pk[j / 2] = __uint_as_float(pack_f16x2(p[0], p[1]));
                        pk[j / 2 + 1] = __uint_as_float(pack_f16x2(p[2], p[3]));
                    }
                    // over S columns that have been read: P of position j lies in column j / 2
                    tmem_st16(tS + lane_off + (tt & 1) * T + j0 / 2, pk);
                }
                l = __fmaf_rn(l, al, __fadd_rn(__fadd_rn(ts[0], ts[1]), __fadd_rn(ts[2], ts[3])));
                m = mn;
                // O is rescaled once P V of the tile before has completed
                if (i >= 1 && __any_sync(0xffffffffu, mine && al != 1.f)) {
                    if (!WW(pfree((tt - 1) & 1), ((tt - 1) >> 1) & 1u)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < HD / 32; ++k) {
                        float o[32];
#pragma unroll
                        for (int q2 = 0; q2 < 2; ++q2) tmem_ld16(tO + lane_off + k * 32 + q2 * 16, o + q2 * 16);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __fmul_rn(o[e], al);
#pragma unroll
                        for (int q2 = 0; q2 < 2; ++q2) tmem_st16(tO + lane_off + k * 32 + q2 * 16, o + q2 * 16);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(pready(tt & 1));
                __syncwarp();
                if (lane == 0) mbar_arrive(emptyS(sc));
            }
            if (!ok) break;
            // hand m and l to the epilogue warps (once they are done with the previous item's)
            if (MULTI && jl > 0 && !WW(ofree, (jl - 1) & 1u)) break;
            ml_sm[rho] = make_float2(m, l);
            mbar_arrive(mlready);
            t += I.ntiles;
            ++jl;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tS, S::TMEM_COLS);
    }
}

struct CombineArgs {
    const int32_t* ctx_len;
    const int32_t* n_rows;
    int R, Hq, nslot, nsink, max_len, window, sinks, shift;
    const float* opart;
    const float2* ml;
    const uint16_t* gate;
    long long gate_stride;
    uint16_t* out;
    long long out_stride;
};

// One CTA per (row, q head): w_s = 2^(m_s - M) over the row's live slots s in order, out = sum w_s O_s /
// sum w_s l_s.  CB_GROUPS groups of threads each add the slots of one residue, then the groups'
// sums are added in order: fixed by the row alone, and a long context's partials (140 splits at
// 131072) come in CB_GROUPS times fewer dependent steps.
constexpr int CB_GROUPS = 8;
constexpr int CB_SLOTS = 1 << 10;   // slots whose weights are staged at a time

template <int HD>
__global__ void __launch_bounds__(CB_GROUPS* HD / 4) attn_q8_combine_kernel(const __grid_constant__ CombineArgs C) {
    griddep_launch();
    griddep_wait();
    constexpr int LN = HD / 4, NT = CB_GROUPS * LN;
    __shared__ float2 wl[CB_SLOTS];
    __shared__ float4 acc_sm[CB_GROUPS][LN];
    __shared__ float l_sm[CB_GROUPS], wmax[NT / 32];
    const int hq = blockIdx.x % C.Hq;
    const long long br = blockIdx.x / C.Hq;
    const int b = static_cast<int>(br / C.R), r = static_cast<int>(br % C.R), tid = threadIdx.x;
    const int nr = q8_rows(C.n_rows, b, C.R), L0 = C.ctx_len[b];
    if (r >= nr || L0 < 1 || L0 > C.max_len - nr + 1) return;
    const int len = L0 + r;
    // the row's slots: those of the sinks it sees beside its window, then its window's
    const int first = q8_first(L0, C.shift, C.nsink);
    const int from = C.window ? max(0, len - C.window) : 0, upto = min(C.sinks, from);
    const int n0 = upto ? q8_split_of(upto - 1) + 1 : 0;             // splits with a sink
    const int s0 = max(n0, q8_split_of(from)), ns = n0 + q8_split_of(len - 1) + 1 - s0;
    auto slot = [&](int i) {
        const int s = i < n0 ? i : s0 + i - n0;
        return s < C.nsink ? s : s - first + C.nsink;
    };
    const long long idx0 = (br * C.Hq + hq) * C.nslot;
    float M = NEG_INF;
    for (int i = tid; i < ns; i += NT) M = fmaxf(M, C.ml[idx0 + slot(i)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if ((tid & 31) == 0) wmax[tid >> 5] = M;
    __syncthreads();
    M = wmax[0];
    for (int w = 1; w < NT / 32; ++w) M = fmaxf(M, wmax[w]);
    const int grp = tid / LN, ln = tid % LN;
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < ns; c0 += CB_SLOTS) {
        const int n = min(CB_SLOTS, ns - c0);
        __syncthreads();
        for (int i = tid; i < n; i += NT) {
            const float2 v = C.ml[idx0 + slot(c0 + i)];
            wl[i] = make_float2(exp2f(__fsub_rn(v.x, M)), v.y);
        }
        __syncthreads();
#pragma unroll 4
        for (int i = grp; i < n; i += CB_GROUPS) {
            const float2 w = wl[i];
            const float4 o = __ldcg(reinterpret_cast<const float4*>(C.opart + (idx0 + slot(c0 + i)) * HD) + ln);
            L = __fmaf_rn(w.x, w.y, L);
            a.x = __fmaf_rn(w.x, o.x, a.x);
            a.y = __fmaf_rn(w.x, o.y, a.y);
            a.z = __fmaf_rn(w.x, o.z, a.z);
            a.w = __fmaf_rn(w.x, o.w, a.w);
        }
    }
    acc_sm[grp][ln] = a;
    if (ln == 0) l_sm[grp] = L;
    __syncthreads();
    if (grp) return;
    for (int g = 1; g < CB_GROUPS; ++g) {
        const float4 o = acc_sm[g][ln];
        L = __fadd_rn(L, l_sm[g]);
        a.x = __fadd_rn(a.x, o.x), a.y = __fadd_rn(a.y, o.y), a.z = __fadd_rn(a.z, o.z), a.w = __fadd_rn(a.w, o.w);
    }
    float y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __fadd_rn(__fdiv_rn(y[e], L), 0.f);
    if (C.gate) {
        const uint2 g = *reinterpret_cast<const uint2*>(C.gate + br * C.gate_stride + static_cast<long long>(hq) * HD + 4 * ln);
        const float gv[4] = {__uint_as_float(g.x << 16), __uint_as_float(g.x & 0xffff0000u), __uint_as_float(g.y << 16),
                             __uint_as_float(g.y & 0xffff0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fmul_rn(y[e], __frcp_rn(__fadd_rn(1.f, expf(-gv[e]))));
    }
    *reinterpret_cast<uint2*>(C.out + br * C.out_stride + static_cast<long long>(hq) * HD + 4 * ln) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Slots of a row and, of them, the sinks': without a window the splits up to max_len; with one the
// sinks' splits and as many as a window and the rows behind it can touch.
inline int slots(int R, int max_len, int window, int sinks, int* nsink) {
    const int all = q8_split_of(max_len - 1) + 1;
    *nsink = 0;
    if (!window || window >= max_len) return all;
    const int ns = sinks ? q8_split_of(min(sinks, max_len) - 1) + 1 : 0;
    const long long w = (static_cast<long long>(window) + R - 2) / Q8_SHORT + 2;
    if (ns + w >= all) return all;   // then no slot is left out and none counts as a sink's
    *nsink = ns;
    return ns + static_cast<int>(w);
}

inline bool sizes_ok(int B, int R, int Hq, int hd, int max_ctx, int window, int sinks) {
    return B >= 1 && B <= 65535 && R >= 1 && R <= XV_KMAX && Hq >= 1 && (hd == 64 || hd == 128 || hd == 256) && max_ctx >= 1 &&
           max_ctx <= (1 << 30) && window >= 0 && sinks >= 0 && static_cast<long long>(B) * R * Hq <= (1ll << 30);
}

template <int HD>
xv_status launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const Q8Args& a, const CombineArgs& c, cudaStream_t s) {
    using S = Shape<HD>;
    int sms = 0;
    if (xv_status st = kernel_smem_once(reinterpret_cast<const void*>(attn_q8_kernel<HD, true>), S::SMEM, false, "attn_q8: set shared memory size"))
        return st;
    if (xv_status st = kernel_smem_once(reinterpret_cast<const void*>(attn_q8_kernel<HD, false>), S::SMEM, false, "attn_q8: set shared memory size"))
        return st;
    if (xv_status st = device_sm_count(&sms)) return st;
    const long long n_items = static_cast<long long>(a.nslot) * ((a.R * a.G + 63) / 64) * a.Hkv * a.B;
    if (n_items > (1ll << 30)) return fail(XV_ERR_UNSUPPORTED, "attn_q8: %lld work items", n_items);
    const int room = sms * S::PER_SM;
    const bool multi = n_items > 2ll * room;
    const dim3 grid(static_cast<unsigned>(multi ? room : n_items));
    trace_pre(s);
    if (multi) launch_k(attn_q8_kernel<HD, true>, grid, dim3(S::THREADS), S::SMEM, s, tmK, tmV, a);
    else launch_k(attn_q8_kernel<HD, false>, grid, dim3(S::THREADS), S::SMEM, s, tmK, tmV, a);
    const long long rows = static_cast<long long>(a.B) * a.R * a.Hq, seen = a.window && a.window < a.max_len ? a.window + a.sinks : a.max_len;
    if (xv_status st = launched("attn_q8_kernel", s, K_ATTN_Q8, (2ll * HD + 8) * a.B * a.Hkv * seen + 2 * rows * HD + 4 * rows * a.nslot * (HD + 2)))
        return st;
    trace_pre(s);
    launch_k(attn_q8_combine_kernel<HD>, dim3(static_cast<unsigned>(rows)), dim3(CB_GROUPS * HD / 4), 0, s, c);
    return launched("attn_q8_combine_kernel", s, K_ATTN_Q8, 4 * rows * a.nslot * (HD + 2) + 2 * rows * HD * (c.gate ? 2 : 1));
}

xv_status attn_q8(const uint16_t* q, long long q_stride, const xv_kv_q8* cache, const KvPages& kv, int Lmax,
                  const int32_t* ctx_len, const int32_t* n_rows, int R, int B, int Hq, int Hkv, int hd, int max_ctx, int window,
                  int sinks, float scale, const uint16_t* gate, long long gate_stride, uint16_t* out, long long out_stride,
                  void* ws, size_t ws_bytes, cudaStream_t s) {
    if (!q || !ctx_len || !out) return fail(XV_ERR_ARG, "attn_q8: null q, ctx_len or out");
    if (R < 1 || B < 1 || Hq < 1 || Hkv < 1) return fail(XV_ERR_ARG, "attn_q8: need R, B, Hq and Hkv >= 1");
    if (Hq % Hkv) return fail(XV_ERR_ARG, "attn_q8: Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
    if (max_ctx < 1 || max_ctx > Lmax) return fail(XV_ERR_ARG, "attn_q8: max_ctx = %d outside [1, Lmax = %d]", max_ctx, Lmax);
    if (window < 0 || sinks < 0) return fail(XV_ERR_ARG, "attn_q8: window and sinks must not be negative");
    const long long w = static_cast<long long>(Hq) * hd;
    if (q_stride < w || out_stride < w || (gate && gate_stride < w)) return fail(XV_ERR_ARG, "attn_q8: a row stride is below its row");
    if (hd != 64 && hd != 128 && hd != 256) return fail(XV_ERR_UNSUPPORTED, "attn_q8: hd must be 64, 128 or 256 (got %d)", hd);
    if (R > XV_KMAX || B > 65535 || Hkv > 65535 || !sizes_ok(B, R, Hq, hd, max_ctx, window, sinks))
        return fail(XV_ERR_UNSUPPORTED, "attn_q8: R above %d, B or Hkv above 65535, or B*R*Hq above 2^30", XV_KMAX);
    if (!aligned16(q) || !aligned16(out) || !aligned16(gate) || q_stride % 8 || out_stride % 8 || (gate && gate_stride % 8))
        return fail(XV_ERR_UNSUPPORTED, "attn_q8: rows must be 16-byte aligned");
    const size_t need = xv_attn_q8_workspace_size(B, R, Hq, hd, max_ctx, window, sinks);
    if (!ws || ws_bytes < need) return fail(XV_ERR_WORKSPACE, "attn_q8: workspace of %zu bytes needed", need);
    if (!aligned16(ws)) return fail(XV_ERR_UNSUPPORTED, "attn_q8: workspace must be 16-byte aligned");
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "attn_q8: device error word unavailable");
    CUtensorMap tmK, tmV;
    const uint64_t dims[3] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(kv.page), static_cast<uint64_t>(kv.n_pages) * Hkv};
    const uint64_t strides[2] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(kv.page) * hd};
    const uint32_t box[3] = {static_cast<uint32_t>(hd < 128 ? hd : 128), static_cast<uint32_t>(T), 1};
    const CUtensorMapSwizzle sw = hd < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (xv_status st = encode_tiled(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, cache->k, dims, strides, box, sw)) return st;
    if (xv_status st = encode_tiled(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, cache->v, dims, strides, box, sw)) return st;
    int nsink;
    const int nslot = slots(R, max_ctx, window, sinks, &nsink);
    const int win = window < max_ctx ? window : 0;   // a window that holds every row is none
    const int shift = nslot < q8_split_of(max_ctx - 1) + 1 ? win : 0;
    const size_t rows = static_cast<size_t>(B) * R * Hq * nslot;
    float* opart = static_cast<float*>(ws);
    float2* ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + round256(rows * hd * sizeof(float)));
    const Q8Args a{q, q_stride, kv, cache->k_scale, cache->v_scale, ctx_len, n_rows, R, Hq / Hkv, Hq, Hkv, B, nslot, nsink, max_ctx,
                   win, win ? sinks : 0, shift, scale * 1.4426950408889634f, opart, ml, err};
    const CombineArgs c{ctx_len, n_rows, R, Hq, nslot, nsink, max_ctx, win, win ? sinks : 0, shift, opart, ml, gate, gate_stride, out,
                        out_stride};
    return hd == 256 ? launch<256>(tmK, tmV, a, c, s) : hd == 128 ? launch<128>(tmK, tmV, a, c, s) : launch<64>(tmK, tmV, a, c, s);
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

int xv_attn_q8_split_begin(int s) { return s < 0 ? -1 : q8_split_begin(s); }

size_t xv_attn_q8_workspace_size(int B, int R, int Hq, int hd, int max_ctx, int window, int sinks) {
    if (!sizes_ok(B, R, Hq, hd, max_ctx, window, sinks)) return 0;
    int nsink;
    const size_t rows = static_cast<size_t>(B) * R * Hq * slots(R, max_ctx, window, sinks, &nsink);
    return round256(rows * hd * sizeof(float)) + round256(rows * sizeof(float2));
}

xv_status xv_attn_decode_rows_q8(const uint16_t* q, long long q_stride, const xv_kv_q8* cache, const int32_t* ctx_len,
                                 const int32_t* n_rows, int R, int B, int Hq, int Hkv, int hd, int Lmax, int max_ctx,
                                 int window, int sinks, float scale, const uint16_t* gate, long long gate_stride,
                                 uint16_t* out, long long out_stride, void* ws, size_t ws_bytes, xv_stream s) {
    if (xv_status st = kv_q8_check(cache, "attn_q8")) return st;
    if (xv_status st = kv_contiguous_check(B, Hkv, hd, Lmax, "attn_q8")) return st;
    return attn_q8(q, q_stride, cache, kv_contiguous(B, Lmax), Lmax, ctx_len, n_rows, R, B, Hq, Hkv, hd, max_ctx, window, sinks,
                   scale, gate, gate_stride, out, out_stride, ws, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

xv_status xv_attn_decode_rows_q8_paged(const uint16_t* q, long long q_stride, const xv_kv_q8* cache, const xv_kv_pages* pages,
                                       const int32_t* ctx_len, const int32_t* n_rows, int R, int B, int Hq, int Hkv, int hd,
                                       int max_ctx, int window, int sinks, float scale, const uint16_t* gate,
                                       long long gate_stride, uint16_t* out, long long out_stride, void* ws, size_t ws_bytes,
                                       xv_stream s) {
    if (xv_status st = kv_q8_check(cache, "attn_q8")) return st;
    if (B < 1 || Hkv < 1 || hd < 1) return fail(XV_ERR_ARG, "attn_q8: need B, Hkv and hd >= 1");
    KvPages kv;
    int Lmax;
    if (xv_status st = kv_pages_check(pages, Hkv, hd, &kv, &Lmax)) return st;
    return attn_q8(q, q_stride, cache, kv, Lmax, ctx_len, n_rows, R, B, Hq, Hkv, hd, max_ctx, window, sinks, scale, gate,
                   gate_stride, out, out_stride, ws, ws_bytes, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

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
// 128; a row goes through its tiles in order, a tile without a position it sees leaves its m, l and O
// as they were, and its splits are joined in a fixed order.  A row's bits depend on its own length,
// q and what it sees, not on the rows and sequences beside it.
//
// The products run on tcgen05 in fp8, the cache's codes straight from their TMA stages as the
// 128-row operand A, the few query rows as N:
//   S^T = K Q^T    [128 positions x rows].  A bf16 q is the sum of two e4m3 values (the nearest, and
//                  the nearest to what is left), side by side in N; their two results are added.  A row
//                  is scaled by a power of two first, its largest value into [128, 256).
//   O^T += V^T P^T [dims x rows].  P is rounded to fp16 and goes in as the exact sum of four e5m2
//                  values: e5m2 is fp16's upper byte, so cutting the byte off three times leaves
//                  nothing (11 bits of significand, 3 by 3).  What is left after two is scaled by
//                  2^6, against e5m2's smallest value, and has an accumulator of its own.  P_SHIFT
//                  puts p at up to 2^15: P keeps weights to 2^-19 of the reference at full precision
//                  and to 2^-29 at all (a long context can hold half its weight in such), and the
//                  reference may stay up to RESCALE_SLACK below the row's largest t_j.
// With rows in M instead (a first form: 64 rows of 128 used, P in fp16, V widened to fp16 by warps of
// their own) a thread had a row and went through a tile's positions one by one: 2300 to 3500 cycles a
// tile of 64, where the codes of 128 take 2800 to arrive (hd 256).  Here a thread has a position, its
// scales are two registers, a batch's rows of one token cost what they are, and V is never widened.
//
// Kernel 1 (attn_q8_kernel): work items (slot, row tile, kv head, sequence); a slot is a split, or
// with a window one of the splits that the window and the sinks can touch.  One CTA per item where
// all fit at once, else persistent CTAs that walk contiguous ranges of equal cost.  Kernel 2
// (attn_q8_combine_kernel) joins each row's splits, where there are several.
#include <algorithm>
#include <climits>
#include <cmath>

#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

constexpr int T = 128;                 // positions per tile, in two halves of 64 (a page is a multiple of 64)
constexpr float NEG_INF = -INFINITY;
constexpr float P_SHIFT = 7.f, RESCALE_SLACK = 8.f;
constexpr float DEAD = -3e38f;         // the reference of a row that has seen nothing: t - DEAD passes any slack
constexpr float LOW_SCALE = 64.f;      // P's last two terms

// Split boundaries: every 256 positions below Q8_NEAR, 512 below Q8_FAR, 1024 beyond.  A short context
// wants its splits spread over the machine (one verify at 2183: 512 instead of 256 costs 1.4 us of 14.6),
// a batch wants few items (32 sequences at 4000 to 8000: 256 up to 4096 costs 5 us of 65), a long context
// few partial results (131072: 512 instead of 1024 costs 3 us of 69).
constexpr int Q8_NEAR = 2048, Q8_FAR = 32768, Q8_NS = Q8_NEAR / 256, Q8_FS = Q8_NS + (Q8_FAR - Q8_NEAR) / 512;
static_assert(256 % T == 0 && 1024 <= 8 * T, "a lane per half tile of an item");
__host__ __device__ inline int q8_split_begin(int s) {
    return s < Q8_NS ? s * 256 : s < Q8_FS ? Q8_NEAR + (s - Q8_NS) * 512 : Q8_FAR + (s - Q8_FS) * 1024;
}
// The split that position p lies in.
__host__ __device__ inline int q8_split_of(int p) {
    return p < Q8_NEAR ? p / 256 : p < Q8_FAR ? Q8_NS + (p - Q8_NEAR) / 512 : Q8_FS + (p - Q8_FAR) / 1024;
}

// NR: rows of a row tile, padded (a multiple of 8, as 2 NR is an N of the MMAs).
template <int HD, int NR>
struct Shape {
    static constexpr int KROW = HD < 128 ? HD : 128;          // bytes of a code row in a swizzled block
    static constexpr int KB = HD / KROW;                      // code blocks [128 positions][KROW] per tile
    static constexpr int KBLK = T * KROW;
    static constexpr int CODE = T * HD;                       // one K or V tile of codes
    static constexpr int MB = HD > 128 ? 2 : 1;               // 128-dim blocks of O^T (hd 64: lanes 64.. unused)
    static constexpr int QBLK = 2 * NR * KROW;                // Q block: nearest terms, then what is left
    static constexpr int Q = KB * QBLK;
    static constexpr int PT = T * 2 * NR;                     // terms 1 and 3, or 2 and 4, of a tile's P
    static constexpr int PB = NR <= 24 ? 2 : 1;               // P buffers
    // two CTAs per SM where their registers and rings allow it
    static constexpr int PER_SM = HD <= 128 && NR <= 16 ? 2 : 1;
    // softmax warpgroups of RW rows each: one thread's 48 rows took 3000 cycles a tile, and three times the code
    static constexpr int RW = NR % 16 ? 8 : 16, WG = NR / RW;
    static constexpr int THREADS = 128 * (WG + 2);
    static constexpr int RAW = PER_SM == 1 || NR == 8 ? 8 : 6;           // tiles of scales
    static constexpr int ITEMS = 8;                           // items on their way
    static constexpr int STATIC = 3 * RAW * T * 4 + 15 * NR * 4 + ITEMS * 208 + 64;
    static constexpr int ROOM = (PER_SM == 2 ? 233472 / 2 - 1024 : 232448) - STATIC - 1024 - 512 - Q - PB * 2 * PT;
    static constexpr int STAGES = ROOM / CODE;
    static constexpr int SV = STAGES < 10 ? (STAGES + 1) / 2 : 5, SK = STAGES < 10 ? STAGES - SV : 5;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + Q;
    static constexpr int V_OFF = K_OFF + SK * CODE;
    static constexpr int P_OFF = V_OFF + SV * CODE;
    static constexpr int BAR_OFF = P_OFF + PB * 2 * PT;
    static constexpr int N_BARS = 2 * (SK + SV + RAW + ITEMS) + 4 + PB + 4;
    static constexpr int SMEM = 1024 + BAR_OFF + 8 * N_BARS;
    static constexpr uint32_t O_COL = 4 * NR;                 // S twice, then O: MB blocks, each per warpgroup [terms 1, 2 | terms 3, 4]
    static constexpr int COLS = 4 * NR + MB * 2 * NR;
    static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(NR % 8 == 0 && NR <= 64 && COLS <= 512 && PER_SM * TMEM_COLS <= 512, "");
    static_assert(SK >= 2 && SV >= 2 && 8 * N_BARS <= 512 && QBLK % 1024 == 0, "");
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
    int tile_rows, nrt;  // rows of a row tile, row tiles
    Divisor by_g, by_nrt, by_hkv, by_nslot, by_page;
    int nslot, nsink;    // slots per row, of which the first nsink are the sinks' splits
    int max_len, window, sinks;
    int shift;           // the window, where the slots past the sinks' begin at it; 0: slots are splits
    int joined;          // nslot = 1, and each CTA makes its rows' output of their only split
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

// What a row tile of a sequence sees: positions below `end` for its last row; none of its rows those in
// [sinks, lo).
struct Sight {
    int L0, rows, row_base, end, lo, sinks;   // rows <= 0: nothing to do
    int from, upto;                           // every row sees [from, upto)
    __device__ __forceinline__ void of(const Q8Args& A, int b, int rt) {
        const int nr = q8_rows(A.n_rows, b, A.R);
        L0 = __ldg(A.ctx_len + b);
        row_base = rt * A.tile_rows;
        rows = min(nr * A.G - row_base, A.tile_rows);
        if (L0 < 1 || L0 > A.max_len - nr + 1) rows = 0;
        end = lo = sinks = from = upto = 0;
        if (rows <= 0) return;
        // what other rows see beside a row changes nothing of it
        end = L0 + A.by_g.div(row_base + rows - 1);
        upto = L0 + A.by_g.div(row_base);
        if (A.window) from = max(0, end - A.window);
        if (A.window && upto > A.window) lo = upto - A.window, sinks = A.sinks;
    }
    // whether a row sees any of the 64 positions at p
    __device__ __forceinline__ bool half(int p) const { return p < end && (p + 64 > lo || p < sinks); }
    // tiles of sinks before those of the windows
    __device__ __forceinline__ int heads() const { return min(lo / T, (min(sinks, lo) + T - 1) / T); }
    // cost of the splits before split s: one a tile, one a split
    __device__ __forceinline__ int cost(int s) const {
        const int last = q8_split_of(end - 1) + 1, h = heads(), n = s >= last ? (end + T - 1) / T : q8_split_begin(s) / T;
        const int hs = h ? q8_split_of(h * T - 1) + 1 : 0, m = min(s, last);
        return min(n, h) + max(0, n - max(lo / T, h)) + min(m, hs) + max(0, m - max(q8_split_of(lo), hs));
    }
};

constexpr int Q_COST = 1;   // in tiles

// Split of slot s, where the slots past the sinks' begin at split `first`.
__device__ __forceinline__ int q8_slot_split(int s, int nsink, int first) { return s < nsink ? s : first + s - nsink; }

// The work items of a CTA in order, those that see nothing left out.
struct Item {
    int it, slot, rt, g, b, first;
    Sight v;
    int p_begin, ntiles, head, skip;   // live tiles: the split's first `head`, then from tile head + skip on
    __device__ __forceinline__ int pos(int i) const { return p_begin + (i < head ? i : i + skip) * T; }
    __device__ __forceinline__ void sight(const Q8Args& A) {
        v.of(A, b, rt);
        first = q8_first(v.L0, A.shift, A.nsink);
    }
    __device__ __forceinline__ void place(const Q8Args& A) {
        const int split = q8_slot_split(slot, A.nsink, first);
        p_begin = q8_split_begin(split);
        const int nt = (max(0, min(q8_split_begin(split + 1), v.end) - p_begin) + T - 1) / T;
        const int low = min(nt, max(0, v.lo - p_begin) / T);   // first tile that a window reaches
        head = min(low, (max(0, v.sinks - p_begin) + T - 1) / T);
        skip = low - head;
        ntiles = v.rows > 0 ? nt - skip : 0;
    }
    // the first live item of [i, it1); false if there is none
    __device__ __forceinline__ bool open(const Q8Args& A, int i, int it1) {
        it = i;
        if (it >= it1) return false;
        const int tile = A.by_nslot.div(i), head = A.by_nrt.div(tile);
        slot = i - tile * A.nslot;
        rt = tile - head * A.nrt;
        b = A.by_hkv.div(head);
        g = head - b * A.Hkv;
        sight(A);
        place(A);
        return ntiles > 0 || next(A, it1);
    }
    __device__ __forceinline__ bool next(const Q8Args& A, int it1) {
        for (;;) {
            ++it;
            if (++slot == A.nslot || v.rows <= 0 || p_begin >= v.end) {   // splits past the end: none is live
                it += A.nslot - slot;
                slot = 0;
                if (++rt == A.nrt) {
                    rt = 0;
                    if (++g == A.Hkv) g = 0, ++b;
                }
                if (it >= it1) return false;
                sight(A);
            }
            if (it >= it1) return false;
            place(A);
            if (ntiles > 0) return true;
        }
    }
    __device__ __forceinline__ bool same_q(const Item& o) const { return b == o.b && g == o.g && rt == o.rt; }
};

// The items [it[0], it[1]) of persistent CTA c of n: equal shares of the cost (measured: 1.4 to 1.6 us a tile, 1 to
// 1.2 an item, some more where the Q changes).  One warp.  (What it takes
// the CTA waits for: with divisions in 64 bits and a look at the same sequence three times 3.5 us.)
__device__ __forceinline__ void q8_range(const Q8Args& A, int c, int n, int* it) {
    const int lane = threadIdx.x & 31;
    long long total = 0, before = 0, at0 = 0, at1 = 0;
    it[0] = it[1] = A.nslot * A.nrt * A.Hkv * A.B;   // where no cost is left
#pragma unroll 1
    for (int pass = A.B > 32 ? 0 : 1; pass < 2; ++pass) {   // the total, which 32 sequences show at once; the shares
#pragma unroll 1
        for (int b0 = 0; b0 < A.B; b0 += 32) {
            Sight v;
            v.rows = 0;
            int one = 0, tiles = 0;   // cost of a row tile of a head, live row tiles
            if (b0 + lane < A.B) v.of(A, b0 + lane, 0);
            if (v.rows > 0) {
                one = Q_COST + v.cost(1 << 24);
                tiles = A.nrt == 1 ? 1 : (q8_rows(A.n_rows, b0 + lane, A.R) * A.G + A.tile_rows - 1) / A.tile_rows;
            }
            long long x = static_cast<long long>(one) * (tiles * A.Hkv);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += o;
            }
            const long long all = __shfl_sync(0xffffffffu, x, 31);
            if (pass == 0 || A.B <= 32) total += all;
            if (pass == 0) continue;
            if (b0 == 0) {   // shares of total / n, the first total % n of them one more
                const bool small = total < (1ll << 31);
                const long long share = small ? static_cast<unsigned>(total) / static_cast<unsigned>(n) : total / n;
                const int more = static_cast<int>(total - share * n);
                at0 = share * c + min(c, more);
                at1 = share * (c + 1) + min(c + 1, more);
            }
            // an item belongs to the CTA in whose share its cost begins
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                long long off = (e ? at1 : at0) - before;
                if (off < 0 || off >= all) continue;
                const int own = __ffs(__ballot_sync(0xffffffffu, x > off)) - 1;
                off -= own ? __shfl_sync(0xffffffffu, x, own - 1) : 0;
                const int o1 = __shfl_sync(0xffffffffu, one, own), tl = __shfl_sync(0xffffffffu, tiles, own);
                const int pair = static_cast<int>(off) / o1, in = static_cast<int>(off) - pair * o1;   // (head, row tile), cost in it
                Sight w;
                w.L0 = __shfl_sync(0xffffffffu, v.L0, own);
                w.end = __shfl_sync(0xffffffffu, v.end, own);
                w.lo = __shfl_sync(0xffffffffu, v.lo, own);
                w.sinks = __shfl_sync(0xffffffffu, v.sinks, own);
                const int first = q8_first(w.L0, A.shift, A.nsink);
                int slot = 0;   // the first whose cost begins at `in` or later
#pragma unroll 1
                for (int s = 0; s < A.nslot; s += 32) {
                    // (the first item of a row tile begins with its Q)
                    const int ahead = w.cost(q8_slot_split(s + lane, A.nsink, first)), begin = ahead ? ahead + Q_COST : 0;
                    const unsigned less = __ballot_sync(0xffffffffu, s + lane < A.nslot && begin < in);
                    slot += __popc(less);
                    if (less != 0xffffffffu) break;
                }
                const int h = tl == 1 ? pair : pair / tl;
                it[e] = (((b0 + own) * A.Hkv + h) * A.nrt + pair - h * tl) * A.nslot + slot;
            }
            before += all;
        }
    }
}

// An item as the CTA's warps get it.
struct Work {
    int ntiles, p_begin, head, skip, slot;   // ntiles = 0: no more items
    int fresh, pre;                          // its Q is another than the last item's; the next item's is the same
    int b, g;
    Sight v;
    int z[16], row[16];   // half h of tile i at 2 i + h: head of the pools, row in it; z < 0 where no row sees it
    __device__ __forceinline__ int pos(int i) const { return p_begin + (i < head ? i : i + skip) * T; }
};
static_assert(sizeof(Work) <= 208, "");

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
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Live Q rows of an item -> rows of N, as two e4m3 terms of q 2^e (the row's largest magnitude in
// [128, 256)) in swizzled blocks, and fac[row] = sl2 2^-e; the rows behind them become 0.
// NT threads (whole warps) from t0.
template <int HD, int NR, int NT>
__device__ __forceinline__ void load_q(uint8_t* sq, float* fac, const Q8Args& A, const Work& I, int t0) {
    using S = Shape<HD, NR>;
    constexpr int LPH = HD / 8, RPP = NT / LPH, UN = (NR + RPP - 1) / RPP < 4 ? (NR + RPP - 1) / RPP : 4;
    const int n = I.v.rows, c = t0 % LPH;
#pragma unroll 1
    for (int r0 = 0; r0 < NR; r0 += RPP * UN) {
        uint4 v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int row = r0 + k * RPP + t0 / LPH;
            v[k] = make_uint4(0, 0, 0, 0);
            if (row < n) {
                const int r = A.by_g.div(I.v.row_base + row), h = I.g * A.G + I.v.row_base + row - r * A.G;
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
            if (row >= NR) continue;
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
            uint8_t* dst = sq + blk * S::QBLK + row * S::KROW + sw * 16 + (byte & 8);
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(dst + NR * S::KROW) = make_uint2(lo[0], lo[1]);
            if (c == 0) fac[row] = __fmul_rn(A.sl2, __uint_as_float(static_cast<uint32_t>(127 - e) << 23));
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
// MN-major operand of bytes in swizzled rows of ROW dims, 8 positions of them (8 ROW bytes) after another.
// ROW = 128 fills M; with ROW = 64 the upper half of M repeats the lower (a stride of 0).
template <int ROW>
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t saddr) {
    uint64_t d = sw128_mnmajor_desc(saddr, 0, 8 * ROW);
    if (ROW == 64) d ^= static_cast<uint64_t>(2 ^ 4) << 61;
    return d;
}
// MN-major operand of bytes without swizzle: cores of 8 positions x 16 bytes of N, positions 128 bytes
// a core, the next 16 of N `n_stride` bytes further.
__device__ __forceinline__ uint64_t mnmajor_plain_desc(uint32_t saddr, uint32_t n_stride) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128u >> 4) << 16;
    d |= static_cast<uint64_t>(n_stride >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator, A e4m3.
constexpr uint32_t idesc_f8(int M, int N, bool b_e5m2, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (b_e5m2 ? (1u << 10) : 0u) | (a_mn_major ? (1u << 15) : 0u) | (b_mn_major ? (1u << 16) : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D (+)= A B^T, operands in shared memory.
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 lanes x 32 bits, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
                 "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Barriers of a softmax warpgroup; with a flag, whether any thread's is set.
__device__ __forceinline__ void wg_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool wg_any(int id, bool f) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, %2, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(r)
                 : "r"(f ? 1u : 0u), "r"(id)
                 : "memory");
    return r != 0;
}
// L2 policy of lines read once, or of any.
__device__ __forceinline__ uint64_t l2_policy(bool once) {
    uint64_t p;
    if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
// Sums of the warp's lanes, N values each: halves of the values go to halves of the lanes, so that it
// takes about N shuffles.  The lane's sums end in v[0..] and are those of `first` on; the tree over the
// lanes is the same for every N.
template <int N, int OFF>
__device__ __forceinline__ int warp_sums(float* v, int lane, int* first) {
    if constexpr (OFF == 0) return N;
    else if constexpr (N % 2 == 0) {
        const bool up = lane & OFF;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float send = up ? v[i] : v[i + N / 2];
            v[i] = __fadd_rn(up ? v[i + N / 2] : v[i], __shfl_xor_sync(0xffffffffu, send, OFF));
        }
        if (up) *first += N / 2;
        return warp_sums<N / 2, OFF / 2>(v, lane, first);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xffffffffu, v[i], OFF));
        return warp_sums<N, OFF / 2>(v, lane, first);
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

constexpr int CB_SUMS = 16;   // a row's splits are joined in so many sums

// The slots of a row that hold what it sees: those of the sinks it sees beside its window, then its window's.
struct RowSlots {
    int first, nsink, n0, s0, n;
    __device__ __forceinline__ RowSlots(const CombineArgs& C, int L0, int r) {
        const int len = L0 + r, from = C.window ? max(0, len - C.window) : 0, upto = min(C.sinks, from);
        first = q8_first(L0, C.shift, C.nsink);
        nsink = C.nsink;
        n0 = upto ? q8_split_of(upto - 1) + 1 : 0;   // splits with a sink
        s0 = max(n0, q8_split_of(from));
        n = n0 + q8_split_of(len - 1) + 1 - s0;
    }
    __device__ __forceinline__ int operator[](int i) const {
        const int s = i < n0 ? i : s0 + i - n0;
        return s < nsink ? s : s - first + nsink;
    }
};
// Whether row r of sequence b is there (L0: the first row's length).
__device__ __forceinline__ bool q8_row(const CombineArgs& C, int b, int r, int* L0) {
    const int nr = q8_rows(C.n_rows, b, C.R);
    *L0 = C.ctx_len[b];
    return r < nr && *L0 >= 1 && *L0 <= C.max_len - nr + 1;
}
// Four dims of a row's output from their sum and the weights': br = b R + r.
template <int HD>
__device__ __forceinline__ void q8_output(const CombineArgs& C, int br, int hq, int dim, float4 y, float sum) {
    // one reciprocal, as its rounding and the product's are far below the output's
    const float inv = __frcp_rn(sum);
    float out[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = __fadd_rn(__fmul_rn(out[e], inv), 0.f);
    if (C.gate) {
        const uint2 g = *reinterpret_cast<const uint2*>(C.gate + br * C.gate_stride + hq * HD + dim);
        const float gv[4] = {__uint_as_float(g.x << 16), __uint_as_float(g.x & 0xffff0000u), __uint_as_float(g.y << 16),
                             __uint_as_float(g.y & 0xffff0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = __fmul_rn(out[e], __frcp_rn(__fadd_rn(1.f, expf(-gv[e]))));
    }
    *reinterpret_cast<uint2*>(C.out + br * C.out_stride + hq * HD + dim) = make_uint2(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]));
}
// Four dims of a row whose only slot is 0: the bits that attn_q8_combine_kernel gives for one slot.
template <int HD>
__device__ __forceinline__ void q8_join_one(const CombineArgs& C, int b, int r, int hq, int dim) {
    int L0;
    if (!q8_row(C, b, r, &L0)) return;
    const int br = b * C.R + r;
    const long long row = static_cast<long long>(br) * C.Hq + hq;
    const float2 v = __ldcg(C.ml + row);
    const float4 o = __ldcg(reinterpret_cast<const float4*>(C.opart + row * HD + dim));
    const float w = ex2_approx(__fsub_rn(v.x, v.x));   // 1, or NaN
    const float4 y = make_float4(__fmaf_rn(w, o.x, 0.f), __fmaf_rn(w, o.y, 0.f), __fmaf_rn(w, o.z, 0.f), __fmaf_rn(w, o.w, 0.f));
    q8_output<HD>(C, br, hq, dim, y, __fmaf_rn(w, v.y, 0.f));
}

// Warps of a CTA and what they do per tile t (counted over the CTA's items):
//   0..4 WG - 1   softmax, warpgroup w for rows RW w.., a thread per position: S out of tensor memory,
//          t_j, mask; the references stand unless some row's t_j passes its by RESCALE_SLACK (or the
//          tile is an item's first): then the tile's maxima are found, and references, l and O moved;
//          P to shared memory, l per thread
//   then 4 an item's O, m and l to the workspace, while the next item's first tiles run
//   1      TMA of the K and V codes into their rings
//   1      MMAs: S(t + 1) = K Q^T, then O += V^T P(t); the S that overwrites S(t - 1) is issued after
//          the P V of that tile, whose P was made of it
//   1      the positions' scales: ks, log2(vs) and 1 / vs into a ring
//   1      the items, with their pages looked up, for all the others.  (With every warp stepping through
//          the items itself the code outgrew the instruction caches: 113 KB, and 20 cycles an instruction.)
template <int HD, int NR>
__global__ void __launch_bounds__(Shape<HD, NR>::THREADS, Shape<HD, NR>::PER_SM)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Q8Args A,
                   const __grid_constant__ CombineArgs C) {
    using S = Shape<HD, NR>;
    constexpr int SK = S::SK, SV = S::SV, RAW = S::RAW, PB = S::PB, RW = S::RW, WG = S::WG;
    constexpr int IT = S::ITEMS;
    constexpr int W_OUT = 4 * WG, W_TMA = W_OUT + 4, W_MMA = W_TMA + 1, W_SC = W_TMA + 2, W_IT = W_TMA + 3;   // warps
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) float sc_k[RAW][T], sc_v[RAW][T], sc_i[RAW][T];
    __shared__ __align__(16) float q_fac[2][NR], mo_sm[NR], al_sm[NR], wmax[4][NR], l_sm[4][NR], m_sm[NR];
    __shared__ long long at_sm[NR];
    __shared__ Work items[IT];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int s_abort;
    const uint32_t rawb = smem_u32(smem_raw);
    const uint32_t base = (rawb + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - rawb);
    auto sK = [&](int st) { return base + S::K_OFF + st * S::CODE; };
    auto sV = [&](int st) { return base + S::V_OFF + st * S::CODE; };
    const uint32_t bar0 = base + S::BAR_OFF;
    auto fullK = [&](int st) { return bar0 + 8u * st; };
    auto emptyK = [&](int st) { return bar0 + 8u * (SK + st); };
    const uint32_t bar1 = bar0 + 8u * 2 * SK;
    auto fullV = [&](int st) { return bar1 + 8u * st; };
    auto emptyV = [&](int st) { return bar1 + 8u * (SV + st); };
    const uint32_t bar2 = bar1 + 8u * 2 * SV;
    auto fullS = [&](int st) { return bar2 + 8u * st; };
    auto emptyS = [&](int st) { return bar2 + 8u * (RAW + st); };
    const uint32_t bx = bar2 + 8u * 2 * RAW;
    auto sbar = [&](int j) { return bx + 8u * j; };            // S of a tile is complete
    auto pready = [&](int j) { return bx + 8u * (2 + j); };    // its P is in shared memory, its S has been read
    auto pfree = [&](int j) { return bx + 8u * (4 + j); };     // its P V is complete
    const uint32_t by = bx + 8u * (4 + PB);
    const uint32_t done = by, ofree = by + 8, qready = by + 16, mlready = by + 24, bi = by + 32;
    auto fullI = [&](int n) { return bi + 8u * (n % IT); };
    auto emptyI = [&](int n) { return bi + 8u * (IT + n % IT); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 32 * W_TMA) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        for (int st = 0; st < SK; ++st) mbar_init(fullK(st), 1), mbar_init(emptyK(st), 1);
        for (int st = 0; st < SV; ++st) mbar_init(fullV(st), 1), mbar_init(emptyV(st), 1);
        for (int st = 0; st < RAW; ++st) mbar_init(fullS(st), 1), mbar_init(emptyS(st), 4 * WG);
        for (int st = 0; st < IT; ++st) mbar_init(fullI(st), 1), mbar_init(emptyI(st), 4 * WG + 7);
        for (int j = 0; j < 2; ++j) mbar_init(sbar(j), 1), mbar_init(pready(j), 128 * WG);
        for (int j = 0; j < PB; ++j) mbar_init(pfree(j), 1);
        mbar_init(done, 1);
        mbar_init(ofree, 128);
        mbar_init(qready, 128 * WG);
        mbar_init(mlready, 128 * WG);
        fence_mbar_init();
        s_abort = 0;
    }
    __syncthreads();
    griddep_wait();
    // The tensor memory's columns, for the warps that use them.  No limit bounds the wait for them: the MMA warp takes
    // them once the kernels before are done, which may have none yet themselves, and lets the kernels behind go only
    // then (the GEMM takes its own before it waits for this one: at hd 64 both fit an SM's memory, but 512 columns and
    // 64 not its tensor memory).
    auto columns = [&]() -> uint32_t {
        asm volatile("barrier.cta.sync 8, %0;" ::"n"(128 * (WG + 1) + 32) : "memory");
        tc_fence_after();
        return tmem_slot;
    };

    auto W = [&](uint32_t bar, uint32_t par) -> bool { return mbar_try_wait(bar, par) || wait_slow(bar, par, &s_abort, A.err); };
    // the same verdict for every lane of a warp
    auto WW = [&](uint32_t bar, uint32_t par) -> bool { return __all_sync(0xffffffffu, W(bar, par)); };
    // the n-th item is there, and is not the end
    auto item = [&](int n) -> bool { return WW(fullI(n), (n / IT) & 1u) && items[n % IT].ntiles > 0; };
    // the warp has no more use for it
    auto item_done = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(emptyI(n));
    };

    if (warp == W_IT) {
        // ---- items
        int it[2] = {static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.x) + 1};   // one item per CTA
        if (static_cast<int>(gridDim.x) < A.nslot * A.nrt * A.Hkv * A.B) q8_range(A, blockIdx.x, gridDim.x, it);
        Item I;
        bool more = I.open(A, it[0], it[1]), fresh = true;
        for (int n = 0;; ++n) {
            if (n >= IT && !WW(emptyI(n), ((n / IT) & 1u) ^ 1u)) break;
            Work& w = items[n % IT];
            if (!more) {
                if (lane == 0) {
                    w.ntiles = 0;
                    mbar_arrive(fullI(n));
                }
                break;
            }
            const int p = I.pos(lane >> 1) + 64 * (lane & 1);
            int z = -1, row = p;
            if (lane < 2 * I.ntiles && I.v.half(p)) {
                int page = I.b;
                if (A.kv.table) {
                    const int j = A.by_page.div(p);
                    row = p - j * A.kv.page;
                    page = A.kv.table[static_cast<long long>(I.b) * A.kv.max_pages + j];
                    if (page < 0 || page >= A.kv.n_pages) {
                        atomicOr(A.err, ERR_BAD_PAGE);
                        page = 0;
                    }
                }
                z = page * A.Hkv + I.g;
            }
            if (lane < 16) w.z[lane] = z, w.row[lane] = row;
            if (lane == 0) {
                w.ntiles = I.ntiles, w.p_begin = I.p_begin, w.head = I.head, w.skip = I.skip, w.slot = I.slot;
                w.b = I.b, w.g = I.g, w.v = I.v;
            }
            const Item was = I;
            more = I.next(A, it[1]);
            const bool pre = more && I.same_q(was);
            if (lane == 0) w.fresh = fresh, w.pre = pre;
            fresh = !pre;
            __syncwarp();
            if (lane == 0) mbar_arrive(fullI(n));
        }
        // lengths and counts outside their range see nothing, and are recorded
        for (int b = blockIdx.x + gridDim.x * lane; b < A.B; b += gridDim.x * 32) {
            const int raw = A.n_rows ? A.n_rows[b] : A.R, nr = min(max(raw, 0), A.R), L0 = A.ctx_len[b];
            if (raw != nr) atomicOr(A.err, ERR_BAD_COUNT);
            if (nr > 0 && (L0 < 1 || L0 > A.max_len - nr + 1)) atomicOr(A.err, ERR_BAD_LENGTH);
        }
    } else if (warp == W_TMA) {
        // ---- TMA: K before V of a tile, the order in which their stages come free
        // (codes that one row tile reads once are the first to leave L2, and the partial results stay)
        const uint64_t policy = l2_policy(A.nrt == 1);
        int t = 0;
        for (int n = 0; item(n); ++n) {
            const Work& w = items[n % IT];
            const int nt = w.ntiles;
            bool ok = true;
            for (int i = 0; ok && i < nt; ++i, ++t) {
#pragma unroll 1
                for (int side = 0; ok && side < 2; ++side) {
                    const int NS = side ? SV : SK, st = t % NS;
                    const uint32_t fb = side ? fullV(st) : fullK(st), dst0 = side ? sV(st) : sK(st);
                    if (t >= NS) ok = WW(side ? emptyV(st) : emptyK(st), ((t / NS) & 1u) ^ 1u);
                    if (ok && lane == 0) {
                        const CUtensorMap* map = side ? &tmV : &tmK;
                        const int z0 = w.z[2 * i], z1 = w.z[2 * i + 1];
                        mbar_arrive_expect_tx(fb, (z0 >= 0 ? S::CODE / 2 : 0) + (z1 >= 0 ? S::CODE / 2 : 0));
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            const int z = h ? z1 : z0, row = w.row[2 * i + h];
                            if (z < 0) continue;
#pragma unroll
                            for (int cb = 0; cb < S::KB; ++cb)
                                tma_load_3d_hint(dst0 + cb * S::KBLK + h * S::KBLK / 2, map, cb * S::KROW, row, z, fb, policy);
                        }
                    }
                    // a stage that will not be filled ends the loads; what has been issued is waited for
                }
                if (!ok) break;
            }
            item_done(n);
            if (!ok) break;
        }
        // every issued copy lands before the CTA may leave
        for (int j = t > SK ? t - SK : 0; j < t; ++j) mbar_wait(fullK(j % SK), (j / SK) & 1u, A.err);
        for (int j = t > SV ? t - SV : 0; j < t; ++j) mbar_wait(fullV(j % SV), (j / SV) & 1u, A.err);
    } else if (warp == W_SC) {
        // ---- scales: every lane copies those of its four positions RAW - 2 tiles ahead, and makes of them,
        // in their place, what the softmax needs
        int t = 0;   // tiles copied
        auto make = [&](int m) {
            const int st = m % RAW;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float vs = sc_v[st][lane + 32 * k];
                const float vc = fminf(fmaxf(vs, 0x1p-40f), 0x1p60f);              // a NaN becomes 2^-40
                sc_v[st][lane + 32 * k] = vs != vs ? vs : lg2_approx(vc);          // a NaN scale speaks through t_j alone
                sc_i[st][lane + 32 * k] = __frcp_rn(vc);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fullS(st));
        };
        bool ok = true, live = true;
        int m = 0, n = 0, i = 0, nt = 0;
        // (one loop for the copies ahead, for both, and for what is left to make)
        while (ok && (live || m < t)) {
            if (live && i == nt) {
                if (nt) item_done(n++);
                live = item(n);
                i = 0;
                nt = live ? items[n % IT].ntiles : 0;
            }
            if (live) {
                const Work& w = items[n % IT];
                const int st = t % RAW, left = w.v.end - w.pos(i);
                ok = t < RAW || WW(emptyS(st), ((t / RAW) & 1u) ^ 1u);
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int z = w.z[2 * i + h];
                    const long long at = static_cast<long long>(z) * A.kv.page + w.row[2 * i + h];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = lane + 32 * k;
                        const bool in = z >= 0 && 64 * h + j < left;
                        cp_async4(smem_u32(&sc_k[st][64 * h + j]), A.k_scale + (in ? at + j : 0), in);
                        cp_async4(smem_u32(&sc_v[st][64 * h + j]), A.v_scale + (in ? at + j : 0), in);
                    }
                }
                ++t;
                ++i;
            }
            cp_async_commit();   // a group per round, an empty one past the last tile
            if (t - m > RAW - 2 || !live) {
                cp_async_wait<RAW - 2>();
                if (!live) cp_async_wait_all();
                make(m++);
            }
        }
        cp_async_wait_all();
    } else if (warp == W_MMA) {
        // ---- MMAs
        tmem_alloc(smem_u32(&tmem_slot), S::TMEM_COLS);
        tmem_relinquish();
        griddep_launch();
        tc_fence_before();
        const uint32_t tS = columns(), tO = tS + S::O_COL;
        if (lane == 0) {
            constexpr uint32_t IDS = idesc_f8(128, 2 * NR, false, false, false), IDO = idesc_f8(128, 2 * NR, true, true, true);
            constexpr int KS = S::KROW / 32;   // MMAs of 32 codes per block row
            const uint32_t sQ = base + S::Q_OFF;
            auto qk = [&](int tt) -> bool {
                const int st = tt % SK;
                if (!W(fullK(st), (tt / SK) & 1u)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < HD / 32; ++ks)
                    mma_fp8(tS + (tt & 1) * 2 * NR, kmajor_desc<S::KROW>(sK(st) + (ks / KS) * S::KBLK + (ks % KS) * 32),
                            kmajor_desc<S::KROW>(sQ + (ks / KS) * S::QBLK + (ks % KS) * 32), IDS, ks > 0 ? 1u : 0u);
                tc_commit(sbar(tt & 1));
                tc_commit(emptyK(st));
                return true;
            };
            int t = 0, nq = 0;
            bool ok = true;
            for (int n = 0; ok && W(fullI(n), (n / IT) & 1u); ++n) {
                const int nt = items[n % IT].ntiles;
                const bool fresh = items[n % IT].fresh, pre = items[n % IT].pre;
                mbar_arrive(emptyI(n));
                if (!nt) break;
                // with the last item's Q, this one's first S went out before the last P V
                if (fresh && (!W(qready, nq++ & 1u) || !qk(t))) break;
                for (int i = 0; i < nt; ++i) {
                    const int tt = t + i, sv = tt % SV;
                    if ((i + 1 < nt || pre) && !qk(tt + 1)) { ok = false; break; }
                    if (i == 0 && n > 0 && !W(ofree, (n - 1) & 1u)) { ok = false; break; }
                    if (!W(fullV(sv), (tt / SV) & 1u) || !W(pready(tt & 1), (tt >> 1) & 1u)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sP = base + S::P_OFF + (tt % PB) * 2 * S::PT;
#pragma unroll
                    for (int mb = 0; mb < S::MB; ++mb)
#pragma unroll
                        for (int kk = 0; kk < T / 32; ++kk) {   // 32 positions
                            const uint64_t ad = mnmajor_desc<S::KROW>(sV(sv) + mb * S::KBLK + kk * 32 * S::KROW);
                            mma_fp8(tO + mb * 2 * NR, ad, mnmajor_plain_desc(sP + kk * 512, T * 16), IDO, (i > 0 || kk > 0) ? 1u : 0u);
                            mma_fp8(tO + mb * 2 * NR, ad, mnmajor_plain_desc(sP + S::PT + kk * 512, T * 16), IDO, 1u);
                        }
                    tc_commit(pfree(tt % PB));
                    tc_commit(emptyV(sv));
                }
                t += nt;
            }
            tc_commit(done);   // every MMA issued is complete before the CTA may leave
            mbar_wait(done, 0u, A.err);
        }
    } else if (warp >= W_OUT) {
        // ---- epilogue: thread = dim of O^T (tensor memory lane), modulo 128
        const int d = tid - 32 * W_OUT;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16, tO = columns() + S::O_COL;
        int t = 0;
        for (int n = 0; item(n); ++n) {
            t += items[n % IT].ntiles;
            const int rows = items[n % IT].v.rows, tl = t - 1;
            item_done(n);
            if (!WW(mlready, n & 1u) || !WW(pfree(tl % PB), (tl / PB) & 1u)) break;
            tc_fence_after();
            if (HD >= 128 || warp < W_OUT + 2) {
                constexpr int CH = RW;   // rows at a time: a warpgroup's
#pragma unroll 1
                for (int c = 0; c < S::MB * NR; c += CH) {
                    const int mb = c / NR, r0 = c % NR;
                    if (r0 >= rows) continue;
                    float a[CH], b[CH];
                    const uint32_t col = tO + lane_off + mb * 2 * NR + 2 * r0;
                    if constexpr (CH == 16) {
                        tmem_ld16(col, a);
                        tmem_ld16(col + RW, b);
                    } else {
                        tmem_ld8(col, a);
                        tmem_ld8(col + RW, b);
                    }
                    tmem_ld_wait();
                    float* out = A.opart + mb * 128 + d;
#pragma unroll
                    for (int e = 0; e < CH; ++e)
                        if (r0 + e < rows) out[at_sm[r0 + e] * HD] = __fmaf_rn(b[e], 1.f / LOW_SCALE, a[e]);
                }
            }
            if (d < rows)
                A.ml[at_sm[d]] = make_float2(m_sm[d], __fadd_rn(__fadd_rn(l_sm[0][d], l_sm[1][d]), __fadd_rn(l_sm[2][d], l_sm[3][d])));
            tc_fence_before();
            mbar_arrive(ofree);   // O, m and l may be overwritten by the next item
        }
    } else {
        // ---- softmax: thread = position of the tile (tensor memory lane), rows r_wg..  A wait that gives up
        // breaks no loop here, so that the four warps meet at the same barriers (later waits return at once)
        const int wg = warp >> 2, r_wg = wg * RW, pt = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t cS = columns() + lane_off + r_wg, cO = cS + S::O_COL + r_wg;
        int t = 0, nq = 0;
        long long at = 0;   // of row r_wg + pt in the workspace, slot 0
        for (int n = 0;; ++n) {
            if (wg_any(1 + wg, !item(n))) break;
            const Work& I = items[n % IT];
            if (I.fresh) {
                // every S of the old Q is complete (this warp has seen the last), and the MMA warp issues
                // none of this item until qready
                load_q<HD, NR, 128 * WG>(smem + S::Q_OFF, q_fac[(nq + 1) & 1], A, I, tid);
                fence_proxy_async_smem();
                mbar_arrive(qready);
                const int gr = I.v.row_base + r_wg + pt, r = A.by_g.div(gr);
                at = ((static_cast<long long>(I.b) * A.R + r) * A.Hq + I.g * A.G + gr - r * A.G) * A.nslot;
                WW(qready, nq & 1u);   // the other warps' factors too
                ++nq;
            }
            const int nt = I.ntiles;
            const float* fac = q_fac[nq & 1] + r_wg;
            float l[RW], m = NEG_INF;   // l of this thread's positions; m of row r_wg + pt
#pragma unroll
            for (int r = 0; r < RW; ++r) l[r] = 0.f;
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const int tt = t + i, st = tt % RAW, p0 = I.pos(i);
                const bool whole = p0 >= I.v.from && p0 + T <= I.v.upto;
                WW(fullS(st), (tt / RAW) & 1u);
                const float ks = sc_k[st][pt], lv = sc_v[st][pt], iv = sc_i[st][pt];
                __syncwarp();
                if (lane == 0) mbar_arrive(emptyS(st));
                WW(sbar(tt & 1), (tt >> 1) & 1u);
                tc_fence_after();
                float s[RW], lo[RW];   // t_j of the rows
                if constexpr (RW == 16) {
                    tmem_ld16(cS + (tt & 1) * 2 * NR, s);
                    tmem_ld16(cS + (tt & 1) * 2 * NR + NR, lo);
                } else {
                    tmem_ld8(cS + (tt & 1) * 2 * NR, s);
                    tmem_ld8(cS + (tt & 1) * 2 * NR + NR, lo);
                }
                tmem_ld_wait();
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 c = *reinterpret_cast<const float4*>(fac + r);
                    float* x = s + r;
                    add2(x[0], x[1], lo[r], lo[r + 1]);
                    add2(x[2], x[3], lo[r + 2], lo[r + 3]);
                    mul2(x[0], x[1], c.x, c.y);
                    mul2(x[2], x[3], c.z, c.w);
                    fma2(x[0], x[1], ks, ks, lv, lv);
                    fma2(x[2], x[3], ks, ks, lv, lv);
                }
                if (!whole) {
                    // row n / G of length L0 + n / G (n = row_base + r) sees p from r = r_lo on, and with a
                    // window to r_hi unless p is a sink
                    const int p = p0 + pt;
                    const long long n0 = I.v.row_base + r_wg;
                    const long long r_lo = p >= I.v.end ? RW : static_cast<long long>(p - I.v.L0 + 1) * A.G - n0;
                    const long long r_hi = !A.window || p < A.sinks ? RW : (static_cast<long long>(p) + A.window - I.v.L0 + 1) * A.G - n0;
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (r < r_lo || r >= r_hi) s[r] = NEG_INF;
                    // V codes that were not loaded or lie behind every row: zeros, as 0 times their NaN is NaN
                    const bool gap = p >= I.v.end || !I.v.half(p0 + (pt & 64));
                    if (wg == 0 && __any_sync(0xffffffffu, gap)) {
                        const int sv = tt % SV;
                        WW(fullV(sv), (tt / SV) & 1u);
                        if (gap) {
#pragma unroll 1
                            for (int c = 0; c < HD; c += 16)
                                *reinterpret_cast<uint4*>(smem + S::V_OFF + sv * S::CODE + c / S::KROW * S::KBLK + pt * S::KROW +
                                                          c % S::KROW) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                bool move = i == 0;
                if (!move) {
                    float over = NEG_INF;
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 mo = *reinterpret_cast<const float4*>(mo_sm + r_wg + r);
                        over = fmaxf(fmaxf(fmaxf(over, __fsub_rn(s[r], mo.x)), fmaxf(__fsub_rn(s[r + 1], mo.y), __fsub_rn(s[r + 2], mo.z))),
                                     __fsub_rn(s[r + 3], mo.w));
                    }
                    move = wg_any(1 + wg, over > P_SHIFT + RESCALE_SLACK);
                }
                if (move) {
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 x = make_float4(warp_max(s[r]), warp_max(s[r + 1]), warp_max(s[r + 2]), warp_max(s[r + 3]));
                        if (lane == 0) *reinterpret_cast<float4*>(&wmax[warp & 3][r_wg + r]) = x;
                    }
                    wg_sync(1 + wg);
                    bool scaled = false;
                    if (pt < RW) {
                        const int r = r_wg + pt;
                        const float mx = fmaxf(fmaxf(wmax[0][r], wmax[1][r]), fmaxf(wmax[2][r], wmax[3][r]));
                        const float old = m == NEG_INF ? DEAD : __fsub_rn(m, P_SHIFT);
                        float al = 1.f;
                        if (__fsub_rn(mx, old) > P_SHIFT + RESCALE_SLACK) {
                            if (m != NEG_INF) al = ex2_approx(__fsub_rn(m, mx));
                            m = mx;
                        }
                        mo_sm[r] = m == NEG_INF ? DEAD : __fsub_rn(m, P_SHIFT);
                        al_sm[r] = al;
                        scaled = al != 1.f;
                    }
                    if (wg_any(1 + wg, scaled)) {
                        // O once P V of the tile before has completed
                        WW(pfree((tt - 1) % PB), ((tt - 1) / PB) & 1u);
                        tc_fence_after();
#pragma unroll
                        for (int r = 0; r < RW; ++r) l[r] = __fmul_rn(l[r], al_sm[r_wg + r]);
#pragma unroll 1
                        for (int c = 0; c < S::MB * 2 * RW; c += 8) {
                            const uint32_t col = cO + c / (2 * RW) * 2 * NR + c % (2 * RW);
                            float o[8];
                            tmem_ld8(col, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __fmul_rn(o[e], al_sm[r_wg + c % RW + e]);
                            tmem_st8(col, o);
                        }
                        tmem_st_wait();
                    }
                }
                if (tt >= PB) WW(pfree(tt % PB), ((tt / PB) & 1u) ^ 1u);
                // a thread's bytes of N: per warpgroup [terms 1 | terms 3], and [terms 2 | terms 4]
                uint8_t* P = smem + S::P_OFF + (tt % PB) * 2 * S::PT + wg * (RW / 8) * T * 16 + pt * 16;
                uint32_t a[RW / 2], b[RW / 2];
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 mo = *reinterpret_cast<const float4*>(mo_sm + r_wg + r);
                    float* x = s + r;
                    add2(x[0], x[1], -mo.x, -mo.y);
                    add2(x[2], x[3], -mo.z, -mo.w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = ex2_approx(x[e]);
                    fma2_acc(l[r], l[r + 1], x[0], x[1], iv, iv);
                    fma2_acc(l[r + 2], l[r + 3], x[2], x[3], iv, iv);
                    uint32_t u = pack_f16x2(x[0], x[1]), v = pack_f16x2(x[2], x[3]);
                    constexpr uint32_t TOP = 0xff00ff00u, UP = 0x54005400u;   // LOW_SCALE, twice
                    a[r / 4] = __byte_perm(u, v, 0x7531);
                    u = sub_f16x2(u, u & TOP), v = sub_f16x2(v, v & TOP);
                    b[r / 4] = __byte_perm(u, v, 0x7531);
                    u = mul_f16x2(sub_f16x2(u, u & TOP), UP), v = mul_f16x2(sub_f16x2(v, v & TOP), UP);
                    a[RW / 4 + r / 4] = __byte_perm(u, v, 0x7531);
                    u = sub_f16x2(u, u & TOP), v = sub_f16x2(v, v & TOP);
                    b[RW / 4 + r / 4] = __byte_perm(u, v, 0x7531);
                }
#pragma unroll
                for (int c = 0; c < RW / 8; ++c) {
                    *reinterpret_cast<uint4*>(P + c * T * 16) = make_uint4(a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]);
                    *reinterpret_cast<uint4*>(P + S::PT + c * T * 16) = make_uint4(b[4 * c], b[4 * c + 1], b[4 * c + 2], b[4 * c + 3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(pready(tt & 1));
            }
            // hand m and l to the epilogue warps (once they are done with the previous item's)
            if (n > 0) WW(ofree, (n - 1) & 1u);
            int r0 = r_wg;
            const int ns = warp_sums<RW, 16>(l, lane, &r0);   // (lanes that hold the same sums write the same)
#pragma unroll
            for (int k = 0; k < RW; ++k)
                if (k < ns) l_sm[warp & 3][r0 + k] = l[k];
            if (pt < RW && r_wg + pt < I.v.rows) m_sm[r_wg + pt] = m, at_sm[r_wg + pt] = at + I.slot;
            mbar_arrive(mlready);
            item_done(n);
            t += nt;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem_slot, S::TMEM_COLS);
    }
    if (A.joined) {
        __threadfence_block();
        const int rt = blockIdx.x % A.nrt, g = blockIdx.x / A.nrt % A.Hkv, b = blockIdx.x / A.nrt / A.Hkv;
        const int last = min((rt + 1) * A.tile_rows, A.R * A.G);
        for (int k = tid; k < A.tile_rows * (HD / 4); k += S::THREADS) {
            const int gr = rt * A.tile_rows + k / (HD / 4), r = gr / A.G;
            if (gr < last) q8_join_one<HD>(C, b, r, g * A.G + gr - r * A.G, k % (HD / 4) * 4);
        }
    }
}

// One CTA per (row, q head): w_s = 2^(m_s - M) over the row's live slots s in order, out = sum w_s O_s /
// sum w_s l_s.  The i-th of them belongs to the sum of residue i mod CB_SUMS, and those sums are added in
// order: fixed by the row alone, whether G = 4 groups of threads have 4 residues each (few slots, or
// many rows) or 16 have one (many slots of few rows: their loads are in flight together).
constexpr int CB_SLOTS = 1 << 10;   // slots whose m and l are staged at a time

template <int HD, int G>
__global__ void __launch_bounds__(G* HD / 4) attn_q8_combine_kernel(const __grid_constant__ CombineArgs C) {
    griddep_launch();
    griddep_wait();
    constexpr int LN = HD / 4, NT = G * LN, PER = CB_SUMS / G;
    __shared__ float2 wl[CB_SLOTS];
    __shared__ float4 acc_sm[CB_SUMS][LN];
    __shared__ float l_sm[CB_SUMS], wmax[NT / 32];
    const int row = blockIdx.x, br = row / C.Hq, hq = row - br * C.Hq, b = br / C.R, r = br - b * C.R, tid = threadIdx.x;
    int L0;
    if (!q8_row(C, b, r, &L0)) return;
    const RowSlots slot(C, L0, r);
    const int ns = slot.n;
    const float2* ml = C.ml + static_cast<long long>(row) * C.nslot;
    const float4* op = reinterpret_cast<const float4*>(C.opart + static_cast<long long>(row) * C.nslot * HD) + tid % LN;
    float M = NEG_INF;
#pragma unroll 1
    for (int i = tid; i < ns; i += NT) {
        const float2 v = __ldcg(ml + slot[i]);
        if (i < CB_SLOTS) wl[i] = v;
        M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if ((tid & 31) == 0) wmax[tid >> 5] = M;
    __syncthreads();
    M = wmax[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) M = fmaxf(M, wmax[w]);
    const int grp = tid / LN, ln = tid % LN;
    float L[PER];
    float4 a[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) L[k] = 0.f, a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c0 = 0; c0 < ns; c0 += CB_SLOTS) {
        const int n = min(CB_SLOTS, ns - c0);
        if (c0) {
            __syncthreads();
            for (int i = tid; i < n; i += NT) wl[i] = __ldcg(ml + slot[c0 + i]);
            __syncthreads();
        }
        constexpr int UN = 8 / PER;   // 8 loads in flight
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += CB_SUMS * UN) {
            float4 o[UN][PER];
#pragma unroll
            for (int u = 0; u < UN; ++u)
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const int i = i0 + u * CB_SUMS + grp + k * G;
                    if (i < n) o[u][k] = __ldcg(op + static_cast<long long>(slot[c0 + i]) * LN);
                }
#pragma unroll
            for (int u = 0; u < UN; ++u)
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const int i = i0 + u * CB_SUMS + grp + k * G;
                    if (i >= n) continue;
                    const float w = ex2_approx(__fsub_rn(wl[i].x, M));
                    L[k] = __fmaf_rn(w, wl[i].y, L[k]);
                    a[k].x = __fmaf_rn(w, o[u][k].x, a[k].x);
                    a[k].y = __fmaf_rn(w, o[u][k].y, a[k].y);
                    a[k].z = __fmaf_rn(w, o[u][k].z, a[k].z);
                    a[k].w = __fmaf_rn(w, o[u][k].w, a[k].w);
                }
        }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        acc_sm[grp + k * G][ln] = a[k];
        if (ln == 0) l_sm[grp + k * G] = L[k];
    }
    __syncthreads();
    if (tid >= LN) return;
    float4 y = acc_sm[0][tid];
    float sum = l_sm[0];
#pragma unroll
    for (int g = 1; g < CB_SUMS; ++g) {
        const float4 o = acc_sm[g][tid];
        sum = __fadd_rn(sum, l_sm[g]);
        y.x = __fadd_rn(y.x, o.x), y.y = __fadd_rn(y.y, o.y), y.z = __fadd_rn(y.z, o.z), y.w = __fadd_rn(y.w, o.w);
    }
    q8_output<HD>(C, br, hq, 4 * tid, y, sum);
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Slots of a row and, of them, the sinks': without a window the splits up to max_len; with one the
// sinks' splits and as many as a window and the rows behind it can touch.
inline int slots(int R, int max_len, int window, int sinks, int* nsink) {
    const int all = q8_split_of(max_len - 1) + 1;
    *nsink = 0;
    if (!window || window >= max_len) return all;
    const int ns = sinks ? q8_split_of(min(sinks, max_len) - 1) + 1 : 0;
    const long long w = (static_cast<long long>(window) + R - 2) / 256 + 2;
    if (ns + w >= all) return all;   // then no slot is left out and none counts as a sink's
    *nsink = ns;
    return ns + static_cast<int>(w);
}

inline bool sizes_ok(int B, int R, int Hq, int hd, int max_ctx, int window, int sinks) {
    return B >= 1 && B <= 65535 && R >= 1 && R <= XV_KMAX && Hq >= 1 && (hd == 64 || hd == 128 || hd == 256) && max_ctx >= 1 &&
           max_ctx <= (1 << 30) && window >= 0 && sinks >= 0 && static_cast<long long>(B) * R * Hq <= (1ll << 30);
}

// Row tiles: as few as 64 rows allow, and of even sizes.
inline int row_tiles(int rows) { return (rows + 63) / 64; }

template <int HD, int NR>
xv_status launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, Q8Args& a, const CombineArgs& c, cudaStream_t s) {
    using S = Shape<HD, NR>;
    const auto kern = attn_q8_kernel<HD, NR>;
    const void* fn = reinterpret_cast<const void*>(kern);
    int sms = 0;
    if (xv_status st = kernel_smem_once(fn, S::SMEM, true, "attn_q8: set shared memory size")) return st;
    if (xv_status st = device_sm_count(&sms)) return st;
    const long long n_tiles = static_cast<long long>(a.nrt) * a.Hkv * a.B, n_items = n_tiles * a.nslot;
    if (n_items > (1ll << 30)) return fail(XV_ERR_UNSUPPORTED, "attn_q8: %lld work items", n_items);
    const int room = sms * S::PER_SM;
    // The only split of each row is its output: a second kernel would begin 1.5 to 3 us after the first
    // one's end (one token at 128: 6.9 us with it, 6.3 us without; clusters that join up to 16 splits took
    // 15.2 us for one verify at 2183, the second kernel 14.6)
    a.joined = n_items <= room && a.nslot == 1;
    trace_pre(s);
    launch_k(kern, dim3(static_cast<unsigned>(std::min<long long>(room, n_items))), dim3(S::THREADS), S::SMEM, s, tmK, tmV, a, c);
    const long long rows = static_cast<long long>(a.B) * a.R * a.Hq, seen = a.window ? std::min(a.window + static_cast<long long>(a.sinks), static_cast<long long>(a.max_len)) : a.max_len;
    return launched("attn_q8_kernel", s, K_ATTN_Q8, (2ll * HD + 8) * a.B * a.Hkv * seen + 2 * rows * HD + 4 * rows * a.nslot * (HD + 2));
}

template <int HD>
xv_status launch(const CUtensorMap& tmK, const CUtensorMap& tmV, Q8Args& a, const CombineArgs& c, cudaStream_t s) {
    const int n = a.tile_rows;
    if (xv_status st = n <= 8    ? launch_attn<HD, 8>(tmK, tmV, a, c, s)
                       : n <= 16 ? launch_attn<HD, 16>(tmK, tmV, a, c, s)
                       : n <= 24 ? launch_attn<HD, 24>(tmK, tmV, a, c, s)
                       : n <= 32 ? launch_attn<HD, 32>(tmK, tmV, a, c, s)
                       : n <= 48 ? launch_attn<HD, 48>(tmK, tmV, a, c, s)
                                 : launch_attn<HD, 64>(tmK, tmV, a, c, s))
        return st;
    if (a.joined) return XV_OK;
    const long long rows = static_cast<long long>(a.B) * a.R * a.Hq;
    // (with the first kernel's division of an SM's memory: another one would wait for the SMs to empty)
    auto go = [&](auto kern, int threads) -> xv_status {
        if (xv_status st = kernel_smem_once(reinterpret_cast<const void*>(kern), 0, true, "attn_q8: set shared memory size")) return st;
        trace_pre(s);
        launch_k(kern, dim3(static_cast<unsigned>(rows)), dim3(threads), 0, s, c);
        return XV_OK;
    };
    int sms = 0;
    if (xv_status st = device_sm_count(&sms)) return st;
    // 16 groups for many slots of few rows, 1024 threads per SM at most.  The whole call with 16 and with 4, in us:
    // 32 rows of 128 slots 53.6, 56.1; 128 of 30 43.9, 44.9; 192 of 128 71.2, 69.3; 1536 of 62 135, 118
    const bool wide = a.nslot > 2 * CB_SUMS && rows * 4 * HD <= 1024ll * sms;
    if (xv_status st = wide ? go(attn_q8_combine_kernel<HD, 16>, 4 * HD) : go(attn_q8_combine_kernel<HD, 4>, HD)) return st;
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
    sinks = std::min(sinks, max_ctx);   // further ones are behind every row (and sums with them would pass 2^31)
    const size_t need = xv_attn_q8_workspace_size(B, R, Hq, hd, max_ctx, window, sinks);
    if (!ws || ws_bytes < need) return fail(XV_ERR_WORKSPACE, "attn_q8: workspace of %zu bytes needed", need);
    if (!aligned16(ws)) return fail(XV_ERR_UNSUPPORTED, "attn_q8: workspace must be 16-byte aligned");
    unsigned* err = device_error_word();
    if (!err) return fail(XV_ERR_CUDA, "attn_q8: device error word unavailable");
    CUtensorMap tmK, tmV;
    const uint64_t dims[3] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(kv.page), static_cast<uint64_t>(kv.n_pages) * Hkv};
    const uint64_t strides[2] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(kv.page) * hd};
    const uint32_t box[3] = {static_cast<uint32_t>(hd < 128 ? hd : 128), static_cast<uint32_t>(T / 2), 1};
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
    const int grp = R * (Hq / Hkv), nrt = row_tiles(grp);
    Q8Args a{q, q_stride, kv, cache->k_scale, cache->v_scale, ctx_len, n_rows, R, Hq / Hkv, Hq, Hkv, B,
             (grp + nrt - 1) / nrt, nrt, Divisor(Hq / Hkv), Divisor(nrt), Divisor(Hkv), Divisor(nslot), Divisor(kv.page), nslot, nsink, max_ctx, win, win ? sinks : 0, shift, 0, scale * 1.4426950408889634f, opart, ml, err};
    const CombineArgs c{ctx_len, n_rows, R, Hq, nslot, nsink, max_ctx, win, win ? sinks : 0, shift, opart, ml, gate, gate_stride, out,
                        out_stride};
    return hd == 256 ? launch<256>(tmK, tmV, a, c, s) : hd == 128 ? launch<128>(tmK, tmV, a, c, s) : launch<64>(tmK, tmV, a, c, s);
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

int xv_attn_q8_split_begin(int s) {
    constexpr int LAST = Q8_FS + (INT_MAX - Q8_FAR) / 1024;   // the last split that begins below 2^31
    return s < 0 ? -1 : s > LAST ? INT_MAX : q8_split_begin(s);
}

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

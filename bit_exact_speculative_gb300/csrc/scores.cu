// Log probabilities of given tokens, entropies and top alternatives of rows of logits.
//
// For a row x of V logits:
//     m = max x,  S = sum exp(x_i - m),  D = sum exp(x_i - m) (x_i - m),
//     logprob(t) = (x_t - m) - log S,   entropy = log S - D / S,
// and the n largest x_i, the lowest index first among equals (a NaN below every number).
//
// A row is cut into chunks of SC_CHUNK logits, a chunk into a share of 32 logits per thread; a warp's
// shares give one (m, S, D), and a row's are joined in order.  Chunks, shares and the order of every sum
// are fixed by V alone, so a row has the same bits in a call of any number of rows, at any position and
// alignment.
//
// Persistent CTAs take equal runs of the call's chunks, each logit read once: bulk copies of whole
// 16-byte pieces bring a ring of chunks into shared memory (rows may start at any address: the pieces
// that hold a chunk's two ends are read whole), from where a thread takes every 256th logit.  Most rows
// lie in one CTA, which finishes them; of a row that reaches into other CTAs each leaves its warps' sums
// and its n best in the workspace, and the one that ends last (an atomic counter) joins them.
// (A CTA per chunk, its loads straight into registers: 392 us for 2048 rows of 151936, of 184 at the
// memory's rate, and 54 us for 500 rows of 50257 bf16 logits, whose odd rows were read one by one.)
//
// The exponentials alone are 512 cycles a chunk and SM, where the memory's rate leaves 720 for bf16
// logits, so what is done per logit and per chunk is kept small: no barrier but one a row, two logits an
// instruction, no reduction wider than a warp before a row's end, a warp of its own for the ring and one
// for the ends of rows (the join, the token's logit, the lists), while the others go on with the next
// row: 500 rows of 50257 bf16 logits took 33 us with a row's end in one of the computing warps.
//
// Each warp keeps the 32 best of its shares of a row, one a lane, in order.  A logit has to pass the n-th
// of them, and what n logits of the warps' reach: with k = n / 8, rounded up, the (n / k)-th largest of
// their k-th best (in a row's first chunk: of their lanes' best).  A few that pass are put in one by one,
// more by a bitonic sort and merge, and at a row's end the best of the warps' lists are taken.  (With one
// list for the CTA, and a barrier a chunk for it, 2048 rows of 151936 took 234 us with n = 1, 290 us with
// n = 20.)
#include <algorithm>
#include <cmath>

#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

constexpr int SC_THREADS = 256, SC_WARPS = SC_THREADS / 32;
constexpr int SC_KEYS = 512;                        // lists' keys at a time
constexpr int SC_PER = 32;                          // logits per thread
constexpr int SC_CHUNK = SC_THREADS * SC_PER;
constexpr int SC_V_MAX = 1 << 19;
constexpr int SC_C_MAX = SC_V_MAX / SC_CHUNK;
constexpr int SC_G_MAX = 1024;                      // CTAs
constexpr int SC_HEADER = SC_G_MAX * 4;             // their counters, wherever the rest lies
constexpr float LOG2E = 1.4426950408889634f;
static_assert(XV_TOP_MAX <= 32 && SC_WARPS == 8 && SC_KEYS >= 32 * SC_WARPS, "a lane each");

// Ring of chunks: as many as fit beside the CTAs of an SM.
template <typename T>
struct Ring {
    static constexpr int PER_SM = 2, N = sizeof(T) == 4 ? 3 : 5;
    static constexpr int BYTES = SC_CHUNK * static_cast<int>(sizeof(T)) + 16;   // any alignment
    static constexpr int STRIDE = (BYTES + 127) / 128 * 128;
    static constexpr int SMEM = N * STRIDE + 128;
    static_assert(PER_SM * (SMEM + 15 * 1024 + 1024) <= 228 * 1024, "");
};

using Key = unsigned long long;   // (1 + order of the value) << 32 | ~index: larger is better, 0 is none

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
    unsigned* cnt;     // [SC_G_MAX], zero between calls: of the row that starts in a CTA and leaves it
    float4* part;      // [CTAs][C][SC_WARPS] (m, S, D, -) of that row
    Key* keys;         // [CTAs][2][top] n best of the row that entered the CTA, and of the one that leaves it
    unsigned* err;
};

// Unsigned order of a float: NaN 1, then -inf .. +inf, -0 as +0; 0 is none.
__device__ __forceinline__ unsigned order_of(float x) {
    const unsigned u = __float_as_uint(__fadd_rn(x, 0.f));
    return x != x ? 1u : ((u & 0x80000000u) ? ~u : u | 0x80000000u) + 1u;
}
__device__ __forceinline__ float value_of(unsigned o) {
    --o;
    return o == 0 ? __uint_as_float(0x7fc00000u) : __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_to_f32(x); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Sorts a warp's bitonic keys, the largest into lane 0.
__device__ __forceinline__ Key bitonic_down(Key k, int lane) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const Key o = __shfl_xor_sync(0xffffffffu, k, off);
        k = (lane & off) == 0 ? (k > o ? k : o) : (k < o ? k : o);
    }
    return k;
}
// The 32 best of two sorted lists (the largest in lane 0), the second one read backwards.
__device__ __forceinline__ Key merge_best(Key list, Key backwards, int lane) {
    return bitonic_down(list > backwards ? list : backwards, lane);
}
__device__ __forceinline__ Key reversed(Key k, int lane) { return __shfl_sync(0xffffffffu, k, 31 - lane); }
// The n best of a warp's sorted lists, one per lane, `have` keys long (0: none): n times the largest head.
// The k-th best ends in lane k.
__device__ __forceinline__ Key best_of_heads(const Key* list, int have, int n, int lane) {
    Key h = have > 0 ? list[0] : 0, next = have > 1 ? list[1] : 0, mine = 0;
    int at = 1;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        const unsigned hi = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(h >> 32));
        const unsigned lo = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(h >> 32) == hi ? static_cast<unsigned>(h) : 0u);
        const Key w = static_cast<Key>(hi) << 32 | lo;
        if (lane == k) mine = w;
        if (h == w) {
            h = next;
            next = ++at < have ? list[at] : 0;
        }
    }
    return mine;
}
// Sorts a warp's keys, the smallest into lane 0.
__device__ __forceinline__ Key sort_up(Key k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int off = size / 2; off > 0; off >>= 1) {
            const Key o = __shfl_xor_sync(0xffffffffu, k, off);
            const bool up = (lane & size) == 0 || size == 32, low = (lane & off) == 0;
            k = low == up ? (k < o ? k : o) : (k > o ? k : o);
        }
    return k;
}

// The q-th largest of 8 words in shared memory, as they are now.
__device__ __forceinline__ unsigned largest8(uint32_t at, int q, int lane) {
    unsigned v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + 4 * (lane % 8)) : "memory");
    int reach = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) reach += __shfl_sync(0xffffffffu, v, k) >= v;
    return __reduce_max_sync(0xffffffffu, reach >= q ? v : 0u);
}

// Barrier of the warps that compute.
__device__ __forceinline__ void sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(SC_THREADS) : "memory"); }

template <typename T, bool TOP>
__global__ void __launch_bounds__(SC_THREADS + 64, Ring<T>::PER_SM) logprobs_kernel(const __grid_constant__ ScoreArgs A) {
    griddep_launch();
    using R = Ring<T>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[R::N], empty[R::N], ends[2], freed[2];
    __shared__ Key lists[2][TOP ? 32 * SC_WARPS : 1], others[TOP ? SC_KEYS : 1];   // of the warps at a row's end; of other CTAs
    __shared__ __align__(16) unsigned floors[2][SC_WARPS];   // what part_n of a warp's logits reach, by the row's parity
    __shared__ float pm[SC_C_MAX * SC_WARPS], ps[SC_C_MAX * SC_WARPS], pd[SC_C_MAX * SC_WARPS];   // [chunk][warp]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, top = A.top, C = A.C;
    const uint32_t raw = smem_u32(smem_raw), ring = (raw + 127u) & ~127u;
    uint8_t* bufs = smem_raw + (ring - raw);
    if (tid == 0) {
        for (int st = 0; st < R::N; ++st) mbar_init(smem_u32(&full[st]), 1), mbar_init(smem_u32(&empty[st]), SC_WARPS);
        for (int k = 0; k < 2; ++k) mbar_init(smem_u32(&ends[k]), SC_WARPS), mbar_init(smem_u32(&freed[k]), 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    const int rows = A.n_rows ? min(max(*A.n_rows, 0), A.M) : A.M;
    const int n_chunks = rows * C;   // below 2^31
    const int G = min(static_cast<int>(gridDim.x), n_chunks);   // CTAs with a chunk at least
    if (static_cast<int>(blockIdx.x) >= G) return;
    const int i0 = static_cast<int>(static_cast<long long>(blockIdx.x) * n_chunks / G);
    const int i1 = static_cast<int>((blockIdx.x + 1ll) * n_chunks / G);

    const T* base = static_cast<const T*>(A.logits);
    int row = i0 / C, c = i0 - row * C;
    // a row's sums and lists stand in one of two buffers, while the next row fills the other; a row of more
    // than half the chunks there can be has both
    const int bufs2 = C <= SC_C_MAX / 2 ? 2 : 1, half = SC_C_MAX / 2 * SC_WARPS;
    if (warp == SC_WARPS) {
        // ---- the chunks into the ring, in whole 16-byte pieces
        if (lane) return;
        const int count = i1 - i0;
        int j = 0;
        for (; j < count; ++j) {
            const int st = j % R::N;
            if (j >= R::N && !mbar_wait(smem_u32(&empty[st]), ((j / R::N) & 1u) ^ 1u, A.err)) break;
            const uintptr_t a = reinterpret_cast<uintptr_t>(base + row * A.ld + c * SC_CHUNK);
            const uintptr_t lo = a & ~static_cast<uintptr_t>(15);
            const uintptr_t hi = (a + min(SC_CHUNK, A.V - c * SC_CHUNK) * sizeof(T) + 15) & ~static_cast<uintptr_t>(15);
            const uint32_t bar = smem_u32(&full[st]);
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(hi - lo));
            bulk_load(ring + st * R::STRIDE, reinterpret_cast<const void*>(lo), static_cast<uint32_t>(hi - lo), bar);
            if (++c == C) c = 0, ++row;
        }
        // every copy issued lands before the CTA leaves
        for (int k = max(0, j - R::N); k < j; ++k) mbar_wait(smem_u32(&full[k % R::N]), (k / R::N) & 1u, A.err);
        return;
    }

    if (warp == SC_WARPS + 1) {
        // ---- the ends of rows, and of the run
        bool ok = true;
        for (int i = i0, seg = 0; i < i1; ++seg, ++row, c = 0) {
            const int first_c = c, last_c = min(C - 1, c + i1 - i - 1), buf = seg % bufs2;
            const bool row_ends = last_c == C - 1;
            i += last_c - first_c + 1;
            float *pmr = pm + buf * half, *psr = ps + buf * half, *pdr = pd + buf * half;
            const int token = __ldg(A.tokens + row);
            const float token_x = token >= 0 && token < A.V ? to_float(__ldg(base + row * A.ld + token)) : 0.f;
            if (ok) ok = mbar_wait(smem_u32(&ends[buf]), (seg / bufs2) & 1u, A.err);
            bool last = true;
            Key list = 0;
            if (TOP) {
                // (a head takes 200 cycles, the merges 2300)
                if (top <= 8) list = best_of_heads(lists[buf] + lane * 32, lane < SC_WARPS ? top : 0, top, lane);
                else {
                    const Key* l = lists[buf];
                    auto two = [&](int w) { return merge_best(l[w * 32 + lane], l[w * 32 + 63 - lane], lane); };
                    const Key a = merge_best(two(0), reversed(two(2), lane), lane), b = merge_best(two(4), reversed(two(6), lane), lane);
                    list = merge_best(a, reversed(b, lane), lane);
                }
            }
            if (first_c != 0 || !row_ends) {
                // the row lies in CTAs a to z; ((i + 1) G - 1) / n_chunks is the CTA of chunk i
                const long long r0 = static_cast<long long>(row) * C;
                const int a = static_cast<int>(((r0 + 1) * G - 1) / n_chunks), z = static_cast<int>(((r0 + C) * G - 1) / n_chunks);
                float4* gp = A.part + static_cast<long long>(a) * C * SC_WARPS;
                for (int k = first_c * SC_WARPS + lane; k < (last_c + 1) * SC_WARPS; k += 32) __stcg(gp + k, make_float4(pmr[k], psr[k], pdr[k], 0.f));
                if (TOP && lane < top) __stcg(A.keys + (2ll * blockIdx.x + (first_c == 0)) * top + lane, list);
                __threadfence();
                __syncwarp();
                unsigned seen = 0;
                if (lane == 0) seen = atomicAdd(A.cnt + a, 1u);
                last = __shfl_sync(0xffffffffu, seen, 0) == static_cast<unsigned>(z - a);
                if (last) {
                    if (lane == 0) A.cnt[a] = 0;
                    __threadfence();
#pragma unroll 8
                    for (int k = lane; k < C * SC_WARPS; k += 32) {
                        const float4 q = __ldcg(gp + k);
                        pmr[k] = q.x, psr[k] = q.y, pdr[k] = q.z;
                    }
                    if (TOP) {
                        // lane 0 has the list so far, the others a CTA's each
                        list = lane < top ? __ldcg(A.keys + (2ll * a + 1) * top + lane) : 0;
                        const int most = min(31, SC_KEYS / top - 1);
                        for (int g = a + 1; g <= z; g += most) {
                            const int nl = min(most, z + 1 - g);
                            if (lane < top) others[lane] = list;
                            // list h of the round, key j: after the first, in order
#pragma unroll 8
                            for (int k = lane; k < nl * top; k += 32) {
                                const int h = k / top;
                                others[top + k] = __ldcg(A.keys + 2ll * (g + h) * top + k - h * top);
                            }
                            __syncwarp();
                            list = best_of_heads(others + lane * top, lane <= nl ? top : 0, top, lane);
                            __syncwarp();
                        }
                    }
                    __syncwarp();
                }
            }
            if (last) {
                float mrow = -INFINITY;
                for (int k = lane; k < C * SC_WARPS; k += 32)
                    if (psr[k] != 0.f) mrow = fmaxf(mrow, pmr[k]);   // S = 0: nothing but -inf
                mrow = warp_max(mrow);
                for (int k = lane; k < C * SC_WARPS; k += 32) {
                    const float off = __fsub_rn(pmr[k], mrow), S = psr[k];
                    pmr[k] = S == 0.f ? 0.f : expf(off);
                    // a share of finite mask values, far below the row's maximum: its weight is 0 from off = -104 on, and
                    // -1e30 S, S <= 1024, stays finite beside it (0 times infinity is not 0)
                    pdr[k] = S == 0.f ? 0.f : __fmaf_rn(fmaxf(off, -1e30f), S, pdr[k]);
                }
                __syncwarp();
                float S = 0.f, D = 0.f;   // of a warp's shares, in lanes 0 to 7 and again in the others
#pragma unroll 4
                for (int k = lane % SC_WARPS; k < C * SC_WARPS; k += SC_WARPS) {
                    S = __fmaf_rn(pmr[k], psr[k], S);
                    D = __fmaf_rn(pmr[k], pdr[k], D);
                }
#pragma unroll
                for (int off = SC_WARPS / 2; off > 0; off >>= 1) {
                    S = __fadd_rn(S, __shfl_xor_sync(0xffffffffu, S, off));
                    D = __fadd_rn(D, __shfl_xor_sync(0xffffffffu, D, off));
                }
                const float logs = logf(S);
                const bool empty = S == 0.f;   // every logit -inf
                auto score = [&](float xv) { return empty ? -INFINITY : __fsub_rn(__fsub_rn(xv, mrow), logs); };
                if (lane == 0) {
                    if (A.entropy) A.entropy[row] = empty ? 0.f : __fsub_rn(logs, __fdiv_rn(D, S));
                    const bool in = token >= 0 && token < A.V;
                    if (!in && token != -1) atomicOr(A.err, ERR_BAD_TOKEN);
                    A.logprob[row] = in ? score(token_x) : token == -1 ? 0.f : __uint_as_float(0x7fc00000u);
                }
                if (TOP && lane < top) {
                    const long long o = static_cast<long long>(row) * top + lane;
                    A.ids[o] = static_cast<int32_t>(~static_cast<unsigned>(list));
                    A.lps[o] = score(value_of(static_cast<unsigned>(list >> 32)));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&freed[buf]));
        }
        return;
    }

    Key list = 0, least = 0;      // the lane's of the warp's best; a new key has to pass the last of n
    unsigned floor = 0;
    // part_w warps with part_n logits each make n at least
    const int part_n = (top + SC_WARPS - 1) / SC_WARPS, part_w = part_n ? (top + part_n - 1) / part_n : 0;
    int first_c = c;              // of this row in this CTA
    int st = 0, ph = 0;
    int seg = 0;                  // rows begun in this CTA
    bool ok = true;
    for (int i = i0; i < i1; ++i) {
        const int at0 = c * SC_CHUNK, n = min(SC_CHUNK, A.V - at0);
        const int buf = seg % bufs2;
        // (a wait that gave up is recorded; what follows reads stale logits, but ends)
        if (ok) ok = mbar_wait(smem_u32(&full[st]), ph, A.err);
        const T* x = reinterpret_cast<const T*>(bufs + st * R::STRIDE + (reinterpret_cast<uintptr_t>(base + row * A.ld + at0) & 15)) + tid;
        float v[SC_PER];
        if (n == SC_CHUNK) {
#pragma unroll
            for (int k = 0; k < SC_PER; ++k) v[k] = to_float(x[k * SC_THREADS]);
        } else {
#pragma unroll
            for (int k = 0; k < SC_PER; ++k) v[k] = k * SC_THREADS + tid < n ? to_float(x[k * SC_THREADS]) : -INFINITY;
        }
        if (c == first_c && seg >= bufs2 && ok) ok = mbar_wait(smem_u32(&freed[buf]), (seg / bufs2 - 1) & 1u, A.err);
        float mx4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int k = 4; k < SC_PER; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], v[k]);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));   // NaN only if all are
        if (TOP) {
            // (0 where every logit of the thread is NaN, masked or behind the row)
            const unsigned need = static_cast<unsigned>(least >> 32), best = mx > -INFINITY ? order_of(mx) : 0u;
            if (c == first_c) {
                unsigned b = best;
                for (int k = part_n;; --k) {   // the part_n-th largest
                    floor = __reduce_max_sync(0xffffffffu, b);
                    if (k == 1) break;
                    if (lane == __ffs(__ballot_sync(0xffffffffu, b == floor)) - 1) b = 0;
                }
                if (lane == 0) floors[seg & 1][warp] = floor;
                sync();
            }
            unsigned pass = largest8(smem_u32(floors[seg & 1]), part_w, lane);
            const bool some = best > need && best >= pass;
            pass = max(pass, need);
            const bool rest = pass <= order_of(-INFINITY);   // what is not a number above -inf counts, too
            if (__any_sync(0xffffffffu, some || rest)) {
                const float low = rest ? -INFINITY : value_of(pass);
                unsigned hit = 0;
#pragma unroll
                for (int k = 0; k < SC_PER; ++k) hit |= v[k] < low ? 0u : 1u << k;
                if (rest && n < SC_CHUNK) hit &= n > tid ? 0xffffffffu >> (31 - (n - tid - 1) / SC_THREADS) : 0u;
                for (;;) {
                    Key mine = 0;   // the lane's next that passes
                    while (hit) {
                        const int k = __ffs(hit) - 1;
                        mine = static_cast<Key>(order_of(to_float(x[k * SC_THREADS]))) << 32 | static_cast<unsigned>(~(at0 + k * SC_THREADS + tid));
                        if (mine > least) break;
                        mine = 0;
                        hit &= hit - 1;
                    }
                    const unsigned who = __ballot_sync(0xffffffffu, mine != 0);
                    if (!who) break;
                    if (__popc(who) > 4) {
                        list = merge_best(list, sort_up(mine, lane), lane);
                        hit &= hit - 1;
                    } else {
                        const int src = __ffs(who) - 1;
                        const Key key = __shfl_sync(0xffffffffu, mine, src), before = __shfl_up_sync(0xffffffffu, list, 1);
                        const int at = __popc(__ballot_sync(0xffffffffu, list > key));
                        list = lane < at ? list : lane == at ? key : before;
                        if (lane == src) hit &= hit - 1;
                    }
                    least = __shfl_sync(0xffffffffu, list, top - 1);
                }
                floor = max(floor, static_cast<unsigned>(__shfl_sync(0xffffffffu, list, part_n - 1) >> 32));
                if (lane == 0) floors[seg & 1][warp] = floor;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[st]));   // the stage may be filled again
        const float m = warp_max(mx), ref = m > -INFINITY ? m : 0.f;
        float s4[4] = {0.f, 0.f, 0.f, 0.f}, d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < SC_PER; k += 2) {
            if (k % 8 == 0 && k * SC_THREADS >= n) break;   // behind the row: they would add 0
            float a = v[k], b = v[k + 1];
            add2(a, b, -ref, -ref);
            float ea = a, eb = b;
            mul2(ea, eb, LOG2E, LOG2E);
            ea = ex2_approx(ea), eb = ex2_approx(eb);
            add2(s4[k & 3], s4[(k & 3) + 1], ea, eb);
            fma2_acc(d4[k & 3], d4[(k & 3) + 1], ea, eb, fmaxf(a, -3e38f), fmaxf(b, -3e38f));   // exp(-inf) (-inf) is 0 here
        }
        const float s = warp_sum(__fadd_rn(__fadd_rn(s4[0], s4[1]), __fadd_rn(s4[2], s4[3])));
        const float d = warp_sum(__fadd_rn(__fadd_rn(d4[0], d4[1]), __fadd_rn(d4[2], d4[3])));
        if (lane == 0) {
            const int k = buf * half + c * SC_WARPS + warp;
            pm[k] = ref, ps[k] = s, pd[k] = d;
        }
        if (++st == R::N) st = 0, ph ^= 1;
        const bool row_ends = c == C - 1;
        if (!row_ends && i + 1 < i1) {
            ++c;
            continue;
        }
        if (TOP) lists[buf][warp * 32 + lane] = list;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ends[buf]));
        ++seg;
        ++row;
        c = first_c = 0;
        list = least = 0;
    }
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool sizes_ok(int M, int V, int top) {
    return M >= 1 && V >= 1 && V <= SC_V_MAX && top >= 0 && top <= XV_TOP_MAX && top <= V &&
           static_cast<long long>(M) * ceil_div(V, SC_CHUNK) < (1ll << 31);
}

// CTAs at most
inline size_t ctas(int M, int C) { return std::min<size_t>(SC_G_MAX, static_cast<size_t>(M) * C); }

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
    w += SC_HEADER;
    a.part = reinterpret_cast<float4*>(w);
    w += ctas(M, C) * C * SC_WARPS * sizeof(float4);
    a.keys = reinterpret_cast<Key*>(w);
    int sms = 0;
    if (xv_status st = device_sm_count(&sms)) return st;
    auto go = [&](auto kern, int smem, int per_sm) -> xv_status {
        if (xv_status st = kernel_smem_once(reinterpret_cast<const void*>(kern), smem, true, "logprobs: set shared memory size")) return st;
        const size_t grid = std::min(ctas(M, C), static_cast<size_t>(sms) * per_sm);
        trace_pre(s);
        launch_k(kern, dim3(static_cast<unsigned>(grid)), dim3(SC_THREADS + 64), smem, s, a);
        return XV_OK;
    };
    using F = Ring<float>;
    using H = Ring<uint16_t>;
    if (xv_status st = f32 ? (top ? go(logprobs_kernel<float, true>, F::SMEM, F::PER_SM) : go(logprobs_kernel<float, false>, F::SMEM, F::PER_SM))
                           : (top ? go(logprobs_kernel<uint16_t, true>, H::SMEM, H::PER_SM)
                                  : go(logprobs_kernel<uint16_t, false>, H::SMEM, H::PER_SM)))
        return st;
    return launched("logprobs_kernel", s, K_LOGPROBS, (f32 ? 4ll : 2ll) * M * V + M * (12ll + 8 * top));
}

}  // namespace
}  // namespace xv

using namespace xv;

extern "C" {

size_t xv_logprobs_workspace_size(int M, int V, int top) {
    if (!sizes_ok(M, V, top)) return 0;
    const int C = ceil_div(V, SC_CHUNK);
    const size_t n = ctas(M, C);
    return SC_HEADER + round256(n * C * SC_WARPS * sizeof(float4) + 2 * n * top * sizeof(Key));
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

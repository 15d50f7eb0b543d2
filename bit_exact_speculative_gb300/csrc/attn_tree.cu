// Attention of a tree of drafted tokens over a bf16 KV cache, on tcgen05, with the bits of decode.
//
// Every row (node, q head) attends to the cache's ctx positions and to its own path, and is computed
// by the operations of a decode row at its position (attn.cu): splits at fixed absolute positions,
// tiles of 64 positions, an fp32 online softmax over the tiles in order with the sum l taken position
// by position, P rounded to bf16 (the tensor core takes it in V's type), P V accumulated 16 positions (one
// MMA K step) at a time, the splits combined in split order.  A tree changes nothing of that below
// position 16 * (ctx / 16): those positions are the same for every row.  Above, rows disagree about what
// stands at a position:
//   - scores: Q K^T against all nodes at once (one 64-column tile, each score its own dot product); a
//     row masks the nodes off its path.  Nodes are numbered after their parents, so a row's path in
//     node order is in position order, and adding the masked zeros leaves its sum's bits alone;
//   - P V: the 16 positions of one K step stay one K step.  For every node t that is the last of its
//     path inside a 16-position group (a leaf, or the group's last position), a block of 16 V rows is
//     gathered: the cache's rows below ctx, then t's ancestors in the group, zeros past t.  A row has
//     its p in the block its path runs through, p = 0 in all others, and blocks go in position order,
//     so what each row accumulates, K step by K step, is a decode row's sequence with no-ops between.
// A non-finite V value would turn those no-ops into NaN (0 * inf), so the gather replaces it by zero
// and the epilogue adds p * v itself, for the rows whose path holds it.
//
// Work items (split, row tile, kv head, sequence); a row tile is up to 128 rows: as many whole nodes,
// Hq/Hkv rows each, as fit, spread evenly over the tiles.  Per item, as in attn.cu: K and V tiles by
// TMA into rings, Q by TMA into the A operand, S = Q K^T and O += P V in tensor memory, softmax one
// thread per row.  An SM does 128 x 64 scores per K tile whatever rows hold nodes (63 nodes x 6 q heads
// per kv head: three tiles of 126 rows; 64 nodes: four of 96), so wide trees over long contexts are bound
// by the tensor core and the softmax, small ones by the K/V stream, batches of short contexts by their
// trees' tails, which do not overlap in a CTA, single short contexts by latency.
//
// Measured (24 q / 4 kv heads of 256 unless said): 8 nodes at 131072 positions 101 us, 5.3 TB/s of K and V;
// 64 nodes there 272 us, 757 TFLOP/s; 32 x 13 nodes at 4000 to 8000, 32 / 8 heads of 128, 178 us, 4.0 TB/s, and
// at 1000 to 2000 93 us, 2.2 TB/s; 16 nodes at 2183 16.6 us; 8 nodes at 128, 2 / 1 heads of 64, 6.4 us.
#include <cmath>

#include "xv_internal.h"
#include "xv_ptx.cuh"

namespace xv {
namespace {

constexpr int T = ATTN_TILE;
constexpr float NEG_INF = -INFINITY;
constexpr float RESCALE_SLACK = 2.f;   // as the decode rows' (log2 units)
typedef unsigned long long u64;

// Shared-memory plan (offsets from a 1024-byte aligned base), 128-byte swizzle throughout:
//   Q      CB blocks of [128 rows][64 dims]
//   K ring SK stages of CB blocks of [64 positions][64 dims]; V ring SV stages, the same (SV even)
//   PB[2]  [128 rows][64 slots] bf16, the P of the block steps; at hd 256 they take the stage of the
//          tree's K tile, which is done with by then
//   barriers, hand-over values, tree info
// P of the cache's tiles goes through tensor memory: at hd 256 the 32 KB it would take here are the
// third K stage.
struct TreeInfo;
template <int HD>
struct TreeShape {
    static constexpr int CB = HD / 64;
    static constexpr int QBLK = 128 * 128;
    static constexpr int BLK = T * 128;
    static constexpr int TILE_BYTES = CB * BLK;
    static constexpr bool PB_IN_K = HD == 256;
    static constexpr int SK = HD == 256 ? 3 : 5;
    static constexpr int SV = HD == 256 ? 2 : 4;
    static constexpr int K_OFF = CB * QBLK;
    static constexpr int V_OFF = K_OFF + SK * TILE_BYTES;
    static constexpr int PB_OFF = V_OFF + SV * TILE_BYTES;
    static constexpr int BAR_OFF = PB_OFF + (PB_IN_K ? 0 : 2 * QBLK);
    static constexpr int N_BARS = 2 * SK + 2 * SV + 28;
    static constexpr int M_OFF = BAR_OFF + 8 * ((N_BARS + 1) / 2 * 2);   // float[128]
    static constexpr int SUM_OFF = M_OFF + 512;                          // float[2][128]
    static constexpr int INFO_OFF = SUM_OFF + 1024;
    // the plan needs its base on a 1024-byte boundary: dynamic shared memory starts on one (it is all
    // this kernel has); with room to spare a full kilobyte of slack is taken all the same
    static constexpr int SLACK = HD == 256 ? 0 : 1024;
    // tensor-memory columns: S[2] (64 each), O (HD; at hd 64 and 128 two of them, item by item), the
    // tree's scores (64), P[2] (32 each)
    static constexpr int NO = HD == 256 ? 1 : 2;
    static constexpr uint32_t TMEM_COLS = 512;
};

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
    int G, NT, nrt, nsplit;   // q heads per kv head; nodes per row tile, row tiles, splits the launch is sized for
    float* opart;             // partial outputs, [B][Hkv][nsplit][row tile][HD / 4][rows of the tile][4]
    float2* ml;               // [B*N*Hq][nsplit]
    int32_t* nsp;             // [B*N] splits of each node's rows
};

// warps 0-3 softmax of an item's even tiles, tail and epilogue, 4-7 softmax of its odd tiles (thread =
// row = TMEM lane) and the gather, 8 K, 9 V and the tree's info, 10 Q and Q K^T, 11 P V.  Three warps per
// SM sub-partition leave each thread 168 registers, a thirteenth would leave 128: the softmax then
// waits on its own dependences and spills (32 x 13 nodes at 4000 to 8000 positions: 178 us, 265 with 128).
constexpr int TREE_THREADS = 384;

struct TreeItem {
    int b, g, rt, split, ctx, n, p_begin;
    int nfull;        // whole tiles of cache positions
    int c;            // cache positions of the tail tile (the tile that holds position ctx)
    bool tail0, tail1;   // this split holds the tail tile; the tile after it
    bool live;
    __device__ __forceinline__ bool tail() const { return tail0 || tail1; }
    __device__ __forceinline__ int kreg() const { return nfull + (tail0 && c > 0 ? 1 : 0); }      // K tiles of cache positions
    __device__ __forceinline__ int vreg() const { return nfull + (tail0 && c >= 16 ? 1 : 0); }    // V tiles of them
    __device__ __forceinline__ int node0(int NT) const { return rt * NT; }
};

// what follows from b, rt and split
__device__ __forceinline__ void tree_item_split(TreeItem& I, int NT) {
    I.p_begin = attn_split_begin(I.split);
    const int p_end = attn_split_begin(I.split + 1), t0 = I.ctx - I.c;
    I.nfull = I.p_begin < t0 ? (min(t0, p_end) - I.p_begin) / T : 0;
    I.tail0 = t0 >= I.p_begin && t0 < p_end;
    // a node stands in the tile after the tail when its depth is at least T - c
    I.tail1 = I.n - 1 >= T - I.c && t0 + T >= I.p_begin && t0 + T < p_end;
    I.live = I.rt * NT < I.n && (I.nfull > 0 || I.tail0 || I.tail1);
}

__device__ __forceinline__ TreeItem tree_item_at(const TreeArgs& A, int b, int g, int rt, int split) {
    TreeItem I;
    I.b = b, I.g = g, I.rt = rt, I.split = split;
    const int ctx = __ldg(A.ctx_len + b), n = A.n_nodes ? __ldg(A.n_nodes + b) : A.N;
    const bool bad = ctx < 0 || ctx > A.max_ctx;   // no nodes then
    I.ctx = bad ? 0 : ctx;
    I.n = bad ? 0 : min(max(n, 0), A.N);
    I.c = I.ctx & (T - 1);
    tree_item_split(I, A.NT);
    return I;
}

// Out of line, like everything below that runs once per item: the roles' loops share the SM's
// instruction cache, and the code around them decides how much of it they get.  Items go by value: one
// whose address is taken lives in local memory, and the loops read it there.
__device__ __noinline__ TreeItem tree_item(const TreeArgs& A, int it, int rt) {
    // items are numbered split-fastest, then row tiles (rt < 0) or those of row tile rt alone
    const int split = it % A.nsplit, tile = it / A.nsplit, head = rt < 0 ? tile / A.nrt : tile;
    return tree_item_at(A, head / A.Hkv, head % A.Hkv, rt < 0 ? tile % A.nrt : rt, split);
}

// ctx or n_nodes out of range: once per sequence
__device__ __forceinline__ void tree_report(const TreeArgs& A, int b) {
    const int ctx = __ldg(A.ctx_len + b), n = A.n_nodes ? __ldg(A.n_nodes + b) : A.N;
    if (ctx < 0 || ctx > A.max_ctx) atomicOr(A.err, ERR_BAD_LENGTH);
    if (n < 0 || n > A.N) atomicOr(A.err, ERR_BAD_COUNT);
}

// The items [*it0, *it1) of persistent CTA `blockIdx.x`: contiguous shares of the batch by weight, so that
// sequences of different lengths even out (32 x 13 nodes at 4000 to 8000 positions: 242 us with shares of
// equal item counts, 215 so).  A tile weighs 1, an item ITEM_WEIGHT more (1 to 4 measured alike) and a
// tree's tail TAIL_WEIGHT (64 nodes at 32768 positions: 99 us with 4 to 8, 90 with 16; 8 x 40 nodes at
// 9000: 123 and 115).  A cut is a weight between 0 and the total; its item is found from prefix sums over
// the sequences, a run of them per thread.  `sm`: one word per warp and the two results, not written
// before the next barrier.
//
// Where all trees have all row tiles (and at least 7/8 of the CTAs form whole bundles), a share goes to a
// bundle of nrt CTAs, one per row tile (*rt; else -1): they read the same K and V tiles at the same time,
// once from HBM and then from L2.  With a share per CTA the row tiles of a split ran far apart (63 nodes in
// three row tiles at 131072 positions: 306 us, 245 so).
constexpr int ITEM_WEIGHT = 4, TAIL_WEIGHT = 16;
__device__ __forceinline__ int tree_weight(int split) { return split * ITEM_WEIGHT + attn_split_begin(split) / T; }   // splits before
__device__ __noinline__ void tree_share(const TreeArgs& A, long long* sm, int* it0, int* it1, int* rt) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
    const int run = (A.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x), b0 = min(tid * run, A.B), b1 = min(b0 + run, A.B);
    // row tiles with a node; weight of each of sequence b's (kv head, row tile) pairs
    auto tiles = [&](int b, int& weight) -> int {
        const int ctx = __ldg(A.ctx_len + b), n = min(max(A.n_nodes ? __ldg(A.n_nodes + b) : A.N, 0), A.N);
        if (ctx < 0 || ctx > A.max_ctx) return 0;
        weight = attn_split_count(ctx + n) * ITEM_WEIGHT + (ctx + n) / T + TAIL_WEIGHT;
        return (n + A.NT - 1) / A.NT * A.Hkv;
    };
    long long own = 0;
    bool full = true;
    for (int b = b0; b < b1; ++b) {
        int w = 0;
        const int t = tiles(b, w);
        full = full && (t == 0 || t == A.nrt * A.Hkv);
        if (blockIdx.x == 0) tree_report(A, b);
        own += static_cast<long long>(t) * w;
    }
    long long incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) sm[warp] = incl;
    if (tid < 2) sm[n_warps + tid] = -1;   // past the last item
    const int bundles = gridDim.x / A.nrt;
    const bool bundled = __syncthreads_and(full) && bundles * A.nrt * 8 >= static_cast<int>(gridDim.x) * 7;
    long long total = 0, before = incl - own;
    for (int w = 0; w < n_warps; ++w) {
        if (w < warp) before += sm[w];
        total += sm[w];
    }
    const int per = bundled ? A.nrt : 1, share = blockIdx.x / per, shares = gridDim.x / per;   // CTAs a share has
    *rt = bundled ? static_cast<int>(blockIdx.x) % A.nrt : -1;
    total /= per, before /= per, own /= per;   // without remainders
    for (int e = 0; e < 2 && share < shares; ++e) {
        long long x = total * (share + e) / shares;
        if (x < before || x >= before + own) continue;
        x -= before;
        for (int b = b0; b < b1; ++b) {
            int w = 0;
            const int t = tiles(b, w) / per;
            const long long all = static_cast<long long>(t) * w;
            if (x >= all) {
                x -= all;
                continue;
            }
            const int j = static_cast<int>(x / w), rest = static_cast<int>(x - static_cast<long long>(j) * w), live = t / A.Hkv;   // row tiles
            int split = 0;   // the cut goes to the nearer end of the item it falls into
            while (split < A.nsplit && tree_weight(split) + tree_weight(split + 1) <= 2 * rest) ++split;
            sm[n_warps + e] = ((static_cast<long long>(b) * A.Hkv + j / live) * (A.nrt / per) + j % live) * A.nsplit + split;
            break;
        }
    }
    __syncthreads();
    const int end = A.B * A.Hkv * (A.nrt / per) * A.nsplit;
    *it0 = sm[n_warps] < 0 ? end : static_cast<int>(sm[n_warps]);
    *it1 = sm[n_warps + 1] < 0 ? end : static_cast<int>(sm[n_warps + 1]);
}

// What the rows of one tail item know about their tree; positions are relative to the tail tile.
struct TreeInfo {
    u64 anc[XV_KMAX];          // the path from the root: ancestors and the node itself
    uint8_t pos[XV_KMAX];      // c + depth (16-byte aligned)
    u64 tile0;                 // nodes standing in the tail tile
    u64 ends;                  // nodes at the last position of a 16-position group
    u64 vbad;                  // nodes whose V holds a non-finite value (set by the gather)
    unsigned cbad;             // the same for the cache positions of the blocks' first group
    uint8_t rep[XV_KMAX];      // the terminal node whose block holds the node
    uint8_t idx[XV_KMAX];      // block number of a terminal node
    uint8_t list[XV_KMAX];     // terminal node of a block: blocks by group, then node
    int nb0, nb1;              // blocks of the tail tile, of the tile after it
};

// Parent of node i as the tree has it (-1 past the last); the load, apart from its use.
__device__ __forceinline__ int tree_parent(const TreeArgs& A, const TreeItem& I, int i) {
    return i < I.n ? __ldg(A.parent + static_cast<long long>(I.b) * A.N + i) : -1;
}

// Fills the info of an item (one warp, nodes lane and lane + 32, whose parents are par0 and par1).
__device__ __noinline__ void tree_info(TreeInfo* S, const TreeArgs& A, const TreeItem I, int lane, int par0, int par1) {
    constexpr unsigned ALL = 0xffffffffu;
    int8_t* jump = reinterpret_cast<int8_t*>(S->list);   // list is filled last
    int par[2] = {par0, par1};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        if (par[u] < -1 || par[u] >= i) {
            atomicOr(A.err, ERR_BAD_TREE);
            par[u] = -1;
        }
        S->anc[i] = 1ull << i;
        jump[i] = static_cast<int8_t>(par[u]);
    }
    __syncwarp();
    for (int span = 1; span < I.n; span <<= 1) {   // pointer doubling
        u64 a[2];
        int8_t j[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = lane + 32 * u, p = jump[i];
            a[u] = S->anc[i] | (p >= 0 ? S->anc[p] : 0ull);
            j[u] = p >= 0 ? jump[p] : -1;
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            S->anc[lane + 32 * u] = a[u];
            jump[lane + 32 * u] = j[u];
        }
        __syncwarp();
    }
    u64 kid = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (par[u] >= 0) kid |= 1ull << par[u];
    kid = (static_cast<u64>(__reduce_or_sync(ALL, static_cast<unsigned>(kid >> 32))) << 32) |
          __reduce_or_sync(ALL, static_cast<unsigned>(kid));
    int pos[2];
    bool real[2], last[2], term[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        real[u] = i < I.n;
        pos[u] = I.c + __popcll(S->anc[i]) - 1;
        S->pos[i] = static_cast<uint8_t>(pos[u]);
        last[u] = real[u] && (pos[u] & 15) == 15;
        term[u] = real[u] && (last[u] || !((kid >> i) & 1));
    }
    auto mask = [&](const bool* f) { return (static_cast<u64>(__ballot_sync(ALL, f[1])) << 32) | __ballot_sync(ALL, f[0]); };
    const u64 terms = mask(term), ends = mask(last);
    const bool first[2] = {real[0] && pos[0] < T, real[1] && pos[1] < T};
    const u64 tile0 = mask(first);
    __syncwarp();
    // nodes below each of the lane's two (and themselves): the ancestors' bits, transposed by ballots
    // (a walk over 43 terminal nodes took 10000 cycles)
    const u64 anc[2] = {S->anc[lane], S->anc[lane + 32]};
    u64 below[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const unsigned lo = static_cast<unsigned>(anc[0] >> (32 * h)), hi = static_cast<unsigned>(anc[1] >> (32 * h));
#pragma unroll 2
        for (int i = 0; i < 32 && 32 * h + i < I.n; ++i) {
            const unsigned b0 = __ballot_sync(ALL, (lo >> i) & 1), b1 = __ballot_sync(ALL, (hi >> i) & 1);
            if (lane == i) below[h] = (static_cast<u64>(b1) << 32) | b0;
        }
    }
    // the block of a node: the lowest terminal node at or below it in its group
    int rep[2] = {0, 0};
    const int g0 = I.c >> 4, g1 = (I.c + I.n - 1) >> 4;   // groups that nodes can stand in
#pragma unroll 1
    for (int grp = g0; grp <= g1; ++grp) {
        const bool in[2] = {real[0] && (pos[0] >> 4) == grp, real[1] && (pos[1] >> 4) == grp};
        const u64 gm = mask(in) & terms;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (in[u]) rep[u] = __ffsll(static_cast<long long>(below[u] & gm)) - 1;
    }
    // the blocks this row tile's nodes run through
    u64 need = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        S->rep[i] = static_cast<uint8_t>(rep[u]);
        if (real[u] && i >= I.node0(A.NT) && i < I.node0(A.NT) + A.NT) need |= (1ull << rep[u]) | (anc[u] & ends);
    }
    need = (static_cast<u64>(__reduce_or_sync(ALL, static_cast<unsigned>(need >> 32))) << 32) |
           __reduce_or_sync(ALL, static_cast<unsigned>(need));
    int before = 0, nb0 = 0;
#pragma unroll 1
    for (int grp = g0; grp <= g1; ++grp) {
        const bool in[2] = {((need >> lane) & 1) && (pos[0] >> 4) == grp, ((need >> (lane + 32)) & 1) && (pos[1] >> 4) == grp};
        const u64 gm = mask(in);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (in[u]) {
                const int i = lane + 32 * u, x = before + __popcll(gm & ((1ull << i) - 1));
                S->idx[i] = static_cast<uint8_t>(x);
                S->list[x] = static_cast<uint8_t>(i);
            }
        before += __popcll(gm);
        if (grp < 4) nb0 = before;
    }
    if (lane == 0) {
        S->tile0 = tile0;
        S->ends = ends;
        S->vbad = 0;
        S->cbad = 0;
        S->nb0 = nb0;
        S->nb1 = before - nb0;
    }
}

// Page of position p of sequence b and the row inside it; an entry outside the pool is recorded and
// replaced by page 0.
__device__ __forceinline__ int tree_page(const KvPages& kv, int b, int p, int* row, unsigned* err) {
    if (!kv.table) {
        *row = p;
        return b;
    }
    const int j = p / kv.page;
    *row = p - j * kv.page;
    int pg = __ldg(kv.table + static_cast<long long>(b) * kv.max_pages + j);
    if (pg < 0 || pg >= kv.n_pages) {
        atomicOr(err, ERR_BAD_PAGE);
        pg = 0;
    }
    return pg;
}

// Whether a pair of bf16 values holds a non-finite one: an exponent field of all ones carries into
// the sign's place.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// Rare: non-finite values of a gathered block replaced by zeros, and whose they were noted.  A lane goes over the
// 16 bytes that it wrote of every `rows`-th row.
__device__ __noinline__ void gather_fix(TreeInfo* S, uint8_t* d, int quarter, int ch, int first, int rows, int who) {
    for (int r0 = 0; r0 < 16; r0 += rows) {
        const int r = r0 + first, s = quarter * 16 + r, w = __shfl_sync(0xffffffffu, who, r);
        uint32_t* e = reinterpret_cast<uint32_t*>(d + s * 128 + (((ch & 7) ^ (s & 7)) * 16));
        uint32_t any = 0;
        for (int k = 0; k < 4; ++k) {
            any |= non_finite(e[k]);
            if ((e[k] & 0x7F80u) == 0x7F80u) e[k] &= 0xFFFF0000u;
            if ((e[k] & 0x7F800000u) == 0x7F800000u) e[k] &= 0x0000FFFFu;
        }
        if (any) {
            if (w < 64) atomicOr(&S->vbad, 1ull << w);
            else atomicOr(&S->cbad, 1u << (w - 64));
        }
    }
}

// Gathers the V rows of block x (16 slots) into its quarter of a V stage, by one warp.  A lane finds
// the source row of slot lane % 16; a row is HD / 8 chunks of 16 bytes, all of a lane's loads in
// flight together; non-finite values are dropped and noted on the way.
template <int HD>
__device__ __noinline__ void gather_block(TreeInfo* S, const TreeArgs& A, const TreeItem I, uint8_t* dst, int x, int quarter, int lane) {
    constexpr int CH = HD / 8, ROWS = 32 / CH, U = 16 / ROWS;
    const int term = S->list[x], tp = S->pos[term], p = (tp & ~15) + (lane & 15);
    const uint16_t* src = nullptr;
    int who = 0;   // node, or 64 + position of a cache row in its group
    if (p < I.c) {
        int row;
        const long long z = static_cast<long long>(tree_page(A.kv, I.b, I.ctx - I.c + p, &row, A.err)) * A.Hkv + I.g;
        src = A.vc + (z * A.kv.page + row) * HD;
        who = 64 + (lane & 15);
    } else if (p <= tp) {
        u64 m = S->anc[term];   // the ancestor tp - p steps up: a path's nodes ascend
        for (int up = tp - p; up > 0; --up) m ^= 1ull << (63 - __clzll(static_cast<long long>(m)));
        who = 63 - __clzll(static_cast<long long>(m));
        src = A.src + (static_cast<long long>(I.b) * A.N + who) * A.src_stride + static_cast<long long>(A.Hkv + I.g) * HD;
    }
    __syncwarp();
    const int ch = lane % CH;
    uint8_t* d = dst + (ch >> 3) * (T * 128);
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const u64 q = __shfl_sync(0xffffffffu, reinterpret_cast<u64>(src), u * ROWS + lane / CH);
        v[u] = make_uint4(0, 0, 0, 0);
        if (q) v[u] = __ldg(reinterpret_cast<const uint4*>(q) + ch);
    }
    uint32_t bad = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int s = quarter * 16 + u * ROWS + lane / CH;
        bad |= non_finite(v[u].x) | non_finite(v[u].y) | non_finite(v[u].z) | non_finite(v[u].w);
        *reinterpret_cast<uint4*>(d + s * 128 + (((ch & 7) ^ (s & 7)) * 16)) = v[u];
    }
    if (__any_sync(0xffffffffu, bad)) gather_fix(S, d, quarter, ch, lane / CH, ROWS, who);
}

__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    tmem_ld_wait();
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float* s) {
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld16(taddr + c * 16, s + c * 16);
    tmem_ld_wait();
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
                 "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// MMA issue.  One thread issues an SM's MMAs, and what it computes for each one bounds the kernel as
// soon as a tile's MMAs are short: with both 64-bit descriptors put together from addresses per MMA
// it needed ~150 cycles each (20 a tile at hd 256), three times the tensor core's own time.  So a
// descriptor's constant upper half stays in the instruction and its lower half (the address / 16, and
// an MN-major operand's block stride) is one add away from a base formed once per tile, four K steps
// to an asm statement.
constexpr uint32_t DESC_HI = (1u << 30) | (1u << 14) | (1024u >> 4);   // 128-byte swizzle, version, 8-row groups 1024 bytes apart
// Arrival that hands over tensor memory and nothing else: after tc_fence_before it needs no release of
// its own, and a releasing one waits for the thread's stores to global memory (2400 cycles after the
// read-out of O at hd 128).
__device__ __forceinline__ void arrive_tc(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead = 16u) { return ((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16); }

// D (+)= A B^T over 64 K elements, A and B K-major in shared memory (K steps 32 bytes apart);
// acc: whether the first of them accumulates.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(DESC_HI)
        : "memory");
}
// One K step (16 positions), A in tensor memory (a row per lane, two K elements per column) or
// K-major in shared memory, B MN-major.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(DESC_HI)
        : "memory");
}
// The four K steps of a whole tile's P V: P's are 8 columns apart, V's 2048 bytes.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 b, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 b, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 b, {y, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(DESC_HI)
        : "memory");
}

// Two fp32 operations in one instruction, each rounded as the single one.
__device__ __forceinline__ void mul2(float& a, float& b, float x) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x));
}
__device__ __forceinline__ void add2(float& a, float& b, float x) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Largest of 64 scores (a maximum is exact in any order; NaN are passed over).
__device__ __forceinline__ float max32(const float* s) {
    float x[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
    for (int j = 0; j < 32; j += 2) x[(j / 2) & 3] = max3(x[(j / 2) & 3], s[j], s[j + 1]);
    return fmaxf(max3(x[0], x[1], x[2]), x[3]);
}
// The running maximum after a tile whose largest score is mx, and what O and l are rescaled by.
__device__ __forceinline__ float new_max(float m, float mx) { return (m == NEG_INF || mx > __fadd_rn(m, RESCALE_SLACK)) ? mx : m; }
__device__ __forceinline__ float alpha(float m, float mn) { return (mn == NEG_INF || mn == m) ? 1.f : ex2_approx(__fsub_rn(m, mn)); }
// p = exp2(s - m) of 32 scores: packs them as bf16 pairs and adds them to ts in order (the decode
// rows' operations; the p of a row that has seen no score yet are 0).
__device__ __forceinline__ void exp_half(float* s, float m, uint32_t* pk, float& ts) {
    if (m == NEG_INF) {   // rare: no score, or only NaN, so far
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = NEG_INF;
        m = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) add2(s[j], s[j + 1], -m);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        s[j] = ex2_approx(s[j]), s[j + 1] = ex2_approx(s[j + 1]);
        ts = __fadd_rn(__fadd_rn(ts, s[j]), s[j + 1]);
        pk[j / 2] = pack_bf16x2(s[j], s[j + 1]);
    }
}

// The rest of a bounded wait whose first test failed.
__device__ __noinline__ bool tree_wait(uint32_t bar, uint32_t par, unsigned* err, volatile int* abort) {
    if (*abort) return false;
    if (mbar_wait_sleep(bar, par, err)) return true;
    *abort = 1;
    return false;
}

// Rare: what the non-finite V values left out by the gather add to a row's partial output, p * v
// each (p is the row's bf16 weight: 0 * inf is a NaN as in the product).  Whole warps; op is the
// row's partial, null for rows that have none in this split.
struct TreeBad {
    u64 path, in0, vbad;
    unsigned cbad, cnz;
    float m0, m1;      // reference maxima of the tail tile and of the tile after it
    uint32_t scores;   // the row's tree scores in tensor memory
    bool use0, use1;   // which of the two tiles this split holds
    int b, g, ctx, c, hd, pitch;
    float* op;
};
__device__ __noinline__ void tree_add_bad(const TreeArgs& A, const TreeBad& F) {
    auto add = [&](const uint16_t* v, float p) {
        for (int k = 0; k < F.hd; ++k)
            if ((v[k] & 0x7F80) == 0x7F80) {
                float& o = F.op[(k >> 2) * F.pitch + (k & 3)];
                o = __fmaf_rn(p, bf16_to_f32(v[k]), o);
            }
    };
    for (u64 e = F.vbad; e; e &= e - 1) {
        const int i = __ffsll(static_cast<long long>(e)) - 1;
        __syncwarp();
        const float s = __fmul_rn(tmem_ld1(F.scores + i), A.sl2);
        const bool first = (F.in0 >> i) & 1;
        if (F.op && ((F.path >> i) & 1) && (first ? F.use0 : F.use1))
            add(A.src + (static_cast<long long>(F.b) * A.N + i) * A.src_stride + static_cast<long long>(A.Hkv + F.g) * F.hd,
                bf16_to_f32(f32_to_bf16(ex2_approx(__fsub_rn(s, first ? F.m0 : F.m1)))));
    }
    for (unsigned e = F.cbad; e; e &= e - 1) {
        const int i = __ffs(e) - 1;
        int row;
        const long long z = static_cast<long long>(tree_page(A.kv, F.b, F.ctx - F.c + (F.c & ~15) + i, &row, A.err)) * A.Hkv + F.g;
        if (F.op) add(A.vc + (z * A.kv.page + row) * F.hd, (F.cnz >> i) & 1 ? 1.f : 0.f);
    }
    __syncwarp();
}

// Whether a CTA of one item forms the output of its rows itself: up to DIRECT_MAX values (64 positions: 16 x 64
// values 6.4 us, with the combine 8.3; 64 x 128 12.2 and 12.8; 24 x 256 with a gate 10.4 and 10.6; 96 x 256 with a
// gate 26.3 and 17.6).
constexpr int DIRECT_MAX = 6144;
__host__ __device__ inline bool tree_direct(int rows, int hd) { return rows * hd <= DIRECT_MAX; }
// A value of the output: acc / L, with the gate's product where there is one.  At hd 64 and 256 the quotient
// is rounded to bf16 before that product, as the decode rows round it; they take no hd 128, so there the
// product is rounded alone.
__device__ __forceinline__ uint16_t tree_out(float acc, float L, const uint16_t* gate, int hd) {
    float y = __fdiv_rn(acc, L);
    if (gate) y = __fmul_rn(hd == 128 ? y : bf16_to_f32(f32_to_bf16(y)), __frcp_rn(__fadd_rn(1.f, expf(-bf16_to_f32(*gate)))));
    return f32_to_bf16(y);
}

template <int HD, bool MULTI>
__global__ void __launch_bounds__(TREE_THREADS, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmT,
                     const __grid_constant__ TreeArgs A) {
    using S = TreeShape<HD>;
    constexpr int CB = S::CB, SK = S::SK, SV = S::SV, TILE_BYTES = S::TILE_BYTES, BLK = S::BLK, QBLK = S::QBLK;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    TreeInfo& info = *reinterpret_cast<TreeInfo*>(smem + S::INFO_OFF);
    float* m_sm = reinterpret_cast<float*>(smem + S::M_OFF);         // running maximum after the last tile
    float* sum_sm = reinterpret_cast<float*>(smem + S::SUM_OFF);     // [2][128] sums of the odd tiles
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::INFO_OFF + sizeof(TreeInfo));
    volatile int& s_abort = *reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t sQ = base;
    auto sK = [&](int st) { return base + S::K_OFF + st * TILE_BYTES; };
    auto sV = [&](int st) { return base + S::V_OFF + st * TILE_BYTES; };
    const uint32_t bar0 = base + S::BAR_OFF;
    auto fullK = [&](int st) { return bar0 + 8u * st; };
    auto emptyK = [&](int st) { return bar0 + 8u * (SK + st); };
    auto fullV = [&](int st) { return bar0 + 8u * (2 * SK + st); };
    auto emptyV = [&](int st) { return bar0 + 8u * (2 * SK + SV + st); };
    const uint32_t bx = bar0 + 8u * (2 * SK + 2 * SV);
    // by the softmax group j of a cache tile: i & 1 for an item's i-th whole tile, 0 for its tail tile
    auto sbar = [&](int j) { return bx + 8u * j; };           // S[j] written
    auto sfree = [&](int j) { return bx + 8u * (2 + j); };    // S[j] read
    auto pready = [&](int j) { return bx + 8u * (4 + j); };   // P[j] written (and O rescaled)
    // the P V step of group j's tile n has completed: two barriers per group, as a wait may come while
    // the tile before is still on its way
    auto pfree = [&](int j, int n) { return bx + 8u * (j ? 25 + (n & 1) : (n & 1) ? 6 : 7); };
    auto mpub = [&](int j) { return bx + 8u * (8 + j); };     // the running maximum after the tile is known (to the next tile's group)
    // by the parity of a block step's number
    auto bready = [&](int j) { return bx + 8u * (10 + j); };
    auto bfree = [&](int j) { return bx + 8u * (12 + j); };
    // once per tail item: the tree's scores written; all that it holds (scores, info) read; its info
    // filled and its V tiles requested (every stage's last use but one is then complete, so the
    // gather's waits on the stages are never two phases behind); its blocks gathered
    const uint32_t tbar = bx + 8u * 14, tfree = bx + 8u * 15, tready = bx + 8u * 16, vdone = bx + 8u * 17;
    const uint32_t qfull = bx + 8u * 19, qdone = bx + 8u * 20, done = bx + 8u * 22;
    auto ofree = [&](int j) { return bx + 8u * (j ? 18 : 21); };   // by O buffer: read out
    // by the parity of group 1's tile: its sum is in shared memory.  Two of them, as group 1 may end its
    // next tile before group 0 comes to take this one's sum.
    auto spub = [&](int j) { return bx + 8u * (23 + j); };
    const uint32_t done2 = bx + 8u * 27;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // one CTA per item: the block (row tile, kv head and sequence, split), splits slowest; persistent
    // CTAs: a contiguous range numbered split-fastest (consecutive items mostly share Q)
    int it0 = 0, it1 = 1, only_rt = -1;
    // barrier i of the list above; the stages' barriers come first
    if (tid < S::N_BARS && base - raw <= S::SLACK) {
        const int j = tid - (2 * SK + 2 * SV);
        // arrivals: 1 where a thread or the hardware arrives; a softmax group's 128 on sfree, pready,
        // mpub, bready, spub and ofree
        constexpr u64 BY_GROUP = 0x1A40F3Cull;
        int count = 1;
        if (j < 0) count = tid >= 2 * SK && tid < 2 * SK + SV ? 5 : 1;   // fullV: the gather's warps and V's
        else if ((BY_GROUP >> j) & 1) count = 128;
        else if (j == 15) count = 128 + 1 + 4;   // tfree: group 0, P V, group 1's warps
        else if (j == 17) count = 4;                 // vdone: group 1's warps
        mbar_init(bar0 + 8u * tid, count);
        fence_mbar_init();
    }
    if (tid == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmT);
        if (base - raw <= S::SLACK) s_abort = 0;
    }
    griddep_wait();
    int first = 0;
    TreeItem I0;
    if constexpr (MULTI) {
        tree_share(A, reinterpret_cast<long long*>(&info), &it0, &it1, &only_rt);
        I0.live = false;
        for (first = it0; first < it1; ++first) {
            I0 = tree_item(A, first, only_rt);
            if (I0.live) break;
        }
    } else {
        I0 = tree_item_at(A, blockIdx.y / A.Hkv, blockIdx.y % A.Hkv, blockIdx.x, blockIdx.z);
        first = I0.live ? 0 : 1;
        if (tid == 0 && I0.g == 0 && I0.rt == 0 && I0.split == 0) tree_report(A, I0.b);
    }
    if (first >= it1 || base - raw > S::SLACK) {
        if (first < it1 && tid == 0) atomicOr(A.err, ERR_WAIT_TIMEOUT);   // an unaligned base: see SLACK
        griddep_launch();
        return;   // no tensor memory was set up
    }
    // the next item, in the roles' loops; within a row tile without the call, whose divisions and loads
    // took 2500 cycles in a role's way
    auto next = [&](int it, TreeItem& I) {
        if (!MULTI || it >= it1) return;
        if (++I.split < A.nsplit) tree_item_split(I, A.NT);
        else I = tree_item(A, it, only_rt);
    };
    int par0 = -1, par1 = -1;   // a single item's parents, on their way meanwhile
    if (!MULTI && warp == 9) {
        par0 = tree_parent(A, I0, lane);
        par1 = tree_parent(A, I0, lane + 32);
    }
    if (warp == 10) {
        tmem_alloc(smem_u32(tmem_slot), S::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // one split per row and few rows: the partials stay in shared memory, where the K and V rings were,
    // and the whole CTA forms the output from them, without the combine's launch
    const bool direct = !MULTI && A.nsplit == 1 && tree_direct(A.NT * A.G, HD);
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tO0 = tmem + 128, tT = tO0 + S::NO * HD, tP = tT + 64;

    // bounded waits; after the first one that gives up, every later one that would have to wait returns at once
    auto W = [&](uint32_t bar, uint32_t par) -> bool { return mbar_try_wait(bar, par) || tree_wait(bar, par, A.err, &s_abort); };
    // two barriers tested side by side
    auto W2 = [&](uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) -> bool {
        const bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1);
        return (r0 || tree_wait(b0, p0, A.err, &s_abort)) && (r1 || tree_wait(b1, p1, A.err, &s_abort));
    };
    // a wait for one's own copies or MMAs before leaving: also after an abort
    auto drain = [&](uint32_t bar, uint32_t par) {
        int none = 0;
        if (!mbar_try_wait(bar, par)) tree_wait(bar, par, A.err, &none);
    };
    auto WW = [&](uint32_t bar, uint32_t par) -> bool { return __all_sync(0xffffffffu, W(bar, par)); };
    auto same_q = [](const TreeItem& x, int b, int g, int rt) { return x.b == b && x.g == g && x.rt == rt; };

    if (warp == 8) {
        // ---- K tiles of the cache, then the tree's
        if (lane == 0) {
            int t = 0;
            bool ok = true;
            TreeItem I = I0;
            for (int it = first; ok && it < it1; next(++it, I)) {
                if (!I.live) continue;
                const int nreg = I.kreg(), nk = nreg + (I.tail() ? 1 : 0);
                for (int i = 0; i < nk; ++i) {
                    const int st = t % SK;
                    if (t >= SK && !W(emptyK(st), ((t / SK) & 1u) ^ 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(fullK(st), TILE_BYTES);
                    if (i < nreg) {
                        int row;
                        const int z = tree_page(A.kv, I.b, I.p_begin + i * T, &row, A.err) * A.Hkv + I.g;
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb) tma_load_3d(sK(st) + cb * BLK, &tmK, cb * 64, row, z, fullK(st));
                    } else {
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb) tma_load_2d(sK(st) + cb * BLK, &tmT, I.g * HD + cb * 64, I.b * A.N, fullK(st));
                    }
                    ++t;
                }
            }
            for (int j = t > SK ? t - SK : 0; j < t; ++j) drain(fullK(j % SK), (j / SK) & 1u);
        }
    } else if (warp == 9) {
        // ---- V tiles of the cache (a tail's block steps are group 1's), then what there is to know of
        // a tail item's tree
        int t = 0, nt = 0;
        unsigned mine = 0;   // bit j: use t - 1 - j of the ring was a copy of this warp's
        bool ok = true;
        TreeItem I = I0;
        for (int it = first; ok && it < it1; next(++it, I)) {
            if (!I.live) continue;
            if (lane == 0) {
                const int nv = I.vreg();
                for (int i = 0; i < nv; ++i, ++t) {
                    const int st = t % SV;
                    if (t >= SV && !W(emptyV(st), ((t / SV) & 1u) ^ 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(fullV(st), TILE_BYTES);
                    for (int k = 0; k < 4; ++k) mbar_arrive(fullV(st));   // a gathered stage's other arrivals
                    int row;
                    const int z = tree_page(A.kv, I.b, I.p_begin + i * T, &row, A.err) * A.Hkv + I.g;
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) tma_load_3d(sV(st) + cb * BLK, &tmV, cb * 64, row, z, fullV(st));
                    mine = mine << 1 | 1u;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok || !I.tail()) continue;
            if (MULTI) {
                par0 = tree_parent(A, I, lane);
                par1 = tree_parent(A, I, lane + 32);
            }
            if (nt > 0 && !WW(tfree, (nt - 1) & 1u)) break;
            ++nt;
            tree_info(&info, A, I, lane, par0, par1);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(tready);
                int steps = (I.tail0 ? (info.nb0 + 3) / 4 : 0) + (I.tail1 ? (info.nb1 + 3) / 4 : 0);
                for (; ok && steps > 0; --steps) {
                    ok = t < SV || W(emptyV(t % SV), ((t / SV) & 1u) ^ 1u);
                    if (!ok) break;
                    mbar_arrive(fullV(t % SV));   // the fifth arrival keeps this warp in step with the ring
                    mine <<= 1;
                    ++t;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // every issued copy lands before the CTA may leave
        if (lane == 0)
            for (int j = 1; j <= SV && j <= t; ++j)
                if ((mine >> (j - 1)) & 1) drain(fullV((t - j) % SV), ((t - j) / SV) & 1u);
    } else if (warp == 10) {
        // ---- Q of every item whose (sequence, kv head, row tile) differs from the one before, and Q K^T,
        // as far ahead as the two score buffers allow.  It and P V are issued by a warp each:
        // a tile's barrier tests and commits take an issuer ~1000 cycles beside the ~1000 of its MMAs,
        // and with one issuer for both the tensor core stood idle meanwhile.
        if (lane == 0) {
            constexpr uint32_t IDS = idesc_bf16_f32(128, T);
            int st = 0, n0 = 0, n1 = 0, nt = 0, nq = 0, qb = -1, qg = -1, qrt = -1;
            uint32_t ph = 0;
            bool ok = true;
            TreeItem I = I0;
            for (int it = first; ok && it < it1; next(++it, I)) {
                if (!I.live) continue;
                if (!same_q(I, qb, qg, qrt)) {
                    if (nq > 0) {
                        tc_commit(qdone);
                        if (!W(qdone, (nq - 1) & 1u)) break;
                    }
                    mbar_arrive_expect_tx(qfull, CB * A.NT * A.G * 128);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) tma_load_3d(sQ + cb * QBLK, &tmQ, cb * 64, I.g * A.G, I.b * A.N + I.rt * A.NT, qfull);
                    if (!W(qfull, nq++ & 1u)) break;
                    qb = I.b, qg = I.g, qrt = I.rt;
                }
                const int nreg = I.kreg(), nqk = nreg + (I.tail() ? 1 : 0);
#pragma unroll 1
                for (int i = 0; i < nqk; ++i) {
                    uint32_t d, ready;
                    if (i >= nreg) {   // the tree's scores
                        ok = W(fullK(st), ph) && (nt == 0 || W(tfree, (nt - 1) & 1u));
                        ++nt;
                        d = tT;
                        ready = tbar;
                    } else {
                        const uint32_t odd = i < I.nfull ? i & 1 : 0;
                        const uint32_t n = odd ? n1++ : n0++;
                        ok = n == 0 ? W(fullK(st), ph) : W2(fullK(st), ph, sfree(odd), (n - 1) & 1u);
                        d = tS + odd * T;
                        ready = sbar(odd);
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t q = desc_lo(sQ), k = desc_lo(sK(st));
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) mma4_ss(d, q + cb * (QBLK / 16), k + cb * (BLK / 16), IDS, cb > 0 ? 1u : 0u);
                    tc_commit(ready);
                    // at hd 256 the tree's stage goes on as the block steps' P and is freed by their end
                    if (!S::PB_IN_K || i < nreg) tc_commit(emptyK(st));
                    if (++st == SK) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // only now: the combine's CTAs, launched as the first SMs fall idle, would all crowd onto those
            // (16 nodes at 131072 positions: 131 us, so 111)
            griddep_launch();
            if (nq > 0) drain(qfull, (nq - 1) & 1u);   // every issued copy lands before the CTA may leave
            tc_commit(done);   // every MMA issued is complete before the CTA may leave
            drain(done, 0u);
        }
    } else if (warp == 11) {
        // ---- P V
        if (lane == 0) {
            constexpr uint32_t IDO = idesc_bf16_f32(128, HD, true);
            constexpr uint32_t VBLK = CB > 1 ? BLK : 1024;   // as in attn.cu: unused with a single block
            // tk: K tiles; np_g: steps of group g's tiles; bs: block steps; v: V tiles; nitem: items with a step
            int tk = 0, np_0 = 0, np_1 = 0, bs = 0, v = 0, nt = 0, nitem = 0;
            bool ok = true;
            TreeItem I = I0;
            for (int it = first; ok && it < it1; next(++it, I)) {
                if (!I.live) continue;
                const int nreg = I.kreg();
                bool first_pv = true;
                const int ob = nitem % S::NO;
                const uint32_t tO = tO0 + ob * HD;
                // an item's first step overwrites its O buffer: the epilogue before has read it
                auto begin_pv = [&]() -> bool { return !first_pv || nitem < S::NO || W(ofree(ob), (nitem / S::NO - 1) & 1u); };
#pragma unroll 1
                for (int i = 0; i < nreg; ++i) {
                    const bool odd = i < I.nfull && (i & 1);
                    const int ksteps = i < I.nfull ? 4 : I.c / 16, sv = v % SV, n = odd ? np_1++ : np_0++;
                    ok = begin_pv() && (ksteps == 0 ? W(pready(odd), n & 1u) : W2(pready(odd), n & 1u, fullV(sv), (v / SV) & 1u));
                    if (!ok) break;
                    if (ksteps > 0) {
                        tc_fence_after();
                        const uint32_t b = desc_lo(sV(sv), VBLK), p = tP + (odd ? 32 : 0);
                        if (ksteps == 4) {
                            mma4_ts(tO, p, b, IDO, first_pv ? 0u : 1u);
                        } else {
#pragma unroll 1
                            for (int kk = 0; kk < ksteps; ++kk) mma_ts(tO, p + kk * 8, b + kk * 128, IDO, !first_pv || kk > 0 ? 1u : 0u);
                        }
                        first_pv = false;
                    }
                    tc_commit(pfree(odd, n));
                    if (ksteps > 0) {
                        tc_commit(emptyV(sv));
                        ++v;
                    }
                }
                tk += nreg;
                if (ok && I.tail()) {
                    if (!W(tready, nt & 1u)) break;
                    const int nb0 = I.tail0 ? info.nb0 : 0, nb1 = I.tail1 ? info.nb1 : 0;
                    mbar_arrive(tfree);   // the info is not read here any more
                    ++nt;
                    const uint32_t sPB = S::PB_IN_K ? sK(tk % SK) : base + S::PB_OFF;   // the tree's K stage
                    ++tk;
#pragma unroll 1
                    for (int x = 0, left = nb0; ok && (left > 0 || x < 1); ) {
                        if (left <= 0) {   // the tile after the tail
                            ++x;
                            left = nb1;
                            continue;
                        }
                        const int sv = v % SV, nblk = min(4, left);
                        ok = begin_pv() && W(bready(bs & 1), (bs >> 1) & 1u) && W(fullV(sv), (v / SV) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a = desc_lo(sPB + (bs & 1) * QBLK), b = desc_lo(sV(sv), VBLK);
#pragma unroll 1
                        for (int kk = 0; kk < nblk; ++kk) mma_ss(tO, a + kk * 2, b + kk * 128, IDO, !first_pv || kk > 0 ? 1u : 0u);
                        first_pv = false;
                        tc_commit(bfree(bs & 1));
                        tc_commit(emptyV(sv));
                        ++v;
                        ++bs;
                        left -= 4;
                    }
                }
                if (!first_pv) ++nitem;
            }
            tc_commit(done2);
            drain(done2, 0u);
        }
    } else {
        // ---- softmax: thread = row rho of the tile (node rho / G, q head rho % G).  Group 0 (warps
        // 0-3) takes an item's even tiles, group 1 the odd ones: while one exponentiates, the other
        // loads and takes its maximum.  The running maximum is handed from tile to tile as soon as it
        // is known; group 0 keeps l, adding an odd tile's sum when it comes to its own next tile.
        const int grp = warp >> 2, rho = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int nl = rho / A.G, gh = rho - nl * A.G;
        // n: own tiles; n1 (group 0): tiles of group 1 taken; n0 (group 1): tiles of group 0 in the
        // items before; npub (group 1): maxima taken from group 0; tv (group 1): V tiles and block steps;
        // nitem: items with a P V step
        int n = 0, n1 = 0, n0 = 0, npub = 0, bs = 0, nt = 0, tk = 0, tv = 0, nitem = 0;
        uint32_t tO = tO0;
        int pitch = 0;   // floats between a row's pieces of four columns in the partials
        bool ok = true;
        // O (once a P V step of the item has been issued; `bar` completes with its last) times al
        auto rescale = [&](float al, bool any_pv, uint32_t bar, uint32_t par) -> bool {
            if (!any_pv || !__any_sync(0xffffffffu, al != 1.f)) return true;
            if (!WW(bar, par)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD / 64; ++c) {
                float o[64];
                tmem_ld64(tO + lane_off + c * 64, o);
#pragma unroll
                for (int e = 0; e < 64; e += 2) mul2(o[e], o[e + 1], al);
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) tmem_st16(tO + lane_off + c * 64 + q4 * 16, o + q4 * 16);
            }
            tmem_st_wait();
            return true;
        };
        // O of an item to its rows' partials (null: a row without one), once its last P V step has
        // completed.  The partials hold four columns of a tile's rows side by side, so a lane writes its
        // own row and a warp whole 128-byte lines (with [row][HD] partials, rows transposed by shuffles,
        // the 128 columns of a warp took 4700 cycles).
        auto store_o = [&](float* op) {
            if (__any_sync(0xffffffffu, op != nullptr)) {
#pragma unroll 1
                for (int c = 0; c < HD / 64; ++c) {
                    float o[64];
                    tmem_ld64(tO + lane_off + c * 64, o);
                    if (op)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            *reinterpret_cast<float4*>(op + (c * 16 + j) * pitch) = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            }
            tc_fence_before();
        };
        TreeItem I = I0;
        for (int it = first; ok && it < it1; next(++it, I)) {
            if (!I.live) continue;
            const int node = I.node0(A.NT) + nl;
            const bool valid = nl < A.NT && node < I.n;
            const long long brow = static_cast<long long>(I.b) * A.N + node, idx = (brow * A.Hq + I.g * A.G + gh) * A.nsplit + I.split;
            const int tile0 = I.rt * A.NT, tile_rows = min(A.NT, A.N - tile0) * A.G;
            float* const part = direct ? reinterpret_cast<float*>(smem + S::K_OFF) + rho * 4 : A.opart + (((static_cast<long long>(I.b) * A.Hkv + I.g) * A.nsplit + I.split) * A.N + tile0) * A.G * HD + rho * 4;
            pitch = tile_rows * 4;
            tO = tO0 + nitem % S::NO * HD;
            float m = NEG_INF, l = 0.f;
            // group 0: the maximum and, when its own exponentials are done, the sum of the odd tile
            // before its next one or the item's end
            float al_odd = 1.f;
            auto take_max = [&]() -> bool {
                if (!WW(mpub(1), n1 & 1u)) return false;
                const float mo = m_sm[rho];
                al_odd = alpha(m, mo);
                m = mo;
                return true;
            };
            auto take_sum = [&]() -> bool {
                if (!WW(spub(n1 & 1), (n1 >> 1) & 1u)) return false;
                l = __fadd_rn(__fmul_rn(l, al_odd), sum_sm[(n1 & 1) * 128 + rho]);
                ++n1;
                return true;
            };
#pragma unroll 1
            for (int i = grp; i < I.nfull; i += 2) {
                if (!WW(sbar(grp), n & 1u)) { ok = false; break; }
                tc_fence_after();
                float mx = NEG_INF;
#pragma unroll
                for (int h = 0; h < T; h += 32) {   // its maximum
                    float s[32];
                    tmem_ld16(tS + lane_off + grp * T + h, s);
                    tmem_ld16(tS + lane_off + grp * T + h + 16, s + 16);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mul2(s[j], s[j + 1], A.sl2);
                    mx = fmaxf(mx, max32(s));
                }
                if (grp == 0) {
                    if (i > 0 && !take_max()) { ok = false; break; }
                } else {
                    if (!WW(mpub(0), npub & 1u)) { ok = false; break; }
                    ++npub;
                    m = m_sm[rho];
                }
                const float mn = new_max(m, mx);
                // a row that is no node's holds whatever its Q was: it must not have O rescaled for it
                const float al = valid ? alpha(m, mn) : 1.f;
                m = mn;
                if (grp == 1 || i + 1 < I.nfull) {   // someone takes it
                    m_sm[rho] = mn;
                    mbar_arrive(mpub(grp));
                }
                float sum = 0.f;
                if (n > 0 && !WW(pfree(grp, n - 1), ((n - 1) >> 1) & 1u)) { ok = false; break; }
                tc_fence_after();
                // the scores again, in two turns of one loop: unrolled it is twice the code and registers, and
                // warps that wait for instructions were a fifth of the stalls (64 nodes at 131072 positions
                // 309 us unrolled, 279 so; 32 x 13 nodes at 4000 to 8000: 199, 181)
#pragma unroll 1
                for (int h = 0; h < T; h += 32) {
                    float s[32];
                    uint32_t pk[16];
                    tmem_ld16(tS + lane_off + grp * T + h, s);
                    tmem_ld16(tS + lane_off + grp * T + h + 16, s + 16);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mul2(s[j], s[j + 1], A.sl2);
                    exp_half(s, mn, pk, sum);
                    tmem_st16u(tP + grp * 32 + h / 2 + lane_off, pk);
                }
                tc_fence_before();
                arrive_tc(sfree(grp));
                if (grp == 0) {
                    if (i > 0 && !take_sum()) { ok = false; break; }
                    l = __fadd_rn(__fmul_rn(l, al), sum);
                } else {
                    sum_sm[(n & 1) * 128 + rho] = sum;
                    mbar_arrive(spub(n & 1));
                }
                // the P V step before is the other group's
                const int before = grp ? n0 + i / 2 : n1 - 1;
                if (!rescale(al, i > 0, pfree(1 - grp, before), (before >> 1) & 1u)) { ok = false; break; }
                tmem_st_wait();
                tc_fence_before();
                arrive_tc(pready(grp));
                ++n;
            }
            if (!ok) break;
            if (grp == 1) {
                // tails' softmax and epilogues are group 0's; here the V rows of the block steps, a
                // block per warp
                n0 += (I.nfull + 1) / 2 + (I.tail0 && I.c > 0 ? 1 : 0);
                tv += I.vreg();
                if (!I.tail()) {
                    // a split below ctx: whole tiles, an even number, the last one this group's.  Its O
                    // is read out here while group 0 begins the next item.
                    if (!WW(pfree(1, n - 1), ((n - 1) >> 1) & 1u)) break;
                    tc_fence_after();
                    store_o(valid ? part : nullptr);
                    arrive_tc(ofree(nitem % S::NO));
                    ++nitem;
                    continue;
                }
                if (!WW(tready, nt & 1u)) break;
                ++nt;
                if (I.nfull > 0 || I.tail0 || info.nb1 > 0) ++nitem;   // a tail tile always has a block
#pragma unroll 1
                for (int half = 0; ok && half < 2; ++half) {
                    if (half ? !I.tail1 : !I.tail0) continue;
                    const int nb0 = info.nb0, x1 = half ? nb0 + info.nb1 : nb0;
#pragma unroll 1
                    for (int x0 = half ? nb0 : 0; x0 < x1; x0 += 4, ++tv) {
                        const int st = tv % SV, x = x0 + (warp & 3);
                        if (tv >= SV && !WW(emptyV(st), ((tv / SV) & 1u) ^ 1u)) { ok = false; break; }
                        if (x < x1) gather_block<HD>(&info, A, I, smem + (sV(st) - base), x, warp & 3, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(fullV(st));
                    }
                }
                __syncwarp();
                if (ok && lane == 0) {
                    mbar_arrive(vdone);
                    mbar_arrive(tfree);
                }
                continue;
            }
            const bool last_odd = I.nfull > 0 && !(I.nfull & 1);
            if (last_odd && (!take_max() || !take_sum())) break;
            if (!I.tail()) {   // the rest is group 1's
                if (valid) A.ml[idx] = make_float2(m, l);
                ++nitem;
                tk += I.kreg();
                continue;
            }
            // completes with the last P V step of the item's whole tiles
            const int last = (last_odd ? n1 : n) - 1;
            const uint32_t last_bar = pfree(last_odd, last), last_par = (last >> 1) & 1u;
            const int tail_st = (tk + I.kreg()) % SK;   // K stage of the tree's tile
            tk += I.kreg() + 1;
            uint8_t* prow = smem + (S::PB_IN_K ? S::K_OFF + tail_st * TILE_BYTES : S::PB_OFF) + rho * 128;
            bool any_pv = I.nfull > 0, any_block = false;
            u64 path = 0, in0 = 0;
            float m0 = NEG_INF;      // the reference max of the tail tile (the rare epilogue's)
            unsigned cnz = 0;        // cache positions of the first block group whose p is not 0
            int npos = 0;            // position of the node, relative to the tail tile
            if (!WW(tready, nt & 1u) || !WW(tbar, nt & 1u)) break;
            tc_fence_after();
            path = valid ? info.anc[node] : 0;
            npos = valid ? info.pos[node] : 0;
            in0 = info.tile0;
            // block of the path in each of the 8 groups of the two tiles (255: none)
            uint32_t blk[2] = {~0u, ~0u};
            auto set_blk = [&](int g16, int x) {
                const int sh = 8 * (g16 & 3);
                if (g16 < 4) blk[0] = (blk[0] & ~(255u << sh)) | (static_cast<uint32_t>(x) << sh);
                else blk[1] = (blk[1] & ~(255u << sh)) | (static_cast<uint32_t>(x) << sh);
            };
            if (valid) {
                for (u64 e = path & info.ends; e; e &= e - 1) {
                    const int a = __ffsll(static_cast<long long>(e)) - 1;
                    set_blk(info.pos[a] >> 4, info.idx[a]);
                }
                set_blk(npos >> 4, info.idx[info.rep[node]]);
            }
            __syncwarp();
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (half ? !I.tail1 : !I.tail0) continue;
                const u64 mine = half ? path & ~in0 : path & in0;
                const bool has_a = !half && I.c > 0;
                const u64 a_mask = has_a && valid ? (1ull << I.c) - 1 : 0ull;
                // scores 16 r .. 16 r + 15 of the cache's part of the tile (r < 4) or of the tree
                // (r - 4), -inf where this row does not look; 16 at a time in rolled loops, as
                // this code runs once per item
                float s[16];
                auto load16 = [&](int r) {
                    tmem_ld16((r < 4 ? tS : tT - 64) + lane_off + 16 * r, s);
                    tmem_ld_wait();
                    const unsigned in = static_cast<unsigned>((r < 4 ? a_mask >> (16 * r) : mine >> (16 * r - 64))) & 0xFFFFu;
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = (in >> j) & 1 ? __fmul_rn(s[j], A.sl2) : NEG_INF;
                };
                float mx = NEG_INF, sum = 0.f;
                if (has_a) {
                    if (!WW(sbar(0), n & 1u)) { ok = false; break; }
                    tc_fence_after();
                }
                // the parts that hold a cache position or a node
                const int r0 = has_a ? 0 : 4, ra = (I.c + 15) / 16, r1 = 4 + (I.n + 15) / 16;
#pragma unroll 1
                for (int r = r0; r < r1; r = r + 1 == ra ? 4 : r + 1) {
                    load16(r);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) mx = max3(mx, s[j], s[j + 1]);
                }
                const float mn = new_max(m, mx), al = alpha(m, mn);
                const bool dead = mn == NEG_INF;
                // the last P V step so far: a block step of the tail tile, or a cache tile's
                if (!(any_block ? rescale(al, true, bfree((bs - 1) & 1), ((bs - 1) >> 1) & 1u)
                                : rescale(al, any_pv, last_bar, last_par))) {
                    ok = false;
                    break;
                }
                // p of 16 scores as bf16 pairs (0 where no score has been seen at all)
                uint32_t pk[8];
                auto exp16 = [&](float& ts) {
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float a0 = dead ? 0.f : ex2_approx(__fsub_rn(s[j], mn)), a1 = dead ? 0.f : ex2_approx(__fsub_rn(s[j + 1], mn));
                        ts = __fadd_rn(__fadd_rn(ts, a0), a1);
                        pk[j / 2] = pack_bf16x2(a0, a1);
                    }
                };
                // the first group's cache positions, in whose block p stands before the nodes'
                uint32_t sh[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                const int gs = half ? -1 : I.c >> 4;
                if (has_a) {
                    if (n > 0 && !WW(pfree(0, n - 1), ((n - 1) >> 1) & 1u)) { ok = false; break; }
                    tc_fence_after();
                }
#pragma unroll 1
                for (int r = r0; r < r1; r = r + 1 == ra ? 4 : r + 1) {
                    load16(r);
                    exp16(sum);
                    if (r < 4) {
                        tmem_st8(tP + lane_off + 8 * r, pk);   // its first c / 16 K steps are used
                        if (r == gs) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                sh[e] = pk[e];
                                cnz |= ((pk[e] & 0x7FFFu) ? 1u << (2 * e) : 0u) | ((pk[e] & 0x7FFF0000u) ? 2u << (2 * e) : 0u);
                            }
                        }
                    }
                }
                if (has_a) {
                    tmem_st_wait();
                    tc_fence_before();
                    arrive_tc(sfree(0));
                    mbar_arrive(pready(0));
                    ++n;
                }
                l = __fadd_rn(__fmul_rn(l, al), sum);
                m = mn;
                if (!half) m0 = mn;
                const int nb = half ? info.nb1 : info.nb0, xb = half ? info.nb0 : 0;
                const uint32_t bl = blk[half];
#pragma unroll 1
                for (int x0 = 0; x0 < nb; x0 += 4, ++bs) {
                    if (bs >= 2 && !WW(bfree(bs & 1), ((bs - 2) >> 1) & 1u)) { ok = false; break; }
                    uint8_t* pr = prow + (bs & 1) * QBLK;
                    // per group of the tile a byte: where the row's block begins in its swizzled row
                    // of 128 bytes, 255 if the block is none of the step's four
                    uint32_t at = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const unsigned b8 = (bl >> (8 * q)) & 255u, x = b8 - xb;
                        at |= (b8 != 255u && (x >> 2) == static_cast<unsigned>(x0) >> 2 ? (((x & 3u) * 2u) ^ (rho & 7u)) * 16u : 255u) << (8 * q);
                    }
                    const bool here = at != ~0u;
#pragma unroll
                    for (int c = 0; c < T / 8; ++c) *reinterpret_cast<uint4*>(pr + c * 16) = make_uint4(0, 0, 0, 0);
                    if (gs >= 0) {
                        const unsigned o = (at >> (8 * gs)) & 255u;
                        if (o != 255u) {
                            *reinterpret_cast<uint4*>(pr + o) = make_uint4(sh[0], sh[1], sh[2], sh[3]);
                            *reinterpret_cast<uint4*>(pr + (o ^ 16u)) = make_uint4(sh[4], sh[5], sh[6], sh[7]);
                        }
                    }
                    if (__any_sync(0xffffffffu, here)) {
                        float unused = 0.f;
#pragma unroll 1
                        for (int r = 4; 16 * (r - 4) < I.n; ++r) {   // the tree's p again, to their slots
                            const unsigned in = here ? static_cast<unsigned>(mine >> (16 * r - 64)) & 0xFFFFu : 0u;
                            if (!__any_sync(0xffffffffu, in)) continue;
                            load16(r);
                            exp16(unused);
                            const uint4 ps = *reinterpret_cast<const uint4*>(info.pos + 16 * (r - 4));
                            const uint32_t pw[4] = {ps.x, ps.y, ps.z, ps.w};
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                if (j == 8 && 16 * (r - 4) + 8 >= I.n) break;
                                // node 16 (r - 4) + j at position p: byte 2 (p % 16) of the block of group p / 16 % 4
                                const uint32_t p = pw[j / 4] >> (8 * (j & 3));
                                const unsigned o = (at >> ((p >> 1) & 24u)) & 255u;
                                if (((in >> j) & 1) && o != 255u)
                                    *reinterpret_cast<uint16_t*>(pr + (o ^ ((p & 15u) * 2u))) =
                                        static_cast<uint16_t>(j & 1 ? pk[j / 2] >> 16 : pk[j / 2]);
                            }
                            __syncwarp();
                        }
                    }
                    __syncwarp();
                    fence_proxy_async_smem();
                    tc_fence_before();
                    mbar_arrive(bready(bs & 1));
                    any_block = true;
                }
                if (!ok) break;
            }
            if (!ok || !WW(vdone, nt & 1u)) break;
            // ---- epilogue: m, l and O of the rows that reach into this split
            const bool live = valid && I.ctx - I.c + npos >= I.p_begin;
            if (I.tail0 && valid && I.g == 0 && gh == 0) A.nsp[brow] = attn_split_count(I.ctx - I.c + npos + 1);
            if (any_pv || any_block) {
                if (!(any_block ? WW(bfree((bs - 1) & 1), ((bs - 1) >> 1) & 1u) : WW(last_bar, last_par))) break;
                tc_fence_after();
                const u64 vbad = info.vbad;
                const unsigned cbad = info.cbad;
                store_o(live ? part : nullptr);
                if (vbad || cbad) {
                    const TreeBad F{path, in0, vbad, cbad, cnz, m0, m, tT + lane_off, I.tail0, I.tail1, I.b, I.g, I.ctx, I.c, HD, pitch,
                                    live ? part : nullptr};
                    tree_add_bad(A, F);
                }
                if (direct) {
                    m_sm[rho] = m;
                    sum_sm[rho] = l;
                } else if (live)
                    A.ml[idx] = make_float2(m, l);
                arrive_tc(ofree(nitem % S::NO));
                ++nitem;
            }
            mbar_arrive(tfree);
            if (S::PB_IN_K && tid == 0) mbar_arrive(emptyK(tail_st));
            ++nt;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 10) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM_COLS);
    }
    if (direct) {   // the combine's operations for one split
        const int node0 = I0.node0(A.NT), rows = min(A.NT, I0.n - node0) * A.G, pitch = min(A.NT, A.N - node0) * A.G * 4;
        const float* part = reinterpret_cast<const float*>(smem + S::K_OFF);
        for (int e = tid; e < rows * (HD / 4); e += TREE_THREADS) {
            const int row = e / (HD / 4), c4 = e % (HD / 4), i = row / A.G, h = I0.g * A.G + row - i * A.G;
            const float4 o = *reinterpret_cast<const float4*>(part + c4 * pitch + row * 4);
            const float w = exp2f(__fsub_rn(m_sm[row], fmaxf(NEG_INF, m_sm[row]))), L = __fadd_rn(0.f, __fmul_rn(w, sum_sm[row]));
            const long long br = static_cast<long long>(I0.b) * A.N + node0 + i, c = static_cast<long long>(h) * HD + c4 * 4;
            const float a[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                A.out[br * A.out_stride + c + k] = tree_out(__fadd_rn(0.f, __fmul_rn(w, a[k])), L, A.gate ? A.gate + br * A.gate_stride + c + k : nullptr, HD);
        }
    }
}

// Combine of a row's splits, the decode rows' operations: w_s = exp2(m_s - M), L += w_s l_s,
// acc += w_s o_s in split order, out = acc / L (and the output gate).  A warp owns 16 columns of eight
// rows, four per lane: each of its loads takes whole 128-byte lines of the partials.  The four lanes of a
// row read its m and l and form its weights, each weight once a warp; eight splits are in flight.
// 13312 rows of 128 in 10 splits 18 us, 1536 rows of 256 in 71 splits 26 us.
constexpr int COMB_THREADS = 128;

__global__ void __launch_bounds__(COMB_THREADS) attn_tree_combine_kernel(const __grid_constant__ TreeArgs A, int hd) {
    griddep_launch();
    griddep_wait();
    // rows here run node by node within a sequence and kv head: [B][Hkv][N][G]
    const int per = hd / 16, lane = threadIdx.x & 31, row8 = lane & 7, c4 = lane >> 3;
    const int wid = static_cast<int>(blockIdx.x) * (COMB_THREADS / 32) + (threadIdx.x >> 5);
    const int rows = A.N * A.G, groups = (rows + 7) / 8;
    const int col = wid % per * 16 + 4 * c4, bg = wid / per / groups, r = (wid / per - bg * groups) * 8 + row8;
    const int b = bg / A.Hkv, g = bg - b * A.Hkv;
    if (b >= A.B) return;
    const int ctx = A.ctx_len[b], n = A.n_nodes ? A.n_nodes[b] : A.N;
    const int i = r / A.G, h = g * A.G + r - i * A.G;
    const bool on = r < rows && i < n && ctx >= 0 && ctx <= A.max_ctx;   // else reported by the split kernel
    const long long br = static_cast<long long>(b) * A.N + i;
    const int ns = on ? min(A.nsp[br], A.nsplit) : 0, ns_max = __reduce_max_sync(0xffffffffu, ns);
    const float2* ml = A.ml + (br * A.Hq + h) * A.nsplit;
    const int tile0 = i / A.NT * A.NT, pitch = min(A.NT, A.N - tile0) * A.G * 4;   // of its row tile
    const long long split_len = static_cast<long long>(rows) * hd;
    const float* op = A.opart + static_cast<long long>(bg) * A.nsplit * split_len + static_cast<long long>(tile0) * A.G * hd +
                      static_cast<long long>(col / 4) * pitch + (r - tile0 * A.G) * 4;
    float M = NEG_INF;
#pragma unroll 8
    for (int s = c4; s < ns; s += 4) M = fmaxf(M, ml[s].x);
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
    float L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;
#pragma unroll 1
    for (int s0 = 0; s0 < ns_max; s0 += U, op += U * split_len) {
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < ns) o[u] = *reinterpret_cast<const float4*>(op + u * split_len);
        float w[U / 4], wl[U / 4];
#pragma unroll
        for (int k = 0; k < U / 4; ++k) {
            const float2 v = s0 + 4 * k + c4 < ns ? ml[s0 + 4 * k + c4] : make_float2(NEG_INF, 0.f);
            w[k] = exp2f(__fsub_rn(v.x, M));
            wl[k] = __fmul_rn(w[k], v.y);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float x = __shfl_sync(0xffffffffu, w[u / 4], u % 4 * 8 + row8), xl = __shfl_sync(0xffffffffu, wl[u / 4], u % 4 * 8 + row8);
            if (s0 + u < ns) {
                L = __fadd_rn(L, xl);
                a[0] = __fadd_rn(a[0], __fmul_rn(x, o[u].x));
                a[1] = __fadd_rn(a[1], __fmul_rn(x, o[u].y));
                a[2] = __fadd_rn(a[2], __fmul_rn(x, o[u].z));
                a[3] = __fadd_rn(a[3], __fmul_rn(x, o[u].w));
            }
        }
    }
    if (!on) return;
    const long long c = static_cast<long long>(h) * hd + col;
    uint16_t* out = A.out + br * A.out_stride + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = tree_out(a[e], L, A.gate ? A.gate + br * A.gate_stride + c + e : nullptr, hd);
}

inline size_t r256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int TREE_MAX_CTX = 1 << 30;   // positions are ints, and a tree stands past the last one
constexpr long long TREE_MAX_ROWS = 1ll << 30;

size_t tree_workspace(int B, int N, int Hq, int hd, int max_ctx) {
    const size_t rows = static_cast<size_t>(B) * N * Hq * attn_split_count(max_ctx + N);
    return r256(rows * hd * sizeof(float)) + r256(rows * sizeof(float2)) + r256(4ull * B * N);
}

template <int HD>
constexpr int tree_smem() {
    return TreeShape<HD>::SLACK + TreeShape<HD>::INFO_OFF + static_cast<int>(sizeof(TreeInfo)) + 16;
}
static_assert(tree_smem<256>() <= 227 * 1024 && tree_smem<128>() <= 227 * 1024 && tree_smem<64>() <= 227 * 1024, "shared memory");

template <int HD>
xv_status tree_launch_split(const CUtensorMap* tm, const TreeArgs& a, bool* combined, cudaStream_t s) {
    constexpr int SMEM = tree_smem<HD>();
    int sms = 0;
    for (const void* f : {reinterpret_cast<const void*>(attn_tree_kernel<HD, true>), reinterpret_cast<const void*>(attn_tree_kernel<HD, false>)})
        if (xv_status st = kernel_smem_once(f, SMEM, false, "attn_tree: set shared memory size")) return st;
    if (xv_status st = device_sm_count(&sms)) return st;
    const long long n_items = static_cast<long long>(a.nsplit) * a.nrt * a.Hkv * a.B;
    if (n_items > (1ll << 30)) return fail(XV_ERR_UNSUPPORTED, "attn_tree: %lld work items", n_items);
    // past two waves of items, persistent CTAs (the rule of the decode rows' launch); rows of one split
    // are finished by the split kernel where its CTA has one item
    const bool multi = n_items > 2ll * sms;
    *combined = !multi && a.nsplit == 1 && tree_direct(a.NT * a.G, HD);
    trace_pre(s);
    if (multi) launch_k(attn_tree_kernel<HD, true>, dim3(sms), dim3(TREE_THREADS), SMEM, s, tm[0], tm[1], tm[2], tm[3], a);
    else launch_k(attn_tree_kernel<HD, false>, dim3(a.nrt, a.Hkv * a.B, a.nsplit), dim3(TREE_THREADS), SMEM, s, tm[0], tm[1], tm[2], tm[3], a);
    return launched("attn_tree_kernel", s, K_ATTN_TREE,
                    4ll * a.B * a.Hkv * a.max_ctx * HD + 4ll * a.B * a.N * (a.Hq + a.Hkv) * HD + 4ll * a.B * a.N * a.Hq * a.nsplit * (HD + 2));
}

xv_status tree_launch(TreeArgs a, int hd, void* ws, cudaStream_t s) {
    a.err = device_error_word();
    if (!a.err) return fail(XV_ERR_CUDA, "attn_tree: device error word unavailable");
    a.G = a.Hq / a.Hkv;
    const int fit = 128 / a.G;             // whole nodes a row tile holds
    a.nrt = ceil_div(a.N, fit);
    a.NT = ceil_div(a.N, a.nrt);
    a.nsplit = attn_split_count(a.max_ctx + a.N);
    const size_t rows = static_cast<size_t>(a.B) * a.N * a.Hq * a.nsplit;
    a.opart = static_cast<float*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + r256(rows * hd * sizeof(float)));
    a.nsp = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(a.ml) + r256(rows * sizeof(float2)));
    CUtensorMap tm[4];
    const uint64_t u = 2;
    const uint64_t qd[3] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.B) * a.N};
    const uint64_t qs[2] = {hd * u, a.q_stride * u};
    const uint32_t qb[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(a.NT)};
    if (xv_status st = encode_tiled(&tm[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
    const uint64_t kd[3] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(a.kv.page), static_cast<uint64_t>(a.kv.n_pages) * a.Hkv};
    const uint64_t ks[2] = {hd * u, static_cast<uint64_t>(a.kv.page) * hd * u};
    const uint32_t kb[3] = {64, static_cast<uint32_t>(T), 1};
    if (xv_status st = encode_tiled(&tm[1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.kc, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
    if (xv_status st = encode_tiled(&tm[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.vc, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
    const uint64_t td[2] = {static_cast<uint64_t>(a.Hkv) * hd, static_cast<uint64_t>(a.B) * a.N};
    const uint64_t tst[1] = {a.src_stride * u};
    const uint32_t tb[2] = {64, static_cast<uint32_t>(T)};
    if (xv_status st = encode_tiled(&tm[3], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.src, td, tst, tb, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
    bool combined = false;
    xv_status st = hd == 256 ? tree_launch_split<256>(tm, a, &combined, s)
                 : hd == 128 ? tree_launch_split<128>(tm, a, &combined, s) : tree_launch_split<64>(tm, a, &combined, s);
    if (st || combined) return st;
    const long long nrow = static_cast<long long>(a.B) * a.N * a.Hq;
    trace_pre(s);
    const long long warps = static_cast<long long>(a.B) * a.Hkv * ((a.N * a.G + 7) / 8) * (hd / 16);
    launch_k(attn_tree_combine_kernel, dim3(static_cast<unsigned>(ceil_div(warps, COMB_THREADS / 32))), dim3(COMB_THREADS), 0, s, a, hd);
    return launched("attn_tree_combine_kernel", s, K_ATTN_TREE, 4ll * nrow * a.nsplit * (hd + 2) + 2ll * nrow * hd * (a.gate ? 2 : 1));
}

xv_status tree_checks(const TreeArgs& a, int hd, int Lmax, const void* ws, size_t ws_bytes) {
    if (!a.q || !a.kc || !a.vc || !a.ctx_len || !a.src || !a.parent || !a.out) return fail(XV_ERR_ARG, "attn_tree: null pointer");
    if (a.B < 1 || a.N < 1 || a.Hq < 1 || a.Hkv < 1 || Lmax < 1) return fail(XV_ERR_ARG, "attn_tree: sizes must be positive");
    if (a.N > XV_KMAX) return fail(XV_ERR_UNSUPPORTED, "attn_tree: N = %d exceeds %d", a.N, XV_KMAX);
    if (a.Hq % a.Hkv) return fail(XV_ERR_ARG, "attn_tree: Hq must be a multiple of Hkv");
    if (hd != 64 && hd != 128 && hd != 256) return fail(XV_ERR_UNSUPPORTED, "attn_tree: hd must be 64, 128 or 256 (got %d)", hd);
    if (a.Hq / a.Hkv > 128) return fail(XV_ERR_UNSUPPORTED, "attn_tree: more than 128 q heads per kv head");
    if (a.max_ctx < 0 || a.max_ctx > Lmax) return fail(XV_ERR_ARG, "attn_tree: need 0 <= max_ctx <= Lmax");
    if (a.max_ctx > TREE_MAX_CTX) return fail(XV_ERR_UNSUPPORTED, "attn_tree: max_ctx exceeds 2^30 positions");
    if (a.B > 65535 || a.Hkv > 65535) return fail(XV_ERR_UNSUPPORTED, "attn_tree: B and Hkv must be below 65536");
    if (static_cast<long long>(a.B) * a.N * a.Hq > TREE_MAX_ROWS) return fail(XV_ERR_UNSUPPORTED, "attn_tree: more than 2^30 rows");
    if (static_cast<long long>(a.kv.n_pages) * a.Hkv >= (1ll << 31)) return fail(XV_ERR_UNSUPPORTED, "attn_tree: cache too large");
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
    if (B < 1 || B > 65535 || N < 1 || N > XV_KMAX || Hq < 1 || (hd != 64 && hd != 128 && hd != 256)) return 0;
    if (max_ctx < 0 || max_ctx > TREE_MAX_CTX || static_cast<long long>(B) * N * Hq > TREE_MAX_ROWS) return 0;
    return tree_workspace(B, N, Hq, hd, max_ctx);
}

xv_status xv_attn_tree(const uint16_t* q, long long q_stride, const uint16_t* kc, const uint16_t* vc,
                       const int32_t* ctx_len, const uint16_t* kv_src, long long src_stride, const int32_t* parent,
                       const int32_t* n_nodes, int N, int B, int Hq, int Hkv, int hd, int Lmax, int max_ctx, float scale,
                       const uint16_t* gate, long long gate_stride, uint16_t* out, long long out_stride, void* ws,
                       size_t ws_bytes, xv_stream s) {
    TreeArgs a{q, q_stride, kc, vc, kv_contiguous(B, Lmax), ctx_len, kv_src, src_stride, parent, n_nodes, N, B, Hq, Hkv,
               max_ctx, scale * 1.4426950408889634f, gate, gate_stride, out, out_stride, nullptr, 0, 0, 0, 0, nullptr, nullptr,
               nullptr};
    if (xv_status st = tree_checks(a, hd, Lmax, ws, ws_bytes)) return st;
    return tree_launch(a, hd, ws, reinterpret_cast<cudaStream_t>(s));
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
               max_ctx, scale * 1.4426950408889634f, gate, gate_stride, out, out_stride, nullptr, 0, 0, 0, 0, nullptr, nullptr,
               nullptr};
    if (xv_status st = tree_checks(a, hd, Lmax, ws, ws_bytes)) return st;
    return tree_launch(a, hd, ws, reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"

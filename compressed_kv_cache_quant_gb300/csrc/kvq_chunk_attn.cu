// kv_chunk_attn: attention of a run of new tokens per sequence over an fp16 layer's pages; kv_tree_attn, where the new
// tokens are trees of drafts; kv_latent_expanded_attn, a run over keys and values expanded from latent rows.
//
// Bound: the tensor cores from a few dozen query rows per kv head on (4 d flops per visible pair), below
// that the bytes of the cache.  One CTA takes up to 256 query rows of one kv head as two tiles of 128:
// row r is new token r / GQ, query head r % GQ of the group, so that the heads of a group share every
// staged K/V tile and a short run still fills rows.  Tiles of 128 cached tokens are eight pages, each
// fetched through the block table by one TMA box of 4 KB: groups of eight rows, a group's two halves of
// 64 values behind one another, 128-byte swizzle.
//
//   warps 8-11 give most of their registers to the softmax warps; 10 and 11 do nothing else
//   warp 9     loads: Q once, then K and V tiles into a ring of shared-memory stages
//   warp 8     issues tcgen05.mma: S_i = Q_i K^T into TMEM, O_i += P_i V with P_i read from TMEM
//   warps 0-3  softmax of tile 0: one thread per row, S from TMEM, P as fp16 back over S
//   warps 4-7  softmax of tile 1
//
// While one tile's softmax runs, the tensor cores work for the other one.  O stays in TMEM over the whole
// loop.  A row's weights are taken against an anchor, which cancels at the end: 2^7 below the row's maximum when
// it is set, and set anew (O rescaled) when a weight would pass 2^15.99.  A rescale holds up its tile for about 900
// cycles, so one row's turn is the turn of every row of its warp whose maximum has grown: 2048 tokens under a
// 4096-token window take 115 us in a graph, 117 us with anchors at the maximum that move for a growth beyond 2^14;
// anchors 2^7 below it that move one by one cost 16% more.
//
// P is one fp16 rounding of a weight, since the tensor cores take P and V in one type: off by 2^-11 of itself, or
// by 2^-25 where it is subnormal.  Against a largest weight of 2^7 or more that is 2^-32, so what many small weights
// add up to beside a dominant token is kept: 131072 of them lose under 2^-15 of the whole.  The rounding shows beside
// the fp16 output's own: 2.5e-4 to 2.9e-4 of the output (normwise) where the output's rounding alone is 2.1e-4.  A
// second half of P would bring that down for half as many products again.
//
// Measured (32 q / 8 kv heads): a causal prompt of 16384 tokens 1.35 ms, 1.63 PFLOP/s of the needed products,
// in a short run, 1.44 ms under the power limit of a long one; five drafted tokens of eight 32K sequences
// 171 us, 6.0 TB/s.  A turn (two tiles, 128 cached tokens) takes about 2700 cycles against 2048 of products:
// a tile's softmax takes 1250 (128 exponentials per row, 4-5 cycles each per warp), then its 768 last cycles
// of products and some 300 of signals close its chain, and the issuing warp spends 100 cycles on every wait,
// ready or not.
#include <algorithm>
#include <type_traits>

#include "kvq_attn_mod.cuh"
#include "kvq_latent.cuh"
#include "kvq_tc.cuh"
#include "kvq_tree.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int PG = KVQ_BLOCK_TOKENS;
constexpr int CA_NT = 384;
constexpr int CA_ROWS = 256;             // query rows per CTA
constexpr int CA_KEYS = 128;             // cached tokens per tile
constexpr int CA_NS = 4;                 // K or V tiles in the ring
constexpr int CA_TILE = 128 * D * 2;     // bytes of a Q, K or V tile
constexpr int CA_HALF = CA_TILE / 2;     // a Q tile is two halves of 128 rows x 128 bytes
constexpr int CA_SMEM = 2 * CA_TILE + CA_NS * CA_TILE + 1024;
constexpr int EX_QC = (D + KVQ_LATENT_ROPE) / 64;   // expanded form: halves of a query or key row of 192 values
constexpr int EX_NS = 8;                 // its ring, in pieces of CA_HALF: five per tile
constexpr int EX_SMEM = 2 * EX_QC * CA_HALF + EX_NS * CA_HALF + 1024;
constexpr float CA_HEAD = 7.0f;          // log2 of a row's largest weight when its anchor is set
constexpr float CA_TOP = 15.99f;         // log2 of the largest weight before the anchor is set anew (fp16 ends at 2^16)
constexpr float CA_FAR = 1048576.0f;     // scores (log2) beyond which they are rounded before the anchor is taken off

// TMEM columns: S (and P over it) of the two tiles, then their O
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
constexpr uint32_t IDESC_QK = idesc_f16(128, 128), IDESC_PV = IDESC_QK | KVQ_B_MN;   // (V's rows run along K)

struct ChunkArgs {
    const int32_t *bt, *seq_lens, *q_starts;
    const int32_t* parents;       // kv_tree_attn: of every row
    const int32_t* k_starts;      // kv_latent_expanded_attn: first key of every sequence, in place of seq_lens
    int64_t n_keys;
    int64_t num_blocks;
    int32_t batch, max_blocks, max_len, max_new, H, GQ, n_splits;
    int32_t items, heads_first;   // groups of new tokens, at most; which of heads and groups runs faster in the grid
    int64_t n_rows;
    KvqModArgs mod;
    uint16_t* out;
    float* lse;
    float* part;   // [item][split][CA_ROWS][D]
    float2* ml;    // [item][split][CA_ROWS] anchor (log2) and sum
    KvqWsHeader* hdr;
};

// ---------------------------------------------------------------- what a CTA works on

// A CTA's next group of the expanded form, from the warp that loads to the others.
struct Job {
    int32_t h, item, split, row0, rows, pos0, T, it0, nt;   // row0, pos0: its first query's row and place; rows 0: the end
};

struct Shared {
    uint64_t q_full, kv_full[EX_NS], kv_empty[EX_NS], s_full[2], p_full[2][2], o_full[2], drain;
    uint64_t q_empty, job_full[2], job_empty[2], cta_full;
    __align__(16) uint32_t cta[4];                // answer of a request for a CTA that was not launched yet
    Job job[2];
    uint32_t tmem;
    int32_t abort;
    int32_t item_b, item_tok;                     // sequence and first new token of this CTA
    int32_t doc_min, sink_max, lo_min, hi_max;    // over its rows
};

// What the new tokens are: a run; nodes of trees (kv_tree_attn); a run over expanded latent rows
// (kv_latent_expanded_attn).
enum Kind { RUN, TREES, EXPANDED };

// Tokens of sequence b; -1 where its keys lie outside the call's.
__device__ __forceinline__ int seq_len(const ChunkArgs& a, int b) {
    if (a.k_starts == nullptr) return a.seq_lens[b];
    const int64_t k0 = a.k_starts[b], k1 = a.k_starts[b + 1];
    return k0 < 0 || k1 < k0 || k1 > a.n_keys ? -1 : (int)(k1 - k0);
}

// Sequence b's new tokens: *first row and count; false (flagged) when its lengths do not fit the call.
__device__ __forceinline__ bool seq_rows(const ChunkArgs& a, int b, int* first, int* n) {
    *first = a.q_starts[b];
    const int64_t cnt = (int64_t)a.q_starts[b + 1] - *first;
    const int T = seq_len(a, b);
    *n = 0;
    if (*first < 0 || cnt < 0 || cnt > a.max_new || *first + cnt > a.n_rows || T < cnt || T > a.max_len) {
        kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return false;
    }
    *n = (int)cnt;
    return true;
}

// One warp finds item x: the x-th group of `tpc` new tokens, sequences in order, a sequence's last group
// (the one that sees most) first.  b = -1 when there is none.
__device__ __forceinline__ void find_item(const ChunkArgs& a, int x, int tpc, int* b_out, int* tok_out) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    *b_out = -1;
    *tok_out = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        int first, n = 0;
        if (b < a.batch) seq_rows(a, b, &first, &n);
        const int g = (n + tpc - 1) / tpc;
        int incl = g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const bool mine = x >= base + incl - g && x < base + incl;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who) {
            const int src = __ffs(who) - 1;
            *b_out = b0 + src;
            *tok_out = __shfl_sync(0xffffffffu, (base + incl - 1 - x) * tpc, src);
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }
// bits of the columns [a, b) of a tile in its w-th word of 32
__device__ __forceinline__ uint32_t columns(int a, int b, int w) {
    return b > a ? below(b - 32 * w) & ~below(a - 32 * w) : 0u;
}

// Eight words to a 16-byte aligned place; in one store where it is 32-byte aligned (`wide`).  A thread has a row of its
// own, so a store touches 32 lines: with 16 bytes each the outputs of 256 rows take 3.0 us, with 32 bytes 1.7 (four lanes
// that exchange their pieces and write 64 bytes of a row: 3.8).
__device__ __forceinline__ void store8(void* to, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Asks for a CTA of this grid that was not launched yet; it will not be, and the caller does its work.
__device__ __forceinline__ void next_cta_request(uint32_t to, uint64_t* bar) {
    bar_expect(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to),
                 "r"(saddr(bar))
                 : "memory");
}
// The answer: its place in the grid, or false when all have been launched (then no further request is allowed).
__device__ __forceinline__ bool next_cta_answer(uint32_t at, int* x, int* y) {
    uint32_t some, px, py;
    asm volatile(
        "{\n.reg .b128 r;\n.reg .pred p;\nld.shared.b128 r, [%3];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\nmov.u32 %2, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, r;\n}"
        : "=r"(some), "=r"(px), "=r"(py)
        : "r"(at)
        : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (the next answer is written by the asynchronous proxy)
    *x = (int)px, *y = (int)py;
    return some != 0;
}

// TREE: the new tokens are nodes of trees.  A node's interval ends with the cached tokens before them, and its path
// adds a few bits among the last columns; positions go by depth.
//
// EXPANDED: a key has 128 values of its head and 64 that all heads share, so a query row has three halves; keys and
// values lie in one piece per sequence.  The ring then holds 16 KB pieces, three of a K tile and two of a V tile (of 64
// tokens each): 1.6 tiles, since two query tiles take 96 KB.  A CTA works through several groups: while the softmax warps
// end one, the loading warp asks for another that no CTA has begun and fetches its queries and first keys; all barriers and
// the ring go on counting.  With a CTA per group 7 us passed between the last turn of one and the first of the next
// (five prompts of 333-4001 tokens, 16 heads: 116 instead of 109 us).
template <bool CAP, bool BIAS, Kind KIND>
__global__ void __launch_bounds__(CA_NT, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ ChunkArgs a) {
    constexpr bool TREE = KIND == TREES, EXP = KIND == EXPANDED;
    constexpr int Q_TILE = EXP ? EX_QC * CA_HALF : CA_TILE;
    extern __shared__ unsigned char raw[];
    __shared__ Shared S;
    __shared__ int4 seen_of[EXP ? 1 : CA_ROWS];   // lo, hi, doc, sink of every token
    __shared__ std::conditional_t<TREE, KvqTree, int> tree;
    // places of the columns from the first node's tile on, less ctx
    __shared__ __align__(16) float place_of[TREE && BIAS ? KVQ_TREE_MAX + CA_KEYS : 4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int GQ = a.GQ, tpc = CA_ROWS / GQ;
    const auto place = [&](int x, int* h, int* item) {
        *h = a.heads_first ? x % a.H : x / a.items;
        *item = a.heads_first ? x / a.H : x % a.items;
    };
    int split = blockIdx.y, h, item;
    place(blockIdx.x, &h, &item);
    const uint32_t sq = (saddr(raw) + 1023) & ~1023u, skv = sq + 2 * Q_TILE;
    kvq_pdl_begin();
    int b = 0, tok0 = 0, first = 0, n = 0, T = 0, ntok = 0;
    if constexpr (EXP) {
        if (tid == 0) S.abort = 0;
    } else {
        if (warp == 0) {
            int of, tok;
            find_item(a, item, tpc, &of, &tok);
            if (lane == 0) {
                S.item_b = of, S.item_tok = tok;
                S.abort = 0;
                S.doc_min = S.lo_min = INT32_MAX;
                S.sink_max = S.hi_max = 0;
            }
        }
        __syncthreads();
        b = S.item_b, tok0 = S.item_tok;
        if (b < 0) return;
        first = a.q_starts[b], n = a.q_starts[b + 1] - first, T = seq_len(a, b);
        ntok = min(tpc, n - tok0);
    }
    int rows = ntok * GQ, nq = rows > 128 ? 2 : 1;
    const int ctx = T - n;   // cached tokens before the new ones
    if constexpr (TREE) {
        if (tid < n) kvq_tree_fetch(tree, a.parents + first, tid, a.hdr);
        __syncthreads();
        if (tid < n) kvq_tree_walk(tree, tid, ctx & 31);
        __syncthreads();   // (of the nodes' paths a row reads its own, of their depths all)
        if (BIAS && tid < KVQ_TREE_MAX + CA_KEYS) {
            const int k = tid - ctx % CA_KEYS;
            place_of[tid] = (float)(k < 0 ? k : k < n ? (int)tree.depth[k] : 0);
        }
    }
    if (!EXP && tid < ntok) {
        const int i = tok0 + tid;
        const int doc = a.mod.doc_start ? a.mod.doc_start[first + i] : 0;
        KvqSee see;
        if constexpr (TREE) {
            const int pos = ctx + tree.depth[i];
            see = kvq_see(a.mod, pos, ctx, 0, doc);
            // ancestors the document or the window leaves out, by the rules of the cached tokens
            if (doc > ctx || a.mod.window > 0) {
                for (int k = i, at = pos; k >= 0; k = tree.parent[k], --at) {
                    if (at < doc || (a.mod.window > 0 && at <= pos - a.mod.window && at - max(doc, 0) >= a.mod.n_sink))
                        tree.path[i][(k + (ctx & 31)) >> 5] &= ~(1u << ((k + ctx) & 31));
                }
            }
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w <= KVQ_TREE_WORDS; ++w) any |= tree.path[i][w];
            if (any) {
                atomicMin(&S.lo_min, ctx);
                atomicMax(&S.hi_max, T);
            }
        } else {
            see = kvq_see(a.mod, ctx + i, T, a.mod.prefix_len ? a.mod.prefix_len[b] : 0, doc);
        }
        seen_of[tid] = make_int4(see.lo, see.hi, see.doc, see.sink);
        if (see.lo < see.hi) {
            atomicMin(&S.lo_min, see.lo);
            atomicMax(&S.hi_max, see.hi);
        }
        if (see.doc < see.sink) {
            atomicMin(&S.doc_min, see.doc);
            atomicMax(&S.sink_max, see.sink);
        }
    }
    if (tid == 0) {
        bar_init(&S.q_full, 1);
        for (int i = 0; i < (EXP ? EX_NS : CA_NS); ++i) {
            bar_init(&S.kv_full[i], 1);
            bar_init(&S.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&S.s_full[i], 1);
            bar_init(&S.p_full[i][0], 4);
            bar_init(&S.p_full[i][1], 4);
            bar_init(&S.o_full[i], 1);
        }
        bar_init(&S.drain, 1);
        if (EXP) {
            bar_init(&S.q_empty, 1);
            bar_init(&S.cta_full, 1);
            for (int i = 0; i < 2; ++i) {
                bar_init(&S.job_full[i], 1);
                bar_init(&S.job_empty[i], 1 + 8);   // the issuing lane and the softmax warps
            }
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem)), "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = S.tmem;
    // tiles some row sees: [a1, b1) for the sinks, then [a2, b2); this split takes [it0, it1) of the list
    int a1 = 0, b1 = 0, a2 = 0, b2 = 0;
    if (!EXP && S.doc_min < S.sink_max) a1 = S.doc_min / CA_KEYS, b1 = (S.sink_max + CA_KEYS - 1) / CA_KEYS;
    if (!EXP && S.lo_min < S.hi_max) a2 = max(S.lo_min / CA_KEYS, b1), b2 = max(a2, (S.hi_max + CA_KEYS - 1) / CA_KEYS);
    const int total = b1 - a1 + b2 - a2;
    const int per = (total + a.n_splits - 1) / a.n_splits;
    int it0 = min(total, split * per), nt = min(total, it0 + per) - it0;
    int row0 = first + tok0, pos0 = ctx + tok0;   // the first query's row and place
    const auto tile_of = [&](int it) { return it < b1 - a1 ? a1 + it : a2 + (it - (b1 - a1)); };

    // 384 threads are launched with 168 registers each: 256 * 232 + 128 * 40 is the same total
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 9 && (EXP || nt > 0)) {
            // ---- loads
            const auto queries = [&] {
                bar_expect(&S.q_full, nq * Q_TILE);
                for (int i = 0; i < nq; ++i)
                    for (int c = 0; c < Q_TILE / CA_HALF; ++c)
                        tma_3d(sq + i * Q_TILE + c * CA_HALF, &map_q, 64 * c, h * GQ, row0 + i * (128 / GQ), &S.q_full);
            };
            if constexpr (EXP) {
                // A tile is five pieces of a list that goes round the ring: K's three, V's two.  A piece's place was that of the
                // piece eight before, and every place has its own barriers.
                int p = 0, k = 0, loads = 0;   // pieces, groups and groups with keys so far
                int x = blockIdx.x, asked = 0;
                bool more = true;
                while (more && !aborted(&S.abort)) {
                    place(x, &h, &item);
                    find_item(a, item, tpc, &b, &tok0);
                    if (b >= 0) {
                        first = a.q_starts[b], n = a.q_starts[b + 1] - first, T = seq_len(a, b);
                        rows = min(tpc, n - tok0), nq = rows > 128 ? 2 : 1;
                        row0 = first + tok0, pos0 = T - n + tok0;
                        const int tiles = (pos0 + rows + CA_KEYS - 1) / CA_KEYS, each = (tiles + a.n_splits - 1) / a.n_splits;
                        it0 = min(tiles, split * each), nt = min(tiles, it0 + each) - it0;
                        if (k >= 2) bar_wait(&S.abort, a.hdr, &S.job_empty[k & 1], ((k >> 1) & 1) ^ 1);
                        if (lane == 0) {
                            S.job[k & 1] = Job{h, item, split, row0, rows, pos0, T, it0, nt};
                            bar_arrive(&S.job_full[k & 1]);
                        }
                        __syncwarp();
                        ++k;
                        if (nt > 0 && elect()) {
                            if (loads > 0) bar_wait(&S.abort, a.hdr, &S.q_empty, (loads & 1) ^ 1);
                            if (!*(volatile int32_t*)&S.abort) queries();
                            int key = a.k_starts[b] + it0 * CA_KEYS;
                            for (int j = 0, at = p; j < nt; ++j, key += CA_KEYS) {
#pragma unroll
                                for (int c = 0; c < 5; ++c, ++at) {
                                    uint64_t* full = &S.kv_full[at % EX_NS];
                                    if (at >= EX_NS) bar_wait(&S.abort, a.hdr, &S.kv_empty[at % EX_NS], ((at / EX_NS) & 1) ^ 1);
                                    if (*(volatile int32_t*)&S.abort) break;
                                    const uint32_t to = skv + at % EX_NS * CA_HALF;
                                    bar_expect(full, CA_HALF);
                                    if (c < 2)
                                        tma_3d(to, &map_k, 64 * c, h, key, full);
                                    else if (c == 2)
                                        tma_3d(to, &map_r, 0, key, 0, full);
                                    else
                                        for (int y = 0; y < 2; ++y)
                                            tma_3d(to + y * (CA_HALF / 2), &map_v, 64 * y, h, key + 64 * (c - 3), full);
                                }
                                if (*(volatile int32_t*)&S.abort) break;
                            }
                        }
                        __syncwarp();
                        p += 5 * nt, loads += nt > 0;
                    }
                    if (aborted(&S.abort)) break;
                    if (lane == 0) next_cta_request(saddr(S.cta), &S.cta_full);
                    __syncwarp();
                    bar_wait(&S.abort, a.hdr, &S.cta_full, asked++ & 1);
                    more = next_cta_answer(saddr(S.cta), &x, &split);
                    __syncwarp();
                }
                if (k >= 2) bar_wait(&S.abort, a.hdr, &S.job_empty[k & 1], ((k >> 1) & 1) ^ 1);
                if (lane == 0) {
                    S.job[k & 1].rows = 0;
                    bar_arrive(&S.job_full[k & 1]);
                }
                __syncwarp();
            } else {
                if (lane == 0) queries();
                __syncwarp();
                const int pg = lane & 7;   // lanes 0-7 look up one page each
                const int nowhere = (int)(a.num_blocks * a.H * (PG / 8));  // a group of rows behind the pool: zeros
                // where this lane's page of the j-th tile begins, in groups of 8 rows: it is looked up a tile ahead,
                // before the wait for V's stage
                const auto group_of = [&](int j) {
                    const int t = tile_of(it0 + j), lp = t * (CA_KEYS / PG) + pg;
                    uint32_t need;  // bit per page: some row sees a token of it
                    if (a.mod.doc_start == nullptr) {
                        const int p0 = lp * PG;
                        need = __ballot_sync(0xffffffffu, (p0 < S.hi_max && p0 + PG > S.lo_min) ||
                                                              (p0 < S.sink_max && p0 + PG > S.doc_min));
                    } else {
                        uint32_t bits = 0;
                        for (int k = lane; k < ntok; k += 32) {
                            const int4 e = seen_of[k];
                            const int p0 = t * (CA_KEYS / PG);
                            if (e.x < e.y) bits |= below((e.y + PG - 1) / PG - p0) & ~below(e.x / PG - p0);
                            if (e.z < e.w) bits |= below((e.w + PG - 1) / PG - p0) & ~below(e.z / PG - p0);
                            if (TREE) bits |= below((T + PG - 1) / PG - p0) & ~below(ctx / PG - p0);
                        }
                        need = __reduce_or_sync(0xffffffffu, bits);
                    }
                    int y = nowhere;
                    if (need >> pg & 1) {
                        const int32_t page = a.bt[(int64_t)b * a.max_blocks + lp];
                        if (page >= 0 && page < a.num_blocks)
                            y = (page * a.H + h) * (PG / 8);
                        else if (lane == pg)
                            kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
                    }
                    return y;
                };
                // one elected lane issues from uniform registers: a copy per lane would be issued one by one just
                // the same, at 79 cycles each
                const auto fetch = [&](int slot, const CUtensorMap* map, const int* at) {
                    const int st = slot % CA_NS;
                    if (slot >= CA_NS) bar_wait(&S.abort, a.hdr, &S.kv_empty[st], ((slot / CA_NS) & 1) ^ 1);
                    const bool ok = !aborted(&S.abort);
                    if (ok && elect()) {
                        bar_expect(&S.kv_full[st], CA_TILE);
#pragma unroll
                        for (int k = 0; k < 8; ++k) tma_page(skv + st * CA_TILE + k * (PG * D * 2), map, at[k], &S.kv_full[st]);
                    }
                    __syncwarp();
                    return ok;
                };
                bool ok = true;
                int y = group_of(0);
                for (int j = 0; j < nt && ok; ++j) {
                    int at[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) at[k] = __shfl_sync(0xffffffffu, y, k);
                    ok = fetch(2 * j, &map_k, at);
                    if (j + 1 < nt) y = group_of(j + 1);
                    ok = ok && fetch(2 * j + 1, &map_v, at);
                }
            }
        }
        if (warp == 8 && (EXP || nt > 0)) {
            // ---- tensor cores.  The whole warp walks the loop and one elected lane issues, so that the
            // descriptors stay in uniform registers.  All 512 TMEM columns are this CTA's, so they start at
            // column 0.  A descriptor is its low word plus constants: the low words are made opaque in every
            // step, or the compiler keeps all 64 of a step's descriptors in (spilled) registers, and the
            // reloads hold up every product (110 instead of 64 cycles each).
            const uint32_t hi_q = (uint32_t)(smem_desc(0, 16, 1024) >> 32),
                           hi_kv = (uint32_t)(smem_desc(0, 16, EXP ? 1024 : 2048) >> 32);
            const uint32_t lq = (uint32_t)smem_desc(sq, 16, 0), lk = (uint32_t)smem_desc(skv, 16, 0),
                           lv = (uint32_t)smem_desc(skv, EXP ? CA_HALF / 2 : 1024, 0);
            const auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; };
            const auto qk = [&](int i, int st) {
                if (elect()) {
                    uint32_t x = lq + (i * CA_TILE >> 4), y = lk + (st * CA_TILE >> 4);
                    asm volatile("" : "+r"(x), "+r"(y));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        mma_ss(TM_S + 128 * i, desc(hi_q, x + (((k >> 2) * CA_HALF + (k & 3) * 32) >> 4)),
                               desc(hi_kv, y + (((k >> 2) * 1024 + (k & 3) * 32) >> 4)), IDESC_QK, k > 0);
                    }
                    tc_commit(&S.s_full[i]);
                }
            };
            const auto pv = [&](int i, int st, int half, bool acc) {
                if (elect()) {
                    uint32_t y = lv + (st * CA_TILE >> 4);
                    asm volatile("" : "+r"(y));
#pragma unroll
                    for (int k = 4 * half; k < 4 * half + 4; ++k)
                        mma_ts(TM_O + 128 * i, TM_S + 128 * i + 8 * k, desc(hi_kv, y + (k * 4096 >> 4)), IDESC_PV, acc || k > 0);
                }
            };
            const auto commit = [&](uint64_t* bar) {
                if (elect()) tc_commit(bar);
            };
            if constexpr (EXP) {
                // one lane walks the loop
                if (elect()) {
                    int p0 = 0, loads = 0, turns[2] = {0, 0};   // pieces, groups with keys and tiles so far
                    const auto scores = [&](int i, int j) {
#pragma unroll
                        for (int c = 0; c < EX_QC; ++c) {
                            const int p = p0 + 5 * j + c;
                            if (i == 0) bar_wait(&S.abort, a.hdr, &S.kv_full[p % EX_NS], (p / EX_NS) & 1);
                            uint32_t x = lq + (i * Q_TILE + c * CA_HALF >> 4), y = lk + (p % EX_NS * CA_HALF >> 4);
                            asm volatile("" : "+r"(x), "+r"(y));
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ss(TM_S + 128 * i, desc(hi_q, x + 2 * k), desc(hi_kv, y + 2 * k), IDESC_QK, c + k > 0);
                            if (i == nq - 1) tc_commit(&S.kv_empty[p % EX_NS]);
                        }
                        tc_commit(&S.s_full[i]);
                        if (i == nq - 1 && j == nt - 1) tc_commit(&S.q_empty);
                    };
                    for (int g = 0;; ++g) {
                        bar_wait(&S.abort, a.hdr, &S.job_full[g & 1], (g >> 1) & 1);
                        if (*(volatile int32_t*)&S.abort) break;
                        rows = S.job[g & 1].rows, nt = S.job[g & 1].nt;
                        bar_arrive(&S.job_empty[g & 1]);
                        if (rows == 0) break;
                        if (nt == 0) continue;
                        nq = rows > 128 ? 2 : 1;
                        bar_wait(&S.abort, a.hdr, &S.q_full, loads++ & 1);
                        for (int i = 0; i < nq; ++i) scores(i, 0);
                        for (int j = 0; j < nt; ++j) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if (i == nq) break;
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const int p = p0 + 5 * j + 3 + half;
                                    // (V first: this lane waits for P some 700 cycles, so here it costs nothing)
                                    if (i == 0) bar_wait(&S.abort, a.hdr, &S.kv_full[p % EX_NS], (p / EX_NS) & 1);
                                    bar_wait(&S.abort, a.hdr, &S.p_full[i][half], (turns[i] + j) & 1);
                                    tc_after();
                                    uint32_t y = lv + (p % EX_NS * CA_HALF >> 4);
                                    asm volatile("" : "+r"(y));
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        mma_ts(TM_O + 128 * i, TM_S + 128 * i + 8 * (4 * half + k), desc(hi_kv, y + (k * 2048 >> 4)), IDESC_PV,
                                               j > 0 || half + k > 0);
                                    if (i == nq - 1) tc_commit(&S.kv_empty[p % EX_NS]);
                                }
                                if (j + 1 < nt)
                                    scores(i, j + 1);
                                else
                                    tc_commit(&S.o_full[i]);
                            }
                        }
                        p0 += 5 * nt, turns[0] += nt;
                        if (nq == 2) turns[1] += nt;
                    }
                }
                __syncwarp();
            } else {
                bar_wait(&S.abort, a.hdr, &S.q_full, 0);
                bar_wait(&S.abort, a.hdr, &S.kv_full[0], 0);
                tc_after();
                qk(0, 0);
                if (nq > 1) qk(1, 0);
                commit(&S.kv_empty[0]);
                for (int j = 0; j < nt; ++j) {
                    const int sv = (2 * j + 1) % CA_NS, sk = (2 * j + 2) % CA_NS;
                    const bool more = j + 1 < nt;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i == nq) break;
                        bar_wait(&S.abort, a.hdr, &S.p_full[i][0], j & 1);
                        tc_after();
                        pv(i, sv, 0, j > 0);
                        bar_wait(&S.abort, a.hdr, &S.p_full[i][1], j & 1);
                        tc_after();
                        pv(i, sv, 1, true);
                        if (i == nq - 1) commit(&S.kv_empty[sv]);
                        if (more) {
                            if (i == 0) bar_wait(&S.abort, a.hdr, &S.kv_full[sk], ((2 * j + 2) / CA_NS) & 1);
                            qk(i, sk);
                        } else {
                            commit(&S.o_full[i]);
                        }
                    }
                    if (more) commit(&S.kv_empty[sk]);
                }
            }
        }
    } else {
        // ---- softmax: thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int i = warp >> 2, r = tid;   // row of the CTA
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);  // TMEM lanes 32 (warp % 4) ..
        const uint32_t ts = lane_base + TM_S + 128 * i, to = lane_base + TM_O + 128 * i;
        int p0 = 0, turns = 0, outs = 0;   // expanded form: pieces of the ring, this tile's turns and outputs so far
        for (int g = 0;; ++g) {
            if constexpr (EXP) {
                // (a group of at most 128 rows is tile 0's alone: these warps may wait for as long as it has tiles)
                bar_wait(&S.abort, a.hdr, &S.job_full[g & 1], (g >> 1) & 1, KVQ_SPIN * (1 + min(nt >> 6, 4095)));
                if (aborted(&S.abort)) break;
                const Job w = S.job[g & 1];
                __syncwarp();
                if (lane == 0) bar_arrive(&S.job_empty[g & 1]);
                if (w.rows == 0) break;
                h = w.h, item = w.item, split = w.split, row0 = w.row0, rows = w.rows, pos0 = w.pos0, T = w.T, it0 = w.it0, nt = w.nt;
                nq = rows > 128 ? 2 : 1;
            }
            const bool valid = r < rows;
            const int tok = r / GQ;
            int4 see = make_int4(0, 0, 0, 0);
            int maxlo = 0, minhi = INT32_MAX;   // over the warp's rows: tiles between need no mask
            if (valid) {
                see = EXP ? make_int4(0, pos0 + tok + 1, 0, 0) : seen_of[tok];
                maxlo = see.x, minhi = see.y;
            }
            maxlo = __reduce_max_sync(0xffffffffu, maxlo);
            minhi = __reduce_min_sync(0xffffffffu, minhi);
            int pos = pos0 + tok;
            if constexpr (TREE) pos = ctx + (valid ? tree.depth[tok0 + tok] : 0);
            // what the row sees of the w-th 32 columns of the tile at t0
            const auto seen_bits = [&](int t0, int w) {
                if constexpr (TREE) {   // (from shared memory: kept in registers over the loop, some of them spill)
                    if (!valid) return 0u;
                    const int4 e = seen_of[tok];
                    return columns(e.x - t0, e.y - t0, w) | columns(e.z - t0, e.w - t0, w) | kvq_tree_bits(tree, tok0 + tok, t0 + 32 * w, ctx);
                }
                return columns(see.x - t0, see.y - t0, w) | columns(see.z - t0, see.w - t0, w);
            };
            const float slope2 = BIAS && valid ? a.mod.slopes[h * GQ + r % GQ] * KVQ_LOG2E : 0.0f;
            float m = valid ? -INFINITY : INFINITY, l = 0.0f;   // (no row: weights 0, never a new anchor)
            if (i < nq) {
                for (int j = 0; j < nt; ++j) {
                    const int t0 = (EXP ? it0 + j : tile_of(it0 + j)) * CA_KEYS;
                    // rows at and behind T may hold anything: 0 * NaN must not reach O
                    const bool tail = T < t0 + CA_KEYS && (EXP || (T & (PG - 1)) != 0) && T > t0;
                    const auto v_wait = [&] {
                        if (EXP) {
                            for (int p = p0 + 5 * j + 3; p < p0 + 5 * j + 5; ++p)
                                bar_wait(&S.abort, a.hdr, &S.kv_full[p % EX_NS], (p / EX_NS) & 1);
                        } else {
                            bar_wait(&S.abort, a.hdr, &S.kv_full[(2 * j + 1) % CA_NS], ((2 * j + 1) / CA_NS) & 1);
                        }
                    };
                    bar_wait(&S.abort, a.hdr, &S.s_full[i], (turns + j) & 1);
                    // tile 0's weights stand for V's arrival too (its products are issued after these waits, and tile
                    // 1's after tile 0's): the issuing warp is the busier one.  1.38 -> 1.36 ms for the prompt
                    if (!EXP && i == 0) v_wait();
                    if (tail) {
                        v_wait();
                        const uint32_t base = skv + (2 * j + 1) % CA_NS * CA_TILE;
                        const int r0 = T - t0, r1 = EXP ? CA_KEYS : (r0 + PG - 1) / PG * PG;
                        for (int x = tid & 127; x < (r1 - r0) * 16; x += 128) {
                            const int row = r0 + (x >> 4);
                            const uint32_t at = EXP ? skv + (p0 + 5 * j + 3 + (row >> 6)) % EX_NS * CA_HALF + (x & 1) * (CA_HALF / 2) +
                                                          (row & 63) * 128 + ((x >> 1) & 7) * 16
                                                    : base + (row >> 3) * 2048 + (x & 1) * 1024 + (row & 7) * 128 + ((x >> 1) & 7) * 16;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        if (CAP) {
                            // The form of the cap below is the warp's choice, by the size of its scores: neither these rows
                            // nor queries that are not the sequence's have a part in it, or what they hold would change
                            // the others' last bits.
                            tc_after();
#pragma unroll 1
                            for (int c = r0; c < r1; ++c) tm_st1(ts + c, 0);
                            tm_wait_st();
                        }
                    }
                    tc_after();
                    float s[128];
                    tm_ld128(ts, reinterpret_cast<uint32_t*>(s));
                    float scale = a.mod.pre;
                    if (CAP) {
                        float big[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int c = 0; c < 128; c += 4) {
                            big[0] = max3(big[0], fabsf(s[c]), fabsf(s[c + 1]));
                            big[1] = max3(big[1], fabsf(s[c + 2]), fabsf(s[c + 3]));
                        }
                        if (__all_sync(0xffffffffu, !valid || fmaxf(big[0], big[1]) * a.mod.pre <= 0.75f)) {
                            // the usual case: tanh x = x P(x^2) on |x| <= 3/4, P the polynomial through the Chebyshev
                            // points, 6e-7 relative; 3.5 instructions per score (below they are 2 special-function
                            // results on top of the weight's one: packed documents 87 us instead of 73)
                            const float z = a.mod.post;
                            const uint64_t pre2 = pair(a.mod.pre, a.mod.pre);
                            const uint64_t c0 = pair(0.999999463558197f * z, 0.999999463558197f * z),
                                           c1 = pair(-0.3332834839820862f * z, -0.3332834839820862f * z),
                                           c2 = pair(0.13259831070899963f * z, 0.13259831070899963f * z),
                                           c3 = pair(-0.05008019134402275f * z, -0.05008019134402275f * z),
                                           c4 = pair(0.012950727716088295f * z, 0.012950727716088295f * z);
#pragma unroll
                            for (int c = 0; c < 128; c += 2) {
                                const uint64_t x = mul2(pair(s[c], s[c + 1]), pre2), u = mul2(x, x);
                                unpair(mul2(x, fma2(fma2(fma2(fma2(c4, u, c3), u, c2), u, c1), u, c0)), &s[c], &s[c + 1]);
                            }
                        } else {
                            // tanh x = 1 - 2 / (1 + e^2x), 5e-7 absolute: ex2's and rcp's 2^-22, and three fp32 roundings
                            const float k2 = a.mod.pre * (2.0f * KVQ_LOG2E), p2 = -2.0f * a.mod.post;
#pragma unroll
                            for (int c = 0; c < 128; ++c) s[c] = fmaf(p2, rcp(1.0f + ex2(s[c] * k2)), a.mod.post);
                        }
                        scale = 1.0f;
                    }
                    if (BIAS) {
                        const float from = (float)(pos - t0);   // (whole numbers: exact below 2^24)
                        const float mul = CAP ? 1.0f : a.mod.pre;
                        bool nodes = false;
                        if constexpr (TREE) {
                            nodes = t0 + CA_KEYS > ctx;
                            if (nodes) {
                                const float depth = (float)(pos - ctx);
                                const float4* at = reinterpret_cast<const float4*>(place_of + (t0 - ctx / CA_KEYS * CA_KEYS));
#pragma unroll
                                for (int c = 0; c < 128; c += 4) {
                                    const float4 p = at[c / 4];
                                    s[c] = fmaf(s[c], mul, -slope2 * fabsf(depth - p.x));
                                    s[c + 1] = fmaf(s[c + 1], mul, -slope2 * fabsf(depth - p.y));
                                    s[c + 2] = fmaf(s[c + 2], mul, -slope2 * fabsf(depth - p.z));
                                    s[c + 3] = fmaf(s[c + 3], mul, -slope2 * fabsf(depth - p.w));
                                }
                            }
                        }
                        if (nodes) {
                        } else if (TREE || a.mod.prefix_len == nullptr) {
                            // what is seen is not ahead: -slope (from - c), linear in the column
                            const float at0 = -slope2 * from;
                            const uint64_t mul_2 = pair(mul, mul);
#pragma unroll
                            for (int c = 0; c < 128; c += 2) {
                                const uint64_t b = pair(fmaf(slope2, (float)c, at0), fmaf(slope2, (float)(c + 1), at0));
                                unpair(CAP ? add2(pair(s[c], s[c + 1]), b) : fma2(pair(s[c], s[c + 1]), mul_2, b), &s[c], &s[c + 1]);
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 128; ++c) s[c] = fmaf(s[c], mul, -slope2 * fabsf(from - (float)c));
                        }
                        scale = 1.0f;
                    }
                    if (t0 < maxlo || t0 + CA_KEYS > minhi) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            // an edge crosses few of a warp's words of 32 columns
                            const uint32_t bits = seen_bits(t0, w);
                            if (__all_sync(0xffffffffu, bits == ~0u)) continue;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(bits >> c & 1)) s[32 * w + c] = -INFINITY;
                        }
                    }
                    // The first half's weights are taken with the anchor so far, while the tile's maximum is still being
                    // found; only when that is too far above a row's anchor are they taken again.
                    uint32_t p[32];
                    uint64_t sum2[2];
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    // The steps of a pair are spread over eight turns of the loop, so that no instruction waits
                    // for the one before; the maximum's comparisons fill the gaps of the first half.
                    const auto weights = [&](int c, bool with_max) {
                        const float ms = m == -INFINITY ? 0.0f : m;
                        const uint64_t scale2 = pair(scale, scale), ms2 = pair(-ms, -ms);
                        uint64_t t[32];
                        float e[64];
#pragma unroll
                        for (int x = 0; x < 32 + 8; ++x) {
                            if (x < 32) {
                                t[x] = fma2(pair(s[c + 2 * x], s[c + 2 * x + 1]), scale2, ms2);
                                if (with_max) {
                                    mx4[x & 1] = max3(mx4[x & 1], s[2 * x], s[2 * x + 1]);
                                    mx4[2 + (x & 1)] = max3(mx4[2 + (x & 1)], s[64 + 2 * x], s[64 + 2 * x + 1]);
                                }
                            }
                            if (x >= 4 && x < 36) {
                                unpair(t[x - 4], &e[2 * (x - 4)], &e[2 * (x - 4) + 1]);
                                e[2 * (x - 4)] = ex2(e[2 * (x - 4)]);
                                e[2 * (x - 4) + 1] = ex2(e[2 * (x - 4) + 1]);
                            }
                            if (x >= 8) {
                                const int y = x - 8;
                                sum2[y & 1] = add2(sum2[y & 1], pair(e[2 * y], e[2 * y + 1]));
                                p[y] = half2_bits(e[2 * y], e[2 * y + 1]);
                            }
                        }
                    };
                    const auto rescale = [&](float f) {
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tm_ld32(to + c, o);
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tm_st32(to + c, o);
                        }
                    };
                    const auto hand_over = [&](int c) {   // the products start on the first half of the keys
                        tm_st32(ts + c / 2, p);
                        tm_wait_st();
                        tc_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(&S.p_full[i][c / 64]);
                    };
                    // A weight's exponent s * scale - m is rounded once, behind the difference.  That is exact enough until an
                    // fp32 step of m is no longer far below 1: a row's largest weight would be 2^(m's rounding error), 0 or
                    // infinite.  Then the products are rounded like m itself, from S as it still lies in TMEM (an own path,
                    // since a change of s in the loop below costs every prompt 3%).
                    const auto far_tile = [&] {
                        const auto seen = [&](int c) {
                            return seen_bits(t0, c >> 5) >> (c & 31) & 1;
                        };
                        uint32_t v[32];
                        float top = -INFINITY;
                        for (int c = 0; c < 128; c += 32) {
                            tm_ld32(ts + c, v);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (seen(c + x)) top = fmaxf(top, __fmul_rn(__uint_as_float(v[x]), scale));
                        }
                        const float anchor = fmaxf(m, top - CA_HEAD);
                        const float f = m == anchor ? 1.0f : ex2(m - anchor);
                        m = anchor;
                        l *= f;
                        if (j > 0) rescale(f);
                        const float ms = m == -INFINITY ? 0.0f : m;
                        for (int c = 0; c < 128; c += 64) {
#pragma unroll
                            for (int k = 0; k < 64; k += 32) {
                                tm_ld32(ts + c + k, v);
#pragma unroll
                                for (int x = 0; x < 32; x += 2) {
                                    const float e0 = seen(c + k + x) ? ex2(__fmul_rn(__uint_as_float(v[x]), scale) - ms) : 0.0f;
                                    const float e1 = seen(c + k + x + 1) ? ex2(__fmul_rn(__uint_as_float(v[x + 1]), scale) - ms) : 0.0f;
                                    l += e0 + e1;
                                    p[(k + x) / 2] = half2_bits(e0, e1);
                                }
                            }
                            hand_over(c);
                        }
                    };
                    // At most two turns (with far_tile in place of a third): behind a move of m the largest exponent is
                    // CA_HEAD and the roundings of m, under 1/8 up to CA_FAR.
                    bool done = false;
                    for (;;) {
                        sum2[0] = sum2[1] = 0;
                        weights(0, true);
                        const float top = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
                        // the exponent of the row's largest weight, rounded as the weights' are
                        const float most = fmaf(top, scale, -m);
                        if (!__any_sync(0xffffffffu, most > CA_TOP || (m == -INFINITY && top > m))) break;
                        // one row's turn is every row's: an anchor that would have to follow later is set now
                        const bool grew = most > CA_HEAD;
                        const float mx = top * scale;
                        if (!CAP && !BIAS && __any_sync(0xffffffffu, grew && fabsf(mx) > CA_FAR)) {
                            far_tile();
                            done = true;
                            break;
                        }
                        const float anchor = mx - CA_HEAD;
                        const float f = grew ? ex2(m - anchor) : 1.0f;
                        if (grew) m = anchor;
                        l *= f;
                        if (j > 0) rescale(f);
                    }
                    if (done) continue;
                    hand_over(0);
                    weights(64, false);
                    hand_over(64);
                    float l0, l1;
                    unpair(add2(sum2[0], sum2[1]), &l0, &l1);
                    l += l0 + l1;
                }
                // ---- this row's output
                if (nt > 0) bar_wait(&S.abort, a.hdr, &S.o_full[i], outs & 1);
                if (!aborted(&S.abort)) {
                    tc_after();
                    const int64_t out_row = (int64_t)(row0 + tok) * a.H * GQ + h * GQ + r % GQ;
                    const int64_t part_row = (((int64_t)item * a.H + h) * a.n_splits + split) * CA_ROWS + r;
                    const bool wide = ((uintptr_t)a.out & 31u) == 0;
                    const float inv = a.n_splits > 1 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        if (nt > 0) {
                            tm_ld32(to + c, o);
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = 0;
                        }
                        if (!valid) continue;
                        if (a.n_splits > 1) {
                            if (nt == 0) continue;
#pragma unroll
                            for (int x = 0; x < 32; x += 8) store8(a.part + part_row * D + c + x, o + x, true);
                        } else {
                            uint32_t w[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                w[x] = half2_bits(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
#pragma unroll
                            for (int x = 0; x < 16; x += 8) store8(a.out + out_row * D + c + 2 * x, w + x, wide);
                        }
                    }
                    if (valid && a.n_splits > 1 && nt > 0) a.ml[part_row] = make_float2(m, l);
                    if (valid && a.n_splits == 1 && a.lse != nullptr)
                        a.lse[out_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * KVQ_LN2;
                }
                turns += nt, outs += nt > 0;
            }
            if (!EXP) break;
            p0 += 5 * nt;
        }
    }
    __syncwarp();
    __syncthreads();
    if (*(volatile int32_t*)&S.abort) {
        drain_after_abort(warp == 8 && lane == 0, &S.drain);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
}

// Joins the splits of an item's rows, a warp per row, in their order, and leaves the workspace zeroed.  A split without a
// tile wrote nothing, one without a visible token a sum of 0.  MANY: the splits that wrote are found first and their rows
// fetched sixteen at a time (a tree of 25 nodes in 16 splits 20.0 -> 18.8 us, a window of six tokens in 38 splits 61 -> 20);
// with few splits that takes longer than reading all of them (64 nodes in two splits 219 -> 235 us).
constexpr int CJ_NW = 8, CJ_MANY = 8, CJ_G = 16;
template <bool MANY>
__global__ void __launch_bounds__(32 * CJ_NW) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
    __shared__ int item[4];   // its sequence, first new token, the sequence's first row, rows of the item
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int GQ = a.GQ, tpc = CA_ROWS / GQ, h = blockIdx.y, r = blockIdx.z * CJ_NW + warp;
    kvq_pdl_begin();
    if (warp == 0) {
        int b, tok;
        find_item(a, blockIdx.x, tpc, &b, &tok);
        if (lane == 0) {
            item[0] = b, item[1] = tok;
            if (b >= 0) {
                item[2] = a.q_starts[b];
                item[3] = min(tpc, a.q_starts[b + 1] - item[2] - tok) * GQ;
            }
        }
    }
    __syncthreads();
    if (item[0] < 0 || r >= item[3]) return;
    const int tok = item[1], first = item[2];
    const int64_t p0 = ((int64_t)blockIdx.x * a.H + h) * a.n_splits * CA_ROWS + r;
    const auto ml_at = [&](int s) { return a.ml + p0 + (int64_t)s * CA_ROWS; };
    float2 mine = lane < a.n_splits ? *ml_at(lane) : make_float2(0.0f, 0.0f);
    float mx = mine.y != 0.0f ? mine.x : -INFINITY;
    for (int s = lane + 32; s < a.n_splits; s += 32) {
        const float2 v = *ml_at(s);
        if (v.y != 0.0f) mx = fmaxf(mx, v.x);
    }
    mx = kvq_warp_max(mx);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float y = 0.0f;
    if constexpr (MANY) {
        for (int s0 = 0; s0 < a.n_splits; s0 += 32) {
            if (s0 > 0) mine = s0 + lane < a.n_splits ? *ml_at(s0 + lane) : make_float2(0.0f, 0.0f);
            const unsigned some = __ballot_sync(0xffffffffu, mine.y != 0.0f);
            const unsigned written = __ballot_sync(0xffffffffu, mine.x != 0.0f || mine.y != 0.0f);
            if (mine.x != 0.0f || mine.y != 0.0f) *ml_at(s0 + lane) = make_float2(0.0f, 0.0f);
            const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int g = 0; g < 32 && written >> g; g += CJ_G) {
                float4* const part = reinterpret_cast<float4*>(a.part + (p0 + (int64_t)(s0 + g) * CA_ROWS) * D) + lane;
                float4 w[CJ_G];
#pragma unroll
                for (int k = 0; k < CJ_G; ++k) w[k] = some >> (g + k) & 1 ? part[k * CA_ROWS * (D / 4)] : zero;
#pragma unroll
                for (int k = 0; k < CJ_G; ++k)
                    if (written >> (g + k) & 1) part[k * CA_ROWS * (D / 4)] = zero;
#pragma unroll
                for (int k = 0; k < CJ_G; ++k) {
                    const float2 v = make_float2(__shfl_sync(0xffffffffu, mine.x, g + k), __shfl_sync(0xffffffffu, mine.y, g + k));
                    const bool one = some >> (g + k) & 1;
                    const float f = one ? exp2f(v.x - mx) : 0.0f;
                    x.x += one ? f * w[k].x : 0.0f;
                    x.y += one ? f * w[k].y : 0.0f;
                    x.z += one ? f * w[k].z : 0.0f;
                    x.w += one ? f * w[k].w : 0.0f;
                    y += f * v.y;
                }
            }
        }
    } else {
#pragma unroll 8
        for (int s = 0; s < a.n_splits; ++s) {
            const float2 v = *ml_at(s);
            const float4 w = reinterpret_cast<const float4*>(a.part + (p0 + (int64_t)s * CA_ROWS) * D)[lane];
            const bool some = v.y != 0.0f;
            const float f = some ? exp2f(v.x - mx) : 0.0f;
            x.x += some ? f * w.x : 0.0f;
            x.y += some ? f * w.y : 0.0f;
            x.z += some ? f * w.z : 0.0f;
            x.w += some ? f * w.w : 0.0f;
            y += f * v.y;
        }
        // (behind the loads: a store between them would hold up the next one)
        for (int s = 0; s < a.n_splits; ++s)
            reinterpret_cast<float4*>(a.part + (p0 + (int64_t)s * CA_ROWS) * D)[lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncwarp();
        for (int s = lane; s < a.n_splits; s += 32) *ml_at(s) = make_float2(0.0f, 0.0f);
    }
    const float inv = y == 0.0f ? 0.0f : 1.0f / y;
    const int64_t out_row = (int64_t)(first + tok + r / GQ) * a.H * GQ + h * GQ + r % GQ;
    reinterpret_cast<uint2*>(a.out + out_row * D)[lane] =
        make_uint2(half2_bits(x.x * inv, x.y * inv), half2_bits(x.z * inv, x.w * inv));
    if (a.lse != nullptr && lane == 0) a.lse[out_row] = y == 0.0f ? -INFINITY : (mx + log2f(y)) * KVQ_LN2;
}

// ---------------------------------------------------------------- host

int check_rows(int64_t n_rows, int32_t max_new, const char* fn) {
    KVQ_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX && max_new >= 0 && (n_rows == 0 || max_new > 0), KVQ_ERR_INVALID_ARG,
                "%s: n_rows / max_new", fn);
    return KVQ_OK;
}

int check_tree_rows(int64_t n_rows, int32_t max_new, const char* fn) {
    const int st = check_rows(n_rows, max_new, fn);
    if (st) return st;
    KVQ_REQUIRE(max_new <= KVQ_TREE_MAX, KVQ_ERR_UNSUPPORTED, "%s: max_new %d (at most %d)", fn, max_new, KVQ_TREE_MAX);
    return KVQ_OK;
}

struct ChunkPlan {
    int64_t items;   // groups of new tokens over all sequences, at most
    int n_splits;
    size_t off_ml, off_part, bytes;
};

// Enough (item, kv head) CTAs fill the SMs by themselves; fewer are split along the cache, into the number
// of parts whose waves take least: a CTA's beginning and end cost about as much as 12 of its tiles (five
// drafted tokens of eight 32K sequences: 64 CTAs in 2 parts, one wave, 173 us; in 7 parts, three full waves,
// 182 us), the join's launch as 3, and the parts' rows are written, read and zeroed, 0.036 tiles' time per CTA
// of 256 rows (200 new tokens of 1000: 32 CTAs whole 19.9 us, in 2 parts 22.6 us; 500 of 8000: 91 us, in 2
// parts 62 us).  `least`: tiles of a part; two for trees, which are few rows (25 nodes behind 4096 tokens, two kv heads:
// in 7 parts of five tiles 24.7 us, in 16 20.4 us).
ChunkPlan chunk_plan(int H, int GQ, int32_t batch, int32_t max_len, int64_t n_rows, int32_t max_new, int least = 4) {
    ChunkPlan p;
    const int tpc = CA_ROWS / GQ;
    const int64_t by_max = batch * (((int64_t)max_new + tpc - 1) / tpc);
    p.items = std::max<int64_t>(1, std::min(by_max, n_rows / tpc + batch));
    const int64_t ctas = p.items * H, sms = kvq_num_sms();
    const int tiles = (max_len + CA_KEYS - 1) / CA_KEYS;
    p.n_splits = 1;
    if (ctas < sms) {
        const int most = (int)std::min<int64_t>(std::max(1, tiles / least), 4 * sms / ctas);
        const double full = std::min(1.0, (double)max_new * GQ / CA_ROWS);   // how much of a CTA's rows is used
        double best = 0.0;
        for (int s = 1; s <= most; ++s) {
            const int64_t waves = (ctas * s + sms - 1) / sms;
            double cost = (double)waves * ((tiles + s - 1) / s + 12);
            if (s > 1) cost += 3.0 + 0.036 * full * (double)(ctas * s);
            if (s == 1 || cost < best) best = cost, p.n_splits = s;
        }
    }
    const size_t rows = p.n_splits > 1 ? (size_t)ctas * p.n_splits * CA_ROWS : 0;
    p.off_ml = sizeof(KvqWsHeader);
    p.off_part = kvq_round_up(p.off_ml + rows * sizeof(float2), 256);
    p.bytes = kvq_round_up(p.off_part + rows * D * sizeof(float), 256);
    return p;
}

ChunkPlan chunk_plan(const kvq_layout* L, const kvq_seqs* S, int64_t n_rows, int32_t max_new, bool tree) {
    return chunk_plan(L->n_kv_heads, L->n_q_heads / L->n_kv_heads, S->batch, S->max_len, n_rows, max_new, tree ? 2 : 4);
}

// A call with something to do: its groups over all heads are a grid's x.
int check_plan(const ChunkPlan& p, int H, int32_t batch, int64_t n_rows, const char* fn) {
    KVQ_REQUIRE(batch == 0 || n_rows == 0 || p.items <= INT32_MAX / H, KVQ_ERR_UNSUPPORTED, "%s: n_rows", fn);
    return KVQ_OK;
}
size_t plan_bytes(const ChunkPlan& p, int H, int32_t batch, int64_t n_rows, const char* fn) {
    return check_plan(p, H, batch, n_rows, fn) ? 0 : p.bytes;
}

// Fills in what follows from the plan and launches the kernel and, over parts of the cache, their join.
template <typename Kernel>
int launch_chunk(Kernel kernel, int smem, const ChunkPlan& p, ChunkArgs& a, const CUtensorMap& map_q, const CUtensorMap& map_k,
                 const CUtensorMap& map_v, const CUtensorMap& map_r, void* ws, cudaStream_t stream, const char* fn) {
    a.n_splits = p.n_splits;
    a.items = (int32_t)p.items;
    a.hdr = static_cast<KvqWsHeader*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.off_ml);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_part);
    // The longest groups come first.  In a few waves, the heads' long groups run side by side, or the last
    // head's would start late (packed documents: 92 -> 82 us); in many waves one head after the other, so
    // that all CTAs read the same K and V (a 16384-token prompt: 1.38 instead of 1.42 ms).
    a.heads_first = p.items * a.H <= 6 * (int64_t)kvq_num_sms();
    const int rc = kvq_prepare_kernel((const void*)kernel, smem);
    if (rc) return rc;
    cudaError_t e = kvq_launch_pdl(kernel, dim3((unsigned)(p.items * a.H), p.n_splits), dim3(CA_NT), smem, stream, map_q, map_k,
                                   map_v, map_r, a);
    if (e == cudaSuccess && p.n_splits > 1)
        e = kvq_launch_pdl(p.n_splits > CJ_MANY ? chunk_join_kernel<true> : chunk_join_kernel<false>,
                           dim3((unsigned)p.items, a.H, CA_ROWS / CJ_NW), dim3(32 * CJ_NW), 0, stream, a);
    if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return KVQ_OK;
}

}  // namespace

extern "C" size_t kv_chunk_attn_ws(const kvq_layout* L, const kvq_seqs* S, int64_t n_rows, int32_t max_new) {
    if (kvq_check_layout(L, "kv_chunk_attn_ws", true) || kvq_check_seqs_sizes(S, "kv_chunk_attn_ws") ||
        kvq_check_max_len(S, "kv_chunk_attn_ws") || check_rows(n_rows, max_new, "kv_chunk_attn_ws"))
        return 0;
    return plan_bytes(chunk_plan(L, S, n_rows, max_new, false), L->n_kv_heads, S->batch, n_rows, "kv_chunk_attn_ws");
}

// kv_chunk_attn, or with `tree` kv_tree_attn.
static int chunk_attn(const char* fn, bool tree, const kvq_layout* L, const kvq_pool* P, const kvq_seqs* S, const uint16_t* q,
                      const int32_t* parents, const int32_t* q_starts, int64_t n_rows, int32_t max_new,
                      const kvq_attn_mod* mod, uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    kvq_clear_error();
    int st = kvq_check_layout(L, fn, true);
    if (st) return st;
    KVQ_REQUIRE(L->bits == 16, KVQ_ERR_UNSUPPORTED, "%s: bits %d (an fp16 layer)", fn, L->bits);
    st = kvq_check_seqs(S, fn);
    if (!st) st = kvq_check_max_len(S, fn);
    if (st) return st;
    KVQ_REQUIRE(P && P->k16 && P->v16 && P->num_blocks > 0, KVQ_ERR_INVALID_ARG, "%s: pool needs k16 and v16", fn);
    const int64_t pool_rows = P->num_blocks * L->n_kv_heads * PG;
    KVQ_REQUIRE(P->num_blocks <= INT32_MAX && pool_rows <= INT32_MAX && L->n_kv_heads <= 65535, KVQ_ERR_UNSUPPORTED,
                "%s: more than 2^31 - 1 rows in the pool", fn);
    st = tree ? check_tree_rows(n_rows, max_new, fn) : check_rows(n_rows, max_new, fn);
    if (st) return st;
    ChunkArgs a;
    st = kvq_mod_args(mod, fn, &a.mod);
    if (st) return st;
    KVQ_REQUIRE(!tree || a.mod.prefix_len == nullptr, KVQ_ERR_UNSUPPORTED, "%s: prefix_len (trees have no prefix)", fn);
    const ChunkPlan p = chunk_plan(L, S, n_rows, max_new, tree);
    st = kvq_check_ws(ws, ws_bytes, p.bytes, fn);
    if (st) return st;
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && q_starts && (!tree || parents) && (S->block_table || S->max_len == 0), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out | (uintptr_t)P->k16 | (uintptr_t)P->v16) & 15u) == 0,
                KVQ_ERR_INVALID_ARG, "%s: q, out, k16 and v16 must be 16-byte aligned", fn);
    st = check_plan(p, L->n_kv_heads, S->batch, n_rows, fn);
    if (st) return st;
    const int H = L->n_kv_heads, GQ = L->n_q_heads / H;
    CUtensorMap map_q, map_k, map_v;
    const uint64_t qd[3] = {D, (uint64_t)L->n_q_heads, (uint64_t)n_rows};
    const uint64_t qs[2] = {D * 2, (uint64_t)L->n_q_heads * D * 2};
    const uint32_t qb[3] = {64, (uint32_t)GQ, (uint32_t)(128 / GQ)};
    const uint64_t kd[4] = {64, 8, 2, (uint64_t)pool_rows / 8}, ks[3] = {D * 2, 64 * 2, 8 * D * 2};
    const uint32_t kb[4] = {64, 8, 2, PG / 8};
    st = make_map(&map_q, q, 3, qd, qs, qb, fn);
    if (!st) st = make_map(&map_k, P->k16, 4, kd, ks, kb, fn);
    if (!st) st = make_map(&map_v, P->v16, 4, kd, ks, kb, fn);
    if (st) return st;
    a.num_blocks = P->num_blocks;
    a.bt = S->block_table, a.seq_lens = S->seq_lens, a.q_starts = q_starts, a.parents = parents;
    a.k_starts = nullptr, a.n_keys = 0;
    a.batch = S->batch, a.max_blocks = S->max_blocks, a.max_len = S->max_len, a.max_new = max_new;
    a.H = H, a.GQ = GQ;
    a.n_rows = n_rows;
    a.out = out, a.lse = lse;
    const auto go = [&](auto kernel) {
        return launch_chunk(kernel, CA_SMEM, p, a, map_q, map_k, map_v, map_q, ws, kvq_stream(stream), fn);
    };
    const bool cap = a.mod.post != 0.0f, bias = a.mod.slopes != nullptr;
    if (tree) {
        if (cap) return bias ? go(chunk_attn_kernel<true, true, TREES>) : go(chunk_attn_kernel<true, false, TREES>);
        return bias ? go(chunk_attn_kernel<false, true, TREES>) : go(chunk_attn_kernel<false, false, TREES>);
    }
    if (cap) return bias ? go(chunk_attn_kernel<true, true, RUN>) : go(chunk_attn_kernel<true, false, RUN>);
    return bias ? go(chunk_attn_kernel<false, true, RUN>) : go(chunk_attn_kernel<false, false, RUN>);
}

extern "C" int kv_chunk_attn(const kvq_layout* L, const kvq_pool* P, const kvq_seqs* S, const uint16_t* q,
                             const int32_t* q_starts, int64_t n_rows, int32_t max_new, const kvq_attn_mod* mod,
                             uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    return chunk_attn("kv_chunk_attn", false, L, P, S, q, nullptr, q_starts, n_rows, max_new, mod, out, lse, ws, ws_bytes,
                      stream);
}

extern "C" size_t kv_tree_attn_ws(const kvq_layout* L, const kvq_seqs* S, int64_t n_rows, int32_t max_new) {
    if (kvq_check_layout(L, "kv_tree_attn_ws", true) || kvq_check_seqs_sizes(S, "kv_tree_attn_ws") ||
        kvq_check_max_len(S, "kv_tree_attn_ws") || check_tree_rows(n_rows, max_new, "kv_tree_attn_ws"))
        return 0;
    return plan_bytes(chunk_plan(L, S, n_rows, max_new, true), L->n_kv_heads, S->batch, n_rows, "kv_tree_attn_ws");
}

extern "C" int kv_tree_attn(const kvq_layout* L, const kvq_pool* P, const kvq_seqs* S, const uint16_t* q,
                            const int32_t* parents, const int32_t* q_starts, int64_t n_rows, int32_t max_new,
                            const kvq_attn_mod* mod, uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    return chunk_attn("kv_tree_attn", true, L, P, S, q, parents, q_starts, n_rows, max_new, mod, out, lse, ws, ws_bytes,
                      stream);
}

static int check_expanded(int32_t batch, int32_t n_heads, int64_t n_rows, int32_t max_new, int32_t max_len, const char* fn) {
    KVQ_REQUIRE(batch >= 0 && max_len >= 0, KVQ_ERR_INVALID_ARG, "%s: negative sizes", fn);
    KVQ_REQUIRE(max_len <= 1 << 30, KVQ_ERR_UNSUPPORTED, "%s: max_len %d (at most 2^30)", fn, max_len);
    return check_latent_rows(n_heads, n_rows, max_new, false, fn);
}

extern "C" size_t kv_latent_expanded_attn_ws(int32_t batch, int32_t n_heads, int64_t n_rows, int32_t max_new, int32_t max_len) {
    kvq_clear_error();
    if (check_expanded(batch, n_heads, n_rows, max_new, max_len, "kv_latent_expanded_attn_ws")) return 0;
    return plan_bytes(chunk_plan(n_heads, 1, batch, max_len, n_rows, max_new), n_heads, batch, n_rows, "kv_latent_expanded_attn_ws");
}

extern "C" int kv_latent_expanded_attn(int32_t batch, int32_t n_heads, const uint16_t* q, const uint16_t* k_nope,
                                       int64_t kn_stride, int64_t kn_head_stride, const uint16_t* k_rope, int64_t kr_stride,
                                       const uint16_t* v, int64_t v_stride, int64_t v_head_stride, int64_t n_keys,
                                       const int32_t* q_starts, const int32_t* k_starts, int64_t n_rows, int32_t max_new,
                                       int32_t max_len, float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                       void* stream) {
    static const char* fn = "kv_latent_expanded_attn";
    kvq_clear_error();
    int st = check_expanded(batch, n_heads, n_rows, max_new, max_len, fn);
    ChunkArgs a;
    if (!st) st = kvq_mod_args(nullptr, fn, &a.mod);
    if (!st) st = latent_scale(scale, fn, &a.mod.pre);
    if (st) return st;
    a.mod.lin = a.mod.pre;
    const ChunkPlan p = chunk_plan(n_heads, 1, batch, max_len, n_rows, max_new);
    st = kvq_check_ws(ws, ws_bytes, p.bytes, fn);
    if (st) return st;
    KVQ_REQUIRE(n_keys >= 0 && n_keys <= INT32_MAX - CA_KEYS, KVQ_ERR_INVALID_ARG, "%s: n_keys", fn);
    if (batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(n_keys > 0, KVQ_ERR_INVALID_ARG, "%s: queries without keys", fn);
    KVQ_REQUIRE(q && out && q_starts && k_starts && k_nope && k_rope && v, KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_nope | (uintptr_t)k_rope | (uintptr_t)v) & 15u) == 0,
                KVQ_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned", fn);
    KVQ_REQUIRE((kn_stride | kn_head_stride | kr_stride | v_stride | v_head_stride) % 8 == 0, KVQ_ERR_INVALID_ARG,
                "%s: strides must be multiples of 8", fn);
    // (a tensor map's strides are below 2^40 bytes)
    KVQ_REQUIRE(kn_stride >= D && kn_head_stride >= D && v_stride >= D && v_head_stride >= D && kr_stride >= KVQ_LATENT_ROPE &&
                    std::max({kn_stride, kn_head_stride, kr_stride, v_stride, v_head_stride}) < (int64_t)1 << 39,
                KVQ_ERR_INVALID_ARG, "%s: a stride below the row's width, or above 2^39", fn);
    st = check_plan(p, n_heads, batch, n_rows, fn);
    if (st) return st;
    const uint64_t H = n_heads;
    CUtensorMap map_q, map_k, map_v, map_r;
    const uint64_t qd[3] = {D + KVQ_LATENT_ROPE, H, (uint64_t)n_rows}, qs[2] = {(D + KVQ_LATENT_ROPE) * 2, H * (D + KVQ_LATENT_ROPE) * 2};
    const uint64_t kd[3] = {D, H, (uint64_t)n_keys}, ks[2] = {(uint64_t)kn_head_stride * 2, (uint64_t)kn_stride * 2},
                   vs[2] = {(uint64_t)v_head_stride * 2, (uint64_t)v_stride * 2};
    const uint64_t rd[3] = {KVQ_LATENT_ROPE, (uint64_t)n_keys, 1}, rs[2] = {(uint64_t)kr_stride * 2, 16};
    const uint32_t rows128[3] = {64, 1, 128}, rows64[3] = {64, 1, 64}, shared128[3] = {64, 128, 1};
    st = make_map(&map_q, q, 3, qd, qs, rows128, fn);
    if (!st) st = make_map(&map_k, k_nope, 3, kd, ks, rows128, fn);
    if (!st) st = make_map(&map_v, v, 3, kd, vs, rows64, fn);
    if (!st) st = make_map(&map_r, k_rope, 3, rd, rs, shared128, fn);
    if (st) return st;
    a.num_blocks = 0;
    a.bt = a.seq_lens = a.parents = nullptr;
    a.q_starts = q_starts, a.k_starts = k_starts, a.n_keys = n_keys;
    a.batch = batch, a.max_blocks = 0, a.max_len = max_len, a.max_new = max_new;
    a.H = n_heads, a.GQ = 1;
    a.n_rows = n_rows;
    a.out = out, a.lse = lse;
    return launch_chunk(chunk_attn_kernel<false, false, EXPANDED>, EX_SMEM, p, a, map_q, map_k, map_v, map_r, ws,
                        kvq_stream(stream), fn);
}

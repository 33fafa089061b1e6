// kv_latent_attn: absorbed attention over a latent layer, whose rows (576 values of fp16 per token) are the keys, and
// their first 512 values the values, of every head.
//
// Bound: the bytes of the rows for few query rows (1152 bytes and 2176 flops per query row and token), the tensor
// cores from some 100 query rows per sequence on.  Query rows are (new token, head) pairs, side by side in memory.  A
// token's row is read from its page by a TMA box of 16 tokens: groups of eight rows, a group's nine chunks of 64 values
// behind one another, 128-byte swizzle.
//
// Up to 32 query rows per sequence (latent_attn_kernel), steps of 48 tokens; the same staged rows serve both products:
//
//   S   = Q K^T      64 rows (32 at most in use) x 48 tokens    A = Q, B = the rows along their 576 values
//   O^T = V^T P^T    512 values x rows      A = the rows' first 512 values in four blocks of 128, B = P
//
// O transposed, because rows of 512 values would fill TMEM (M = 64 uses half of its lanes) and leave no place for S; as
// O^T they take a block's columns each, and the second product shrinks with the rows.  48 tokens, because three stages of
// them fit, and a step's products (1730 cycles) take less than its bytes at the rate of HBM (2350); with 64 tokens in two
// stages the loads' latency shows (32 sequences of 4096 to 32767 tokens, 16 heads: 169 us), with 32 in five the issuing
// lane is the bound (124 us).
//
//   warps 0-3  softmax: warp w has rows 16w .. 16w + 15 (M = 64 puts them into 16 lanes per warp), read as fragments
//              of 16 rows by 8 columns, two rows per thread; then the output
//   warp 4     issues tcgen05.mma: S of the next step before O^T of this one
//   warp 5     loads, and brings the pages of two steps later into L2
//
// More query rows: pairs of CTAs, further below.
//
// The steps of all sequences and row groups are one list, cut into equal ranges, one per SM (or pair): a CTA works
// through its range segment by segment, and a second launch joins the row groups that a cut runs through (groups of a few
// steps are left whole).  Weights are
// taken against an anchor per row as in kv_chunk_attn: 2^7 below the row's maximum when it is set, set anew (O rescaled)
// when a weight would pass 2^15.99; their exponents are differences of rounded products, so that far scores stay exact
// enough.
//
// Measured (in a graph): that batch 118 us, 5.8 TB/s (6.2 in this launch, 7 us of join); 131072 tokens of one sequence
// 43 us; one of 1025 tokens 11 us.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "kvq_attn_mod.cuh"
#include "kvq_latent.cuh"
#include "kvq_tc.cuh"
#include "kvq_tree.cuh"

namespace {

constexpr int PG = KVQ_BLOCK_TOKENS;
constexpr int LAT = KVQ_LATENT_DIM, ROT = KVQ_LATENT_ROPE, ROW = LAT + ROT;
constexpr int LA_NT = 192;
constexpr int LA_ROWS = 32;               // query rows per CTA, at most
constexpr int LA_KEYS = 48;               // tokens per step
constexpr int LA_FAR = 2;                 // steps that pages are brought into L2 ahead of their load
constexpr int LA_NS = 3;                  // stages: as many as fit
constexpr int LA_CHUNKS = ROW / 64;
constexpr int LA_GROUP = LA_CHUNKS * 1024;              // bytes of eight staged rows
constexpr int LA_STAGE = LA_KEYS / 8 * LA_GROUP;
constexpr int LA_SMEM = 232448 - 1024;    // dynamic shared memory of a CTA, at most (static: under 1 KB)
constexpr int la_smem(int nr) { return 1024 + nr * (ROW * 2 + 2 * 128) + LA_NS * LA_STAGE; }
static_assert(la_smem(LA_ROWS) <= LA_SMEM && la_smem(16) + LA_STAGE > LA_SMEM, "stages");
constexpr float LA_HEAD = 7.0f;           // log2 of a row's largest weight when its anchor is set
constexpr float LA_TOP = 15.99f;          // log2 of the largest weight before the anchor is set anew
constexpr int LA_WHOLE = 6;               // steps of a row group that is not cut, at most
// TMEM columns: O (O^T in four blocks of 64), two S.  All of them are the CTA's, so they start at column 0.
constexpr uint32_t TM_O = 0, TM_S = 256, TM_COLS = 512;

struct LatArgs {
    const int32_t *bt, *seq_lens, *q_starts, *parents;
    int64_t n_rows, num_blocks;
    int32_t batch, max_blocks, max_len, max_new, H, items;   // items: row groups, at most
    int32_t whole;                                        // a CTA (or pair) takes one row group, none is cut
    int32_t nr;                                           // rows per CTA (or pair) as the products see them: 16, 32 or 128
    float scale2;                                         // of a score, in log2 units
    uint16_t* out;
    float* lse;
    float* part;   // [slot][nr][LAT]
    float2* ml;    // [slot][nr] anchor (log2) and sum
    int4* cuts;    // [row group][nr] of a row in parts: its first part's CTA + 1, its parts, its row of the output
    KvqWsHeader* hdr;
};

// ---------------------------------------------------------------- the list of steps

struct Seq {
    int32_t first, n, T;   // first row of the call, new tokens, tokens
    int32_t groups, steps; // of nr query rows; of KEYS tokens, per group
};

template <int KEYS>
__device__ __forceinline__ Seq seq_at(const LatArgs& a, int b) {
    Seq s = {0, 0, 0, 0, 0};
    const int first = a.q_starts[b], T = a.seq_lens[b];
    const int64_t cnt = (int64_t)a.q_starts[b + 1] - first;
    if (first < 0 || cnt < 0 || cnt > a.max_new || first + cnt > a.n_rows || T < cnt || T > a.max_len) {
        kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return s;
    }
    s.first = first, s.n = (int)cnt, s.T = T;
    s.groups = (int)(((uint32_t)s.n * a.H + a.nr - 1) / (uint32_t)a.nr);   // (rows of all heads are below 2^31)
    s.steps = s.groups > 0 ? (T + KEYS - 1) / KEYS : 0;
    return s;
}

// A CTA's range, segment by segment: `cnt` steps of one row group from `step` on, of which the first nt hold a token
// that some row of the group sees; those end before token `end`.
template <int KEYS>
struct Segment {
    int32_t at, end_at;   // where it begins in the list, and where the CTA's range ends
    int32_t item;         // row groups before it, over all sequences
    int32_t b, group, step, cnt, nt, end;
    Seq s;
    __device__ __forceinline__ void clip(const LatArgs& a) {
        cnt = min(end_at - at, s.steps - step);
        end = s.T;
        if (a.parents == nullptr) {
            const uint32_t last = min((uint32_t)s.n * a.H, (uint32_t)(group + 1) * a.nr) - 1;
            end = s.T - s.n + (int)(last / (uint32_t)a.H) + 1;
        }
        nt = max(0, min(cnt, (end + KEYS - 1) / KEYS - step));
    }
    __device__ __forceinline__ bool next(const LatArgs& a) {
        at += cnt;
        if (at >= end_at) return false;
        step = 0;
        ++item;
        if (++group == s.groups) {
            group = 0;
            do {
                if (++b >= a.batch) return false;
                s = seq_at<KEYS>(a, b);
            } while (s.steps == 0);
        }
        clip(a);
        return true;
    }
};

// One warp: the first segment (b = -1: none) of the index-th of `count` CTAs, or pairs of them, and the steps of each
// (where groups are not cut, the index-th group).  Steps of all sequences are below 2^31.
template <int KEYS>
__device__ __forceinline__ Segment<KEYS> first_segment(const LatArgs& a, int index, int count, int* per_out) {
    const int lane = threadIdx.x & 31;
    const Seq none = {0, 0, 0, 0, 0};
    const Seq mine = lane < a.batch ? seq_at<KEYS>(a, lane) : none;   // (of the first 32 sequences, kept)
    const auto share = [&](const Seq& s) { return a.whole ? s.groups : s.groups * s.steps; };
    int sum = share(mine);
    for (int b = lane + 32; b < a.batch; b += 32) sum += share(seq_at<KEYS>(a, b));
    const int total = (int)__reduce_add_sync(0xffffffffu, (unsigned)sum);
    const int per = a.whole ? 1 : max(1, (int)((uint32_t)(total + count - 1) / (uint32_t)count));
    *per_out = per;
    Segment<KEYS> g = {0, 0, 0, -1, 0, 0, 0, 0, 0, none};
    const int64_t x64 = (int64_t)per * index;
    if (x64 >= total) return g;
    const int x = (int)x64;
    int base = 0, items = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const Seq s = b0 == 0 ? mine : b0 + lane < a.batch ? seq_at<KEYS>(a, b0 + lane) : none;
        const int steps = share(s);
        int incl = steps, incl_items = s.groups;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o), v = __shfl_up_sync(0xffffffffu, incl_items, o);
            if (lane >= o) incl += u, incl_items += v;
        }
        const unsigned who = __ballot_sync(0xffffffffu, x >= base + incl - steps && x < base + incl);
        if (who) {
            const int src = __ffs(who) - 1;
            const auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
            g.s = Seq{of(s.first), of(s.n), of(s.T), of(s.groups), of(s.steps)};
            const uint32_t in = (uint32_t)(x - of(base + incl - steps));
            g.b = b0 + src;
            if (a.whole) {
                g.end_at = g.s.steps;
                g.group = (int)in;
            } else {
                g.at = x, g.end_at = min(x + per, total);
                g.group = (int)(in / (uint32_t)g.s.steps);
                g.step = (int)in - g.group * g.s.steps;
            }
            g.item = of(items + incl_items - s.groups) + g.group;
            g.clip(a);
            return g;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
        items += __shfl_sync(0xffffffffu, incl_items, 31);
    }
    return g;
}

// A place in a ring of n: the index, and the parity of the rounds before it.
struct Place {
    int i = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) i = 0, round ^= 1;
    }
};

struct Shared {
    uint64_t q_full, q_free, kv_full[LA_NS], kv_empty[LA_NS], s_full[2], p_full[2], pv_done[2], drain;
    uint32_t tmem;
    int32_t abort;
    Segment<LA_KEYS> seg;
    int32_t per;       // steps per CTA
    float factor[64];  // (of 64 rows: M of the first product)
};

__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// one barrier of the softmax warps; true when some thread's x is
__device__ __forceinline__ bool sm_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// 16 lanes by 48 columns: of column group k (8 columns), v[4k] and v[4k + 1] are row lane / 4, columns 2 (lane % 4) and
// the one behind it, v[4k + 2] and v[4k + 3] the same of row lane / 4 + 8
__device__ __forceinline__ void tm_ld_frag(uint32_t addr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%24];\n"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%25];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
          "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23])
        : "r"(addr), "r"(addr + 32)
        : "memory");
}

// A row's path to its root, 32 nodes per word, walked through the parents.
__device__ __forceinline__ void walk_path(const LatArgs& a, int first, int tok, uint32_t* path) {
    for (int k = tok; k >= 0;) {
#pragma unroll
        for (int w = 0; w < KVQ_TREE_WORDS; ++w)
            if (k >> 5 == w) path[w] |= 1u << (k & 31);
        const int p = a.parents[first + k];
        if (p < -1 || p >= k) kvq_dev_flag(a.hdr, KVQ_DEV_BAD_INDEX, p);
        k = p < -1 || p >= k ? -1 : p;
    }
}
// 32 bits of it from node `from` on
__device__ __forceinline__ uint32_t path_bits(const uint32_t* path, int from) {
    const int at = from >> 5;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < KVQ_TREE_WORDS; ++i) {
        if (i == at) lo = path[i];
        if (i == at + 1) hi = path[i];
    }
    return __funnelshift_r(lo, hi, from & 31);
}

__global__ void __launch_bounds__(LA_NT, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_rows,
                       const __grid_constant__ LatArgs a) {
    constexpr int NG = LA_KEYS / 8;
    extern __shared__ unsigned char raw[];
    __shared__ Shared S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // queries, stages, weights: with nr below 64 the first product reads behind the queries, into the stages, for
    // rows of S that nothing looks at
    if (tid == 64) map_prefetch(&map_q), map_prefetch(&map_rows);
    const uint32_t sq = (saddr(raw) + 1023) & ~1023u, skv = sq + a.nr * ROW * 2, sp = skv + LA_NS * LA_STAGE,
                   p_bytes = a.nr * 128;   // (a row of weights takes 128 bytes, as the swizzle wants it)
    // (what does not read global memory goes before the wait for the launch before)
    if (tid == 32) {
        bar_init(&S.q_full, 1);
        bar_init(&S.q_free, 1);
        for (int i = 0; i < LA_NS; ++i) {
            bar_init(&S.kv_full[i], 1);
            bar_init(&S.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&S.s_full[i], 1);
            bar_init(&S.p_full[i], 4);
            bar_init(&S.pv_done[i], 1);
        }
        bar_init(&S.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem)), "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    kvq_pdl_begin();
    if (warp == 0) {
        int per;
        const Segment<LA_KEYS> g = first_segment<LA_KEYS>(a, blockIdx.x, gridDim.x, &per);
        if (lane == 0) S.seg = g, S.per = per, S.abort = 0;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = S.tmem;
    Segment<LA_KEYS> g = S.seg;

    if (g.b < 0) {
        // no work
    } else if (warp == 5) {
        // ---- loads
        const int nowhere = (int)(a.num_blocks * (PG / 8));   // a group of rows behind the pool: zeros
        Place st;
        int loaded = 0;    // steps so far
        bool ok = true;
        for (int seg = 0; ok;) {
            // lanes 0 .. LA_KEYS / 16 - 1 look up one page each, a step ahead
            const auto group_of = [&](int j) {
                const int lp = (g.step + j) * (LA_KEYS / PG) + lane;
                if (j >= g.nt || lane >= LA_KEYS / PG || lp * PG >= g.end) return nowhere;
                const int32_t page = a.bt[(int64_t)g.b * a.max_blocks + lp];
                if (page >= 0 && page < a.num_blocks) return page * (PG / 8);
                kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
                return nowhere;
            };
            int y = group_of(0), ahead[LA_FAR];
#pragma unroll
            for (int k = 0; k < LA_FAR; ++k) ahead[k] = group_of(1 + k);
            if (g.nt > 0) {
                if (seg > 0) bar_wait(&S.abort, a.hdr, &S.q_free, (seg - 1) & 1);
                ok = !aborted(&S.abort);
                if (ok && elect()) {
                    bar_expect(&S.q_full, a.nr * ROW * 2);
                    tma_3d(sq, &map_q, 0, g.s.first * a.H + g.group * a.nr, 0, &S.q_full);
                }
                __syncwarp();
                ++seg;
            }
            for (int j = 0; j < g.nt && ok; ++j, ++loaded) {
                const int pages = min(LA_KEYS / PG, (g.end - (g.step + j) * LA_KEYS + PG - 1) / PG);
                int to[LA_KEYS / PG];
#pragma unroll
                for (int k = 0; k < LA_KEYS / PG; ++k) to[k] = __shfl_sync(0xffffffffu, y, k);
                if (loaded >= LA_NS) bar_wait(&S.abort, a.hdr, &S.kv_empty[st.i], st.round ^ 1);
                ok = !aborted(&S.abort);
                if (ok && elect()) {
                    bar_expect(&S.kv_full[st.i], pages * PG * ROW * 2);
#pragma unroll
                    for (int k = 0; k < LA_KEYS / PG; ++k)
                        if (k < pages) tma_page(skv + st.i * LA_STAGE + k * (PG * ROW * 2), &map_rows, to[k], &S.kv_full[st.i]);
                }
                __syncwarp();
                if (ahead[LA_FAR - 1] != nowhere) tma_page_prefetch(&map_rows, ahead[LA_FAR - 1]);
                y = ahead[0];
#pragma unroll
                for (int k = 0; k + 1 < LA_FAR; ++k) ahead[k] = ahead[k + 1];
                ahead[LA_FAR - 1] = group_of(j + 1 + LA_FAR);
                st.next(LA_NS);
            }
            if (!g.next(a)) break;
        }
    } else if (warp == 4) {
        // ---- tensor cores: one lane walks the loop (elected anew for every batch, it starts some 100 cycles later)
        if (elect()) {
            const uint32_t hi_q = (uint32_t)(smem_desc(0, 16, 1024) >> 32), hi_kv = (uint32_t)(smem_desc(0, 16, LA_GROUP) >> 32);
            const uint32_t lq = (uint32_t)smem_desc(sq, 16, 0), lk = (uint32_t)smem_desc(skv, 16, 0),
                           lv = (uint32_t)smem_desc(skv, 1024, 0), lp = (uint32_t)smem_desc(sp, 16, 0);
            const uint32_t idesc_s = idesc_f16(64, LA_KEYS), idesc_o = idesc_f16(128, a.nr) | KVQ_A_MN;
            const auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; };
            const uint32_t q_chunk = (uint32_t)a.nr * 128 >> 4;
            Place in, s, out, p;   // stage and S of the next first product, stage and P of the next second one
            const auto qk = [&] {
                bar_wait(&S.abort, a.hdr, &S.kv_full[in.i], in.round);
                tc_after();
                {
                    uint32_t x = lq, y = lk + (in.i * LA_STAGE >> 4);
                    asm volatile("" : "+r"(x), "+r"(y));
#pragma unroll
                    for (int c = 0; c < LA_CHUNKS; ++c) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ss(TM_S + s.i * LA_KEYS, desc(hi_q, x + 2 * k), desc(hi_kv, y + (c * 1024 >> 4) + 2 * k), idesc_s, c + k > 0);
                        x += q_chunk;
                    }
                    // (all products so far: where S is there, so is O^T of two steps before, and P's place is free)
                    tc_commit(&S.s_full[s.i]);
                }
                in.next(LA_NS);
                s.next(2);
            };
            for (int seg = 0;;) {
                const int nt = g.nt;
                if (nt > 0) {
                    bar_wait(&S.abort, a.hdr, &S.q_full, seg & 1);
                    ++seg;
                    qk();
                    if (nt == 1) tc_commit(&S.q_free);
                }
                for (int j = 0; j < nt; ++j) {
                    if (j + 1 < nt) {
                        qk();
                        if (j + 2 == nt) tc_commit(&S.q_free);
                    }
                    bar_wait(&S.abort, a.hdr, &S.p_full[p.i], p.round);
                    tc_after();
                    {
                        uint32_t y = lv + (out.i * LA_STAGE >> 4), z = lp + (p.i * p_bytes >> 4);
                        asm volatile("" : "+r"(y), "+r"(z));
#pragma unroll
                        for (int d = 0; d < LAT / 128; ++d)
#pragma unroll
                            for (int k = 0; k < LA_KEYS / 16; ++k)
                                mma_ss(TM_O + 64 * d, desc(hi_kv, y + ((k * 2 * LA_GROUP + d * 2048) >> 4)), desc(hi_q, z + 2 * k), idesc_o,
                                       j > 0 || k > 0);
                        tc_commit(&S.kv_empty[out.i]);
                        tc_commit(&S.pv_done[p.i]);
                    }
                    out.next(LA_NS);
                    p.next(2);
                }
                if (!g.next(a)) break;
            }
        }
    } else {
        // ---- softmax: a thread has columns 8k + 2 (lane % 4) and the one behind of rows ra and ra + 8
        const uint32_t lane_base = tmem + ((uint32_t)warp << 21);   // TMEM lanes 32 warp ..
        const int ra = 16 * warp + (lane >> 2), c0 = 2 * (lane & 3);
        const bool tree = a.parents != nullptr;
        // `done`: the step before.  Where S of a step is there, O^T of two steps before is, so that of the step before is
        // at most one phase of its barrier away
        Place st, s_at, done;
        do {
            const int nt = g.nt, end = g.end, ctx = g.s.T - g.s.n;
            const int row0 = g.group * a.nr;   // of the sequence
            const int rows = min(a.nr, g.s.n * a.H - row0);
            const bool active = 16 * warp < rows;
            bool valid[2];
            int cut[2];                                     // every token before it is seen
            uint32_t path[2][KVQ_TREE_WORDS] = {};
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                valid[i] = ra + 8 * i < rows;
                const int tok = valid[i] ? (int)((uint32_t)(row0 + ra + 8 * i) / (uint32_t)a.H) : 0;
                cut[i] = valid[i] ? (tree ? ctx : ctx + tok + 1) : 0;
                if (tree && valid[i]) walk_path(a, g.s.first, tok, path[i]);
            }
            const int full = __reduce_min_sync(0xffffffffu, min(cut[0], cut[1]));
            for (int j = 0; j < nt; ++j, done = s_at, st.next(LA_NS), s_at.next(2)) {
                const int t0 = (g.step + j) * LA_KEYS;
                bar_wait(&S.abort, a.hdr, &S.s_full[s_at.i], s_at.round);
                tc_after();
                if (end < t0 + LA_KEYS) {
                    // rows at and behind the end may hold anything: 0 * NaN must not reach O^T
                    const uint32_t base = skv + st.i * LA_STAGE;
                    const int r0 = end - t0;
                    for (int x = tid; x < (LA_KEYS - r0) * (LAT / 8); x += 128) {
                        const int row = r0 + x / (LAT / 8), c = x % (LAT / 8);
                        const uint32_t to = base + (row >> 3) * LA_GROUP + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
                    }
                }
                float s[4 * NG];
                float top[2] = {-INFINITY, -INFINITY};
                bool far = false;
                if (active) {
                    tm_ld_frag(lane_base + TM_S + s_at.i * LA_KEYS, s);
#pragma unroll
                    for (int c = 0; c < 4 * NG; ++c) s[c] = __fmul_rn(s[c], a.scale2);
                    if (t0 + LA_KEYS > full) {   // (full: what every row of the warp sees all of)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint64_t bits = (uint64_t)below(cut[i] - t0 - 32) << 32 | below(cut[i] - t0);
                            if (tree && valid[i])
                                bits |= (uint64_t)path_bits(path[i], t0 + 32 - ctx) << 32 | path_bits(path[i], t0 - ctx);
                            bits >>= c0;
#pragma unroll
                            for (int k = 0; k < NG; ++k) {
                                if (!(bits >> (8 * k) & 1)) s[4 * k + 2 * i] = -INFINITY;
                                if (!(bits >> (8 * k) & 2)) s[4 * k + 2 * i + 1] = -INFINITY;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int k = 0; k < NG; ++k) top[i] = max3(top[i], s[4 * k + 2 * i], s[4 * k + 2 * i + 1]);
                        // a first anchor, or a weight that would leave fp16's range (any lane of the row's four tells)
                        far |= m[i] == -INFINITY ? top[i] > m[i] : top[i] - m[i] > LA_TOP;
                    }
                }
                if (sm_any(far)) {
                    // one row's turn is every row's: an anchor that would have to follow later is set now
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        float f = 1.0f;
                        if (m[i] == -INFINITY ? x > m[i] : x - m[i] > LA_HEAD) {
                            const float anchor = x - LA_HEAD;
                            f = ex2(m[i] - anchor);
                            m[i] = anchor;
                            l[i] *= f;
                        }
                        if ((lane & 3) == 0) S.factor[ra + 8 * i] = f;
                    }
                    if (j > 0) {
                        bar_wait(&S.abort, a.hdr, &S.pv_done[done.i], done.round);
                        tc_after();
                        sm_any(false);
                        for (int d = 0; d < LAT / 128; ++d)
                            for (int c = 0; c < a.nr; c += 16) {
                                uint32_t o[16];
                                tm_ld16(lane_base + TM_O + 64 * d + c, o);
#pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * S.factor[c + x]);
                                tm_st16(lane_base + TM_O + 64 * d + c, o);
                            }
                        tm_wait_st();
                    }
                }
                if (active) {
                    const uint32_t to = sp + s_at.i * p_bytes + (ra >> 3) * 1024 + (ra & 7) * 128 + 4 * (lane & 3);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float ms = m[i] == -INFINITY ? 0.0f : m[i];
                        float sum[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int k = 0; k < NG; ++k) {
                            const float e0 = ex2(s[4 * k + 2 * i] - ms), e1 = ex2(s[4 * k + 2 * i + 1] - ms);
                            sum[k & 1] += e0 + e1;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 1024 * i + ((k ^ (ra & 7)) << 4)), "r"(half2_bits(e0, e1))
                                         : "memory");
                        }
                        l[i] += sum[0] + sum[1];
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&S.p_full[s_at.i]);
            }
            // ---- the segment's rows: to the output, or as a part of them
            const bool whole = g.step == 0 && g.cnt == g.s.steps, last = g.step + g.cnt == g.s.steps;
            const int out_row = g.s.first * a.H + row0;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (g.step == 0 ? 1 : 0);
            if (nt > 0) bar_wait(&S.abort, a.hdr, &S.pv_done[done.i], done.round);
            tc_after();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int r = ra + 8 * i;
                if (!valid[i] || (lane & 3) != 0) continue;
                if (whole) {
                    S.factor[r] = sum == 0.0f ? 0.0f : 1.0f / sum;
                    if (a.lse != nullptr) a.lse[out_row + r] = sum == 0.0f ? -INFINITY : (m[i] + log2f(sum)) * KVQ_LN2;
                } else {
                    a.ml[slot * a.nr + r] = make_float2(m[i], sum);
                    if (last && g.item < a.items) {   // (more only where q_starts is not ascending)
                        const int c0 = (g.at - g.step) / S.per;
                        a.cuts[(int64_t)g.item * a.nr + r] = make_int4(c0 + 1, (int)blockIdx.x - c0 + 1, out_row + r, 0);
                    }
                }
            }
            sm_any(false);
            if (nt > 0 && !aborted(&S.abort)) {
                const int dim = 32 * warp + lane;
                for (int c = 0; c < rows; c += 16) {
                    float* part = a.part + (slot * a.nr + c) * LAT + dim;
                    uint16_t* out = a.out + (int64_t)(out_row + c) * LAT + dim;
                    const int n = min(16, rows - c);
#pragma unroll
                    for (int d = 0; d < LAT / 128; ++d) {
                        uint32_t o[16];
                        tm_ld16(lane_base + TM_O + 64 * d + c, o);
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            if (x >= n) break;
                            if (whole)
                                out[x * LAT + 128 * d] = kvq_f2h(__uint_as_float(o[x]) * S.factor[c + x]);
                            else
                                part[x * LAT + 128 * d] = __uint_as_float(o[x]);
                        }
                    }
                }
            }
            tc_before();   // (O^T is read before the next segment's first weights are handed over)
        } while (g.next(a));
    }
    __syncwarp();
    __syncthreads();
    if (*(volatile int32_t*)&S.abort) drain_after_abort(warp == 4 && lane == 0, &S.drain);
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 4)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
}

// ---------------------------------------------------------------- many query rows: pairs of CTAs
//
// 128 query rows, 64 per CTA, and 64 tokens per step.  S = Q K^T is one product of both (M = 128, N = 64): a CTA stages
// its rows' queries and the keys of half of the tokens.  O = P V keeps its rows as they are (M = 128, N = 256, twice): a
// CTA stages half of the 512 values of all tokens, so that O takes 256 of its TMEM columns (a CTA of a pair keeps 64 rows
// of M = 128 in 128 lanes: lanes 64 and up have the second half of the columns).  Half a token's values is thus staged
// twice, since one descriptor serves both CTAs, and at different places they cannot read it.
//
// Rank 1's weights (and its values, zeroed rows and reads of TMEM) are handed to rank 0 in three steps, each ordered: its
// softmax warps arrive at a barrier of their own CTA, one lane there (warp 4's) waits for them and arrives at rank 0's
// with a release to the cluster, and rank 0's issuing lane waits with an acquire.  The release takes some 2000 cycles, so S
// is two steps ahead of O; in the softmax warps themselves, it would hold them up (five drafted tokens as below 233 us; by
// the lane with S one step ahead 178 us).
//
// Bound: the shared-memory reads of the products, 128 bytes per cycle: 24 cycles for each of the 36 products of S, 64 for
// each of the eight of O, 1376 per step; and the way of the weights: a place of theirs is written, handed over, read and
// free again in two steps.  Two stages of keys and of values fit beside 64 rows of queries,
// too few for the latency of HBM, which L2 takes up (three steps ahead).  Five drafted tokens of eight sequences of
// 12001 to 16384 tokens, 128 heads: 152 us, 1.02 PFLOP/s, of which the join 12 us.
constexpr int LB_KEYS = 64;
constexpr int LB_K = LB_KEYS / 2 * ROW * 2;      // bytes of a CTA's keys of a step
constexpr int LB_V = LB_KEYS * LAT;              // and of its values (two bytes each, half of them)
constexpr int LB_V_GROUP = 4 * 1024;             // eight rows of its four chunks
constexpr int LB_NS = 2;
constexpr int LB_NT = 224;                       // softmax 0-3, products 4, keys 5, values 6
constexpr int LB_FAR = 3;                        // steps that keys are brought into L2 ahead of their load
constexpr int LB_Q = 64 * ROW * 2, LB_P = 64 * 128;
constexpr int LB_SMEM = 1024 + LB_Q + LB_NS * (LB_K + LB_V) + 2 * LB_P;

struct SharedPair {
    uint64_t q_full, q_free, k_full[LB_NS], k_empty[LB_NS], v_full[LB_NS], v_empty[LB_NS], s_full[3], p_full[2], p_here[2], pv_done[2];
    uint32_t tmem;
    int32_t abort, per;
    Segment<LB_KEYS> seg;
    float half[128];      // what the two threads of a row have to tell one another
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(LB_NT, 1)
    latent_pair_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ LatArgs a) {
    extern __shared__ unsigned char raw[];
    __shared__ SharedPair S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    if (tid == 64) map_prefetch(&map_q), map_prefetch(&map_k), map_prefetch(&map_v);
    const int pair = blockIdx.x >> 1;
    const uint32_t sq = (saddr(raw) + 1023) & ~1023u, sk = sq + LB_Q, sv = sk + LB_NS * LB_K, sp = sv + LB_NS * LB_V;
    // (what does not read global memory goes before the wait for the launch before)
    if (tid == 32) {
        bar_init(&S.q_full, 1);
        bar_init(&S.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&S.k_full[i], 1);
            bar_init(&S.k_empty[i], 1);
            bar_init(&S.v_full[i], 1);
            bar_init(&S.v_empty[i], 1);
            bar_init(&S.p_full[i], 4 + 1);   // rank 0: its softmax warps, and the other CTA's by one lane
            bar_init(&S.p_here[i], 4);       // rank 1: its softmax warps
            bar_init(&S.pv_done[i], 1);
        }
        for (int i = 0; i < 3; ++i) bar_init(&S.s_full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem)), "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    cluster_sync();   // (both CTAs' barriers and TMEM are there)
    tc_after();
    kvq_pdl_begin();
    if (warp == 0) {
        int per;
        const Segment<LB_KEYS> g = first_segment<LB_KEYS>(a, pair, gridDim.x >> 1, &per);
        if (lane == 0) S.seg = g, S.per = per, S.abort = 0;
    }
    __syncthreads();
    const uint32_t tmem = S.tmem;
    Segment<LB_KEYS> g = S.seg;

    if (g.b < 0) {
        // no work for this pair
    } else if (warp == 5) {
        // ---- queries and keys: they signal rank 0, which issues the products.  Two stages are too few for the latency of
        // HBM, so a step's pages are brought into L2 LB_FAR steps before
        const int nowhere = (int)(a.num_blocks * (PG / 8));   // a group of rows behind the pool: zeros
        Place st;
        int loaded = 0;
        bool ok = true;
        for (int seg = 0; ok;) {
            // lanes 0 and 1 look up one of this CTA's two pages of a step each
            const auto group_of = [&](int j) {
                const int lp = (g.step + j) * (LB_KEYS / PG) + 2 * (int)rank + lane;
                if (j >= g.nt || lane >= 2 || lp * PG >= g.end) return nowhere;
                const int32_t page = a.bt[(int64_t)g.b * a.max_blocks + lp];
                if (page >= 0 && page < a.num_blocks) return page * (PG / 8);
                kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
                return nowhere;
            };
            int y[LB_FAR + 1];   // of the steps j .. j + LB_FAR
#pragma unroll
            for (int k = 0; k <= LB_FAR; ++k) y[k] = group_of(k);
            if (g.nt > 0) {
                if (seg > 0) bar_wait(&S.abort, a.hdr, &S.q_free, (seg - 1) & 1);
                ok = !aborted(&S.abort);
                if (ok && elect()) {
                    if (rank == 0) bar_expect(&S.q_full, 2 * LB_Q);
                    tma_3d_pair(sq, &map_q, 0, g.s.first * a.H + g.group * a.nr + 64 * (int)rank, 0, saddr_in(&S.q_full, 0));
                }
                __syncwarp();
                ++seg;
            }
            for (int j = 0; j < g.nt && ok; ++j, ++loaded) {
                const int pages = min(LB_KEYS / PG, (g.end - (g.step + j) * LB_KEYS + PG - 1) / PG);
                int to[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) to[k] = __shfl_sync(0xffffffffu, y[0], k);
                if (loaded >= LB_NS) bar_wait(&S.abort, a.hdr, &S.k_empty[st.i], st.round ^ 1);
                ok = !aborted(&S.abort);
                if (ok && elect()) {
                    if (rank == 0) bar_expect(&S.k_full[st.i], pages * PG * ROW * 2);
                    const uint32_t bar = saddr_in(&S.k_full[st.i], 0);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (2 * (int)rank + k < pages) tma_page_pair(sk + st.i * LB_K + k * (PG * ROW * 2), &map_k, to[k], bar);
                }
                __syncwarp();
                if (y[LB_FAR] != nowhere && lane < 2) tma_page_prefetch(&map_k, y[LB_FAR]);
#pragma unroll
                for (int k = 0; k < LB_FAR; ++k) y[k] = y[k + 1];
                y[LB_FAR] = group_of(j + 1 + LB_FAR);
                st.next(LB_NS);
            }
            if (!g.next(a)) break;
        }
    } else if (warp == 6) {
        // ---- values: they stay within the CTA
        const int nowhere = (int)(a.num_blocks * (PG / 8));
        Place st;
        int loaded = 0;
        for (bool ok = true; ok;) {
            const auto group_of = [&](int j) {   // (what is no page the keys' warp flags)
                const int lp = (g.step + j) * (LB_KEYS / PG) + lane;
                if (j >= g.nt || lane >= LB_KEYS / PG || lp * PG >= g.end) return nowhere;
                const int32_t page = a.bt[(int64_t)g.b * a.max_blocks + lp];
                return page >= 0 && page < a.num_blocks ? page * (PG / 8) : nowhere;
            };
            int y = group_of(0);
            for (int j = 0; j < g.nt && ok; ++j, ++loaded) {
                const int pages = min(LB_KEYS / PG, (g.end - (g.step + j) * LB_KEYS + PG - 1) / PG);
                int to[LB_KEYS / PG];
#pragma unroll
                for (int k = 0; k < LB_KEYS / PG; ++k) to[k] = __shfl_sync(0xffffffffu, y, k);
                if (loaded >= LB_NS) bar_wait(&S.abort, a.hdr, &S.v_empty[st.i], st.round ^ 1);
                ok = !aborted(&S.abort);
                if (ok && elect()) {
                    bar_expect(&S.v_full[st.i], pages * PG * LAT);
#pragma unroll
                    for (int k = 0; k < LB_KEYS / PG; ++k)
                        if (k < pages) tma_4d(sv + st.i * LB_V + k * (PG * LAT), &map_v, 0, 0, 4 * (int)rank, to[k], &S.v_full[st.i]);
                }
                __syncwarp();
                y = group_of(j + 1);
                st.next(LB_NS);
            }
            if (!g.next(a)) break;
        }
    } else if (warp == 4) {
        // ---- tensor cores: one lane of rank 0
        if (rank == 0 && elect()) {
            const uint32_t hi_q = (uint32_t)(smem_desc(0, 16, 1024) >> 32), hi_k = (uint32_t)(smem_desc(0, 16, LA_GROUP) >> 32),
                           hi_v = (uint32_t)(smem_desc(0, 16, LB_V_GROUP) >> 32);
            const uint32_t lq = (uint32_t)smem_desc(sq, 16, 0), lk = (uint32_t)smem_desc(sk, 16, 0),
                           lv = (uint32_t)smem_desc(sv, 1024, 0), lp = (uint32_t)smem_desc(sp, 16, 0);
            constexpr uint32_t idesc_s = idesc_f16(128, LB_KEYS), idesc_o = idesc_f16(128, 256) | KVQ_B_MN;
            const auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; };
            Place in, s, out;   // stage and buffer (of three) of the next S; stage and buffer of the next O
            const auto qk = [&] {
                bar_wait(&S.abort, a.hdr, &S.k_full[in.i], in.round);
                tc_after();
                uint32_t x = lq, y = lk + (in.i * LB_K >> 4);
                asm volatile("" : "+r"(x), "+r"(y));
#pragma unroll
                for (int c = 0; c < LA_CHUNKS; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss_pair(TM_S + s.i * (LB_KEYS / 2), desc(hi_q, x + (c * 8192 >> 4) + 2 * k),
                                    desc(hi_k, y + (c * 1024 >> 4) + 2 * k), idesc_s, c + k > 0);
                // (all products so far: where S is there, so is O of three steps before)
                tc_commit_pair(&S.s_full[s.i]);
                tc_commit_pair(&S.k_empty[in.i]);
                in.next(2);
                s.next(3);
            };
            for (int seg = 0;;) {
                if (g.nt > 0) {
                    bar_wait(&S.abort, a.hdr, &S.q_full, seg & 1);
                    ++seg;
                    qk();
                    if (g.nt > 1) qk();
                    if (g.nt <= 2) tc_commit_pair(&S.q_free);
                }
                for (int j = 0; j < g.nt; ++j) {
                    if (j + 2 < g.nt) {
                        qk();
                        if (j + 3 == g.nt) tc_commit_pair(&S.q_free);
                    }
                    bar_wait<true>(&S.abort, a.hdr, &S.p_full[out.i], out.round);
                    tc_after();
                    uint32_t y = lv + (out.i * LB_V >> 4), z = lp + (out.i * LB_P >> 4);
                    asm volatile("" : "+r"(y), "+r"(z));
#pragma unroll
                    for (int k = 0; k < LB_KEYS / 16; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mma_ss_pair(TM_O + 128 * h, desc(hi_q, z + 2 * k), desc(hi_v, y + ((k * 2 * LB_V_GROUP + h * 2048) >> 4)),
                                        idesc_o, j > 0 || k > 0);
                    tc_commit_pair(&S.v_empty[out.i]);
                    tc_commit_pair(&S.pv_done[out.i]);
                    out.next(2);
                }
                if (!g.next(a)) break;
            }
        } else if (rank == 1 && elect()) {
            // ---- hands this CTA's weights to rank 0
            const uint32_t p_full[2] = {saddr_in(&S.p_full[0], 0), saddr_in(&S.p_full[1], 0)};
            Place at;
            do {
                for (int j = 0; j < g.nt; ++j, at.next(2)) {
                    bar_wait(&S.abort, a.hdr, &S.p_here[at.i], at.round);
                    tc_after();
                    tc_before();
                    bar_arrive_in(p_full[at.i]);
                }
            } while (g.next(a));
        }
        __syncwarp();
    } else {
        // ---- softmax: thread t has half of the step's columns of row t % 64, and the same half of O's
        const uint32_t lane_base = tmem + ((uint32_t)warp << 21);   // TMEM lanes 32 warp ..
        const int r = tid & 63, half = tid >> 6;
        const bool tree = a.parents != nullptr;
        uint64_t* const handed = rank == 0 ? S.p_full : S.p_here;
        Place s_at, at, done;   // buffer of S; of the weights, and stage; `done`: the step before
        do {
            const int nt = g.nt, end = g.end, ctx = g.s.T - g.s.n;
            const int row0 = g.group * a.nr + 64 * (int)rank;   // of the sequence
            const int rows = min(64, g.s.n * a.H - row0);       // (below 1: none in this CTA)
            const bool valid = r < rows;
            uint32_t path[KVQ_TREE_WORDS] = {};
            const int tok = valid ? (int)((uint32_t)(row0 + r) / (uint32_t)a.H) : 0;
            const int cut = valid ? (tree ? ctx : ctx + tok + 1) : 0;    // every token before it is seen
            if (tree && valid) walk_path(a, g.s.first, tok, path);
            const int full = __reduce_min_sync(0xffffffffu, cut);
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < nt; ++j, done = at, at.next(2), s_at.next(3)) {
                const int t0 = (g.step + j) * LB_KEYS, c0 = t0 + 32 * half;
                bar_wait(&S.abort, a.hdr, &S.s_full[s_at.i], s_at.round);
                tc_after();
                float s[32];
                tm_ld32(lane_base + TM_S + s_at.i * (LB_KEYS / 2), reinterpret_cast<uint32_t*>(s));
#pragma unroll
                for (int c = 0; c < 32; ++c) s[c] = __fmul_rn(s[c], a.scale2);
                if (c0 + 32 > full) {   // (full: what every row of the warp sees all of)
                    uint32_t bits = below(cut - c0);
                    if (tree && valid) bits |= path_bits(path, c0 - ctx);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(bits >> c & 1)) s[c] = -INFINITY;
                }
                float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 32; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x) t4[x] = max3(t4[x], s[c + 2 * x], s[c + 2 * x + 1]);
                float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                // a first anchor, or a weight that would leave fp16's range (either thread of a row tells)
                const bool turn = sm_any(m == -INFINITY ? top > m : top - m > LA_TOP);
                if (j >= 2) bar_wait(&S.abort, a.hdr, &S.pv_done[at.i], at.round ^ 1);   // the weights' place is free
                if (turn) {
                    // one row's turn is every row's: an anchor that would have to follow later is set now
                    S.half[tid] = top;
                    sm_any(false);
                    top = fmaxf(top, S.half[tid ^ 64]);
                    float f = 1.0f;
                    if (m == -INFINITY ? top > m : top - m > LA_HEAD) {
                        const float anchor = top - LA_HEAD;
                        f = ex2(m - anchor);
                        m = anchor;
                        l *= f;
                    }
                    if (j > 0) {
                        bar_wait(&S.abort, a.hdr, &S.pv_done[done.i], done.round);
                        tc_after();
#pragma unroll 1
                        for (int c = 0; c < 256; c += 32) {
                            uint32_t o[32];
                            tm_ld32(lane_base + TM_O + c, o);
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tm_st32(lane_base + TM_O + c, o);
                        }
                        tm_wait_st();
                    }
                }
                const float ms = m == -INFINITY ? 0.0f : m;
                float sum[2] = {0.0f, 0.0f};
                const uint32_t to = sp + at.i * LB_P + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
                for (int c = 0; c < 32; c += 8) {
                    uint32_t p[4];
#pragma unroll
                    for (int x = 0; x < 8; x += 2) {
                        const float e0 = ex2(s[c + x] - ms), e1 = ex2(s[c + x + 1] - ms);
                        sum[(x >> 1) & 1] += e0 + e1;
                        p[x / 2] = half2_bits(e0, e1);
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((4 * half + (c >> 3)) ^ (r & 7)) << 4)), "r"(p[0]),
                                 "r"(p[1]), "r"(p[2]), "r"(p[3])
                                 : "memory");
                }
                l += sum[0] + sum[1];
                // the weights stand for the values' arrival, too
                bar_wait(&S.abort, a.hdr, &S.v_full[at.i], at.round);
                if (end < t0 + LB_KEYS) {
                    // rows at and behind the end may hold anything: 0 * NaN must not reach O
                    const uint32_t base = sv + at.i * LB_V;
                    const int r0 = end - t0;
                    for (int x = tid; x < (LB_KEYS - r0) * 32; x += 128) {
                        const int row = r0 + (x >> 5), c = x & 31;
                        const uint32_t z = base + (row >> 3) * LB_V_GROUP + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(z), "r"(0) : "memory");
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&handed[at.i]);
            }
            // ---- the segment's rows: to the output, or as a part of them
            const bool whole = g.step == 0 && g.cnt == g.s.steps, last = g.step + g.cnt == g.s.steps;
            const int out_row = g.s.first * a.H + row0;
            const int64_t slot = 2 * (int64_t)pair + (g.step == 0 ? 1 : 0);
            const int in_group = 64 * (int)rank + r;
            if (nt > 0) bar_wait(&S.abort, a.hdr, &S.pv_done[done.i], done.round);
            tc_after();
            S.half[tid] = l;
            sm_any(false);
            l += S.half[tid ^ 64];   // (one sum of two, whichever thread takes it)
            sm_any(false);
            const float f = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            if (valid && half == 0) {
                if (whole) {
                    if (a.lse != nullptr) a.lse[out_row + r] = l == 0.0f ? -INFINITY : (m + log2f(l)) * KVQ_LN2;
                } else {
                    a.ml[slot * a.nr + in_group] = make_float2(m, l);
                    if (last && g.item < a.items) {
                        const int p0 = (g.at - g.step) / S.per;
                        a.cuts[(int64_t)g.item * a.nr + in_group] = make_int4(p0 + 1, pair - p0 + 1, out_row + r, 0);
                    }
                }
            }
            if (nt > 0) {
                // Through the weights' place (16 KB, free until the next segment's first ones), 32 values of every thread at a
                // time, so that a warp writes whole lines: written by the rows' threads they take 10000 cycles.
                // Thread t's 16-byte pieces lie at t * 128, piece k at k ^ (t % 8).
                const bool ok = !aborted(&S.abort);
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t o[32];
                    tm_ld32(lane_base + TM_O + c, o);
                    if (whole) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            o[x] = half2_bits(__uint_as_float(o[2 * x]) * f, __uint_as_float(o[2 * x + 1]) * f);
                    }
                    const int pieces = whole ? 4 : 8;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < pieces)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sp + tid * 128 + ((k ^ (tid & 7)) << 4)), "r"(o[4 * k]),
                                         "r"(o[4 * k + 1]), "r"(o[4 * k + 2]), "r"(o[4 * k + 3])
                                         : "memory");
                    sm_any(false);
                    for (int x = tid; x < 128 * pieces; x += 128) {
                        const int t = whole ? x >> 2 : x >> 3, k = x & (pieces - 1), row = t & 63, at_dim = 256 * (t >> 6) + c;
                        if (!ok || row >= rows) continue;
                        uint4 w;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                     : "r"(sp + t * 128 + ((k ^ (t & 7)) << 4))
                                     : "memory");
                        if (whole)
                            *reinterpret_cast<uint4*>(a.out + (int64_t)(out_row + row) * LAT + at_dim + 8 * k) = w;
                        else
                            *reinterpret_cast<uint4*>(a.part + (slot * a.nr + 64 * (int)rank + row) * LAT + at_dim + 4 * k) = w;
                    }
                    sm_any(false);
                }
            }
            tc_before();   // (O is read before the next segment's first weights are handed over)
        } while (g.next(a));
    }
    __syncwarp();
    __syncthreads();
    if (*(volatile int32_t*)&S.abort) {
        // a wait gave up: this pair's own copies and products land before it ends (far above a copy's time)
        const long long began = clock64();
        while (clock64() - began < 4000000) __nanosleep(1000);
    }
    tc_before();
    __syncthreads();
    cluster_sync();   // (neither ends while the other may still signal it or read its shared memory)
    tc_after();
    if (warp == 4)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
}

// ---------------------------------------------------------------- the join of a row's parts
//
// In the order of their CTAs, so that results do not depend on the run, and the workspace is left zeroed.  A row's first
// part is its CTA's last segment, the others are their CTAs' first ones.  Weights of the parts: 2^(anchor - largest
// anchor); a part without a visible token wrote no row.  (Joined by the CTA whose part came last, the work is spread over
// too few threads: 57 us more for 40 row groups of 128 rows in three parts each.)

__device__ __forceinline__ int64_t part_slot(const LatArgs& a, int c0, int i, int r) {
    return ((int64_t)2 * (c0 + i) + (i == 0 ? 1 : 0)) * a.nr + r;
}

// A warp per row: 16 values per lane.
constexpr int LJ_NW = 8;
__global__ void __launch_bounds__(32 * LJ_NW) latent_join_kernel(const __grid_constant__ LatArgs a, int n_rows) {
    const int lane = threadIdx.x & 31, row = blockIdx.x * LJ_NW + (threadIdx.x >> 5);
    if (row >= n_rows) return;
    kvq_pdl_begin();
    const int4 cut = a.cuts[row];
    if (cut.x == 0) return;
    const int c0 = cut.x - 1, n = cut.y, r = row % a.nr;
    float mx = -INFINITY, y = 0.0f;
    float2 v = make_float2(0.0f, 0.0f);
    for (int i = lane; i < n; i += 32) {
        v = a.ml[part_slot(a, c0, i, r)];
        if (v.y != 0.0f) mx = fmaxf(mx, v.x);
    }
    mx = kvq_warp_max(mx);
    float4 o[4] = {};
    for (int i0 = 0; i0 < n; i0 += 32) {
        float f = 0.0f;
        if (i0 + lane < n) {
            float2* const at = a.ml + part_slot(a, c0, i0 + lane, r);
            if (n > 32) v = *at;
            f = v.y != 0.0f ? exp2f(v.x - mx) : 0.0f;
            y += f * v.y;
            *at = make_float2(0.0f, 0.0f);
        }
        const int m = min(32, n - i0);
#pragma unroll 4
        for (int i = 0; i < m; ++i) {
            const float4* part = reinterpret_cast<const float4*>(a.part + part_slot(a, c0, i0 + i, r) * LAT) + lane;
            const float w = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 p = part[32 * x];
                o[x].x += w * p.x, o[x].y += w * p.y, o[x].z += w * p.z, o[x].w += w * p.w;
            }
        }
    }
    // (behind the loads: a store between them would hold up the next one)
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            reinterpret_cast<float4*>(a.part + part_slot(a, c0, i, r) * LAT)[lane + 32 * x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // (every lane's sum is over its own parts, joined in one order)
    y = kvq_warp_sum(y);
    const float inv = y == 0.0f ? 0.0f : 1.0f / y;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        reinterpret_cast<uint2*>(a.out + (int64_t)cut.z * LAT)[lane + 32 * x] =
            make_uint2(half2_bits(o[x].x * inv, o[x].y * inv), half2_bits(o[x].z * inv, o[x].w * inv));
    if (lane == 0) {
        a.cuts[row] = make_int4(0, 0, 0, 0);
        if (a.lse != nullptr) a.lse[cut.z] = y == 0.0f ? -INFINITY : (mx + log2f(y)) * KVQ_LN2;
    }
}

// Few rows of many parts: a cluster of LQ CTAs per row, 128 / LQ threads per part with four values each, LQ_GR parts at a
// time.
constexpr int LQ = 4, LQ_W = 128 / LQ, LQ_GR = 16;
__global__ void __cluster_dims__(LQ, 1, 1) __launch_bounds__(LQ_W * LQ_GR) latent_join_wide_kernel(const __grid_constant__ LatArgs a) {
    __shared__ float weight[KVQ_LATENT_MAX_CTAS];
    __shared__ float4 sums[LQ_GR][LQ_W];
    const int tid = threadIdx.x, lane = tid & 31, quarter = blockIdx.x % LQ;
    int4* const cut_at = a.cuts + blockIdx.x / LQ;
    const int r = blockIdx.x / LQ % a.nr;
    kvq_pdl_begin();
    const int4 cut = *cut_at;
    if (cut.x == 0) return;   // (a cluster's CTAs read the same)
    const int c0 = cut.x - 1, n = cut.y;
    const auto part_of = [&](int i) { return reinterpret_cast<float4*>(a.part + part_slot(a, c0, i, r) * LAT) + quarter * LQ_W + tid % LQ_W; };
    if (tid < 32) {
        float mx = -INFINITY, y = 0.0f;
        for (int i = lane; i < n; i += 32) {
            const float2 v = a.ml[part_slot(a, c0, i, r)];
            if (v.y != 0.0f) mx = fmaxf(mx, v.x);
        }
        mx = kvq_warp_max(mx);
        for (int i = lane; i < n; i += 32) {
            const float2 v = a.ml[part_slot(a, c0, i, r)];
            const float f = v.y != 0.0f ? exp2f(v.x - mx) : 0.0f;
            weight[i] = f;
            y += f * v.y;
        }
        y = kvq_warp_sum(y);
        const float inv = y == 0.0f ? 0.0f : 1.0f / y;
        for (int i = lane; i < n; i += 32) weight[i] *= inv;
        if (lane == 0 && quarter == 0 && a.lse != nullptr) a.lse[cut.z] = y == 0.0f ? -INFINITY : (mx + log2f(y)) * KVQ_LN2;
    }
    __syncthreads();
    cluster_sync();   // (the others have read what is zeroed below)
    if (quarter == 0) {
        for (int i = tid; i < n; i += LQ_W * LQ_GR) a.ml[part_slot(a, c0, i, r)] = make_float2(0.0f, 0.0f);
        if (tid == 0) *cut_at = make_int4(0, 0, 0, 0);
    }
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int grp = tid / LQ_W;
#pragma unroll 8
    for (int i = grp; i < n; i += LQ_GR) {
        const float4 v = *part_of(i);
        const float f = weight[i];
        o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
    }
    for (int i = grp; i < n; i += LQ_GR) *part_of(i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    sums[grp][tid % LQ_W] = o;
    __syncthreads();
    if (grp > 0) return;
    for (int k = 1; k < LQ_GR; ++k) {
        const float4 v = sums[k][tid];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    reinterpret_cast<uint2*>(a.out + (int64_t)cut.z * LAT)[quarter * LQ_W + tid] = make_uint2(half2_bits(o.x, o.y), half2_bits(o.z, o.w));
}

struct LatPlan {
    bool pairs, whole;
    int nr, keys, ctas;   // ctas: CTAs, or pairs of them
    int64_t items, steps;   // row groups and steps of the list, at most
    size_t smem, off_ml, off_cuts, off_part, bytes;
};

// Pairs of CTAs that run at the same time on the current device (asked once per device).
int latent_pairs() {
    static std::mutex mu;
    static std::vector<int> found;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return kvq_num_sms() / 2;
    }
    std::lock_guard<std::mutex> lk(mu);
    if ((int)found.size() <= dev) found.resize(dev + 1, 0);
    if (found[dev] == 0) {
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (kvq_num_sms() / 2));
        cfg.blockDim = dim3(LB_NT);
        cfg.dynamicSmemBytes = LB_SMEM;
        if (kvq_prepare_kernel((const void*)latent_pair_kernel, LB_SMEM) != KVQ_OK ||
            cudaOccupancyMaxActiveClusters(&n, latent_pair_kernel, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            return kvq_num_sms() / 2;
        }
        found[dev] = n;
    }
    return found[dev];
}

// Fills in p, or refuses what the kernels' 32-bit numbers do not hold.  The arguments are those that check_latent_rows and
// kvq_check_max_len let through, so every product here is below 2^63.
int latent_plan(const kvq_seqs* S, int32_t n_heads, int64_t n_rows, int32_t max_new, const char* fn, LatPlan* plan) {
    LatPlan& p = *plan;
    KVQ_REQUIRE(n_rows * n_heads <= INT32_MAX - 128, KVQ_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 query rows", fn);
    const int64_t most = (int64_t)max_new * n_heads;   // query rows of a sequence
    p.pairs = most > LA_ROWS;
    p.nr = p.pairs ? 128 : std::max(16, (int)((most + 15) / 16 * 16));
    const int64_t groups = (most + p.nr - 1) / p.nr, by_rows = n_rows * n_heads / p.nr + S->batch;
    // (the batch's groups by max_new, where they are the fewer)
    p.items = std::max<int64_t>(1, S->batch > 0 && groups > by_rows / S->batch ? by_rows : S->batch * groups);
    p.keys = p.pairs ? LB_KEYS : LA_KEYS;
    const int64_t each = (S->max_len + p.keys - 1) / p.keys;
    const int at_once = std::min(p.pairs ? latent_pairs() : kvq_num_sms(), KVQ_LATENT_MAX_CTAS);
    p.steps = p.items * each;
    KVQ_REQUIRE(p.items * p.nr <= INT32_MAX / 8 && p.steps <= INT32_MAX - KVQ_LATENT_MAX_CTAS, KVQ_ERR_UNSUPPORTED,
                "%s: more than 2^31 steps (queries times max_len)", fn);
    // Few steps per row group: one CTA takes them all, since parts and their join cost more (12 sequences of 53-69 tokens, 60
    // rows each 14.1 -> 10.1 us, four of 200-300, 128 rows 16.3 -> 12.5; seven steps of 16 rows 10.7 in parts, 13.7 in one).
    p.whole = p.items <= at_once && each <= LA_WHOLE;
    const int64_t cut = std::max<int64_t>(1, std::min<int64_t>(p.steps, at_once));
    p.ctas = (int)(p.whole ? p.items : cut);
    p.smem = p.pairs ? LB_SMEM : la_smem(p.nr);
    const size_t rows = (size_t)2 * cut * p.nr;   // (of either kind, so that a workspace serves every shorter max_len)
    p.off_ml = sizeof(KvqWsHeader);
    p.off_cuts = kvq_round_up(p.off_ml + rows * sizeof(float2), 256);
    p.off_part = kvq_round_up(p.off_cuts + (size_t)p.items * p.nr * sizeof(int4), 256);
    p.bytes = kvq_round_up(p.off_part + rows * LAT * sizeof(float), 256);
    return KVQ_OK;
}

}  // namespace

extern "C" size_t kv_latent_attn_ws(const kvq_seqs* S, int32_t n_heads, int64_t n_rows, int32_t max_new) {
    static const char* fn = "kv_latent_attn_ws";
    LatPlan p;
    if (kvq_check_seqs_sizes(S, fn) || kvq_check_max_len(S, fn) || check_latent_rows(n_heads, n_rows, max_new, false, fn) ||
        latent_plan(S, n_heads, n_rows, max_new, fn, &p))
        return 0;
    return p.bytes;
}

extern "C" int kv_latent_attn(const kvq_latent* C, const kvq_seqs* S, int32_t n_heads, const uint16_t* q,
                              const int32_t* parents, const int32_t* q_starts, int64_t n_rows, int32_t max_new, float scale,
                              uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    static const char* fn = "kv_latent_attn";
    kvq_clear_error();
    int st = kvq_check_latent(C, fn);
    if (!st) st = kvq_check_seqs(S, fn);
    if (!st) st = kvq_check_max_len(S, fn);
    if (!st) st = check_latent_rows(n_heads, n_rows, max_new, parents != nullptr, fn);
    LatArgs a;
    if (!st) st = latent_scale(scale, fn, &a.scale2);
    if (st) return st;
    LatPlan p;
    st = latent_plan(S, n_heads, n_rows, max_new, fn, &p);
    if (!st) st = kvq_check_ws(ws, ws_bytes, p.bytes, fn);
    if (st) return st;
    KVQ_REQUIRE(C->num_blocks * PG <= INT32_MAX, KVQ_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows in the pool", fn);
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && q_starts && (S->block_table || S->max_len == 0), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out) & 15u) == 0, KVQ_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", fn);
    CUtensorMap map_q, map_rows, map_v;
    const uint64_t qd[3] = {64, (uint64_t)n_rows * n_heads, LA_CHUNKS}, qs[2] = {ROW * 2, 128};
    const uint32_t qb[3] = {64, (uint32_t)(p.pairs ? 64 : p.nr), LA_CHUNKS};
    const uint64_t rd[4] = {64, 8, LA_CHUNKS, (uint64_t)C->num_blocks * (PG / 8)}, rs[3] = {ROW * 2, 128, 8 * ROW * 2};
    const uint32_t rb[4] = {64, 8, LA_CHUNKS, PG / 8}, vb[4] = {64, 8, LAT / 128, PG / 8};
    st = make_map(&map_q, q, 3, qd, qs, qb, fn);
    if (!st) st = make_map(&map_rows, C->rows, 4, rd, rs, rb, fn);
    if (!st && p.pairs) st = make_map(&map_v, C->rows, 4, rd, rs, vb, fn);
    if (st) return st;
    a.bt = S->block_table, a.seq_lens = S->seq_lens, a.q_starts = q_starts, a.parents = parents;
    a.n_rows = n_rows, a.num_blocks = C->num_blocks;
    a.batch = S->batch, a.max_blocks = S->max_blocks, a.max_len = S->max_len, a.max_new = max_new, a.H = n_heads, a.whole = p.whole, a.nr = p.nr, a.items = (int)p.items;
    a.out = out, a.lse = lse, a.hdr = static_cast<KvqWsHeader*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.off_ml);
    a.cuts = reinterpret_cast<int4*>(static_cast<char*>(ws) + p.off_cuts);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_part);
    const void* const kernel = p.pairs ? (const void*)latent_pair_kernel : (const void*)latent_attn_kernel;
    st = kvq_prepare_kernel(kernel, (int)p.smem);
    if (st) return st;
    cudaError_t e = p.pairs ? kvq_launch_pdl(latent_pair_kernel, dim3(2 * p.ctas), dim3(LB_NT), p.smem, kvq_stream(stream), map_q,
                                             map_rows, map_v, a)
                            : kvq_launch_pdl(latent_attn_kernel, dim3(p.ctas), dim3(LA_NT), p.smem, kvq_stream(stream), map_q,
                                             map_rows, a);
    if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    if (p.whole || p.ctas == 1) return KVQ_OK;
    const int64_t group_rows = p.items * p.nr;
    // A cluster per row where rows are few and parts many, else a warp per row.  Both sides, one token of sequences of 1000,
    // 2000 and 8000 (time with clusters by time with warps): 16 heads, one sequence 0.27 to 0.57, eight (128 rows) 0.86 to
    // 0.93, twelve (192 rows, 12 parts) 0.95 to 0.98, thirteen 0.97 to 1.01, fourteen 1.03 to 1.06, twenty 1.08 to 1.25;
    // pairs, one and two sequences of 128 heads (256 rows) 0.54 to 0.87 and 0.87 to 1.02, three 1.03 to 1.18 (but 0.86 to 0.94
    // of 64 heads, whose groups are half empty).
    const bool wide = p.ctas > 6 && (group_rows <= 128 || (group_rows <= 256 && p.ctas >= 12 * p.items));
    e = wide
            ? kvq_launch_pdl(latent_join_wide_kernel, dim3((unsigned)group_rows * LQ), dim3(LQ_W * LQ_GR), 0, kvq_stream(stream), a)
            : kvq_launch_pdl(latent_join_kernel, dim3((unsigned)((group_rows + LJ_NW - 1) / LJ_NW)), dim3(32 * LJ_NW), 0,
                             kvq_stream(stream), a, (int)group_rows);
    if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return KVQ_OK;
}

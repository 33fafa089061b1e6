// kv_chunk_attn: attention of a run of new tokens per sequence over an fp16 layer's pages.
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
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kvq_attn_mod.cuh"

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
constexpr uint32_t CA_SPIN = 1u << 16;   // bound on the polls of one mbarrier wait
constexpr float CA_HEAD = 7.0f;          // log2 of a row's largest weight when its anchor is set
constexpr float CA_TOP = 15.99f;         // log2 of the largest weight before the anchor is set anew (fp16 ends at 2^16)
constexpr float CA_FAR = 1048576.0f;     // scores (log2) beyond which they are rounded before the anchor is taken off

// TMEM columns: S (and P over it) of the two tiles, then their O
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;

struct ChunkArgs {
    const int32_t *bt, *seq_lens, *q_starts;
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

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
// a page of one kv head: the map's dims are 64 values, 8 rows, 2 halves of a row, groups of 8 rows
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int group, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(0), "r"(group), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: start address, byte offsets between the 64-element
// blocks of a matrix whose rows run along K (`lead`), and between groups of eight rows (`group`).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t group) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(group >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// f16 x f16 -> f32, M = 128, N = 128; bit 16: B's rows run along K (V), else along N (K)
constexpr uint32_t IDESC_QK = (1u << 4) | (128u / 8 << 17) | (128u / 16 << 24);
constexpr uint32_t IDESC_PV = IDESC_QK | (1u << 16);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

#define R8(v, o) "=r"((v)[o]), "=r"((v)[o + 1]), "=r"((v)[o + 2]), "=r"((v)[o + 3]), "=r"((v)[o + 4]), "=r"((v)[o + 5]), "=r"((v)[o + 6]), "=r"((v)[o + 7])
#define W8(v, o) "r"((v)[o]), "r"((v)[o + 1]), "r"((v)[o + 2]), "r"((v)[o + 3]), "r"((v)[o + 4]), "r"((v)[o + 5]), "r"((v)[o + 6]), "r"((v)[o + 7])
// 32 columns of this thread's lane; the wait is part of the statement, so nothing reads v before it
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24)
        : "r"(addr)
        : "memory");
}
// all 128 columns of a score tile
__device__ __forceinline__ void tm_ld128(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24), R8(v, 32), R8(v, 40), R8(v, 48), R8(v, 56), R8(v, 64), R8(v, 72), R8(v, 80),
          R8(v, 88), R8(v, 96), R8(v, 104), R8(v, 112), R8(v, 120)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        W8(v, 0), W8(v, 8), W8(v, 16), W8(v, 24)
        : "memory");
}
__device__ __forceinline__ void tm_st1(uint32_t addr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// two fp32 values per instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- what a CTA works on

struct Shared {
    uint64_t q_full, kv_full[CA_NS], kv_empty[CA_NS], s_full[2], p_full[2][2], o_full[2], drain;
    uint32_t tmem;
    int32_t abort;
    int32_t item_b, item_tok;                     // sequence and first new token of this CTA
    int32_t doc_min, sink_max, lo_min, hi_max;    // over its rows
    int4 see[CA_ROWS];                            // lo, hi, doc, sink of every token
};

__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for a phase of bar.  After CA_SPIN polls it flags the timeout, and every wait of the CTA that is
// not over by then returns at once: the roles run through to their ends without waiting, on data that is
// not valid, so no step needs a branch for the failure; only the loads stop (a barrier must not be armed
// twice).  Most waits of the issuing warps find their phase done: one poll and nothing else.
__device__ __forceinline__ void bar_wait(Shared& S, KvqWsHeader* hdr, uint64_t* bar, uint32_t parity) {
    const uint32_t at = saddr(bar);
    for (uint32_t it = 0; !bar_done(at, parity); ++it) {
        if ((it & 63) != 63) continue;
        if (*(volatile int32_t*)&S.abort) return;
        if (it > CA_SPIN) {
            *(volatile int32_t*)&S.abort = 1;
            kvq_dev_flag(hdr, KVQ_DEV_TIMEOUT, (int32_t)blockIdx.x);
            return;
        }
    }
}
__device__ __forceinline__ bool aborted(Shared& S) {
    return __any_sync(0xffffffffu, *(volatile int32_t*)&S.abort != 0);
}

// Sequence b's new tokens: *first row and count; false (flagged) when its lengths do not fit the call.
__device__ __forceinline__ bool seq_rows(const ChunkArgs& a, int b, int* first, int* n) {
    *first = a.q_starts[b];
    const int64_t cnt = (int64_t)a.q_starts[b + 1] - *first;
    const int T = a.seq_lens[b];
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

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(CA_NT, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ ChunkArgs a) {
    extern __shared__ unsigned char raw[];
    __shared__ Shared S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int GQ = a.GQ, tpc = CA_ROWS / GQ, split = blockIdx.y;
    const int h = a.heads_first ? blockIdx.x % a.H : blockIdx.x / a.items;
    const int item = a.heads_first ? blockIdx.x / a.H : blockIdx.x % a.items;
    const uint32_t sq = (saddr(raw) + 1023) & ~1023u, skv = sq + 2 * CA_TILE;
    kvq_pdl_begin();
    if (warp == 0) {
        int b, tok;
        find_item(a, item, tpc, &b, &tok);
        if (lane == 0) {
            S.item_b = b, S.item_tok = tok;
            S.abort = 0;
            S.doc_min = S.lo_min = INT32_MAX;
            S.sink_max = S.hi_max = 0;
        }
    }
    __syncthreads();
    const int b = S.item_b, tok0 = S.item_tok;
    if (b < 0) return;
    const int first = a.q_starts[b], n = a.q_starts[b + 1] - first, T = a.seq_lens[b];
    const int ntok = min(tpc, n - tok0), rows = ntok * GQ;
    const int nq = rows > 128 ? 2 : 1;
    if (tid < ntok) {
        const int i = tok0 + tid;
        const KvqSee see = kvq_see(a.mod, T - n + i, T, a.mod.prefix_len ? a.mod.prefix_len[b] : 0,
                                   a.mod.doc_start ? a.mod.doc_start[first + i] : 0);
        S.see[tid] = make_int4(see.lo, see.hi, see.doc, see.sink);
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
        for (int i = 0; i < CA_NS; ++i) {
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
    if (S.doc_min < S.sink_max) a1 = S.doc_min / CA_KEYS, b1 = (S.sink_max + CA_KEYS - 1) / CA_KEYS;
    if (S.lo_min < S.hi_max) a2 = max(S.lo_min / CA_KEYS, b1), b2 = max(a2, (S.hi_max + CA_KEYS - 1) / CA_KEYS);
    const int total = b1 - a1 + b2 - a2;
    const int per = (total + a.n_splits - 1) / a.n_splits;
    const int it0 = min(total, split * per), it1 = min(total, it0 + per), nt = it1 - it0;
    const auto tile_of = [&](int it) { return it < b1 - a1 ? a1 + it : a2 + (it - (b1 - a1)); };

    // 384 threads are launched with 168 registers each: 256 * 232 + 128 * 40 is the same total
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 9 && nt > 0) {
            // ---- loads
            if (lane == 0) {
                bar_expect(&S.q_full, nq * CA_TILE);
                for (int i = 0; i < nq; ++i)
                    for (int c = 0; c < 2; ++c)
                        tma_3d(sq + i * CA_TILE + c * CA_HALF, &map_q, 64 * c, h * GQ, first + tok0 + i * (128 / GQ), &S.q_full);
            }
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
                        const int4 e = S.see[k];
                        const int p0 = t * (CA_KEYS / PG);
                        if (e.x < e.y) bits |= below((e.y + PG - 1) / PG - p0) & ~below(e.x / PG - p0);
                        if (e.z < e.w) bits |= below((e.w + PG - 1) / PG - p0) & ~below(e.z / PG - p0);
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
                if (slot >= CA_NS) bar_wait(S, a.hdr, &S.kv_empty[st], ((slot / CA_NS) & 1) ^ 1);
                const bool ok = !aborted(S);
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
        if (warp == 8 && nt > 0) {
            // ---- tensor cores.  The whole warp walks the loop and one elected lane issues, so that the
            // descriptors stay in uniform registers.  All 512 TMEM columns are this CTA's, so they start at
            // column 0.  A descriptor is its low word plus constants: the low words are made opaque in every
            // step, or the compiler keeps all 64 of a step's descriptors in (spilled) registers, and the
            // reloads hold up every product (110 instead of 64 cycles each).
            const uint32_t hi_q = (uint32_t)(smem_desc(0, 16, 1024) >> 32), hi_kv = (uint32_t)(smem_desc(0, 16, 2048) >> 32);
            const uint32_t lq = (uint32_t)smem_desc(sq, 16, 0), lk = (uint32_t)smem_desc(skv, 16, 0),
                           lv = (uint32_t)smem_desc(skv, 1024, 0);
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
            bar_wait(S, a.hdr, &S.q_full, 0);
            bar_wait(S, a.hdr, &S.kv_full[0], 0);
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
                    bar_wait(S, a.hdr, &S.p_full[i][0], j & 1);
                    tc_after();
                    pv(i, sv, 0, j > 0);
                    bar_wait(S, a.hdr, &S.p_full[i][1], j & 1);
                    tc_after();
                    pv(i, sv, 1, true);
                    if (i == nq - 1) commit(&S.kv_empty[sv]);
                    if (more) {
                        if (i == 0) bar_wait(S, a.hdr, &S.kv_full[sk], ((2 * j + 2) / CA_NS) & 1);
                        qk(i, sk);
                    } else {
                        commit(&S.o_full[i]);
                    }
                }
                if (more) commit(&S.kv_empty[sk]);
            }
        }
    } else {
        // ---- softmax: thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int i = warp >> 2, r = tid;   // row of the CTA
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);  // TMEM lanes 32 (warp % 4) ..
        const uint32_t ts = lane_base + TM_S + 128 * i, to = lane_base + TM_O + 128 * i;
        const bool valid = r < rows;
        const int tok = r / GQ;
        int4 see = make_int4(0, 0, 0, 0);
        int maxlo = 0, minhi = INT32_MAX;   // over the warp's rows: tiles between need no mask
        if (valid) {
            see = S.see[tok];
            maxlo = see.x, minhi = see.y;
        }
        maxlo = __reduce_max_sync(0xffffffffu, maxlo);
        minhi = __reduce_min_sync(0xffffffffu, minhi);
        const int pos = T - n + tok0 + tok;
        const float slope2 = BIAS && valid ? a.mod.slopes[h * GQ + r % GQ] * KVQ_LOG2E : 0.0f;
        float m = valid ? -INFINITY : INFINITY, l = 0.0f;   // (no row: weights 0, never a new anchor)
        if (i < nq) {
            for (int j = 0; j < nt; ++j) {
                const int t0 = tile_of(it0 + j) * CA_KEYS;
                // rows at and behind T may hold anything: 0 * NaN must not reach O
                const bool tail = T < t0 + CA_KEYS && (T & (PG - 1)) != 0 && T > t0;
                bar_wait(S, a.hdr, &S.s_full[i], j & 1);
                // tile 0's weights stand for V's arrival too (its products are issued after these waits, and tile
                // 1's after tile 0's): the issuing warp is the busier one.  1.38 -> 1.36 ms for the prompt
                if (i == 0) bar_wait(S, a.hdr, &S.kv_full[(2 * j + 1) % CA_NS], ((2 * j + 1) / CA_NS) & 1);
                if (tail) {
                    bar_wait(S, a.hdr, &S.kv_full[(2 * j + 1) % CA_NS], ((2 * j + 1) / CA_NS) & 1);
                    const uint32_t base = skv + (2 * j + 1) % CA_NS * CA_TILE;
                    const int r0 = T - t0, r1 = (r0 + PG - 1) / PG * PG;
                    for (int x = tid & 127; x < (r1 - r0) * 16; x += 128) {
                        const int row = r0 + (x >> 4);
                        const uint32_t at = base + (row >> 3) * 2048 + (x & 1) * 1024 + (row & 7) * 128 + ((x >> 1) & 7) * 16;
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
                    if (a.mod.prefix_len == nullptr) {
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
                        const uint32_t bits = columns(see.x - t0, see.y - t0, w) | columns(see.z - t0, see.w - t0, w);
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
                        return (columns(see.x - t0, see.y - t0, c >> 5) | columns(see.z - t0, see.w - t0, c >> 5)) >> (c & 31) & 1;
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
            if (nt > 0) bar_wait(S, a.hdr, &S.o_full[i], 0);
            if (!aborted(S)) {
                tc_after();
                const int64_t out_row = (int64_t)(first + tok0 + tok) * a.H * GQ + h * GQ + r % GQ;
                const int64_t part_row = (((int64_t)item * a.H + h) * a.n_splits + split) * CA_ROWS + r;
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
                        uint4* dst = reinterpret_cast<uint4*>(a.part + part_row * D + c);
#pragma unroll
                        for (int x = 0; x < 32; x += 4) dst[x / 4] = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + c);
                        uint32_t w[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            w[x] = half2_bits(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
#pragma unroll
                        for (int x = 0; x < 16; x += 4) dst[x / 4] = make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
                    }
                }
                if (valid && a.n_splits > 1) a.ml[part_row] = make_float2(m, l);
                if (valid && a.n_splits == 1 && a.lse != nullptr)
                    a.lse[out_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * KVQ_LN2;
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (*(volatile int32_t*)&S.abort) {
        // a wait gave up: let this CTA's own copies and products land (again with a limit) before it ends
        if (warp == 8 && lane == 0) {
            tc_commit(&S.drain);
            for (uint32_t it = 0; it < CA_SPIN && !bar_done(saddr(&S.drain), 0); ++it) {}
        }
        const long long began = clock64();
        while (clock64() - began < 2000000) __nanosleep(1000);  // about a millisecond: far above a copy's time
        __syncthreads();
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
}

// Joins the splits of an item's rows, a warp per row, in their order, and leaves the workspace zeroed.
constexpr int CJ_NW = 8;
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
    float mx = -INFINITY;
    for (int s = lane; s < a.n_splits; s += 32) mx = fmaxf(mx, a.ml[p0 + (int64_t)s * CA_ROWS].x);
    mx = kvq_warp_max(mx);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float y = 0.0f;
#pragma unroll 8
    for (int s = 0; s < a.n_splits; ++s) {
        const int64_t row = p0 + (int64_t)s * CA_ROWS;
        const float2 v = a.ml[row];
        const float4 w = reinterpret_cast<const float4*>(a.part + row * D)[lane];
        const bool some = v.y != 0.0f;   // (a split without a visible token wrote no row)
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
    for (int s = lane; s < a.n_splits; s += 32) a.ml[p0 + (int64_t)s * CA_ROWS] = make_float2(0.0f, 0.0f);
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
// parts 62 us).
ChunkPlan chunk_plan(const kvq_layout* L, const kvq_seqs* S, int64_t n_rows, int32_t max_new) {
    ChunkPlan p;
    const int GQ = L->n_q_heads / L->n_kv_heads, tpc = CA_ROWS / GQ;
    const int64_t by_max = S->batch * (((int64_t)max_new + tpc - 1) / tpc);
    p.items = std::max<int64_t>(1, std::min(by_max, n_rows / tpc + S->batch));
    const int64_t ctas = p.items * L->n_kv_heads, sms = kvq_num_sms();
    const int tiles = (S->max_len + CA_KEYS - 1) / CA_KEYS;
    p.n_splits = 1;
    if (ctas < sms) {
        const int most = (int)std::min<int64_t>(std::max(1, tiles / 4), 4 * sms / ctas);
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

// A tensor map of fp16 values in boxes whose innermost extent is 64 values, 128-byte swizzle.
int make_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
             const char* fn) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static std::atomic<Encode> found_encode{nullptr};   // (threads that make the first call together each look it up)
    Encode encode = found_encode.load(std::memory_order_relaxed);
    if (encode == nullptr) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || f == nullptr) {
            cudaGetLastError();
            return kvq_fail(KVQ_ERR_CUDA, "%s: the driver has no cuTensorMapEncodeTiled", fn);
        }
        encode = reinterpret_cast<Encode>(f);
        found_encode.store(encode, std::memory_order_relaxed);
    }
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const auto fill = [&] {
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void*>(base),
                      reinterpret_cast<const cuuint64_t*>(dims), reinterpret_cast<const cuuint64_t*>(strides), box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = fill();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // the thread has made no runtime call yet that makes its device's context current, as a launch would
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = fill();
    }
    if (r != CUDA_SUCCESS) return kvq_fail(KVQ_ERR_CUDA, "%s: tensor map (%d)", fn, (int)r);
    return KVQ_OK;
}

}  // namespace

extern "C" size_t kv_chunk_attn_ws(const kvq_layout* L, const kvq_seqs* S, int64_t n_rows, int32_t max_new) {
    if (kvq_check_layout(L, "kv_chunk_attn_ws", true) || kvq_check_seqs_sizes(S, "kv_chunk_attn_ws") ||
        kvq_check_max_len(S, "kv_chunk_attn_ws") || check_rows(n_rows, max_new, "kv_chunk_attn_ws"))
        return 0;
    return chunk_plan(L, S, n_rows, max_new).bytes;
}

extern "C" int kv_chunk_attn(const kvq_layout* L, const kvq_pool* P, const kvq_seqs* S, const uint16_t* q,
                             const int32_t* q_starts, int64_t n_rows, int32_t max_new, const kvq_attn_mod* mod,
                             uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    static const char* fn = "kv_chunk_attn";
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
    st = check_rows(n_rows, max_new, fn);
    if (st) return st;
    ChunkArgs a;
    st = kvq_mod_args(mod, fn, &a.mod);
    if (st) return st;
    const ChunkPlan p = chunk_plan(L, S, n_rows, max_new);
    st = kvq_check_ws(ws, ws_bytes, p.bytes, fn);
    if (st) return st;
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && q_starts && (S->block_table || S->max_len == 0), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out | (uintptr_t)P->k16 | (uintptr_t)P->v16) & 15u) == 0,
                KVQ_ERR_INVALID_ARG, "%s: q, out, k16 and v16 must be 16-byte aligned", fn);
    KVQ_REQUIRE(p.items * L->n_kv_heads <= INT32_MAX, KVQ_ERR_UNSUPPORTED, "%s: n_rows", fn);
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
    a.bt = S->block_table, a.seq_lens = S->seq_lens, a.q_starts = q_starts;
    a.batch = S->batch, a.max_blocks = S->max_blocks, a.max_len = S->max_len, a.max_new = max_new;
    a.H = H, a.GQ = GQ, a.n_splits = p.n_splits;
    a.n_rows = n_rows;
    a.out = out, a.lse = lse;
    a.hdr = static_cast<KvqWsHeader*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.off_ml);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_part);
    a.items = (int32_t)p.items;
    // The longest groups come first.  In a few waves, the heads' long groups run side by side, or the last
    // head's would start late (packed documents: 92 -> 82 us); in many waves one head after the other, so
    // that all CTAs read the same K and V (a 16384-token prompt: 1.38 instead of 1.42 ms).
    a.heads_first = p.items * H <= 6 * (int64_t)kvq_num_sms();
    const dim3 grid((unsigned)(p.items * H), p.n_splits);
    const auto go = [&](auto kernel) {
        const int rc = kvq_prepare_kernel((const void*)kernel, CA_SMEM);
        if (rc) return rc;
        cudaError_t e = kvq_launch_pdl(kernel, grid, dim3(CA_NT), CA_SMEM, kvq_stream(stream), map_q, map_k, map_v, a);
        if (e == cudaSuccess && p.n_splits > 1)
            e = kvq_launch_pdl(chunk_join_kernel, dim3((unsigned)p.items, H, CA_ROWS / CJ_NW), dim3(32 * CJ_NW), 0, kvq_stream(stream), a);
        if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
        return (int)KVQ_OK;
    };
    const bool cap = a.mod.post != 0.0f, bias = a.mod.slopes != nullptr;
    if (cap) return bias ? go(chunk_attn_kernel<true, true>) : go(chunk_attn_kernel<true, false>);
    return bias ? go(chunk_attn_kernel<false, true>) : go(chunk_attn_kernel<false, false>);
}

// kv_decode_attn: attention of one new token per sequence over an fp16 layer's pages, split over the
// cache's length and joined.
//
// Bound: bytes.  Every visible K and V row is read once for the H_q/H_kv <= 8 query heads of its kv head,
// 8 flop per byte at most, so both products run on mma.sync m16n8k16 fragments that come straight from
// global memory in 16-byte loads, without shared memory:
//   S^T = K q^T   A = 16 tokens of a page, B = the group's query heads as the 8 columns.  A sum over
//                 channels may take them in any order, so lane (g, t) holds the 16-byte chunks t, t+4,
//                 t+8, t+12 of token g (and g + 8) and the query's fragments use the same order.
//   O^T = V^T p   A = 16 dims x 16 tokens.  Lane (g, t) loads chunks g and g + 8 of tokens 2t, 2t+1, 2t+8,
//                 2t+9; a byte permute pairs neighbouring tokens, and row g of product j is dim 8g + j.
//                 p enters as two fp16 halves, against exact fp16 V; sums are fp32.  The halves are taken of
//                 2^15 p, so that both use fp16's whole range: p is off by 2^-22 of itself down to 2^-18 of the
//                 warp's largest weight, and by 2^-40 of that below.
// p^T reaches the B operand through movmatrix.  A warp owns whole pages (8 KB of loads in flight per warp,
// K of the next page issued as soon as the current one is consumed), keeps its own running maximum and
// sum, and meets the others once, at the end.
//
// Measured: sixteen sequences of 4096-32767 tokens, 32 kv heads, 720 us (6.7 TB/s, 99% of the measured copy
// rate); one of 131072 tokens, 8 kv heads, capped scores, 86 us (92%); one of 4096 tokens, 2 kv heads, 8.8
// us in a graph: two dependent loads, two or three pages per warp at about 1 us each, two cluster barriers.
#include <algorithm>

#include "kvq_attn_mod.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int PG = KVQ_BLOCK_TOKENS;
// How a (sequence, kv head) row is cut into parts and joined:
//   DA_CLUSTER  short contexts: up to 8 CTAs of DA_WIDE warps, which join through their shared memories
//   DA_TICKET   few rows: one CTA of DA_WIDE warps per SM, whose warps meet in shared memory, so that few
//               parts are left for the part that arrives last to join
//   DA_SECOND   many rows: three CTAs of DA_SLIM warps per SM, so that one CTA's loads fill another's beginning
//               and end; a second launch joins
enum { DA_SECOND = 0, DA_TICKET = 1, DA_CLUSTER = 2 };
constexpr int DA_WIDE = 12, DA_SLIM = 4;
// pages per warp up to which DA_CLUSTER is taken: where 8 CTAs leave SMs idle (4096 tokens, 2 kv heads: 9.4
// instead of 10.5 us; 8192: 13.1 instead of 11.5), and where they do not (4 x 4000 tokens, 8 kv heads: 14.0
// instead of 15.8 us)
constexpr int DA_FEW_PAGES = 4, DA_MOST_PAGES = 12;
constexpr float DA_LIFT = 32768.0f;   // the scale of the weights in the value product: the largest is 2^15
constexpr int DA_JOIN = 4;      // warps per CTA of the second launch
constexpr int DA_TICKETS = 56;  // rows whose arrivals fit the workspace header's spare words
constexpr int SO_ROW = D + 4;   // floats of a head's row in shared memory

struct DecArgs {
    const uint16_t *k16, *v16, *q;
    int64_t num_blocks;
    const int32_t *bt, *seq_lens;
    int32_t max_blocks, max_len, H, GQ;
    KvqModArgs mod;
    float *out, *lse;
    float* part;        // [B][H][n_splits][GQ][D] unnormalised outputs
    float2* ml;         // [B][H][n_splits][GQ] running maximum (log2) and sum
    KvqWsHeader* hdr;
    int32_t n_splits, pps;
    int32_t mode;       // DA_*
};

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 bits_float2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
__device__ __forceinline__ uint4 ldg_stream(const uint16_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

struct Page {
    uint4 k[8];  // token g: chunks t + 4i; then token g + 8
    uint4 v[8];  // tokens 2t, 2t+1, 2t+8, 2t+9: chunk g; then chunk g + 8
};

__device__ __forceinline__ void load_k(Page& P, const uint16_t* rows, int g, int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        P.k[i] = ldg_stream(rows + g * D + 8 * (t + 4 * i));
        P.k[4 + i] = ldg_stream(rows + (g + 8) * D + 8 * (t + 4 * i));
    }
}
__device__ __forceinline__ void load_v(Page& P, const uint16_t* rows, int g, int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
        P.v[i] = ldg_stream(rows + tok * D + 8 * g);
        P.v[4 + i] = ldg_stream(rows + tok * D + 64 + 8 * g);
    }
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// one score in the log2 domain; `away` = |i - j|
template <bool CAP, bool BIAS>
__device__ __forceinline__ float score(const KvqModArgs& m, float dot, float slope2, int away) {
    float s = CAP ? kvq_capped(m, dot) : dot * m.pre;
    if (BIAS) s = fmaf(-slope2, (float)away, s);
    return s;
}

// The pages the newest token of sequence b sees: n1 from p1 (sinks), then n2 from p2; the parts they
// are cut into.  Returns false for a length out of bounds.
struct Span {
    KvqSee see;
    int T, p1, n1, p2, n, used;
    __device__ __forceinline__ int logical(int u) const { return u < n1 ? p1 + u : p2 + (u - n1); }
};
__device__ __forceinline__ bool span_of(const DecArgs& a, int b, Span* s) {
    s->T = a.seq_lens[b];
    if (s->T < 0 || s->T > a.max_len) return false;
    s->see = KvqSee{0, 0, 0, 0};
    if (s->T > 0)
        s->see = kvq_see(a.mod, s->T - 1, s->T, a.mod.prefix_len ? a.mod.prefix_len[b] : 0,
                         a.mod.doc_start ? a.mod.doc_start[b] : 0);
    const KvqSee& e = s->see;
    s->p1 = e.doc / PG;
    s->n1 = e.sink > e.doc ? (e.sink + PG - 1) / PG - s->p1 : 0;
    s->p2 = max(e.lo / PG, s->n1 > 0 ? s->p1 + s->n1 : 0);
    s->n = s->n1 + (e.lo < e.hi ? max(0, (e.hi + PG - 1) / PG - s->p2) : 0);
    s->used = max(1, (s->n + a.pps - 1) / a.pps);
    return true;
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the value of a shared variable in the CTA of this rank of the cluster
__device__ __forceinline__ float peer(const float* p, int rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// Adds part r of a row (four dims per lane), weighted against the row's maximum.  The part is zeroed behind
// all loads (drop_part): a store between them would hold up the next one.
__device__ __forceinline__ void join_part(const DecArgs& a, int64_t r, int lane, float mx, float4* x, float* y) {
    const float2 v = __ldcg(&a.ml[r]);
    const float4 w = __ldcg(reinterpret_cast<const float4*>(a.part + r * D) + lane);
    const float f = v.x == -INFINITY ? 0.0f : exp2f(v.x - mx);
    x->x += f * w.x;
    x->y += f * w.y;
    x->z += f * w.z;
    x->w += f * w.w;
    *y += f * v.y;
}
__device__ __forceinline__ void drop_part(const DecArgs& a, int64_t r, int lane) {
    reinterpret_cast<float4*>(a.part + r * D)[lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}
__device__ __forceinline__ void finish_row(const DecArgs& a, int64_t r, int lane, float mx, float4 x, float y) {
    const float inv = y == 0.0f ? 0.0f : 1.0f / y;  // nothing visible: 0
    reinterpret_cast<float4*>(a.out + r * D)[lane] = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (a.lse != nullptr && lane == 0) a.lse[r] = y == 0.0f ? -INFINITY : (mx + log2f(y)) * KVQ_LN2;
}

template <bool CAP, bool BIAS, int DA_NW>
__global__ void __launch_bounds__(32 * DA_NW) decode_attn_kernel(DecArgs a) {
    constexpr int DA_NT = 32 * DA_NW;
    extern __shared__ __align__(16) float so[];   // [DA_NW][GQ][SO_ROW] unnormalised outputs
    __shared__ float sm[DA_NW][8], sl[DA_NW][8];
    __shared__ float cm[8], cl[8];   // the CTA's maximum and sum per head, for its cluster
    __shared__ int is_last;
    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int GQ = a.GQ, Hq = a.H * GQ;
    kvq_pdl_begin();
    // what does not depend on the length is on its way while the length is: the query's fragments (head g of
    // the group, channels in the order of the key chunks) and, where page u of the list is page u of the
    // table, this warp's first table entry
    uint4 qf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        qf[i] = g < GQ ? *reinterpret_cast<const uint4*>(a.q + ((int64_t)b * Hq + h * GQ + g) * D + 8 * (t + 4 * i))
                       : make_uint4(0, 0, 0, 0);
    const int32_t* bt = a.bt + (int64_t)b * a.max_blocks;
    const bool straight = a.mod.window == 0 && a.mod.doc_start == nullptr;
    const int64_t u_first = (int64_t)split * a.pps + warp;
    const int32_t early = straight && u_first * PG < a.max_len ? bt[u_first] : -1;
    Span sp;
    if (!span_of(a, b, &sp)) {
        if (tid == 0 && split == 0) kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return;
    }
    const bool cluster = DA_NW == DA_WIDE && a.mode == DA_CLUSTER;
    if (split >= sp.used && !cluster) return;
    const KvqSee see = sp.see;
    const int T = sp.T, u0 = split * a.pps, u1 = min(sp.n, u0 + a.pps);

    float slope[2] = {0.0f, 0.0f};
    if (BIAS) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * t + e < GQ) slope[e] = a.mod.slopes[h * GQ + 2 * t + e] * KVQ_LOG2E;
    }
    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    // rows of page u of this CTA's range; page 0 stands in for a bad id (flagged, the output is not valid)
    const auto rows_at = [&](int32_t page) -> int64_t {
        if (page < 0 || page >= a.num_blocks) {
            if (lane == 0) kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
            page = 0;
        }
        return ((int64_t)page * a.H + h) * PG * D;
    };
    const auto rows_of = [&](int u) { return rows_at(bt[sp.logical(u)]); };
    Page P;
    int u = u0 + warp;
    int64_t row = 0, next = 0;
    if (u < u1) {
        row = straight ? rows_at(early) : rows_of(u);
        load_k(P, a.k16 + row, g, t);
        load_v(P, a.v16 + row, g, t);
    }
    if (u + DA_NW < u1) next = rows_of(u + DA_NW);
    for (; u < u1; u += DA_NW) {
        // two chains of four products: half the latency, and half the sums that round
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mma16816(s, P.k[i].x, P.k[4 + i].x, P.k[i].y, P.k[4 + i].y, qf[i].x, qf[i].y);
            mma16816(s2, P.k[i].z, P.k[4 + i].z, P.k[i].w, P.k[4 + i].w, qf[i].z, qf[i].w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += s2[i];
        const bool more = u + DA_NW < u1;
        row = next;
        if (more) load_k(P, a.k16 + row, g, t);
        if (u + 2 * DA_NW < u1) next = rows_of(u + 2 * DA_NW);

        const int j0 = sp.logical(u) * PG;
        const bool whole = j0 >= see.lo && j0 + PG <= see.hi;
        const bool in0 = see(j0 + g), in1 = see(j0 + g + 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            s[e] = in0 ? score<CAP, BIAS>(a.mod, s[e], slope[e], abs(T - 1 - j0 - g)) : -INFINITY;
            s[2 + e] = in1 ? score<CAP, BIAS>(a.mod, s[2 + e], slope[e], abs(T - 1 - j0 - g - 8)) : -INFINITY;
        }
        float mn[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[e], s[2 + e]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            mn[e] = fmaxf(m[e], x);
        }
        if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = mn[e] > m[e] ? exp2f(m[e] - mn[e]) : 1.0f;
                m[e] = mn[e];
                l[e] *= f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j][e] *= f;
                    o[j][2 + e] *= f;
                }
            }
        }
        float p[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float ms = m[e] == -INFINITY ? 0.0f : m[e];   // (nothing but scores of -inf so far: weights 0)
            p[e] = in0 ? exp2f(s[e] - ms) * DA_LIFT : 0.0f;
            p[2 + e] = in1 ? exp2f(s[2 + e] - ms) * DA_LIFT : 0.0f;
            l[e] += p[e] + p[2 + e];
        }
        const uint32_t h0 = half2_bits(p[0], p[1]), h1 = half2_bits(p[2], p[3]);
        const float2 f0 = bits_float2(h0), f1 = bits_float2(h1);
        const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
        const uint32_t c0 = transpose8x8(half2_bits(p[0] - f0.x, p[1] - f0.y));
        const uint32_t c1 = transpose8x8(half2_bits(p[2] - f1.x, p[3] - f1.y));
        if (!whole) {  // rows nobody sees may hold anything, also NaN: 0 * NaN must not reach the sum
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!see(j0 + 2 * t + (i & 1) + 8 * (i >> 1))) P.v[i] = P.v[4 + i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
            const uint32_t a0 = __byte_perm(word(P.v[0], j >> 1), word(P.v[1], j >> 1), sel);
            const uint32_t a1 = __byte_perm(word(P.v[4], j >> 1), word(P.v[5], j >> 1), sel);
            const uint32_t a2 = __byte_perm(word(P.v[2], j >> 1), word(P.v[3], j >> 1), sel);
            const uint32_t a3 = __byte_perm(word(P.v[6], j >> 1), word(P.v[7], j >> 1), sel);
            mma16816(o[j], a0, a1, a2, a3, b0, b1);
            mma16816(o[j], a0, a1, a2, a3, c0, c1);
        }
        if (more) load_v(P, a.v16 + row, g, t);
    }

    // the warps' states into shared memory, their scale taken off (a power of two: exact)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= 1.0f / DA_LIFT;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] *= 1.0f / DA_LIFT;
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
        if (g == 0) {
            sm[warp][2 * t + e] = m[e];
            sl[warp][2 * t + e] = l[e];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (2 * t + e >= GQ) break;
            float* dst = so + (warp * GQ + 2 * t + e) * SO_ROW + 64 * c + 8 * g;
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4*>(dst + j) = make_float4(o[j][2 * c + e], o[j + 1][2 * c + e],
                                                                  o[j + 2][2 * c + e], o[j + 3][2 * c + e]);
        }
    }
    __syncthreads();
    const int64_t bh = (int64_t)b * a.H + h;
    for (int i = tid; i < GQ * (D / 4); i += DA_NT) {   // four dims of a head per thread
        const int e = i / (D / 4), d = 4 * (i % (D / 4));
        float mx = sm[0][e];
#pragma unroll
        for (int w = 1; w < DA_NW; ++w) mx = fmaxf(mx, sm[w][e]);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < DA_NW; ++w) {
            const float f = sm[w][e] == -INFINITY ? 0.0f : exp2f(sm[w][e] - mx);
            const float4 z = *reinterpret_cast<const float4*>(&so[(w * GQ + e) * SO_ROW + d]);
            x.x += f * z.x, x.y += f * z.y, x.z += f * z.z, x.w += f * z.w;
            y += f * sl[w][e];
        }
        if (cluster) {
            *reinterpret_cast<float4*>(&so[e * SO_ROW + d]) = x;   // (nobody else reads these elements)
            if (d == 0) cm[e] = mx, cl[e] = y;
        } else if (sp.used == 1) {
            const int64_t r = (int64_t)b * Hq + h * GQ + e;
            const float inv = y == 0.0f ? 0.0f : 1.0f / y;
            *reinterpret_cast<float4*>(a.out + r * D + d) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
            if (a.lse != nullptr && d == 0) a.lse[r] = y == 0.0f ? -INFINITY : (mx + log2f(y)) * KVQ_LN2;
        } else {
            const int64_t r = (bh * a.n_splits + split) * GQ + e;
            *reinterpret_cast<float4*>(a.part + r * D + d) = x;
            if (d == 0) a.ml[r] = make_float2(mx, y);
        }
    }
    if (cluster) {
        // every CTA takes its share of the outputs and adds up all parts, in their order
        cluster_sync();
        const int n_parts = gridDim.x;
        for (int i = split * DA_NT + tid; i < GQ * D; i += n_parts * DA_NT) {
            const int e = i / D, d = i % D;
            float mx = -INFINITY, x = 0.0f, y = 0.0f;
            float pm[8], pl[8], px[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int rank = min(s, n_parts - 1);
                pm[s] = peer(&cm[e], rank);
                pl[s] = peer(&cl[e], rank);
                px[s] = peer(&so[e * SO_ROW + d], rank);
                if (s < n_parts) mx = fmaxf(mx, pm[s]);
            }
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                if (s >= n_parts) continue;
                // (a part without a maximum holds zeros, or NaN where all that it sees is NaN: that has to show)
                const float f = pm[s] == -INFINITY ? 0.0f : exp2f(pm[s] - mx);
                x += f * px[s];
                y += f * pl[s];
            }
            const int64_t r = (int64_t)b * Hq + h * GQ + e;
            a.out[r * D + d] = y == 0.0f ? 0.0f : x / y;
            if (a.lse != nullptr && d == 0) a.lse[r] = y == 0.0f ? -INFINITY : (mx + log2f(y)) * KVQ_LN2;
        }
        cluster_sync();   // no CTA ends while another reads its shared memory
        return;
    }
    if (DA_NW != DA_WIDE || a.mode != DA_TICKET || sp.used == 1) return;
    // the part that arrives last joins the row's parts, in their order, and leaves the workspace zeroed
    __threadfence();
    __syncthreads();
    int32_t* ticket = &a.hdr->pad[bh];
    if (tid == 0) is_last = atomicAdd(ticket, 1) == sp.used - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    constexpr int MOST = DA_NW;           // DA_NW / GQ warps per head, each takes every so-many-th part
    const int per = max(1, MOST / GQ), e = warp % GQ, turn = warp / GQ;
    const int64_t first = bh * a.n_splits * GQ + e;
    float mx = -INFINITY, y = 0.0f;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (turn < per) {
        for (int s = lane; s < sp.used; s += 32) mx = fmaxf(mx, __ldcg(&a.ml[first + (int64_t)s * GQ]).x);
        mx = kvq_warp_max(mx);
#pragma unroll 8
        for (int s = turn; s < sp.used; s += per) join_part(a, first + (int64_t)s * GQ, lane, mx, &x, &y);
        for (int s = turn; s < sp.used; s += per) drop_part(a, first + (int64_t)s * GQ, lane);
        float* dst = so + (turn * GQ + e) * SO_ROW;
        reinterpret_cast<float4*>(dst)[lane] = x;
        if (lane == 0) dst[D] = y;
    }
    __syncthreads();  // also: every warp has read the maxima
    for (int64_t i = tid; i < (int64_t)sp.used * GQ; i += DA_NT) a.ml[bh * a.n_splits * GQ + i] = make_float2(0.0f, 0.0f);
    if (tid == 0) *ticket = 0;
    if (turn != 0) return;
    for (int w = 1; w < per; ++w) {
        const float* src = so + (w * GQ + e) * SO_ROW;
        const float4 z = reinterpret_cast<const float4*>(src)[lane];
        x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
        y += src[D];
    }
    finish_row(a, (int64_t)b * Hq + h * GQ + e, lane, mx, x, y);
}

// Joins the parts of one (sequence, query head) in their order and leaves the workspace zeroed.  The
// warps take every DA_JOIN-th part, so the loads of a long split list overlap.
__global__ void __launch_bounds__(32 * DA_JOIN) decode_join_kernel(DecArgs a) {
    __shared__ float4 so[DA_JOIN][32];
    __shared__ float sl[DA_JOIN];
    const int hq = blockIdx.x, b = blockIdx.y, h = hq / a.GQ, e = hq % a.GQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    kvq_pdl_begin();
    Span sp;
    if (!span_of(a, b, &sp) || sp.used == 1) return;
    const int64_t first = (((int64_t)b * a.H + h) * a.n_splits) * a.GQ + e;
    float mx = -INFINITY;
    for (int s = lane; s < sp.used; s += 32) mx = fmaxf(mx, a.ml[first + (int64_t)s * a.GQ].x);
    mx = kvq_warp_max(mx);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float y = 0.0f;
#pragma unroll 4
    for (int s = warp; s < sp.used; s += DA_JOIN) join_part(a, first + (int64_t)s * a.GQ, lane, mx, &x, &y);
    for (int s = warp; s < sp.used; s += DA_JOIN) drop_part(a, first + (int64_t)s * a.GQ, lane);
    so[warp][lane] = x;
    if (lane == 0) sl[warp] = y;
    __syncthreads();  // also: every warp has read the maxima
    for (int s = threadIdx.x; s < sp.used; s += 32 * DA_JOIN) a.ml[first + (int64_t)s * a.GQ] = make_float2(0.0f, 0.0f);
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < DA_JOIN; ++w) {
        const float4 z = so[w][lane];
        x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
        y += sl[w];
    }
    finish_row(a, (int64_t)b * a.H * a.GQ + hq, lane, mx, x, y);
}

struct DecPlan {
    int n_splits, pps, mode;
    size_t off_ml, off_part, bytes;
};

// Splits by size alone.  Short contexts: a cluster per row, as many CTAs as there are SMs per row, 8 at most.
// Few rows whose work is either one sequence (equal parts) or not long: as many parts as there are SMs per
// row, one wave.  Else parts of equal pages, small enough for about eight waves, so that the long sequences
// of a batch do not finish alone, with 8 pages per warp at least.
DecPlan dec_plan(const kvq_layout* L, const kvq_seqs* S) {
    DecPlan p;
    const int H = L->n_kv_heads, GQ = L->n_q_heads / H, B = std::max(S->batch, 1);
    const int pages = std::max(1, (S->max_len + PG - 1) / PG);
    const int64_t rows = (int64_t)B * H, sms = kvq_num_sms();
    const int ctas = (int)std::min<int64_t>({8, std::max<int64_t>(1, sms / rows), (pages + DA_WIDE - 1) / DA_WIDE});
    const auto up = [](int64_t x, int64_t m) { return (x + m - 1) / m * m; };
    if (rows <= sms && pages <= ctas * DA_WIDE * (sms / rows > 8 ? DA_FEW_PAGES : DA_MOST_PAGES)) {
        p.mode = DA_CLUSTER;
        p.pps = (int)up((pages + ctas - 1) / ctas, DA_WIDE);
    } else if (rows <= DA_TICKETS && (B == 1 || rows * pages <= 16 * DA_WIDE * sms)) {
        const int64_t want = std::max<int64_t>(1, sms / rows);
        p.mode = DA_TICKET;
        p.pps = (int)up((pages + want - 1) / want, DA_WIDE);
    } else {
        const int64_t slots = 3 * sms, want = std::max<int64_t>(1, (rows <= slots ? slots : 8 * slots) / rows);
        p.mode = DA_SECOND;
        p.pps = (int)up(std::max<int64_t>((pages + want - 1) / want, 8 * DA_SLIM), DA_SLIM);
    }
    p.n_splits = (pages + p.pps - 1) / p.pps;
    const size_t parts = p.n_splits > 1 && p.mode != DA_CLUSTER ? (size_t)rows * p.n_splits * GQ : 0;
    p.off_ml = sizeof(KvqWsHeader);
    p.off_part = kvq_round_up(p.off_ml + parts * sizeof(float2), 256);
    p.bytes = kvq_round_up(p.off_part + parts * D * sizeof(float), 256);
    return p;
}

}  // namespace

extern "C" size_t kv_decode_attn_ws(const kvq_layout* L, const kvq_seqs* S) {
    if (kvq_check_layout(L, "kv_decode_attn_ws", true) || kvq_check_seqs_sizes(S, "kv_decode_attn_ws") ||
        kvq_check_max_len(S, "kv_decode_attn_ws"))
        return 0;
    return dec_plan(L, S).bytes;
}

extern "C" int kv_decode_attn(const kvq_layout* L, const kvq_pool* P, const kvq_seqs* S, const uint16_t* q,
                              const kvq_attn_mod* mod, float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    static const char* fn = "kv_decode_attn";
    kvq_clear_error();
    int st = kvq_check_layout(L, fn, true);
    if (st) return st;
    KVQ_REQUIRE(L->bits == 16, KVQ_ERR_UNSUPPORTED, "%s: bits %d (an fp16 layer)", fn, L->bits);
    st = kvq_check_seqs(S, fn);
    if (!st) st = kvq_check_max_len(S, fn);
    if (st) return st;
    KVQ_REQUIRE(P && P->k16 && P->v16 && P->num_blocks > 0, KVQ_ERR_INVALID_ARG, "%s: pool needs k16 and v16", fn);
    KVQ_REQUIRE(S->batch <= 65535 && L->n_kv_heads <= 65535, KVQ_ERR_UNSUPPORTED, "%s: batch or heads", fn);
    DecArgs a;
    st = kvq_mod_args(mod, fn, &a.mod);
    if (st) return st;
    const DecPlan p = dec_plan(L, S);
    st = kvq_check_ws(ws, ws_bytes, p.bytes, fn);
    if (st) return st;
    if (S->batch == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && (S->block_table || S->max_len == 0), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out | (uintptr_t)P->k16 | (uintptr_t)P->v16) & 15u) == 0,
                KVQ_ERR_INVALID_ARG, "%s: q, out, k16 and v16 must be 16-byte aligned", fn);
    a.k16 = P->k16, a.v16 = P->v16, a.q = q;
    a.num_blocks = P->num_blocks;
    a.bt = S->block_table, a.seq_lens = S->seq_lens;
    a.max_blocks = S->max_blocks, a.max_len = S->max_len;
    a.H = L->n_kv_heads, a.GQ = L->n_q_heads / L->n_kv_heads;
    a.out = out, a.lse = lse;
    a.hdr = static_cast<KvqWsHeader*>(ws);
    a.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.off_ml);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_part);
    a.n_splits = p.n_splits, a.pps = p.pps;
    const dim3 grid(p.n_splits, L->n_kv_heads, S->batch);
    const bool cap = a.mod.post != 0.0f, bias = a.mod.slopes != nullptr;
    a.mode = p.mode;
    const int nw = p.mode == DA_SECOND ? DA_SLIM : DA_WIDE;
    const auto go = [&](auto kernel) {
        // the two halves of a 128-byte line are asked for by neighbouring loads: with the smallest L1 the
        // second one goes out again (948 instead of 732 us for sixteen sequences of 4K-32K)
        const int rc = kvq_prepare_kernel((const void*)kernel, nw * 8 * SO_ROW * (int)sizeof(float), true);
        if (rc) return rc;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(32 * nw);
        cfg.dynamicSmemBytes = (size_t)nw * a.GQ * SO_ROW * sizeof(float);
        cfg.stream = kvq_stream(stream);
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {(unsigned)p.n_splits, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = p.mode == DA_CLUSTER ? 2 : 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
        if (e == cudaSuccess && p.n_splits > 1 && p.mode == DA_SECOND)
            e = kvq_launch_pdl(decode_join_kernel, dim3(L->n_q_heads, S->batch), dim3(32 * DA_JOIN), 0, kvq_stream(stream), a);
        if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
        return (int)KVQ_OK;
    };
    if (nw == DA_WIDE) {
        if (cap) return bias ? go(decode_attn_kernel<true, true, DA_WIDE>) : go(decode_attn_kernel<true, false, DA_WIDE>);
        return bias ? go(decode_attn_kernel<false, true, DA_WIDE>) : go(decode_attn_kernel<false, false, DA_WIDE>);
    }
    if (cap) return bias ? go(decode_attn_kernel<true, true, DA_SLIM>) : go(decode_attn_kernel<true, false, DA_SLIM>);
    return bias ? go(decode_attn_kernel<false, true, DA_SLIM>) : go(decode_attn_kernel<false, false, DA_SLIM>);
}

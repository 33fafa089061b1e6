// kv_rope_append and kv_latent_append: a run of new tokens per sequence into the pages, normed and rotated on
// the way, so that no rotated copy is written and read again.
//
// Bound: bytes (about 3 flops per byte).  One CTA takes a few rows of the call.  Its last warp finds each row's
// sequence, page and position (three loads in sequence) while the others' first head rows are on their way; 256
// threads then compute the rows' cosines and sines once into shared memory, and every group of lanes takes whole
// head rows in two 16-byte loads per lane, as kv_qk_norm_rope does.  Angles are 64-bit turns.  Every value is
// rounded once, from fp32 to the cache's type.
//
// Measured (in a graph): two prompts of 16001 and 16384 tokens, bf16, normed, 32 + 8 + 8 heads into E4M3 pages 121 us,
// 6.0 TB/s (89% of the copy rate); 16385 latent rows with the rotated part of 16 heads 23 us, 4.5 TB/s, where 2.7 waves of
// CTAs (2049, five per SM) each begin with the chain of lookups; one token of 16 sequences 3 us.  More loads per lane cost
// CTAs per SM and more time (24 -> 34 us with four head rows on their way).
#include <algorithm>
#include <cmath>

#include "kvq_new_rows.cuh"
#include "kvq_rope.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int PG = KVQ_BLOCK_TOKENS;
constexpr int AP_NT = 256;
constexpr int AP_TOK = 8;      // most rows per CTA

struct AppendArgs {
    KvqNewRows rows;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *qw, *kw;
    float eps, mscale;
    const uint64_t* steps;
    int32_t rot, Hq, H;        // Hq: 0 without queries
    uint16_t* qo;
    void *k_pages, *v_pages;
    uint16_t* kT;
    float* k_absmax;
    int32_t t_cap;
};

// fp32 x8 -> E4M3 x8, round to nearest even, finite values saturate at +-448
__device__ __forceinline__ uint2 pack_e4m3(const float* x) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm("{\n.reg .b16 a, b;\ncvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
            "mov.b32 %0, {a, b};\n}"
            : "=r"(w[i])
            : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]));
    return make_uint2(w[0], w[1]);
}

template <typename T, bool INTER, bool FP8>
__global__ void __launch_bounds__(AP_NT) rope_append_kernel(const __grid_constant__ AppendArgs a, int tok_per_cta) {
    __shared__ __align__(16) float2 cs[AP_TOK][D / 2];
    __shared__ __align__(16) float wt[2][D];
    __shared__ int64_t at[AP_TOK];
    __shared__ int32_t pos[AP_TOK];
    const int64_t t0 = (int64_t)blockIdx.x * tok_per_cta;
    const int nt = (int)min((int64_t)tok_per_cta, a.rows.n_rows - t0);
    const int l = threadIdx.x & 7, heads = a.Hq + 2 * a.H;
    int ca, cb;
    chunks<INTER>(l, a.rot, &ca, &cb);
    kvq_pdl_begin();
    int t = 0, h = threadIdx.x >> 3;
    const auto settle = [&] {
        while (h >= heads) h -= heads, ++t;
    };
    settle();
    uint4 x4, y4;
    const auto fetch = [&] {
        if (t >= nt) return;
        const int64_t tok = t0 + t;
        const T* src = h < a.Hq         ? static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)h * D
                       : h < a.Hq + a.H ? static_cast<const T*>(a.k) + tok * a.k_stride + (int64_t)(h - a.Hq) * D
                                        : static_cast<const T*>(a.v) + tok * a.v_stride + (int64_t)(h - a.Hq - a.H) * D;
        x4 = *reinterpret_cast<const uint4*>(src + 8 * ca);
        y4 = *reinterpret_cast<const uint4*>(src + 8 * cb);
    };
    fetch();
    if (threadIdx.x < D) {
        if (a.qw != nullptr) wt[0][threadIdx.x] = a.qw[threadIdx.x];
        if (a.kw != nullptr) wt[1][threadIdx.x] = a.kw[threadIdx.x];
    }
    if (threadIdx.x >= AP_NT - 32) kvq_find_rows(a.rows, t0, nt, at, pos);
    __syncthreads();
    const int half = a.rot >> 1;
    for (int i = threadIdx.x; i < nt * (D / 2); i += AP_NT) {
        const int k = i / (D / 2), p = i % (D / 2);
        if (p < half) cs[k][pair_entry<INTER>(p)] = kvq_cos_sin(pos[k], a.steps[p], a.mscale);
    }
    __syncthreads();
    while (t < nt) {
        float x[8], y[8];
        unpack(x4, x, (T*)nullptr);
        unpack(y4, y, (T*)nullptr);
        const int tn = t, hn = h;
        h += AP_NT / 8;
        settle();
        fetch();
        const bool is_q = hn < a.Hq, is_v = hn >= a.Hq + a.H;
        if (!is_v) {
            if ((is_q ? a.qw : a.kw) != nullptr) norm_row(x, y, wt[is_q ? 0 : 1], ca, cb, a.eps);
            turn_row<INTER>(x, y, cs[tn], l, ca, cb, a.rot);
        }
        const int64_t to = at[tn];
        if (is_q) {
            if (to == KVQ_ROW_NONE) continue;
            uint16_t* dst = a.qo + ((t0 + tn) * a.Hq + hn) * D;
            *reinterpret_cast<uint4*>(dst + 8 * ca) = pack_half(x);
            *reinterpret_cast<uint4*>(dst + 8 * cb) = pack_half(y);
        } else {
            if (to < 0) continue;
            const int g = hn - a.Hq - (is_v ? a.H : 0);
            const int64_t off = (((to / PG) * a.H + g) * PG + to % PG) * D;
            void* pages = is_v ? a.v_pages : a.k_pages;
            if (FP8) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + off + 8 * ca) = pack_e4m3(x);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + off + 8 * cb) = pack_e4m3(y);
            } else {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pages) + off + 8 * ca) = pack_half(x);
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pages) + off + 8 * cb) = pack_half(y);
            }
        }
    }
}

// The same into an fp16 layer with a channel-major copy of its keys and their channels' maxima.  A CTA takes the new
// tokens of eight places of a sequence (0 .. 7 modulo 8), so that a channel's values are one 16-byte piece of the copy, and
// up to SC_HEADS key heads with their part of the queries and values: first those as above, then the keys, which are
// written to their pages and, through shared memory, to the copy.  A row is on its way while the one before is turned.  (As a
// second launch over the rows just written: 32 us for 4097 tokens of 32 + 8 + 8 heads, here 23; with all heads in one CTA
// 3.5K tokens of 40 + 40 + 40 heads took 94 instead of 63 us.)
constexpr int SC_TOK = 8, SC_HEADS = 8;
template <typename T, bool INTER>
__global__ void __launch_bounds__(AP_NT, 4) rope_append_scored_kernel(const __grid_constant__ AppendArgs a, int heads) {
    __shared__ __align__(16) float2 cs[SC_TOK][D / 2];
    __shared__ __align__(16) float wt[2][D];
    __shared__ __align__(16) uint16_t keys[SC_HEADS][SC_TOK][D];
    __shared__ int32_t who[4];          // sequence, its first new row here, that row's place, rows here
    __shared__ int32_t pos[SC_TOK];
    __shared__ int32_t page;
    const int tid = threadIdx.x, l = tid & 7, grp = tid >> 3, lane = tid & 31;
    int ca, cb;
    chunks<INTER>(l, a.rot, &ca, &cb);
    kvq_pdl_begin();
    if (tid < D) {
        if (a.qw != nullptr) wt[0][tid] = a.qw[tid];
        if (a.kw != nullptr) wt[1][tid] = a.kw[tid];
    }
    if (tid >= AP_NT - 32) {
        if (lane == 0) who[0] = -1;
        __syncwarp();
        int base = 0;
        for (int b0 = 0; b0 < a.rows.batch; b0 += 32) {
            const int b = b0 + lane;
            int first = 0, n = 0, len = 0;
            if (b < a.rows.batch) kvq_new_rows_of(a.rows, b, &first, &n, &len);
            const int lo = (len - n) / SC_TOK, tiles = n > 0 ? (len - 1) / SC_TOK + 1 - lo : 0;
            int incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const int mine = (int)blockIdx.x - (base + incl - tiles);
            if (mine >= 0 && mine < tiles) {
                const int at = max(len - n, (lo + mine) * SC_TOK);
                who[0] = b, who[1] = first + at - (len - n), who[2] = at, who[3] = min(len, (lo + mine + 1) * SC_TOK) - at;
                page = kvq_page_at(a.rows, b, at / PG);
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        __syncwarp();
        if (who[0] >= 0 && lane < who[3]) pos[lane] = a.rows.pos != nullptr ? a.rows.pos[who[1] + lane] : who[2] + lane;
    }
    __syncthreads();
    const int b = who[0], r0 = who[1], place = who[2], nt = who[3];
    if (b < 0) return;
    for (int i = tid; i < nt * (D / 2); i += AP_NT) {
        const int k = i / (D / 2), p = i % (D / 2);
        if (p < a.rot >> 1) cs[k][pair_entry<INTER>(p)] = kvq_cos_sin(pos[k], a.steps[p], a.mscale);
    }
    __syncthreads();
    // (the rows here share a page)
    const auto row_at = [&](int g, int k) { return (((int64_t)page * a.H + g) * PG + place % PG + k) * D; };
    const int g0 = blockIdx.y * heads, ng = min(heads, a.H - g0);   // this CTA's key heads
    uint4 kx4, ky4;
    const auto fetch_key = [&](int i) {
        const int k = i / ng, g = i - k * ng;
        const T* src = static_cast<const T*>(a.k) + (r0 + k) * a.k_stride + (int64_t)(g0 + g) * D;
        kx4 = *reinterpret_cast<const uint4*>(src + 8 * ca);
        ky4 = *reinterpret_cast<const uint4*>(src + 8 * cb);
    };
    if (grp < nt * ng) fetch_key(grp);
    // its queries and values, the next row on its way
    const int share = (a.Hq + a.H + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * share, nh = min(share, a.Hq + a.H - h0);
    uint4 x4, y4;
    const auto fetch = [&](int i) {
        const int k = i / nh, h = h0 + i - k * nh;
        const T* src = h < a.Hq ? static_cast<const T*>(a.q) + (r0 + k) * a.q_stride + (int64_t)h * D
                                : static_cast<const T*>(a.v) + (r0 + k) * a.v_stride + (int64_t)(h - a.Hq) * D;
        x4 = *reinterpret_cast<const uint4*>(src + 8 * ca);
        y4 = *reinterpret_cast<const uint4*>(src + 8 * cb);
    };
    const int n_rows = nt * max(nh, 0);
    if (grp < n_rows) fetch(grp);
    for (int i = grp; i < n_rows; i += AP_NT / 8) {
        const int k = i / nh, h = h0 + i - k * nh;
        const bool is_q = h < a.Hq;
        float x[8], y[8];
        unpack(x4, x, (T*)nullptr);
        unpack(y4, y, (T*)nullptr);
        if (i + AP_NT / 8 < n_rows) fetch(i + AP_NT / 8);
        uint16_t* dst;
        if (is_q) {
            if (a.qw != nullptr) norm_row(x, y, wt[0], ca, cb, a.eps);
            turn_row<INTER>(x, y, cs[k], l, ca, cb, a.rot);
            dst = a.qo + ((int64_t)(r0 + k) * a.Hq + h) * D;
        } else {
            if (page < 0) continue;
            dst = static_cast<uint16_t*>(a.v_pages) + row_at(h - a.Hq, k);
        }
        *reinterpret_cast<uint4*>(dst + 8 * ca) = pack_half(x);
        *reinterpret_cast<uint4*>(dst + 8 * cb) = pack_half(y);
    }
    if (page < 0) return;
    // keys
    for (int i = grp; i < nt * ng; i += AP_NT / 8) {
        const int k = i / ng, g = i - k * ng;
        float x[8], y[8];
        unpack(kx4, x, (T*)nullptr);
        unpack(ky4, y, (T*)nullptr);
        if (i + AP_NT / 8 < nt * ng) fetch_key(i + AP_NT / 8);
        if (a.kw != nullptr) norm_row(x, y, wt[1], ca, cb, a.eps);
        turn_row<INTER>(x, y, cs[k], l, ca, cb, a.rot);
        const uint4 u = pack_half(x), v = pack_half(y);
        uint16_t* dst = static_cast<uint16_t*>(a.k_pages) + row_at(g0 + g, k);
        *reinterpret_cast<uint4*>(dst + 8 * ca) = u;
        *reinterpret_cast<uint4*>(dst + 8 * cb) = v;
        *reinterpret_cast<uint4*>(&keys[g][k][8 * ca]) = u;
        *reinterpret_cast<uint4*>(&keys[g][k][8 * cb]) = v;
    }
    __syncthreads();
    for (int i = tid; i < ng * D; i += AP_NT) {
        const int g = i / D, c = i % D;
        const int64_t ch = ((int64_t)b * a.H + g0 + g) * D + c;
        const float so_far = a.k_absmax[ch];
        __align__(16) uint16_t w[SC_TOK];
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < SC_TOK; ++k) {
            w[k] = k < nt ? keys[g][k][c] : (uint16_t)0;
            top = fmaxf(top, fabsf(kvq_h2f(w[k])));
        }
        uint16_t* dst = a.kT + ch * a.t_cap + place;
        if (nt == SC_TOK) {
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(w);
        } else {
#pragma unroll
            for (int k = 0; k < SC_TOK; ++k)
                if (k < nt) dst[k] = w[k];
        }
        // (maxima are not negative, so their bits are ordered as integers; the order of arrival does not matter, and a
        // maximum only grows: most CTAs find theirs passed already)
        if (top > so_far) atomicMax(reinterpret_cast<int*>(a.k_absmax + ch), __float_as_int(top));
    }
}

// ---------------------------------------------------------------- latent rows

constexpr int LAT = KVQ_LATENT_DIM, ROT = KVQ_LATENT_ROPE, ROW = LAT + ROT;

struct LatentArgs {
    KvqNewRows rows;
    const void *c, *k, *q;
    int64_t c_stride, k_stride, q_stride, q_head, qo_stride, qo_head;
    const float* cw;
    float eps, mscale;
    const uint64_t* steps;
    int32_t Hq;
    uint16_t *pages, *qo;
};

// A token's work comes in warps: its latent row (16 values per lane), then its rotated rows of 64 values, the key's
// and the query heads', eight rows per warp (four lanes per row, 16 values per lane).
template <typename T, bool INTER>
__global__ void __launch_bounds__(AP_NT, 5) latent_append_kernel(const __grid_constant__ LatentArgs a, int tok_per_cta) {
    __shared__ __align__(16) float2 cs[AP_TOK][ROT / 2];
    __shared__ int64_t at[AP_TOK];
    __shared__ int32_t pos[AP_TOK];
    const int64_t t0 = (int64_t)blockIdx.x * tok_per_cta;
    const int nt = (int)min((int64_t)tok_per_cta, a.rows.n_rows - t0);
    const int lane = threadIdx.x & 31, l = lane & 3, quad = lane >> 2;
    const int per = 1 + (a.Hq + 1 + 7) / 8;   // warps of work per token
    kvq_pdl_begin();
    int t = 0, u = threadIdx.x >> 5;          // token and its warp of work
    const auto settle = [&] {
        while (u >= per) u -= per, ++t;
    };
    settle();
    uint4 x4, y4;
    const auto fetch = [&] {
        if (t >= nt) return;
        const int64_t tok = t0 + t;
        const T* src;
        int ca = lane, cb = lane + 32;
        if (u == 0) {
            src = static_cast<const T*>(a.c) + tok * a.c_stride;
        } else {
            const int row = (u - 1) * 8 + quad;
            ca = l, cb = l + 4;
            if (row > a.Hq) return;
            src = row == 0 ? static_cast<const T*>(a.k) + tok * a.k_stride
                           : static_cast<const T*>(a.q) + tok * a.q_stride + (row - 1) * a.q_head;
        }
        x4 = *reinterpret_cast<const uint4*>(src + 8 * ca);
        y4 = *reinterpret_cast<const uint4*>(src + 8 * cb);
    };
    fetch();
    if (threadIdx.x >= AP_NT - 32) kvq_find_rows(a.rows, t0, nt, at, pos);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * (ROT / 2); i += AP_NT) {
        const int k = i / (ROT / 2), p = i % (ROT / 2);
        // by the lane that uses them: entries 8j + 2l and 8j + 2l + 1 hold the j-th two pairs of lane l
        const int of = INTER ? (p >> 2) & 3 : p >> 3, nth = INTER ? (p >> 4) * 4 + (p & 3) : p & 7;
        cs[k][((nth >> 1) * 4 + of) * 2 + (nth & 1)] = kvq_cos_sin(pos[k], a.steps[p], a.mscale);
    }
    __syncthreads();
    while (t < nt) {
        float x[8], y[8];
        unpack(x4, x, (T*)nullptr);
        unpack(y4, y, (T*)nullptr);
        const int tn = t, un = u;
        u += AP_NT / 32;
        settle();
        fetch();
        const int64_t to = at[tn];
        if (un == 0) {
            if (a.cw != nullptr) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
                const float inv = 1.0f / sqrtf(kvq_warp_sum(ss) * (1.0f / LAT) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 p = *reinterpret_cast<const float4*>(a.cw + 8 * lane + i);
                    const float4 q = *reinterpret_cast<const float4*>(a.cw + 8 * (lane + 32) + i);
                    x[i] *= inv * p.x, x[i + 1] *= inv * p.y, x[i + 2] *= inv * p.z, x[i + 3] *= inv * p.w;
                    y[i] *= inv * q.x, y[i + 1] *= inv * q.y, y[i + 2] *= inv * q.z, y[i + 3] *= inv * q.w;
                }
            }
            if (to < 0) continue;
            uint16_t* dst = a.pages + to * ROW;
            *reinterpret_cast<uint4*>(dst + 8 * lane) = pack_half(x);
            *reinterpret_cast<uint4*>(dst + 8 * (lane + 32)) = pack_half(y);
            continue;
        }
        const int row = (un - 1) * 8 + quad;
        if (row > a.Hq) continue;
        const float4* f = reinterpret_cast<const float4*>(cs[tn]) + l;
        if (INTER) {
            turn_two(&x[0], &x[1], &x[2], &x[3], f[0]), turn_two(&x[4], &x[5], &x[6], &x[7], f[4]);
            turn_two(&y[0], &y[1], &y[2], &y[3], f[8]), turn_two(&y[4], &y[5], &y[6], &y[7], f[12]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) turn_two(&x[2 * j], &y[2 * j], &x[2 * j + 1], &y[2 * j + 1], f[4 * j]);
        }
        if (row == 0 ? to < 0 : to == KVQ_ROW_NONE) continue;
        uint16_t* dst = row == 0 ? a.pages + to * ROW + LAT : a.qo + (t0 + tn) * a.qo_stride + (row - 1) * a.qo_head;
        *reinterpret_cast<uint4*>(dst + 8 * l) = pack_half(x);
        *reinterpret_cast<uint4*>(dst + 8 * (l + 4)) = pack_half(y);
    }
}

// Rows per CTA: one until every SM has CTAs enough to hide the loads' latency, then more, which share the CTA's start; of
// many heads fewer, some 384 head rows.  What that limit gives, over nine numbers of tokens from 1300 to 12000 and two cache
// types (time with it by time without): 64 + 64 + 64 heads 0.78 to 1.00, 0.92 on average (5500 tokens 78 and 100 us);
// 32 + 32 + 32 heads 0.84 to 1.00, 0.97; 40 + 40 + 40 heads 0.83 to 1.25, 0.94 (2000 tokens, the worst, 27 and 22 us: with
// the limit a second wave begins); latent rows with 128 heads 0.84 to 1.04, 0.97, with 64 heads 0.97 to 1.11, 1.02.
int rows_per_cta(int64_t n_rows, int heads) {
    const int64_t sms = kvq_num_sms();
    return std::min(n_rows <= 8 * sms ? 1 : n_rows <= 32 * sms ? 4 : AP_TOK, std::max(1, 384 / heads));
}

}  // namespace

extern "C" size_t kv_rope_append_ws(void) { return sizeof(KvqWsHeader); }

extern "C" int kv_rope_append(const kvq_layout* L, const kvq_pool* P, const kvq_seqs* S, const kvq_rope* rope,
                              const uint64_t* steps, float mscale, int32_t dtype, int64_t n_rows,
                              const int32_t* row_starts, const int32_t* positions, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* q_weight,
                              const float* k_weight, float eps, uint16_t* q_out, void* ws, size_t ws_bytes, void* stream) {
    static const char* fn = "kv_rope_append";
    kvq_clear_error();
    int st = kvq_check_layout(L, fn, false);
    if (!st) st = kvq_check_seqs(S, fn);
    if (!st) st = kvq_check_rope(rope, fn);
    if (!st) st = kvq_check_ws(ws, ws_bytes, kv_rope_append_ws(), fn);
    if (st) return st;
    const bool fp8 = L->bits == KVQ_BITS_E4M3;
    KVQ_REQUIRE(fp8 || L->bits == 16, KVQ_ERR_UNSUPPORTED, "%s: bits %d (an fp16 or an E4M3 layer)", fn, L->bits);
    KVQ_REQUIRE(dtype == KVQ_F16 || dtype == KVQ_BF16, KVQ_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    // (a token's head rows are counted in 32 bits)
    KVQ_REQUIRE(L->n_q_heads <= 1 << 16 && L->n_kv_heads <= 1 << 16, KVQ_ERR_UNSUPPORTED, "%s: %d + %d heads (at most 65536 each)",
                fn, L->n_q_heads, L->n_kv_heads);
    KVQ_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX, KVQ_ERR_INVALID_ARG, "%s: n_rows", fn);
    KVQ_REQUIRE(P != nullptr && S->batch <= P->max_seqs, KVQ_ERR_INVALID_ARG, "%s: NULL pool, or batch above max_seqs", fn);
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    st = kvq_check_new_rows(S, row_starts, P->num_blocks, fn);
    if (st) return st;
    KVQ_REQUIRE(k && v && !q == !q_out, KVQ_ERR_INVALID_ARG, "%s: k and v, and q with q_out or neither", fn);
    KVQ_REQUIRE(q || !q_weight, KVQ_ERR_INVALID_ARG, "%s: a weight without its rows", fn);
    KVQ_REQUIRE(rope->rot_dim == 0 || steps, KVQ_ERR_INVALID_ARG, "%s: NULL steps", fn);
    KVQ_REQUIRE(std::isfinite(mscale) && std::isfinite(eps) && eps >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: mscale / eps", fn);
    const int64_t wq = (int64_t)L->n_q_heads * D, wk = (int64_t)L->n_kv_heads * D;
    KVQ_REQUIRE((!q || q_stride >= wq) && k_stride >= wk && v_stride >= wk, KVQ_ERR_INVALID_ARG,
                "%s: a token stride below the row's width", fn);
    KVQ_REQUIRE(((q ? q_stride : 0) | k_stride | v_stride) % 8 == 0, KVQ_ERR_INVALID_ARG,
                "%s: strides must be multiples of 8", fn);
    KVQ_REQUIRE(kvq_aligned16(q) && kvq_aligned16(k) && kvq_aligned16(v) && kvq_aligned16(q_out), KVQ_ERR_INVALID_ARG,
                "%s: rows must be 16-byte aligned", fn);
    KVQ_REQUIRE(!q || q != q_out || (dtype == KVQ_F16 && q_stride == wq), KVQ_ERR_INVALID_ARG,
                "%s: in place needs fp16 rows without gaps", fn);
    AppendArgs a;
    a.rows = KvqNewRows{row_starts, S->seq_lens, S->block_table, positions, n_rows, P->num_blocks,
                        S->batch, S->max_blocks, S->max_len, static_cast<KvqWsHeader*>(ws)};
    a.kT = nullptr, a.k_absmax = nullptr, a.t_cap = 0;
    if (fp8) {
        a.k_pages = P->k_codes, a.v_pages = P->v_codes;
    } else {
        a.k_pages = P->k16, a.v_pages = P->v16;
        KVQ_REQUIRE((P->kT == nullptr) == (P->k_absmax == nullptr), KVQ_ERR_INVALID_ARG, "%s: kT with k_absmax or neither", fn);
        if (P->kT != nullptr) {
            KVQ_REQUIRE(P->t_cap > 0 && P->t_cap % 8 == 0 && kvq_aligned16(P->kT), KVQ_ERR_INVALID_ARG,
                        "%s: kT must be 16-byte aligned, t_cap a multiple of 8", fn);
            a.kT = P->kT, a.k_absmax = P->k_absmax, a.t_cap = P->t_cap;
            a.rows.max_len = std::min(a.rows.max_len, P->t_cap);
        }
    }
    KVQ_REQUIRE(a.k_pages && a.v_pages && kvq_aligned16(a.k_pages) && kvq_aligned16(a.v_pages), KVQ_ERR_INVALID_ARG,
                "%s: the pool needs 16-byte aligned K and V pages", fn);
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.qw = q_weight, a.kw = k_weight;
    a.eps = eps, a.mscale = mscale, a.steps = steps, a.rot = rope->rot_dim;
    a.Hq = q ? L->n_q_heads : 0, a.H = L->n_kv_heads;
    a.qo = q_out;
    const auto launched = [&](cudaError_t e) {
        return e == cudaSuccess ? (int)KVQ_OK : kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    };
    if (a.kT != nullptr) {
        // n new tokens of a sequence touch at most n / 8 + 2 groups of eight places
        const int64_t tiles = n_rows / SC_TOK + 2 * (int64_t)S->batch;
        KVQ_REQUIRE(tiles <= INT32_MAX, KVQ_ERR_UNSUPPORTED, "%s: batch", fn);
        // Fewer key heads per CTA while CTAs are few: 1820 tokens of 8 heads, 230 groups, 13 us by four and 17 by eight;
        // 8192 tokens of 32 heads, 1026 groups, 120 and 108 (98 with four CTAs per SM).
        const int heads = tiles * ((a.H + SC_HEADS - 1) / SC_HEADS) >= 3 * (int64_t)kvq_num_sms() ? SC_HEADS : SC_HEADS / 2;
        const auto go = [&](auto kernel) {
            return launched(kvq_launch_pdl(kernel, dim3((unsigned)tiles, (a.H + heads - 1) / heads), dim3(AP_NT), 0,
                                           kvq_stream(stream), a, heads));
        };
        if (dtype == KVQ_F16)
            return rope->interleaved ? go(rope_append_scored_kernel<__half, true>) : go(rope_append_scored_kernel<__half, false>);
        return rope->interleaved ? go(rope_append_scored_kernel<__nv_bfloat16, true>)
                                 : go(rope_append_scored_kernel<__nv_bfloat16, false>);
    }
    const int tpc = rows_per_cta(n_rows, a.Hq + 2 * a.H);
    const unsigned grid = (unsigned)((n_rows + tpc - 1) / tpc);
    const auto go = [&](auto kernel) {
        return launched(kvq_launch_pdl(kernel, dim3(grid), dim3(AP_NT), 0, kvq_stream(stream), a, tpc));
    };
    const auto by_layout = [&](auto type) {
        using T = decltype(type);
        if (fp8) return rope->interleaved ? go(rope_append_kernel<T, true, true>) : go(rope_append_kernel<T, false, true>);
        return rope->interleaved ? go(rope_append_kernel<T, true, false>) : go(rope_append_kernel<T, false, false>);
    };
    return dtype == KVQ_F16 ? by_layout(__half()) : by_layout(__nv_bfloat16());
}

extern "C" int kv_latent_append(const kvq_latent* C, const kvq_seqs* S, const kvq_rope* rope, const uint64_t* steps,
                                float mscale, int32_t dtype, int64_t n_rows, const int32_t* row_starts,
                                const int32_t* positions, const void* c, int64_t c_stride, const void* k_rope,
                                int64_t k_stride, const float* c_weight, float eps, int32_t n_heads, const void* q,
                                int64_t q_stride, int64_t q_head_stride, uint16_t* q_out, int64_t q_out_stride,
                                int64_t q_out_head_stride, void* ws, size_t ws_bytes, void* stream) {
    static const char* fn = "kv_latent_append";
    kvq_clear_error();
    int st = kvq_check_latent(C, fn);
    if (!st) st = kvq_check_seqs(S, fn);
    if (!st) st = kvq_check_rope(rope, fn);
    if (!st) st = kvq_check_ws(ws, ws_bytes, kv_rope_append_ws(), fn);
    if (st) return st;
    KVQ_REQUIRE(rope->rot_dim == ROT, KVQ_ERR_UNSUPPORTED, "%s: rot_dim %d (a latent row's rotated part is 64)", fn,
                rope->rot_dim);
    KVQ_REQUIRE(dtype == KVQ_F16 || dtype == KVQ_BF16, KVQ_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    KVQ_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX, KVQ_ERR_INVALID_ARG, "%s: n_rows", fn);
    KVQ_REQUIRE(!q == !q_out && (q ? n_heads > 0 && n_heads <= 1 << 16 : n_heads == 0) , KVQ_ERR_INVALID_ARG,
                "%s: q with q_out and n_heads, or none of them", fn);
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    st = kvq_check_new_rows(S, row_starts, C->num_blocks, fn);
    if (st) return st;
    KVQ_REQUIRE(c && k_rope && steps, KVQ_ERR_INVALID_ARG, "%s: NULL c / k_rope / steps", fn);
    KVQ_REQUIRE(std::isfinite(mscale) && std::isfinite(eps) && eps >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: mscale / eps", fn);
    KVQ_REQUIRE(c_stride >= LAT && k_stride >= ROT, KVQ_ERR_INVALID_ARG, "%s: a token stride below the row's width", fn);
    // (a head's 64 values within a token's stride, or tokens within a head's: any order of the two)
    KVQ_REQUIRE(!q || (q_stride >= ROT && q_head_stride >= ROT && q_out_stride >= ROT && q_out_head_stride >= ROT),
                KVQ_ERR_INVALID_ARG, "%s: a query stride below the row's width", fn);
    KVQ_REQUIRE((c_stride | k_stride | (q ? q_stride | q_head_stride | q_out_stride | q_out_head_stride : 0)) % 8 == 0,
                KVQ_ERR_INVALID_ARG, "%s: strides must be multiples of 8", fn);
    KVQ_REQUIRE(kvq_aligned16(c) && kvq_aligned16(k_rope) && kvq_aligned16(q) && kvq_aligned16(q_out) &&
                    ((uintptr_t)c_weight & 15u) == 0, KVQ_ERR_INVALID_ARG, "%s: rows and c_weight must be 16-byte aligned", fn);
    KVQ_REQUIRE(!q || q != q_out || (dtype == KVQ_F16 && q_stride == q_out_stride && q_head_stride == q_out_head_stride),
                KVQ_ERR_INVALID_ARG, "%s: in place needs fp16 queries and one set of strides", fn);
    LatentArgs a;
    a.rows = KvqNewRows{row_starts, S->seq_lens, S->block_table, positions, n_rows, C->num_blocks,
                        S->batch, S->max_blocks, S->max_len, static_cast<KvqWsHeader*>(ws)};
    a.c = c, a.k = k_rope, a.q = q;
    a.c_stride = c_stride, a.k_stride = k_stride;
    a.q_stride = q_stride, a.q_head = q_head_stride, a.qo_stride = q_out_stride, a.qo_head = q_out_head_stride;
    a.cw = c_weight, a.eps = eps, a.mscale = mscale, a.steps = steps;
    a.Hq = n_heads;
    a.pages = C->rows, a.qo = q_out;
    const int tpc = rows_per_cta(n_rows, a.Hq + 4);
    const unsigned grid = (unsigned)((n_rows + tpc - 1) / tpc);
    const auto go = [&](auto kernel) {
        const cudaError_t e = kvq_launch_pdl(kernel, dim3(grid), dim3(AP_NT), 0, kvq_stream(stream), a, tpc);
        if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
        return (int)KVQ_OK;
    };
    if (dtype == KVQ_F16)
        return rope->interleaved ? go(latent_append_kernel<__half, true>) : go(latent_append_kernel<__half, false>);
    return rope->interleaved ? go(latent_append_kernel<__nv_bfloat16, true>) : go(latent_append_kernel<__nv_bfloat16, false>);
}

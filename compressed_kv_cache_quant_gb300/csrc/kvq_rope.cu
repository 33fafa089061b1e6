// kv_qk_norm_rope: RMS norms of the query and key heads and their rotary positions in one pass over a
// projection's rows, and the host helper that lays out the rotation's frequencies.
//
// Positions.  A pair that turns f radians per position is at angle p * f.  At long positions an fp32
// product loses it (p * f near 1e5 rad has 8e-3 rad steps) and fp64 arithmetic is slow on this GPU, so
// frequencies are kept in turns as 64-bit fractions, step = f / 2pi * 2^64: the wrapping integer product
// p * step is p times the step modulo one turn, without any rounding, so positions add nothing to the step's own
// error.  That is fp64's (kvq_rope_steps: a power, a logarithm for some scalings, a few roundings): at most 2^-48 of
// the step and one unit of 2^-63, 2^-33 turns at position 131072.  The angle's top bits as a signed fp32 fraction go
// to sincospif.
//
// Bound: bytes (every head row is read and written once, about 3 flops per byte).  One CTA takes a few
// tokens: 256 threads compute the tokens' cosines and sines once into shared memory (64 pairs per token,
// reused by every head), then every group of 8 lanes takes whole head rows, 16 values per lane as two
// 16-byte loads, so a row's norm is three shuffles and both members of every pair are in one lane.  A row's
// loads are issued while the one before is worked on.  Measured: 32768 tokens of 32 + 8 + 8 bf16 heads with
// norms 125 us (6.45 TB/s, 95% of the measured copy rate); eight tokens 1.9 us in a graph.
#include <algorithm>
#include <cmath>

#include "kvq_rope.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int RP_NT = 256;
constexpr int RP_GROUPS = RP_NT / 8;  // head rows in flight per CTA
constexpr int RP_TOK = 8;             // most tokens per CTA

struct RopeArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *qw, *kw;
    float eps, mscale;
    const int32_t* pos;
    const uint64_t* steps;
    int32_t rot, Hq, Hk, Hv;  // Hq / Hk / Hv: head rows per token of q, k and v (0 when absent)
    int64_t n;
    uint16_t *qo, *ko, *vo;
};

// One head row of a lane's group: where it is read and written, its weight, whether it is rotated.
struct Row {
    const void* src;
    uint16_t* dst;
    const float* w;   // its weights in shared memory, or NULL
    bool turn;
};
template <typename T>
__device__ __forceinline__ Row row_of(const RopeArgs& a, int64_t tok, int h, const float (*wt)[D]) {
    Row r;
    if (h < a.Hq) {
        r.src = static_cast<const T*>(a.q) + tok * a.q_stride + h * D;
        r.dst = a.qo + (tok * a.Hq + h) * D;
        r.w = a.qw != nullptr ? wt[0] : nullptr;
        r.turn = true;
    } else if (h < a.Hq + a.Hk) {
        r.src = static_cast<const T*>(a.k) + tok * a.k_stride + (h - a.Hq) * D;
        r.dst = a.ko + (tok * a.Hk + h - a.Hq) * D;
        r.w = a.kw != nullptr ? wt[1] : nullptr;
        r.turn = true;
    } else {
        r.src = static_cast<const T*>(a.v) + tok * a.v_stride + (h - a.Hq - a.Hk) * D;
        r.dst = a.vo + (tok * a.Hv + h - a.Hq - a.Hk) * D;
        r.w = nullptr;
        r.turn = false;
    }
    return r;
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(RP_NT) norm_rope_kernel(const __grid_constant__ RopeArgs a, int tok_per_cta) {
    __shared__ __align__(16) float2 cs[RP_TOK][D / 2];
    __shared__ __align__(16) float wt[2][D];
    const int64_t t0 = (int64_t)blockIdx.x * tok_per_cta;
    const int nt = (int)min((int64_t)tok_per_cta, a.n - t0);
    const int l = threadIdx.x & 7;
    const int rows = a.Hq + a.Hk + a.Hv;
    int ca, cb;
    chunks<INTER>(l, a.rot, &ca, &cb);
    kvq_pdl_begin();
    // the first rows are on their way while the angles are computed, every further row while the one
    // before is
    int t = 0, h = threadIdx.x >> 3;
    const auto settle = [&] {
        while (h >= rows) h -= rows, ++t;
    };
    settle();
    Row r;
    uint4 x4, y4;
    const auto fetch = [&] {
        if (t >= nt) return;
        r = row_of<T>(a, t0 + t, h, wt);
        x4 = *reinterpret_cast<const uint4*>(static_cast<const T*>(r.src) + 8 * ca);
        y4 = *reinterpret_cast<const uint4*>(static_cast<const T*>(r.src) + 8 * cb);
    };
    fetch();
    if (threadIdx.x < D) {
        if (a.qw != nullptr) wt[0][threadIdx.x] = a.qw[threadIdx.x];
        if (a.kw != nullptr) wt[1][threadIdx.x] = a.kw[threadIdx.x];
    }
    const int half = a.rot >> 1;
    for (int i = threadIdx.x; i < nt * (D / 2); i += RP_NT) {
        const int k = i / (D / 2), p = i % (D / 2);
        if (p >= half) continue;
        cs[k][pair_entry<INTER>(p)] = kvq_cos_sin(a.pos[t0 + k], a.steps[p], a.mscale);
    }
    __syncthreads();
    while (t < nt) {
        float x[8], y[8];
        unpack(x4, x, (T*)nullptr);
        unpack(y4, y, (T*)nullptr);
        const Row now = r;
        const int tn = t;
        h += RP_GROUPS;
        settle();
        fetch();
        if (now.w != nullptr) norm_row(x, y, now.w, ca, cb, a.eps);
        if (now.turn) turn_row<INTER>(x, y, cs[tn], l, ca, cb, a.rot);
        *reinterpret_cast<uint4*>(now.dst + 8 * ca) = pack_half(x);
        *reinterpret_cast<uint4*>(now.dst + 8 * cb) = pack_half(y);
    }
}

}  // namespace

extern "C" int kvq_rope_steps(const kvq_rope* r, uint64_t* steps, float* mscale) {
    kvq_clear_error();
    const int st = kvq_check_rope(r, "kvq_rope_steps");
    if (st) return st;
    KVQ_REQUIRE(mscale != nullptr && (steps != nullptr || r->rot_dim == 0), KVQ_ERR_INVALID_ARG,
                "kvq_rope_steps: NULL output");
    *mscale = 1.0f;
    if (r->rot_dim == 0) return KVQ_OK;
    const double two_pi = 6.283185307179586476925;
    const int R = r->rot_dim;
    KVQ_REQUIRE(std::isfinite(r->base) && r->base > 1.0, KVQ_ERR_INVALID_ARG, "kvq_rope_steps: base must exceed 1");
    KVQ_REQUIRE(r->scaling >= KVQ_ROPE_PLAIN && r->scaling <= KVQ_ROPE_KNEES, KVQ_ERR_UNSUPPORTED,
                "kvq_rope_steps: scaling %d", r->scaling);
    const bool ramp = r->scaling == KVQ_ROPE_YARN || r->scaling == KVQ_ROPE_KNEES;
    KVQ_REQUIRE(r->scaling == KVQ_ROPE_PLAIN || (std::isfinite(r->factor) && r->factor >= 1.0), KVQ_ERR_INVALID_ARG,
                "kvq_rope_steps: factor must be at least 1");
    if (ramp) {
        KVQ_REQUIRE(r->original_len > 0 && std::isfinite(r->low) && std::isfinite(r->high) && r->low > 0 && r->high > 0,
                    KVQ_ERR_INVALID_ARG, "kvq_rope_steps: original_len, low and high must be positive");
        KVQ_REQUIRE(r->scaling == KVQ_ROPE_YARN ? r->low > r->high : r->low < r->high, KVQ_ERR_INVALID_ARG,
                    "kvq_rope_steps: YaRN wants low > high (fast and slow turns), knees low < high");
    }
    double base = r->base;
    if (r->scaling == KVQ_ROPE_NTK) base *= pow(r->factor, (double)R / (R - 2));
    double edge_lo = 0.0, edge_hi = 0.0;
    if (r->scaling == KVQ_ROPE_YARN) {
        const auto pair_of = [&](double turns) { return R * log(r->original_len / (turns * two_pi)) / (2.0 * log(base)); };
        edge_lo = std::max(floor(pair_of(r->low)), 0.0);
        edge_hi = std::min(ceil(pair_of(r->high)), (double)(R - 1));
        *mscale = (float)(0.1 * log(r->factor) + 1.0);
    }
    for (int i = 0; i < R / 2; ++i) {
        double f = pow(base, -2.0 * i / R);
        double keep = 1.0;  // share of the unscaled frequency
        if (r->scaling == KVQ_ROPE_LINEAR) keep = 0.0;
        if (r->scaling == KVQ_ROPE_YARN)
            keep = 1.0 - std::min(std::max((i - edge_lo) / std::max(edge_hi - edge_lo, 1e-3), 0.0), 1.0);
        if (r->scaling == KVQ_ROPE_KNEES) {
            const double turns = r->original_len * f / two_pi;
            keep = std::min(std::max((turns - r->low) / (r->high - r->low), 0.0), 1.0);
        }
        if (r->scaling != KVQ_ROPE_PLAIN && r->scaling != KVQ_ROPE_NTK) f = f * keep + f / r->factor * (1.0 - keep);
        // f <= 1 rad: below 0.16 turns, far from the 64-bit limit.  Split so that the double's 53 bits
        // are scaled exactly.
        steps[i] = (uint64_t)llrint(ldexp(f / two_pi, 63)) << 1;
    }
    return KVQ_OK;
}

extern "C" int kv_qk_norm_rope(const kvq_layout* L, const kvq_rope* rope, const uint64_t* steps, float mscale,
                               int32_t dtype, int64_t n_tokens, const int32_t* positions, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               const float* q_weight, const float* k_weight, float eps, uint16_t* q_out,
                               uint16_t* k_out, uint16_t* v_out, void* stream) {
    static const char* fn = "kv_qk_norm_rope";
    kvq_clear_error();
    int st = kvq_check_layout(L, fn, false);
    if (st) return st;
    st = kvq_check_rope(rope, fn);
    if (st) return st;
    KVQ_REQUIRE(dtype == KVQ_F16 || dtype == KVQ_BF16, KVQ_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    KVQ_REQUIRE(n_tokens >= 0, KVQ_ERR_INVALID_ARG, "%s: n_tokens", fn);
    if (n_tokens == 0) return KVQ_OK;  // (an empty tensor has no address)
    KVQ_REQUIRE(q || k || v, KVQ_ERR_INVALID_ARG, "%s: no rows given", fn);
    KVQ_REQUIRE(!q == !q_out && !k == !k_out && !v == !v_out, KVQ_ERR_INVALID_ARG,
                "%s: every input needs its output, and the other way round", fn);
    KVQ_REQUIRE((q || !q_weight) && (k || !k_weight), KVQ_ERR_INVALID_ARG, "%s: a weight without its rows", fn);
    KVQ_REQUIRE(rope->rot_dim == 0 || !(q || k) || (positions && steps), KVQ_ERR_INVALID_ARG,
                "%s: NULL positions / steps", fn);
    KVQ_REQUIRE(std::isfinite(mscale) && std::isfinite(eps) && eps >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: mscale / eps", fn);
    const int64_t wq = (int64_t)L->n_q_heads * D, wk = (int64_t)L->n_kv_heads * D;
    KVQ_REQUIRE((!q || q_stride >= wq) && (!k || k_stride >= wk) && (!v || v_stride >= wk), KVQ_ERR_INVALID_ARG,
                "%s: a token stride below the row's width", fn);
    KVQ_REQUIRE((q_stride | k_stride | v_stride) % 8 == 0, KVQ_ERR_INVALID_ARG, "%s: strides must be multiples of 8",
                fn);
    KVQ_REQUIRE(kvq_aligned16(q) && kvq_aligned16(k) && kvq_aligned16(v) && kvq_aligned16(q_out) && kvq_aligned16(k_out) && kvq_aligned16(v_out),
                KVQ_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned", fn);
    // in place only where every row is written where it was read (v in place would be no work at all)
    KVQ_REQUIRE((!q || q != q_out || (dtype == KVQ_F16 && q_stride == wq)) &&
                    (!k || k != k_out || (dtype == KVQ_F16 && k_stride == wk)) &&
                    (!v || v != v_out || (dtype == KVQ_F16 && v_stride == wk)),
                KVQ_ERR_INVALID_ARG, "%s: in place needs fp16 rows without gaps", fn);
    RopeArgs a;
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.qw = q_weight, a.kw = k_weight;
    a.eps = eps, a.mscale = mscale;
    a.pos = positions, a.steps = steps;
    a.rot = q || k ? rope->rot_dim : 0;   // (v alone is cast: positions and steps may then be NULL)
    a.Hq = q ? L->n_q_heads : 0, a.Hk = k ? L->n_kv_heads : 0, a.Hv = v ? L->n_kv_heads : 0;
    a.n = n_tokens;
    a.qo = q_out, a.ko = k_out, a.vo = v_out;
    // one token per CTA until every SM has CTAs enough to hide the loads' latency, then more, which share the
    // CTA's start: 4 (2000 tokens 9.3 us, with 8 10.8 us), and RP_TOK when there are many waves of them
    // (32768 tokens 125 us, with 4 127 us, with 2 133 us)
    const int64_t sms = kvq_num_sms();
    const int tpc = n_tokens <= 8 * sms ? 1 : n_tokens <= 32 * sms ? 4 : RP_TOK;
    const int64_t grid = (n_tokens + tpc - 1) / tpc;
    KVQ_REQUIRE(grid <= INT32_MAX, KVQ_ERR_UNSUPPORTED, "%s: n_tokens", fn);
    const auto go = [&](auto kernel) {
        const cudaError_t e = kvq_launch_pdl(kernel, dim3((unsigned)grid), dim3(RP_NT), 0, kvq_stream(stream), a, tpc);
        if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
        return (int)KVQ_OK;
    };
    if (dtype == KVQ_F16)
        return rope->interleaved ? go(norm_rope_kernel<__half, true>) : go(norm_rope_kernel<__half, false>);
    return rope->interleaved ? go(norm_rope_kernel<__nv_bfloat16, true>) : go(norm_rope_kernel<__nv_bfloat16, false>);
}

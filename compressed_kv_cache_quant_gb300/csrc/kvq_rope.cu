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
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "kvq_internal.cuh"

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

__device__ __forceinline__ void unpack(const uint4& w, float* x, __half*) {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void unpack(const uint4& w, float* x, __nv_bfloat16*) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack_half(const float* x) {
    uint4 w;
    __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    return w;
}

// the pairs (u, v) and (p, q) by the angles whose cosines and sines are f = (cos, sin, cos, sin)
__device__ __forceinline__ void turn_two(float* u, float* v, float* p, float* q, float4 f) {
    const float x = *u, y = *v, z = *p, w = *q;
    *u = x * f.x - y * f.y;
    *v = y * f.x + x * f.y;
    *p = z * f.z - w * f.w;
    *q = w * f.z + z * f.w;
}

// The two 8-value chunks of a head row that lane l (< 8) of a group holds.  Half layout: chunk c pairs
// with chunk c + rot/16, and the chunks behind the rotated part go to the remaining lanes.
template <bool INTER>
__device__ __forceinline__ void chunks(int l, int rot, int* a, int* b) {
    const int half = rot >> 4;
    if (INTER) {
        *a = l;
        *b = l + 8;
    } else if (l < half) {
        *a = l;
        *b = l + half;
    } else {
        *a = 2 * l;
        *b = 2 * l + 1;
    }
}

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
    // cosines and sines by the lane that uses them: entry 8j + l holds the j-th two pairs of lane l, so that
    // a group's 16-byte loads cover neighbouring words
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
        const uint64_t ph = (uint64_t)(int64_t)a.pos[t0 + k] * a.steps[p];
        float s, c;
        sincospif(__ll2float_rn((long long)ph) * 1.0842021724855044e-19f, &s, &c);  // * 2^-63: half turns
        const int lane = INTER ? (p >> 2) & 7 : p >> 3, nth = INTER ? (p >> 5) * 4 + (p & 3) : p & 7;
        cs[k][((nth >> 1) * 8 + lane) * 2 + (nth & 1)] = make_float2(c * a.mscale, s * a.mscale);
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
        if (now.w != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
            // the 8 lanes of a group run the same trip count, so the mask is the group's own lanes
            const unsigned m = 0xffu << (threadIdx.x & 24);
            ss += __shfl_xor_sync(m, ss, 1);
            ss += __shfl_xor_sync(m, ss, 2);
            ss += __shfl_xor_sync(m, ss, 4);
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 u = *reinterpret_cast<const float4*>(now.w + 8 * ca + i);
                const float4 v = *reinterpret_cast<const float4*>(now.w + 8 * cb + i);
                x[i] *= inv * u.x, x[i + 1] *= inv * u.y, x[i + 2] *= inv * u.z, x[i + 3] *= inv * u.w;
                y[i] *= inv * v.x, y[i + 1] *= inv * v.y, y[i + 2] *= inv * v.z, y[i + 3] *= inv * v.w;
            }
        }
        if (now.turn) {
            const float4* f = reinterpret_cast<const float4*>(cs[tn]) + l;
            if (INTER) {
                if (8 * ca < a.rot) turn_two(&x[0], &x[1], &x[2], &x[3], f[0]), turn_two(&x[4], &x[5], &x[6], &x[7], f[8]);
                if (8 * cb < a.rot) turn_two(&y[0], &y[1], &y[2], &y[3], f[16]), turn_two(&y[4], &y[5], &y[6], &y[7], f[24]);
            } else if (16 * l < a.rot) {
#pragma unroll
                for (int j = 0; j < 4; ++j) turn_two(&x[2 * j], &y[2 * j], &x[2 * j + 1], &y[2 * j + 1], f[8 * j]);
            }
        }
        *reinterpret_cast<uint4*>(now.dst + 8 * ca) = pack_half(x);
        *reinterpret_cast<uint4*>(now.dst + 8 * cb) = pack_half(y);
    }
}

int rope_spec_ok(const kvq_rope* r, const char* fn) {
    KVQ_REQUIRE(r != nullptr, KVQ_ERR_INVALID_ARG, "%s: NULL rope", fn);
    KVQ_REQUIRE(r->rot_dim >= 0 && r->rot_dim <= D && r->rot_dim % 16 == 0, KVQ_ERR_UNSUPPORTED,
                "%s: rot_dim %d (a multiple of 16 up to 128)", fn, r->rot_dim);
    KVQ_REQUIRE(r->interleaved == 0 || r->interleaved == 1, KVQ_ERR_INVALID_ARG, "%s: interleaved", fn);
    return KVQ_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

extern "C" int kvq_rope_steps(const kvq_rope* r, uint64_t* steps, float* mscale) {
    kvq_clear_error();
    const int st = rope_spec_ok(r, "kvq_rope_steps");
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
    st = rope_spec_ok(rope, fn);
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
    KVQ_REQUIRE(aligned16(q) && aligned16(k) && aligned16(v) && aligned16(q_out) && aligned16(k_out) && aligned16(v_out),
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

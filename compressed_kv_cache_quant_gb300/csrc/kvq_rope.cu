// kv_qk_norm_rope: RMS norms of the query and key heads and their rotary positions in one pass over a
// projection's rows, and the host helper that lays out the rotation's frequencies.
//
// Positions.  A pair that turns f radians per position is at angle p * f.  At long positions an fp32
// product loses it (p * f near 1e5 rad has 8e-3 rad steps) and fp64 arithmetic is slow on this GPU, so
// frequencies are kept in turns as 64-bit fractions, step = round(f / 2pi * 2^64): the wrapping integer
// product p * step IS the angle modulo one turn, off by at most |p| * 2^-65 turns.  Its top bits as a
// signed fp32 fraction go to sincospif.
//
// Bound: bytes (every head row is read and written once, about 3 flops per byte).  One CTA takes a few
// tokens: 256 threads compute the tokens' cosines and sines once into shared memory (64 pairs per token,
// reused by every head), then every group of 8 lanes takes whole head rows, 16 values per lane as two
// 16-byte loads, so a row's norm is three shuffles and both members of every pair are in one lane.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "kvq_internal.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int RP_NT = 256;
constexpr int RP_GROUPS = RP_NT / 8;  // head rows in flight per CTA
constexpr int RP_TOK = 4;             // most tokens per CTA

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

template <typename T, bool INTER>
__global__ void __launch_bounds__(RP_NT) norm_rope_kernel(RopeArgs a, int tok_per_cta) {
    __shared__ float2 cs[RP_TOK][D / 2];
    const int64_t t0 = (int64_t)blockIdx.x * tok_per_cta;
    const int nt = (int)min((int64_t)tok_per_cta, a.n - t0);
    const int half = a.rot >> 1;
    for (int i = threadIdx.x; i < nt * (D / 2); i += RP_NT) {
        const int t = i / (D / 2), p = i % (D / 2);
        if (p >= half) continue;
        const uint64_t ph = (uint64_t)(int64_t)a.pos[t0 + t] * a.steps[p];
        float s, c;
        sincospif(__ll2float_rn((long long)ph) * 1.0842021724855044e-19f, &s, &c);  // * 2^-63: half turns
        cs[t][p] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();
    const int l = threadIdx.x & 7;
    const int rows = a.Hq + a.Hk + a.Hv;
    int ca, cb;
    chunks<INTER>(l, a.rot, &ca, &cb);
    for (int r = threadIdx.x >> 3; r < nt * rows; r += RP_GROUPS) {
        const int t = r / rows, h = r % rows;
        const int64_t tok = t0 + t;
        const T* src;
        uint16_t* dst;
        const float* w = nullptr;
        bool turn = true;
        if (h < a.Hq) {
            src = static_cast<const T*>(a.q) + tok * a.q_stride + h * D;
            dst = a.qo + (tok * a.Hq + h) * D;
            w = a.qw;
        } else if (h < a.Hq + a.Hk) {
            src = static_cast<const T*>(a.k) + tok * a.k_stride + (h - a.Hq) * D;
            dst = a.ko + (tok * a.Hk + h - a.Hq) * D;
            w = a.kw;
        } else {
            src = static_cast<const T*>(a.v) + tok * a.v_stride + (h - a.Hq - a.Hk) * D;
            dst = a.vo + (tok * a.Hv + h - a.Hq - a.Hk) * D;
            turn = false;
        }
        float x[8], y[8];
        unpack(*reinterpret_cast<const uint4*>(src + 8 * ca), x, (T*)nullptr);
        unpack(*reinterpret_cast<const uint4*>(src + 8 * cb), y, (T*)nullptr);
        if (w != nullptr) {
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
            for (int i = 0; i < 8; ++i) {
                x[i] *= inv * w[8 * ca + i];
                y[i] *= inv * w[8 * cb + i];
            }
        }
        if (turn) {
            if (INTER) {
                if (8 * ca < a.rot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = cs[t][4 * ca + i];
                        const float u = x[2 * i], v = x[2 * i + 1];
                        x[2 * i] = u * f.x - v * f.y;
                        x[2 * i + 1] = v * f.x + u * f.y;
                    }
                }
                if (8 * cb < a.rot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = cs[t][4 * cb + i];
                        const float u = y[2 * i], v = y[2 * i + 1];
                        y[2 * i] = u * f.x - v * f.y;
                        y[2 * i + 1] = v * f.x + u * f.y;
                    }
                }
            } else if (16 * l < a.rot) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = cs[t][8 * l + i];
                    const float u = x[i], v = y[i];
                    x[i] = u * f.x - v * f.y;
                    y[i] = v * f.x + u * f.y;
                }
            }
        }
        *reinterpret_cast<uint4*>(dst + 8 * ca) = pack_half(x);
        *reinterpret_cast<uint4*>(dst + 8 * cb) = pack_half(y);
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
    a.rot = rope->rot_dim;
    a.Hq = q ? L->n_q_heads : 0, a.Hk = k ? L->n_kv_heads : 0, a.Hv = v ? L->n_kv_heads : 0;
    a.n = n_tokens;
    a.qo = q_out, a.ko = k_out, a.vo = v_out;
    // one token per CTA until every SM has CTAs enough to hide the loads' latency, then RP_TOK, which
    // shares the launch and the angles' latency
    const int tpc = n_tokens <= 8 * (int64_t)kvq_num_sms() ? 1 : RP_TOK;
    const int64_t grid = (n_tokens + tpc - 1) / tpc;
    KVQ_REQUIRE(grid <= INT32_MAX, KVQ_ERR_UNSUPPORTED, "%s: n_tokens", fn);
    const auto go = [&](auto kernel) {
        kernel<<<(unsigned)grid, RP_NT, 0, kvq_stream(stream)>>>(a, tpc);
        return kvq_launch_status(fn);
    };
    if (dtype == KVQ_F16)
        return rope->interleaved ? go(norm_rope_kernel<__half, true>) : go(norm_rope_kernel<__half, false>);
    return rope->interleaved ? go(norm_rope_kernel<__nv_bfloat16, true>) : go(norm_rope_kernel<__nv_bfloat16, false>);
}

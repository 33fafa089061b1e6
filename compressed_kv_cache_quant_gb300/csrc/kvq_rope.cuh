// What kv_qk_norm_rope, kv_rope_append and kv_latent_append share: 16-byte groups of fp16 and bf16 values, the
// rotation of pairs, and the angle of a position.
#pragma once

#include <cuda_bf16.h>

#include "kvq_internal.cuh"

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

// Where pair p's cosine and sine lie in a token's 64 entries: by the lane that uses them, entries 16j + 2l and
// 16j + 2l + 1 hold the j-th two pairs of lane l, so that a group's 16-byte loads cover neighbouring words.
template <bool INTER>
__device__ __forceinline__ int pair_entry(int p) {
    const int lane = INTER ? (p >> 2) & 7 : p >> 3, nth = INTER ? (p >> 5) * 4 + (p & 3) : p & 7;
    return ((nth >> 1) * 8 + lane) * 2 + (nth & 1);
}

// The head row that a group of 8 lanes holds (chunks ca and cb of each lane), rotated by its token's entries.
template <bool INTER>
__device__ __forceinline__ void turn_row(float* x, float* y, const float2* cs, int l, int ca, int cb, int rot) {
    const float4* f = reinterpret_cast<const float4*>(cs) + l;
    if (INTER) {
        if (8 * ca < rot) turn_two(&x[0], &x[1], &x[2], &x[3], f[0]), turn_two(&x[4], &x[5], &x[6], &x[7], f[8]);
        if (8 * cb < rot) turn_two(&y[0], &y[1], &y[2], &y[3], f[16]), turn_two(&y[4], &y[5], &y[6], &y[7], f[24]);
    } else if (16 * l < rot) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn_two(&x[2 * j], &y[2 * j], &x[2 * j + 1], &y[2 * j + 1], f[8 * j]);
    }
}

// The same row normed: y = x w / sqrt(mean x^2 + eps), w the weights in shared memory.  Every lane of the group
// makes the same call, so the mask is the group's own lanes.
__device__ __forceinline__ void norm_row(float* x, float* y, const float* w, int ca, int cb, float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
    const unsigned m = 0xffu << (threadIdx.x & 24);
    ss += __shfl_xor_sync(m, ss, 1);
    ss += __shfl_xor_sync(m, ss, 2);
    ss += __shfl_xor_sync(m, ss, 4);
    const float inv = 1.0f / sqrtf(ss * (1.0f / KVQ_HEAD_DIM) + eps);
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(w + 8 * ca + i);
        const float4 v = *reinterpret_cast<const float4*>(w + 8 * cb + i);
        x[i] *= inv * u.x, x[i + 1] *= inv * u.y, x[i + 2] *= inv * u.z, x[i + 3] *= inv * u.w;
        y[i] *= inv * v.x, y[i + 1] *= inv * v.y, y[i + 2] *= inv * v.z, y[i + 3] *= inv * v.w;
    }
}

// Cosine and sine of position pos under a pair's step (its turns per position as a 64-bit fraction: the wrapping
// product is the angle modulo one turn, without a rounding).
__device__ __forceinline__ float2 kvq_cos_sin(int32_t pos, uint64_t step, float mscale) {
    const uint64_t ph = (uint64_t)(int64_t)pos * step;
    float s, c;
    sincospif(__ll2float_rn((long long)ph) * 1.0842021724855044e-19f, &s, &c);  // * 2^-63: half turns
    return make_float2(c * mscale, s * mscale);
}

// Checks the fields of a rotation that a kernel reads.
static inline int kvq_check_rope(const kvq_rope* r, const char* fn) {
    KVQ_REQUIRE(r != nullptr, KVQ_ERR_INVALID_ARG, "%s: NULL rope", fn);
    KVQ_REQUIRE(r->rot_dim >= 0 && r->rot_dim <= KVQ_HEAD_DIM && r->rot_dim % 16 == 0, KVQ_ERR_UNSUPPORTED,
                "%s: rot_dim %d (a multiple of 16 up to 128)", fn, r->rot_dim);
    KVQ_REQUIRE(r->interleaved == 0 || r->interleaved == 1, KVQ_ERR_INVALID_ARG, "%s: interleaved", fn);
    return KVQ_OK;
}

static inline bool kvq_aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

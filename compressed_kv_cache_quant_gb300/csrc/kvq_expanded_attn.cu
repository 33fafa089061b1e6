// kv_latent_expanded_attn.
//
// A warp per (row, head): the query and the running output in registers, a softmax with a running maximum over the
// keys that the row sees.
#include <algorithm>
#include <cmath>

#include "kvq_attn_mod.cuh"
#include "kvq_latent.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int PG = KVQ_BLOCK_TOKENS;
constexpr int LAT = KVQ_LATENT_DIM, ROT = KVQ_LATENT_ROPE, ROW = LAT + ROT;

__device__ __forceinline__ int find_seq(const int32_t* starts, int batch, int64_t row) {
    int b = 0;
    while (b < batch && starts[b + 1] <= row) ++b;
    return b;
}

struct ExpArgs {
    const uint16_t *q, *kn, *kr, *v;
    int64_t kn_stride, kn_head, kr_stride, v_stride, v_head, n_keys, n_rows;
    const int32_t *q_starts, *k_starts;
    int32_t batch, H, max_new, max_len;
    float scale2;
    uint16_t* out;
    float* lse;
    KvqWsHeader* hdr;
};

__global__ void __launch_bounds__(128) expanded_simple_kernel(ExpArgs a) {
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
    kvq_pdl_begin();
    const int b = find_seq(a.q_starts, a.batch, row);
    if (b >= a.batch || row < a.q_starts[b] || h >= a.H) return;
    const int first = a.q_starts[b], k0 = a.k_starts[b];
    const int64_t cnt = (int64_t)a.q_starts[b + 1] - first, T = (int64_t)a.k_starts[b + 1] - k0;
    if (first < 0 || k0 < 0 || cnt < 0 || cnt > a.max_new || first + cnt > a.n_rows || T < cnt || T > a.max_len || k0 + T > a.n_keys) {
        kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return;
    }
    const uint16_t* qr = a.q + (row * a.H + h) * (D + ROT);
    float q[6], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    for (int x = 0; x < 6; ++x) q[x] = kvq_h2f(qr[lane + 32 * x]);
    const int end = (int)(T - cnt + (row - first) + 1);
    for (int j = 0; j < end; ++j) {
        const uint16_t* kn = a.kn + (int64_t)(k0 + j) * a.kn_stride + h * a.kn_head;
        const uint16_t* kr = a.kr + (int64_t)(k0 + j) * a.kr_stride;
        const uint16_t* v = a.v + (int64_t)(k0 + j) * a.v_stride + h * a.v_head;
        float s = 0.0f;
        for (int x = 0; x < 4; ++x) s = fmaf(q[x], kvq_h2f(kn[lane + 32 * x]), s);
        for (int x = 0; x < 2; ++x) s = fmaf(q[4 + x], kvq_h2f(kr[lane + 32 * x]), s);
        s = kvq_warp_sum(s) * a.scale2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn, l = l * f + p;
        for (int x = 0; x < 4; ++x) o[x] = o[x] * f + p * kvq_h2f(v[lane + 32 * x]);
    }
    uint16_t* dst = a.out + (row * a.H + h) * D;
    for (int x = 0; x < 4; ++x) dst[lane + 32 * x] = kvq_f2h(l > 0.0f ? o[x] / l : 0.0f);
    if (a.lse != nullptr && lane == 0) a.lse[row * a.H + h] = l > 0.0f ? (m + log2f(l)) * KVQ_LN2 : -INFINITY;
}

}  // namespace

static int check_expanded(int32_t batch, int32_t n_heads, int64_t n_rows, int32_t max_new, int32_t max_len, const char* fn) {
    KVQ_REQUIRE(batch >= 0 && max_len >= 0, KVQ_ERR_INVALID_ARG, "%s: negative sizes", fn);
    KVQ_REQUIRE(max_len <= 1 << 30, KVQ_ERR_UNSUPPORTED, "%s: max_len %d (at most 2^30)", fn, max_len);
    return check_latent_rows(n_heads, n_rows, max_new, false, fn);
}

extern "C" size_t kv_latent_expanded_attn_ws(int32_t batch, int32_t n_heads, int64_t n_rows, int32_t max_new, int32_t max_len) {
    kvq_clear_error();
    if (check_expanded(batch, n_heads, n_rows, max_new, max_len, "kv_latent_expanded_attn_ws")) return 0;
    return sizeof(KvqWsHeader);
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
    ExpArgs a;
    if (!st) st = latent_scale(scale, fn, &a.scale2);
    if (!st) st = kvq_check_ws(ws, ws_bytes, kv_latent_expanded_attn_ws(batch, n_heads, n_rows, max_new, max_len), fn);
    if (st) return st;
    KVQ_REQUIRE(n_keys >= 0 && n_keys <= INT32_MAX, KVQ_ERR_INVALID_ARG, "%s: n_keys", fn);
    if (batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && q_starts && k_starts && (n_keys == 0 || (k_nope && k_rope && v)), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_nope | (uintptr_t)k_rope | (uintptr_t)v) & 15u) == 0,
                KVQ_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned", fn);
    KVQ_REQUIRE((kn_stride | kn_head_stride | kr_stride | v_stride | v_head_stride) % 8 == 0, KVQ_ERR_INVALID_ARG,
                "%s: strides must be multiples of 8", fn);
    KVQ_REQUIRE(kn_stride >= D && kn_head_stride >= D && v_stride >= D && v_head_stride >= D && kr_stride >= ROT,
                KVQ_ERR_INVALID_ARG, "%s: a stride below the row's width", fn);
    a.q = q, a.kn = k_nope, a.kr = k_rope, a.v = v;
    a.kn_stride = kn_stride, a.kn_head = kn_head_stride, a.kr_stride = kr_stride, a.v_stride = v_stride, a.v_head = v_head_stride;
    a.n_keys = n_keys, a.n_rows = n_rows, a.q_starts = q_starts, a.k_starts = k_starts;
    a.batch = batch, a.H = n_heads, a.max_new = max_new, a.max_len = max_len;
    a.out = out, a.lse = lse, a.hdr = static_cast<KvqWsHeader*>(ws);
    const cudaError_t e = kvq_launch_pdl(expanded_simple_kernel, dim3((unsigned)n_rows, (n_heads + 3) / 4), dim3(128), 0, kvq_stream(stream), a);
    if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return KVQ_OK;
}

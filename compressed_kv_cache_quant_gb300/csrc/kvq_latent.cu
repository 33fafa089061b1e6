// kv_latent_attn and kv_latent_expanded_attn.
//
// A warp per (row, head): the query and the running output in registers, a softmax with a running maximum over the
// keys that the row sees.
#include <algorithm>
#include <cmath>

#include "kvq_attn_mod.cuh"
#include "kvq_tree.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int PG = KVQ_BLOCK_TOKENS;
constexpr int LAT = KVQ_LATENT_DIM, ROT = KVQ_LATENT_ROPE, ROW = LAT + ROT;

struct LatArgs {
    const uint16_t *q, *rows;
    const int32_t *bt, *seq_lens, *q_starts, *parents;
    int64_t n_rows, num_blocks;
    int32_t batch, max_blocks, max_len, max_new, H;
    float scale2;    // in log2 units
    uint16_t* out;
    float* lse;
    KvqWsHeader* hdr;
};

__device__ __forceinline__ int find_seq(const int32_t* starts, int batch, int64_t row) {
    int b = 0;
    while (b < batch && starts[b + 1] <= row) ++b;
    return b;
}

__global__ void __launch_bounds__(128) latent_simple_kernel(LatArgs a) {
    __shared__ KvqTree tree;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
    kvq_pdl_begin();
    const int b = find_seq(a.q_starts, a.batch, row);
    if (b >= a.batch || row < a.q_starts[b]) return;
    const int first = a.q_starts[b], T = a.seq_lens[b];
    const int64_t cnt = (int64_t)a.q_starts[b + 1] - first;
    if (first < 0 || cnt < 0 || cnt > a.max_new || first + cnt > a.n_rows || T < cnt || T > a.max_len) {
        kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return;
    }
    const int n = (int)cnt, i = (int)(row - first), ctx = T - n;
    if (a.parents != nullptr) {
        for (int k = threadIdx.x; k < n; k += 128) kvq_tree_fetch(tree, a.parents + first, k, a.hdr);
        __syncthreads();
        if (threadIdx.x == 0) kvq_tree_walk(tree, i);
        __syncthreads();
    }
    if (h >= a.H) return;
    const uint16_t* qr = a.q + (row * a.H + h) * ROW;
    float q[ROW / 32], o[LAT / 32], m = -INFINITY, l = 0.0f;
    for (int x = 0; x < ROW / 32; ++x) q[x] = kvq_h2f(qr[lane + 32 * x]);
    for (int x = 0; x < LAT / 32; ++x) o[x] = 0.0f;
    const int end = a.parents ? T : ctx + i + 1;
    for (int j = 0; j < end; ++j) {
        if (a.parents && j >= ctx && !(tree.path[i][(j - ctx) >> 5] >> ((j - ctx) & 31) & 1)) continue;
        const int32_t page = a.bt[(int64_t)b * a.max_blocks + j / PG];
        if (page < 0 || page >= a.num_blocks) {
            kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
            continue;
        }
        const uint16_t* kr = a.rows + ((int64_t)page * PG + j % PG) * ROW;
        float k[ROW / 32], s = 0.0f;
        for (int x = 0; x < ROW / 32; ++x) k[x] = kvq_h2f(kr[lane + 32 * x]), s = fmaf(q[x], k[x], s);
        s = kvq_warp_sum(s) * a.scale2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn, l = l * f + p;
        for (int x = 0; x < LAT / 32; ++x) o[x] = o[x] * f + p * k[x];
    }
    uint16_t* dst = a.out + (row * a.H + h) * LAT;
    for (int x = 0; x < LAT / 32; ++x) dst[lane + 32 * x] = kvq_f2h(l > 0.0f ? o[x] / l : 0.0f);
    if (a.lse != nullptr && lane == 0) a.lse[row * a.H + h] = l > 0.0f ? (m + log2f(l)) * KVQ_LN2 : -INFINITY;
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

int check_latent_rows(int32_t n_heads, int64_t n_rows, int32_t max_new, bool tree, const char* fn) {
    KVQ_REQUIRE(n_heads > 0 && n_heads <= 1 << 16, KVQ_ERR_INVALID_ARG, "%s: n_heads", fn);
    KVQ_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX && max_new >= 0 && (n_rows == 0 || max_new > 0), KVQ_ERR_INVALID_ARG,
                "%s: n_rows / max_new", fn);
    KVQ_REQUIRE(!tree || max_new <= KVQ_TREE_MAX, KVQ_ERR_UNSUPPORTED, "%s: max_new %d (trees: at most %d)", fn, max_new,
                KVQ_TREE_MAX);
    return KVQ_OK;
}

// the scale of a score in log2 units, combined in fp64 and rounded once
int latent_scale(float scale, const char* fn, float* scale2) {
    KVQ_REQUIRE(std::isfinite(scale) && scale >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    *scale2 = (float)((scale > 0.0f ? (double)scale : 0.07216878364870322) * 1.44269504088896340736);   // 1/sqrt(192)
    KVQ_REQUIRE(std::isfinite(*scale2), KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    return KVQ_OK;
}

}  // namespace

extern "C" size_t kv_latent_attn_ws(const kvq_seqs* S, int32_t n_heads, int64_t n_rows, int32_t max_new) {
    static const char* fn = "kv_latent_attn_ws";
    if (kvq_check_seqs_sizes(S, fn) || kvq_check_max_len(S, fn) || check_latent_rows(n_heads, n_rows, max_new, false, fn)) return 0;
    return sizeof(KvqWsHeader);
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
    if (!st) st = kvq_check_ws(ws, ws_bytes, kv_latent_attn_ws(S, n_heads, n_rows, max_new), fn);
    if (st) return st;
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && q_starts && (S->block_table || S->max_len == 0), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out) & 15u) == 0, KVQ_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", fn);
    a.q = q, a.rows = C->rows, a.bt = S->block_table, a.seq_lens = S->seq_lens, a.q_starts = q_starts, a.parents = parents;
    a.n_rows = n_rows, a.num_blocks = C->num_blocks;
    a.batch = S->batch, a.max_blocks = S->max_blocks, a.max_len = S->max_len, a.max_new = max_new, a.H = n_heads;
    a.out = out, a.lse = lse, a.hdr = static_cast<KvqWsHeader*>(ws);
    const cudaError_t e = kvq_launch_pdl(latent_simple_kernel, dim3((unsigned)n_rows, (n_heads + 3) / 4), dim3(128), 0, kvq_stream(stream), a);
    if (e != cudaSuccess) return kvq_fail(KVQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return KVQ_OK;
}

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

// kv_chunk_attn: attention of a run of new tokens per sequence over an fp16 layer's pages.
//
// One warp per (new token, query head), four dims per lane: the plain recurrence of the running maximum
// and sum over the visible tokens, in fp32.
#include <algorithm>

#include "kvq_attn_mod.cuh"

namespace {

constexpr int D = KVQ_HEAD_DIM;
constexpr int PG = KVQ_BLOCK_TOKENS;
constexpr int CA_NT = 128;

struct ChunkArgs {
    const uint16_t *k16, *v16, *q;
    int64_t num_blocks;
    const int32_t *bt, *seq_lens, *q_starts;
    int32_t batch, max_blocks, max_len, max_new, H, GQ;
    int64_t n_rows;
    KvqModArgs mod;
    uint16_t* out;
    float* lse;
    KvqWsHeader* hdr;
};

__global__ void __launch_bounds__(CA_NT) chunk_attn_kernel(ChunkArgs a) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int Hq = a.H * a.GQ;
    const int64_t item = (int64_t)blockIdx.x * (CA_NT / 32) + (threadIdx.x >> 5);
    const int i = (int)(item / Hq), hq = (int)(item % Hq);
    const int first = a.q_starts[b], n = a.q_starts[b + 1] - first, T = a.seq_lens[b];
    if (first < 0 || n < 0 || n > a.max_new || (int64_t)first + n > a.n_rows || T < n || T > a.max_len) {
        if (item == 0 && lane == 0) kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return;
    }
    if (i >= n) return;
    const int64_t row = ((int64_t)first + i) * Hq + hq;
    const int pos = T - n + i;
    const KvqSee see = kvq_see(a.mod, pos, T, a.mod.prefix_len ? a.mod.prefix_len[b] : 0,
                               a.mod.doc_start ? a.mod.doc_start[first + i] : 0);
    const float slope = a.mod.slopes ? a.mod.slopes[hq] * KVQ_LOG2E : 0.0f;
    float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    for (int c = 0; c < 4; ++c) q[c] = kvq_h2f(a.q[row * D + 4 * lane + c]);
    for (int j = see.sink > see.doc ? see.doc : see.lo; j < see.hi; ++j) {
        if (!see(j)) {
            j = max(j, see.lo - 1);
            continue;
        }
        const int32_t page = a.bt[(int64_t)b * a.max_blocks + j / PG];
        if (page < 0 || page >= a.num_blocks) {
            if (lane == 0) kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
            continue;
        }
        const int64_t at = (((int64_t)page * a.H + hq / a.GQ) * PG + j % PG) * D + 4 * lane;
        float s = 0.0f;
        for (int c = 0; c < 4; ++c) s += q[c] * kvq_h2f(a.k16[at + c]);
        s = kvq_warp_sum(s);
        s = a.mod.post != 0.0f ? a.mod.post * kvq_tanh(s * a.mod.pre) : s * a.mod.pre;
        s -= slope * (float)abs(pos - j);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
        for (int c = 0; c < 4; ++c) o[c] = o[c] * f + p * kvq_h2f(a.v16[at + c]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int c = 0; c < 4; ++c) a.out[row * D + 4 * lane + c] = kvq_f2h(o[c] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * KVQ_LN2;
}

int check_rows(int64_t n_rows, int32_t max_new, const char* fn) {
    KVQ_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX && max_new >= 0 && (n_rows == 0 || max_new > 0), KVQ_ERR_INVALID_ARG,
                "%s: n_rows / max_new", fn);
    return KVQ_OK;
}

}  // namespace

extern "C" size_t kv_chunk_attn_ws(const kvq_layout* L, const kvq_seqs* S, int64_t n_rows, int32_t max_new) {
    if (kvq_check_layout(L, "kv_chunk_attn_ws", true) || kvq_check_seqs_sizes(S, "kv_chunk_attn_ws") ||
        check_rows(n_rows, max_new, "kv_chunk_attn_ws"))
        return 0;
    return sizeof(KvqWsHeader);
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
    if (st) return st;
    KVQ_REQUIRE(P && P->k16 && P->v16 && P->num_blocks > 0, KVQ_ERR_INVALID_ARG, "%s: pool needs k16 and v16", fn);
    KVQ_REQUIRE(S->batch <= 65535 && L->n_kv_heads <= 65535, KVQ_ERR_UNSUPPORTED, "%s: batch or heads", fn);
    st = check_rows(n_rows, max_new, fn);
    if (st) return st;
    ChunkArgs a;
    st = kvq_mod_args(mod, fn, &a.mod);
    if (st) return st;
    st = kvq_check_ws(ws, ws_bytes, sizeof(KvqWsHeader), fn);
    if (st) return st;
    if (S->batch == 0 || n_rows == 0) return KVQ_OK;
    KVQ_REQUIRE(q && out && q_starts && (S->block_table || S->max_len == 0), KVQ_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    KVQ_REQUIRE((((uintptr_t)q | (uintptr_t)out | (uintptr_t)P->k16 | (uintptr_t)P->v16) & 15u) == 0,
                KVQ_ERR_INVALID_ARG, "%s: q, out, k16 and v16 must be 16-byte aligned", fn);
    a.k16 = P->k16, a.v16 = P->v16, a.q = q;
    a.num_blocks = P->num_blocks;
    a.bt = S->block_table, a.seq_lens = S->seq_lens, a.q_starts = q_starts;
    a.batch = S->batch, a.max_blocks = S->max_blocks, a.max_len = S->max_len, a.max_new = max_new;
    a.H = L->n_kv_heads, a.GQ = L->n_q_heads / L->n_kv_heads;
    a.n_rows = n_rows;
    a.out = out, a.lse = lse;
    a.hdr = static_cast<KvqWsHeader*>(ws);
    const int64_t items = (int64_t)max_new * L->n_q_heads;
    const dim3 grid((unsigned)((items + CA_NT / 32 - 1) / (CA_NT / 32)), S->batch);
    chunk_attn_kernel<<<grid, CA_NT, 0, kvq_stream(stream)>>>(a);
    return kvq_launch_status(fn);
}

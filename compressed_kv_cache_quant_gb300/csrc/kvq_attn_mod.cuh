// The score forms shared by kv_decode_attn and kv_chunk_attn: host checks, kernel arguments and which
// cached tokens a query row sees.
#pragma once

#include <cmath>

#include "kvq_internal.cuh"

#define KVQ_LOG2E 1.4426950408889634f
#define KVQ_LN2 0.6931471805599453f

struct KvqModArgs {
    // a score q.k in the log2 domain: without a cap dot * pre; with one post * tanh(dot * pre)
    float pre, post;
    int32_t window, n_sink;  // window 0: none
    const float* slopes;
    const int32_t* prefix_len;
    const int32_t* doc_start;
};

// Fills m from the caller's descriptor (NULL: the plain softmax of q.k/sqrt(d)).
static inline int kvq_mod_args(const kvq_attn_mod* mod, const char* fn, KvqModArgs* m) {
    const float dflt = 0.08838834764831845f;  // 1/sqrt(128)
    *m = KvqModArgs{dflt * KVQ_LOG2E, 0.0f, 0, 0, nullptr, nullptr, nullptr};
    if (mod == nullptr) return KVQ_OK;
    KVQ_REQUIRE(std::isfinite(mod->scale) && mod->scale >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    KVQ_REQUIRE(std::isfinite(mod->softcap) && mod->softcap >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: softcap", fn);
    KVQ_REQUIRE(mod->window >= 0 && mod->n_sink >= 0, KVQ_ERR_INVALID_ARG, "%s: window / n_sink", fn);
    const float scale = mod->scale > 0.0f ? mod->scale : dflt;
    if (mod->softcap > 0.0f) {
        m->pre = scale / mod->softcap;
        m->post = mod->softcap * KVQ_LOG2E;
        KVQ_REQUIRE(std::isfinite(m->pre) && std::isfinite(m->post), KVQ_ERR_INVALID_ARG, "%s: scale / softcap", fn);
    } else {
        m->pre = scale * KVQ_LOG2E;
    }
    m->window = mod->window;
    m->n_sink = mod->n_sink;
    m->slopes = mod->slopes;
    m->prefix_len = mod->prefix_len;
    m->doc_start = mod->doc_start;
    return KVQ_OK;
}

// The cached tokens a query sees: [lo, hi) and, under a window, its document's first tokens [doc, sink).
struct KvqSee {
    int32_t lo, hi, doc, sink;
    __device__ __forceinline__ bool operator()(int j) const { return j < hi && (j >= lo || (j >= doc && j < sink)); }
};

// The query at position i of a sequence of T tokens (0 <= i < T).
__device__ __forceinline__ KvqSee kvq_see(const KvqModArgs& m, int i, int T, int prefix, int doc) {
    KvqSee s;
    s.doc = max(doc, 0);
    s.hi = min(max(i + 1, prefix), T);
    s.lo = s.doc;
    s.sink = s.doc;
    if (m.window > 0) {
        s.lo = max(s.doc, i - m.window + 1);
        s.sink = min(s.doc < T ? s.doc + min(m.n_sink, T) : s.doc, s.hi);
    }
    return s;
}

// tanh to about 1 ulp of the larger of |x| and its use: 1 - 2/(1 + e^2x) away from zero (absolute error
// 1e-7), the odd series near zero, where the former cancels.
__device__ __forceinline__ float kvq_tanh(float x) { return tanhf(x); }

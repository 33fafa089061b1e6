// The score forms shared by kv_decode_attn, kv_chunk_attn and kv_tree_attn: host checks, kernel arguments and which
// cached tokens a query row sees.
#pragma once

#include <cmath>

#include "kvq_internal.cuh"

#define KVQ_LOG2E 1.4426950408889634f
#define KVQ_LN2 0.6931471805599453f

struct KvqModArgs {
    // a score q.k in the log2 domain: without a cap dot * pre; with one post * tanh(dot * pre)
    float pre, post;
    float lin;               // the score without its cap: dot * lin
    int32_t window, n_sink;  // window 0: none
    const float* slopes;
    const int32_t* prefix_len;
    const int32_t* doc_start;
};

// Fills m from the caller's descriptor (NULL: the plain softmax of q.k/sqrt(d)).
static inline int kvq_mod_args(const kvq_attn_mod* mod, const char* fn, KvqModArgs* m) {
    // constants are combined in fp64 and rounded once
    const double dflt = 0.08838834764831844055, log2e = 1.44269504088896340736;  // 1/sqrt(128)
    const float plain = (float)(dflt * log2e);
    *m = KvqModArgs{plain, 0.0f, plain, 0, 0, nullptr, nullptr, nullptr};
    if (mod == nullptr) return KVQ_OK;
    KVQ_REQUIRE(std::isfinite(mod->scale) && mod->scale >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    KVQ_REQUIRE(std::isfinite(mod->softcap) && mod->softcap >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: softcap", fn);
    KVQ_REQUIRE(mod->window >= 0 && mod->n_sink >= 0, KVQ_ERR_INVALID_ARG, "%s: window / n_sink", fn);
    const double scale = mod->scale > 0.0f ? (double)mod->scale : dflt;
    m->lin = (float)(scale * log2e);
    KVQ_REQUIRE(std::isfinite(m->lin), KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    if (mod->softcap > 0.0f) {
        m->pre = (float)(scale / mod->softcap);
        m->post = (float)(mod->softcap * log2e);
        KVQ_REQUIRE(std::isfinite(m->pre) && std::isfinite(m->post), KVQ_ERR_INVALID_ARG, "%s: scale / softcap", fn);
    } else {
        m->pre = m->lin;
    }
    m->window = mod->window;
    m->n_sink = mod->n_sink;
    m->slopes = mod->slopes;
    m->prefix_len = mod->prefix_len;
    m->doc_start = mod->doc_start;
    return KVQ_OK;
}

// Positions and counts of pages and tiles are 32-bit numbers, and sums of two of them have to be, too.
static inline int kvq_check_max_len(const kvq_seqs* S, const char* fn) {
    KVQ_REQUIRE(S->max_len <= 1 << 30, KVQ_ERR_UNSUPPORTED, "%s: max_len %d (at most 2^30)", fn, S->max_len);
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

// cap * tanh(scale * dot / cap) in the log2 domain.  A cap many times the scores leaves s(1 + x^2 Q(x^2)), s
// the plain score and x = s/cap: on |x| <= 3/4 (Q the polynomial through the Chebyshev points, 3e-8 of the
// score) s is rounded twice in all, where a rounded tanh near 1/5 times the cap is off by 2e-6 in the weight.
__device__ __forceinline__ float kvq_capped(const KvqModArgs& m, float dot) {
    const float x = dot * m.pre, u = x * x;
    if (!(u <= 0.5625f)) return m.post * tanhf(x);
    float q = 0.001914540189318359f;
    q = fmaf(q, u, -0.0079409284517169f);
    q = fmaf(q, u, 0.02161884680390358f);
    q = fmaf(q, u, -0.05393656715750694f);
    q = fmaf(q, u, 0.13333185017108917f);
    q = fmaf(q, u, -0.3333333134651184f);
    const float s = dot * m.lin;
    return fmaf(s, u * q, s);
}

// What the two attention forms of latent layers share: host checks and the default scale.
#pragma once

#include <cmath>

#include "kvq_internal.cuh"

constexpr int KVQ_LATENT_MAX_CTAS = 256;   // CTAs or pairs of the absorbed form, at most

static inline int check_latent_rows(int32_t n_heads, int64_t n_rows, int32_t max_new, bool tree, const char* fn) {
    KVQ_REQUIRE(n_heads > 0 && n_heads <= 1 << 16, KVQ_ERR_INVALID_ARG, "%s: n_heads", fn);
    KVQ_REQUIRE(n_rows >= 0 && n_rows <= INT32_MAX && max_new >= 0 && (n_rows == 0 || max_new > 0), KVQ_ERR_INVALID_ARG,
                "%s: n_rows / max_new", fn);
    KVQ_REQUIRE(!tree || max_new <= KVQ_TREE_MAX, KVQ_ERR_UNSUPPORTED, "%s: max_new %d (trees: at most %d)", fn, max_new,
                KVQ_TREE_MAX);
    return KVQ_OK;
}

// the scale of a score in log2 units, combined in fp64 and rounded once
static inline int latent_scale(float scale, const char* fn, float* scale2) {
    KVQ_REQUIRE(std::isfinite(scale) && scale >= 0.0f, KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    *scale2 = (float)((scale > 0.0f ? (double)scale : 0.07216878364870322) * 1.44269504088896340736);   // 1/sqrt(192)
    KVQ_REQUIRE(std::isfinite(*scale2), KVQ_ERR_INVALID_ARG, "%s: scale", fn);
    return KVQ_OK;
}

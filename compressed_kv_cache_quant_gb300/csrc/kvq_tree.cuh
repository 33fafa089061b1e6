// Trees of drafted tokens, shared by kv_tree_attn and kv_latent_attn.  Node i of a sequence is its i-th new token;
// its parent is an earlier node, or -1 where it hangs from the last cached token.
#pragma once

#include "kvq_internal.cuh"

constexpr int KVQ_TREE_WORDS = KVQ_TREE_MAX / 32;

struct KvqTree {
    int16_t parent[KVQ_TREE_MAX];
    int16_t depth[KVQ_TREE_MAX];                        // nodes above it
    // bit `shift` + k: it is node k or hangs below it (and sees it); shift: the nodes' first place modulo 32, so that a
    // word is 32 columns of the cache
    uint32_t path[KVQ_TREE_MAX][KVQ_TREE_WORDS + 1];
};

// One thread per node: fetches its parent (a flagged -1 where the entry is no earlier node).  A barrier follows.
__device__ __forceinline__ void kvq_tree_fetch(KvqTree& t, const int32_t* parents, int i, KvqWsHeader* hdr) {
    const int32_t p = parents[i];
    if (p < -1 || p >= i) kvq_dev_flag(hdr, KVQ_DEV_BAD_INDEX, p);
    t.parent[i] = (int16_t)(p < -1 || p >= i ? -1 : p);
}

// One thread per node: its depth and path.  A path goes down in the nodes' order, so the walk ends.
__device__ __forceinline__ void kvq_tree_walk(KvqTree& t, int i, int shift) {
#pragma unroll
    for (int w = 0; w <= KVQ_TREE_WORDS; ++w) t.path[i][w] = 0;
    int above = -1;
    for (int k = i; k >= 0; k = t.parent[k]) {
        t.path[i][(k + shift) >> 5] |= 1u << ((k + shift) & 31);
        ++above;
    }
    t.depth[i] = (int16_t)above;
}

// What node i sees of the 32 columns from `column` on, a multiple of 32; ctx: the nodes' first place.
__device__ __forceinline__ uint32_t kvq_tree_bits(const KvqTree& t, int i, int column, int ctx) {
    const uint32_t w = (uint32_t)((column >> 5) - (ctx >> 5));
    return w <= (uint32_t)KVQ_TREE_WORDS ? t.path[i][w] : 0u;
}

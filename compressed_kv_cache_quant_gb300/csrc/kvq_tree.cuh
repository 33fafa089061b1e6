// Trees of drafted tokens, shared by kv_tree_attn and kv_latent_attn.  Node i of a sequence is its i-th new token;
// its parent is an earlier node, or -1 where it hangs from the last cached token.
#pragma once

#include "kvq_internal.cuh"

constexpr int KVQ_TREE_WORDS = KVQ_TREE_MAX / 32;

struct KvqTree {
    int16_t parent[KVQ_TREE_MAX];
    int16_t depth[KVQ_TREE_MAX];                    // nodes above it
    uint32_t path[KVQ_TREE_MAX][KVQ_TREE_WORDS];    // bit k: it is node k or hangs below it (and sees it)
};

// One thread per node: fetches its parent (a flagged -1 where the entry is no earlier node).  A barrier follows.
__device__ __forceinline__ void kvq_tree_fetch(KvqTree& t, const int32_t* parents, int i, KvqWsHeader* hdr) {
    const int32_t p = parents[i];
    if (p < -1 || p >= i) kvq_dev_flag(hdr, KVQ_DEV_BAD_INDEX, p);
    t.parent[i] = (int16_t)(p < -1 || p >= i ? -1 : p);
}

// One thread per node: its depth and path.  A path goes down in the nodes' order, so the walk ends.
__device__ __forceinline__ void kvq_tree_walk(KvqTree& t, int i) {
#pragma unroll
    for (int w = 0; w < KVQ_TREE_WORDS; ++w) t.path[i][w] = 0;
    int above = -1;
    for (int k = i; k >= 0; k = t.parent[k]) {
        t.path[i][k >> 5] |= 1u << (k & 31);
        ++above;
    }
    t.depth[i] = (int16_t)above;
}

// 32 bits of node i's path from node `from` on (which may lie outside the tree).
__device__ __forceinline__ uint32_t kvq_tree_bits(const KvqTree& t, int i, int from) {
    const int w = from >> 5;   // (floor)
    const uint32_t lo = w >= 0 && w < KVQ_TREE_WORDS ? t.path[i][w] : 0u;
    const uint32_t hi = w + 1 >= 0 && w + 1 < KVQ_TREE_WORDS ? t.path[i][w + 1] : 0u;
    return __funnelshift_r(lo, hi, from & 31);
}

// Runs of new tokens in a paged cache: which sequence a row of the call belongs to, and where it goes.  Shared by
// the operators that write new rows.
#pragma once

#include "kvq_internal.cuh"

struct KvqNewRows {
    const int32_t *starts, *lens, *bt;   // row_starts, seq_lens, block_table
    const int32_t* pos;                  // the rows' positions, or NULL: their places in the sequence
    int64_t n_rows, num_blocks;
    int32_t batch, max_blocks, max_len;  // max_len: of what the call can hold, t_cap included
    KvqWsHeader* hdr;
};

// Sequence b's new rows: *first and their number; false (flagged) when its lengths do not fit the call.
__device__ __forceinline__ bool kvq_new_rows_of(const KvqNewRows& a, int b, int* first, int* n, int* T) {
    *first = a.starts[b];
    const int64_t cnt = (int64_t)a.starts[b + 1] - *first;
    *T = a.lens[b];
    *n = 0;
    if (*first < 0 || cnt < 0 || *first + cnt > a.n_rows || *T < cnt || *T > a.max_len) {
        kvq_dev_flag(a.hdr, KVQ_DEV_BAD_LENGTH, b);
        return false;
    }
    *n = (int)cnt;
    return true;
}

// A page of sequence b, or -1 (flagged) when its table entry is none.
__device__ __forceinline__ int32_t kvq_page_at(const KvqNewRows& a, int b, int lp) {
    const int32_t page = a.bt[(int64_t)b * a.max_blocks + lp];
    if (page >= 0 && page < a.num_blocks) return page;
    kvq_dev_flag(a.hdr, KVQ_DEV_BAD_PAGE, page);
    return -1;
}

constexpr int64_t KVQ_ROW_NO_PAGE = -1;   // its table entry is no page: queries alone are written
constexpr int64_t KVQ_ROW_NONE = -2;      // behind the last sequence, or of one whose lengths do not fit: untouched

// One warp finds where rows r0 .. r0 + nt - 1 (nt <= 8) go: at[k] = page * 16 + slot, or KVQ_ROW_*, and their
// positions.  A row's sequence is the number of sequences that end at or before it.
__device__ __forceinline__ void kvq_find_rows(const KvqNewRows& a, int64_t r0, int nt, int64_t* at, int32_t* pos) {
    const int lane = threadIdx.x & 31;
    int b = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int64_t end = b0 + lane < a.batch ? (int64_t)a.starts[b0 + lane + 1] : INT64_MAX;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = __popc(__ballot_sync(0xffffffffu, end <= r0 + k));
            if (lane == k) b += c;
        }
    }
    if (lane >= nt) return;
    const int64_t row = r0 + lane;
    int64_t to = KVQ_ROW_NONE;
    int32_t p = 0;
    int first, n, T;
    if (b < a.batch && kvq_new_rows_of(a, b, &first, &n, &T) && row >= first && row < (int64_t)first + n) {
        p = T - n + (int)(row - first);
        const int32_t page = kvq_page_at(a, b, p / KVQ_BLOCK_TOKENS);
        to = page < 0 ? KVQ_ROW_NO_PAGE : (int64_t)page * KVQ_BLOCK_TOKENS + p % KVQ_BLOCK_TOKENS;
        if (a.pos != nullptr) p = a.pos[row];
    }
    at[lane] = to;
    pos[lane] = p;
}

// Host checks shared by the calls; n_rows == 0 and batch == 0 are the caller's.
static inline int kvq_check_new_rows(const kvq_seqs* S, const int32_t* row_starts, int64_t num_blocks, const char* fn) {
    KVQ_REQUIRE(row_starts && S->block_table, KVQ_ERR_INVALID_ARG, "%s: NULL row_starts / block table", fn);
    KVQ_REQUIRE(num_blocks > 0 && num_blocks <= INT32_MAX, KVQ_ERR_INVALID_ARG, "%s: num_blocks", fn);
    KVQ_REQUIRE(S->max_len <= 1 << 30, KVQ_ERR_UNSUPPORTED, "%s: max_len %d (at most 2^30)", fn, S->max_len);
    return KVQ_OK;
}

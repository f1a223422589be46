// rows.h -- what the kernels of row plans, of 8-bit rows and of drafted trees see:
// their parameters and launchers (attn_rows.cuh, kv_q8.cu, tree.cu).
#pragma once

#include "fanout_internal.h"

namespace fanout {

// What a cache holds a value in: bf16, e2m1 with a scale per 16 values (kv_q4.cu), e4m3
// (kv_q8.cu).
enum class Pool : int32_t { bf16 = 0, q4 = 1, q8 = 2 };

// A row plan's attention. masks != null: drafted trees (the rows of a branch see its keys
// before them, and of themselves those that their masks name); tok_pos then holds the
// number of keys before a row's branch's drafted tokens for every row, and behind them
// ([R], [R]) every row's own key.
struct RowParams : SplitParams {
    const uint32_t* masks;     // [R][mask_words]
    const int32_t* positions;  // [R], read with a window only; or null
    int32_t mask_words;
};

constexpr int kMaxTreeTokens = 1024;  // drafted tokens of a branch

// 8-bit rows in and out of the pools.
struct Q8RowParams {
    const __nv_bfloat16* k_rows;
    const __nv_bfloat16* v_rows;
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    uint8_t* k_pool;
    uint8_t* v_pool;
    const int64_t* slots;
    int32_t* err;
    int64_t k_stride, v_stride;  // elements between rows
    int64_t n_slots;             // num_pages * page_size
    int32_t n_rows, H_kv, page_shift;
    int32_t align32;  // 1: every 16 values of a row start on 32 bytes
    float k_scale, v_scale;
    float k_rcp, v_rcp;  // 1 / scale, rounded to nearest
};

// Drafted trees: their rows' masks, positions and slots; the accepted path; the accepted
// rows moved together. Every pointer is device memory.
struct TreeParams {
    const int32_t* parents;      // [R]: rows grouped by branch
    const int32_t* page_table;   // [B][max_pages]
    const int32_t* suffix_lens;  // [B]: without the drafted tokens
    const int32_t* lens;         // [B]: drafted tokens
    uint32_t* masks;             // [R][words]
    int32_t* positions;          // [R]
    int64_t* slots;              // [R]
    const int64_t* draft;        // [R]
    const int64_t* target;       // [R]
    const int64_t* first;        // [B]
    int32_t* path;               // [R]: written by accept, read by keep
    int32_t* counts;             // [B]
    int64_t* next;               // [B]
    uint8_t* k_pool;
    uint8_t* v_pool;
    int32_t* err;
    int32_t num_branches, R, words, window, sinks, prefix_len, page_size, max_pages, num_pages, H_kv;
    Pool pool;
};

// Whether two arrays of n >= 1 rows share a byte. A row is `row` values of 2 bytes, the next
// one starts a_stride (b_stride) >= row values behind it; rows of one array may lie between
// those of the other.
inline bool rows_overlap(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t n,
                         int64_t row) {
    using Wide = __int128;  // (n strides may pass 64 bits)
    const Wide as = 2 * static_cast<Wide>(a_stride), bs = 2 * static_cast<Wide>(b_stride), len = 2 * row;
    const Wide a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    if (a0 >= b0 + (n - 1) * bs + len || b0 >= a0 + (n - 1) * as + len) return false;
    for (Wide i = 0, j = 0; i < n && j < n;) {  // past the rows that end first
        const Wide x = a0 + i * as, y = b0 + j * bs;
        if (x + len <= y) i += (y - len - x) / as + 1;
        else if (y + len <= x) j += (x - len - y) / bs + 1;
        else return true;
    }
    return false;
}

cudaError_t launch_attn_rows(const RowParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, int grid, cudaStream_t stream);
cudaError_t launch_attn_rows_q4(const RowParams& p, const CUtensorMap& tm_q, int grid,
                                cudaStream_t stream);
cudaError_t launch_attn_rows_q8(const RowParams& p, const CUtensorMap& tm_q,
                                const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                                cudaStream_t stream);
cudaError_t launch_attn_tree(const RowParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, Pool pool, int grid, cudaStream_t stream);
cudaError_t launch_q8_rows(const Q8RowParams& p, bool read, cudaStream_t stream);
cudaError_t launch_tree_rows(const TreeParams& p, cudaStream_t stream);
cudaError_t launch_tree_accept(const TreeParams& p, cudaStream_t stream);
cudaError_t launch_kv_keep(const TreeParams& p, cudaStream_t stream);

}  // namespace fanout

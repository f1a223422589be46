// rows_api.cpp -- the C entry points of the device page tables, of the 4-bit and 8-bit
// rows and of drafted trees: argument checks and launches (kernels in tables.cu,
// kv_q4.cu, kv_q8.cu, tree.cu).
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/fanout.h"
#include "plan.h"

using namespace fanout;

namespace {

int status_from_cuda(cudaError_t e) { return e == cudaSuccess ? FANOUT_OK : FANOUT_ECUDA; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether two arrays share a byte. What a table call reads must not be what it writes:
// its blocks do not wait for one another.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && a_bytes > 0 && b_bytes > 0 && x < y + static_cast<uint64_t>(b_bytes) &&
           y < x + static_cast<uint64_t>(a_bytes);
}
struct Array {
    const void* at;
    int64_t bytes;
};
template <size_t N, size_t M>
bool any_overlap(const Array (&read)[N], const Array (&written)[M]) {
    for (const Array& r : read)
        for (const Array& w : written)
            if (overlap(r.at, r.bytes, w.at, w.bytes)) return true;
    return false;
}

int launch_checked_tables(TableParams& p, fanout_stream_t stream) {
    const cudaError_t ce = err_word_ptr(&p.err);
    if (ce != cudaSuccess) return status_from_cuda(ce);
    return status_from_cuda(launch_tables(p, reinterpret_cast<cudaStream_t>(stream)));
}

// What the two fork calls share (clear: see TableParams).
int fork_device(const int32_t* prefix_pages, int32_t prefix_len, int32_t num_branches,
                const int32_t* suffix_lens, int32_t page_size, const int32_t* free_pages,
                int32_t n_free, const int32_t* used_in, int32_t* used_out, int32_t* page_table,
                int32_t max_pages_per_branch, int32_t* cow_pairs, int32_t clear,
                fanout_stream_t stream) {
    if (prefix_len < 0 || num_branches < 0 || page_size <= 0 || n_free < 0 ||
        max_pages_per_branch < 0)
        return FANOUT_EINVAL;
    if (num_branches > kMaxTableBranches || max_pages_per_branch > kMaxTablePages)
        return FANOUT_EUNSUPPORTED;
    const int64_t n_prefix = (static_cast<int64_t>(prefix_len) + page_size - 1) / page_size;
    if (num_branches > 0 && n_prefix > max_pages_per_branch) return FANOUT_EINVAL;
    if (num_branches > 0 && (!suffix_lens || (n_prefix > 0 && !prefix_pages) ||
                             (max_pages_per_branch > 0 && !page_table)))
        return FANOUT_EINVAL;
    if (n_free > 0 && !free_pages) return FANOUT_EINVAL;
    if (used_out && used_out == used_in) return FANOUT_EINVAL;
    for (const void* ptr : {static_cast<const void*>(prefix_pages),
                            static_cast<const void*>(suffix_lens),
                            static_cast<const void*>(free_pages),
                            static_cast<const void*>(used_in), static_cast<const void*>(used_out),
                            static_cast<const void*>(page_table),
                            static_cast<const void*>(cow_pairs)})
        if (!aligned(ptr, 4)) return FANOUT_EINVAL;
    const int64_t table_bytes = 4LL * num_branches * max_pages_per_branch;
    const int64_t n_full = prefix_len / page_size;
    // The whole prefix pages may be those of a row of the table itself: it is given its
    // own entries.
    const int64_t into = reinterpret_cast<intptr_t>(prefix_pages) - reinterpret_cast<intptr_t>(page_table);
    const bool own_row = max_pages_per_branch > 0 && into >= 0 && into < table_bytes &&
                         into % (4LL * max_pages_per_branch) == 0;
    const Array read[] = {{prefix_pages, own_row ? 0 : 4 * n_full},
                          {n_full < n_prefix && cow_pairs ? prefix_pages + n_full : nullptr, 4},
                          {suffix_lens, 4LL * num_branches},
                          {free_pages, 4LL * n_free},
                          {used_in, 4}};
    const Array written[] = {{page_table, table_bytes}, {cow_pairs, 8LL * num_branches}, {used_out, 4}};
    if (any_overlap(read, written)) return FANOUT_EINVAL;
    TableParams p{};
    p.prefix_pages = prefix_pages;
    p.suffix_lens = suffix_lens;
    p.free_pages = free_pages;
    p.used_in = used_in;
    p.used_out = used_out;
    p.page_table = page_table;
    p.cow_pairs = cow_pairs;
    p.num_branches = num_branches;
    p.prefix_len = prefix_len;
    p.page_size = page_size;
    p.n_free = n_free;
    p.max_pages = max_pages_per_branch;
    p.clear = clear;
    return launch_checked_tables(p, stream);
}

// What the two row calls check alike.
int check_rows(const void* k_rows, const void* v_rows, const void* k_pages, const void* v_pages,
               const int64_t* slots, int32_t n_rows, int64_t k_stride, int64_t v_stride,
               int32_t num_pages, int32_t H_kv, int32_t d, int32_t page_size, float k_scale,
               float v_scale) {
    if (n_rows < 0 || num_pages <= 0 || H_kv <= 0 || d <= 0 || page_size <= 0) return FANOUT_EINVAL;
    if (d != kHD) return FANOUT_EUNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return FANOUT_EUNSUPPORTED;
    if (!pool_scale_ok(k_scale) || !pool_scale_ok(v_scale)) return FANOUT_EINVAL;
    if (static_cast<int64_t>(n_rows) * H_kv >= (1LL << 31)) return FANOUT_EUNSUPPORTED;
    if (n_rows == 0) return FANOUT_OK;
    const int64_t row = static_cast<int64_t>(H_kv) * d;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
        return FANOUT_EINVAL;
    if (!k_rows || !v_rows || !k_pages || !v_pages || !slots) return FANOUT_EINVAL;
    if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_pages, 16) ||
        !aligned(v_pages, 16) || !aligned(slots, 8))
        return FANOUT_EINVAL;
    return FANOUT_OK;
}

int run_rows(Q4RowParams& p, bool read, int32_t page_size, fanout_stream_t stream) {
    const void* k = read ? static_cast<const void*>(p.k_out) : p.k_rows;
    const void* v = read ? static_cast<const void*>(p.v_out) : p.v_rows;
    if (read && rows_overlap(k, p.k_stride, v, p.v_stride, p.n_rows, static_cast<int64_t>(p.H_kv) * kHD))
        return FANOUT_EINVAL;
    p.align32 = aligned(k, 32) && aligned(v, 32) && p.k_stride % 16 == 0 && p.v_stride % 16 == 0;
    p.k_rcp6 = 1.0f / (6.0f * p.k_scale);
    p.v_rcp6 = 1.0f / (6.0f * p.v_scale);
    p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    const cudaError_t ce = err_word_ptr(&p.err);
    if (ce != cudaSuccess) return status_from_cuda(ce);
    return status_from_cuda(launch_q4_rows(p, read, reinterpret_cast<cudaStream_t>(stream)));
}

// A size in bytes, where arguments may be such that its product passes 64 bits (exact up to
// 2^53).
int64_t bytes_of(double n) { return n < 9e18 ? static_cast<int64_t>(n) : INT64_MAX; }

int run_rows_q8(Q8RowParams& p, bool read, int32_t page_size, fanout_stream_t stream) {
    const void* k = read ? static_cast<const void*>(p.k_out) : p.k_rows;
    const void* v = read ? static_cast<const void*>(p.v_out) : p.v_rows;
    const double row = static_cast<double>(p.H_kv) * kHD, last = p.n_rows - 1;
    const int64_t pool = bytes_of(row * static_cast<double>(p.n_slots));
    const Array pools[] = {{p.k_pool, pool}, {p.v_pool, pool}};
    const Array rows[] = {{k, bytes_of(2 * (last * static_cast<double>(p.k_stride) + row))},
                          {v, bytes_of(2 * (last * static_cast<double>(p.v_stride) + row))}};
    const Array slots[] = {{p.slots, 8LL * p.n_rows}};
    if (any_overlap(rows, pools) || (read ? any_overlap(slots, rows) : any_overlap(slots, pools)) ||
        (!read && overlap(p.k_pool, pool, p.v_pool, pool)) ||
        (read && rows_overlap(k, p.k_stride, v, p.v_stride, p.n_rows, static_cast<int64_t>(p.H_kv) * kHD)))
        return FANOUT_EINVAL;
    p.align32 = aligned(k, 32) && aligned(v, 32) && p.k_stride % 16 == 0 && p.v_stride % 16 == 0;
    p.k_rcp = 1.0f / p.k_scale;
    p.v_rcp = 1.0f / p.v_scale;
    p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    const cudaError_t ce = err_word_ptr(&p.err);
    if (ce != cudaSuccess) return status_from_cuda(ce);
    return status_from_cuda(launch_q8_rows(p, read, reinterpret_cast<cudaStream_t>(stream)));
}

// Whether every array is there when the call has rows (`any`) and starts where its type does.
struct Typed {
    const void* at;
    uintptr_t align;
    bool needed;
};
template <size_t N>
bool arrays_ok(const Typed (&arrays)[N]) {
    for (const Typed& a : arrays)
        if ((a.needed && !a.at) || !aligned(a.at, a.align)) return false;
    return true;
}
template <size_t N>
bool any_overlap_among(const Array (&written)[N]) {
    for (size_t i = 0; i < N; ++i)
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(written[i].at, written[i].bytes, written[j].at, written[j].bytes))
                return true;
    return false;
}

}  // namespace

namespace fanout {
// Quotients by 6 gs and sc gs (sc from 2^-9 to 448) and the values themselves
// stay normal fp32 numbers inside these bounds.
bool pool_scale_ok(float gs) { return gs >= 1e-30f && gs <= 1e30f; }
}  // namespace fanout

extern "C" {

int fanout_fork_device(const int32_t* prefix_pages, int32_t prefix_len, int32_t num_branches,
                       const int32_t* suffix_lens, int32_t page_size, const int32_t* free_pages,
                       int32_t n_free, const int32_t* used_in, int32_t* used_out,
                       int32_t* page_table, int32_t max_pages_per_branch, int32_t* cow_pairs,
                       fanout_stream_t stream) {
    return fork_device(prefix_pages, prefix_len, num_branches, suffix_lens, page_size, free_pages,
                       n_free, used_in, used_out, page_table, max_pages_per_branch, cow_pairs, 0,
                       stream);
}

int fanout_fork_device_new(const int32_t* prefix_pages, int32_t prefix_len, int32_t num_branches,
                           const int32_t* suffix_lens, int32_t page_size,
                           const int32_t* free_pages, int32_t n_free, const int32_t* used_in,
                           int32_t* used_out, int32_t* page_table, int32_t max_pages_per_branch,
                           int32_t* cow_pairs, fanout_stream_t stream) {
    return fork_device(prefix_pages, prefix_len, num_branches, suffix_lens, page_size, free_pages,
                       n_free, used_in, used_out, page_table, max_pages_per_branch, cow_pairs, 1,
                       stream);
}

int fanout_extend_device(int32_t* page_table, int32_t num_branches, int32_t max_pages_per_branch,
                         int32_t prefix_len, const int32_t* suffix_lens, const int32_t* add_lens,
                         int32_t page_size, const int32_t* free_pages, int32_t n_free,
                         const int32_t* used_in, int32_t* used_out, int64_t* slots,
                         int64_t n_slots, fanout_stream_t stream) {
    if (num_branches < 0 || max_pages_per_branch < 0 || prefix_len < 0 || page_size <= 0 ||
        n_free < 0 || n_slots < 0 || n_slots > 0x7fffffff)
        return FANOUT_EINVAL;
    if (num_branches > kMaxTableBranches) return FANOUT_EUNSUPPORTED;
    if (num_branches > 0 &&
        (!suffix_lens || !add_lens || (max_pages_per_branch > 0 && !page_table)))
        return FANOUT_EINVAL;
    if (n_free > 0 && !free_pages) return FANOUT_EINVAL;
    if (n_slots > 0 && !slots) return FANOUT_EINVAL;
    if (used_out && used_out == used_in) return FANOUT_EINVAL;
    for (const void* ptr : {static_cast<const void*>(page_table),
                            static_cast<const void*>(suffix_lens),
                            static_cast<const void*>(add_lens),
                            static_cast<const void*>(free_pages),
                            static_cast<const void*>(used_in),
                            static_cast<const void*>(used_out)})
        if (!aligned(ptr, 4)) return FANOUT_EINVAL;
    if (!aligned(slots, 8)) return FANOUT_EINVAL;
    const int64_t table_bytes = 4LL * num_branches * max_pages_per_branch;
    const Array read[] = {{suffix_lens, 4LL * num_branches},
                          {add_lens, 4LL * num_branches},
                          {free_pages, 4LL * n_free},
                          {used_in, 4}};
    const Array written[] = {{page_table, table_bytes}, {slots, 8 * n_slots}, {used_out, 4}};
    if (any_overlap(read, written) || overlap(slots, 8 * n_slots, page_table, table_bytes))
        return FANOUT_EINVAL;
    TableParams p{};
    p.extend = 1;
    p.suffix_lens = suffix_lens;
    p.add_lens = add_lens;
    p.free_pages = free_pages;
    p.used_in = used_in;
    p.used_out = used_out;
    p.page_table = page_table;
    p.slots = slots;
    p.n_slots = n_slots;
    p.num_branches = num_branches;
    p.prefix_len = prefix_len;
    p.page_size = page_size;
    p.n_free = n_free;
    p.max_pages = max_pages_per_branch;
    return launch_checked_tables(p, stream);
}

int fanout_kv_append_q4(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                        void* k_pages, void* v_pages, const int64_t* slots, int32_t n_rows,
                        int32_t num_pages, int32_t H_kv, int32_t d, int32_t page_size,
                        float k_scale, float v_scale, fanout_stream_t stream) {
    const int st = check_rows(k_new, v_new, k_pages, v_pages, slots, n_rows, k_stride, v_stride,
                              num_pages, H_kv, d, page_size, k_scale, v_scale);
    if (st != FANOUT_OK || n_rows == 0) return st;
    Q4RowParams p{};
    p.k_rows = static_cast<const __nv_bfloat16*>(k_new);
    p.v_rows = static_cast<const __nv_bfloat16*>(v_new);
    p.k_pool = static_cast<uint8_t*>(k_pages);
    p.v_pool = static_cast<uint8_t*>(v_pages);
    p.slots = slots;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_slots = static_cast<int64_t>(num_pages) * page_size;
    p.n_rows = n_rows;
    p.H_kv = H_kv;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return run_rows(p, false, page_size, stream);
}

int fanout_kv_read_q4(const void* k_pages, const void* v_pages, const int64_t* slots,
                      int32_t n_rows, int32_t num_pages, int32_t H_kv, int32_t d,
                      int32_t page_size, float k_scale, float v_scale, void* k_out, void* v_out,
                      int64_t k_stride, int64_t v_stride, fanout_stream_t stream) {
    const int st = check_rows(k_out, v_out, k_pages, v_pages, slots, n_rows, k_stride, v_stride,
                              num_pages, H_kv, d, page_size, k_scale, v_scale);
    if (st != FANOUT_OK || n_rows == 0) return st;
    Q4RowParams p{};
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.v_out = static_cast<__nv_bfloat16*>(v_out);
    p.k_pool = static_cast<uint8_t*>(const_cast<void*>(k_pages));
    p.v_pool = static_cast<uint8_t*>(const_cast<void*>(v_pages));
    p.slots = slots;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_slots = static_cast<int64_t>(num_pages) * page_size;
    p.n_rows = n_rows;
    p.H_kv = H_kv;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return run_rows(p, true, page_size, stream);
}

int fanout_kv_append_q8(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                        void* k_pages, void* v_pages, const int64_t* slots, int32_t n_rows,
                        int32_t num_pages, int32_t H_kv, int32_t d, int32_t page_size,
                        float k_scale, float v_scale, fanout_stream_t stream) {
    const int st = check_rows(k_new, v_new, k_pages, v_pages, slots, n_rows, k_stride, v_stride,
                              num_pages, H_kv, d, page_size, k_scale, v_scale);
    if (st != FANOUT_OK || n_rows == 0) return st;
    Q8RowParams p{};
    p.k_rows = static_cast<const __nv_bfloat16*>(k_new);
    p.v_rows = static_cast<const __nv_bfloat16*>(v_new);
    p.k_pool = static_cast<uint8_t*>(k_pages);
    p.v_pool = static_cast<uint8_t*>(v_pages);
    p.slots = slots;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_slots = static_cast<int64_t>(num_pages) * page_size;
    p.n_rows = n_rows;
    p.H_kv = H_kv;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return run_rows_q8(p, false, page_size, stream);
}

int fanout_kv_read_q8(const void* k_pages, const void* v_pages, const int64_t* slots,
                      int32_t n_rows, int32_t num_pages, int32_t H_kv, int32_t d,
                      int32_t page_size, float k_scale, float v_scale, void* k_out, void* v_out,
                      int64_t k_stride, int64_t v_stride, fanout_stream_t stream) {
    const int st = check_rows(k_out, v_out, k_pages, v_pages, slots, n_rows, k_stride, v_stride,
                              num_pages, H_kv, d, page_size, k_scale, v_scale);
    if (st != FANOUT_OK || n_rows == 0) return st;
    Q8RowParams p{};
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.v_out = static_cast<__nv_bfloat16*>(v_out);
    p.k_pool = static_cast<uint8_t*>(const_cast<void*>(k_pages));
    p.v_pool = static_cast<uint8_t*>(const_cast<void*>(v_pages));
    p.slots = slots;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_slots = static_cast<int64_t>(num_pages) * page_size;
    p.n_rows = n_rows;
    p.H_kv = H_kv;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return run_rows_q8(p, true, page_size, stream);
}

int fanout_tree_rows(const int32_t* parents, const int32_t* page_table, int32_t num_branches,
                     int32_t max_pages_per_branch, int32_t prefix_len, const int32_t* suffix_lens,
                     const int32_t* add_lens, int32_t page_size, int64_t n_rows,
                     int32_t mask_words, int32_t window, uint32_t* masks, int32_t* positions,
                     int64_t* slots, fanout_stream_t stream) {
    return fanout_tree_rows_sinks(parents, page_table, num_branches, max_pages_per_branch, prefix_len,
                                  suffix_lens, add_lens, page_size, n_rows, mask_words, window, 0,
                                  masks, positions, slots, stream);
}

int fanout_tree_rows_sinks(const int32_t* parents, const int32_t* page_table, int32_t num_branches,
                           int32_t max_pages_per_branch, int32_t prefix_len,
                           const int32_t* suffix_lens, const int32_t* add_lens, int32_t page_size,
                           int64_t n_rows, int32_t mask_words, int32_t window, int32_t sinks,
                           uint32_t* masks, int32_t* positions, int64_t* slots,
                           fanout_stream_t stream) {
    if (num_branches < 0 || max_pages_per_branch < 0 || prefix_len < 0 || page_size <= 0 ||
        n_rows < 0 || mask_words <= 0 || window < 0 || sinks < 0 || (window == 0 && sinks > 0))
        return FANOUT_EINVAL;
    if (num_branches > kMaxTableBranches || mask_words > kMaxTreeTokens / 32 || n_rows > 0x7fffffff)
        return FANOUT_EUNSUPPORTED;
    if (n_rows == 0) return FANOUT_OK;
    const bool some = num_branches > 0;
    const Typed arrays[] = {{parents, 4, some},     {page_table, 4, some && max_pages_per_branch > 0},
                            {suffix_lens, 4, some}, {add_lens, 4, some},
                            {masks, 4, true},       {positions, 4, true},
                            {slots, 8, true}};
    if (!arrays_ok(arrays)) return FANOUT_EINVAL;
    const Array read[] = {{parents, 4 * n_rows},
                          {page_table, 4LL * num_branches * max_pages_per_branch},
                          {suffix_lens, 4LL * num_branches},
                          {add_lens, 4LL * num_branches}};
    const Array written[] = {{masks, 4 * n_rows * mask_words}, {positions, 4 * n_rows}, {slots, 8 * n_rows}};
    if (any_overlap(read, written) || any_overlap_among(written)) return FANOUT_EINVAL;
    TreeParams p{};
    p.parents = parents;
    p.page_table = page_table;
    p.suffix_lens = suffix_lens;
    p.lens = add_lens;
    p.masks = masks;
    p.positions = positions;
    p.slots = slots;
    p.num_branches = num_branches;
    p.R = static_cast<int32_t>(n_rows);
    p.words = mask_words;
    p.window = window;
    p.sinks = sinks;
    p.prefix_len = prefix_len;
    p.page_size = page_size;
    p.max_pages = max_pages_per_branch;
    const cudaError_t ce = err_word_ptr(&p.err);
    if (ce != cudaSuccess) return status_from_cuda(ce);
    return status_from_cuda(launch_tree_rows(p, reinterpret_cast<cudaStream_t>(stream)));
}

int fanout_tree_accept(const int32_t* parents, const int64_t* draft_tokens,
                       const int64_t* target_tokens, const int64_t* first_tokens,
                       const int32_t* add_lens, int32_t num_branches, int64_t n_rows,
                       int32_t* path, int32_t* counts, int64_t* next_tokens,
                       fanout_stream_t stream) {
    if (num_branches < 0 || n_rows < 0) return FANOUT_EINVAL;
    if (num_branches > kMaxTableBranches || n_rows > 0x7fffffff) return FANOUT_EUNSUPPORTED;
    if (n_rows == 0 && num_branches == 0) return FANOUT_OK;
    const bool some = num_branches > 0, rows = n_rows > 0;
    const Typed arrays[] = {{parents, 4, rows},       {draft_tokens, 8, rows},
                            {target_tokens, 8, rows}, {first_tokens, 8, some},
                            {add_lens, 4, some},      {path, 4, rows},
                            {counts, 4, some},        {next_tokens, 8, some}};
    if (!arrays_ok(arrays)) return FANOUT_EINVAL;
    const Array read[] = {{parents, 4 * n_rows},
                          {draft_tokens, 8 * n_rows},
                          {target_tokens, 8 * n_rows},
                          {first_tokens, 8LL * num_branches},
                          {add_lens, 4LL * num_branches}};
    const Array written[] = {{path, 4 * n_rows}, {counts, 4LL * num_branches}, {next_tokens, 8LL * num_branches}};
    if (any_overlap(read, written) || any_overlap_among(written)) return FANOUT_EINVAL;
    TreeParams p{};
    p.parents = parents;
    p.draft = draft_tokens;
    p.target = target_tokens;
    p.first = first_tokens;
    p.lens = add_lens;
    p.path = path;
    p.counts = counts;
    p.next = next_tokens;
    p.num_branches = num_branches;
    p.R = static_cast<int32_t>(n_rows);
    const cudaError_t ce = err_word_ptr(&p.err);
    if (ce != cudaSuccess) return status_from_cuda(ce);
    return status_from_cuda(launch_tree_accept(p, reinterpret_cast<cudaStream_t>(stream)));
}

int fanout_kv_keep(void* k_pages, void* v_pages, int32_t kv_type, const int32_t* page_table,
                   int32_t num_branches, int32_t max_pages_per_branch, int32_t prefix_len,
                   const int32_t* suffix_lens, const int32_t* add_lens, const int32_t* path,
                   const int32_t* counts, int64_t n_rows, int32_t num_pages, int32_t H_kv,
                   int32_t d, int32_t page_size, fanout_stream_t stream) {
    if (kv_type != FANOUT_KV_BF16 && kv_type != FANOUT_KV_Q4 && kv_type != FANOUT_KV_Q8)
        return FANOUT_EINVAL;
    if (num_branches < 0 || max_pages_per_branch < 0 || prefix_len < 0 || n_rows < 0 ||
        num_pages <= 0 || H_kv <= 0 || d <= 0 || page_size <= 0)
        return FANOUT_EINVAL;
    if (d != kHD) return FANOUT_EUNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return FANOUT_EUNSUPPORTED;
    if (num_branches > kMaxTableBranches || n_rows > 0x7fffffff ||
        static_cast<int64_t>(num_branches) * H_kv > 0x7fffffff)
        return FANOUT_EUNSUPPORTED;
    if (n_rows == 0 || num_branches == 0) return FANOUT_OK;
    const Typed arrays[] = {{k_pages, 16, true}, {v_pages, 16, true},
                            {page_table, 4, max_pages_per_branch > 0},
                            {suffix_lens, 4, true}, {add_lens, 4, true},
                            {path, 4, true}, {counts, 4, true}};
    if (!arrays_ok(arrays)) return FANOUT_EINVAL;
    const double row = kv_type == FANOUT_KV_BF16 ? 2 * kHD : kv_type == FANOUT_KV_Q4 ? kQ4RowBytes : kHD;
    const int64_t pool = bytes_of(row * num_pages * H_kv * page_size);
    const Array read[] = {{page_table, 4LL * num_branches * max_pages_per_branch},
                          {suffix_lens, 4LL * num_branches},
                          {add_lens, 4LL * num_branches},
                          {path, 4 * n_rows},
                          {counts, 4LL * num_branches}};
    const Array written[] = {{k_pages, pool}, {v_pages, pool}};
    if (any_overlap(read, written) || any_overlap_among(written)) return FANOUT_EINVAL;
    TreeParams p{};
    p.page_table = page_table;
    p.suffix_lens = suffix_lens;
    p.lens = add_lens;
    p.path = const_cast<int32_t*>(path);
    p.counts = const_cast<int32_t*>(counts);
    p.k_pool = static_cast<uint8_t*>(k_pages);
    p.v_pool = static_cast<uint8_t*>(v_pages);
    p.pool = static_cast<Pool>(kv_type);
    p.num_branches = num_branches;
    p.R = static_cast<int32_t>(n_rows);
    p.prefix_len = prefix_len;
    p.page_size = page_size;
    p.max_pages = max_pages_per_branch;
    p.num_pages = num_pages;
    p.H_kv = H_kv;
    const cudaError_t ce = err_word_ptr(&p.err);
    if (ce != cudaSuccess) return status_from_cuda(ce);
    return status_from_cuda(launch_kv_keep(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// tree.cu -- what a step with drafted tokens does around its attention, on the device: the
// masks, positions and cache slots of the drafted rows, the path that the model's tokens
// follow through a tree, and the accepted rows moved together in the cache.
//
// Branch b drafted T_b tokens; token t has parent[t] < t (-1: none) and sits in the cache
// at key n_b + t, n_b = prefix_len + suffix_lens[b].
//   depth(t) = 0 without a parent, depth(parent[t]) + 1 else; position = n_b + depth(t);
//   bit u of t's mask: u is t or an ancestor of t less than `window` levels above it, or one
//   at a position below `sinks`;
//   accepted: from no node on, the child of lowest index that was drafted as the token
//   picked at its parent (first[b] at none), until there is none;
//   kept: row n_b + i := row n_b + path[i]. A path ascends, so path[i] >= i, and a row is
//   never overwritten before it has been read, whatever runs of moves are read at once.
//
// Rows are grouped by branch, so every CTA adds up the lengths of all branches itself (as
// tables.cu does): no CTA waits for another and all come to the same verdict on the
// lengths. All three are a launch and a chain of dependent reads (lengths, parents, steps
// up or down a tree in shared memory, table, rows), which is what bounds them: back to back
// in a graph 2.7, 2.6 and 3.2 us for 8 branches of 32 drafted tokens (8 KV heads). Masks are
// found a word of 32 tokens at a time, so that a token steps from word to word and not from
// parent to parent; of every token's children the accepted one is found at once, so that the
// path is a step a token in shared memory. (A chain of 64 tokens: 3.3 and 4.1 us, not 10 and
// 15; of 1024: 28 and 33, not 660 and 200.) A call costs the host 5 to 11 us from Python, so
// a step's calls issued one by one are bound by the host.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "launch_after.cuh"
#include "rows.h"

namespace fanout {
namespace {

constexpr int kThreads = 128;
constexpr int kErrInval = 1;  // FANOUT_EINVAL
constexpr int64_t kMaxTokens = 0x7fffffff;

struct Sums {
    int64_t part[2][kThreads / 32];
    int32_t bad;
};

// Rows before branch b_first, and all of them; false when some length is not valid.
// place: the branches' places in the cache are checked as well.
__device__ bool sum_rows(const TreeParams& p, Sums& sm, int32_t b_first, bool place, int64_t& before,
                         int64_t& all) {
    if (threadIdx.x == 0) sm.bad = 0;
    __syncthreads();
    before = all = 0;
    bool ok = true;
    for (int b = threadIdx.x; b < p.num_branches; b += kThreads) {
        const int32_t n = __ldcg(p.lens + b);
        ok &= n >= 0 && n <= kMaxTreeTokens && (p.words == 0 || n <= 32 * p.words);
        if (place) {
            const int32_t s = __ldcg(p.suffix_lens + b);
            const int64_t end = static_cast<int64_t>(p.prefix_len) + s + n;
            ok &= s >= 0 && end <= kMaxTokens &&
                  end <= static_cast<int64_t>(p.max_pages) * p.page_size;
        }
        all += n;
        if (b < b_first) before += n;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, d);
        before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    if ((threadIdx.x & 31) == 0) {
        sm.part[0][threadIdx.x >> 5] = all;
        sm.part[1][threadIdx.x >> 5] = before;
    }
    if (!ok) sm.bad = 1;
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        all += sm.part[0][w];
        before += sm.part[1][w];
    }
    return !sm.bad && all <= p.R;
}

// A CTA's run of consecutive items.
__device__ __forceinline__ void run_of(int32_t items, int32_t& i0, int32_t& i1) {
    const int32_t per = (items + gridDim.x - 1) / gridDim.x;
    i0 = min(items, static_cast<int32_t>(blockIdx.x) * per);
    i1 = min(items, i0 + per);
}

// ------------------------------------------------------------ masks, positions, slots
__global__ void __launch_bounds__(kThreads) tree_rows_kernel(const TreeParams p) {
    after_previous();
    __shared__ Sums sums;
    // of every token: its ancestors (and itself) in its word of 32 tokens, and the first
    // ancestor in a word below (-1: none)
    __shared__ uint32_t family[kMaxTreeTokens];
    __shared__ int32_t below[kMaxTreeTokens];
    int32_t b0, b1;
    run_of(p.num_branches, b0, b1);
    int64_t row, all;
    const bool ok = sum_rows(p, sums, b0, true, row, all);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.err, 0, kErrInval);
    // rows behind the last token, or all of a refused call: nothing may be written or
    // seen through them
    for (int64_t r = (ok ? all : 0) + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; r < p.R;
         r += static_cast<int64_t>(gridDim.x) * kThreads) {
        for (int w = 0; w < p.words; ++w) p.masks[r * p.words + w] = 0u;
        p.positions[r] = 0;
        p.slots[r] = -1;
    }
    if (!ok) return;
    for (int32_t b = b0; b < b1; ++b) {
        const int32_t T = __ldcg(p.lens + b), n = p.prefix_len + __ldcg(p.suffix_lens + b);
        __syncthreads();
        for (int t = threadIdx.x; (t & ~31) < T; t += kThreads) {  // a warp a word
            int32_t up = t < T ? __ldcg(p.parents + row + t) : -1;
            if (up < -1 || up >= t) {  // reported, and taken as none
                atomicCAS(p.err, 0, kErrInval);
                up = -1;
            }
            // A run of ancestors in the word, from the token up, is doubled five times:
            // its tokens, the next one in the word (-1: none) or else the one below.
            uint32_t run = 1u << (t & 31);
            int32_t next = up >= (t & ~31) ? up & 31 : -1, out = up;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int from = max(next, 0);
                const uint32_t r = __shfl_sync(0xffffffffu, run, from);
                const int32_t o = __shfl_sync(0xffffffffu, out, from);
                const int32_t x = __shfl_sync(0xffffffffu, next, from);
                if (next >= 0) {
                    run |= r;
                    out = o;
                    next = x;
                }
            }
            family[t] = run;
            below[t] = out;
        }
        __syncthreads();
        for (int t = threadIdx.x; t < T; t += kThreads) {
            uint32_t* mask = p.masks + (row + t) * p.words;
            for (int w = (t >> 5) + 1; w < p.words; ++w) mask[w] = 0u;
            // of the tokens from t up, those from the `far`-th on are among the first keys
            int far = 1 << 30;
            if (p.window > 0 && p.sinks > n) {
                far = n - p.sinks;
                for (int u = t; u >= 0; u = below[u]) far += __popc(family[u]);
            }
            int depth = 0, word = t >> 5;
            for (int u = t; u >= 0; u = below[u]) {  // ancestors come in descending order
                uint32_t bits = family[u];
                const int count = __popc(bits), left = p.window - depth;
                const int low = depth + count - max(depth, far);
                if (p.window > 0 && count > left && count > low) {
                    // the `left` nearest: the highest; the `low` nearest the root: the lowest
                    uint32_t keep = left <= 0 ? 0u : ~0u << __fns(bits, 0, count - left + 1);
                    if (low > 0) keep |= (1u << __fns(bits, 0, low + 1)) - 1u;
                    bits &= keep;
                }
                depth += count;
                for (; word > (u >> 5); --word) mask[word] = 0u;
                mask[word--] = bits;
            }
            for (; word >= 0; --word) mask[word] = 0u;
            p.positions[row + t] = n + depth - 1;
            const int32_t key = n + t;
            const int32_t i = static_cast<int32_t>(static_cast<uint32_t>(key) /
                                                   static_cast<uint32_t>(p.page_size));
            const int32_t page = __ldcg(p.page_table + static_cast<int64_t>(b) * p.max_pages + i);
            if (page < 0) atomicCAS(p.err, 0, kErrInval);
            p.slots[row + t] =
                page < 0 ? -1 : static_cast<int64_t>(page) * p.page_size + (key - i * p.page_size);
        }
        row += T;
    }
}

// ------------------------------------------------------------ the accepted path
__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const TreeParams p) {
    after_previous();
    __shared__ Sums sums;
    __shared__ int64_t target[kMaxTreeTokens];
    __shared__ int32_t child[kMaxTreeTokens + 1];  // behind each token (0: behind none) the accepted one
    __shared__ int32_t list[kMaxTreeTokens];
    __shared__ int32_t taken;
    int32_t b0, b1;
    run_of(p.num_branches, b0, b1);
    int64_t row, all;
    const bool ok = sum_rows(p, sums, b0, false, row, all);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.err, 0, kErrInval);
    for (int64_t r = (ok ? all : 0) + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; r < p.R;
         r += static_cast<int64_t>(gridDim.x) * kThreads)
        p.path[r] = -1;
    for (int32_t b = b0; b < b1; ++b) {
        if (!ok) {
            if (threadIdx.x == 0) {
                p.counts[b] = 0;
                p.next[b] = -1;
            }
            continue;
        }
        const int32_t T = __ldcg(p.lens + b);
        const int64_t first = __ldcg(p.first + b);
        __syncthreads();
        for (int t = threadIdx.x; t <= T; t += kThreads) {
            child[t] = kMaxTreeTokens;
            if (t < T) target[t] = __ldcg(p.target + row + t);
        }
        __syncthreads();
        for (int t = threadIdx.x; t < T; t += kThreads) {
            int32_t up = __ldcg(p.parents + row + t);
            if (up < -1 || up >= t) {  // reported, and taken as none
                atomicCAS(p.err, 0, kErrInval);
                up = -1;
            }
            if (__ldcg(p.draft + row + t) == (up < 0 ? first : target[up])) atomicMin(child + up + 1, t);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int32_t at = -1, count = 0;
            for (int32_t t = child[0]; t < kMaxTreeTokens; t = child[t + 1]) {
                list[count++] = t;
                at = t;
            }
            p.counts[b] = count;
            p.next[b] = at < 0 ? first : target[at];
            taken = count;
        }
        __syncthreads();
        for (int t = threadIdx.x; t < T; t += kThreads) p.path[row + t] = t < taken ? list[t] : -1;
        row += T;
    }
}

// ------------------------------------------------------------ the kept rows
// A row of a (page, KV head) block in pieces of 16 or 8 bytes, lane `l` of 16 each.
template <Pool F>
struct RowOf {
    using Piece = uint2;
    static constexpr int kLanes = F == Pool::q4 ? 9 : 16;
    static __device__ __forceinline__ int64_t at(int64_t block, int32_t slot, int32_t ps, int l) {
        if (F == Pool::q8) return (block * ps + slot) * kHD + l * 8;
        const int64_t base = block * ps * kQ4RowBytes;  // 4 bits: codes, then scales
        return l < 8 ? base + slot * 64 + l * 8 : base + ps * 64 + slot * 8;
    }
};
template <>
struct RowOf<Pool::bf16> {
    using Piece = uint4;
    static constexpr int kLanes = 16;
    static __device__ __forceinline__ int64_t at(int64_t block, int32_t slot, int32_t ps, int l) {
        return (block * ps + slot) * (2 * kHD) + l * 16;
    }
};

constexpr int kHeadsPerItem = kThreads / 32;  // a warp a KV head
constexpr int kMoves = 4;                     // rows read before any is written

template <Pool F>
__global__ void __launch_bounds__(kThreads) kv_keep_kernel(const TreeParams p) {
    after_previous();
    using Row = RowOf<F>;
    __shared__ Sums sums;
    const int32_t groups = (p.H_kv + kHeadsPerItem - 1) / kHeadsPerItem;
    int32_t i0, i1;
    run_of(p.num_branches * groups, i0, i1);
    int64_t row, all;
    const bool ok = sum_rows(p, sums, i0 / groups, true, row, all);
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(p.err, 0, kErrInval);
        return;
    }
    const int lane = threadIdx.x & 31, l = lane & 15;
    uint8_t* const pool = lane < 16 ? p.k_pool : p.v_pool;
    int32_t last = i0 / groups;
    for (int32_t item = i0; item < i1; ++item) {
        const int32_t b = item / groups;
        if (b != last) row += __ldcg(p.lens + last);
        last = b;
        const int32_t h = (item - b * groups) * kHeadsPerItem + (threadIdx.x >> 5);
        if (h >= p.H_kv) continue;
        const int32_t T = __ldcg(p.lens + b), count = __ldcg(p.counts + b);
        const int32_t n = p.prefix_len + __ldcg(p.suffix_lens + b);
        const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
        // a path that does not ascend inside the branch moves nothing
        bool good = count >= 0 && count <= T, ascends = true;
        for (int i = lane; i < (good ? count : 0); i += 32) {
            const int32_t from = __ldcg(p.path + row + i);
            const int32_t before = i > 0 ? __ldcg(p.path + row + i - 1) : -1;
            ascends = ascends && from > before && from < T;
        }
        good = good && ascends;
        if (!__all_sync(0xffffffffu, good)) {
            if (lane == 0) atomicCAS(p.err, 0, kErrInval);
            continue;
        }
        for (int32_t c0 = 0; c0 < count; c0 += 32) {
            // lane i: the places of move c0 + i
            int32_t from = 0, slot_s = 0, slot_d = 0, page_s = -1, page_d = -1;
            const int32_t to = c0 + lane;
            if (to < count) {
                from = __ldcg(p.path + row + to);
                auto place = [&](int32_t key, int32_t& page, int32_t& slot) {
                    const int32_t i = static_cast<int32_t>(static_cast<uint32_t>(key) /
                                                           static_cast<uint32_t>(p.page_size));
                    page = __ldcg(table + i);
                    slot = key - i * p.page_size;
                    if (page < 0 || page >= p.num_pages) {
                        atomicCAS(p.err, 0, kErrInval);
                        page = -1;
                    }
                };
                if (from != to) {
                    place(n + from, page_s, slot_s);
                    place(n + to, page_d, slot_d);
                }
            }
            if (!__any_sync(0xffffffffu, page_s >= 0)) continue;  // all in place
            const int32_t moves = min(32, count - c0);
            for (int32_t m = 0; m < moves; m += kMoves) {
                typename Row::Piece v[kMoves];
                int64_t dst[kMoves];
                bool move[kMoves];
#pragma unroll
                for (int k = 0; k < kMoves; ++k) {  // (lanes past the last move hold no pages)
                    const int32_t ps = __shfl_sync(0xffffffffu, page_s, (m + k) & 31);
                    const int32_t pd = __shfl_sync(0xffffffffu, page_d, (m + k) & 31);
                    const int32_t ss = __shfl_sync(0xffffffffu, slot_s, (m + k) & 31);
                    const int32_t sd = __shfl_sync(0xffffffffu, slot_d, (m + k) & 31);
                    move[k] = ps >= 0 && pd >= 0 && l < Row::kLanes;
                    dst[k] = Row::at(static_cast<int64_t>(pd) * p.H_kv + h, sd, p.page_size, l);
                    if (move[k])
                        v[k] = *reinterpret_cast<const typename Row::Piece*>(
                            pool + Row::at(static_cast<int64_t>(ps) * p.H_kv + h, ss, p.page_size, l));
                }
#pragma unroll
                for (int k = 0; k < kMoves; ++k)
                    if (move[k]) *reinterpret_cast<typename Row::Piece*>(pool + dst[k]) = v[k];
            }
        }
    }
}

int grid_for(int64_t items) {
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(items, 8LL * sms)));
}

}  // namespace

cudaError_t launch_tree_rows(const TreeParams& p, cudaStream_t stream) {
    return launch_after(tree_rows_kernel, grid_for(p.num_branches), kThreads, 0, stream, p);
}

cudaError_t launch_tree_accept(const TreeParams& p, cudaStream_t stream) {
    return launch_after(tree_accept_kernel, grid_for(p.num_branches), kThreads, 0, stream, p);
}

cudaError_t launch_kv_keep(const TreeParams& p, cudaStream_t stream) {
    const int groups = (p.H_kv + kHeadsPerItem - 1) / kHeadsPerItem;
    const int grid = grid_for(static_cast<int64_t>(p.num_branches) * groups);
    auto* kernel = p.pool == Pool::bf16 ? kv_keep_kernel<Pool::bf16>
                   : p.pool == Pool::q4 ? kv_keep_kernel<Pool::q4>
                                        : kv_keep_kernel<Pool::q8>;
    return launch_after(kernel, grid, kThreads, 0, stream, p);
}

}  // namespace fanout

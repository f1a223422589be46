// tables.cu -- branch page tables and slot maps built on the device.
//
// The device counterparts of fanout_fork / fanout_fork_cow and fanout_extend
// ("AHBM Agentic Runtime Architecture" section 3.1: a branch's table is
// [shared prefix pages] + [private pages]): the lengths, the free list and the
// number of its entries already handed out are device memory, so a step needs
// no host round trip and the calls can be captured in a graph.
//
// Mathematics: with P shared and S_b private tokens, pages of ps tokens and
// A_b tokens to add, branch b takes n_b pages (fork: ceil((P + S_b) / ps) minus
// the whole prefix pages; extend: ceil((P + S_b + A_b) / ps) - ceil((P + S_b) /
// ps)); its first one is entry used + sum_{i < b} n_i of the free list, and its
// first new row is sum_{i < b} A_i.
//
// Every CTA computes that exclusive scan over all branches for itself (two
// loads and a few shuffles per branch, from L2), so no CTA waits for another
// and all of them come to the same verdict on the lengths: a negative length, a
// row too narrow, a list too short or too few slots leaves the table untouched (or
// fills a new one with -1).
// Measured: extend of 8 branches 8.2 us (a launch and three dependent reads), fork of
// 1024 branches over 4096 prefix pages 12.3 us for 18.4 MB (2.7 us at the copy rate:
// the scan in front of the copies and one wave of blocks are the rest).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fanout_internal.h"

namespace fanout {
namespace {

constexpr int kThreads = 256;
constexpr int kErrInval = 1;  // FANOUT_EINVAL
constexpr int64_t kMaxTokens = 0x7fffffff;

struct Scan {
    int32_t page_off[kMaxTableBranches + 1];  // pages taken before branch b
    int32_t row_off[kMaxTableBranches + 1];   // new rows before branch b (extend)
    int64_t part[2][kThreads / 32];
    int32_t bad;
};

// Exclusive block scan of one value per thread; every thread gets the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += t;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    return before + incl - v;
}

// Pages of up to kMaxTokens tokens, in 32 bits: with 64-bit divisions the scan over
// 1024 branches took three quarters of a fork's time.
__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t ps) {
    return static_cast<int32_t>(
        (static_cast<uint32_t>(tokens) + static_cast<uint32_t>(ps) - 1u) / static_cast<uint32_t>(ps));
}

// Pages that forked branch b needs (at least the prefix's n_prefix); false when its
// lengths are not valid. Tokens are counted in 64 bits.
__device__ __forceinline__ bool fork_pages(const TableParams& p, int32_t b, int32_t n_prefix,
                                           int32_t& need) {
    const int32_t S = __ldg(p.suffix_lens + b);
    const int64_t end = static_cast<int64_t>(p.prefix_len) + S;
    need = n_prefix;
    if (S < 0 || end > kMaxTokens) return false;
    need = max(need, pages_of(end, p.page_size));
    return need <= p.max_pages;
}

// Pages that branch b holds and needs after its growth, and its new rows.
__device__ __forceinline__ bool branch_pages(const TableParams& p, int32_t b, int32_t& held,
                                             int32_t& need, int32_t& rows) {
    const int32_t S = __ldg(p.suffix_lens + b), A = __ldg(p.add_lens + b);
    const int64_t end = static_cast<int64_t>(p.prefix_len) + S + A;
    if (S < 0 || A < 0 || end > kMaxTokens) {
        held = need = rows = 0;
        return false;
    }
    rows = A;
    held = pages_of(end - A, p.page_size);
    need = pages_of(end, p.page_size);
    return need <= p.max_pages;
}

// The scan over all branches into sm, for an extension (each thread a contiguous run
// of them).
// Returns whether the call is valid; `used` is the free list's first entry.
__device__ bool scan_branches(const TableParams& p, Scan& sm, int32_t& used, int64_t& pages,
                              int64_t& rows) {
    if (threadIdx.x == 0) sm.bad = 0;
    __syncthreads();
    used = p.used_in ? *p.used_in : 0;
    const int per = (p.num_branches + kThreads - 1) / kThreads;
    const int b0 = min(p.num_branches, static_cast<int>(threadIdx.x) * per);
    const int b1 = min(p.num_branches, b0 + per);
    int64_t np = 0, nr = 0;
    bool ok = true;
    for (int b = b0; b < b1; ++b) {
        int32_t held, need, r;
        ok &= branch_pages(p, b, held, need, r);
        np += need - held;
        nr += r;
    }
    int64_t pos = block_scan(np, sm.part[0], pages);
    int64_t row = block_scan(nr, sm.part[1], rows);
    if (!ok) sm.bad = 1;
    __syncthreads();
    if (sm.bad || used < 0 || (pages > 0 && used + pages > p.n_free) ||
        (p.slots && rows > p.n_slots) || rows > kMaxTokens)
        return false;
    for (int b = b0; b < b1; ++b) {  // lengths again: cheaper than keeping them
        int32_t held, need, r;
        branch_pages(p, b, held, need, r);
        sm.page_off[b] = static_cast<int32_t>(pos);
        sm.row_off[b] = static_cast<int32_t>(row);
        pos += need - held;
        row += r;
    }
    if (threadIdx.x == 0) {
        sm.page_off[p.num_branches] = static_cast<int32_t>(pages);
        sm.row_off[p.num_branches] = static_cast<int32_t>(rows);
    }
    __syncthreads();
    return true;
}

// Largest b < n with off[b] <= v (the branch whose run holds entry v).
__device__ __forceinline__ int32_t branch_of(const int32_t* off, int32_t n, int32_t v) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (off[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A CTA takes a run of consecutive (branch, kRun table entries) items. Of the scan
// it needs the pages taken before its first branch and the total (for the verdict),
// so it only adds up the lengths; the later branches' starts follow one by one.
// A row's entries come from the prefix list, the branch's run of the free list, -1.
constexpr int kQuads = 2;  // runs of 4 entries a thread takes of an item
constexpr int kRun = 4 * kQuads * kThreads;

__global__ void __launch_bounds__(kThreads) fork_kernel(const TableParams p) {
    __shared__ int64_t part[2][kThreads / 32];
    __shared__ int32_t bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    const int32_t used = p.used_in ? *p.used_in : 0;
    const int32_t n_full = p.prefix_len / p.page_size;
    const bool partial = p.prefix_len % p.page_size != 0;
    const int32_t n_prefix = n_full + (partial ? 1 : 0);
    const int32_t runs = max(1, (p.max_pages + kRun - 1) / kRun);
    const int32_t items = p.num_branches * runs;  // <= 2^12 * 2^13 (host check)
    const int32_t per = (items + gridDim.x - 1) / gridDim.x;
    const int32_t it0 = min(items, static_cast<int32_t>(blockIdx.x) * per);
    const int32_t it1 = min(items, it0 + per);
    int32_t b = it0 / runs, run = it0 - b * runs;
    int64_t mine = 0, all = 0;
    bool ok = true;
    for (int i = threadIdx.x; i < p.num_branches; i += kThreads) {
        int32_t need;
        ok &= fork_pages(p, i, n_prefix, need);
        all += need - n_full;
        if (i < b) mine += need - n_full;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, d);
        mine += __shfl_xor_sync(0xffffffffu, mine, d);
    }
    if ((threadIdx.x & 31) == 0) {
        part[0][threadIdx.x >> 5] = all;
        part[1][threadIdx.x >> 5] = mine;
    }
    if (!ok) bad = 1;
    __syncthreads();
    all = mine = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        all += part[0][w];
        mine += part[1][w];
    }
    ok = !bad && used >= 0 && (all == 0 || used + all <= p.n_free);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (p.used_out) *p.used_out = used + (ok ? static_cast<int32_t>(all) : 0);
        if (!ok) atomicCAS(p.err, 0, kErrInval);
    }
    if (!ok) {
        // No page may be copied or read by what follows: the pairs, and the entries of a
        // table that held nothing before, become -1.
        for (int32_t it = it0; it < it1; ++it) {
            if (run == 0 && threadIdx.x == 0 && partial && p.cow_pairs) {
                p.cow_pairs[2 * b] = -1;
                p.cow_pairs[2 * b + 1] = -1;
            }
            int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
            const int32_t end = p.clear ? min(p.max_pages, (run + 1) * kRun) : 0;
            for (int32_t i = run * kRun + static_cast<int32_t>(threadIdx.x); i < end; i += kThreads)
                row[i] = -1;
            if (++run == runs) {
                run = 0;
                ++b;
            }
        }
        return;
    }
    const int32_t* list = p.free_pages + used + mine - n_full;  // of branch b, by table entry
    // 16-byte copies where every row and the prefix list start on 16 bytes
    const bool quads = p.max_pages % 4 == 0 &&
                       ((reinterpret_cast<uintptr_t>(p.page_table) |
                         reinterpret_cast<uintptr_t>(p.prefix_pages)) & 15u) == 0;
    for (int32_t it = it0; it < it1; ++it) {
        int32_t need;
        fork_pages(p, b, n_prefix, need);
        int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
        int4 v[kQuads];
#pragma unroll
        for (int u = 0; u < kQuads; ++u) {
            const int32_t i = run * kRun + 4 * (u * kThreads + static_cast<int>(threadIdx.x));
            auto entry = [&](int32_t e) {
                return e < n_full ? __ldg(p.prefix_pages + e) : e < need ? __ldg(list + e) : -1;
            };
            if (i + 3 < n_full && quads) v[u] = __ldg(reinterpret_cast<const int4*>(p.prefix_pages + i));
            else if (i < p.max_pages) v[u] = make_int4(entry(i), entry(i + 1), entry(i + 2), entry(i + 3));
        }
#pragma unroll
        for (int u = 0; u < kQuads; ++u) {
            const int32_t i = run * kRun + 4 * (u * kThreads + static_cast<int>(threadIdx.x));
            if (i >= p.max_pages) continue;
            if (quads) {
                *reinterpret_cast<int4*>(row + i) = v[u];
            } else {
                row[i] = v[u].x;
                if (i + 1 < p.max_pages) row[i + 1] = v[u].y;
                if (i + 2 < p.max_pages) row[i + 2] = v[u].z;
                if (i + 3 < p.max_pages) row[i + 3] = v[u].w;
            }
        }
        if (partial && p.cow_pairs && run == 0 && threadIdx.x == 0) {
            p.cow_pairs[2 * b] = p.prefix_pages[n_full];
            p.cow_pairs[2 * b + 1] = list[n_full];
        }
        if (++run == runs) {
            run = 0;
            ++b;
            list += need - n_full;
        }
    }
}

__global__ void __launch_bounds__(kThreads) extend_kernel(const TableParams p) {
    __shared__ Scan sm;
    int32_t used;
    int64_t pages, rows;
    const bool ok = scan_branches(p, sm, used, pages, rows);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (p.used_out) *p.used_out = used + (ok ? static_cast<int32_t>(pages) : 0);
        if (!ok) atomicCAS(p.err, 0, kErrInval);
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (!ok) {  // no row of a refused call may be written by what follows
        if (p.slots)
            for (int64_t r = t0; r < p.n_slots; r += stride) p.slots[r] = -1;
        return;
    }
    for (int64_t e = t0; e < pages; e += stride) {
        const int32_t b = branch_of(sm.page_off, p.num_branches, static_cast<int32_t>(e));
        const int32_t held = pages_of(static_cast<int64_t>(p.prefix_len) + p.suffix_lens[b],
                                      p.page_size);
        p.page_table[static_cast<int64_t>(b) * p.max_pages + held +
                     (static_cast<int32_t>(e) - sm.page_off[b])] = p.free_pages[used + e];
    }
    if (!p.slots) return;
    for (int64_t r = t0; r < p.n_slots; r += stride) {
        int64_t slot = -1;
        if (r < rows) {
            const int32_t b = branch_of(sm.row_off, p.num_branches, static_cast<int32_t>(r));
            const int32_t before = p.prefix_len + p.suffix_lens[b];  // <= kMaxTokens (scan)
            const int32_t pos = before + (static_cast<int32_t>(r) - sm.row_off[b]);
            const int32_t held = pages_of(before, p.page_size);
            const int32_t i = static_cast<int32_t>(static_cast<uint32_t>(pos) /
                                                   static_cast<uint32_t>(p.page_size));
            // a page taken by this call comes from the list: the table entry may
            // be another CTA's store
            const int32_t page = i >= held
                                     ? p.free_pages[used + sm.page_off[b] + (i - held)]
                                     : p.page_table[static_cast<int64_t>(b) * p.max_pages + i];
            if (page >= 0) slot = static_cast<int64_t>(page) * p.page_size + (pos - i * p.page_size);
            else atomicCAS(p.err, 0, kErrInval);
        }
        p.slots[r] = slot;
    }
}

}  // namespace

cudaError_t launch_tables(const TableParams& p, cudaStream_t stream) {
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (p.extend) {
        const int64_t work = std::max<int64_t>(p.slots ? p.n_slots : 0, p.num_branches);
        const int64_t blocks = (work + 4 * kThreads - 1) / (4 * kThreads);
        const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, 2 * sms)));
        extend_kernel<<<grid, kThreads, 0, stream>>>(p);
    } else {
        const int64_t items =
            static_cast<int64_t>(p.num_branches) * std::max(1, (p.max_pages + kRun - 1) / kRun);
        const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(items, 4 * sms)));
        fork_kernel<<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace fanout

// attn_rows.cuh -- fan-out attention of row plans, for sm_103a: over bf16 pools with a
// sliding window and first keys that stay visible, over pools held in 4 or 8 bits (with or
// without a window), and for trees of drafted tokens over any of them. Instances:
// attn_rows.cu, attn_rows_q8.cu, attn_tree.cu.
//
// Units, tiles and the online softmax are those of attn_fwd.cu (128 query rows x
// 128 keys, base 2, the reference maximum m raised only when a row's maximum passes
// it by 2^8). A row plan gives every token's position in a table, so that rows of
// different branches share a unit whatever their windows; a unit may sweep its first
// keys as tiles in front of its own range; its range may begin inside a page.
//
// GB300 mapping, one persistent CTA per SM:
//   warp 0      producer. bf16 pools: TMA boxes, a page of a KV head each, into a
//               ring of 32 KB tiles. 4-bit pools: page blocks by cp.async.bulk into
//               a ring of raw tiles (9 KB: 128 rows of 72 bytes). 8-bit pools: TMA boxes
//               of 128-byte rows, K into the ring that the products read, V into one of
//               raw tiles. Q by TMA as soon as its buffer is free. Page ids are checked
//               before they are read through;
//   warp 1      TMEM owner;
//   warp 3      tcgen05 issuer: the whole warp runs the issue loop, so that its
//               addresses stay warp-uniform, and one elected lane issues. (An issuer
//               for each group lets the groups' softmaxes coincide: a bf16 prefill of
//               2048 tokens took 1755 us, not 1243.);
//   warps 4-11  two softmax groups of 4 warps, thread = row;
//   warps 12-19 4-bit pools: turn Q tiles into f16 and widen raw tiles into the swizzled
//               16-bit ring (4 warps the K tiles, 4 Q and the V tiles): with 4 warps for
//               both, a decode step waited for them (35 us against 31 with 8). 8-bit
//               pools: warps 12-15, Q and the V tiles.
// Keys of a tile that no row of the unit sees are zeros in shared memory, whatever
// the pool holds there (K tiles of 8 bits: their scores are masked).
//
// A unit of two query tiles gives each group one of them. A unit of one query
// tile (decode) is split over the groups by keys instead: even tiles (counted over
// the CTA) go to group 0, odd ones to group 1, each with its own S, (m, l) and O in
// TMEM, and the two are joined at the unit's end (64 columns of O each), so that two
// tiles' softmaxes overlap. (All eight softmax warps on every tile, two to a row,
// was slower: their phases coincide, and the exponentials' pipe idles between.)
// TMEM: S_0 = 0, S_1 = 128, O_0 = 256, O_1 = 384 (512 columns).
//
// 4-bit pools. The rows of a cache (kv_q4.cu) are e2m1 codes with one e4m3 scale per
// 16 values; the tensor core gets f16 tiles that hold the cached values exactly: a
// code has 2 significant bits and a group scale 4, their product 6, and it lies
// between 2^-10 and 2688.
//   S = Q K^T from shared memory, Q as f16 too: its rows are scaled by the power
//   of two that brings their largest element into [2^14, 2^15) (undone in the
//   row's softmax scale), so bf16's 8 bits fit f16's 11, and only elements below
//   2^-28 of the row's largest lose bits;
//   O += P V with P from TMEM, P = 2^(x - m + 7): at most 2^15, and its rounding is
//   f16's half step of 2^-11 (bf16's, as for bf16 pools, would be 2^-8); a P below
//   2^-21 of the row's reference has a step of 2^-31 of it. The 2^7 is taken out
//   of l and of the output, where V's pool scale goes too (K's: softmax scale).
// Widening is one conversion (a byte of two codes to an f16 pair) and one packed
// product per two values: both run at 64 lanes a cycle and SM (measured), so a K
// and a V tile take 256 cycles of either pipe, under the 2048 that the four products
// of two query tiles (1024: the two of one) take on the tensor core. Bit tricks on
// bf16 tiles took 2.5 times the instructions: a prefill step was 2.1 times slower.
// The codes of a word come out as values 0 2 4 6 1 3 5 7 of its 8; K and Q keep
// that order (it is summed over), V's columns are put back when O is stored.
//
// 8-bit pools. The rows are e4m3 codes (kv_q8.cu), and a row of 128 is one line of a
// swizzled K-major tile, so K goes to the tensor core as it is cached: S is an e4m3
// product, Q in two e4m3 parts (convert_q), over twice the values at twice f16's rate. It
// accumulates in fp32 (sums of 128 products over all of e4m3's range: off by at most 2^-20
// of the sum of their magnitudes, measured). V is widened to f16 (exact) for the product with P, which
// needs f16's range: in e4m3 a P below 2^-18 of its row's largest would be lost, and
// behind a first key that takes most of a row there may be thousands of such.
//
// Drafted trees. A row sees the keys before its branch's drafted tokens as in a window,
// and of the drafted ones those of its mask, read as 32 bits for 32 columns in the one to
// nine tiles that hold them; every other tile is the same as without a tree.
//
// What bounds it (GB300, L2 flushed, whole calls). Two query tiles: the chain of a
// group, S product (512 cycles), softmax, hand-off (400), P.V product (512); P lies over
// S, and two S and two O are all of TMEM, so S cannot be doubled. Cycles a key tile and
// pair of query tiles, whose products are 2048: bf16 2750 (softmax 1300), 8 bits 2900,
// 4 bits 3150 (softmax 1600: the widening warps take issue slots). Products keep
// their 512 cycles beside 60 bytes a cycle of other shared-memory traffic and full TMEM
// reading (measured), so neither is the bound. Halving S to double it (64 keys each) was
// slower: a product of 64 keys takes 384 cycles, not 256, as Q is read twice, and with
// both groups' softmaxes always running each took twice as long (1714 us against 1461 of
// an 8-bit prefill then). A boundary between units costs about 10000 cycles (epilogue,
// next Q, masked tiles).
//   4-bit prefill, 2048 rows x 64 heads over 32768 keys: 1440 us, 1480 TFLOP/s
//   8-bit, the same: 1300 us (in a row of calls, power-limited, 1366), 1640 TFLOP/s
//   4-bit, 32 branches of 1..32 tokens over 65536 shared keys: 829 us, 1205 TFLOP/s
//   8-bit, 32 branches of 1..64 drafted tokens over 65536 shared keys: 1500 us, 1505 TFLOP/s
//   bf16, 8 branches of 32 drafted tokens over 32768 shared keys: 184 us, 1516 TFLOP/s
//   bf16, 32 branches of 1..32 tokens over 16384 keys, window 2048: 94 us, 387 TFLOP/s
//   bf16 prefill, 4096 rows x 64 heads, window 1024: 158 us, 874 TFLOP/s
// One query tile (decode), 8 rows x 64 heads over 32768 keys: 28 us for 42.5 MB in 4
// bits, 25 us for 76 MB in 8, in a row of calls (bf16 pools through attn_fwd.cu: 45 us for
// 151 MB): of 41000 cycles a CTA 6000 pass until the first S and 6000 behind the last P;
// its 18 tiles take 1575 each, two groups in turn (softmax 1400, wait for the products
// 1450). Shorter chains gained little there (rows copied into a tile's idle half, so that
// a row's keys were split over two warps, gained nothing). Window 4096: 21 us, four tiles
// a CTA, start and epilogue.
// Every wait is bounded, as in attn_fwd.cu.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "launch_after.cuh"
#include "ptx_fp8.cuh"
#include "ptx_sm100.cuh"
#include "row_unit.cuh"
#include "rows.h"

namespace fanout {
namespace {

constexpr int kTileBytes = kBN * kHD * 2;   // one widened K or V tile
constexpr int kHalfBytes = kTileBytes / 2;  // 128 rows x 64 columns (128 B rows)
constexpr int kQBytes = kBM * kHD * 2;
constexpr float kRescaleLog2 = 8.0f;  // lazy rescale threshold (base-2 units)
constexpr int kErrTimeout = 5;        // FANOUT_ETIMEOUT
constexpr int kErrCuda = 3;           // FANOUT_ECUDA
constexpr uint64_t kLingerNs = 1000000;  // a CTA's stay after a wait has given up
constexpr int kGroupWarps = 4;
constexpr int kWarpSoftmax = 4;  // first softmax warp
constexpr int kWarpWiden = 12;   // first widening warp
constexpr int kFacBufs = 4;      // units whose row factors are held
// Barriers of a softmax group: S there; the first half of P there (and O rescaled), all of
// it; a unit's last product done; two for the join.
enum { SFULL = 0, PHALF = 1, PFULL = 2, ODONE = 3, JOIN = 4, kGroupBars = 6 };

// What differs between the pools: threads, registers a thread at launch and after the
// warpgroups' split (whose sum must not exceed what the block was launched with), rings.
template <int NQ, Pool F>
struct Cfg {
    static constexpr bool kQ4 = F == Pool::q4, kQ8 = F == Pool::q8;
    static constexpr bool kF16 = kQ4 || kQ8;  // V tiles are widened to f16, Q is scaled by row
    static constexpr int kWidenWarps = kQ4 ? 8 : kQ8 ? 4 : 0;
    static constexpr int kThreads = 32 * (kWarpWiden + kWidenWarps);
    static constexpr int kRegsLaunch = kQ4 ? 96 : 128, kRegsSoftmax = kQ4 ? 144 : 176;
    static constexpr int kRegsWiden = kQ4 ? 64 : 80, kRegsOther = kQ4 ? 64 : 80;
    static_assert(!kF16 || kRegsSoftmax * 256 + kRegsWiden * 32 * kWidenWarps + kRegsOther * 128 <=
                               kRegsLaunch * kThreads,
                  "register split");
    // K and V tiles that the products read (8-bit pools: K as it is cached), raw ones.
    static constexpr int kKStages = !kQ8 ? 2 : NQ == 1 ? 4 : 2, kVStages = 2;
    static constexpr int kStages = kKStages + kVStages;
    static constexpr int kKBytes = kQ8 ? kBN * kHD : kTileBytes;
    static constexpr int kRaw = kQ4 ? (NQ == 1 ? 6 : 2) : kQ8 ? (NQ == 1 ? 3 : 2) : 0;
    static constexpr int kRawBytes = kQ4 ? kBN * kQ4RowBytes : kBN * kHD;
    // The product over P's first half starts while the softmax works on its second. (bf16
    // pools, window prefill 164 -> 158 us, window over 32 branches 99 -> 97; 8 bits, prefill
    // 1411 -> 1400; 4 bits, prefill 1449 -> 1428, but 32 branches over 65536 keys 823 -> 846,
    // so not there.)
    static constexpr bool kEarlyP = !kQ4;
    // P is 2^lift times the probability's numerator
    static constexpr float kLiftLog2 = kF16 ? 7.0f : 0.0f, kUnlift = kF16 ? 0.0078125f : 1.0f;
    static constexpr uint32_t kIdescQK = kQ8   ? ptx::idesc_e4m3_f32(kBM, kBN)
                                         : kQ4 ? ptx::idesc_f16_f32(kBM, kBN, false, false)
                                               : ptx::idesc_bf16_f32(kBM, kBN, false, false);
    static constexpr uint32_t kIdescPV = kF16 ? ptx::idesc_f16_f32(kBM, kHD, false, true)
                                              : ptx::idesc_bf16_f32(kBM, kHD, false, true);
    // Ring positions: K tiles are even, V tiles odd. bf16 and 4-bit pools have one ring
    // for both, and the warps that widen one kind wait for its stages only: with an
    // odd ring a stage would change kind, and a warp could take the phase before last of
    // its barrier for the last. 8-bit pools have a ring for each.
    static_assert(kQ8 || (kStages == 4 && kRaw % 2 == 0), "rings of K/V pairs");
    static constexpr int kSmemQ = 0;
    static constexpr int kSmemRing = NQ * kQBytes;
    static constexpr int kSmemRaw = kSmemRing + kKStages * kKBytes + kVStages * kTileBytes;
    static constexpr int kSmemBar = kSmemRaw + kRaw * kRawBytes;
    static constexpr int BAR_FULL = 0;
    static constexpr int BAR_EMPTY = kStages;
    static constexpr int BAR_RFULL = 2 * kStages;
    static constexpr int BAR_REMPTY = BAR_RFULL + kRaw;
    static constexpr int BAR_QFULL = BAR_REMPTY + kRaw;  // + x
    static constexpr int BAR_QFREE = BAR_QFULL + NQ;     // + x
    static constexpr int BAR_QREADY = BAR_QFREE + NQ;    // + x
    static constexpr int BAR_OFREE = BAR_QREADY + NQ;
    static constexpr int BAR_AUX = BAR_OFREE + 1;
    static constexpr int BAR_DRAIN = BAR_AUX + 1;
    static constexpr int BAR_GROUP = BAR_DRAIN + 1;  // + kGroupBars x + {SFULL, ...}
    static constexpr int kNumBars = BAR_GROUP + 2 * kGroupBars;
    static constexpr int kSmemMisc = kSmemBar + kNumBars * 8;
    static constexpr int kSmemJoin = (kSmemMisc + 16 + 15) & ~15;  // float2 [2][2][128]
    static constexpr int kSmemFac = kSmemJoin + 2 * 2 * kBM * 8;  // uint8 [kFacBufs][NQ][128]
    static constexpr int kSmemTotal = kSmemFac + (kF16 ? kFacBufs * NQ * kBM : 0);
    static constexpr int kSmemAlloc = kSmemTotal;
    static_assert(kSmemAlloc <= 232448, "shared memory per CTA");
    static_assert(kSmemBar % 16 == 0 && kSmemRaw % 128 == 0, "shared-memory alignment");

    // The stage of a ring position, and the parity of its use.
    __device__ static __forceinline__ uint32_t stage(uint32_t pos) {
        if constexpr (!kQ8) return pos % kStages;
        return (pos & 1u) ? kKStages + (pos >> 1) % kVStages : (pos >> 1) % kKStages;
    }
    __device__ static __forceinline__ uint32_t parity(uint32_t pos) {
        if constexpr (!kQ8) return (pos / kStages) & 1u;
        return ((pos & 1u) ? (pos >> 1) / kVStages : (pos >> 1) / kKStages) & 1u;
    }
    // The raw stage of tile `pos` (8-bit pools: V tiles only) and the parity of its use.
    __device__ static __forceinline__ uint32_t raw_stage(uint32_t pos) {
        return kQ8 ? (pos >> 1) % (kRaw > 0 ? kRaw : 1) : pos % (kRaw > 0 ? kRaw : 1);
    }
    __device__ static __forceinline__ uint32_t raw_parity(uint32_t pos) {
        return ((kQ8 ? pos >> 1 : pos) / (kRaw > 0 ? kRaw : 1)) & 1u;
    }
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;

template <int NQ, Pool F>
struct Smem {
    using C = Cfg<NQ, F>;
    uint32_t base;  // shared-window address of the 1024-aligned base
    uint8_t* ptr;   // generic pointer to the same place
    __device__ uint32_t bar(int i) const { return base + C::kSmemBar + 8u * i; }
    __device__ uint32_t gbar(int x, int which) const { return bar(C::BAR_GROUP + kGroupBars * x + which); }
    __device__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(ptr + C::kSmemMisc); }
    __device__ volatile int* abort_flag() const {
        return reinterpret_cast<volatile int*>(ptr + C::kSmemMisc + 4);
    }
    __device__ uint32_t tile(uint32_t pos) const {
        if constexpr (!C::kQ8) return base + C::kSmemRing + (pos % C::kStages) * kTileBytes;
        const uint32_t v = base + C::kSmemRing + C::kKStages * C::kKBytes;
        return (pos & 1u) ? v + (pos >> 1) % C::kVStages * kTileBytes
                          : base + C::kSmemRing + (pos >> 1) % C::kKStages * C::kKBytes;
    }
    // Exponent of the power of two that row `row` of the n-th load of Q buffer x
    // was multiplied with, plus 127 (a byte).
    __device__ uint8_t* fac(uint32_t n, int x, int row) const {
        return ptr + C::kSmemFac + ((n % kFacBufs) * NQ + x) * kBM + row;
    }
};

// Wait of a whole warp (every lane returns the same). Bounded: false once another
// wait of the CTA has given up, or after p.wait_limit_ns; the site goes into the
// CTA's abort word, which the kernel reports at its end. Every role's waits are
// inlined, and the roles share an instruction cache that their code overflows, so
// this is kept short.
template <int NQ, Pool F>
__device__ __forceinline__ bool warp_wait(const RowParams& p, const Smem<NQ, F>& sm, uint32_t bar,
                                          uint32_t parity, int site) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; !__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)); ++i) {
        if ((i & 63u) != 0) continue;
        const uint64_t now = ptx::globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *sm.abort_flag() != 0 || now - t0 > p.wait_limit_ns)) {
            if (*sm.abort_flag() == 0) *sm.abort_flag() = site;
            return false;
        }
    }
    return true;
}

// Query tiles of a unit.
template <int NQ>
__device__ __forceinline__ int unit_nq(const Unit& u, int tpt) {
    return (NQ == 2 && u.n_tok > tpt) ? 2 : 1;
}

// The tiles of a unit, in sweep order: its first keys, then its own range.
struct Tiles {
    int n_first, first_begin, first_end, begin, end, key_begin, n;
    __device__ Tiles(const RowParams& p, const Unit& u)
        : n_first(first_tiles(u, p.split_at)),
          first_begin(fanout::first_begin(u, p.split_at)),
          first_end(u.pos_base),
          begin(range_begin(u, p.page_size)),
          end(u.key_end),
          key_begin(u.key_begin),
          n(n_first + range_tiles(u, p.page_size)) {}
    // first key, one past the last key, first key that some row sees
    __device__ __forceinline__ void tile(int j, int& kt, int& last, int& front) const {
        const bool f = j < n_first;
        kt = f ? first_begin + j * kBN : begin + (j - n_first) * kBN;
        last = min(kt + kBN, f ? first_end : end);
        front = f ? 0 : max(0, key_begin - kt);
    }
};

// ------------------------------------------------------------------ producer
template <int NQ, Pool F>
__device__ void producer_warp(const RowParams& p, const Smem<NQ, F>& sm, const CUtensorMap* tm_q,
                              const CUtensorMap* tm_k, const CUtensorMap* tm_v) {
    using C = Cfg<NQ, F>;
    const int lane = threadIdx.x & 31;
    volatile int* abort = sm.abort_flag();
    const int ps = p.page_size;
    const int64_t block = static_cast<int64_t>(ps) * kQ4RowBytes;
    // the barriers of tile `pos` in the ring this warp fills: raw tiles (8-bit pools: V
    // only), or the tiles that the products read
    auto is_raw = [](uint32_t pos) { return C::kQ4 || (C::kQ8 && (pos & 1u)); };
    auto full_of = [&](uint32_t pos) {
        return is_raw(pos) ? sm.bar(C::BAR_RFULL + C::raw_stage(pos))
                           : sm.bar(C::BAR_FULL + C::stage(pos));
    };
    auto parity_of = [&](uint32_t pos) { return is_raw(pos) ? C::raw_parity(pos) : C::parity(pos); };
    uint32_t it = 0;                // tiles issued
    // bf16 pools: a V tile that holds rows no row of the unit sees (in front of
    // tail_front, from tail_valid) is zeroed there when its pages have landed, which
    // the warp waits for only after the next K tile is on its way. (K's such rows stay:
    // their scores are masked, whatever they are.)
    uint32_t n_aux = 0;             // such tiles finished
    bool aux_pending = false;
    uint32_t tail_pos = 0;
    int tail_front = 0, tail_valid = 0;
    uint32_t q_loads[NQ] = {};      // loads of each Q buffer so far
    bool ok = true;

    // Q tile x of unit u into its buffer, whose last S products have completed.
    auto load_q = [&](const Unit& u, int x) {
        if (lane == 0) {
            const uint32_t qb = sm.bar(C::BAR_QFULL + x);
            const int box_bytes = p.G * p.tpt * 128;  // one half of one query tile
            ptx::mbar_arrive_expect_tx(qb, static_cast<uint32_t>(2 * box_bytes));
            const uint32_t dst = sm.base + C::kSmemQ + x * kQBytes;
            const int y = u.kv_head * p.G, z = u.tok_begin + x * p.tpt;
            ptx::tma_load_3d(dst, tm_q, qb, 0, y, z);
            ptx::tma_load_3d(dst + kHalfBytes, tm_q, qb, 64, y, z);
        }
    };
    auto q_free = [&](int x) {
        return q_loads[x] == 0 ||
               ptx::mbar_test_wait(sm.bar(C::BAR_QFREE + x), (q_loads[x] - 1) & 1u);
    };

    auto zero_tail = [&]() {
        const uint32_t dst = sm.tile(tail_pos);
        for (int i = lane; i < (kBN - tail_valid + tail_front) * 16; i += 32) {
            const int r = (i >> 4) < tail_front ? i >> 4 : tail_valid + (i >> 4) - tail_front;
            const uint32_t ch = i & 15;
            ptx::st_shared_v4(dst + (ch >> 3) * kHalfBytes + r * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full_of(tail_pos));
        aux_pending = false;
        ++n_aux;
    };

    const int ui_end = p.cta_first[blockIdx.x + 1];
    for (int ui = p.cta_first[blockIdx.x]; ui < ui_end && ok; ++ui) {
        const Unit u = p.units[ui];
        const Tiles tl(p, u);
        const int nq = unit_nq<NQ>(u, p.tpt);
        if (lane == 0 && ui + 1 < ui_end) {  // the next unit's Q into L2
            const Unit un = p.units[ui + 1];
            for (int x = 0; x < unit_nq<NQ>(un, p.tpt); ++x) {
                const int y = un.kv_head * p.G, z = un.tok_begin + x * p.tpt;
                ptx::tma_prefetch_3d(tm_q, 0, y, z);
                ptx::tma_prefetch_3d(tm_q, 64, y, z);
            }
        }
        // The unit's Q waits for the previous unit's last S products while its
        // raw tiles already flow: Q goes out as soon as its buffer is seen free.
        int q_next = 0;
        auto try_q = [&]() {
            while (q_next < nq && __shfl_sync(0xffffffffu, q_free(q_next), 0)) {
                load_q(u, q_next);
                ++q_loads[q_next];
                ++q_next;
            }
        };
        // Waits for a barrier of this warp, sending Q when it can.
        auto wait_for = [&](uint32_t bar, uint32_t parity, int site) {
            uint64_t t0 = 0;
            for (uint32_t i = 0;; ++i) {
                try_q();
                if (q_next == nq) return warp_wait<NQ, F>(p, sm, bar, parity, site);
                if (__all_sync(0xffffffffu, ptx::mbar_test_wait(bar, parity))) return true;
                if ((i & 63u) == 63u) {
                    const uint64_t now = ptx::globaltimer_ns();
                    if (t0 == 0) t0 = now;
                    if (__any_sync(0xffffffffu, *abort != 0 || now - t0 > p.wait_limit_ns)) {
                        if (*abort == 0) *abort = site;
                        return false;
                    }
                }
            }
        };
        auto finish_tail = [&]() {
            if (!wait_for(sm.bar(C::BAR_AUX), n_aux & 1u, 3)) return false;
            zero_tail();
            return true;
        };
        const int32_t* table = p.page_table + static_cast<int64_t>(u.branch) * p.max_pages;
        for (int run = tl.n_first > 0 ? 0 : 1; run < 2 && ok; ++run) {
            const int begin = run == 0 ? tl.first_begin : tl.begin;
            const int end = run == 0 ? tl.first_end : tl.end;
            const int n_tiles = (end - begin + kBN - 1) / kBN;
            const int n_pages = (end - begin + ps - 1) / ps;
            const int ppt = kBN / ps;  // pages per tile: 1, 2, 4 or 8 (divides 32)
            // page ids, 32 per window, loaded one window ahead
            auto load_window = [&](int w) -> int {
                const int idx = w * 32 + lane;
                return idx < n_pages ? table[begin / ps + idx] : 0;
            };
            int win = 0, win_cur = load_window(0), win_nxt = load_window(1);
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int n_pg = min(ppt, n_pages - j * ppt);
                if (((j * ppt) >> 5) != win) {
                    win = (j * ppt) >> 5;
                    win_cur = win_nxt;
                    win_nxt = load_window(win + 1);
                }
                const int page = __shfl_sync(0xffffffffu, win_cur, ((j * ppt) & 31) + (lane & 7));
                const int page_ok = lane < n_pg ? checked_page(p, page) : 0;
                const int64_t head = static_cast<int64_t>(page_ok) * p.H_kv + u.kv_head;
                // rows of the tile that no row of the unit sees: before front, from n_valid
                const int front = run == 1 && j == 0 ? tl.key_begin - tl.begin : 0;
                const int n_valid = min(kBN, end - (begin + j * kBN));
                for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                    if (!C::kF16 && kv == 1 && aux_pending && !(ok = finish_tail())) break;
                    const uint32_t empty = is_raw(it) ? sm.bar(C::BAR_REMPTY + C::raw_stage(it))
                                                      : sm.bar(C::BAR_EMPTY + C::stage(it));
                    ok = wait_for(empty, parity_of(it) ^ 1u, 2);
                    if (!ok) break;
                    const uint32_t full = full_of(it);
                    if (C::kQ4) {
                        if (lane == 0)
                            ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(n_pg) *
                                                                 static_cast<uint32_t>(block));
                        __syncwarp();
                        if (lane < n_pg)
                            ptx::bulk_load(sm.base + C::kSmemRaw + C::raw_stage(it) * C::kRawBytes +
                                               lane * static_cast<uint32_t>(block),
                                           (kv == 0 ? p.k_pool : p.v_pool) + head * block,
                                           static_cast<uint32_t>(block), full);
                    } else if (C::kQ8) {
                        // a row is one swizzled line; scores of rows past the pages are masked
                        const uint32_t dst =
                            kv == 0 ? sm.tile(it)
                                    : sm.base + C::kSmemRaw + C::raw_stage(it) * C::kRawBytes;
                        if (lane == 0)
                            ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(n_pg * ps) * 128u);
                        __syncwarp();
                        if (lane < n_pg)
                            ptx::tma_load_2d(dst + static_cast<uint32_t>(lane * ps) * 128u,
                                             kv == 0 ? tm_k : tm_v, full, 0,
                                             static_cast<int>(head * ps));
                    } else {
                        const bool partial = kv == 1 && (n_valid < kBN || front > 0);
                        const uint32_t bar = partial ? sm.bar(C::BAR_AUX) : full;
                        const uint32_t dst = sm.tile(it);
                        if (lane == 0)
                            ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n_pg * ps) * 256u);
                        __syncwarp();
                        if (lane < n_pg) {
                            const CUtensorMap* tm = kv == 0 ? tm_k : tm_v;
                            const int row = static_cast<int>(head * ps);
                            const uint32_t off = static_cast<uint32_t>(lane * ps) * 128u;
                            ptx::tma_load_2d(dst + off, tm, bar, 0, row);
                            ptx::tma_load_2d(dst + kHalfBytes + off, tm, bar, 64, row);
                        }
                        if (partial) {
                            aux_pending = true;
                            tail_pos = it;
                            tail_front = front;
                            tail_valid = n_valid;
                        }
                    }
                }
            }
        }
        // Q buffers not seen free so far
        for (; ok && q_next < nq; try_q())
            if (q_loads[q_next] > 0)
                ok = warp_wait<NQ, F>(p, sm, sm.bar(C::BAR_QFREE + q_next),
                                       (q_loads[q_next] - 1) & 1u, 1);
    }
    if (!C::kF16 && ok && aux_pending) {
        ok = warp_wait<NQ, F>(p, sm, sm.bar(C::BAR_AUX), n_aux & 1u, 3);
        if (ok) zero_tail();
    }
    // (see attn_fwd.cu: the merge grid may start once every copy is issued)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!ok && lane == 0) {
        // Drain: every copy this warp started must land before the CTA exits.
        // (A V tile that still waits for its pages is covered by the AUX barrier: its
        // full barrier never completes.)
        // The last tiles, as many as a ring holds (8-bit pools: the larger of two rings; a
        // tile before a ring's last ones has landed, and its wait ends at once or, where
        // its stage is two uses on, runs out).
        constexpr uint32_t kRing = C::kQ4 ? C::kRaw : C::kQ8 ? 2 * C::kKStages : C::kStages;
        const uint32_t n = it < kRing ? it : kRing;
        for (uint32_t i = it - n; i != it; ++i)
            if (!aux_pending || i != tail_pos)
                ptx::mbar_wait(full_of(i), parity_of(i), p.wait_limit_ns, nullptr);
        if (aux_pending) ptx::mbar_wait(sm.bar(C::BAR_AUX), n_aux & 1u, p.wait_limit_ns, nullptr);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
            if (q_loads[x] > 0)
                ptx::mbar_wait(sm.bar(C::BAR_QFULL + x), (q_loads[x] - 1) & 1u, p.wait_limit_ns,
                               nullptr);
    }
}

// ------------------------------------------------------------------ Q tiles
// The warps that widen V tiles turn a unit's loaded Q tiles into what the products take,
// in place, before its first V tile (which S, and so Q, comes before): 4 lanes a row, 32
// values each, in pieces of 16 bytes. They find the row's largest exponent, scale by a
// power of two and store. Rows behind the unit's last are left as they are (their scores
// are never used).
//
// 4-bit pools: f16, the 8 values of a piece in the order the widened K tiles have.
//
// 8-bit pools: K stays in e4m3, so Q goes to the product in two e4m3 parts: a bf16 value
// has 8 significant bits, e4m3 four, and x = upper + lower with upper = x rounded to e4m3
// and lower the exact rest, whose own 4 bits hold it. A row's largest element goes into
// [2^7, 2^8); elements below 2^-9 of that lose bits, each at most half of e4m3's smallest
// step of 2^-9, 2^-17 of the row's largest. A step of the product takes 32 values: their
// upper parts replace the first two of the four pieces that held them, their lower parts
// the last two, and the step runs over the same 32 values of K twice. A row with an
// infinity or a NaN is NaN.
template <int NQ, Pool F>
__device__ __forceinline__ bool convert_q(const RowParams& p, const Smem<NQ, F>& sm, const Unit& u, int w,
                                          uint32_t (&loads)[2]) {
    using C = Cfg<NQ, F>;
    const int lane = threadIdx.x & 31, q = (lane & 3) * 4;
    const int nq = unit_nq<NQ>(u, p.tpt);
    for (int x = 0; x < nq; ++x) {
        const uint32_t n = x == 0 ? loads[0]++ : loads[1]++;
        if (!warp_wait<NQ, F>(p, sm, sm.bar(C::BAR_QFULL + x), n & 1u, 50)) return false;
        const int rows = min(p.tpt, u.n_tok - x * p.tpt) * p.G;
        // (whole warps go round: a row's lanes exchange its largest exponent)
#pragma unroll 1
        for (int row0 = w * 8; row0 < rows; row0 += 8 * kGroupWarps) {
            const int row = row0 + (lane >> 2);
            const uint32_t at = sm.base + C::kSmemQ + x * kQBytes + row * 128;
            const uint32_t swz = static_cast<uint32_t>(row & 7) << 4;
            auto piece = [&](int c) { return at + (c >> 3) * kHalfBytes + (((c & 7) << 4) ^ swz); };
            uint4 v[4];
            uint32_t t = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = ptx::ld_shared_v4(piece(q + c));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                t = ptx::max_nan_bf16x2(t, v[c].x & 0x7fff7fffu);
                t = ptx::max_nan_bf16x2(t, v[c].y & 0x7fff7fffu);
                t = ptx::max_nan_bf16x2(t, v[c].z & 0x7fff7fffu);
                t = ptx::max_nan_bf16x2(t, v[c].w & 0x7fff7fffu);
            }
            t = ptx::max_nan_bf16x2(t, __shfl_xor_sync(0xffffffffu, t, 1));
            t = ptx::max_nan_bf16x2(t, __shfl_xor_sync(0xffffffffu, t, 2));
            const int e = max((t >> 7) & 0xff, (t >> 23) & 0xff);
            // f16: largest element to [2^14, 2^15); tiny rows times at most 2^100
            const int k = e == 255 ? 0 : min((C::kQ8 ? 134 : 141) - e, 100);
            const float f = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
            auto lo = [f](uint32_t b) { return __uint_as_float(b << 16) * f; };
            auto hi = [f](uint32_t b) { return __uint_as_float(b & 0xffff0000u) * f; };
            if (row >= rows) continue;
            if constexpr (C::kQ8) {
                uint32_t up[8], rest[8];  // 4 values each
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // (f16 holds the scaled values' 8 bits down to 2^-17)
                    ptx::split_e4m3x4(ptx::pack_f16x2(lo(v[c].x), hi(v[c].x)),
                                      ptx::pack_f16x2(lo(v[c].y), hi(v[c].y)), up[2 * c], rest[2 * c]);
                    ptx::split_e4m3x4(ptx::pack_f16x2(lo(v[c].z), hi(v[c].z)),
                                      ptx::pack_f16x2(lo(v[c].w), hi(v[c].w)), up[2 * c + 1],
                                      rest[2 * c + 1]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (e == 255) up[i] = 0x7f7f7f7fu;
                    if (e == 255) rest[i] = 0u;
                }
                ptx::st_shared_v4(piece(q), up[0], up[1], up[2], up[3]);
                ptx::st_shared_v4(piece(q + 1), up[4], up[5], up[6], up[7]);
                ptx::st_shared_v4(piece(q + 2), rest[0], rest[1], rest[2], rest[3]);
                ptx::st_shared_v4(piece(q + 3), rest[4], rest[5], rest[6], rest[7]);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    ptx::st_shared_v4(piece(q + c), ptx::pack_f16x2(lo(v[c].x), lo(v[c].y)),
                                      ptx::pack_f16x2(lo(v[c].z), lo(v[c].w)),
                                      ptx::pack_f16x2(hi(v[c].x), hi(v[c].y)),
                                      ptx::pack_f16x2(hi(v[c].z), hi(v[c].w)));
            }
            if ((lane & 3) == 0) *sm.fac(n, x, row) = static_cast<uint8_t>(k + 127);
        }
        __syncwarp();
        ptx::fence_proxy_async_smem();  // the MMAs read the tile
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sm.bar(C::BAR_QREADY + x));
    }
    return true;
}

// ------------------------------------------------------------------ widening
// Eight codes to eight f16 values (0 2 4 6 1 3 5 7) times their group's scale.
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
    ptx::f16x2_of_e2m1x8(w, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ptx::mul_f16x2(o[i], scale);
}

// Four warps widen every K (V) tile, 32 rows each. A lane takes 16 bytes of codes
// (32 values, two groups) of a row, 4 rows in all, loaded before any is widened;
// loads are without bank conflicts, and lanes of the upper 64 columns store their
// words in the order 2, 3, 0, 1, so that the 8 lanes of a store phase cover all 8
// sixteen-byte columns. A row that no row of the unit sees gets scale 0 (codes are
// finite whatever they are).
template <int NQ>
__device__ void widen_warp(const RowParams& p, const Smem<NQ, Pool::q4>& sm, int w, bool is_v) {
    using C = Cfg<NQ, Pool::q4>;
    const int lane = threadIdx.x & 31;
    const int ps = p.page_size, ps_shift = 31 - __clz(ps), piece = lane & 3;
    const bool upper = piece >= 2;
    const int row0 = w * 32 + (lane >> 2);
    // scale of the first (second) stored pair of words, of the two loaded
    const uint32_t sel0 = upper ? 0x3232u : 0x1010u, sel1 = upper ? 0x1010u : 0x3232u;
    uint32_t code_at[4], scale_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + 8 * i, slot = r & (ps - 1);
        const uint32_t block = (r - slot) * kQ4RowBytes;
        code_at[i] = block + slot * 64 + piece * 16;
        scale_at[i] = block + ps * 64 + slot * 8 + piece * 2;
    }
    const uint32_t row_at = (piece >> 1) * kHalfBytes + row0 * 128;
    const uint32_t col =
        static_cast<uint32_t>(((piece & 1) * 4) ^ (upper ? 2 : 0) ^ (row0 & 7)) << 4;
    uint32_t it = is_v ? 1u : 0u;  // ring position of these warps' next tile
    uint32_t loads[2] = {0, 0};
    const int ui_end = p.cta_first[blockIdx.x + 1];
    for (int ui = p.cta_first[blockIdx.x]; ui < ui_end; ++ui) {
        const Unit u = p.units[ui];
        if (is_v && !convert_q<NQ, Pool::q4>(p, sm, u, w, loads)) return;
        const Tiles tl(p, u);
        for (int j = 0; j < tl.n; ++j, it += 2) {
            int kt, last, front;
            tl.tile(j, kt, last, front);
            const uint32_t rs = it % C::kRaw, stage = it % C::kStages;
            if (!warp_wait<NQ, Pool::q4>(p, sm, sm.bar(C::BAR_RFULL + rs), (it / C::kRaw) & 1u, 40)) return;
            const uint32_t raw = sm.base + C::kSmemRaw + rs * C::kRawBytes;
            uint4 c[4];
            uint32_t sc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = ptx::ld_shared_v4(raw + code_at[i]);
                const int r = row0 + 8 * i;
                sc[i] = ptx::ld_shared_u16(raw + scale_at[i]);
                if (r < front || kt + r >= last) sc[i] = 0;
            }
            // The raw stage is free once its words are in registers, which a loaded
            // value's use shows and the loads' issue does not (an arrival right behind
            // them let the next copy overwrite words still to be read): a vote over all
            // of them. Should the vote come out true, the stage is freed further down.
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) seen ^= c[i].x ^ c[i].y ^ c[i].z ^ c[i].w ^ sc[i];
            const bool late = __all_sync(0xffffffffu, seen == 0x9e3779b9u);
            if (lane == 0 && !late) ptx::mbar_arrive(sm.bar(C::BAR_REMPTY + rs));
            if (!warp_wait<NQ, Pool::q4>(p, sm, sm.bar(C::BAR_EMPTY + stage), ((it / C::kStages) & 1u) ^ 1u, 41))
                return;
            const uint32_t dst = sm.tile(it) + row_at;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t s = ptx::f16x2_of_e4m3x2(sc[i]);
                const uint32_t s0 = __byte_perm(s, 0u, sel0), s1 = __byte_perm(s, 0u, sel1);
                const uint32_t word[4] = {upper ? c[i].z : c[i].x, upper ? c[i].w : c[i].y,
                                          upper ? c[i].x : c[i].z, upper ? c[i].y : c[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t o[4];
                    widen_word(word[k], k < 2 ? s0 : s1, o);
                    ptx::st_shared_v4(dst + i * 1024 + (col ^ (k << 4)), o[0], o[1], o[2], o[3]);
                }
            }
            ptx::fence_proxy_async_smem();  // the MMAs read the tile
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(sm.bar(C::BAR_FULL + stage));
                if (late) ptx::mbar_arrive(sm.bar(C::BAR_REMPTY + rs));
            }
        }
    }
}

// 8-bit pools: four warps widen every V tile to f16 (exact), 32 rows each. A lane takes 16
// values of a row; the raw tile and the 16-bit one are swizzled alike, and 8 lanes that
// load or store together take 64 values of a row r and of r ^ 5: those differ in the bits
// that keep their loads (of 4 neighbouring pieces) and their stores (of every second) out
// of each other's banks, so that nothing has to be selected. Rows that no row of the unit
// sees become zeros.
template <int NQ>
__device__ void widen_warp_e4m3(const RowParams& p, const Smem<NQ, Pool::q8>& sm, int w) {
    using C = Cfg<NQ, Pool::q8>;
    const int lane = threadIdx.x & 31;
    // lane: piece of the half row, row or its partner, half of the row, one of two row pairs
    const int part = lane & 3, half = (lane >> 3) & 1;
    // rows 0 5, 1 4 (of a group of 8) in the first step, 2 7, 3 6 in the second
    const int row0 = w * 32 + ((lane >> 4) ^ (lane & 4 ? 5 : 0));
    uint32_t it = 1;  // ring position of the next V tile
    uint32_t loads[2] = {0, 0};
    const int ui_end = p.cta_first[blockIdx.x + 1];
    for (int ui = p.cta_first[blockIdx.x]; ui < ui_end; ++ui) {
        const Unit u = p.units[ui];
        if (!convert_q<NQ, Pool::q8>(p, sm, u, w, loads)) return;
        const Tiles tl(p, u);
        for (int j = 0; j < tl.n; ++j, it += 2) {
            int kt, last, front;
            tl.tile(j, kt, last, front);
            const uint32_t rs = C::raw_stage(it), stage = C::stage(it);
            if (!warp_wait<NQ, Pool::q8>(p, sm, sm.bar(C::BAR_RFULL + rs), C::raw_parity(it), 40)) return;
            if (!warp_wait<NQ, Pool::q8>(p, sm, sm.bar(C::BAR_EMPTY + stage), C::parity(it) ^ 1u, 41))
                return;
            const uint32_t raw = sm.base + C::kSmemRaw + rs * C::kRawBytes;
            const uint32_t dst = sm.tile(it) + half * kHalfBytes;
            const bool border = front > 0 || last - kt < kBN;
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {  // two groups of 8 rows at a time
                uint4 c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = row0 ^ (i & 1 ? 2 : 0), line = (r + 16 * g + 8 * (i >> 1)) * 128;
                    c[i] = ptx::ld_shared_v4(raw + line + ((((half << 2) + part) ^ (r & 7)) << 4));
                }
                if (border) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = (row0 ^ (i & 1 ? 2 : 0)) + 16 * g + 8 * (i >> 1);
                        if (r < front || kt + r >= last) c[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = row0 ^ (i & 1 ? 2 : 0);
                    const uint32_t at = dst + (r + 16 * g + 8 * (i >> 1)) * 128;
                    const uint32_t p0 = static_cast<uint32_t>((2 * part) ^ (r & 7)) << 4;
                    uint32_t o[8];
                    ptx::f16x2_of_e4m3x4(c[i].x, o[0], o[1]);
                    ptx::f16x2_of_e4m3x4(c[i].y, o[2], o[3]);
                    ptx::f16x2_of_e4m3x4(c[i].z, o[4], o[5]);
                    ptx::f16x2_of_e4m3x4(c[i].w, o[6], o[7]);
                    ptx::st_shared_v4(at + p0, o[0], o[1], o[2], o[3]);
                    ptx::st_shared_v4(at + (p0 ^ 16u), o[4], o[5], o[6], o[7]);
                }
            }
            // (every word has been used by now, so the raw stage is free)
            ptx::fence_proxy_async_smem();  // the MMAs read the tile
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(sm.bar(C::BAR_REMPTY + rs));
                ptx::mbar_arrive(sm.bar(C::BAR_FULL + stage));
            }
        }
    }
}

// ------------------------------------------------------------------ MMA issuer
// Descriptors: see attn_fwd.cu (the same tile layouts).
__device__ __forceinline__ uint32_t kmajor_step(int kk) {
    return static_cast<uint32_t>((kk >> 2) * (kHalfBytes >> 4) + (kk & 3) * 2);
}

// A value that is the same in all lanes, as the compiler can see: it then keeps what comes
// of it in uniform registers, where a product's operands have to be.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
    return __ballot_sync(0xffffffffu, (v >> (threadIdx.x & 31)) & 1u);
}
// A descriptor from its lower word (uniform) and constants: see ptx::sdesc_sw128.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | 2u << 29;
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return uniform(((saddr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16);
}

// One P.V product: group x's P of its t-th tile times the V tile at ring position
// pos. first: the group's first product of unit k (O is overwritten; both groups
// must have read the previous unit's O); last: its last one there.
struct PvOp {
    int x;
    uint32_t t;
    bool first, last;
    int k;
    uint32_t pos;
};

template <int NQ, Pool F>
struct Issuer {
    using C = Cfg<NQ, F>;
    const RowParams& p;
    const Smem<NQ, F>& sm;
    uint32_t leader;  // 1 in the lane that issues
    bool issued_any = false;

    __device__ __forceinline__ uint32_t full(uint32_t pos) const {
        return sm.bar(C::BAR_FULL + C::stage(pos));
    }
    __device__ __forceinline__ uint32_t full_par(uint32_t pos) const { return C::parity(pos); }
    __device__ __forceinline__ void commit(uint32_t bar) { ptx::mma_commit_if(bar, leader); }
    __device__ __forceinline__ void release(uint32_t pos) {
        commit(sm.bar(C::BAR_EMPTY + C::stage(pos)));
    }
    // Waits for up to four barriers at once, a lane each: a probe is a trip through a
    // busy shared-memory pipe (200 cycles and more), and this warp's trips are what the
    // tensor core waits for.
    __device__ __forceinline__ bool wait(uint32_t bar0, uint32_t par0, uint32_t bar1, uint32_t par1,
                                         uint32_t bar2, uint32_t par2, uint32_t bar3, uint32_t par3,
                                         int site) {
        const uint32_t l = threadIdx.x & 31;
        return warp_wait<NQ, F>(p, sm, l == 1 ? bar1 : l == 2 ? bar2 : l == 3 ? bar3 : bar0,
                                 l == 1 ? par1 : l == 2 ? par2 : l == 3 ? par3 : par0, site);
    }
    // S of group x = Q tile qx times the K tile at pos.
    __device__ __forceinline__ void issue_s(int x, int qx, uint32_t pos) {
        ptx::tc_fence_after();
        const uint32_t dq = desc_lo(sm.base + C::kSmemQ + qx * kQBytes, 16);
        const uint32_t dk = desc_lo(sm.tile(pos), 16);
        const uint32_t d = uniform(128u * x);
#pragma unroll
        for (int kk = 0; kk < kHD / 16; ++kk) {
            if constexpr (C::kQ8)  // 32 values of K times their upper, then their lower parts of Q
                ptx::mma_e4m3_ss_if(d, desc_of(dq + kmajor_step(kk)), desc_of(dk + 2u * (kk >> 1)),
                                    C::kIdescQK, kk > 0, leader);
            else
                ptx::mma_f16_ss_if(d, desc_of(dq + kmajor_step(kk)), desc_of(dk + kmajor_step(kk)),
                                   C::kIdescQK, kk > 0, leader);
        }
        commit(sm.gbar(x, SFULL));
        issued_any = true;
    }
    // P written (and O rescaled), V widened or loaded, O free; and the tile at `next`,
    // which the S product that follows reads (any tile of the ring that is there, if
    // none does). The product over P's first half runs while the softmax still works on
    // its second.
    __device__ __forceinline__ bool issue_pv(const PvOp& op, uint32_t next) {
        const uint32_t pf = sm.gbar(op.x, C::kEarlyP ? PHALF : PFULL);
        const bool of = op.first && op.k > 0;
        if (!wait(pf, op.t & 1u, full(op.pos), full_par(op.pos), of ? sm.bar(C::BAR_OFREE) : pf,
                  of ? (op.k - 1) & 1u : op.t & 1u, full(next), full_par(next), 14))
            return false;
        ptx::tc_fence_after();
        const uint32_t a = uniform(128u * op.x);  // P: 64 columns of 16-bit pairs
        const uint32_t d = kColO + a;
        const uint32_t dv = desc_lo(sm.tile(op.pos), kHalfBytes);
#pragma unroll
        for (int kk = 0; kk < kBN / 32; ++kk)
            ptx::mma_f16_ts_if(d, a + 8u * kk, desc_of(dv + 128u * kk), C::kIdescPV,
                               (!op.first || kk > 0) ? 1u : 0u, leader);
        issued_any = true;
        if (C::kEarlyP) {
            if (!warp_wait<NQ, F>(p, sm, sm.gbar(op.x, PFULL), op.t & 1u, 15)) return false;
            ptx::tc_fence_after();
        }
#pragma unroll
        for (int kk = kBN / 32; kk < kBN / 16; ++kk)
            ptx::mma_f16_ts_if(d, a + 8u * kk, desc_of(dv + 128u * kk), C::kIdescPV, 1u, leader);
        if (op.last) commit(sm.gbar(op.x, ODONE));
        return true;
    }
    // The held P.V of a unit of one query tile, if any.
    __device__ __forceinline__ bool issue_held(const PvOp& op, bool& held) {
        if (!held) return true;
        held = false;
        if (!issue_pv(op, op.pos)) return false;
        release(op.pos);
        return true;
    }
};

// Two query tiles per unit: S_0(j), P.V_1(j-1), S_1(j), P.V_0(j). One query tile:
// S(t) into the buffer of group t mod 2, then P.V(t-1) of the other group; a unit's
// last P.V is held until the next such unit's first S is issued. An S that reuses the
// TMEM of an earlier P is always issued after that P's product. TMEM starts at column
// 0 (the CTA has all of it). One loop with few branches: a state machine over both
// groups' next steps, and loops specialised by ring stage, had longer code paths and
// were slower (a prefill 2237 and 1687 us when this one took 1558).
template <int NQ, Pool F>
__device__ void mma_warp(const RowParams& p, const Smem<NQ, F>& sm) {
    using C = Cfg<NQ, F>;
    Issuer<NQ, F> is{p, sm, ptx::elect_one()};
    // a Q tile is usable when converted (4-bit pools) or loaded
    constexpr int kQBar = C::kF16 ? C::BAR_QREADY : C::BAR_QFULL;
    bool ok = true;
    uint32_t pos = 0;           // ring position of the unit's K_0 (K_j at pos + 2j, V_j behind it)
    uint32_t jt0 = 0, jt1 = 0;  // tiles each softmax group got before
    uint32_t qu0 = 0, qu1 = 0;  // loads of each Q buffer consumed
    PvOp pend{0, 0, false, false, 0, 0};
    bool held = false;
    int k = 0;
    const int ui_end = p.cta_first[blockIdx.x + 1];
    for (int ui = p.cta_first[blockIdx.x]; ui < ui_end && ok; ++ui, ++k) {
        const Unit u = p.units[ui];
        const int n = __shfl_sync(0xffffffffu, Tiles(p, u).n, 0);
        const uint32_t qb0 = sm.bar(kQBar), qb1 = sm.bar(kQBar + NQ - 1);
        if (__shfl_sync(0xffffffffu, unit_nq<NQ>(u, p.tpt), 0) == 2) {
            if (!(ok = is.issue_held(pend, held))) break;
            for (int j = 0; j <= n && ok; ++j) {
                const uint32_t posK = pos + 2u * j, posV = posK + 1u, posVp = posK - 1u;
                if (j < n) {
                    if (j == 0 && !(ok = is.wait(is.full(posK), is.full_par(posK), qb0, qu0 & 1u,
                                                 qb1, qu1 & 1u, qb0, qu0 & 1u, 11)))
                        break;
                    is.issue_s(0, 0, posK);
                    if (j == n - 1) is.commit(sm.bar(C::BAR_QFREE));
                }
                if (j > 0) {
                    if (!(ok = is.issue_pv(PvOp{1, jt1 + j - 1, j == 1, j == n, k, posVp}, posVp))) break;
                    is.release(posVp);
                }
                if (j < n) {
                    is.issue_s(1, NQ - 1, posK);
                    is.release(posK);
                    if (j == n - 1) is.commit(sm.bar(C::BAR_QFREE + NQ - 1));
                    // the next tile's S_0 follows at once
                    if (!(ok = is.issue_pv(PvOp{0, jt0 + j, j == 0, j == n - 1, k, posV},
                                           j + 1 < n ? posV + 1u : posV)))
                        break;
                }
            }
            if (!ok) break;
            jt0 += n;
            jt1 += n;
            ++qu0;
            ++qu1;
        } else {
            if (held && !__all_sync(0xffffffffu, ptx::mbar_test_wait(qb0, qu0 & 1u)) &&
                !(ok = is.issue_held(pend, held)))
                break;
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t posK = pos + 2u * j;
                const int x = (posK >> 1) & 1u;
                const uint32_t fk = is.full(posK), fp = is.full_par(posK);
                if (!(ok = is.wait(fk, fp, j == 0 ? qb0 : fk, j == 0 ? qu0 & 1u : fp, fk, fp, fk, fp, 11)))
                    break;
                is.issue_s(x, 0, posK);
                is.release(posK);
                if (j == n - 1) is.commit(sm.bar(C::BAR_QFREE));
                if (!(ok = is.issue_held(pend, held))) break;
                const uint32_t t = x == 0 ? jt0++ : jt1++;
                pend = PvOp{x, t, j < 2, j >= n - 2, k, posK + 1u};
                held = true;
            }
            if (!ok) break;
            ++qu0;
        }
        pos += 2u * n;
    }
    if (ok) ok = is.issue_held(pend, held);
    if (!ok && is.issued_any) {
        is.commit(sm.bar(C::BAR_DRAIN));
        ptx::mbar_wait(sm.bar(C::BAR_DRAIN), 0, p.wait_limit_ns, nullptr);
    }
}

// ------------------------------------------------------------------ softmax
// Scores a row does not see become -inf in TMEM (tiles at a mask's border only,
// so that the common path carries no masks): it sees columns below lim, and not
// [sink, lo), a bit each of 32. (bf16 pools: 102 us, with two comparisons a column
// 111, for 32 ragged branches in windows of 2048. The 4-bit instances keep the
// comparisons: with bits their whole softmax loop spills, and a prefill step took
// 1528 us, not 1460.)
template <bool Q4>
__device__ __forceinline__ void mask_tile(uint32_t taddr, int lim, int lo, int sink) {
    uint32_t s[32];
#pragma unroll 1
    for (int c0 = 0; c0 < kBN; c0 += 32) {
        auto below = [c0](int n) { return n <= c0 ? 0u : ~0u >> (32 - min(n - c0, 32)); };
        const uint32_t see = below(lim) & (below(sink) | ~below(lo));
        __syncwarp();
        ptx::tmem_ld32(taddr + c0, s);
        ptx::tmem_ld_wait(s);
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (Q4 ? c0 + c >= lim || (c0 + c < lo && c0 + c >= sink) : (see >> c & 1u) == 0)
                s[c] = __float_as_uint(-INFINITY);
        ptx::tmem_st32(taddr + c0, s);
    }
    ptx::tmem_st_wait();
}

// mask_tile for a row of a drafted tree: columns below `last` that are keys before the
// branch's drafted tokens (below ub) and inside the window or among the first keys (as
// in mask_tile), or drafted tokens that the row's mask names, or the row's own (at
// `self`). Drafted token u is column ub + u, so 32 columns are 32 bits of the mask from
// bit c0 - ub on.
__device__ __forceinline__ void mask_tree_tile(uint32_t taddr, int last, int lo, int sink, int ub,
                                               int self, const uint32_t* mask, int words) {
    uint32_t s[32];
#pragma unroll 1
    for (int c0 = 0; c0 < kBN; c0 += 32) {
        auto below = [c0](int n) { return n <= c0 ? 0u : ~0u >> (32 - min(n - c0, 32)); };
        uint32_t see = below(ub) & (below(sink) | ~below(lo));
        if (ub < c0 + 32) {  // (a lane without a row has no mask)
            const int bit = c0 - ub, w = bit >> 5;
            const uint32_t a = mask && w >= 0 && w < words ? mask[w] : 0u;
            const uint32_t b = mask && w >= -1 && w + 1 < words ? mask[w + 1] : 0u;
            uint32_t bits = __funnelshift_r(a, b, bit & 31);
            if (self >= c0 && self < c0 + 32) bits |= 1u << (self - c0);
            see |= bits & ~below(ub);
        }
        see &= below(last);
        __syncwarp();
        ptx::tmem_ld32(taddr + c0, s);
        ptx::tmem_ld_wait(s);
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if ((see >> c & 1u) == 0) s[c] = __float_as_uint(-INFINITY);
        ptx::tmem_st32(taddr + c0, s);
    }
    ptx::tmem_st_wait();
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32], float m) {
    float a[4] = {m, __uint_as_float(s[1]), __uint_as_float(s[2]), __uint_as_float(s[3])};
#pragma unroll
    for (int c = 0; c < 32; c += 2)
        a[(c >> 1) & 3] = ptx::fmax3(a[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    return fmaxf(ptx::fmax3(a[0], a[1], a[2]), a[3]);
}

// P of 32 columns to TMEM (16 columns of 16-bit pairs; bf16 as V for bf16 pools: half
// a step is 2^-8 of each p), their sum, of the unrounded values, added to l.
template <bool kF16>
__device__ __forceinline__ void exp32(const uint32_t (&s)[32], uint32_t taddr, uint64_t sl2,
                                      uint64_t negm, uint64_t (&l)[2]) {
    uint32_t packed[16];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const uint64_t t = ptx::fma_f32x2(
            ptx::f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2, negm);
        const float e0 = ptx::ex2(ptx::lo_f32(t)), e1 = ptx::ex2(ptx::hi_f32(t));
        l[(c >> 1) & 1] = ptx::add_f32x2(l[(c >> 1) & 1], ptx::f32x2(e0, e1));
        packed[c >> 1] = kF16 ? ptx::pack_f16x2(e0, e1) : ptx::pack_bf16x2(e0, e1);
    }
    ptx::tmem_st16(taddr, packed);
}
// The running reference and sum of a row.
struct Running {
    float m = -INFINITY, l = 0.f;
    // A tile's maximum: the factor that O and l take, and the exponent's addend.
    __device__ __forceinline__ float raise(float mx, float lift, float& neg) {
        float corr = 1.f;
        if (mx > m + kRescaleLog2) {
            corr = (m == -INFINITY) ? 0.f : ptx::ex2(m - mx);
            m = mx;
        }
        neg = lift - ((m == -INFINITY) ? 0.f : m);
        return corr;
    }
};

// O's 128 columns times corr, in place.
__device__ __forceinline__ void rescale(uint32_t colO, float corr, uint32_t (&r)[32]) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        __syncwarp();
        ptx::tmem_ld32(colO + 32 * c, r);
        ptx::tmem_ld_wait(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr);
        ptx::tmem_st32(colO + 32 * c, r);
    }
}

// One tile's softmax of this thread's row: P over the first 64 columns of S; `half` runs
// once O is rescaled (where `held`: it holds products) and P's first half is written: the
// product over it need not wait for the rest of the exponentials. (One pass with the
// reference of the tiles before, starting over when it must be raised, was slower: a
// prefill 1661 us against 1583.)
template <bool kF16, typename Half>
__device__ __forceinline__ void softmax_tile(uint32_t colS, uint32_t colO, float sl2, bool held,
                                             bool row_valid, Running& run, Half half) {
    constexpr float kLift = Cfg<1, kF16 ? Pool::q4 : Pool::bf16>::kLiftLog2;
    const uint64_t sl2p = ptx::f32x2(sl2, sl2);
    uint64_t l[2] = {0ull, 0ull};
    uint32_t s0[32];
    float neg;
    // 32 columns at a time, the next ones on their way from TMEM while these are
    // worked on: the maximum from the last columns down, P from the first up
    uint32_t s1[32];
    ptx::tmem_ld32(colS + 96, s1);
    ptx::tmem_ld_wait(s1);
    ptx::tmem_ld32(colS + 64, s0);
    float mx = max32(s1, -INFINITY);
    ptx::tmem_ld_wait(s0);
    ptx::tmem_ld32(colS + 32, s1);
    mx = max32(s0, mx);
    ptx::tmem_ld_wait(s1);
    ptx::tmem_ld32(colS, s0);
    mx = max32(s1, mx);
    ptx::tmem_ld_wait(s0);
    ptx::tmem_ld32(colS + 32, s1);
    mx = max32(s0, mx);
    const float corr = run.raise(mx * sl2, kLift, neg);
    const uint64_t negm = ptx::f32x2(neg, neg);
    // O is rescaled in place: this S was issued after the group's previous product, so
    // that one has completed. (Of a lane without a row nothing is used.)
    if (held && __any_sync(0xffffffffu, row_valid && corr != 1.f)) {
        ptx::tmem_ld_wait(s1);
        rescale(colO, corr, s1);
        ptx::tmem_ld32(colS + 32, s1);
    }
    exp32<kF16>(s0, colS, sl2p, negm, l);
    ptx::tmem_ld_wait(s1);
    ptx::tmem_ld32(colS + 64, s0);
    exp32<kF16>(s1, colS + 16, sl2p, negm, l);
    half();
    ptx::tmem_ld_wait(s0);
    ptx::tmem_ld32(colS + 96, s1);
    exp32<kF16>(s0, colS + 32, sl2p, negm, l);
    ptx::tmem_ld_wait(s1);
    exp32<kF16>(s1, colS + 48, sl2p, negm, l);
    const uint64_t sum = ptx::add_f32x2(l[0], l[1]);
    run.l = run.l * corr + (ptx::lo_f32(sum) + ptx::hi_f32(sum));
}

// 32 columns of a finished row to out (direct) or to its partial block; from 4-bit
// pools put back into their order first (each 8 hold values 0 2 4 6 1 3 5 7). A
// store is a line of its own for every lane, so 32 bytes at once take half as long
// as 16 (an output that is aligned to 16 bytes only gets those).
template <bool Q4>
__device__ __forceinline__ void store32(void* out, float* part_o, int out_bf16,
                                        const uint32_t (&r)[32], bool direct, int64_t orow,
                                        int64_t prow, int c0) {
    auto at = [](int d) { return Q4 ? (d & ~7) + (d & 1) * 4 + ((d & 7) >> 1) : d; };
    auto put = [direct](void* dst, const uint32_t* v) {
        if (!direct || (reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
            ptx::st_global_v8(dst, v);
        } else {
            static_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
            static_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
    };
    uint32_t v[8];
    if (direct && out_bf16) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out) + orow * kHD + c0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int h = 0; h < 8; ++h)
                v[h] = ptx::pack_bf16x2(__uint_as_float(r[at(16 * i + 2 * h)]),
                                        __uint_as_float(r[at(16 * i + 2 * h + 1)]));
            put(dst + 16 * i, v);
        }
    } else {
        float* dst = (direct ? static_cast<float*>(out) + orow * kHD : part_o + prow * kHD) + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int h = 0; h < 8; ++h) v[h] = r[at(8 * i + h)];
            put(dst + 8 * i, v);
        }
    }
}

// Group x: thread i owns row i of the group's query tile (TMEM lane i).
template <int NQ, Pool F, bool Tree>
__device__ void softmax_group(const RowParams& p, const Smem<NQ, F>& sm, uint32_t tmem, int x) {
    using C = Cfg<NQ, F>;
    const int lane = threadIdx.x & 31;
    const int quarter = (threadIdx.x >> 5) & 3;  // TMEM lane quarter this warp may access
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t colS = lane_addr + 128u * x, colO = lane_addr + kColO + 128u * x;
    uint32_t n_load[2] = {0, 0};  // loads of each Q buffer before this unit
    uint32_t jt = 0;                // tiles this group got
    uint32_t ku = 0, ku_other = 0;  // units in which this group and the other got tiles
    uint32_t tile0 = 0;  // K/V tiles before this unit
    int kj = 0;  // joined (one-query-tile) units so far
    // Before the first unit each group makes a dry run of that unit's epilogue (no
    // tiles, no waits, one thread's stores into a scratch sink) while it waits for
    // its first tile anyway: fetched cold, from behind the other CTAs' reads, that
    // code took 2 us of a decode step.
    const int ui_first = p.cta_first[blockIdx.x], ui_end = p.cta_first[blockIdx.x + 1];
    for (int ui = ui_first < ui_end ? ui_first - 1 : ui_first; ui < ui_end; ++ui) {
        const bool dry = ui < ui_first;
        const Unit u = p.units[dry ? ui_first : ui];
        const Tiles tl(p, u);
        const bool pair = unit_nq<NQ>(u, p.tpt) == 2;
        const int tile_tok = pair ? x * p.tpt : 0;
        const bool row_valid = dry ? row == 0 : row < min(p.tpt, u.n_tok - tile_tok) * p.G;
        const bool active = dry || __any_sync(0xffffffffu, row_valid);
        const int tok = u.tok_begin + tile_tok + row / p.G;
        // one past the last key that the row sees (trees: past the keys before its branch's
        // drafted tokens), and one past its position (see the window below)
        const int row_end = row_valid ? p.tok_pos[tok] + (Tree ? 0 : 1) : 0;
        // (a drafted token's position is at most a tree's depth past the keys before it)
        int row_pos1 = row_end + (Tree ? 1 : 0);
        if (Tree && row_valid && p.positions)
            row_pos1 = min(max(p.positions[tok], row_end), row_end + kMaxTreeTokens - 1) + 1;
        const int self = Tree && row_valid ? p.tok_pos[p.R + tok] : 0;
        const uint32_t* const mask =
            Tree && row_valid ? p.masks + static_cast<int64_t>(tok) * p.mask_words : nullptr;
        const int n_tiles = dry ? 0 : tl.n;
        const int j0 = pair ? 0 : (x ^ tile0) & 1, dj = pair ? 1 : 2;
        Running run;
        // the softmax scale, with the power of two that the row of Q carries
        const int xq = pair ? x : 0;
        const uint32_t load = xq == 0 ? n_load[0] : n_load[1];
        if (!dry) {
            ++n_load[0];
            if (pair) ++n_load[1];
        }
        float sl2 = p.scale_log2;
        for (int j = j0; j < n_tiles; j += dj, ++jt) {
            int kt, last, front;
            tl.tile(j, kt, last, front);
            const bool f = j < tl.n_first;
            // (a run of first keys before the range leaves none of them to it)
            const int lim = min(row_end, last) - kt, lo = row_pos1 - p.window - kt;
            const int sink = f || tl.n_first == 0 ? p.sinks - kt : 0;
            // (a lane without a row needs no mask: what it computes stays in its lane)
            const bool full = __all_sync(
                0xffffffffu, !row_valid || (lim >= kBN && (lo <= 0 || sink >= kBN)));
            if (!warp_wait<NQ, F>(p, sm, sm.gbar(x, SFULL), jt & 1u, 20)) return;
            ptx::tc_fence_after();
            // The factor was written before the S product was issued. (Waiting for
            // QREADY here would be wrong: a group without a tile in a unit may find
            // that barrier two phases on.)
            if (C::kF16 && j == j0 && row_valid) {
                const int k = static_cast<int>(*sm.fac(load, xq, row)) - 127;
                // Finite, so that a key of zeros scores 0 with the largest Q too, and
                // not 0, so that a hidden key's -inf stays one (0 * -inf is a NaN) with the
                // smallest: a score is at most 2^34, so 1.2e-38 gives what less would, 0.
                sl2 = fmaxf(fminf(sl2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23), 3e38f),
                            1.2e-38f);
            }
            auto half = [&]() {
                if (!C::kEarlyP) return;
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.gbar(x, PHALF));
            };
            if (active) {
                if constexpr (Tree) {
                    if (!full)
                        mask_tree_tile(colS, last - kt, lo, sink, row_end - kt, self - kt, mask,
                                       p.mask_words);
                } else {
                    if (!full) mask_tile<C::kQ4>(colS, lim, lo, sink);
                }
                softmax_tile<C::kF16>(colS, colO, sl2, j > j0, row_valid, run, half);
            } else {
                half();
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.gbar(x, PFULL));
        }
        const float m_ref = run.m, l_run = run.l * C::kUnlift;  // without P's lift
        const bool direct = u.part < 0;
        const int64_t orow =
            dry ? 0 : static_cast<int64_t>(tok) * p.H_q + u.kv_head * p.G + row % p.G;
        const int64_t prow =
            dry ? 0 : static_cast<int64_t>(u.part) * (kBM * NQ) + (pair ? kBM * x : 0) + row;
        void* const out = dry ? static_cast<void*>(p.sink) : p.out;
        float* const part_o = dry ? p.sink : p.part_o;
        float m_out = m_ref, l_out = l_run, wa = 1.f, wb = 0.f;
        float2* const join = reinterpret_cast<float2*>(sm.ptr + C::kSmemJoin) + (kj & 1) * 2 * kBM;
        const int n_other = pair ? 0 : (n_tiles + j0) >> 1;  // tiles of the other parity
        if (pair) {
            if (!dry) ++ku_other;
        } else if (!dry) {
            // Join the groups: exchange (m, l), then each combines 64 columns.
            join[x * kBM + row] = make_float2(m_ref, l_run);
            __syncwarp();
            // two barriers in turn: a group without a tile in the next unit may
            // arrive there before this one has waited here
            if (lane == 0) ptx::mbar_arrive(sm.gbar(x, JOIN + (kj & 1)));
            if (n_other > 0) ++ku_other;
            if (!warp_wait<NQ, F>(p, sm, sm.gbar(x ^ 1, JOIN + (kj & 1)), (kj >> 1) & 1, 23)) return;
            ++kj;
        }
        if (n_tiles > n_other && !warp_wait<NQ, F>(p, sm, sm.gbar(x, ODONE), ku++ & 1u, 22)) return;
        if (n_other > 0 && !warp_wait<NQ, F>(p, sm, sm.gbar(x ^ 1, ODONE), (ku_other - 1) & 1u, 24))
            return;
        ptx::tc_fence_after();
        if (active) {
            if (!pair) {
                const float2 other = join[(x ^ 1) * kBM + row];
                const float m_a = l_run > 0.f ? m_ref : -INFINITY;
                const float m_b = other.y > 0.f ? other.x : -INFINITY;
                m_out = fmaxf(m_a, m_b);
                wa = m_a == -INFINITY ? 0.f : ptx::ex2(m_a - m_out);
                wb = m_b == -INFINITY ? 0.f : ptx::ex2(m_b - m_out);
                l_out = wa * l_run + wb * other.y;
            }
            const float w = p.o_scale * C::kUnlift * (direct ? (l_out > 0.f ? 1.f / l_out : 0.f) : 1.f);
            wa *= w;
            wb *= w;
            const uint32_t oa = lane_addr + kColO + 128u * x, ob = lane_addr + kColO + 128u * (x ^ 1);
            const int c_end = pair ? kHD : 64 * x + 64;
#pragma unroll 1
            for (int c = pair ? 0 : 64 * x; c < c_end; c += 32) {
                uint32_t r[32], b[32];
                __syncwarp();
                ptx::tmem_ld32(oa + c, r);
                if (!pair) ptx::tmem_ld32(ob + c, b);
                ptx::tmem_ld_wait(r);
                ptx::reg_touch(b);
                // a group without a visible key may never have written its O
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    r[i] = __float_as_uint((wa != 0.f ? wa * __uint_as_float(r[i]) : 0.f) +
                                           (wb != 0.f ? wb * __uint_as_float(b[i]) : 0.f));
                if (row_valid) store32<C::kQ4>(out, part_o, p.out_bf16, r, direct, orow, prow, c);
            }
        }
        if (row_valid && (pair || x == 0)) {
            float2* const ml = dry ? reinterpret_cast<float2*>(p.sink) : p.part_ml;
            float* const lse = dry ? p.sink : p.lse;
            if (!direct) ml[prow] = make_float2(m_out, l_out);
            else if (lse) lse[orow] = (m_out + __log2f(l_out)) * 0.69314718055994531f;
        }
        ptx::tc_fence_before();
        __syncwarp();
        tile0 += n_tiles;
        if (lane == 0 && !dry) ptx::mbar_arrive(sm.bar(C::BAR_OFREE));
    }
}

template <int NQ, Pool F, bool Tree>
__global__ void __launch_bounds__(Cfg<NQ, F>::kThreads, 1)
    attn_rows_kernel(const __grid_constant__ RowParams p, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
    using C = Cfg<NQ, F>;
    // 1024-byte aligned as declared, so that every shared-memory address is a constant
    // (checked below).
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<NQ, F> sm;
    sm.base = ptx::smem_u32(smem_raw);
    sm.ptr = smem_raw;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            // (widened by a group of warps, or loaded)
            ptx::mbar_init(sm.bar(C::BAR_FULL + s),
                           C::kQ4 || (C::kQ8 && s >= C::kKStages) ? kGroupWarps : 1);
            ptx::mbar_init(sm.bar(C::BAR_EMPTY + s), 1);
        }
        for (int s = 0; s < C::kRaw; ++s) {
            ptx::mbar_init(sm.bar(C::BAR_RFULL + s), 1);
            ptx::mbar_init(sm.bar(C::BAR_REMPTY + s), kGroupWarps);
        }
        for (int x = 0; x < NQ; ++x) {
            ptx::mbar_init(sm.bar(C::BAR_QFULL + x), 1);
            ptx::mbar_init(sm.bar(C::BAR_QFREE + x), 1);
            ptx::mbar_init(sm.bar(C::BAR_QREADY + x), kGroupWarps);
        }
        ptx::mbar_init(sm.bar(C::BAR_OFREE), 2 * kGroupWarps);
        ptx::mbar_init(sm.bar(C::BAR_AUX), 1);
        ptx::mbar_init(sm.bar(C::BAR_DRAIN), 1);
        for (int x = 0; x < 2; ++x) {
            ptx::mbar_init(sm.gbar(x, SFULL), 1);
            ptx::mbar_init(sm.gbar(x, PHALF), kGroupWarps);
            ptx::mbar_init(sm.gbar(x, PFULL), kGroupWarps);
            ptx::mbar_init(sm.gbar(x, ODONE), 1);
            ptx::mbar_init(sm.gbar(x, JOIN), kGroupWarps);
            ptx::mbar_init(sm.gbar(x, JOIN + 1), kGroupWarps);
        }
        *sm.abort_flag() = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        if (!C::kQ4) ptx::prefetch_tmap(&tm_k);
        if (!C::kQ4) ptx::prefetch_tmap(&tm_v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(sm.tmem_slot()), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot();
    wait_for_previous();  // up to here nothing of global memory was touched

    if (C::kF16 && warp < kWarpSoftmax) ptx::regs_dec<C::kRegsOther>();
    if (tmem != 0 || (sm.base & 1023u) != 0) {
        // the issuer counts on both; a CTA that gets all TMEM columns gets them from 0
        if (threadIdx.x == 0) atomicCAS(p.err, 0, kErrCuda);
    } else if (warp == 0) {
        producer_warp<NQ, F>(p, sm, &tm_q, &tm_k, &tm_v);
    } else if (warp == 3) {
        mma_warp<NQ, F>(p, sm);
        __syncwarp();
    } else if (warp < kWarpSoftmax) {
        // (only there to make a warpgroup)
    } else if (warp < kWarpWiden) {
        if (C::kF16) ptx::regs_inc<C::kRegsSoftmax>();
        softmax_group<NQ, F, Tree>(p, sm, tmem, (warp - kWarpSoftmax) / kGroupWarps);
    } else {
        if constexpr (C::kF16) ptx::regs_dec<C::kRegsWiden>();
        if constexpr (C::kQ8) {
            widen_warp_e4m3<NQ>(p, sm, warp - kWarpWiden);
        } else if constexpr (C::kQ4) {
            widen_warp<NQ>(p, sm, (warp - kWarpWiden) & 3, warp >= kWarpWiden + kGroupWarps);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    // A role that gave up drained what it had in flight itself, as far as it could; one that
    // had ended before it could not. Copies and products take microseconds to land.
    if (*sm.abort_flag() != 0)
        for (const uint64_t t0 = ptx::globaltimer_ns(); ptx::globaltimer_ns() - t0 < kLingerNs;) {}
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    if (threadIdx.x == 0 && *sm.abort_flag() != 0 && atomicCAS(p.err, 0, kErrTimeout) == 0) {
        p.err[1] = *sm.abort_flag();
        p.err[2] = static_cast<int32_t>(blockIdx.x);
    }
}

template <int NQ, Pool F, bool Tree>
cudaError_t launch_nq(const RowParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                      const CUtensorMap& tm_v, int grid, cudaStream_t stream) {
    // The shared-memory attribute is set once per device (see attn_fwd.cu).
    static std::atomic<bool> attr_set[64];
    static std::mutex attr_mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 64;
    if (!known || !attr_set[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lk(attr_mu);
        if (!known || !attr_set[dev].load(std::memory_order_relaxed)) {
            e = cudaFuncSetAttribute(attn_rows_kernel<NQ, F, Tree>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Cfg<NQ, F>::kSmemAlloc);
            if (e != cudaSuccess) return e;
            if (Cfg<NQ, F>::kF16) {
                // The split asks for what the block was launched with: with fewer registers
                // than it counts on, the softmax warps would wait for more without an end.
                cudaFuncAttributes fa;
                e = cudaFuncGetAttributes(&fa, attn_rows_kernel<NQ, F, Tree>);
                if (e != cudaSuccess) return e;
                if (fa.numRegs < Cfg<NQ, F>::kRegsLaunch) return cudaErrorInvalidConfiguration;
            }
            if (known) attr_set[dev].store(true, std::memory_order_release);
        }
    }
    return launch_after(attn_rows_kernel<NQ, F, Tree>, grid, Cfg<NQ, F>::kThreads, Cfg<NQ, F>::kSmemAlloc,
                        stream, p, tm_q, tm_k, tm_v);
}

}  // namespace
}  // namespace fanout

// pair.cuh - the pieces that every pair kernel shares: shared-memory layout,
// barrier set-up and teardown, operand descriptors, store boxes, and the wide
// tiles' producer step and staggered MMA issue.  kernels.cuh describes the roles,
// barriers and tiles.
#pragma once
#include <cstdint>
#include <cuda.h>
#include "ptx.cuh"

namespace flp {

constexpr int BM = 128;           // rows of A per CTA (TMEM lanes)
constexpr int PM = 256;           // rows of the pair tile (UMMA M)
constexpr int BN = 256;           // columns of the pair tile (UMMA N)
constexpr int BNH = BN / 2;       // rows of B held by each CTA of the pair
constexpr int BK = 64;            // K per pipeline stage (one 128-byte swizzle atom)
constexpr int UMMA_K = 16;        // K per tcgen05.mma (bf16)
constexpr int STAGES = 6;
constexpr int NUM_THREADS = 192;
constexpr int EPI_THREADS = 128;
constexpr int WIDE_THREADS = 64 + 2 * EPI_THREADS;  // wide-tile kernels (forward, dZ, dX + dW): two epilogue groups of four warps
constexpr uint32_t TMEM_COLS = 512;
constexpr uint16_t PAIR_MASK = 0x3;

constexpr uint32_t A_STAGE_BYTES = BM * BK * 2;    // 16 KiB
constexpr uint32_t B_STAGE_BYTES = BNH * BK * 2;   // 16 KiB
constexpr uint32_t PAIR_STAGE_TX = 2 * (A_STAGE_BYTES + B_STAGE_BYTES);  // lands on the leader's barrier
constexpr uint32_t STG_BYTES = 128 * 128;          // one 128-row x 128-byte store box
constexpr uint32_t NUM_STG = 2;
constexpr int SCHED_SLOTS = 4;

constexpr int ERR_BAD_TARGET = 1;
constexpr int ERR_TIMEOUT = 2;

// Offsets inside the (1024-byte aligned) dynamic shared memory block; the
// layout is identical in both CTAs of a pair, which the pair MMA relies on.
constexpr uint32_t SMEM_A = 0;
constexpr uint32_t SMEM_B = SMEM_A + STAGES * A_STAGE_BYTES;
constexpr uint32_t SMEM_STG = SMEM_B + STAGES * B_STAGE_BYTES;
constexpr uint32_t SMEM_BAR = SMEM_STG + NUM_STG * STG_BYTES;
// full[STAGES], empty[STAGES], tfull[2], tempty[2], drain, sched_full[4], sched_empty[4]
constexpr uint32_t NUM_BARS = 2 * STAGES + 4 + 1 + 2 * SCHED_SLOTS;
constexpr uint32_t SMEM_MISC = SMEM_BAR + NUM_BARS * 8;  // tmem slot, abort flag, sched slots
constexpr uint32_t SMEM_TOTAL = SMEM_MISC + 8 + 4 * SCHED_SLOTS;
constexpr uint32_t SMEM_ALLOC = SMEM_TOTAL + 1024;  // slack for 1024-byte alignment

// Shared-memory slots.  Normal tiles: STAGES slots of 16 KiB of A and 16 KiB
// of B (A slots first, then B slots).  Wide tiles (the forward's, and dX tiles
// of the backward): STAGES_W slots of 48 KiB (A, then the B halves of the two
// 256-column sub-tiles), over the same bytes.
constexpr int STAGES_W = 4;
constexpr uint32_t STAGE_W_BYTES = A_STAGE_BYTES + 2 * B_STAGE_BYTES;
constexpr uint32_t PAIR_STAGE_TX_W = 2 * STAGE_W_BYTES;
static_assert(STAGES_W * STAGE_W_BYTES <= SMEM_STG, "wide slots must fit the pipeline region");

__device__ __forceinline__ uint32_t slot_a(bool wide, int s) {
    return wide ? s * STAGE_W_BYTES : SMEM_A + s * A_STAGE_BYTES;
}
__device__ __forceinline__ uint32_t slot_b(bool wide, int s) {
    return wide ? s * STAGE_W_BYTES + A_STAGE_BYTES : SMEM_B + s * B_STAGE_BYTES;
}

struct Smem {
    uint8_t* base;
    uint64_t* full;
    uint64_t* empty;
    uint64_t* tfull;
    uint64_t* tempty;
    uint64_t* drain;
    uint64_t* sched_full;
    uint64_t* sched_empty;
    uint32_t* tmem_slot;
    volatile int* abort_flag;
    volatile int* sched_val;
};

__device__ __forceinline__ Smem smem_layout(uint8_t* raw) {
    Smem s;
    s.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                        ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(s.base + SMEM_BAR);
    s.full = bars;
    s.empty = bars + STAGES;
    s.tfull = bars + 2 * STAGES;
    s.tempty = bars + 2 * STAGES + 2;
    s.drain = bars + 2 * STAGES + 4;
    s.sched_full = bars + 2 * STAGES + 5;
    s.sched_empty = s.sched_full + SCHED_SLOTS;
    s.tmem_slot = reinterpret_cast<uint32_t*>(s.base + SMEM_MISC);
    s.abort_flag = reinterpret_cast<volatile int*>(s.base + SMEM_MISC + 4);
    s.sched_val = reinterpret_cast<volatile int*>(s.base + SMEM_MISC + 8);
    return s;
}

// Records a timeout in the error word and tells both CTAs of the pair to stop
// waiting (the peer's flag is written through the cluster window).
__device__ __forceinline__ void raise_abort(const Smem& sm, int* err) {
    atomicOr(err, ERR_TIMEOUT);
    *sm.abort_flag = 1;
    const uint32_t peer = cluster_ctarank() ^ 1u;
    st_shared_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(sm.abort_flag)), peer), 1u);
}

// Barrier set-up, TMEM allocation on both CTAs, and the cluster handshake that
// makes the peer's barriers visible before any remote arrive or TMA signal.
// sched_arrivals: arrivals that free a slot of the unit hand-off ring (the
// peer's producer, the MMA issuer and every epilogue thread of both CTAs).
// drain_arrivals: threads of both CTAs that drain an accumulator.
__device__ __forceinline__ uint32_t pair_prologue(const Smem& sm, int warp,
                                                  uint32_t sched_arrivals = 2 + 2 * EPI_THREADS,
                                                  uint32_t drain_arrivals = 2 * EPI_THREADS) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sm.tfull[a], 1);
            mbar_init(&sm.tempty[a], drain_arrivals);
        }
        mbar_init(sm.drain, 1);
        for (int s = 0; s < SCHED_SLOTS; ++s) {
            mbar_init(&sm.sched_full[s], 1);
            mbar_init(&sm.sched_empty[s], sched_arrivals);
        }
        *sm.abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(sm.tmem_slot, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    return *sm.tmem_slot;
}

// Teardown: on an abort give copies in flight a bounded grace period, then a
// cluster handshake (no CTA leaves while its peer may still touch its shared
// memory or TMEM) and the pair TMEM release.
__device__ __forceinline__ void pair_epilogue(const Smem& sm, int warp, uint32_t tmem_base) {
    if (*sm.abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// Operand descriptors for UMMA step k (0..3) inside a 64-deep stage.
template <int kMN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int k) {
    if constexpr (kMN == 0)
        return sdesc_sw128(base + k * (UMMA_K * 2), 16, 1024);  // K-major: 32 B inside the atom
    else
        return sdesc_sw128(base + k * (UMMA_K * 128), 8192, 1024);  // MN-major: 16 rows of 128 B
}

// ------------------------------------------------------------ epilogue pieces

// v[idx] for a thread-dependent idx in [0, 32) through a 5-level select tree,
// so the 32 values stay in registers (no dynamically indexed local array).
__device__ __forceinline__ float select32(const uint32_t (&v)[32], int idx) {
    uint32_t a[16], b[8], c[4], d[2];
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] = (idx & 16) ? v[j + 16] : v[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = (idx & 8) ? a[j + 8] : a[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = (idx & 4) ? b[j + 4] : b[j];
#pragma unroll
    for (int j = 0; j < 2; ++j) d[j] = (idx & 2) ? c[j + 2] : c[j];
    return __uint_as_float((idx & 1) ? d[1] : d[0]);
}

// Write 8 x 16-byte chunks of one row into a 128B-swizzled 128-row box.
__device__ __forceinline__ void stage_row(uint32_t box_base, int r, const uint32_t (&w)[32]) {
    const uint32_t row_addr = box_base + r * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        st_shared_v4(row_addr + ((c ^ (r & 7)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                     w[4 * c + 3]);
}

// Two store boxes used in turn: before a box is rewritten, the bulk store
// that last read it must have finished reading.
struct StoreRing {
    uint32_t n = 0;
};

__device__ __forceinline__ uint32_t store_box_acquire(StoreRing& ring, uint8_t* smem, int et) {
    const uint32_t buf = ring.n & 1u;
    if (ring.n >= NUM_STG) {
        if (et == 0) bulk_wait_group_read<NUM_STG - 1>();
        named_bar_sync(1, EPI_THREADS);
    }
    return smem_addr(smem + SMEM_STG + buf * STG_BYTES);
}

__device__ __forceinline__ void store_box_release(StoreRing& ring, uint8_t* smem, int et,
                                                  const CUtensorMap* tmOut, int x, int y, bool add) {
    const uint32_t buf = ring.n & 1u;
    fence_proxy_async_smem();
    named_bar_sync(1, EPI_THREADS);
    if (et == 0) {
        const void* src = smem + SMEM_STG + buf * STG_BYTES;
        if (add)
            tma_reduce_add_2d(tmOut, src, x, y);
        else
            tma_store_2d(tmOut, src, x, y);
        bulk_commit_group();
    }
    ring.n++;
}

// Narrow store boxes: 128 rows x 64 bytes (32 bf16 or 16 fp32 columns,
// 64-byte swizzle), two per epilogue group, so that two groups fit the store
// region.  One box of this thread's row (16 words) is staged and stored (or
// added) in its group's ring, with one named barrier per box: before it,
// thread 0 of the group waits until every earlier bulk store has finished
// reading, so after it the other box (read by the previous store) may be
// rewritten by the next call while this box's store runs.
constexpr uint32_t NBOX_BYTES = BM * 64;
static_assert(2 * 2 * NBOX_BYTES <= NUM_STG * STG_BYTES, "two narrow boxes per epilogue group");

__device__ __forceinline__ void narrow_box_store(StoreRing& ring, uint8_t* box0, uint32_t bar_id, int et, int r,
                                                 const uint32_t* w, const CUtensorMap* out, int x, int y,
                                                 bool add) {
    const uint32_t buf = ring.n & 1u;
    // box buf was last read by the store two boxes back, which thread 0
    // waited for before the previous call's barrier
    uint8_t* box = box0 + buf * NBOX_BYTES;
    const uint32_t row_addr = smem_addr(box) + r * 64;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        st_shared_v4(row_addr + ((c ^ ((r >> 1) & 3)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    fence_proxy_async_smem();
    if (et == 0) bulk_wait_group_read<0>();  // the other box is free again after the barrier
    named_bar_sync(bar_id, EPI_THREADS);
    if (et == 0) {
        if (add)
            tma_reduce_add_2d(out, box, x, y);
        else
            tma_store_2d(out, box, x, y);
        bulk_commit_group();
    }
    ring.n++;
}

// fp32 accumulator columns [c0, c0 + 64) of this thread's row -> 32 packed bf16 pairs.
__device__ __forceinline__ void tmem_row64_to_bf16(uint32_t taddr, uint32_t (&w)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + h * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[h * 16 + j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
    }
}

// ------------------------------------------------------ wide (256 x 512) tiles

// k-blocks issued half by half at each end of a wide tile (at most the number
// of wide slots: those k-blocks' stages stay held until both halves ran)
constexpr int WIDE_EDGE = STAGES_W;

// Producer: one 64-deep k-block of a wide tile whose operands are both K-major
// into wide slot `stage`: this CTA's 128 rows of A (from row a_row) and its
// 128-row halves of the two 256-row B sub-tiles (from rows b_row, b_row + 256).
__device__ __forceinline__ void load_wide_kblock(const Smem& sm, int stage, bool leader,
                                                 const CUtensorMap* tmA, int a_row,
                                                 const CUtensorMap* tmB, int b_row, int kb) {
    if (leader) mbar_arrive_expect_tx(&sm.full[stage], PAIR_STAGE_TX_W);
    const uint32_t bar = mapa_shared(smem_addr(&sm.full[stage]), 0);
    tma_load_2d_pair(sm.base + slot_a(true, stage), tmA, kb * BK, a_row, bar);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        tma_load_2d_pair(sm.base + slot_b(true, stage) + h * B_STAGE_BYTES, tmB, kb * BK, b_row + h * BN, bar);
}

// MMA issuer: every MMA of one wide tile with K-major A and K-major or (B_MN)
// MN-major B (KB k-blocks), half h into accumulator h, then tfull[h] per half.
// `gk` counts the k-blocks consumed so far (slot gk % STAGES_W, fill parity
// (gk / STAGES_W) & 1) and advances by KB; phase0 and phase1 are this tile's
// use parities of the accumulators.  The first and last WIDE_EDGE k-blocks are
// issued half by half: at the end of the tile half 0 completes (and its
// epilogue starts) while the half-1 MMAs of those k-blocks still run, and at
// the start half 0 fills while the previous tile's half 1 is still drained.
// Returns false when a wait ran out.
template <int B_MN = 0>
__device__ __forceinline__ bool wide_tile_mma(const Smem& sm, uint32_t tmem_base, uint32_t& gk,
                                              uint32_t phase0, uint32_t phase1, int KB, uint64_t limit,
                                              volatile int* abort_flag) {
    constexpr uint32_t idesc = idesc_bf16_f32(PM, BN, 0, B_MN);
    auto issue = [&](uint32_t g, int h, int kb) {
        const int s = static_cast<int>(g % STAGES_W);
        const uint32_t a_base = smem_addr(sm.base + slot_a(true, s));
        const uint32_t b_base = smem_addr(sm.base + slot_b(true, s)) + h * B_STAGE_BYTES;
#pragma unroll
        for (int k = 0; k < BK / UMMA_K; ++k)
            umma_bf16_pair(tmem_base + static_cast<uint32_t>(h * BN), operand_desc<0>(a_base, k),
                           operand_desc<B_MN>(b_base, k), idesc, (kb > 0 || k > 0) ? 1u : 0u);
    };
    auto wait_full = [&](uint32_t g) {
        if (!mbar_wait(&sm.full[g % STAGES_W], (g / STAGES_W) & 1u, limit, abort_flag)) return false;
        tc_fence_after();
        return true;
    };
    auto release = [&](uint32_t g) {
        umma_commit_pair_mc(&sm.empty[g % STAGES_W], PAIR_MASK);  // stage free in both CTAs
    };
    const int head = min(WIDE_EDGE, KB);
    const int tail0 = max(head, KB - WIDE_EDGE);
    if (!mbar_wait(&sm.tempty[0], phase0 ^ 1u, limit, abort_flag)) return false;
    tc_fence_after();
    for (int kb = 0; kb < head; ++kb) {
        if (!wait_full(gk + kb)) return false;
        issue(gk + kb, 0, kb);
    }
    if (head == KB) umma_commit_pair_mc(&sm.tfull[0], PAIR_MASK);
    if (!mbar_wait(&sm.tempty[1], phase1 ^ 1u, limit, abort_flag)) return false;
    tc_fence_after();
    for (int kb = 0; kb < head; ++kb) {
        issue(gk + kb, 1, kb);
        release(gk + kb);
    }
    for (int kb = head; kb < tail0; ++kb) {
        if (!wait_full(gk + kb)) return false;
        issue(gk + kb, 0, kb);
        issue(gk + kb, 1, kb);
        release(gk + kb);
    }
    for (int kb = tail0; kb < KB; ++kb) {
        if (!wait_full(gk + kb)) return false;
        issue(gk + kb, 0, kb);
    }
    if (head < KB) umma_commit_pair_mc(&sm.tfull[0], PAIR_MASK);  // half 0 ready in both CTAs
    for (int kb = tail0; kb < KB; ++kb) {
        issue(gk + kb, 1, kb);
        release(gk + kb);
    }
    umma_commit_pair_mc(&sm.tfull[1], PAIR_MASK);  // half 1 ready in both CTAs
    gk += static_cast<uint32_t>(KB);
    return true;
}

}  // namespace flp

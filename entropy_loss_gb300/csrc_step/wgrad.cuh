// wgrad.cuh - the weight gradient of a linear layer whose input was kept as an
// 8-bit checkpoint:  dW[N, K] (+)= dY[M, N]^T X^[M, K].
//
// A checkpoint's values are exact in bf16, so X^ is unpacked once into the
// workspace and the contraction runs on CTA pairs like the head's dW tiles:
// both operands MN-major, 256 x 512 tiles in both TMEM accumulators, four
// 48 KiB slots fed by TMA, the halves staggered at the tile ends, one epilogue
// group per accumulator.  (Unpacking inside this kernel would add 48 KiB of
// shared-memory traffic to the 112 KiB that a 64-deep K step of a tile already
// moves in its 1024 tensor-pipe cycles at 128 bytes a cycle, and every 256
// rows of dW would convert X^ again; the separate pass is a few percent of
// the contraction.)
//
// Whole rounds of tiles over the resident pairs write dW directly.  The tiles
// of the last, incomplete round would leave most pairs idle for a whole tile,
// so their rows of dY and X^ are split into S runs that go to separate fp32
// partial tiles, which a small kernel joins in a fixed order (no atomics).
//
// Bound by the tensor cores: 8192 x 8192 x 5120 (dY rows, dW rows, dW columns) with an
// fp32 dW takes 410 us, 1680 TFLOP/s or 89 % of the measured matrix rate: 380 us in this
// kernel (the tensor pipe busy 77 % of it; the rest is draining the accumulators between
// the four runs of each tile), 20 us unpacking and 11 us in the join.  A bf16 dW, which
// needs no runs, takes 357 us in all.  (A loop of a second or more meets the power cap:
// 450 us at 1885 MHz.)
#pragma once
#include "../csrc/pair.cuh"
#include "vec.cuh"

namespace flp {

struct WgradParams {
    int tn, tk;    // 256-row and 512-column tiles of dW
    int group;     // row tiles that share their column tiles while both are in L2
    int whole;     // tiles that are written directly (units 0 .. whole - 1)
    int splits;    // runs of each other tile
    int units;
    int KB;        // 64-row blocks of dY and X^
    int run;       // 64-row blocks that one accumulation takes (fp32 results)
    int N, K;
    int add;       // whole tiles add into dW
    int bf16_out;  // dW in bf16 (else fp32)
    int* err;
    unsigned long long wait_limit_ns;
    int stall_after;  // < 0: off; else the producers stop after this many blocks (self-test)
};

struct WgradUnit {
    int n0, k0;    // first row and column of the tile
    int kb0, kb1;  // 64-row blocks
    int part;      // partial tile index, -1: written to dW
    int halves;    // 256-column halves that hold columns of dW
    int run;       // blocks accumulated before the accumulators are drained
};

// The tensor cores round an accumulator toward zero at every step, so the error
// of a long sum grows with its length: 3.0e-6 of the result over 8192 rows of
// centred normal values, 1.9e-5 over 32768, 1.1e-3 over 1048576, against 4.8e-7
// over 2048 (values with an offset of half their spread: twice that; a product of
// the same values in fp32 arithmetic 1e-7 to 5e-7).  An fp32 result is
// therefore summed in runs of at most 2048 rows, whose sums are added in memory,
// rounded to nearest (of 4096: 8192 x 8192 x 5120 takes 380 us instead of 410, in one
// run 366, at errors of 1.2e-6 and 3.0e-6).  Draining the accumulators between runs
// costs most when every column goes through memory, so WGRAD_KEEP of a half's 256
// columns are summed in the epilogue's registers (96: 410 us, 64: 420, 32: 432; 128
// spills 148 bytes: 418).  A bf16
// result's own rounding (1.7e-3) leaves nothing of the error of up to 131072 rows (1e-4):
// one run, stored directly.  Above that the error also has a direction (every value
// 1e-3 too small over 1048576 rows), so the result is joined from fp32 sums of runs.
constexpr int WGRAD_RUN = 32;
constexpr int WGRAD_BF16_RUN = 2048;
constexpr int WGRAD_KEEP = 96;

__device__ __forceinline__ WgradUnit wgrad_unit(const WgradParams& p, int u) {
    WgradUnit t;
    int tile = u;
    t.part = -1;
    t.kb0 = 0;
    t.kb1 = p.KB;
    if (u >= p.whole) {
        t.part = u - p.whole;
        tile = p.whole + t.part / p.splits;
        const int s = t.part % p.splits;
        t.kb0 = static_cast<int>(static_cast<long long>(p.KB) * s / p.splits);
        t.kb1 = static_cast<int>(static_cast<long long>(p.KB) * (s + 1) / p.splits);
    }
    const int per = p.group * p.tk;
    const int g = tile / per;
    const int rows = min(p.group, p.tn - g * p.group);
    const int r = tile - g * per;
    t.k0 = r / rows * (2 * BN);
    t.n0 = (g * p.group + r % rows) * PM;
    t.halves = t.k0 + BN < p.K ? 2 : 1;
    t.run = t.part < 0 && p.bf16_out ? t.kb1 - t.kb0 : p.run;
    return t;
}

// NaN in what an epilogue group (half g of a tile, the 128 rows from `rofs` on) would
// still have written to dW, from unit u on: what a timed-out contraction leaves there is
// what dW held, or some of its runs.  Split tiles are left to the join.  Out of line.
__device__ __noinline__ void wgrad_fill_nan(const WgradParams& p, void* dw, int u, int npairs, int g, int rofs, int et) {
    for (; u < p.whole; u += npairs) {
        const WgradUnit t = wgrad_unit(p, u);
        const int k0 = t.k0 + g * BN, n0 = t.n0 + rofs;
        const int cols = min(BN, p.K - k0), rows = min(BM, p.N - n0);
        for (int r = 0; r < rows; ++r)
            for (int c = et; c < cols; c += EPI_THREADS) {
                const long long o = static_cast<long long>(n0 + r) * p.K + k0 + c;
                if (p.bf16_out)
                    static_cast<unsigned short*>(dw)[o] = 0x7fc0;
                else
                    static_cast<uint32_t*>(dw)[o] = 0x7fc00000u;
            }
    }
}

__global__ void __launch_bounds__(WIDE_THREADS, 1)
    flp_wgrad_kernel(const __grid_constant__ CUtensorMap tmY,     // dY, MN-major A (64 x 64 boxes)
                     const __grid_constant__ CUtensorMap tmX,     // X^, MN-major B (64 x 64)
                     const __grid_constant__ CUtensorMap tmDw,    // dW store boxes (128 rows x 64 bytes)
                     const __grid_constant__ CUtensorMap tmPart,  // partial tiles, fp32 [.., 512] (128 x 64 bytes)
                     const __grid_constant__ WgradParams p, void* dw) {
    extern __shared__ uint8_t smem_raw[];
    const Smem sm = smem_layout(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = (rank == 0);
    const int rofs = static_cast<int>(rank) * BM;
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmY);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmDw);
        tma_prefetch_desc(&tmPart);
    }
    if (threadIdx.x == 0) griddep_launch_dependents();
    const uint32_t tmem_base = pair_prologue(sm, warp);
    griddep_wait();  // X^ and the cleared error word are complete from here on
    const uint64_t limit = p.wait_limit_ns;
    volatile int* abort_flag = sm.abort_flag;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true, stalled = false;
            for (int u = pair; u < p.units && ok; u += npairs) {
                const WgradUnit t = wgrad_unit(p, u);
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (p.stall_after >= 0 && issued++ == p.stall_after) {
                        ok = false, stalled = true;  // stop feeding the MMA
                        break;
                    }
                    if (!mbar_wait(&sm.empty[stage], phase ^ 1u, limit, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (leader)
                        mbar_arrive_expect_tx(&sm.full[stage], 2 * (A_STAGE_BYTES + t.halves * B_STAGE_BYTES));
                    const uint32_t bar = mapa_shared(smem_addr(&sm.full[stage]), 0);
                    uint8_t* a = sm.base + slot_a(true, stage);
                    uint8_t* b = sm.base + slot_b(true, stage);
#pragma unroll
                    for (int j = 0; j < BM / 64; ++j)
                        tma_load_2d_pair(a + j * 8192, &tmY, t.n0 + rofs + j * 64, kb * BK, bar);
                    for (int h = 0; h < t.halves; ++h) {
#pragma unroll
                        for (int j = 0; j < BNH / 64; ++j)
                            tma_load_2d_pair(b + h * B_STAGE_BYTES + j * 8192, &tmX,
                                             t.k0 + h * BN + rofs + j * 64, kb * BK, bar);
                    }
                    if (++stage == STAGES_W) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && !stalled) raise_abort(sm, p.err);
        }
    } else if (warp == 1) {
        // ---------------------------------------------- MMA issuer (leader)
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = idesc_bf16_f32(PM, BN, 1, 1);
            uint32_t gk = 0;    // k-blocks consumed so far
            uint32_t uses = 0;  // bit h: parity of the uses of accumulator h so far
            bool ok = true;
            auto issue = [&](uint32_t g, int h, bool first) {
                const int s = static_cast<int>(g % STAGES_W);
                const uint32_t a = smem_addr(sm.base + slot_a(true, s));
                const uint32_t b = smem_addr(sm.base + slot_b(true, s)) + h * B_STAGE_BYTES;
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k)
                    umma_bf16_pair(tmem_base + static_cast<uint32_t>(h * BN), operand_desc<1>(a, k),
                                   operand_desc<1>(b, k), idesc, (!first || k > 0) ? 1u : 0u);
            };
            auto wait_full = [&](uint32_t g) {
                if (!mbar_wait(&sm.full[g % STAGES_W], (g / STAGES_W) & 1u, limit, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            auto release = [&](uint32_t g) { umma_commit_pair_mc(&sm.empty[g % STAGES_W], PAIR_MASK); };
            auto wait_tempty = [&](int h) {
                if (!mbar_wait(&sm.tempty[h], ((uses >> h) & 1u) ^ 1u, limit, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            auto publish = [&](int h) {
                umma_commit_pair_mc(&sm.tfull[h], PAIR_MASK);
                uses ^= 1u << h;
            };
            for (int u = pair; u < p.units && ok; u += npairs) {
                const WgradUnit t = wgrad_unit(p, u);
                for (int kb0 = t.kb0; kb0 < t.kb1 && ok; kb0 += t.run) {
                    const int KB = min(t.run, t.kb1 - kb0);
                    ok = wait_tempty(0);
                    if (t.halves == 1) {
                        for (int kb = 0; kb < KB && ok; ++kb) {
                            ok = wait_full(gk + kb);
                            if (!ok) break;
                            issue(gk + kb, 0, kb == 0);
                            release(gk + kb);
                        }
                        if (ok) publish(0);
                    } else {
                        // halves staggered at both ends of the tile: half 0 completes
                        // (and is drained) under the last half-1 MMAs, and fills while
                        // the previous tile's half 1 is still drained
                        const int head = min(WIDE_EDGE, KB);
                        const int tail0 = max(head, KB - WIDE_EDGE);
                        for (int kb = 0; kb < head && ok; ++kb) {
                            ok = wait_full(gk + kb);
                            if (ok) issue(gk + kb, 0, kb == 0);
                        }
                        if (!ok) break;
                        if (head == KB) publish(0);
                        ok = wait_tempty(1);
                        if (!ok) break;
                        for (int kb = 0; kb < head; ++kb) {
                            issue(gk + kb, 1, kb == 0);
                            release(gk + kb);
                        }
                        for (int kb = head; kb < tail0 && ok; ++kb) {
                            ok = wait_full(gk + kb);
                            if (!ok) break;
                            issue(gk + kb, 0, false);
                            issue(gk + kb, 1, false);
                            release(gk + kb);
                        }
                        for (int kb = tail0; kb < KB && ok; ++kb) {
                            ok = wait_full(gk + kb);
                            if (ok) issue(gk + kb, 0, false);
                        }
                        if (!ok) break;
                        if (head < KB) publish(0);
                        for (int kb = tail0; kb < KB; ++kb) {
                            issue(gk + kb, 1, false);
                            release(gk + kb);
                        }
                        publish(1);
                    }
                    gk += static_cast<uint32_t>(KB);
                }
            }
            if (!ok) raise_abort(sm, p.err);
            umma_commit_pair_mc(sm.drain, 0x1);  // every MMA issued so far has completed
            volatile int no_abort = 0;
            mbar_wait(sm.drain, 0, limit, &no_abort);
        }
    } else {
        // ------------------------- epilogue: group g drains accumulator g
        const int g = (warp - 2) >> 2;
        const int et = threadIdx.x - 64 - g * EPI_THREADS;  // thread 0 issues the bulk stores
        const int q = warp & 3;
        const int r = q * 32 + lane;  // accumulator row == TMEM lane
        const uint32_t tbase = tmem_base + static_cast<uint32_t>(g * BN) + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t tempty = mapa_shared(smem_addr(&sm.tempty[g]), 0);
        const uint32_t bar_box = 1 + 2 * g, bar_vote = 2 + 2 * g;
        uint8_t* box0 = sm.base + SMEM_STG + g * (2 * NBOX_BYTES);
        StoreRing ring;
        uint32_t phase = 0;
        bool ok = true;
        int u = pair;
        for (; u < p.units; u += npairs) {
            const WgradUnit t = wgrad_unit(p, u);
            if (g >= t.halves) continue;
            const bool partial = t.part >= 0;
            const CUtensorMap* out = partial ? &tmPart : &tmDw;
            const int x0 = (partial ? 0 : t.k0) + g * BN;
            const int y0 = (partial ? t.part * PM : t.n0) + rofs;
            const bool bf16_out = !partial && p.bf16_out;
            const int cols = min(BN, p.K - t.k0 - g * BN);  // columns of dW in this half
            // between the runs of a tile the first WGRAD_KEEP columns' sums stay in
            // registers; the others are added to what the earlier runs stored
            const bool runs = t.kb0 + t.run < t.kb1;
            float kept[WGRAD_KEEP];
            auto store32 = [&](int b, const uint32_t* v, bool add) {
                if (b * 32 >= cols) return;  // the whole box lies past dW's last column
                if (bf16_out) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    narrow_box_store(ring, box0, bar_box, et, r, w, out, x0 + b * 32, y0, false);
                } else {
                    narrow_box_store(ring, box0, bar_box, et, r, v, out, x0 + b * 32, y0, add);
                    narrow_box_store(ring, box0, bar_box, et, r, v + 16, out, x0 + b * 32 + 16, y0, add);
                }
            };
            for (int kb0 = t.kb0; kb0 < t.kb1 && ok; kb0 += t.run) {
                const bool ready = mbar_wait(&sm.tfull[g], phase, limit, abort_flag);
                // every thread of the group takes the same branch (the box barriers need all of them)
                if (!named_bar_all(bar_vote, EPI_THREADS, ready)) {
                    ok = false;
                    break;
                }
                phase ^= 1u;
                tc_fence_after();
                const bool first = kb0 == t.kb0, adds = !partial && p.add;
                if (runs) {
#pragma unroll
                    for (int b = 0; b < WGRAD_KEEP / 32; ++b) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tbase + b * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            kept[b * 32 + j] = (first ? 0.f : kept[b * 32 + j]) + __uint_as_float(v[j]);
                    }
                    // a later run adds to what this thread's earlier bulk stores wrote
                    if (!first && et == 0) bulk_wait_group<0>();
                }
#pragma unroll 1
                for (int b = runs ? WGRAD_KEEP / 32 : 0; b < BN / 32; ++b) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tbase + b * 32, v);
                    tmem_wait_ld();
                    if (b == BN / 32 - 1) {
                        tc_fence_before();
                        mbar_arrive_cluster(tempty);
                    }
                    store32(b, v, !first || adds);
                }
                if (runs && kb0 + t.run >= t.kb1) {
#pragma unroll
                    for (int b = 0; b < WGRAD_KEEP / 32; ++b) {
                        uint32_t v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(kept[b * 32 + j]);
                        store32(b, v, adds);
                    }
                }
            }
            if (!ok) break;
        }
        if (!ok) raise_abort(sm, p.err);
        if (et == 0) bulk_wait_group<0>();
        if (!ok) {
            named_bar_sync(bar_vote, EPI_THREADS);  // behind the group's earlier stores
            wgrad_fill_nan(p, dw, u, npairs, g, rofs, et);
        }
    }

    pair_epilogue(sm, warp, tmem_base);
}

struct WgradJoinParams {
    const float* part;  // partial tiles [tile][split][256][512]
    WgradParams g;
    void* dw;           // [N, K]
    int add;
    const int* err;
};

// Sums the partial tiles' splits in order and writes their part of dW (adding
// to what is there, in fp32, when asked).  One block per 2 rows of a tile.
// After a timeout of the contraction the sums are NaN, like what that kernel fills the
// tiles with that it should have written itself, so that no incomplete value passes for
// a result.  4 splits of 16 tiles (33 MB) take 11 us with cold caches,
// bound by the bytes of one short wave of loads.
constexpr int WJ_THREADS = 256;
constexpr int WJ_ROWS = 2;

__global__ void __launch_bounds__(WJ_THREADS) flp_wgrad_join_kernel(const WgradJoinParams p) {
    const int tile = blockIdx.x / (PM / WJ_ROWS);
    const WgradUnit t = wgrad_unit(p.g, p.g.whole + tile * p.g.splits);
    const int r0 = blockIdx.x % (PM / WJ_ROWS) * WJ_ROWS;
    griddep_wait();
    const bool bad = (*p.err & ERR_TIMEOUT) != 0;
    const float* base = p.part + static_cast<long long>(tile) * p.g.splits * (PM * 2 * BN);
    static_assert(WJ_ROWS * 2 * BN / 4 == WJ_THREADS, "four columns a thread");
    __shared__ __align__(16) float rows[WJ_ROWS][2 * BN];
    const int in_block = threadIdx.x / (2 * BN / 4), at = threadIdx.x % (2 * BN / 4);
    const int n = t.n0 + r0 + in_block, k = t.k0 + 4 * at;
    const bool on = n < p.g.N && k < p.g.K;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
        const float* from = base + static_cast<long long>(r0 + in_block) * (2 * BN) + 4 * at;
#pragma unroll 8
        for (int j = 0; j < p.g.splits; ++j) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(from + static_cast<long long>(j) * (PM * 2 * BN)));
            s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
        }
        if (bad) s.x = s.y = s.z = s.w = __uint_as_float(0x7fc00000u);
    }
    if (p.g.K % 4 == 0) {  // dW rows are aligned to four columns (16 bytes, or 8 in bf16)
        if (!on) return;
        const long long o = static_cast<long long>(n) * p.g.K + k;
        if (p.g.bf16_out) {
            *reinterpret_cast<uint2*>(static_cast<bf16*>(p.dw) + o) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
        } else {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.dw) + o);
            float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.add) old = *d;
            *d = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
        }
    } else {  // through shared memory, so that neighbouring threads write neighbouring columns
        *reinterpret_cast<float4*>(&rows[in_block][4 * at]) = s;
        __syncthreads();
        if (n >= p.g.N) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = at + i * (2 * BN / 4);
            if (t.k0 + c >= p.g.K) break;
            const long long o = static_cast<long long>(n) * p.g.K + t.k0 + c;
            if (p.g.bf16_out)
                static_cast<bf16*>(p.dw)[o] = __float2bfloat16_rn(rows[in_block][c]);
            else
                static_cast<float*>(p.dw)[o] = (p.add ? static_cast<float*>(p.dw)[o] : 0.f) + rows[in_block][c];
        }
    }
}

}  // namespace flp

// kernels.cuh - sm_103a kernels of the fused linear log-prob / cross-entropy head.
//
// Every contraction of the path runs on CTA pairs (clusters of two CTAs on two
// SMs) that share an output tile: tcgen05.mma.cta_group::2 with M = 256 (128
// rows of A in each CTA) and N = 256 (B split along N, 128 rows in each CTA),
// fp32 accumulators in both CTAs' TMEM.  For a 256 x 256 tile each SM loads
// 16 KiB of A and 16 KiB of B per 64-deep K step for 2 * 128 * 256 * 64 MACs;
// a wide 256 x 512 tile (both accumulators) loads 48 KiB for twice that.
//
//   flp_fwd_kernel   : z = s X W^T tiles -> online max / sum-exp / (entropy) /
//                      target pick per row -> raw per-split partials
//   flp_merge_kernel : per-split partials -> lse, logprob, entropy
//   flp_dz_kernel    : (bwd.cuh) the dZ tiles of the split backward schedules
//   flp_bwd_kernel   : (bwd.cuh) dX and dW tiles, and all tiles of the fused one
//
// pair.cuh holds the pieces every pair kernel shares; this file the forward and
// the merge.
//
// Roles (192 threads per CTA, one CTA per SM):
//   warp 0      TMA producer (one lane) for this CTA's halves of A and B
//   warp 1      TMEM allocation (both CTAs) and, in the leader CTA (cluster
//               rank 0), the single thread that issues the pair MMAs
//   warps 2..5  epilogue: thread == accumulator row (TMEM lane) of this CTA
// Barriers: both CTAs' TMA loads complete on the leader's `full` barrier; the
// leader's MMA commits are multicast to both CTAs' `empty` (stage free) and
// `tfull` (accumulator ready) barriers; both CTAs' epilogues release an
// accumulator on the leader's `tempty` barrier.  Two 256-column accumulators
// (512 TMEM columns) let a tile's epilogue overlap the next tile's MMAs.
//
// The forward, the dZ kernel and the backward's dX + dW launch run wide tiles
// instead: 256 rows x 512 columns, one per pair, both accumulators (half h of
// the columns in accumulator h), so each SM loads 16 KiB of A and 32 KiB of B
// per K step for twice the MACs (25 % fewer operand bytes per MAC).  They have
// two epilogue groups of four warps (warps 2..5 drain half 0, warps 6..9 half
// 1; 320 threads), and the MMA issuer staggers the halves at both ends of a
// tile so that one half's epilogue runs under the other half's MMAs.
//
// Every mbarrier wait is bounded (globaltimer); on expiry the kernel raises the
// timeout bit in the error word, stops issuing work, lets its copies and MMAs
// in flight finish (a bounded wait), frees its TMEM and returns.
#pragma once
#include <cstdint>
#include <cuda.h>
#include "pair.cuh"

namespace flp {

// ------------------------------------------------------------ forward kernel

struct FwdParams {
    // schedule: units are runs [n0, n1) of 512-column tiles sharing one 256-row pair tile;
    // each unit writes two partials per row (one per 256-column half): S * 2 in all
    int units, Mt, Nt, S, tps, GM;
    int KB;    // K blocks of 64 (H / 64, rounded up)
    int M;     // rows
    int V;     // vocabulary size (column mask)
    long long ignore_index;
    float scale;   // s
    float scale2;  // s * log2(e)
    const long long* y;
    float* part_m;
    float* part_s;
    float* part_t;
    float* zy;
    int* err;
    unsigned long long wait_limit_ns;
    int debug_stall_after;  // < 0: off; else the producers stop after this many stages
};

struct Unit {
    int mt, n0, n1, split;
};

// Units are ordered in groups of GM pair M-tiles; inside a group the split index
// is outermost, so the pairs running at the same time share W tiles while the
// group's X rows stay resident in L2.
__device__ __forceinline__ Unit decode_unit(const FwdParams& p, int u) {
    const int per_group = p.GM * p.S;
    const int g = u / per_group;
    const int first_m = g * p.GM;
    const int gm = min(p.GM, p.Mt - first_m);
    const int r = u - g * per_group;
    Unit t;
    t.split = r / gm;
    t.mt = first_m + (r - t.split * gm);
    t.n0 = t.split * p.tps;
    t.n1 = min(p.Nt, t.n0 + p.tps);
    return t;
}

template <bool kEnt>
__global__ void __launch_bounds__(WIDE_THREADS, 1)
    flp_fwd_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const FwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    const Smem sm = smem_layout(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = (rank == 0);
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (threadIdx.x == 0) griddep_launch_dependents();  // the next launch may be scheduled early
    const uint32_t tmem_base = pair_prologue(sm, warp);
    griddep_wait();  // the previous launch's results (dZ, the error word) are complete from here on
    const uint64_t limit = p.wait_limit_ns;
    volatile int* abort_flag = sm.abort_flag;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int u = pair; u < p.units && ok; u += npairs) {
                const Unit t = decode_unit(p, u);
                for (int nt = t.n0; nt < t.n1 && ok; ++nt) {
                    for (int kb = 0; kb < p.KB; ++kb) {
                        if (p.debug_stall_after >= 0 && issued >= p.debug_stall_after) {
                            ok = false;  // injected stall: stop feeding the MMA
                            break;
                        }
                        if (!mbar_wait(&sm.empty[stage], phase ^ 1u, limit, abort_flag)) {
                            ok = false;
                            break;
                        }
                        load_wide_kblock(sm, stage, leader, &tmA, t.mt * PM + static_cast<int>(rank) * BM,
                                         &tmB, nt * 2 * BN + static_cast<int>(rank) * BNH, kb);
                        ++issued;
                        if (++stage == STAGES_W) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (!ok && p.debug_stall_after < 0) {
                raise_abort(sm, p.err);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------- MMA issuer (leader)
        if (lane == 0 && leader) {
            uint32_t gk = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int u = pair; u < p.units && ok; u += npairs) {
                const Unit t = decode_unit(p, u);
                for (int nt = t.n0; nt < t.n1 && ok; ++nt) {
                    ok = wide_tile_mma(sm, tmem_base, gk, acc_phase, acc_phase, p.KB, limit, abort_flag);
                    acc_phase ^= 1u;
                }
            }
            if (!ok) {
                raise_abort(sm, p.err);
            }
            umma_commit_pair_mc(sm.drain, 0x1);  // every MMA issued so far has completed
            volatile int no_abort = 0;
            mbar_wait(sm.drain, 0, limit, &no_abort);
        }
    } else {
        // --------------------------------------------------------- epilogue
        // two groups of four warps: group g drains accumulator g, the
        // 256-column half g of every 512-column tile
        const int g = (warp - 2) >> 2;
        const int q = warp & 3;           // TMEM lane quadrant of this warp
        const int r = q * 32 + lane;      // accumulator row == TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t tempty_leader = mapa_shared(smem_addr(&sm.tempty[g]), 0);
        const int acc = g;
        uint32_t acc_phase = 0;
        bool ok = true;

        for (int u = pair; u < p.units && ok; u += npairs) {
            const Unit t = decode_unit(p, u);
            const int row = t.mt * PM + static_cast<int>(rank) * BM + r;
            const bool row_ok = row < p.M;
            const long long yv = row_ok ? p.y[row] : -1;
            float run_m = -INFINITY, run_s = 0.f, run_t = 0.f, zyv = 0.f;
            bool found = false;

            for (int nt = t.n0; nt < t.n1; ++nt) {
                if (!mbar_wait(&sm.tfull[acc], acc_phase, limit, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tbase = tmem_base + static_cast<uint32_t>(acc * BN) + lane_off;
                const int col0 = nt * 2 * BN + g * BN;
                const int nvalid = min(BN, p.V - col0);
                const long long tcol = yv - col0;
#pragma unroll 1
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tbase + c * 32, v);
                    tmem_wait_ld();
                    if (c == BN / 32 - 1) {
                        tc_fence_before();
                        mbar_arrive_cluster(tempty_leader);
                    }
                    const long long tc = tcol - c * 32;
                    if (tc >= 0 && tc < 32) {
                        zyv = select32(v, static_cast<int>(tc)) * p.scale;
                        found = true;
                    }
                    const int nv = nvalid - c * 32;
                    if (nv <= 0) continue;
                    if (nv >= 32) {
                        // full chunk: packed fp32 pairs halve the FP32 instruction count
                        uint64_t up[16];
                        const uint64_t sc2 = f2_pack(p.scale2, p.scale2);
                        float cmax = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            up[j] = f2_mul(f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sc2);
                            float a, b;
                            f2_unpack(up[j], a, b);
                            cmax = fmax3(cmax, a, b);
                        }
                        if (cmax > run_m) {
                            const float alpha = ex2_approx(run_m - cmax);
                            if constexpr (kEnt)
                                run_t = (run_s > 0.f) ? alpha * (run_t + run_s * (run_m - cmax)) : 0.f;
                            run_s *= alpha;
                            run_m = cmax;
                        }
                        const uint64_t negm = f2_pack(-run_m, -run_m);
                        uint64_t sacc = f2_pack(0.f, 0.f), tacc = f2_pack(0.f, 0.f);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint64_t d = f2_add(up[j], negm);
                            float d0, d1;
                            f2_unpack(d, d0, d1);
                            const uint64_t e = f2_pack(ex2_approx(d0), ex2_approx(d1));
                            sacc = f2_add(sacc, e);
                            if constexpr (kEnt) tacc = f2_fma(e, d, tacc);
                        }
                        float s0, s1, t0, t1;
                        f2_unpack(sacc, s0, s1);
                        run_s += s0 + s1;
                        if constexpr (kEnt) {
                            f2_unpack(tacc, t0, t1);
                            run_t += t0 + t1;
                        }
                        continue;
                    }
                    // the vocabulary tail: columns >= V are left out of every sum
                    float uu[32];
                    float cmax = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        uu[j] = (j < nv) ? __uint_as_float(v[j]) * p.scale2 : -INFINITY;
                        cmax = fmaxf(cmax, uu[j]);
                    }
                    if (cmax > run_m) {
                        // rescale the running sums to the new maximum; a row that
                        // has seen nothing yet (run_s == 0) has nothing to rescale
                        const float alpha = ex2_approx(run_m - cmax);
                        if constexpr (kEnt)
                            run_t = (run_s > 0.f) ? alpha * (run_t + run_s * (run_m - cmax)) : 0.f;
                        run_s *= alpha;
                        run_m = cmax;
                    }
                    float s0 = 0.f, t0 = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j < nv) {
                            const float d0 = uu[j] - run_m;
                            const float e0 = ex2_approx(d0);
                            s0 += e0;
                            if constexpr (kEnt) t0 = fmaf(e0, d0, t0);
                        }
                    }
                    run_s += s0;
                    if constexpr (kEnt) run_t += t0;
                }
                acc_phase ^= 1u;
            }
            if (!ok) break;

            if (row_ok) {
                const size_t o = static_cast<size_t>(2 * t.split + g) * p.M + row;
                p.part_m[o] = run_m;
                p.part_s[o] = run_s;
                if constexpr (kEnt) p.part_t[o] = run_t;
                if (found) p.zy[row] = zyv;
            }
        }
        if (!ok) {
            raise_abort(sm, p.err);
        }
    }

    pair_epilogue(sm, warp, tmem_base);
}

// ---------------------------------------------------------- fp32 -> bf16

// dst[i] = bf16(src[i]) (round to nearest even): the vocabulary-split
// backward's fp32 dX, accumulated over the chunks, rounded once.  n may be
// any size; the 16-byte vector path runs while 8 elements remain.
__global__ void __launch_bounds__(256) flp_round_bf16_kernel(const float* __restrict__ src,
                                                             uint16_t* __restrict__ dst, int64_t n) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x * 8;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; i < n; i += stride) {
        if (i + 8 <= n) {
            const float4 a = *reinterpret_cast<const float4*>(src + i);
            const float4 b = *reinterpret_cast<const float4*>(src + i + 4);
            uint4 o;
            o.x = pack_bf16x2(a.x, a.y);
            o.y = pack_bf16x2(a.z, a.w);
            o.z = pack_bf16x2(b.x, b.y);
            o.w = pack_bf16x2(b.z, b.w);
            *reinterpret_cast<uint4*>(dst + i) = o;
        } else {
            for (int64_t j = i; j < n; ++j) dst[j] = static_cast<uint16_t>(pack_bf16x2(src[j], 0.f) & 0xFFFFu);
        }
    }
}

// ------------------------------------------------------------- split merge

struct MergeParams {
    int M, S, V;
    long long ignore_index;
    int compute_entropy;
    const long long* y;
    const float* part_m;
    const float* part_s;
    const float* part_t;
    const float* zy;
    float* logprob;
    float* lse;
    float* entropy;
    int* err;
};

// Online combination of two (max, sum-exp, entropy sum) triples in base-2
// units: the sums are rescaled to the larger max; a triple with sum 0 (a split
// that saw no column) contributes nothing, so no 0 * inf arises.
struct Stats {
    float m, s, t;
};

__device__ __forceinline__ Stats combine(Stats a, Stats b) {
    if (!(b.s > 0.f)) return a;
    if (!(a.s > 0.f)) return b;
    const float m = fmaxf(a.m, b.m);
    const float da = a.m - m, db = b.m - m;
    const float ea = exp2f(da), eb = exp2f(db);
    Stats r;
    r.m = m;
    r.s = a.s * ea + b.s * eb;
    r.t = (a.t + a.s * da) * ea + (b.t + b.s * db) * eb;
    return r;
}

constexpr int MERGE_ROWS = 32;   // rows per block (one per lane)
constexpr int MERGE_WAYS = 8;    // warps per block; warp w reads splits w, w + 8, ...
constexpr int MERGE_BATCH = 8;   // splits whose loads a warp has in flight at once

// Combines the per-split partials of each row into the final lse / logprob /
// entropy (the "reduced" and "result" stages kept in buffers separate from the
// raw partials).  Each warp reads a stripe of splits for 32 consecutive rows
// (coalesced), the stripes are combined through shared memory.  Base-2 units
// inside, natural log out.  When the forward tile kernel gave up on a wait
// (timeout bit in the error word) its partials are incomplete: every output
// row is then NaN, so that no stale or partial value passes for a result.
__global__ void __launch_bounds__(MERGE_ROWS * MERGE_WAYS) flp_merge_kernel(const MergeParams p) {
    __shared__ Stats part[MERGE_WAYS][MERGE_ROWS];
    const int lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int i = blockIdx.x * MERGE_ROWS + lane;
    griddep_wait();  // the forward tile kernel's partials and error word are complete
    if (*reinterpret_cast<volatile const int*>(p.err) & ERR_TIMEOUT) {
        if (w == 0 && i < p.M) {
            const float nan = __int_as_float(0x7fc00000);
            p.lse[i] = nan;
            p.logprob[i] = nan;
            if (p.compute_entropy) p.entropy[i] = nan;
        }
        return;
    }
    Stats acc{-INFINITY, 0.f, 0.f};
    if (i < p.M) {
        // splits w, w + 8, w + 16, ... in order; the loads of MERGE_BATCH of
        // them are issued before any is combined (the loop is latency-bound)
        for (int k0 = w; k0 < p.S; k0 += MERGE_BATCH * MERGE_WAYS) {
            Stats v[MERGE_BATCH];
#pragma unroll
            for (int j = 0; j < MERGE_BATCH; ++j) {
                const int k = k0 + j * MERGE_WAYS;
                v[j] = Stats{-INFINITY, 0.f, 0.f};
                if (k < p.S) {
                    const size_t o = static_cast<size_t>(k) * p.M + i;
                    v[j] = Stats{p.part_m[o], p.part_s[o], p.compute_entropy ? p.part_t[o] : 0.f};
                }
            }
#pragma unroll
            for (int j = 0; j < MERGE_BATCH; ++j) acc = combine(acc, v[j]);
        }
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w != 0 || i >= p.M) return;
#pragma unroll
    for (int j = 1; j < MERGE_WAYS; ++j) acc = combine(acc, part[j][lane]);
    const float l2s = log2f(acc.s);
    const float lse = (acc.m + l2s) * LN2;
    p.lse[i] = lse;
    const long long yv = p.y[i];
    float lp, ent = p.compute_entropy ? (l2s - acc.t / acc.s) * LN2 : 0.f;
    if (yv == p.ignore_index) {
        lp = 0.f;
        ent = 0.f;
    } else if (yv < 0 || yv >= p.V) {
        lp = __int_as_float(0x7fc00000);
        atomicOr(p.err, ERR_BAD_TARGET);
    } else {
        lp = p.zy[i] - lse;
    }
    p.logprob[i] = lp;
    if (p.compute_entropy) p.entropy[i] = ent;
}

}  // namespace flp

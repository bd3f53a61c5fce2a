// linear.cuh - a linear layer with bias, activation and residual in its epilogue, and
// what its gradients need:
//     forward   v = x W^T + b,  y = act(v) + r,  v kept in bf16 for the backward pass
//     backward  d = dy act'(v),  dx = d W,  dW = d^T x,  db = column sums of d
// x [M, K], W [N, K], y [M, N] in bf16, sums and everything up to the one rounding of
// each output in fp32 (so y does not carry the rounding of v).
//
// The products x W^T and d W run in one kernel on CTA pairs: 256 x 512 tiles in both TMEM
// accumulators, four 48 KiB slots fed by TMA, the halves staggered at the tile ends, one
// epilogue group per accumulator; W is the K-major operand of the first and the MN-major
// one of the second.  Whole rounds of tiles over the resident pairs write their outputs
// themselves; the tiles of the last, incomplete round (all of them, when rows are few)
// are split along the contraction into fp32 partial tiles, which a small kernel joins in
// a fixed order and takes through the same epilogue.  d is rounded to bf16 by a pass over
// dy and v that also sums db from the unrounded values; dW is the contraction of
// wgrad.cuh.  The rounding (2^-8 of each value) is no more than a bf16 result's own, but an
// fp32 dW would show it: for that one d is written as the sum of two bf16 numbers (2^-16 of
// it), and both are contracted with x, below one another in one product or in two.  Of few
// rows, where W and dW are what takes time, every result is made so; the caller may ask for
// one number or two in all.
//
// Bound by the tensor cores at many rows: 8192 x 4096 -> 16384 (582 us at the measured
// matrix rate) takes 562 us plain, 606 with a bias and gelu_tanh, 720 to 740 with v kept as
// well in a loop that meets the power cap (75 % of the tensor pipe busy; the rest is what
// the epilogue, 65536 outputs a CTA and tile, does not hide: a tile's two accumulators are
// all of TMEM).  Bound by reading W at few rows: 4096 -> 16384 (20 us) 26 us for one row,
// 34 for 16.  In between, up to some 2048 rows, by operands through the L2 and by the joins:
// 512 x 4096 -> 4096 (9 us) 26, where a library product takes 14; 777 x 1000 -> 2047 with
// everything (2 us) 20.  (A graph replay's time, less the 5 us of an empty one.)
#pragma once
#include <type_traits>
#include "../csrc/pair.cuh"
#include "vec.cuh"

namespace flp {

constexpr int LIN_NONE = 0, LIN_RELU = 1, LIN_GELU = 2, LIN_GELU_TANH = 3, LIN_SILU = 4;

// ------------------------------------------------------------------ activation

// All on packed pairs: the epilogues of the products are bound by their instructions.

constexpr float LIN_INV_SQRT_2PI = 0.3989422804014327f;
constexpr float LIN_TANH_U = 1.5957691216057308f;  // gelu_tanh(v) = v sigmoid(u), u = sqrt(8 / pi) (v + 0.044715 v^3)
constexpr float LIN_TANH_3 = 0.044715f;

__device__ __forceinline__ uint64_t f2_rcp(uint64_t v) { return f2_map(v, [](float x) { return rcp_approx(x); }); }
__device__ __forceinline__ uint64_t f2_abs(uint64_t v) { return v & 0x7fffffff7fffffffull; }

// exp(-v^2 / 2), and h = Phi(-|v|) = exp(-v^2 / 2) erfcx(|v| / sqrt 2) / 2, whose relative
// error is that of erfcx: with t = 1 / (1 + 0.375 x), erfcx(x) / 2 = t P(t) for 0 <= x <=
// 9.6 to 6.4e-7, P of degree 6 from a weighted least-squares fit (beyond, h vanishes).
__device__ __forceinline__ void lin_normal_tail(uint64_t v, uint64_t& e, uint64_t& h) {
    e = f2_ex2(f2_mul(f2_mul(v, v), f2_splat(-0.5f * LOG2E)));
    const uint64_t t = f2_rcp(f2_fma(f2_abs(v), f2_splat(0.375f * 0.7071067811865476f), f2_splat(1.f)));
    uint64_t q = f2_splat(0.5f * -0.135095946f);
    q = f2_fma(q, t, f2_splat(0.5f * 0.387937988f));
    q = f2_fma(q, t, f2_splat(0.5f * -0.129597526f));
    q = f2_fma(q, t, f2_splat(0.5f * 0.2830617f));
    q = f2_fma(q, t, f2_splat(0.5f * 0.166664508f));
    q = f2_fma(q, t, f2_splat(0.5f * 0.21568919f));
    q = f2_fma(q, t, f2_splat(0.5f * 0.211339448f));
    h = f2_mul(f2_mul(q, t), e);
}

// -log2(e) u of the two that are v sigmoid(u).
template <int ACT>
__device__ __forceinline__ uint64_t lin_exponent(uint64_t v) {
    if constexpr (ACT == LIN_SILU) return f2_mul(v, f2_splat(-LOG2E));
    return f2_mul(v, f2_fma(f2_mul(v, v), f2_splat(-LOG2E * LIN_TANH_U * LIN_TANH_3), f2_splat(-LOG2E * LIN_TANH_U)));
}

template <int ACT>
__device__ __forceinline__ uint64_t lin_act2(uint64_t v) {
    if constexpr (ACT == LIN_RELU) return f2_map(v, [](float x) { return max_nan(x, 0.f); });
    if constexpr (ACT == LIN_GELU) {  // v Phi(v) = max(v, 0) - |v| Phi(-|v|)
        uint64_t e, h;
        lin_normal_tail(v, e, h);
        const uint64_t a = f2_map(f2_abs(v), [](float x) { return fminf(x, 1e4f); });  // h is 0 by then
        return f2_fma(f2_mul(a, f2_splat(-1.f)), h, f2_map(v, [](float x) { return max_nan(x, 0.f); }));
    }
    if constexpr (ACT == LIN_GELU_TANH || ACT == LIN_SILU)
        return f2_mul(v, f2_rcp(f2_add(f2_ex2(lin_exponent<ACT>(v)), f2_splat(1.f))));
    return v;
}

// act'.  Where |v| is cut off it is 0 or 1 exactly: gelu's exponential has vanished (below
// 2^-126 it is 0), and of the two others e = exp(-u) lies between 2^126, from where its
// reciprocal is 0, and 2^128, so that e p, which gives 1 - p without another exponential,
// is still no NaN.
template <int ACT>
__device__ __forceinline__ uint64_t lin_slope2(uint64_t v) {
    if constexpr (ACT == LIN_RELU) return f2_map(v, [](float x) { return x > 0.f ? 1.f : 0.f; });
    v = f2_map(v, [](float x) {
        constexpr float END = ACT == LIN_GELU_TANH ? 10.03f : ACT == LIN_GELU ? 14.f : 88.f;
        return max_nan(min_nan(x, END), -END);
    });
    if constexpr (ACT == LIN_GELU) {
        uint64_t e, h;
        lin_normal_tail(v, e, h);
        float v0, v1, h0, h1;
        f2_unpack(v, v0, v1);
        f2_unpack(h, h0, h1);
        const uint64_t phi = f2_pack(v0 < 0.f ? h0 : 1.f - h0, v1 < 0.f ? h1 : 1.f - h1);
        return f2_fma(f2_mul(v, f2_splat(LIN_INV_SQRT_2PI)), e, phi);
    }
    uint64_t vdu = v;
    if constexpr (ACT == LIN_GELU_TANH)
        vdu = f2_mul(v, f2_fma(f2_mul(v, v), f2_splat(3.f * LIN_TANH_U * LIN_TANH_3), f2_splat(LIN_TANH_U)));
    const uint64_t e = f2_ex2(lin_exponent<ACT>(v)), p = f2_rcp(f2_add(e, f2_splat(1.f)));
    return f2_fma(f2_mul(vdu, f2_mul(e, p)), p, p);
}

// The same where a few outputs alone are computed: one copy of the code.
__device__ __forceinline__ float lin_act_of(float x, int act) {
    uint64_t v = f2_pack(x, 0.f);
    switch (act) {
        case LIN_RELU: v = lin_act2<LIN_RELU>(v); break;
        case LIN_GELU: v = lin_act2<LIN_GELU>(v); break;
        case LIN_GELU_TANH: v = lin_act2<LIN_GELU_TANH>(v); break;
        case LIN_SILU: v = lin_act2<LIN_SILU>(v); break;
    }
    float hi;
    f2_unpack(v, x, hi);
    return x;
}

// Calls f with the activation as a constant.
template <typename F>
auto lin_with_act(int act, F&& f) {
    switch (act) {
        case LIN_RELU: return f(std::integral_constant<int, LIN_RELU>{});
        case LIN_GELU: return f(std::integral_constant<int, LIN_GELU>{});
        case LIN_GELU_TANH: return f(std::integral_constant<int, LIN_GELU_TANH>{});
        case LIN_SILU: return f(std::integral_constant<int, LIN_SILU>{});
        default: return f(std::integral_constant<int, LIN_NONE>{});
    }
}

// ------------------------------------------------------------------ product

struct LinEpilogue {
    const void* bias;  // [N], or null
    int bias_f32;
    int act;
    const bf16* residual;  // [M, N], or null
    long long ldr;
    bf16* y;
    long long ldy;
    bf16* pre;  // or null
    long long ldpre;
    int vec;       // the rows of y, residual and pre are aligned to 16 bytes
    int bias_vec;  // and so is the bias
};

struct LinParams {
    int tm, tn;   // tiles of 256 rows and of `width` columns
    int width;    // 512, or 256: tiles of one half, in the two accumulators by turns
    int group;    // row tiles that share their column tiles while both are in L2
    int whole;    // tiles that are written directly (units 0 .. whole - 1)
    int splits;   // runs of each other tile; 0: its two halves, written directly
    int units;
    int KB;       // 64-deep blocks of the contraction, over both numbers of d where there are two
    int fold;     // and over one: from here on the blocks of d's low numbers meet those of W again
    int low;      // rows from a row of d to its low numbers (dx alone)
    int M, N;
    float* part;  // partial tiles [tile][split][rows][512]
    int rows;     // of a partial tile: min(M, 256)
    LinEpilogue e;
    int* err;     // error word, or null
    unsigned long long wait_limit_ns;
    int stall_after;  // < 0: off; else the producers stop after this many blocks (self-test)
};

struct LinUnit {
    int m0, n0;    // first row and column of the tile
    int kb0, kb1;  // blocks of the contraction
    int part;      // partial tile index, -1: the outputs are written
    int halves;    // 256-column halves that hold columns (0: none)
};

// The accumulator of the one half of a pair's `it`-th tile.
__device__ __forceinline__ int lin_single(int it) { return it & 1; }

// What epilogue group g drains of a pair's `it`-th tile: the half of a wide tile that lies
// in accumulator g, 128 columns of every tile of one half in a launch of such tiles, or
// the one half of another tile if accumulator g holds it.
struct LinShare {
    int acc;    // -1: nothing
    int col;    // first column, in the tile
    int boxes;  // of 32 columns, up to BN / 32
};
__device__ __forceinline__ LinShare lin_share(const LinParams& p, const LinUnit& t, int g, int it) {
    LinShare s{-1, 0, BN / 32};
    if (p.width == BN) {
        s.acc = lin_single(it), s.col = g * (BN / 2), s.boxes = BN / 64;
    } else if (t.halves == 2) {
        s.acc = g, s.col = g * BN;
    } else if (t.halves == 1 && g == lin_single(it)) {
        s.acc = g;
    }
    s.boxes = max(0, min(s.boxes, (p.N - t.n0 - s.col + 31) / 32));  // the others lie past the last column
    return s;
}

__device__ __forceinline__ LinUnit lin_unit(const LinParams& p, int u) {
    LinUnit t;
    int tile = u;
    t.part = -1;
    t.kb0 = 0;
    t.kb1 = p.KB;
    int from = 0, width = p.width;  // of the tile, the unit's columns
    if (u >= p.whole && p.splits == 0) {
        tile = p.whole + (u - p.whole) / 2;
        from = (u - p.whole) % 2 * BN;
        width = BN;
    } else if (u >= p.whole) {
        t.part = u - p.whole;
        tile = p.whole + t.part / p.splits;
        const int s = t.part % p.splits;
        t.kb0 = static_cast<int>(static_cast<long long>(p.KB) * s / p.splits);
        t.kb1 = static_cast<int>(static_cast<long long>(p.KB) * (s + 1) / p.splits);
    }
    const int per = p.group * p.tn;
    const int g = tile / per;
    const int rows = min(p.group, p.tm - g * p.group);
    const int r = tile - g * per;
    t.n0 = r / rows * p.width + from;
    t.m0 = (g * p.group + r % rows) * PM;
    t.halves = t.n0 >= p.N ? 0 : width > BN && t.n0 + BN < p.N ? 2 : 1;
    if (t.halves == 0) t.kb1 = t.kb0;  // a half past the last column
    return t;
}

// Bias values of 32 columns from c0 on (0 past N or without a bias), added to v.
__device__ __forceinline__ void lin_add_bias(const LinEpilogue& e, int c0, int N, uint64_t (&v)[16]) {
    if (!e.bias) return;
    if (e.bias_vec && c0 + 32 <= N) {
        if (e.bias_f32) {
            const uint4* b = reinterpret_cast<const uint4*>(static_cast<const float*>(e.bias) + c0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 u = __ldg(b + i);
#pragma unroll
                for (int j = 0; j < 2; ++j) v[2 * i + j] = f2_add(v[2 * i + j], Pairs<float>::get(u, j));
            }
        } else {
            const uint4* b = reinterpret_cast<const uint4*>(static_cast<const bf16*>(e.bias) + c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 u = __ldg(b + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * i + j] = f2_add(v[4 * i + j], Pairs<bf16>::get(u, j));
            }
        }
    } else {
        const int c = c0 + (threadIdx.x & 31);  // a lane's column, passed around
        float mine = 0.f;
        if (c < N)
            mine = e.bias_f32 ? static_cast<const float*>(e.bias)[c] : __bfloat162float(static_cast<const bf16*>(e.bias)[c]);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = f2_add(v[j], f2_pack(__shfl_sync(0xffffffffu, mine, 2 * j), __shfl_sync(0xffffffffu, mine, 2 * j + 1)));
    }
}

// A warp's 32 rows x 32 columns between its part of a box (64 bytes a row, swizzled) and
// rows in memory at any alignment: a row at a time, one column a lane.
__device__ __forceinline__ uint32_t lin_box_word(uint32_t row_addr, int r, int word) {
    return row_addr + (((word >> 2) ^ ((r >> 1) & 3)) << 4) + (word & 3) * 4;
}
__device__ __forceinline__ void lin_rows_out(uint32_t box, const uint32_t (&w)[16], bf16* out, long long ld, int row0, int rows,
                                             int c0, int N) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        st_shared_v4(lin_box_word(box + lane * 64, lane, 4 * i), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
    const int n = min(32, rows - row0);
    if (c0 + lane < N) {
        bf16* o = out + row0 * ld + c0 + lane;
#pragma unroll 8
        for (int r = 0; r < n; ++r) {
            const uint32_t u = ld_shared_4(lin_box_word(box + r * 64, r, lane >> 1));
            *reinterpret_cast<unsigned short*>(o + r * ld) = static_cast<unsigned short>(lane & 1 ? u >> 16 : u);
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void lin_rows_in(uint32_t box, uint32_t (&w)[16], const bf16* in, long long ld, int row0, int rows,
                                            int c0, int N) {
    const int lane = threadIdx.x & 31;
    const int n = min(32, rows - row0);
    const bool on = c0 + lane < N;
    const bf16* o = in + row0 * ld + c0 + lane;
    unsigned short u[32];  // every row's load under way at once
#pragma unroll
    for (int r = 0; r < 32; ++r) u[r] = on && r < n ? *reinterpret_cast<const unsigned short*>(o + r * ld) : 0;
#pragma unroll
    for (int r = 0; r < 32; ++r)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(lin_box_word(box + r * 64, r, lane >> 1) + 2 * (lane & 1)), "h"(u[r]) : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 x = ld_shared_16(lin_box_word(box + lane * 64, lane, 4 * i));
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
    __syncwarp();
}

__device__ __forceinline__ void lin_pack(const uint64_t (&v)[16], uint32_t (&w)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float lo, hi;
        f2_unpack(v[j], lo, hi);
        w[j] = pack_bf16x2(lo, hi);
    }
}

// NaN in what epilogue group g (of the 128 rows from `rofs` on) has not finished, from
// unit u on, its pair's `it`-th: what a timed-out product leaves there is no result.
__device__ __noinline__ void lin_fill_nan(const LinParams& p, int u, int it, int npairs, int g, int rofs, int et) {
    for (; u < p.units; u += npairs, ++it) {
        const LinUnit t = lin_unit(p, u);
        const LinShare s = lin_share(p, t, g, it);
        if (s.acc < 0) continue;
        const int m0 = t.m0 + rofs, n0 = t.n0 + s.col;
        const int rows = min(BM, p.M - m0), cols = min(32 * s.boxes, p.N - n0);
        for (int r = 0; r < rows; ++r)
            for (int c = et; c < cols; c += EPI_THREADS) {
                if (t.part >= 0) {
                    p.part[(static_cast<long long>(t.part) * p.rows + rofs + r) * (2 * BN) + s.col + c] = __uint_as_float(0x7fc00000u);
                } else {
                    p.e.y[static_cast<long long>(m0 + r) * p.e.ldy + n0 + c] = __ushort_as_bfloat16(0x7fc0);
                    if (p.e.pre) p.e.pre[static_cast<long long>(m0 + r) * p.e.ldpre + n0 + c] = __ushort_as_bfloat16(0x7fc0);
                }
            }
    }
}

__device__ __forceinline__ void lin_raise(const Smem& sm, int* err) {
    if (err) {
        raise_abort(sm, err);
    } else {
        *sm.abort_flag = 1;
        st_shared_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(sm.abort_flag)), cluster_ctarank() ^ 1u), 1u);
    }
}

template <int B_MN, int ACT>
__global__ void __launch_bounds__(WIDE_THREADS, 1)
    flp_linear_kernel(const __grid_constant__ CUtensorMap tmA,    // x or d, K-major (64 x 128 boxes)
                      const __grid_constant__ CUtensorMap tmB,    // W, K-major (64 x 128) or MN-major (64 x 64)
                      const __grid_constant__ CUtensorMap tmY,    // y store boxes (128 rows x 64 bytes)
                      const __grid_constant__ CUtensorMap tmPre,  // v, the same
                      const __grid_constant__ LinParams p) {
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
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmY);
        tma_prefetch_desc(&tmPre);
    }
    if (threadIdx.x == 0) griddep_launch_dependents();
    const uint32_t tmem_base =
        pair_prologue(sm, warp, 2 + 2 * EPI_THREADS, (p.width == BN ? 4 : 2) * EPI_THREADS);
    griddep_wait();  // aligned copies, d and the cleared error word are complete from here on
    const uint64_t limit = p.wait_limit_ns;
    volatile int* abort_flag = sm.abort_flag;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true, stalled = false;
            for (int u = pair; u < p.units && ok; u += npairs) {
                const LinUnit t = lin_unit(p, u);
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
                    uint8_t* b = sm.base + slot_b(true, stage);
                    const bool again = B_MN == 1 && kb >= p.fold;
                    const int at = (again ? kb - p.fold : kb) * BK;
                    tma_load_2d_pair(sm.base + slot_a(true, stage), &tmA, at, t.m0 + rofs + (again ? p.low : 0), bar);
                    for (int h = 0; h < t.halves; ++h) {
                        const int col = t.n0 + h * BN + rofs;
                        if (B_MN == 0) {
                            tma_load_2d_pair(b + h * B_STAGE_BYTES, &tmB, at, col, bar);
                        } else {
#pragma unroll
                            for (int j = 0; j < BNH / 64; ++j)
                                tma_load_2d_pair(b + h * B_STAGE_BYTES + j * 8192, &tmB, col + j * 64, at, bar);
                        }
                    }
                    if (++stage == STAGES_W) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && !stalled) lin_raise(sm, p.err);
        }
    } else if (warp == 1) {
        // ---------------------------------------------- MMA issuer (leader)
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = idesc_bf16_f32(PM, BN, 0, B_MN);
            uint32_t gk = 0;    // k-blocks consumed so far
            uint32_t uses = 0;  // bit h: parity of the uses of accumulator h so far
            bool ok = true;
            // a tile of one half, into accumulator acc
            auto single = [&](int acc, int KB) {
                if (!mbar_wait(&sm.tempty[acc], (uses >> acc & 1u) ^ 1u, limit, abort_flag)) return false;
                tc_fence_after();
                for (int kb = 0; kb < KB; ++kb, ++gk) {
                    const int s = static_cast<int>(gk % STAGES_W);
                    if (!mbar_wait(&sm.full[s], (gk / STAGES_W) & 1u, limit, abort_flag)) return false;
                    tc_fence_after();
                    const uint32_t a = smem_addr(sm.base + slot_a(true, s)), b = smem_addr(sm.base + slot_b(true, s));
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k)
                        umma_bf16_pair(tmem_base + static_cast<uint32_t>(acc * BN), operand_desc<0>(a, k), operand_desc<B_MN>(b, k),
                                       idesc, (kb > 0 || k > 0) ? 1u : 0u);
                    umma_commit_pair_mc(&sm.empty[s], PAIR_MASK);
                }
                umma_commit_pair_mc(&sm.tfull[acc], PAIR_MASK);
                uses ^= 1u << acc;
                return true;
            };
            int it = 0;
            for (int u = pair; u < p.units && ok; u += npairs, ++it) {
                const LinUnit t = lin_unit(p, u);
                const int KB = t.kb1 - t.kb0;
                if (t.halves == 0) continue;
                if (t.halves == 1) {
                    ok = single(lin_single(it), KB);
                } else {
                    ok = wide_tile_mma<B_MN>(sm, tmem_base, gk, uses & 1u, uses >> 1, KB, limit, abort_flag);
                    uses ^= 3u;
                }
            }
            if (!ok) lin_raise(sm, p.err);
            umma_commit_pair_mc(sm.drain, 0x1);  // every MMA issued so far has completed
            volatile int no_abort = 0;
            mbar_wait(sm.drain, 0, limit, &no_abort);
        }
    } else {
        // ------------------------------------------------- epilogue (lin_share)
        const int g = (warp - 2) >> 2;
        const int et = threadIdx.x - 64 - g * EPI_THREADS;  // thread 0 issues the bulk stores
        const int q = warp & 3;
        const int r = q * 32 + lane;  // accumulator row == TMEM lane
        const uint32_t bar_box = 1 + 2 * g, bar_vote = 2 + 2 * g;
        uint8_t* box0 = sm.base + SMEM_STG + g * (2 * NBOX_BYTES);
        // the warp's rows of the group's boxes, for rows that no bulk store can write (then
        // none reads the boxes)
        const uint32_t box_in = smem_addr(box0) + q * (32 * 64), box_out = box_in + NBOX_BYTES;
        StoreRing ring;
        uint32_t phase = 0;  // bit a: of accumulator a
        bool ok = true;
        int u = pair, it = 0;
        for (; u < p.units; u += npairs, ++it) {
            const LinUnit t = lin_unit(p, u);
            const LinShare share = lin_share(p, t, g, it);
            if (share.acc < 0) continue;
            const bool ready = mbar_wait(&sm.tfull[share.acc], phase >> share.acc & 1u, limit, abort_flag);
            // every thread of the group takes the same branch (the box barriers need all of them)
            if (!named_bar_all(bar_vote, EPI_THREADS, ready)) {
                ok = false;
                break;
            }
            phase ^= 1u << share.acc;
            tc_fence_after();
            const int m0 = t.m0 + rofs, n0 = t.n0 + share.col;
            const int row = m0 + r;
            const int boxes = share.boxes, ahead = p.width == BN ? BN / 64 : BN / 32;
            const uint32_t tbase = tmem_base + static_cast<uint32_t>(share.acc * BN + (p.width == BN ? share.col : 0)) +
                                   (static_cast<uint32_t>(q * 32) << 16);
            const uint32_t tempty = mapa_shared(smem_addr(&sm.tempty[share.acc]), 0);
            auto release = [&]() {
                tc_fence_before();
                mbar_arrive_cluster(tempty);
            };
            if (t.part >= 0) {
                float4* o = reinterpret_cast<float4*>(
                    p.part + (static_cast<long long>(t.part) * p.rows + rofs + r) * (2 * BN) + share.col);
#pragma unroll 1
                for (int b = 0; b < boxes; ++b) {
                    uint32_t raw[32];
                    tmem_ld_32x32b_x32(tbase + b * 32, raw);
                    tmem_wait_ld();
                    if (row < p.M) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            o[b * 8 + i] = make_float4(__uint_as_float(raw[4 * i]), __uint_as_float(raw[4 * i + 1]),
                                                       __uint_as_float(raw[4 * i + 2]), __uint_as_float(raw[4 * i + 3]));
                    }
                }
                release();
                continue;
            }
            uint4 res[4];  // the next box's residual
            auto fetch = [&](int b) {
                const int c0 = n0 + b * 32;
                const uint4* from = reinterpret_cast<const uint4*>(p.e.residual + row * p.e.ldr + c0);
#pragma unroll
                for (int i = 0; i < 4; ++i) res[i] = row < p.M && c0 + 8 * i < p.N ? from[i] : make_uint4(0, 0, 0, 0);
            };
            const bool direct_res = p.e.residual && p.e.vec;
            if (direct_res) fetch(0);
            auto drain = [&](int b, uint32_t(&raw)[32]) {
                if (b >= boxes) return;
                const int c0 = n0 + b * 32;
                uint64_t v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = f2_pack(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1]));
                lin_add_bias(p.e, c0, p.N, v);
                uint32_t w[16];
                if (p.e.pre) {
                    lin_pack(v, w);
                    if (p.e.vec)
                        narrow_box_store(ring, box0, bar_box, et, r, w, &tmPre, c0, m0, false);
                    else if (m0 + q * 32 < p.M)
                        lin_rows_out(box_out, w, p.e.pre, p.e.ldpre, m0 + q * 32, p.M, c0, p.N);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = lin_act2<ACT>(v[j]);
                if (p.e.residual) {
                    if (direct_res) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[4 * i] = res[i].x, w[4 * i + 1] = res[i].y, w[4 * i + 2] = res[i].z, w[4 * i + 3] = res[i].w;
                        if (b + 1 < boxes) fetch(b + 1);
                    } else if (m0 + q * 32 < p.M) {
                        lin_rows_in(box_in, w, p.e.residual, p.e.ldr, m0 + q * 32, p.M, c0, p.N);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = 0;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = f2_add(v[j], f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)));
                }
                lin_pack(v, w);
                if (p.e.vec)
                    narrow_box_store(ring, box0, bar_box, et, r, w, &tmY, c0, m0, false);
                else if (m0 + q * 32 < p.M)
                    lin_rows_out(box_out, w, p.e.y, p.e.ldy, m0 + q * 32, p.M, c0, p.N);
            };
            // a box ahead, so that the accumulator is free for the next tile while two boxes still
            // go through the epilogue
            uint32_t even[32], odd[32];
            auto arrived = [&](uint32_t(&x)[32]) {
                tmem_wait_ld();
                tmem_pin(x);
            };
            tmem_ld_32x32b_x32(tbase, even);
#pragma unroll 1
            for (int b = 0; b < ahead; b += 2) {
                arrived(even);
                tmem_ld_32x32b_x32(tbase + b * 32 + 32, odd);
                if (b + 2 == ahead) {
                    arrived(odd);
                    release();
                }
                drain(b, even);
                if (b + 2 < ahead) {
                    arrived(odd);
                    tmem_ld_32x32b_x32(tbase + b * 32 + 64, even);
                }
                drain(b + 1, odd);
            }
        }
        if (!ok) lin_raise(sm, p.err);
        if (et == 0) bulk_wait_group<0>();
        if (!ok) {
            named_bar_sync(bar_vote, EPI_THREADS);  // behind the group's earlier stores
            lin_fill_nan(p, u, it, npairs, g, rofs, et);
        }
    }

    pair_epilogue(sm, warp, tmem_base);
}

// Sums the partial tiles' splits in order and takes the result through the epilogue.  One
// block per row of a tile; columns a warp apart, so that any alignment coalesces.
constexpr int LJ_THREADS = 128;
__global__ void __launch_bounds__(LJ_THREADS) flp_linear_join_kernel(const __grid_constant__ LinParams p) {
    const int tile = blockIdx.x / p.rows, r = blockIdx.x % p.rows;
    const LinUnit t = lin_unit(p, p.whole + tile * p.splits);
    griddep_wait();
    const long long row = t.m0 + r;
    if (row >= p.M) return;
    const long long step = static_cast<long long>(p.rows) * (2 * BN);
    const float* from = p.part + static_cast<long long>(tile) * p.splits * step + static_cast<long long>(r) * (2 * BN);
    constexpr int C = 2 * BN / LJ_THREADS;
    float v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = 0.f;
    bool on[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = static_cast<int>(threadIdx.x) + i * LJ_THREADS;
        on[i] = at < p.width && t.n0 + at < p.N;
    }
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s)
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (on[i]) v[i] += __ldcs(from + s * step + threadIdx.x + i * LJ_THREADS);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (!on[i]) continue;
        const int c = t.n0 + static_cast<int>(threadIdx.x) + i * LJ_THREADS;
        float x = v[i];
        if (p.e.bias)
            x += p.e.bias_f32 ? static_cast<const float*>(p.e.bias)[c] : __bfloat162float(static_cast<const bf16*>(p.e.bias)[c]);
        if (p.e.pre) p.e.pre[row * p.e.ldpre + c] = __float2bfloat16_rn(x);
        x = lin_act_of(x, p.e.act);
        if (p.e.residual) x += __bfloat162float(p.e.residual[row * p.e.ldr + c]);
        p.e.y[row * p.e.ldy + c] = __float2bfloat16_rn(x);
    }
}

// ------------------------------------------------------------------ turned tiles
//
// For few rows of x: W's rows are the 128 rows of a tile and x's (up to 128, a multiple of
// 16) its columns, so that a tile moves next to nothing but W, and a CTA by itself holds
// 128 columns of y, one a thread.  The `split` CTAs of a cluster share a tile, each with a
// part of the contraction; their fp32 sums are joined through distributed shared memory,
// each CTA taking a part of the rows of x through the epilogue.  Rows that are the sum of
// two bf16 numbers meet each block of W twice.  A bounded wait that runs out makes the tile
// NaN.

constexpr int LT_THREADS = 256;
constexpr int LT_WAYS = LT_THREADS / 128;  // threads that share a column's rows of x
constexpr int LT_STAGES = 12;  // at most
constexpr int LT_MAX_T = 128;
constexpr uint32_t LT_A_BYTES = 128 * BK * 2;

struct LinTurnParams {
    int M, N;
    int KB;      // 64-deep blocks of the contraction
    int nt;      // rows of x in a tile
    int tiles_t; // tiles along the rows of x
    int split;   // CTAs of a tile
    int stages;
    uint32_t cols;  // of TMEM
    int low;        // rows from a row of x to its low part, a second number to be added, or 0
    LinEpilogue e;
    int* err;
    unsigned long long wait_limit_ns;
    int stall_after;
};

struct LinTurnShared {
    uint64_t full[LT_STAGES], empty[LT_STAGES], done, drain;
    uint32_t tmem;
    int abort, bad;  // bad: this CTA's sums are incomplete
};

// Bytes of a stage, and of the shared memory of a launch.
__host__ __device__ inline uint32_t lin_turn_stage(int nt, bool low) {
    return LT_A_BYTES + static_cast<uint32_t>(nt) * (BK * 2) * (low ? 2 : 1);
}

// Column n through the epilogue, for every LT_WAYS * split-th row of x of the tile from
// `first` on: the CTAs' sums [nt][128] added in order.
template <int ACT>
__device__ __forceinline__ void lin_turn_out(const LinTurnParams& p, uint32_t sums, int first, int n, int t0, bool bad) {
    constexpr int G = 8;  // rows under way
    const int rows = min(p.nt, p.M - t0);
    float bias = 0.f;
    if (p.e.bias)
        bias = p.e.bias_f32 ? static_cast<const float*>(p.e.bias)[n] : __bfloat162float(static_cast<const bf16*>(p.e.bias)[n]);
    if (bad) bias = __uint_as_float(0x7fc00000u);
    const int step = LT_WAYS * p.split;
    for (int c0 = first; c0 < rows; c0 += G * step) {
        float v[G], add[G];
        int c[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            c[g] = c0 + g * step;
            v[g] = add[g] = 0.f;
            if (p.e.residual && c[g] < rows) add[g] = __bfloat162float(p.e.residual[(t0 + c[g]) * p.e.ldr + n]);
        }
        for (int i = 0; i < p.split; i += 2) {
            const uint32_t one = mapa_shared(sums, i), two = mapa_shared(sums, i + 1 < p.split ? i + 1 : i);
            float u[2][G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                u[0][g] = u[1][g] = 0.f;
                if (c[g] < rows) u[0][g] = ld_cluster_f32(one + c[g] * 512);
                if (c[g] < rows && i + 1 < p.split) u[1][g] = ld_cluster_f32(two + c[g] * 512);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) v[g] = v[g] + u[0][g] + u[1][g];
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            v[g] += bias;
            if (p.e.pre && c[g] < rows) p.e.pre[(t0 + c[g]) * p.e.ldpre + n] = __float2bfloat16_rn(v[g]);
        }
#pragma unroll
        for (int g = 0; g < G; g += 2) f2_unpack(lin_act2<ACT>(f2_pack(v[g], v[g + 1])), v[g], v[g + 1]);
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (c[g] < rows) p.e.y[(t0 + c[g]) * p.e.ldy + n] = __float2bfloat16_rn(v[g] + add[g]);
    }
}

template <int A_MN>
__global__ void __launch_bounds__(LT_THREADS)
    flp_linear_turned_kernel(const __grid_constant__ CUtensorMap tmW,  // K-major (64 x 128 boxes) or MN-major (64 x 64)
                             const __grid_constant__ CUtensorMap tmX,  // K-major (64 x nt)
                             const __grid_constant__ LinTurnParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ LinTurnShared sh;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = blockIdx.x / p.split;
    const int n0 = tile / p.tiles_t * 128, t0 = tile % p.tiles_t * p.nt;
    const int kb0 = static_cast<int>(static_cast<long long>(p.KB) * rank / p.split);
    const int kb1 = static_cast<int>(static_cast<long long>(p.KB) * (rank + 1) / p.split);
    const uint32_t stage_bytes = lin_turn_stage(p.nt, p.low != 0), x_bytes = static_cast<uint32_t>(p.nt) * (BK * 2);
    volatile int* abort_flag = &sh.abort;
    const uint64_t limit = p.wait_limit_ns;
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.done, 1);
        mbar_init(&sh.drain, 1);
        sh.abort = sh.bad = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem, p.cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    griddep_wait();  // aligned copies and the cleared error word are complete from here on
    auto raise = [&]() {
        if (p.err) atomicOr(p.err, ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (p.stall_after >= 0 && kb - kb0 == p.stall_after) break;  // stop feeding the MMA
                if (!mbar_wait(&sh.empty[stage], phase ^ 1u, limit, abort_flag)) {
                    raise();
                    break;
                }
                uint8_t* a = base + stage * stage_bytes;
                mbar_arrive_expect_tx(&sh.full[stage], stage_bytes);
                if (A_MN == 0) {
                    tma_load_2d(a, &tmW, kb * BK, n0, &sh.full[stage]);
                } else {
                    tma_load_2d(a, &tmW, n0, kb * BK, &sh.full[stage]);
                    tma_load_2d(a + 8192, &tmW, n0 + 64, kb * BK, &sh.full[stage]);
                }
                tma_load_2d(a + LT_A_BYTES, &tmX, kb * BK, t0, &sh.full[stage]);
                if (p.low) tma_load_2d(a + LT_A_BYTES + x_bytes, &tmX, kb * BK, t0 + p.low, &sh.full[stage]);
                if (++stage == p.stages) stage = 0, phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16_f32(128, p.nt, A_MN, 0);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1 && ok; ++kb) {
                ok = mbar_wait(&sh.full[stage], phase, limit, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = smem_addr(base + stage * stage_bytes), b = a + LT_A_BYTES;
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k)
                    umma_bf16(tmem, operand_desc<A_MN>(a, k), operand_desc<0>(b, k), idesc, kb > kb0 || k > 0 ? 1u : 0u);
                if (p.low) {
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k)
                        umma_bf16(tmem, operand_desc<A_MN>(a, k), operand_desc<0>(b + x_bytes, k), idesc, 1u);
                }
                umma_commit(&sh.empty[stage]);
                if (++stage == p.stages) stage = 0, phase ^= 1u;
            }
            if (ok)
                umma_commit(&sh.done);
            else
                raise();
            umma_commit(&sh.drain);  // every MMA issued so far has completed
            volatile int no_abort = 0;
            mbar_wait(&sh.drain, 0, limit, &no_abort);
        }
    } else if (warp < 6) {
        const int q = warp & 3, r = q * 32 + lane;  // accumulator row == TMEM lane
        const bool ok = named_bar_all(1, EPI_THREADS, mbar_wait(&sh.done, 0, limit, abort_flag));
        if (ok) {
            tc_fence_after();
            float* part = reinterpret_cast<float*>(base);  // [nt][128]: every MMA has read its operands
            const int rows = min(p.nt, p.M - t0);
            for (int c = 0; c < rows; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + c + (static_cast<uint32_t>(q * 32) << 16), v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c + j < p.nt) part[(c + j) * 128 + r] = __uint_as_float(v[j]);
            }
        } else {
            raise();
            sh.bad = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (p.split > 1) cluster_sync();  // every CTA's sums are there
    const int r = threadIdx.x % 128, n = n0 + r;
    if (n < p.N) {
        uint32_t bad = 0;
        for (int i = 0; i < p.split; ++i) bad |= ld_cluster_u32(mapa_shared(smem_addr(&sh.bad), i));
        const uint32_t sums = smem_addr(base) + r * 4;
        const int first = rank + static_cast<int>(threadIdx.x) / 128 * p.split;
        switch (p.e.act) {
            case LIN_RELU: lin_turn_out<LIN_RELU>(p, sums, first, n, t0, bad); break;
            case LIN_GELU: lin_turn_out<LIN_GELU>(p, sums, first, n, t0, bad); break;
            case LIN_GELU_TANH: lin_turn_out<LIN_GELU_TANH>(p, sums, first, n, t0, bad); break;
            case LIN_SILU: lin_turn_out<LIN_SILU>(p, sums, first, n, t0, bad); break;
            default: lin_turn_out<LIN_NONE>(p, sums, first, n, t0, bad);
        }
    }
    if (*abort_flag) {  // copies in flight get a bounded grace period
        const uint64_t start = globaltimer_ns();
        while (globaltimer_ns() - start < 2000000ull) {
        }
    }
    __syncthreads();
    if (p.split > 1) cluster_sync();  // no CTA leaves while its sums are read
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.cols);
    }
}

// ------------------------------------------------------------------ one row
//
// One row of x: W is read once, at the pace of memory.  A warp takes R rows of W at a time,
// 8 elements a lane, and keeps their sums in pairs; x, read again for every R rows, comes
// from the caches.  Where W has too few rows for all warps, KW warps of a block share rows
// and split the contraction.

struct LinRowParams {
    const bf16* x;
    const bf16* w;
    long long ldw;
    int N, K;
    int kw;     // warps that share rows: 1, 2, 4, 8
    int chunk;  // of the contraction, each such warp's: a multiple of 256
    LinEpilogue e;
};

constexpr int LR_THREADS = 256;
constexpr int LR_WARPS = LR_THREADS / 32;
constexpr int LR_ROWS = 4;
constexpr int LR_STEPS = 2;  // of 256 elements, under way at once

template <bool LOOSE>
__global__ void __launch_bounds__(LR_THREADS) flp_linear_row_kernel(const __grid_constant__ LinRowParams p) {
    constexpr int R = LR_ROWS, U = LR_STEPS;
    __shared__ __align__(16) uint8_t words[LOOSE ? LR_WARPS * WARP_WORDS_BYTES : 16];
    __shared__ float sums[LR_WARPS][R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage = smem_addr(words) + (LOOSE ? warp * WARP_WORDS_BYTES : 0);
    const int teams = LR_WARPS / p.kw, team = warp / p.kw, part = warp % p.kw;
    const int n0 = (blockIdx.x * teams + team) * R;
    const int k0 = part * p.chunk, k1 = min(p.K, k0 + p.chunk);
    griddep_wait();  // an aligned copy of x
    uint64_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0;
    const Extent all = extent_of<bf16>(p.w, p.N, p.ldw, p.K);
    if (n0 < p.N) {
        for (int k = k0; k < k1; k += 256 * U) {
            uint32_t w[U][R][WarpWords<bf16>::N];
            const bf16* src[U][R];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int n = min(n0 + r, p.N - 1), at = k + u * 256 + lane * 8, left = k1 - at;
                    src[u][r] = p.w + n * p.ldw + at;
                    if constexpr (LOOSE) {
                        load_words<bf16>(w[u][r], src[u][r], left, n == 0 || n == p.N - 1, all);
                    } else {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (left > 0) v = __ldcs(reinterpret_cast<const uint4*>(src[u][r]));
                        w[u][r][0] = v.x, w[u][r][1] = v.y, w[u][r][2] = v.z, w[u][r][3] = v.w;
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k + u * 256 + lane * 8, left = k1 - at;
                // x is aligned and padded to vectors; what lies behind K is zero in a padded
                // copy, and meets zeros of W
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (left > 0) xv = __ldg(reinterpret_cast<const uint4*>(p.x + at));
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    uint4 v;
                    if constexpr (LOOSE)
                        v = settle_words<bf16>(w[u][r], src[u][r], left, stage);
                    else
                        v = make_uint4(w[u][r][0], w[u][r][1], w[u][r][2], w[u][r][3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[r] = f2_fma(Pairs<bf16>::get(v, j), Pairs<bf16>::get(xv, j), acc[r]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float s = warp_sum(f2_sum(acc[r]));
        if (lane == 0) sums[warp][r] = s;
    }
    __syncthreads();
    // one thread per output of the block
    const int j = threadIdx.x, c = blockIdx.x * teams * R + j;
    if (j >= teams * R || c >= p.N) return;
    float v = 0.f;
    for (int q = 0; q < p.kw; ++q) v += sums[j / R * p.kw + q][j % R];
    if (p.e.bias)
        v += p.e.bias_f32 ? static_cast<const float*>(p.e.bias)[c] : __bfloat162float(static_cast<const bf16*>(p.e.bias)[c]);
    if (p.e.pre) p.e.pre[c] = __float2bfloat16_rn(v);
    v = lin_act_of(v, p.e.act);
    if (p.e.residual) v += __bfloat162float(p.e.residual[c]);
    p.e.y[c] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ d and db

struct LinGradParams {
    const bf16* dy;
    long long lddy;
    const bf16* pre;  // with an activation
    long long ldpre;
    int M, N;
    bf16* d;   // [M, Np], or null: not written
    bf16* lo;  // what the rounding to bf16 takes from it, or null
    int Np;
    float* part;  // [row blocks][N]: column sums, or null
    int rows;     // of a row block
};

constexpr int LG_THREADS = 256;
constexpr int LG_WARPS = LG_THREADS / 32;
constexpr int LG_ROWS = 4;  // rows a warp has under way

// What the high numbers leave of d; nothing where one is infinite (inf - inf would be NaN,
// and the products infinite by it alone).
__device__ __forceinline__ uint64_t lin_rest(uint64_t hi, uint64_t d) {
    float h0, h1, r0, r1;
    f2_unpack(hi, h0, h1);
    f2_unpack(f2_fma(hi, f2_splat(-1.f), d), r0, r1);
    return f2_pack(fabsf(h0) == INFINITY ? 0.f : r0, fabsf(h1) == INFINITY ? 0.f : r1);
}

// 256 columns x `rows` rows a block, a row at a time a warp.
template <bool LOOSE, int ACT>
__global__ void __launch_bounds__(LG_THREADS, LOOSE ? 2 : 4) flp_linear_grad_kernel(const __grid_constant__ LinGradParams p) {
    constexpr int P = 4;
    __shared__ __align__(16) uint8_t words[LOOSE ? LG_WARPS * WARP_WORDS_BYTES : 16];
    __shared__ float sums[LG_WARPS][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage = smem_addr(words) + (LOOSE ? warp * WARP_WORDS_BYTES : 0);
    const int col = blockIdx.x * 256 + lane * 8, left = p.N - col;
    const int first = blockIdx.y * p.rows, last = first + min(p.rows, p.M - first);
    griddep_launch_dependents();
    const Extent all_dy = extent_of<bf16>(p.dy, p.M, p.lddy, p.N), all_pre = extent_of<bf16>(p.pre, p.M, p.ldpre, p.N);
    uint64_t sum[P] = {0, 0, 0, 0};
    for (int r0 = first + warp; r0 < last; r0 += LG_WARPS * LG_ROWS) {
        uint32_t a[LG_ROWS][WarpWords<bf16>::N], b[LG_ROWS][WarpWords<bf16>::N];
        auto fetch = [&](uint32_t(&x)[WarpWords<bf16>::N], const bf16* src, bool on, bool edge, const Extent& all) {
            if constexpr (LOOSE) {
                load_words<bf16>(x, src, on ? left : -256, edge, all);
            } else {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (on && left > 0) u = __ldcs(reinterpret_cast<const uint4*>(src));
                x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            }
        };
        auto value = [&](const uint32_t(&x)[WarpWords<bf16>::N], const bf16* src) {
            if constexpr (LOOSE)
                return settle_words<bf16>(x, src, left, stage);
            else
                return make_uint4(x[0], x[1], x[2], x[3]);
        };
#pragma unroll
        for (int i = 0; i < LG_ROWS; ++i) {
            const int r = r0 + i * LG_WARPS;
            const bool on = r < last, edge = r == 0 || r == p.M - 1;
            fetch(a[i], p.dy + r * p.lddy + col, on, edge, all_dy);
            if (ACT != LIN_NONE) fetch(b[i], p.pre + r * p.ldpre + col, on, edge, all_pre);
        }
#pragma unroll
        for (int i = 0; i < LG_ROWS; ++i) {
            const int r = r0 + i * LG_WARPS;
            if (r >= last) break;  // the whole warp
            const uint4 u = value(a[i], p.dy + r * p.lddy + col);
            uint64_t d[P];
#pragma unroll
            for (int j = 0; j < P; ++j) d[j] = Pairs<bf16>::get(u, j);
            if constexpr (ACT != LIN_NONE) {
                const uint4 x = value(b[i], p.pre + r * p.ldpre + col);
#pragma unroll
                for (int j = 0; j < P; ++j) d[j] = f2_mul(d[j], lin_slope2<ACT>(Pairs<bf16>::get(x, j)));
            }
            if (p.d) {
                const uint4 hi = Pairs<bf16>::put(d);
                const long long at = static_cast<long long>(r) * p.Np + col;
                st_global_16(p.d + at, hi, left > 0);
                if (p.lo) {
                    uint64_t rest[P];
#pragma unroll
                    for (int j = 0; j < P; ++j) rest[j] = lin_rest(Pairs<bf16>::get(hi, j), d[j]);
                    st_global_16(p.lo + at, Pairs<bf16>::put(rest), left > 0);
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) sum[j] = f2_add(sum[j], d[j]);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < P; ++j) f2_unpack(sum[j], sums[warp][lane * 8 + 2 * j], sums[warp][lane * 8 + 2 * j + 1]);
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.N) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < LG_WARPS; ++w) s += sums[w][threadIdx.x];
    p.part[static_cast<long long>(blockIdx.y) * p.N + c] = s;
}

// db from the row blocks' sums, in order.
constexpr int LB_WAYS = 32;
__global__ void __launch_bounds__(32 * LB_WAYS) flp_linear_bias_join_kernel(const float* part, int blocks, int N, float* db) {
    __shared__ float sums[LB_WAYS][33];
    const int lane = threadIdx.x & 31, way = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    griddep_launch_dependents();
    griddep_wait();
    float s = 0.f;
    if (c < N)
        for (int b = way; b < blocks; b += LB_WAYS) s += part[static_cast<long long>(b) * N + c];
    sums[way][lane] = s;
    __syncthreads();
    if (way == 0 && c < N) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < LB_WAYS; ++w) s += sums[w][lane];
        db[c] = s;
    }
}

}  // namespace flp

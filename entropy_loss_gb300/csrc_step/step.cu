// step.cu - host side of the first training-step operators declared in
// include/flp.h: argument checks, kernel choice by size and alignment, and
// launches.
#include "balance.cuh"
#include "checkpoint.cuh"
#include "norm.cuh"
#include "step_host.cuh"
#include "wgrad.cuh"

namespace {

using namespace flp;

// ------------------------------------------------------------------ layer norm

inline int64_t ck_cols(int64_t H) { return cdiv(H, CK_BLOCK) * CK_BLOCK; }

// Streaming rows: calls f(shape, threads of a block).  16 elements a thread keep
// a row, its parameters and the column sums in registers while its fixed work per
// row (about 130 instructions) is spread over enough of them: 8 elements a thread
// (twice the warps) took 12 to 50 % longer at 32768 x 4096, 32 (half the warps)
// 17 to 130 %.  Rows of up to 512 elements go to one warp, which needs no block
// barrier; rows above 8192 take more elements a thread.  Two blocks of up to TWO
// threads must fit an SM, which bounds the registers (three of up to 256: forward
// with a checkpoint 118 against 105 us, backward 239 against 127 us).  For the bf16
// forward that pays up to 512 threads, although the loose form of 512 spills: two
// blocks of 384 threads instead of one take 16384 x 6144 from 79 to 64 us, with a
// checkpoint from 94 to 82 us (fp32 from 124 to 134; loose rows with a checkpoint,
// 20000 x 6001, from 204 to 233), two of 512 take 16384 x 8192 from 95 to 83 us (with
// a checkpoint from 112 to 153).  The stages put 32 to 64 KiB per SM in flight.
template <int NV_, int S_, bool WARP_, int MAXT_, int MINB_>
struct StreamShape {
    static constexpr int NV = NV_, S = S_, MAXT = MAXT_, MINB = MINB_;
    static constexpr bool WARP = WARP_;
};

// Shared memory of `vecs` staged vectors per thread, beside them nothing (x: 0), as
// many of a second matrix (1) or of its checkpoint (2).
template <typename T, bool LOOSE>
size_t norm_stage_bytes(int vecs, int threads, int x) {
    const int one = Stage<T, LOOSE>::bytes(threads);
    return static_cast<size_t>(vecs) * (one + (x == 0 ? 0 : x == 1 ? one : threads * wide_v<T>()));
}

template <typename T, int TWO, int S16, typename F>
flp_status norm_stream_shape(int64_t cols, F&& f) {
    constexpr int V = wide_v<T>(), N2 = 16 / V;  // N2 vectors of V = 16 elements
    constexpr int S = V == 8 ? S16 : 2;          // S16: stages of bf16 rows
    const int64_t vecs = cdiv(cols, V);
    if (vecs <= 32) return f(StreamShape<1, 4, true, 256, 1>{}, 256);
    if (vecs <= 64) return f(StreamShape<2, 4, true, 256, 1>{}, 256);
    if constexpr (V == 4)
        if (vecs <= 128) return f(StreamShape<4, 2, true, 256, 1>{}, 256);
    const int threads = static_cast<int>(cdiv(vecs, 32 * N2) * 32);
    if (threads <= 256) return f(StreamShape<N2, S, false, 256, 2>{}, threads);
    if (threads <= 320) return f(StreamShape<N2, S, false, 320, 2>{}, threads);
    if constexpr (TWO >= 384)
        if (threads <= 384) return f(StreamShape<N2, S, false, 384, 2>{}, threads);
    if (threads <= 512) return f(StreamShape<N2, S, false, 512, TWO >= 512 ? 2 : 1>{}, threads);
    return f(StreamShape<2 * N2, 2, false, 512, 1>{}, static_cast<int>(cdiv(vecs, 64 * N2) * 32));
}

flp_status norm_checks(int64_t M, int64_t H, int dtype, int param_dtype, const void* weight, const void* bias) {
    if (M < 0 || H < 1) return fail(FLP_ERR_INVALID_ARG, "M >= 0 and H >= 1 required");
    if (!is_dtype(dtype) || !is_dtype(param_dtype)) return fail(FLP_ERR_INVALID_ARG, "dtypes are FLP_F32 or FLP_BF16");
    if (M > kMaxRows) return fail(FLP_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    if (H > NORM_MAX_H) return fail(FLP_ERR_UNSUPPORTED, "layer norm rows hold at most 16384 elements");
    if (!aligned_to(weight, elem(param_dtype)) || !aligned_to(bias, elem(param_dtype)))
        return fail(FLP_ERR_INVALID_ARG, "weight and bias must be aligned to their elements");
    return FLP_OK;
}

flp_status ck_checks(const void* q, const void* scale) {
    if (!q || !scale) return fail(FLP_ERR_INVALID_ARG, "a checkpoint needs both q and scale");
    if (!aligned16(q)) return fail(FLP_ERR_INVALID_ARG, "checkpoint q must be 16-byte aligned");
    return FLP_OK;
}

// Blocks of a streaming grid: as many as the rows fill, or fit the device.  A group takes
// a second row in the second case alone, `blocks` times the block's rows further on: an
// even number, so that a loose bf16 row of an odd pitch starts at the parity of the one
// before (the SMs come in pairs).
int64_t norm_blocks(int64_t M, int64_t rows_per_block, int sm_count, int64_t blocks_per_sm) {
    return std::max<int64_t>(1, std::min(cdiv(M, rows_per_block), sm_count / 2 * 2 * blocks_per_sm));
}

// Few rows: one cluster of blocks joins its column sums through distributed shared
// memory, without the workspace and the second launch (a row per warp up to 512
// columns, else per block).  A call takes 20 us instead of 23.  On the GPU it is the
// faster form up to 64 rows of 512 columns or fewer and 16 rows of 4096 or more; the
// rule goes on while it takes at most 1 us more (256 x 256 4.8 against 4.0, 256 x 512
// 6.1 against 4.9, 16 x 1024 4.4 against 3.7, 16 x 8192 7.9 against 10.1; twice as many
// rows 5.9 against 4.2, 7.7 against 5.1, 5.2 against 3.8, 9.7 against 10.4, but fp32 10.4
// against 7.8).  Above 8192 columns the sums do not fit beside the rows.
constexpr int kNormBwdCluster = 8;
bool norm_bwd_cluster(int64_t M, int64_t H) { return M <= kNormBwdCluster * (H <= 512 ? 32 : 2) && H <= 8192; }

// The backward's kernel for rows of H columns: calls f(kernel, form), form being what a
// launch of it needs.
struct NormBwdForm {
    int threads;
    int64_t rows;   // of a block at a time
    size_t staged;  // shared memory of the rows under way
    size_t join;    // and of the warps' sums of a cluster's block, before its own 8 H bytes
    size_t most;    // what the kernel's largest block needs
};
template <auto* K>
struct NormBwdKernel {
    static constexpr auto* kernel = K;
};

template <typename T, bool CK, bool LOOSE, typename F>
flp_status norm_bwd_form(int64_t H, F&& f) {
    return norm_stream_shape<T, 320, 4>(H, [&](auto shape, int threads) -> flp_status {
        using X = decltype(shape);
        // above 8192 columns one stage fits beside the weights and sums, or two of aligned
        // bf16 rows with a checkpoint (8192 x 8200 118 us, one stage: 133); two of bf16
        // also where the sums of dy wait there in narrower rows (norm_bwd_db_shared)
        constexpr bool WIDE = norm_bwd_wide<T, X::NV>(), B16 = sizeof(T) == 2;
        constexpr bool DB_SHARED = norm_bwd_db_shared<T, X::NV, X::MAXT, CK, LOOSE>();
        constexpr int S = WIDE && !(CK && !LOOSE && B16) ? 1 : B16 && DB_SHARED ? 2 : X::S;
        constexpr auto* kernel = flp_norm_bwd_stream_kernel<T, X::NV, S, CK, LOOSE, X::WARP, X::MAXT, X::MINB>;
        // a cluster's block holds its warps' sums (a row per warp) and its own after the rows
        constexpr size_t kJoin = X::WARP ? static_cast<size_t>(X::MAXT) * X::NV * wide_v<T>() * 4 : 0;
        constexpr size_t kMostSums = WIDE ? 0 : kJoin + 8ull * (X::WARP ? 32 : X::MAXT) * X::NV * wide_v<T>();
        NormBwdForm form;
        form.threads = threads;
        form.rows = X::WARP ? threads / 32 : 1;
        form.staged = norm_stage_bytes<T, LOOSE>(S * X::NV, threads, CK ? 2 : 1);
        form.join = kJoin;
        form.most = std::max(norm_stage_bytes<T, LOOSE>(S * X::NV, X::MAXT, CK ? 2 : 1), kMostSums);
        return f(NormBwdKernel<kernel>{}, form);
    });
}

// Blocks of the backward's grid in any of its forms (either type, from X or from its
// checkpoint, aligned or loose rows): what the workspace query allows for.
flp_status norm_bwd_most_blocks(int64_t M, int64_t H, int sm_count, int64_t* most) {
    *most = 0;
    auto one = [&](auto t, auto ck, auto loose) {
        return norm_bwd_form<decltype(t), decltype(ck)::value, decltype(loose)::value>(
            H, [&](auto k, const NormBwdForm& form) -> flp_status {
                int per_sm = 0;
                const flp_status st = resident_blocks<decltype(k)::kernel>(form.threads, form.staged, form.most, &per_sm);
                *most = std::max(*most, norm_blocks(M, form.rows, sm_count, per_sm));
                return st;
            });
    };
    auto rows = [&](auto t, auto ck) {
        const flp_status st = one(t, ck, std::true_type{});
        return st == FLP_OK ? one(t, ck, std::false_type{}) : st;
    };
    auto typed = [&](auto t) {
        const flp_status st = rows(t, std::true_type{});
        return st == FLP_OK ? rows(t, std::false_type{}) : st;
    };
    const flp_status st = typed(bf16{});
    return st == FLP_OK ? typed(float{}) : st;
}

// -------------------------------------------------------------- weight gradient

struct WgradPlan {
    int64_t Kp;          // padded columns of X^
    int64_t Np;          // pitch of the aligned copy of dY (0: read in place)
    int tn, tk, whole, rest, splits, units;
    size_t off_x, off_y, off_part, bytes;
};

// Whole rounds of tiles go straight to dW; the rest are split into the number
// of runs that costs least, in the time of a 64-row block of a tile (0.54 us):
// the blocks of a run, and for joining 5 (a launch) and a quarter per partial
// tile (512 KiB written and read back).
// `unpack`: X^ comes from a checkpoint and lies in the workspace.
WgradPlan plan_wgrad(const void* dY, int64_t lddy, int64_t M, int64_t N, int64_t K, int dw_dtype, int pairs,
                     bool unpack = true) {
    WgradPlan w{};
    pairs = std::max(1, pairs);
    w.Kp = ck_cols(K);
    w.Np = rows16(dY, lddy, FLP_BF16) ? 0 : cdiv(N, 8) * 8;
    w.tn = static_cast<int>(cdiv(N, PM));
    w.tk = static_cast<int>(cdiv(K, 2 * BN));
    const int64_t tiles = static_cast<int64_t>(w.tn) * w.tk;
    const int64_t KB = std::max<int64_t>(1, cdiv(M, BK));
    // a TMA store's row pitch; and a bf16 result of many rows is joined from fp32 sums
    const bool direct = (K * elem(dw_dtype)) % 16 == 0 && !(dw_dtype == FLP_BF16 && KB > WGRAD_BF16_RUN);
    w.whole = direct ? static_cast<int>(tiles / pairs * pairs) : 0;
    int64_t rest = tiles - w.whole;
    w.splits = 1;
    if (rest > 0) {
        double best = 1e300;
        const int64_t most = std::min<int64_t>(KB, std::max<int64_t>(1, 4 * pairs / std::max<int64_t>(1, rest)));
        for (int64_t s = 1; s <= std::max<int64_t>(1, most); ++s) {
            const double joined = s > 1 || !direct ? 5.0 + 0.25 * static_cast<double>(rest * s) : 0.0;
            const double cost = static_cast<double>(cdiv(rest * s, pairs) * cdiv(KB, s)) + joined;
            if (cost < best - 1e-9) {
                best = cost;
                w.splits = static_cast<int>(s);
            }
        }
        if (w.splits == 1 && direct) {
            w.whole = static_cast<int>(tiles);
            rest = 0;
        }
    }
    w.rest = static_cast<int>(rest);
    w.units = w.whole + w.rest * w.splits;
    w.off_x = kHeaderBytes;
    w.off_y = w.off_x + (unpack ? align_up(static_cast<size_t>(std::max<int64_t>(M, 1)) * w.Kp * 2, 1024) : 0);
    w.off_part = w.off_y + align_up(static_cast<size_t>(M) * w.Np * 2, 1024);
    w.bytes = w.off_part + static_cast<size_t>(w.rest) * w.splits * PM * 2 * BN * 4;
    return w;
}

flp_status wgrad_checks(const void* dY, int64_t lddy, int64_t M, int64_t N, int64_t K, int dw_dtype) {
    if (M < 0 || N < 1 || K < 1) return fail(FLP_ERR_INVALID_ARG, "M >= 0, N >= 1 and K >= 1 required");
    if (M > kMaxRows - 256 || N > kMaxRows - 1024 || K > kMaxRows - 1024 ||
        cdiv(N, PM) * cdiv(K, 2 * BN) >= (1 << 23))  // partial tiles: below 2^31 rows (more than 4 x pairs are not split)
        return fail(FLP_ERR_UNSUPPORTED, "sizes beyond the 32-bit tiling");
    if (!is_dtype(dw_dtype)) return fail(FLP_ERR_INVALID_ARG, "dW_dtype is FLP_F32 or FLP_BF16");
    if (M > 0 && lddy < N) return fail(FLP_ERR_INVALID_ARG, "row pitch of dY below N");
    if (!aligned_to(dY, 2)) return fail(FLP_ERR_INVALID_ARG, "dY must be aligned to its elements");
    return FLP_OK;
}

// Equal runs of at most WGRAD_RUN blocks.
int wgrad_run(int64_t M) {
    const int64_t KB = cdiv(M, BK);
    return static_cast<int>(cdiv(KB, cdiv(KB, WGRAD_RUN)));
}

// The contraction's shared memory, once per device.
flp_status wgrad_attrs() {
    static bool done[kMaxDevices] = {};
    int dev = 0;
    FLP_CUDA(cudaGetDevice(&dev));  // in range: check_device has run
    std::lock_guard<std::mutex> lk(g_mu);
    if (!done[dev]) {
        FLP_CUDA(cudaFuncSetAttribute(flp_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC));
        done[dev] = true;
    }
    return FLP_OK;
}

// The contraction and the join, dY (pitch ldy) and X^ (cols columns, pitch ldx) being there.
flp_status wgrad_contract(const WgradPlan& w, const void* y, int64_t ldy, const void* x, int64_t cols, int64_t ldx,
                          uint8_t* ws, int64_t M, int64_t N, int64_t K, void* dW, int dw_dtype, int accumulate, int pairs,
                          int run, unsigned long long wait_limit_ns, int stall_after, bool after_kernel, cudaStream_t s) {
    flp_status st;
    const int64_t es = elem(dw_dtype);
    const bool b16 = dw_dtype == FLP_BF16;
    CUtensorMap my, mx, mw, mp;
    if ((st = tmap_2d(&my, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, ldy * 2, 64, 64)) != FLP_OK) return st;
    if ((st = tmap_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, cols, M, ldx * 2, 64, 64)) != FLP_OK) return st;
    const size_t part_rows = static_cast<size_t>(w.rest) * w.splits * PM;
    // without split tiles (or without whole ones) one of the two output maps is
    // not used: it repeats the other
    if (w.rest &&
        (st = tmap_2d(&mp, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + w.off_part, 2 * BN, part_rows, 2 * BN * 4, 16, BM,
                      CU_TENSOR_MAP_SWIZZLE_64B)) != FLP_OK)
        return st;
    if (w.whole &&
        (st = tmap_2d(&mw, b16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dW, K, N, K * es,
                      b16 ? 32 : 16, BM, CU_TENSOR_MAP_SWIZZLE_64B)) != FLP_OK)
        return st;
    if (!w.rest) mp = mw;
    if (!w.whole) mw = mp;
    WgradParams p{};
    p.tn = w.tn;
    p.tk = w.tk;
    p.group = std::min(w.tn, 8);
    p.whole = w.whole;
    p.splits = w.splits;
    p.units = w.units;
    p.KB = static_cast<int>(cdiv(M, BK));
    p.run = run;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.add = accumulate ? 1 : 0;
    p.bf16_out = b16 ? 1 : 0;
    p.err = reinterpret_cast<int*>(ws);
    p.wait_limit_ns = wait_limit_ns;
    p.stall_after = stall_after;
    const int grid = 2 * static_cast<int>(std::min<int64_t>(w.units, pairs));
    st = launch_pairs_n(flp_wgrad_kernel, grid, WIDE_THREADS, s, "flp_wgrad_kernel launch", after_kernel, my, mx, mw, mp, p, dW);
    if (st != FLP_OK || !w.rest) return st;
    WgradJoinParams j{};
    j.part = reinterpret_cast<const float*>(ws + w.off_part);
    j.g = p;
    j.dw = dW;
    j.add = p.add;
    j.err = p.err;
    return launch_step(flp_wgrad_join_kernel, static_cast<int64_t>(w.rest) * (PM / WJ_ROWS), WJ_THREADS, 0, s,
                       "flp_wgrad_join_kernel launch", true, j);
}

// How the vectors of V elements of the rows in p are dealt to threads, `each` per thread.
flp_status ck_places(CkParams& p, int V, bool loose, int each, int64_t* grid) {
    p.per_row = static_cast<unsigned>(loose ? cdiv(p.Hp / V, 32) * 32 : p.Hp / V);
    p.inverse = ~0ull / p.per_row + 1;
    const int64_t total = p.M * p.per_row;
    *grid = cdiv(total, CK_THREADS * each);
    // the row of a vector comes exactly from one multiplication while vectors x vectors per row < 2^64
    if (*grid > INT32_MAX || static_cast<double>(total + (1 << 20)) * p.per_row > 1.8e19)
        return fail(FLP_ERR_UNSUPPORTED, "matrix too large for one launch");
    return FLP_OK;
}

template <typename T, bool LOOSE>
flp_status ck_launch(bool pack, void* x, int64_t ldx, const void* q, const void* scale, int64_t M, int64_t H,
                     cudaStream_t s, int* clear = nullptr) {
    constexpr int V = wide_v<T>();
    CkParams p{};
    p.x = x;
    p.ldx = ldx;
    p.q = static_cast<uint8_t*>(const_cast<void*>(q));
    p.scale = static_cast<uint8_t*>(const_cast<void*>(scale));
    p.M = M;
    p.H = static_cast<int>(H);
    p.Hp = static_cast<int>(ck_cols(H));
    p.clear = clear;
    int64_t grid = 0;
    const flp_status st = ck_places(p, V, LOOSE, pack ? CK_PACK_N : CK_UNPACK_N, &grid);
    if (st != FLP_OK) return st;
    return pack ? launch_step(flp_ck_pack_kernel<T, LOOSE>, grid, CK_THREADS, 0, s, "flp_ck_pack_kernel launch", false, p)
                : launch_step(flp_ck_unpack_kernel<T, LOOSE>, grid, CK_THREADS, 0, s, "flp_ck_unpack_kernel launch",
                              false, p);
}

flp_status ck_run(bool pack, const void* x, int64_t ldx, int dtype, const void* q, const void* scale, int64_t M,
                  int64_t H, cudaStream_t s) {
    if (M < 0 || H < 1) return fail(FLP_ERR_INVALID_ARG, "M >= 0 and H >= 1 required");
    if (!is_dtype(dtype)) return fail(FLP_ERR_INVALID_ARG, "dtype is FLP_F32 or FLP_BF16");
    if (H > INT32_MAX - CK_BLOCK) return fail(FLP_ERR_UNSUPPORTED, "rows of more than 2^31 elements");
    if (M == 0) return FLP_OK;
    flp_status st = ck_checks(q, scale);
    if (st == FLP_OK) st = row_checks(x, ldx, H, dtype, "X must be non-null");
    DevInfo* d;
    if (st == FLP_OK) st = step_device(&d);
    if (st == FLP_OK) st = check_on_current_device(x, "X");
    if (st != FLP_OK) return st;
    void* xx = const_cast<void*>(x);
    const bool loose = !(rows16(x, ldx, dtype) && (H * elem(dtype)) % 16 == 0);
    auto typed = [&](auto t) {
        using T = decltype(t);
        return loose ? ck_launch<T, true>(pack, xx, ldx, q, scale, M, H, s)
                     : ck_launch<T, false>(pack, xx, ldx, q, scale, M, H, s);
    };
    return dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
}

// ----------------------------------------------------------------- balance loss

// Calls f(lanes per row, experts per lane, experts per access) for E experts;
// `vec`: rows are aligned to four elements and hold a multiple of four.
template <typename F>
flp_status balance_shape(int64_t E, bool vec, F&& f) {
#define FLP_SHAPE(L, NE, V)    \
    if (E <= (L) * (NE))       \
        return f(std::integral_constant<int, L>{}, std::integral_constant<int, NE>{}, std::integral_constant<int, V>{});
    FLP_SHAPE(8, 1, 1)
    FLP_SHAPE(16, 1, 1)
    FLP_SHAPE(32, 1, 1)
    if (vec) {
        FLP_SHAPE(32, 2, 2)
        FLP_SHAPE(32, 4, 4)
        FLP_SHAPE(32, 8, 4)
        FLP_SHAPE(32, 16, 4)
        FLP_SHAPE(32, 32, 4)
    } else {
        FLP_SHAPE(32, 2, 1)
        FLP_SHAPE(32, 4, 1)
        FLP_SHAPE(32, 8, 1)
        FLP_SHAPE(32, 16, 1)
        FLP_SHAPE(32, 32, 1)
    }
#undef FLP_SHAPE
    return fail(FLP_ERR_UNSUPPORTED, "at most 1024 experts");
}

constexpr int64_t kBalanceBlocksPerSm = 2;

struct BalancePlan {
    int64_t blocks;
    bool cluster;  // one launch of one cluster
    size_t off_p, off_c, off_n, off_tp, off_tc, off_tn, bytes;
};

BalancePlan plan_balance(int64_t T, int64_t E, int sm_count) {
    BalancePlan b{};
    const int64_t lanes = E <= 8 ? 8 : E <= 16 ? 16 : 32;
    const int64_t rows = BAL_THREADS / lanes;
    b.cluster = cdiv(T, rows) <= BAL_CLUSTER * BAL_CLUSTER_TRIPS;
    b.blocks = std::max<int64_t>(1, std::min(cdiv(T, rows), sm_count * kBalanceBlocksPerSm));
    if (b.cluster) return b;  // no workspace: everything is in shared memory
    size_t at = align_up(static_cast<size_t>(T) * 8, 256);  // the rows' statistics first
    auto take = [&](size_t n) {
        const size_t here = at;
        at += align_up(n, 256);
        return here;
    };
    b.off_p = take(static_cast<size_t>(b.blocks) * E * 4);
    b.off_c = take(static_cast<size_t>(b.blocks) * E * 4);
    b.off_n = take(static_cast<size_t>(b.blocks) * 4);
    b.off_tp = take(static_cast<size_t>(E) * 8);
    b.off_tc = take(static_cast<size_t>(E) * 8);
    b.off_tn = take(8);
    b.bytes = at;
    return b;
}

flp_status balance_checks(int64_t T, int64_t E, int64_t top_k) {
    if (T < 0 || E < 1) return fail(FLP_ERR_INVALID_ARG, "T >= 0 and E >= 1 required");
    if (top_k < 1 || top_k > E) return fail(FLP_ERR_INVALID_ARG, "1 <= top_k <= E required");
    if (E > BAL_MAX_E) return fail(FLP_ERR_UNSUPPORTED, "at most 1024 experts");
    if (T > kMaxRows) return fail(FLP_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    return FLP_OK;
}

}  // namespace

// ------------------------------------------------- for the library's other units

flp_status flp::align_rows(const void* src, int64_t ld, int64_t M, int64_t H, void* dst, int64_t Hp, cudaStream_t s) {
    CkParams a{};
    a.x = const_cast<void*>(src);
    a.ldx = ld;
    a.q = static_cast<uint8_t*>(dst);
    a.M = M;
    a.H = static_cast<int>(H);
    a.Hp = static_cast<int>(Hp);
    int64_t grid = 0;
    const flp_status st = ck_places(a, 8, true, CK_PACK_N, &grid);
    if (st != FLP_OK) return st;
    return launch_step(flp_align_rows_kernel, grid, CK_THREADS, 0, s, "flp_align_rows_kernel launch", false, a);
}

flp_status flp::weight_grad_checks(int64_t M, int64_t N, int64_t K, int dw_dtype) {
    return wgrad_checks(nullptr, N, M, N, K, dw_dtype);
}

size_t flp::weight_grad_bytes(int64_t M, int64_t N, int64_t K, int dw_dtype, int pairs) {
    return plan_wgrad(nullptr, cdiv(N, 8) * 8, M, N, K, dw_dtype, pairs, false).bytes;
}

flp_status flp::weight_grad(const void* dY, int64_t ldy, const void* X, int64_t ldx, int64_t M, int64_t N, int64_t K,
                            void* dW, int dw_dtype, int accumulate, uint8_t* ws, int pairs, bool after_kernel,
                            cudaStream_t s) {
    const flp_status st = wgrad_attrs();
    if (st != FLP_OK) return st;
    const WgradPlan w = plan_wgrad(dY, ldy, M, N, K, dw_dtype, pairs, false);
    return wgrad_contract(w, dY, ldy, X, K, ldx, ws, M, N, K, dW, dw_dtype, accumulate, pairs, wgrad_run(M), kWaitLimitNs, -1,
                          after_kernel, s);
}

// =================================================================== C ABI

extern "C" flp_status flp_layer_norm(const void* X, int64_t ldx, int dtype, const void* weight, const void* bias,
                                     int param_dtype, int64_t M, int64_t H, float eps, void* Y, int64_t ldy,
                                     float* mean, float* rstd, void* q, void* scale, void* stream) {
    flp_status st = norm_checks(M, H, dtype, param_dtype, weight, bias);
    if (st != FLP_OK) return st;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(FLP_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return fail(FLP_ERR_INVALID_ARG, "mean and rstd must be aligned to their elements");
    if (M == 0) return FLP_OK;
    st = row_checks(X, ldx, H, dtype, "X must be non-null");
    if (st == FLP_OK) st = row_checks(Y, ldy, H, dtype, "Y must be non-null");
    if (st == FLP_OK && (q || scale)) st = ck_checks(q, scale);
    DevInfo* d;
    if (st == FLP_OK) st = step_device(&d);
    if (st == FLP_OK) st = check_on_current_device(X, "X");
    if (st != FLP_OK) return st;
    NormFwdParams p{};
    p.x = X;
    p.ldx = ldx;
    p.w = weight;
    p.b = bias;
    p.param_f32 = param_dtype == FLP_F32;
    p.M = M;
    p.H = static_cast<int>(H);
    p.inv_h = static_cast<float>(1.0 / static_cast<double>(H));
    p.eps = eps;
    p.y = Y;
    p.ldy = ldy;
    p.mean = mean;
    p.rstd = rstd;
    p.q = static_cast<uint8_t*>(q);
    p.scale = static_cast<uint8_t*>(scale);
    p.Hp = static_cast<int>(ck_cols(H));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool loose = !(rows16(X, ldx, dtype) && rows16(Y, ldy, dtype) && aligned16(weight) && aligned16(bias) &&
                         (H * elem(dtype)) % 16 == 0);
    auto run = [&](auto t, auto ck, auto is_loose) -> flp_status {
        using T = decltype(t);
        constexpr bool CK = decltype(ck)::value, LOOSE = decltype(is_loose)::value;
        constexpr int TWO = sizeof(T) == 4 || (CK && LOOSE) ? 320 : CK ? 384 : 512;
        // bf16 rows ahead: 32768 x 4096 takes 96, 94, 82 us with 4, 3, 2 of them, with a
        // checkpoint 109, 105, 110 (32768 x 2048: 61, 59, 56; 16384 x 4608: 62, 62, 64)
        constexpr int S16 = CK ? 3 : 2;
        return norm_stream_shape<T, TWO, S16>(CK ? p.Hp : p.H, [&](auto shape, int threads) -> flp_status {
            using X = decltype(shape);
            constexpr auto* kernel = flp_norm_fwd_stream_kernel<T, X::NV, X::S, CK, LOOSE, X::WARP, X::MAXT, X::MINB>;
            const size_t smem = norm_stage_bytes<T, LOOSE>(X::S * X::NV, threads, 0);
            const size_t most = norm_stage_bytes<T, LOOSE>(X::S * X::NV, X::MAXT, 0);
            int per_sm = 0;
            const flp_status r = resident_blocks<kernel>(threads, smem, most, &per_sm);
            if (r != FLP_OK) return r;
            const int64_t rows = X::WARP ? threads / 32 : 1;
            const int64_t blocks = norm_blocks(M, rows, d->sm_count, per_sm);
            p.step = blocks * rows;
            p.step_x = p.step * ldx;
            p.step_y = p.step * ldy;
            p.step_q = p.step * p.Hp;
            p.step_s = p.step_q / CK_BLOCK;
            return launch_step(kernel, blocks, threads, smem, s, "flp_norm_fwd_stream_kernel launch", false, p);
        });
    };
    auto aligned = [&](auto t, auto ck) { return loose ? run(t, ck, std::true_type{}) : run(t, ck, std::false_type{}); };
    auto typed = [&](auto t) { return q ? aligned(t, std::true_type{}) : aligned(t, std::false_type{}); };
    return dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
}

extern "C" flp_status flp_layer_norm_workspace(int64_t M, int64_t H, size_t* bytes) {
    if (!bytes) return fail(FLP_ERR_INVALID_ARG, "bytes must be non-null");
    flp_status st = norm_checks(M, H, FLP_F32, FLP_F32, nullptr, nullptr);
    if (st != FLP_OK) return st;
    DevInfo* d;
    st = step_device(&d);
    if (st != FLP_OK) return st;
    *bytes = 0;
    if (norm_bwd_cluster(M, H)) return FLP_OK;
    int64_t blocks = 0;
    if ((st = norm_bwd_most_blocks(M, H, d->sm_count, &blocks)) != FLP_OK) return st;
    *bytes = static_cast<size_t>(blocks) * 2 * H * 4;
    return FLP_OK;
}

extern "C" flp_status flp_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* q,
                                              const void* scale, int dtype, const void* weight, int param_dtype,
                                              const float* mean, const float* rstd, int64_t M, int64_t H, void* dX,
                                              int64_t lddx, float* dweight, float* dbias, void* workspace,
                                              size_t workspace_bytes, void* stream) {
    flp_status st = norm_checks(M, H, dtype, param_dtype, weight, nullptr);
    if (st != FLP_OK) return st;
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return fail(FLP_ERR_INVALID_ARG, "mean, rstd, dweight and dbias must be aligned to their elements");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DevInfo* d;
    if (M > 0) {
        if ((X != nullptr) == (q != nullptr)) return fail(FLP_ERR_INVALID_ARG, "exactly one of X and its checkpoint");
        if (!mean || !rstd) return fail(FLP_ERR_INVALID_ARG, "mean and rstd must be non-null");
        st = row_checks(dY, lddy, H, dtype, "dY must be non-null");
        if (st == FLP_OK) st = row_checks(dX, lddx, H, dtype, "dX must be non-null");
        if (st == FLP_OK && X) st = row_checks(X, ldx, H, dtype, "X must be non-null");
        if (st == FLP_OK && q) st = ck_checks(q, scale);
    }
    if (st == FLP_OK) st = step_device(&d);
    if (st == FLP_OK && M > 0) st = check_on_current_device(dY, "dY");
    if (st != FLP_OK) return st;
    const bool sums = dweight || dbias;
    int64_t blocks = 0;
    if (M > 0) {
        const bool cluster = norm_bwd_cluster(M, H);
        const bool parts = sums && !cluster;
        if (parts && (!workspace || !aligned16(workspace)))
            return fail(FLP_ERR_WORKSPACE, "layer norm backward workspace null or misaligned");
        NormBwdParams p{};
        p.sums = sums;
        p.cluster = cluster;
        p.dw = dweight;
        p.db = dbias;
        p.dy = dY;
        p.lddy = lddy;
        p.x = X;
        p.ldx = ldx;
        p.q = static_cast<const uint8_t*>(q);
        p.scale = static_cast<const uint8_t*>(scale);
        p.Hp = static_cast<int>(ck_cols(H));
        p.w = weight;
        p.param_f32 = param_dtype == FLP_F32;
        p.mean = mean;
        p.rstd = rstd;
        p.M = M;
        p.H = static_cast<int>(H);
        p.inv_h = static_cast<float>(1.0 / static_cast<double>(H));
        p.dx = dX;
        p.lddx = lddx;
        p.part = static_cast<float*>(workspace);
        const bool loose = !(rows16(dY, lddy, dtype) && rows16(dX, lddx, dtype) && aligned16(weight) &&
                             (!X || rows16(X, ldx, dtype)) && (H * elem(dtype)) % 16 == 0);
        auto run = [&](auto t, auto ck, auto is_loose) -> flp_status {
            using T = decltype(t);
            constexpr bool CK = decltype(ck)::value, LOOSE = decltype(is_loose)::value;
            return norm_bwd_form<T, CK, LOOSE>(H, [&](auto k, const NormBwdForm& form) -> flp_status {
                constexpr auto* kernel = decltype(k)::kernel;
                const size_t smem = std::max(form.staged, cluster ? form.join + 8 * static_cast<size_t>(H) : 0);
                int per_sm = 0;
                const flp_status r = resident_blocks<kernel>(form.threads, form.staged, form.most, &per_sm);
                if (r != FLP_OK) return r;
                blocks = cluster ? kNormBwdCluster : norm_blocks(M, form.rows, d->sm_count, per_sm);
                if (parts && workspace_bytes < static_cast<size_t>(blocks) * 2 * H * 4)
                    return fail(FLP_ERR_WORKSPACE, "layer norm backward workspace too small");
                p.step = blocks * form.rows;
                p.step_dy = p.step * lddy;
                p.step_x = p.step * ldx;
                p.step_dx = p.step * lddx;
                p.step_q = p.step * p.Hp;
                p.step_s = p.step_q / CK_BLOCK;
                return cluster ? launch_cluster<NormBwdParams>(kernel, kNormBwdCluster, form.threads, smem, s,
                                                               "flp_norm_bwd_stream_kernel launch", p)
                               : launch_step(kernel, blocks, form.threads, smem, s, "flp_norm_bwd_stream_kernel launch",
                                             false, p);
            });
        };
        auto aligned = [&](auto t, auto ck) { return loose ? run(t, ck, std::true_type{}) : run(t, ck, std::false_type{}); };
        auto typed = [&](auto t) { return q ? aligned(t, std::true_type{}) : aligned(t, std::false_type{}); };
        st = dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
        if (st != FLP_OK) return st;
    }
    if (!sums || (M > 0 && norm_bwd_cluster(M, H))) return FLP_OK;
    NormJoinParams j{};
    j.part = static_cast<const float*>(workspace);
    j.P = static_cast<int>(blocks);
    j.H = static_cast<int>(H);
    j.dw = dweight;
    j.db = dbias;
    return launch_step(flp_norm_join_kernel, cdiv(2 * H, 32), 1024, 0, s, "flp_norm_join_kernel launch", M > 0, j);
}

extern "C" flp_status flp_checkpoint_pack(const void* X, int64_t ldx, int dtype, int64_t M, int64_t H, void* q,
                                          void* scale, void* stream) {
    return ck_run(true, X, ldx, dtype, q, scale, M, H, static_cast<cudaStream_t>(stream));
}

extern "C" flp_status flp_checkpoint_unpack(const void* q, const void* scale, int64_t M, int64_t H, void* X,
                                            int64_t ldx, int dtype, void* stream) {
    return ck_run(false, X, ldx, dtype, q, scale, M, H, static_cast<cudaStream_t>(stream));
}

extern "C" flp_status flp_checkpoint_weight_grad_workspace(const void* dY, int64_t lddy, int64_t M, int64_t N,
                                                           int64_t K, int dW_dtype, size_t* bytes) {
    if (!bytes) return fail(FLP_ERR_INVALID_ARG, "bytes must be non-null");
    flp_status st = wgrad_checks(dY, lddy, M, N, K, dW_dtype);
    if (st != FLP_OK) return st;
    DevInfo* d;
    st = check_device(&d);
    if (st != FLP_OK) return st;
    *bytes = plan_wgrad(dY, lddy, M, N, K, dW_dtype, d->pairs).bytes;
    return FLP_OK;
}

extern "C" flp_status flp_checkpoint_weight_grad(const void* dY, int64_t lddy, const void* q, const void* scale,
                                                 int64_t M, int64_t N, int64_t K, void* dW, int dW_dtype,
                                                 int accumulate_dW, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
    flp_status st = wgrad_checks(dY, lddy, M, N, K, dW_dtype);
    if (st != FLP_OK) return st;
    if (!dW || !aligned16(dW)) return fail(FLP_ERR_INVALID_ARG, "dW must be non-null and 16-byte aligned");
    if (accumulate_dW && dW_dtype != FLP_F32)
        return fail(FLP_ERR_UNSUPPORTED, "only an fp32 dW accumulates (a bf16 one would be rounded at every call)");
    if (M > 0 && !dY) return fail(FLP_ERR_INVALID_ARG, "dY must be non-null");
    if (M > 0 && (st = ck_checks(q, scale)) != FLP_OK) return st;
    DevInfo* d;
    st = check_device(&d);
    if (st != FLP_OK) return st;
    if ((st = check_on_current_device(dW, "dW")) != FLP_OK) return st;
    if ((st = wgrad_attrs()) != FLP_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const WgradPlan w = plan_wgrad(dY, lddy, M, N, K, dW_dtype, d->pairs);
    if (!workspace || workspace_bytes < w.bytes || !aligned16(workspace))
        return fail(FLP_ERR_WORKSPACE, "weight gradient workspace null, misaligned or too small");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (M == 0) {
        FLP_CUDA(cudaMemsetAsync(ws, 0, sizeof(int), s));  // the error word
        if (!accumulate_dW) FLP_CUDA(cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * elem(dW_dtype), s));
        return FLP_OK;
    }
    if ((st = check_on_current_device(dY, "dY")) != FLP_OK) return st;
    // the pads of the checkpoint's last blocks are unpacked with the rest (they
    // hold zeros); the same kernel clears the error word
    st = ck_launch<bf16, false>(false, ws + w.off_x, w.Kp, q, scale, M, w.Kp, s, reinterpret_cast<int*>(ws));
    if (st != FLP_OK) return st;
    const void* y = dY;
    int64_t ldy = lddy;
    if (w.Np) {
        y = ws + w.off_y;
        ldy = w.Np;
        if ((st = align_rows(dY, lddy, M, N, ws + w.off_y, w.Np, s)) != FLP_OK) return st;
    }
    const int run = wgrad_run(M);
    return wgrad_contract(w, y, ldy, ws + w.off_x, w.Kp, w.Kp, ws, M, N, K, dW, dW_dtype, accumulate_dW, d->pairs, run,
                          kWaitLimitNs, -1, true, s);
}

extern "C" flp_status flp_selftest_weight_grad_timeout(void* workspace, size_t workspace_bytes, int odd, int stall_after,
                                                       int64_t wait_limit_ns, void* stream) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < FLP_SELFTEST_WEIGHT_GRAD_BYTES)
        return fail(FLP_ERR_WORKSPACE, "self-test needs FLP_SELFTEST_WEIGHT_GRAD_BYTES of workspace");
    if (wait_limit_ns <= 0 || wait_limit_ns > 60ll * 1000 * 1000 * 1000)
        return fail(FLP_ERR_INVALID_ARG, "wait_limit_ns must be in (0, 60 s]");
    DevInfo* d;
    flp_status st = check_device(&d);
    if (st != FLP_OK) return st;
    if ((st = check_on_current_device(workspace, "workspace")) != FLP_OK) return st;
    if ((st = wgrad_attrs()) != FLP_OK) return st;
    const int64_t M = 192, N = 136, K = odd ? 521 : 520;
    const WgradPlan w = plan_wgrad(nullptr, N, M, N, K, FLP_F32, 1);
    const size_t off_dy = align_up(w.bytes, 1024);
    if (off_dy + M * N * 2 > FLP_SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET ||
        FLP_SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET + N * K * 4 > FLP_SELFTEST_WEIGHT_GRAD_BYTES)
        return fail(FLP_ERR_UNSUPPORTED, "self-test layout exceeds its workspace");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint8_t* dw = ws + FLP_SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    FLP_CUDA(cudaMemsetAsync(ws, 0, off_dy + M * N * 2, s));  // error word, X^, partial tiles, dY
    FLP_CUDA(cudaMemsetAsync(dw, 0x3f, N * K * 4, s));        // what the result has to replace
    st = wgrad_contract(w, ws + off_dy, N, ws + w.off_x, w.Kp, w.Kp, ws, M, N, K, dw, FLP_F32, 0, 1, 1,
                        static_cast<unsigned long long>(wait_limit_ns), stall_after < 0 ? -1 : stall_after, true, s);
    return st == FLP_OK ? flp_get_error(workspace, stream) : st;
}

extern "C" flp_status flp_balance_loss_workspace(int64_t T, int64_t E, size_t* bytes) {
    if (!bytes) return fail(FLP_ERR_INVALID_ARG, "bytes must be non-null");
    flp_status st = balance_checks(T, E, 1);
    if (st != FLP_OK) return st;
    DevInfo* d;
    st = step_device(&d);
    if (st != FLP_OK) return st;
    *bytes = plan_balance(T, E, d->sm_count).bytes;
    return FLP_OK;
}

extern "C" flp_status flp_balance_loss(const void* logits, int64_t ld, int dtype, const uint8_t* mask,
                                       const int64_t* experts, int64_t T, int64_t E, int64_t top_k, float coef,
                                       float* loss, void* grad, int64_t* counts, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    return flp_balance_loss_ex(logits, ld, dtype, mask, experts, T, E, top_k, coef, loss, grad, dtype, counts, workspace,
                               workspace_bytes, stream);
}

extern "C" flp_status flp_balance_loss_ex(const void* logits, int64_t ld, int dtype, const uint8_t* mask,
                                          const int64_t* experts, int64_t T, int64_t E, int64_t top_k, float coef,
                                          float* loss, void* grad, int grad_dtype, int64_t* counts, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    flp_status st = balance_checks(T, E, top_k);
    if (st != FLP_OK) return st;
    if (!is_dtype(dtype)) return fail(FLP_ERR_INVALID_ARG, "dtype is FLP_F32 or FLP_BF16");
    if (grad_dtype != dtype && grad_dtype != FLP_F32)
        return fail(FLP_ERR_INVALID_ARG, "grad_dtype is the logits' type or FLP_F32");
    if (!loss || !counts) return fail(FLP_ERR_INVALID_ARG, "loss and counts must be non-null");
    if (!aligned_to(loss, 4) || !aligned_to(counts, 8) || !aligned_to(experts, 8))
        return fail(FLP_ERR_INVALID_ARG, "loss, counts and experts must be aligned to their elements");
    if (!std::isfinite(coef)) return fail(FLP_ERR_INVALID_ARG, "coef must be finite");
    if (T > 0 && (st = row_checks(logits, ld, E, dtype, "logits must be non-null")) != FLP_OK) return st;
    if (!aligned_to(grad, elem(grad_dtype)))
        return fail(FLP_ERR_INVALID_ARG, "grad must be aligned to its elements");
    DevInfo* d;
    st = step_device(&d);
    if (st != FLP_OK) return st;
    if (T > 0 && (st = check_on_current_device(logits, "logits")) != FLP_OK) return st;
    const BalancePlan b = plan_balance(T, E, d->sm_count);
    if (b.bytes > 0 && (!workspace || workspace_bytes < b.bytes || !aligned16(workspace)))
        return fail(FLP_ERR_WORKSPACE, "balance loss workspace null, misaligned or too small");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    BalParams p{};
    p.z = logits;
    p.ld = ld;
    p.mask = mask;
    p.experts = reinterpret_cast<const long long*>(experts);
    p.T = T;
    p.E = static_cast<int>(E);
    p.k = static_cast<int>(top_k);
    p.coef = coef;
    p.grad = grad;
    p.grad_f32 = grad_dtype == FLP_F32;
    p.loss = loss;
    p.counts = reinterpret_cast<long long*>(counts);
    p.stat = reinterpret_cast<float2*>(ws);
    p.part_p = reinterpret_cast<float*>(ws + b.off_p);
    p.part_c = reinterpret_cast<int*>(ws + b.off_c);
    p.part_n = reinterpret_cast<int*>(ws + b.off_n);
    p.tot_p = reinterpret_cast<double*>(ws + b.off_tp);
    p.tot_c = reinterpret_cast<long long*>(ws + b.off_tc);
    p.tot_n = reinterpret_cast<long long*>(ws + b.off_tn);
    p.blocks = static_cast<int>(b.blocks);
    const size_t smem = bal_smem(E);
    auto typed = [&](auto t) -> flp_status {
        using T_ = decltype(t);
        const bool vec = E % 4 == 0 && ld % 4 == 0 && aligned_to(logits, 4 * elem(dtype)) && aligned_to(grad, 4 * elem(grad_dtype));
        return balance_shape(E, vec, [&](auto l, auto ne, auto v) -> flp_status {
            constexpr int L = decltype(l)::value, NE = decltype(ne)::value, V = decltype(v)::value;
            if (b.cluster)
                return launch_step(flp_balance_cluster_kernel<T_, L, NE, V>, BAL_CLUSTER, BAL_THREADS, smem, s,
                                   "flp_balance_cluster_kernel launch", false, p);
            flp_status r = launch_step(flp_balance_rows_kernel<T_, L, NE, V>, b.blocks, BAL_THREADS, smem, s,
                                       "flp_balance_rows_kernel launch", false, p);
            if (r == FLP_OK)
                r = launch_step(flp_balance_join_kernel, cdiv(E, 32), 1024, 0, s, "flp_balance_join_kernel launch", true, p);
            if (r == FLP_OK)
                r = launch_step(flp_balance_grad_kernel<T_, L, NE, V>, grad ? b.blocks : 1, BAL_THREADS, 0, s,
                                "flp_balance_grad_kernel launch", true, p);
            return r;
        });
    };
    return dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
}

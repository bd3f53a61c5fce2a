// experts.cu - host side of the expert operators declared in include/flp.h.
#include "experts.cuh"
#include "step_host.cuh"

namespace {

flp_status expert_sizes(int64_t T, int64_t k) {
    if (T < 0 || k < 1) return fail(FLP_ERR_INVALID_ARG, "T >= 0 and k >= 1 required");
    // the movers count a token's choices in steps of up to 32, in 32 bits
    if (k > 1 << 30) return fail(FLP_ERR_UNSUPPORTED, "more than 2^30 choices a token");
    if (T > kMaxRows || T * k > kMaxRows) return fail(FLP_ERR_UNSUPPORTED, "more than 2^31 - 1 slots");
    return FLP_OK;
}

flp_status sort_checks(int64_t T, int64_t k, int64_t E) {
    if (E < 1) return fail(FLP_ERR_INVALID_ARG, "E >= 1 required");
    if (E > SORT_MAX_E) return fail(FLP_ERR_UNSUPPORTED, "at most 1024 experts");
    return expert_sizes(T, k);
}

size_t sort_bytes(int64_t S, int64_t E) { return S <= SORT_ONE_BLOCK ? 0 : static_cast<size_t>(E + 1) * SORT_BLOCKS * 4; }

// The sort's shared memory (a histogram per warp), once per device.
flp_status sort_attrs() {
    static bool done[kMaxDevices] = {};
    int dev = 0;
    FLP_CUDA(cudaGetDevice(&dev));  // in range: step_device has run
    std::lock_guard<std::mutex> lk(g_mu);
    if (!done[dev]) {
        const int most = SORT_WARPS * (SORT_MAX_E + 1) * 4;
        FLP_CUDA(cudaFuncSetAttribute(flp_expert_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        FLP_CUDA(cudaFuncSetAttribute(flp_expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        done[dev] = true;
    }
    return FLP_OK;
}

// What the row movers share: checks of the index arrays, and their parameters.
flp_status move_params(MoveParams& p, int64_t T, int64_t H, int64_t k, int dtype, const int32_t* rows,
                       const int64_t* total, const void* weights, int weight_dtype) {
    flp_status st = expert_sizes(T, k);
    if (st != FLP_OK) return st;
    if (H < 1) return fail(FLP_ERR_INVALID_ARG, "H >= 1 required");
    if (!is_dtype(dtype)) return fail(FLP_ERR_INVALID_ARG, "dtype is FLP_F32 or FLP_BF16");
    if (weights && (!is_dtype(weight_dtype) || !aligned_to(weights, elem(weight_dtype))))
        return fail(FLP_ERR_INVALID_ARG, "weights are FLP_F32 or FLP_BF16 and aligned to their elements");
    if (H > INT32_MAX - 4096) return fail(FLP_ERR_UNSUPPORTED, "rows of more than 2^31 elements");
    if (T == 0) return FLP_OK;
    if (!rows || !total || !aligned_to(rows, 4) || !aligned_to(total, 8))
        return fail(FLP_ERR_INVALID_ARG, "rows and total must be non-null and aligned to their elements");
    p.weights = weights;
    p.weights_f32 = weight_dtype == FLP_F32;
    p.rows = rows;
    p.total = reinterpret_cast<const long long*>(total);
    p.T = T;
    p.k = static_cast<int>(k);
    p.H = static_cast<int>(H);
    return FLP_OK;
}

// Blocks of a grid with a warp for each token and chunk of `vecs` x 32 vectors of its row.
flp_status move_grid(MoveParams& p, int vecs, int dtype, int64_t* grid) {
    p.chunks = static_cast<int>(cdiv(p.H, vecs * 32 * (16 / elem(dtype))));
    *grid = cdiv(p.T * p.chunks, MOVE_WARPS);
    return *grid * MOVE_WARPS > INT32_MAX ? fail(FLP_ERR_UNSUPPORTED, "matrix too large for one launch") : FLP_OK;
}

inline bool rows_vec(const void* p, int64_t ld, int64_t H, int dtype) {
    return rows16(p, ld, dtype) && (H * elem(dtype)) % 16 == 0;
}

// Vectors of aligned rows that are short, else 0.  The short kernels number their threads in
// 32 bits: the tokens of one that would have more go the long rows' way.
inline int64_t short_vecs(const MoveParams& p, int dtype, bool loose) {
    const int64_t vecs = p.H * elem(dtype) / 16;
    return !loose && vecs <= SHORT_VECS && p.T <= INT32_MAX / SHORT_VECS ? vecs : 0;
}

template <typename F>
flp_status move_typed(int dtype, bool loose, F&& f) {
    auto typed = [&](auto t) { return loose ? f(t, std::true_type{}) : f(t, std::false_type{}); };
    return dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
}

}  // namespace

extern "C" flp_status flp_expert_sort_workspace(int64_t T, int64_t k, int64_t E, size_t* bytes) {
    if (!bytes) return fail(FLP_ERR_INVALID_ARG, "bytes must be non-null");
    const flp_status st = sort_checks(T, k, E);
    if (st == FLP_OK) *bytes = sort_bytes(T * k, E);
    return st;
}

extern "C" flp_status flp_expert_sort(const int64_t* experts, int64_t T, int64_t k, int64_t E, int32_t* rows,
                                      int32_t* slots, int64_t* counts, int64_t* offsets, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    flp_status st = sort_checks(T, k, E);
    if (st != FLP_OK) return st;
    if (!counts || !offsets || (T > 0 && (!experts || !rows || !slots)))
        return fail(FLP_ERR_INVALID_ARG, "experts, rows, slots, counts and offsets must be non-null");
    if (!aligned_to(experts, 8) || !aligned_to(rows, 4) || !aligned_to(slots, 4) || !aligned_to(counts, 8) ||
        !aligned_to(offsets, 8))
        return fail(FLP_ERR_INVALID_ARG, "experts, rows, slots, counts and offsets must be aligned to their elements");
    SortParams p{};
    p.S = T * k;
    const size_t need = sort_bytes(p.S, E);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return fail(FLP_ERR_WORKSPACE, "expert sort workspace null, misaligned or too small");
    DevInfo* d;
    if ((st = step_device(&d)) != FLP_OK) return st;
    if ((st = check_on_current_device(counts, "counts")) != FLP_OK) return st;
    if ((st = sort_attrs()) != FLP_OK) return st;
    p.experts = reinterpret_cast<const long long*>(experts);
    p.E = static_cast<int>(E);
    const int64_t most = need ? SORT_BLOCKS : 1;
    p.per = static_cast<int>(std::max<int64_t>(1, cdiv(p.S, most * SORT_THREADS)) * SORT_THREADS);
    p.blocks = static_cast<int>(std::max<int64_t>(1, cdiv(p.S, p.per)));
    p.part = static_cast<int*>(workspace);
    p.rows = rows;
    p.slots = slots;
    p.counts = reinterpret_cast<long long*>(counts);
    p.offsets = reinterpret_cast<long long*>(offsets);
    const size_t smem = static_cast<size_t>(SORT_WARPS) * (E + 1) * 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool two = p.blocks > 1;
    if (two) {
        st = launch_step(flp_expert_count_kernel, p.blocks, SORT_THREADS, smem, s, "flp_expert_count_kernel launch", false, p);
        if (st != FLP_OK) return st;
    }
    return launch_step(flp_expert_place_kernel, p.blocks, SORT_THREADS, smem, s, "flp_expert_place_kernel launch", two, p);
}

extern "C" flp_status flp_expert_gather(const void* X, int64_t ldx, int dtype, int64_t T, int64_t H, int64_t k,
                                        const int32_t* rows, const int64_t* total, void* XS, int64_t ldxs,
                                        void* stream) {
    MoveParams p{};
    flp_status st = move_params(p, T, H, k, dtype, rows, total, nullptr, FLP_F32);
    if (st != FLP_OK || T == 0) return st;
    st = row_checks(X, ldx, H, dtype, "X must be non-null");
    if (st == FLP_OK) st = row_checks(XS, ldxs, H, dtype, "XS must be non-null");
    DevInfo* d;
    if (st == FLP_OK) st = step_device(&d);
    if (st == FLP_OK) st = check_on_current_device(X, "X");
    if (st != FLP_OK) return st;
    p.one = const_cast<void*>(X);
    p.ld_one = ldx;
    p.many = XS;
    p.ld_many = ldxs;
    int64_t grid;
    if ((st = move_grid(p, GATHER_NV, dtype, &grid)) != FLP_OK) return st;
    const bool is_loose = !(rows_vec(X, ldx, H, dtype) && rows_vec(XS, ldxs, H, dtype));
    const int64_t vecs = short_vecs(p, dtype, is_loose);
    return move_typed(dtype, is_loose, [&](auto t, auto loose) {
        if (vecs)
            return launch_step(flp_expert_gather_short_kernel<decltype(t)>, cdiv(T * vecs, MOVE_THREADS), MOVE_THREADS, 0,
                               static_cast<cudaStream_t>(stream), "flp_expert_gather_short_kernel launch", false, p);
        return launch_step(flp_expert_gather_kernel<decltype(t), decltype(loose)::value>, grid, MOVE_THREADS, 0,
                           static_cast<cudaStream_t>(stream), "flp_expert_gather_kernel launch", false, p);
    });
}

extern "C" flp_status flp_expert_combine(const void* YS, int64_t ldys, int dtype, const void* weights, int weight_dtype,
                                         int64_t T, int64_t H, int64_t k, const int32_t* rows, const int64_t* total,
                                         void* Y, int64_t ldy, void* stream) {
    MoveParams p{};
    flp_status st = move_params(p, T, H, k, dtype, rows, total, weights, weight_dtype);
    if (st != FLP_OK || T == 0) return st;
    st = row_checks(YS, ldys, H, dtype, "YS must be non-null");
    if (st == FLP_OK) st = row_checks(Y, ldy, H, dtype, "Y must be non-null");
    DevInfo* d;
    if (st == FLP_OK) st = step_device(&d);
    if (st == FLP_OK) st = check_on_current_device(YS, "YS");
    if (st != FLP_OK) return st;
    p.many = const_cast<void*>(YS);
    p.ld_many = ldys;
    p.one = Y;
    p.ld_one = ldy;
    int64_t grid;
    if ((st = move_grid(p, COMBINE_NV, dtype, &grid)) != FLP_OK) return st;
    const bool is_loose = !(rows_vec(YS, ldys, H, dtype) && rows_vec(Y, ldy, H, dtype));
    const int64_t vecs = short_vecs(p, dtype, is_loose);
    return move_typed(dtype, is_loose, [&](auto t, auto loose) {
        if (vecs)
            return launch_step(flp_expert_combine_short_kernel<decltype(t)>, cdiv(T * vecs, MOVE_THREADS), MOVE_THREADS, 0,
                               static_cast<cudaStream_t>(stream), "flp_expert_combine_short_kernel launch", false, p);
        return launch_step(flp_expert_combine_kernel<decltype(t), decltype(loose)::value>, grid, MOVE_THREADS, 0,
                           static_cast<cudaStream_t>(stream), "flp_expert_combine_kernel launch", false, p);
    });
}

extern "C" flp_status flp_expert_combine_backward(const void* dY, int64_t lddy, const void* YS, int64_t ldys, int dtype,
                                                  const void* weights, int weight_dtype, int64_t T, int64_t H, int64_t k,
                                                  const int32_t* rows, const int64_t* total, void* dYS, int64_t lddys,
                                                  float* dweights, void* stream) {
    MoveParams p{};
    flp_status st = move_params(p, T, H, k, dtype, rows, total, weights, weight_dtype);
    if (st != FLP_OK || T == 0) return st;
    if (!aligned_to(dweights, 4)) return fail(FLP_ERR_INVALID_ARG, "dweights must be aligned to its elements");
    st = row_checks(dY, lddy, H, dtype, "dY must be non-null");
    if (st == FLP_OK && dweights) st = row_checks(YS, ldys, H, dtype, "dweights need YS");
    if (st == FLP_OK) st = row_checks(dYS, lddys, H, dtype, "dYS must be non-null");
    DevInfo* d;
    if (st == FLP_OK) st = step_device(&d);
    if (st == FLP_OK) st = check_on_current_device(dY, "dY");
    if (st != FLP_OK) return st;
    p.one = const_cast<void*>(dY);
    p.ld_one = lddy;
    p.many = dweights ? const_cast<void*>(YS) : nullptr;
    p.ld_many = dweights ? ldys : 0;
    p.out = dYS;
    p.ld_out = lddys;
    p.dweights = dweights;
    int64_t grid;
    if ((st = move_grid(p, CBWD_NV, dtype, &grid)) != FLP_OK) return st;
    // A warp by itself needs no barrier and has no chunks left over: 32768 x 4 x 5120 takes 447
    // us, a block 572, 4096 tokens 68 and 82; of few tokens it would leave most of the GPU idle
    // (1024 x 4 x 4096 25 and 23, 256 x 8 x 7168 50 and 19), unless rows are short.
    const bool warp = T >= 2048 || p.chunks <= 2;
    const bool loose = !(rows_vec(dY, lddy, H, dtype) && rows_vec(dYS, lddys, H, dtype) &&
                         (!dweights || rows_vec(YS, ldys, H, dtype)));
    const int64_t vecs = short_vecs(p, dtype, loose);
    int lanes = 1;
    while (lanes < vecs) lanes *= 2;
    return move_typed(dtype, loose, [&](auto t, auto is_loose) {
        if (vecs)
            return launch_step(flp_expert_combine_bwd_short_kernel<decltype(t)>, cdiv(T * lanes, MOVE_THREADS), MOVE_THREADS, 0,
                               static_cast<cudaStream_t>(stream), "flp_expert_combine_bwd_short_kernel launch", false, p, lanes);
        constexpr bool LOOSE = decltype(is_loose)::value;
        auto go = [&](auto* kernel, int64_t blocks) {
            return launch_step(kernel, blocks, MOVE_THREADS, 0, static_cast<cudaStream_t>(stream),
                               "flp_expert_combine_bwd_kernel launch", false, p);
        };
        return warp ? go(flp_expert_combine_bwd_kernel<decltype(t), LOOSE, true>, cdiv(T, MOVE_WARPS))
                    : go(flp_expert_combine_bwd_kernel<decltype(t), LOOSE, false>, T);
    });
}

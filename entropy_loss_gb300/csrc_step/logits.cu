// logits.cu - host side of the given-logits operators declared in include/flp.h.
#include "logits.cuh"
#include "step_host.cuh"

namespace {

flp_status tlp_checks(const void* logits, int64_t ld, int dtype, const int64_t* targets, int64_t M, int64_t V, float scale) {
    if (M < 0 || V < 1) return fail(FLP_ERR_INVALID_ARG, "M >= 0 and V >= 1 required");
    if (!is_dtype(dtype)) return fail(FLP_ERR_INVALID_ARG, "dtype is FLP_F32 or FLP_BF16");
    if (!(scale > 0.f) || !std::isfinite(scale * LOG2E))
        return fail(FLP_ERR_INVALID_ARG, "scale must be positive and finite");
    if (V > INT32_MAX - 65536) return fail(FLP_ERR_UNSUPPORTED, "rows of more than 2^31 elements");
    if (M > kMaxRows / TLP_CLUSTER) return fail(FLP_ERR_UNSUPPORTED, "too many rows for one launch");
    if (M == 0) return FLP_OK;
    if (!targets || !aligned_to(targets, 8)) return fail(FLP_ERR_INVALID_ARG, "targets must be non-null and aligned");
    return row_checks(logits, ld, V, dtype, "logits must be non-null");
}

// Blocks of a row: as many as finish the rows soonest, in vectors that a resident block
// reads, a row's end costing a block as much as 3000 vectors (2048 rows of 131072 take 108
// us in one block each, 146 in two; 64 rows 15 us in eight blocks each).
int tlp_cluster(int64_t M, int64_t vecs, int64_t resident) {
    int best = 1;
    double least = 1e300;
    for (int c = 1; c <= TLP_CLUSTER; c *= 2) {
        const double cost = static_cast<double>(cdiv(M * c, resident)) * (static_cast<double>(vecs) / c + 3000);
        if (cost < least) least = cost, best = c;
    }
    return best;
}

template <typename T, int THREADS>
flp_status tlp_launch(TlpParams& p, int sm_count, cudaStream_t s) {
    constexpr auto* kernel = flp_token_logprob_kernel<T, THREADS>;
    const int64_t vecs = cdiv(p.V + wide_v<T>() - 1, wide_v<T>());  // at any alignment
    int per_sm = 0;
    const flp_status st = resident_blocks<kernel>(THREADS, 0, 0, &per_sm);
    if (st != FLP_OK) return st;
    p.cluster = vecs <= TLP_NV * THREADS ? 1 : tlp_cluster(p.M, vecs, static_cast<int64_t>(per_sm) * sm_count);
    p.per = static_cast<int>(cdiv(cdiv(vecs, p.cluster), 32) * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.M * p.cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? FLP_OK : cuda_fail(e, "flp_token_logprob_kernel launch");
}

}  // namespace

extern "C" flp_status flp_token_logprob(const void* logits, int64_t ld, int dtype, const int64_t* targets, int64_t M,
                                        int64_t V, int64_t ignore_index, float scale, float* logprob, float* lse,
                                        float* entropy, int64_t top, float* top_logprob, int64_t* top_index, void* stream) {
    flp_status st = tlp_checks(logits, ld, dtype, targets, M, V, scale);
    if (st != FLP_OK) return st;
    if (top < 0 || top > V) return fail(FLP_ERR_INVALID_ARG, "0 <= top <= V required");
    if (top > TLP_MAX_TOP) return fail(FLP_ERR_UNSUPPORTED, "at most 32 alternatives");
    if (M == 0) return FLP_OK;
    if (!logprob || !lse || (top > 0 && (!top_logprob || !top_index)))
        return fail(FLP_ERR_INVALID_ARG, "logprob, lse and the alternatives' outputs must be non-null");
    if (!aligned_to(logprob, 4) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(top_logprob, 4) ||
        !aligned_to(top_index, 8))
        return fail(FLP_ERR_INVALID_ARG, "outputs must be aligned to their elements");
    DevInfo* d;
    if ((st = step_device(&d)) != FLP_OK) return st;
    if ((st = check_on_current_device(logits, "logits")) != FLP_OK) return st;
    TlpParams p{};
    p.x = logits;
    p.ld = ld;
    p.y = reinterpret_cast<const long long*>(targets);
    p.M = M;
    p.V = static_cast<int>(V);
    p.top = static_cast<int>(top);
    p.ignore_index = ignore_index;
    p.scale = scale;
    p.c = scale * LOG2E;
    p.logprob = logprob;
    p.lse = lse;
    p.entropy = entropy;
    p.top_value = top_logprob;
    p.top_index = reinterpret_cast<long long*>(top_index);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto typed = [&](auto t) {
        using T = decltype(t);
        // Short rows in smaller blocks, of which an SM holds more, where there are enough rows
        // to fill it; a row of up to 4 vectors a thread at once in any case.
        const int64_t vecs = cdiv(V, wide_v<T>());
        if (M >= 32 * d->sm_count && vecs <= 1024) return tlp_launch<T, 32>(p, d->sm_count, s);
        if (vecs <= TLP_NV * 128 || (M >= 8 * d->sm_count && vecs <= 4096)) return tlp_launch<T, 128>(p, d->sm_count, s);
        return tlp_launch<T, 256>(p, d->sm_count, s);
    };
    return dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
}

extern "C" flp_status flp_token_logprob_backward(const void* logits, int64_t ld, int dtype, const int64_t* targets,
                                                 int64_t M, int64_t V, int64_t ignore_index, float scale, const float* lse,
                                                 const float* entropy, const float* grad_logprob, const float* grad_entropy,
                                                 void* dlogits, int64_t lddl, void* stream) {
    flp_status st = tlp_checks(logits, ld, dtype, targets, M, V, scale);
    if (st != FLP_OK || M == 0) return st;
    if (!lse) return fail(FLP_ERR_INVALID_ARG, "lse must be non-null");
    if (grad_entropy && !entropy) return fail(FLP_ERR_INVALID_ARG, "the gradient of the entropy needs the entropy");
    if (!aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(grad_logprob, 4) || !aligned_to(grad_entropy, 4))
        return fail(FLP_ERR_INVALID_ARG, "row values must be aligned to their elements");
    if ((st = row_checks(dlogits, lddl, V, dtype, "dlogits must be non-null")) != FLP_OK) return st;
    DevInfo* d;
    if ((st = step_device(&d)) != FLP_OK) return st;
    if ((st = check_on_current_device(logits, "logits")) != FLP_OK) return st;
    TlpBwdParams p{};
    p.x = logits;
    p.ld = ld;
    p.y = reinterpret_cast<const long long*>(targets);
    p.M = M;
    p.V = static_cast<int>(V);
    p.ignore_index = ignore_index;
    p.scale = scale;
    p.lse = lse;
    p.entropy = entropy;
    p.g_lp = grad_logprob;
    p.g_ent = grad_entropy;
    p.dx = dlogits;
    p.lddx = lddl;
    const bool vec = rows16(logits, ld, dtype) && rows16(dlogits, lddl, dtype) && (V * elem(dtype)) % 16 == 0;
    p.chunks = static_cast<int>(cdiv(V, TLPB_NV * 32 * (16 / elem(dtype))));
    const int64_t grid = cdiv(M * p.chunks, TLPB_THREADS / 32);
    if (grid * (TLPB_THREADS / 32) > INT32_MAX) return fail(FLP_ERR_UNSUPPORTED, "matrix too large for one launch");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto* kernel) {
        return launch_step(kernel, grid, TLPB_THREADS, 0, s, "flp_token_logprob_bwd_kernel launch", false, p);
    };
    auto typed = [&](auto t) {
        return vec ? go(flp_token_logprob_bwd_kernel<decltype(t), false>) : go(flp_token_logprob_bwd_kernel<decltype(t), true>);
    };
    return dtype == FLP_BF16 ? typed(bf16{}) : typed(float{});
}

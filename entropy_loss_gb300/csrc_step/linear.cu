// linear.cu - host side of the linear layer declared in include/flp.h.
#include "linear.cuh"
#include "step_host.cuh"

namespace {

// ------------------------------------------------------------------ product

// A step of a tensor core cuts each of its 16 products to a quarter of the last place of the
// accumulator, and their sum to that place, toward zero: 2.4 of these places on average (one
// product of 16 0.4), so a long sum comes out too small.  Of positive products 7e-4 over
// 131072 and 2.8e-3 over 524288; of centred ones 1e-4 over 131072.  A bf16 result's own
// rounding is 1.7e-3: longer contractions are joined from fp32 sums of runs of at most 2048
// 64-deep blocks, as the weight gradient's are.
constexpr int64_t LIN_RUN = 2048;

struct LinPlan {
    int width, tm, tn, whole, rest, splits, units, KB, rows;
    size_t part_bytes;
};

// Tiles of 256 x 512, or of 256 x 256 where they fill the pairs better.  Whole rounds of
// tiles write their outputs; the rest do so too, or are split into their halves (0 splits)
// or along the contraction.  The least of what these cost:
// 0.66 us for a 64-deep block of a wide tile and 0.37 us of a narrow one (the rate at which
// its operands arrive), 3 us for a run's start and end (5 for a half that one epilogue
// group drains by itself), and for joining 4 us (a launch) and
// the partial tiles' bytes, written and read back at 4 TB/s.
// Longer contractions than LIN_RUN blocks are split everywhere, into runs of at most that and
// at least a quarter of it (4096 x 151936 -> 4096 in one run 2607 us, in two 3179, in more
// 2757).
LinPlan plan_linear(int64_t M, int64_t N, int64_t depth, int pairs) {
    LinPlan best{};
    double least = 1e300;
    pairs = std::max(1, pairs);
    for (int width = 2 * BN; width >= BN; width -= BN) {
        LinPlan l{};
        l.width = width;
        l.tm = static_cast<int>(cdiv(M, PM));
        l.tn = static_cast<int>(cdiv(N, width));
        l.KB = static_cast<int>(cdiv(depth, BK));
        l.rows = static_cast<int>(std::min<int64_t>(M, PM));
        const double block = width > BN ? 0.66 : 0.37;
        const int64_t runs = cdiv(l.KB, LIN_RUN), tiles = static_cast<int64_t>(l.tm) * l.tn;
        const int64_t whole = runs > 1 ? 0 : tiles / pairs * pairs, rest = tiles - whole;
        const double tile_mb = static_cast<double>(l.rows) * width * 4 * 2 / 1e6;
        const int64_t most = rest == 0 ? 1 : std::min<int64_t>(l.KB, std::max<int64_t>(runs > 1 ? 4 * runs : 1, 4 * pairs / rest));
        for (int64_t s = width > BN && rest > 0 && runs == 1 ? 0 : runs; s <= most; ++s) {
            const double joined = s > 1 ? 4.0 + tile_mb / 4 * static_cast<double>(rest * s) : 0.0;
            const double last = s == 0 ? static_cast<double>(cdiv(2 * rest, pairs)) * (l.KB * 0.37 + 5.0)
                                       : static_cast<double>(cdiv(rest * s, pairs)) * (static_cast<double>(cdiv(l.KB, s)) * block + 3.0);
            const double cost = static_cast<double>(whole / pairs) * l.KB * block + last + joined;
            if (cost >= least - 1e-9) continue;
            least = cost;
            l.splits = static_cast<int>(s);
            l.whole = static_cast<int>(s == 1 ? tiles : whole);
            l.rest = static_cast<int>(s > 1 ? rest : 0);
            l.units = l.whole + (s == 0 ? static_cast<int>(2 * rest) : l.rest * l.splits);
            l.part_bytes = static_cast<size_t>(l.rest) * l.splits * l.rows * 2 * BN * 4;
            best = l;
        }
    }
    return best;
}

// The products' shared memory, once per device.
flp_status linear_attrs() {
    static bool done[kMaxDevices] = {};
    int dev = 0;
    FLP_CUDA(cudaGetDevice(&dev));  // in range: check_device has run
    std::lock_guard<std::mutex> lk(g_mu);
    if (!done[dev]) {
        FLP_CUDA(cudaFuncSetAttribute(flp_linear_kernel<1, LIN_NONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC));
        FLP_CUDA(cudaFuncSetAttribute(flp_linear_turned_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC));
        FLP_CUDA(cudaFuncSetAttribute(flp_linear_turned_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC));
        for (int act = LIN_NONE; act <= LIN_SILU; ++act) {
            const cudaError_t e = lin_with_act(act, [](auto a) {
                return cudaFuncSetAttribute(flp_linear_kernel<0, decltype(a)::value>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            SMEM_ALLOC);
            });
            if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        }
        done[dev] = true;
    }
    return FLP_OK;
}

// One product and, for split tiles, its join: A [M, depth] and W (w_mn: [depth, N], else
// [N, depth]), rows aligned to 16 bytes; `low`: the M rows below A's are added to them.
flp_status linear_product(const LinPlan& l, const void* a, int64_t lda, const void* w, int64_t ldw, bool w_mn, int64_t M,
                          int64_t N, int64_t depth, const LinEpilogue& e, void* part, int* err, int pairs,
                          unsigned long long wait_limit_ns, int stall_after, bool after_kernel, cudaStream_t s,
                          bool low = false) {
    constexpr auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap ma, mb, my, mp;
    flp_status st = tmap_2d(&ma, BF, a, depth, low ? 2 * M : M, lda * 2, BK, BM);
    if (st == FLP_OK) st = w_mn ? tmap_2d(&mb, BF, w, N, depth, ldw * 2, 64, 64) : tmap_2d(&mb, BF, w, depth, N, ldw * 2, BK, BNH);
    if (st != FLP_OK) return st;
    my = mp = ma;  // where no bulk store writes
    if (e.vec && (st = tmap_2d(&my, BF, e.y, N, M, e.ldy * 2, 32, BM, CU_TENSOR_MAP_SWIZZLE_64B)) != FLP_OK) return st;
    if (e.vec && e.pre && (st = tmap_2d(&mp, BF, e.pre, N, M, e.ldpre * 2, 32, BM, CU_TENSOR_MAP_SWIZZLE_64B)) != FLP_OK)
        return st;
    LinParams p{};
    p.tm = l.tm;
    p.tn = l.tn;
    p.width = l.width;
    p.group = std::min(l.tm, 8);
    p.whole = l.whole;
    p.splits = l.splits;
    p.units = l.units;
    p.KB = l.KB;
    p.fold = static_cast<int>(cdiv(depth, BK));
    p.low = low ? static_cast<int>(M) : 0;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.part = static_cast<float*>(part);
    p.rows = l.rows;
    p.e = e;
    p.err = err;
    p.wait_limit_ns = wait_limit_ns;
    p.stall_after = stall_after;
    const int grid = 2 * static_cast<int>(std::min<int64_t>(l.units, pairs));
    auto go = [&](auto* kernel) {
        return launch_pairs_n(kernel, grid, WIDE_THREADS, s, "flp_linear_kernel launch", after_kernel, ma, mb, my, mp, p);
    };
    st = w_mn ? go(flp_linear_kernel<1, LIN_NONE>)
              : lin_with_act(e.act, [&](auto act) { return go(flp_linear_kernel<0, decltype(act)::value>); });
    if (st != FLP_OK || !l.rest) return st;
    return launch_step(flp_linear_join_kernel, static_cast<int64_t>(l.rest) * l.rows, LJ_THREADS, 0, s,
                       "flp_linear_join_kernel launch", true, p);
}

// ---------------------------------------------------------------- turned tiles

struct LinTurnPlan {
    int nt, tiles_t, tiles_w, split, stages;
    uint32_t cols;  // of TMEM
    size_t smem;
};

// CTAs of a cluster wait for one another while they hold TMEM.  None may wait for TMEM
// itself, or clusters could keep each other from starting: every CTA asks for its columns'
// share of an SM's shared memory, so that those that fit an SM together, of any of these
// launches, find their 512 columns (a CTA of a pair takes the whole SM).
constexpr size_t kSmemPerTmemColumn = 228 * 1024 / 512;

// Rows of x in as few tiles as hold them, evenly; the contraction split over as many CTAs
// as are resident, two an SM.
LinTurnPlan plan_turned(int64_t M, int64_t N, int64_t depth, int sm_count, bool low = false) {
    LinTurnPlan t{};
    t.tiles_t = static_cast<int>(cdiv(M, LT_MAX_T));
    t.nt = static_cast<int>(cdiv(cdiv(M, t.tiles_t), 16) * 16);
    t.tiles_w = static_cast<int>(cdiv(N, 128));
    const int64_t KB = cdiv(depth, BK), tiles = static_cast<int64_t>(t.tiles_t) * t.tiles_w;
    t.split = 1;
    while (t.split * LIN_RUN < (low ? 2 : 1) * KB) t.split *= 2;  // at most 8: linear_turns
    // up to four CTAs a tile, eight of few tiles (4096 x 4096, 16 rows: 19 us with four, 21 with
    // eight; 8192 -> 1024: 21 and 17)
    const int most = tiles * 8 <= sm_count ? 8 : 4;
    while (t.split < most && tiles * t.split * 2 <= 2 * sm_count && t.split * 2 <= KB) t.split *= 2;
    const size_t room = 108 * 1024, stage = lin_turn_stage(t.nt, low);
    t.stages = static_cast<int>(std::min<int64_t>({LT_STAGES, static_cast<int64_t>(room / stage), cdiv(KB, t.split)}));
    for (t.cols = 32; t.cols < static_cast<uint32_t>(t.nt);) t.cols *= 2;
    t.smem = std::max<size_t>({t.stages * stage + 1024, static_cast<size_t>(t.nt) * 128 * 4 + 1024, t.cols * kSmemPerTmemColumn});
    return t;
}

flp_status linear_turned(const LinTurnPlan& t, const void* x, int64_t ldx, const void* w, int64_t ldw, bool w_mn, int64_t M,
                         int64_t N, int64_t depth, const LinEpilogue& e, int* err, unsigned long long wait_limit_ns,
                         int stall_after, bool after_kernel, cudaStream_t s, bool low = false) {
    constexpr auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap mw, mx;
    flp_status st = w_mn ? tmap_2d(&mw, BF, w, N, depth, ldw * 2, 64, 64) : tmap_2d(&mw, BF, w, depth, N, ldw * 2, BK, 128);
    if (st == FLP_OK) st = tmap_2d(&mx, BF, x, depth, low ? 2 * M : M, ldx * 2, BK, static_cast<uint32_t>(t.nt));
    if (st != FLP_OK) return st;
    LinTurnParams p{};
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.KB = static_cast<int>(cdiv(depth, BK));
    p.nt = t.nt;
    p.tiles_t = t.tiles_t;
    p.split = t.split;
    p.stages = t.stages;
    p.cols = t.cols;
    p.low = low ? static_cast<int>(M) : 0;
    p.e = e;
    p.err = err;
    p.wait_limit_ns = wait_limit_ns;
    p.stall_after = stall_after;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(t.tiles_t * t.tiles_w * t.split));
    cfg.blockDim = dim3(LT_THREADS);
    cfg.dynamicSmemBytes = t.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (t.split > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(t.split);
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (after_kernel) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t r = w_mn ? cudaLaunchKernelEx(&cfg, flp_linear_turned_kernel<1>, mw, mx, p)
                               : cudaLaunchKernelEx(&cfg, flp_linear_turned_kernel<0>, mw, mx, p);
    return r == cudaSuccess ? FLP_OK : cuda_fail(r, "flp_linear_turned_kernel launch");
}

// Rows of d that stay the sum of two bf16 numbers in every product unless the caller says
// otherwise: one 64-deep block of dW's, and turned tiles.
constexpr int64_t LIN_FEW = 64;

// Turned tiles where they keep up: while memory sets the pace, or they do not need more
// than one an SM (4096 x 4096: 512 rows 35 us, 39 in pairs' tiles, 1024 rows 48 and 39; 16384
// x 4096: 64 rows 42 and 50, 256 rows 58 and 50).
// A cluster's eight CTAs hold eight runs.
bool linear_turns(int64_t M, int64_t N, int64_t depth, int sm_count, bool low = false) {
    if ((low ? 2 : 1) * cdiv(depth, BK) > 8 * LIN_RUN) return false;
    return M <= 64 || cdiv(M, LT_MAX_T) * cdiv(N, 128) <= sm_count;
}

flp_status linear_row(LinRowParams& p, bool loose, int sm_count, bool after_kernel, cudaStream_t s) {
    // warps of the grid: eight an SM before a row's contraction is split
    p.kw = 1;
    while (p.kw < LR_WARPS && cdiv(p.N, LR_ROWS) * p.kw < 8 * sm_count && p.K > 256 * p.kw) p.kw *= 2;
    p.chunk = static_cast<int>(cdiv(cdiv(p.K, p.kw), 256) * 256);
    return launch_step(loose ? flp_linear_row_kernel<true> : flp_linear_row_kernel<false>, cdiv(p.N, LR_ROWS * (LR_WARPS / p.kw)),
                       LR_THREADS, 0, s, "flp_linear_row_kernel launch", after_kernel, p);
}

flp_status linear_sizes(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1) return fail(FLP_ERR_INVALID_ARG, "M >= 0, N >= 1 and K >= 1 required");
    const int64_t most = kMaxRows - 4096;  // eight chunks of a contraction, each rounded up to 256, end within 32 bits
    if (M > most || N > most || K > most || cdiv(M, PM) * cdiv(N, BN) > (1 << 23) || cdiv(M, PM) * cdiv(K, BN) > (1 << 23))
        return fail(FLP_ERR_UNSUPPORTED, "sizes beyond the 32-bit tiling");
    // partial tiles of a contraction that is split everywhere (512 KiB each)
    auto partial = [](int64_t M, int64_t N, int64_t depth) {
        const int64_t runs = cdiv(depth, BK * LIN_RUN);
        return runs > 1 ? runs * cdiv(M, PM) * cdiv(N, BN) : 0;
    };
    if (partial(M, N, K) > 1 << 22 || partial(M, K, 2 * N) > 1 << 22)
        return fail(FLP_ERR_UNSUPPORTED, "contraction too deep for so many outputs");
    return FLP_OK;
}

flp_status linear_terms(int d_terms, int64_t M) {
    if (d_terms < 0 || d_terms > 2) return fail(FLP_ERR_INVALID_ARG, "d_terms is 0, 1 or 2");
    return d_terms == 2 && M > 1 << 29 ? fail(FLP_ERR_UNSUPPORTED, "sizes beyond the 32-bit tiling") : FLP_OK;
}

flp_status linear_act(int activation) {
    return activation >= FLP_ACT_NONE && activation <= FLP_ACT_SILU ? FLP_OK : fail(FLP_ERR_INVALID_ARG, "unknown activation");
}
static_assert(FLP_ACT_NONE == LIN_NONE && FLP_ACT_RELU == LIN_RELU && FLP_ACT_GELU == LIN_GELU &&
                  FLP_ACT_GELU_TANH == LIN_GELU_TANH && FLP_ACT_SILU == LIN_SILU,
              "one numbering");

inline bool rows_bf16(const void* p, int64_t ld) { return rows16(p, ld, FLP_BF16); }
inline int64_t pad8(int64_t n) { return cdiv(n, 8) * 8; }

// Regions of a workspace, 1 KiB aligned.
struct Regions {
    size_t bytes = 0;
    size_t take(size_t n) {
        const size_t at = bytes;
        bytes += align_up(n, 1024);
        return at;
    }
};

struct LinearLayout {
    LinPlan l;
    LinTurnPlan t;
    size_t off_x, off_w, off_part, bytes;
    bool one, turned, copy_x, copy_w;
};

LinearLayout linear_layout(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K, int sm_count,
                           int pairs) {
    LinearLayout f{};
    f.one = M == 1;
    f.turned = !f.one && linear_turns(M, N, K, sm_count);
    if (f.turned)
        f.t = plan_turned(M, N, K, sm_count);
    else if (!f.one)
        f.l = plan_linear(M, N, K, pairs);
    f.copy_x = !rows_bf16(X, ldx) || (f.one && K % 8 != 0);  // whole vectors of x
    f.copy_w = !f.one && !rows_bf16(W, ldw);
    Regions r;
    f.off_x = r.take(f.copy_x ? M * pad8(K) * 2 : 0);
    f.off_w = r.take(f.copy_w ? N * pad8(K) * 2 : 0);
    f.off_part = r.take(f.l.part_bytes);
    f.bytes = r.bytes;
    return f;
}

struct LinearGradLayout {
    LinPlan l;  // of dx, or
    LinTurnPlan t;
    bool turned;
    size_t off_dw, off_x, off_w, off_d, off_lo, off_part, off_sums, bytes;
    bool copy_x, copy_w, make_d, sums;
    bool two_x, two;  // d as the sum of two bf16 numbers, for dX, and for dW,
    bool stack;       // one below the other with x twice: one product
    int blocks, rows;  // of the column sums
};

// Row blocks of the pass over dy: enough for every SM to hold two blocks of threads, of
// at least 32 rows (the warps' and their loads').
LinearGradLayout linear_grad_layout(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                    int activation, int d_terms, bool want_dx, bool want_dw, bool want_db, int64_t M, int64_t N,
                                    int64_t K, int dw_dtype, int sm_count, int pairs) {
    LinearGradLayout g{};
    const bool rounds = activation != FLP_ACT_NONE && activation != FLP_ACT_RELU;  // whose slopes are 0 and 1
    const bool two = rounds && (d_terms == 2 || (d_terms == 0 && M <= LIN_FEW));
    g.two_x = want_dx && two;
    g.turned = linear_turns(M, K, N, sm_count, g.two_x);
    if (g.turned)
        g.t = plan_turned(M, K, N, sm_count, g.two_x);
    else
        g.l = plan_linear(M, K, g.two_x ? 2 * BK * cdiv(N, BK) : N, pairs);
    g.copy_x = want_dw && !rows_bf16(X, ldx);
    g.copy_w = want_dx && !rows_bf16(W, ldw);
    g.make_d = (want_dx || want_dw) && (activation != FLP_ACT_NONE || !rows_bf16(dY, lddy));
    g.two = want_dw && (two || (rounds && d_terms == 0 && dw_dtype == FLP_F32));
    // x twice costs its copies, 6 M K bytes; a second product a launch and reading and writing dW,
    // 8 N K (two products and one, backward through gelu_tanh: 1 row 4096 -> 16384 213 us and 103,
    // 1024 rows 396 and 314, 2048 rows 2048 -> 2048 91 and 80; 4096 rows 4096 -> 4096 314 and 328,
    // 8192 rows 4096 -> 16384 2060 and 2065).  A second product would round a bf16 dW twice.
    g.stack = g.two && (dw_dtype == FLP_BF16 || M <= LIN_FEW || (M <= N && (M <= 2048 || 4 * M <= N)));
    g.sums = want_db;
    const int64_t strips = cdiv(N, 256);
    g.rows = static_cast<int>(std::max<int64_t>(32, cdiv(cdiv(M, std::max<int64_t>(1, cdiv(8 * sm_count, strips))), 32) * 32));
    while (cdiv(M, g.rows) > 65535) g.rows *= 2;
    g.blocks = static_cast<int>(cdiv(M, g.rows));
    Regions r;
    r.take(kHeaderBytes);  // the error word
    g.off_dw = 0;          // whose region it begins
    if (want_dw) r.bytes = align_up(std::max(r.bytes, weight_grad_bytes(g.stack ? 2 * M : M, N, K, dw_dtype, pairs)), 1024);
    g.off_x = r.take(g.stack ? 2 * M * pad8(K) * 2 : g.copy_x ? M * pad8(K) * 2 : 0);
    g.off_w = r.take(g.copy_w ? N * pad8(K) * 2 : 0);
    g.off_d = r.take(g.make_d ? (g.two || g.two_x ? 2 : 1) * M * pad8(N) * 2 : 0);
    g.off_lo = g.off_d + M * pad8(N) * 2;
    g.off_part = r.take(want_dx ? g.l.part_bytes : 0);
    g.off_sums = r.take(g.sums ? static_cast<size_t>(g.blocks) * N * 4 : 0);
    g.bytes = r.bytes;
    return g;
}

}  // namespace

extern "C" flp_status flp_linear_workspace(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M, int64_t N,
                                           int64_t K, size_t* bytes) {
    if (!bytes) return fail(FLP_ERR_INVALID_ARG, "bytes must be non-null");
    flp_status st = linear_sizes(M, N, K);
    if (st != FLP_OK) return st;
    DevInfo* d;
    if ((st = check_device(&d)) != FLP_OK) return st;
    *bytes = M == 0 ? 0 : linear_layout(X, ldx, W, ldw, M, N, K, d->sm_count, d->pairs).bytes;
    return FLP_OK;
}

extern "C" flp_status flp_linear(const void* X, int64_t ldx, const void* W, int64_t ldw, const void* bias, int bias_dtype,
                                 int activation, const void* residual, int64_t ldr, int64_t M, int64_t N, int64_t K, void* Y,
                                 int64_t ldy, void* pre, int64_t ldpre, void* workspace, size_t workspace_bytes, void* stream) {
    flp_status st = linear_sizes(M, N, K);
    if (st == FLP_OK) st = linear_act(activation);
    if (st != FLP_OK) return st;
    if (bias && (!is_dtype(bias_dtype) || !aligned_to(bias, elem(bias_dtype))))
        return fail(FLP_ERR_INVALID_ARG, "bias is FLP_F32 or FLP_BF16 and aligned to its elements");
    if (M == 0) return FLP_OK;
    st = row_checks(X, ldx, K, FLP_BF16, "X must be non-null");
    if (st == FLP_OK) st = row_checks(W, ldw, K, FLP_BF16, "W must be non-null");
    if (st == FLP_OK) st = row_checks(Y, ldy, N, FLP_BF16, "Y must be non-null");
    if (st == FLP_OK && residual) st = row_checks(residual, ldr, N, FLP_BF16, "residual must be non-null");
    if (st == FLP_OK && pre) st = row_checks(pre, ldpre, N, FLP_BF16, "pre must be non-null");
    DevInfo* d;
    if (st == FLP_OK) st = check_device(&d);
    if (st == FLP_OK) st = check_on_current_device(X, "X");
    if (st == FLP_OK) st = linear_attrs();
    if (st != FLP_OK) return st;
    const LinearLayout f = linear_layout(X, ldx, W, ldw, M, N, K, d->sm_count, d->pairs);
    if (f.bytes > 0 && (!workspace || workspace_bytes < f.bytes || !aligned16(workspace)))
        return fail(FLP_ERR_WORKSPACE, "linear workspace null, misaligned or too small");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    bool after = false;
    if (f.copy_x) {
        if ((st = align_rows(X, ldx, M, K, ws + f.off_x, pad8(K), s)) != FLP_OK) return st;
        X = ws + f.off_x, ldx = pad8(K), after = true;
    }
    if (f.copy_w) {
        if ((st = align_rows(W, ldw, N, K, ws + f.off_w, pad8(K), s)) != FLP_OK) return st;
        W = ws + f.off_w, ldw = pad8(K), after = true;
    }
    LinEpilogue e{};
    e.bias = bias;
    e.bias_f32 = bias_dtype == FLP_F32;
    e.act = activation;
    e.residual = static_cast<const bf16*>(residual);
    e.ldr = ldr;
    e.y = static_cast<bf16*>(Y);
    e.ldy = ldy;
    e.pre = static_cast<bf16*>(pre);
    e.ldpre = ldpre;
    e.vec = rows_bf16(Y, ldy) && N % 8 == 0 && (!residual || rows_bf16(residual, ldr)) && (!pre || rows_bf16(pre, ldpre));
    e.bias_vec = aligned16(bias);
    if (f.one) {
        LinRowParams p{};
        p.x = static_cast<const bf16*>(X);
        p.w = static_cast<const bf16*>(W);
        p.ldw = ldw;
        p.N = static_cast<int>(N);
        p.K = static_cast<int>(K);
        p.e = e;
        return linear_row(p, !(rows_bf16(W, ldw) && K % 8 == 0), d->sm_count, after, s);
    }
    if (f.turned) return linear_turned(f.t, X, ldx, W, ldw, false, M, N, K, e, nullptr, kWaitLimitNs, -1, after, s);
    return linear_product(f.l, X, ldx, W, ldw, false, M, N, K, e, ws + f.off_part, nullptr, d->pairs, kWaitLimitNs, -1, after, s);
}

extern "C" flp_status flp_linear_backward_workspace_ex(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W,
                                                       int64_t ldw, int activation, int d_terms, int want_dX, int want_dW,
                                                       int want_dbias, int64_t M, int64_t N, int64_t K, int dW_dtype, size_t* bytes) {
    if (!bytes) return fail(FLP_ERR_INVALID_ARG, "bytes must be non-null");
    flp_status st = linear_sizes(M, N, K);
    if (st == FLP_OK) st = linear_act(activation);
    if (st == FLP_OK) st = linear_terms(d_terms, M);
    if (st == FLP_OK) st = weight_grad_checks(M, N, K, dW_dtype);
    if (st != FLP_OK) return st;
    DevInfo* d;
    if ((st = check_device(&d)) != FLP_OK) return st;
    *bytes = M == 0 ? 0 : linear_grad_layout(dY, lddy, X, ldx, W, ldw, activation, d_terms, want_dX, want_dW, want_dbias, M, N, K,
                                             dW_dtype, d->sm_count, d->pairs).bytes;
    return FLP_OK;
}

extern "C" flp_status flp_linear_backward_workspace(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W,
                                                    int64_t ldw, int activation, int want_dX, int want_dW, int want_dbias,
                                                    int64_t M, int64_t N, int64_t K, int dW_dtype, size_t* bytes) {
    return flp_linear_backward_workspace_ex(dY, lddy, X, ldx, W, ldw, activation, 0, want_dX, want_dW, want_dbias, M, N, K, dW_dtype,
                                            bytes);
}

extern "C" flp_status flp_linear_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                          const void* pre, int64_t ldpre, int activation, int64_t M, int64_t N, int64_t K,
                                          void* dX, int64_t lddx, void* dW, int dW_dtype, float* dbias, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    return flp_linear_backward_ex(dY, lddy, X, ldx, W, ldw, pre, ldpre, activation, 0, M, N, K, dX, lddx, dW, dW_dtype, dbias,
                                  workspace, workspace_bytes, stream);
}

extern "C" flp_status flp_linear_backward_ex(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                             const void* pre, int64_t ldpre, int activation, int d_terms, int64_t M, int64_t N,
                                             int64_t K, void* dX, int64_t lddx, void* dW, int dW_dtype, float* dbias,
                                             void* workspace, size_t workspace_bytes, void* stream) {
    flp_status st = linear_sizes(M, N, K);
    if (st == FLP_OK) st = linear_act(activation);
    if (st == FLP_OK) st = linear_terms(d_terms, M);
    if (st == FLP_OK) st = weight_grad_checks(M, N, K, dW_dtype);
    if (st != FLP_OK) return st;
    if (!aligned16(dW)) return fail(FLP_ERR_INVALID_ARG, "dW must be 16-byte aligned");
    if (!aligned_to(dbias, 4)) return fail(FLP_ERR_INVALID_ARG, "dbias must be aligned to its elements");
    if (M > 0) {
        st = row_checks(dY, lddy, N, FLP_BF16, "dY must be non-null");
        if (st == FLP_OK && dW) st = row_checks(X, ldx, K, FLP_BF16, "dW needs X");
        if (st == FLP_OK && dX) st = row_checks(W, ldw, K, FLP_BF16, "dX needs W");
        if (st == FLP_OK && dX) st = row_checks(dX, lddx, K, FLP_BF16, "dX must be non-null");
        if (st == FLP_OK && activation != FLP_ACT_NONE)
            st = row_checks(pre, ldpre, N, FLP_BF16, "an activation's gradient needs pre");
        if (st != FLP_OK) return st;
    }
    if (!dX && !dW && !dbias) return FLP_OK;
    DevInfo* d;
    st = check_device(&d);
    if (st == FLP_OK) st = check_on_current_device(M > 0 ? dY : dW ? dW : dbias, "dY");
    if (st == FLP_OK) st = linear_attrs();
    if (st != FLP_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (dW) FLP_CUDA(cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * elem(dW_dtype), s));
        if (dbias) FLP_CUDA(cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, s));
        return FLP_OK;
    }
    const LinearGradLayout g = linear_grad_layout(dY, lddy, X, ldx, W, ldw, activation, d_terms, dX, dW, dbias, M, N, K, dW_dtype,
                                                  d->sm_count, d->pairs);
    if (!workspace || workspace_bytes < g.bytes || !aligned16(workspace))
        return fail(FLP_ERR_WORKSPACE, "linear backward workspace null, misaligned or too small");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int* err = reinterpret_cast<int*>(ws);
    FLP_CUDA(cudaMemsetAsync(err, 0, sizeof(int), s));
    bool after = false;
    if (g.copy_x || g.stack) {
        for (int i = 0; i < (g.stack ? 2 : 1); ++i)
            if ((st = align_rows(X, ldx, M, K, ws + g.off_x + i * M * pad8(K) * 2, pad8(K), s)) != FLP_OK) return st;
        X = ws + g.off_x, ldx = pad8(K), after = true;
    }
    if (g.copy_w) {
        if ((st = align_rows(W, ldw, N, K, ws + g.off_w, pad8(K), s)) != FLP_OK) return st;
        W = ws + g.off_w, ldw = pad8(K), after = true;
    }
    const bool vec = rows_bf16(dY, lddy) && N % 8 == 0 && (activation == FLP_ACT_NONE || rows_bf16(pre, ldpre));
    if (g.make_d || g.sums) {
        LinGradParams p{};
        p.dy = static_cast<const bf16*>(dY);
        p.lddy = lddy;
        p.pre = activation == FLP_ACT_NONE ? nullptr : static_cast<const bf16*>(pre);
        p.ldpre = ldpre;
        p.M = static_cast<int>(M);
        p.N = static_cast<int>(N);
        p.d = g.make_d ? reinterpret_cast<bf16*>(ws + g.off_d) : nullptr;
        p.lo = g.two || g.two_x ? reinterpret_cast<bf16*>(ws + g.off_lo) : nullptr;
        p.Np = static_cast<int>(pad8(N));
        p.part = g.sums ? g.blocks == 1 ? dbias : reinterpret_cast<float*>(ws + g.off_sums) : nullptr;
        p.rows = g.rows;
        const dim3 grid(static_cast<unsigned>(cdiv(N, 256)), static_cast<unsigned>(g.blocks));
        const cudaError_t e = lin_with_act(activation, [&](auto a) {
            if (vec)
                flp_linear_grad_kernel<false, decltype(a)::value><<<grid, LG_THREADS, 0, s>>>(p);
            else
                flp_linear_grad_kernel<true, decltype(a)::value><<<grid, LG_THREADS, 0, s>>>(p);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return cuda_fail(e, "flp_linear_grad_kernel launch");
        if (g.make_d) dY = ws + g.off_d, lddy = pad8(N);
        if (g.sums && g.blocks > 1) {
            st = launch_step(flp_linear_bias_join_kernel, cdiv(N, 32), 32 * LB_WAYS, 0, s, "flp_linear_bias_join_kernel launch", true,
                             reinterpret_cast<const float*>(ws + g.off_sums), g.blocks, static_cast<int>(N), dbias);
            if (st != FLP_OK) return st;
        }
        after = true;
    }
    if (dX) {
        LinEpilogue e{};
        e.y = static_cast<bf16*>(dX);
        e.ldy = lddx;
        e.vec = rows_bf16(dX, lddx) && K % 8 == 0;
        st = g.turned ? linear_turned(g.t, dY, lddy, W, ldw, true, M, K, N, e, err, kWaitLimitNs, -1, after, s, g.two_x)
                      : linear_product(g.l, dY, lddy, W, ldw, true, M, K, N, e, ws + g.off_part, err, d->pairs, kWaitLimitNs, -1, after, s,
                                       g.two_x);
        if (st != FLP_OK) return st;
        after = true;
    }
    if (!dW) return FLP_OK;
    st = weight_grad(dY, lddy, X, ldx, g.stack ? 2 * M : M, N, K, dW, dW_dtype, 0, ws + g.off_dw, d->pairs, after, s);
    if (st != FLP_OK || !g.two || g.stack) return st;
    return weight_grad(ws + g.off_lo, lddy, X, ldx, M, N, K, dW, dW_dtype, 1, ws + g.off_dw, d->pairs, true, s);
}

// M = 192 rows, N = 520 columns (two 256 x 512 tiles, the second of 8 columns), 192 deep:
// three blocks a tile, on one CTA pair; form 1: both tiles through partial tiles of one
// block; forms 2 and 3: turned tiles, in 3 over three CTAs of one block each.
extern "C" flp_status flp_selftest_linear_timeout(void* workspace, size_t workspace_bytes, int form, int stall_after,
                                                  int64_t wait_limit_ns, void* stream) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < FLP_SELFTEST_LINEAR_BYTES)
        return fail(FLP_ERR_WORKSPACE, "self-test needs FLP_SELFTEST_LINEAR_BYTES of workspace");
    if (wait_limit_ns <= 0 || wait_limit_ns > 60ll * 1000 * 1000 * 1000)
        return fail(FLP_ERR_INVALID_ARG, "wait_limit_ns must be in (0, 60 s]");
    if (form < 0 || form > 3) return fail(FLP_ERR_INVALID_ARG, "form must be 0 to 3");
    DevInfo* d;
    flp_status st = check_device(&d);
    if (st == FLP_OK) st = check_on_current_device(workspace, "workspace");
    if (st == FLP_OK) st = linear_attrs();
    if (st != FLP_OK) return st;
    const int64_t M = 192, N = 520, K = 192;
    LinPlan l = plan_linear(M, N, K, 1);
    l.width = 2 * BN;
    l.tn = 2;
    const bool split = form == 1;
    l.splits = split ? 3 : 1;
    l.whole = split ? 0 : 2;
    l.rest = split ? 2 : 0;
    l.units = l.whole + l.rest * l.splits;
    Regions r;
    r.take(kHeaderBytes);
    const size_t off_x = r.take(M * K * 2), off_w = r.take(N * K * 2);
    const size_t zero = r.bytes;
    const size_t off_part = r.take(2ull * 3 * M * 2 * BN * 4);
    if (r.bytes > FLP_SELFTEST_LINEAR_OUTPUT_OFFSET || FLP_SELFTEST_LINEAR_OUTPUT_OFFSET + M * N * 2 > FLP_SELFTEST_LINEAR_BYTES)
        return fail(FLP_ERR_UNSUPPORTED, "self-test layout exceeds its workspace");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LinEpilogue e{};
    e.y = reinterpret_cast<bf16*>(ws + FLP_SELFTEST_LINEAR_OUTPUT_OFFSET);
    e.ldy = N;
    e.vec = 1;
    FLP_CUDA(cudaMemsetAsync(ws, 0, zero, s));                       // error word, x, W
    FLP_CUDA(cudaMemsetAsync(ws + off_part, 0x3f, r.bytes - off_part, s));  // what the partial tiles
    FLP_CUDA(cudaMemsetAsync(e.y, 0x3f, M * N * 2, s));              // and the result have to replace
    const unsigned long long limit = static_cast<unsigned long long>(wait_limit_ns);
    const int stall = stall_after < 0 ? -1 : stall_after;
    int* err = reinterpret_cast<int*>(ws);
    if (form >= 2) {
        LinTurnPlan turned = plan_turned(M, N, K, 1);
        turned.split = form == 3 ? 3 : 1;
        turned.stages = 2;
        st = linear_turned(turned, ws + off_x, K, ws + off_w, K, false, M, N, K, e, err, limit, stall, false, s);
        return st == FLP_OK ? flp_get_error(workspace, stream) : st;
    }
    st = linear_product(l, ws + off_x, K, ws + off_w, K, false, M, N, K, e, ws + off_part, err, 1, limit, stall, false, s);
    return st == FLP_OK ? flp_get_error(workspace, stream) : st;
}

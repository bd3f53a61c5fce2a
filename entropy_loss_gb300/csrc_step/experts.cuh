// experts.cuh - tokens sorted by expert, their rows brought there and back, and
// the gradients.
//
// T tokens choose k experts each: S = T k slots, slot t k + j being token t's j-th
// choice.  A stable counting sort gives every slot a position, slots without an expert
// last.  With total = the number of slots that have one:
//     gather            xs[p] = x[slot(p) / k], 0 from total on
//     combine           y[t]  = sum_j w[t, j] ys[position(t k + j)]     (positions below total)
//     combine backward  dys[p] = w[slot(p)] dy[slot(p) / k], 0 from total on
//                       dw[t, j] = <dy[t], ys[position(t k + j)]>
// and the gather's gradient is the combine without weights.  All four run by token: its
// own row is read or written once, and only the k rows elsewhere are scattered, so
// nothing is read or written twice and no sum needs atomics.  All are bound by memory: of
// the measured copy rate, 32768 x 4 x 5120 in bf16 (tokens x k x width) gathers at 97 %,
// combines at 100 % (248 us) and takes its gradient at 100 % (447 us).
#pragma once
#include "../csrc/ptx.cuh"
#include "vec.cuh"

namespace flp {

// ----------------------------------------------------------------------- sort

constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_MAX_E = 1024;
constexpr int SORT_BLOCKS = 128;            // at most: a warp reads one expert's counts of all blocks at once
constexpr long long SORT_ONE_BLOCK = 8192;  // slots that one block sorts by itself

struct SortParams {
    const long long* experts;  // [S]
    long long S;
    int E;
    int per;     // slots of a block, a multiple of SORT_THREADS
    int blocks;
    int* part;   // [E + 1][SORT_BLOCKS]: each block's slots of each expert
    int* rows;   // [S] position of a slot
    int* slots;  // [S] slot at a position
    long long* counts;   // [E]
    long long* offsets;  // [E + 1]
};

__device__ __forceinline__ int sort_key(const SortParams& p, long long s) {
    const long long e = p.experts[s];
    return e >= 0 && e < p.E ? static_cast<int>(e) : p.E;
}

// This warp's run of the block's slots.
struct SortRun {
    long long lo, hi;
    __device__ __forceinline__ explicit SortRun(const SortParams& p) {
        const long long first = static_cast<long long>(blockIdx.x) * p.per, each = p.per / SORT_WARPS;
        lo = min(p.S, first + (threadIdx.x >> 5) * each);
        hi = min(p.S, lo + each);
    }
};

// hist[warp][e]: the warp's slots of expert e (E: without one).
__device__ __forceinline__ void sort_count(const SortParams& p, int* hist) {
    const int n = p.E + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < SORT_WARPS * n; i += SORT_THREADS) hist[i] = 0;
    __syncthreads();
    const SortRun run(p);
    for (long long s = run.lo + lane; s < run.hi; s += 32) atomicAdd(&hist[warp * n + sort_key(p, s)], 1);
    __syncthreads();
}

__global__ void __launch_bounds__(SORT_THREADS) flp_expert_count_kernel(const SortParams p) {
    extern __shared__ int hist[];
    griddep_launch_dependents();
    sort_count(p, hist);
    const int n = p.E + 1;
    for (int e = threadIdx.x; e < n; e += SORT_THREADS) {
        int sum = 0;
        for (int w = 0; w < SORT_WARPS; ++w) sum += hist[w * n + e];
        p.part[static_cast<long long>(e) * SORT_BLOCKS + blockIdx.x] = sum;
    }
}

// Positions.  A block knows what all blocks count of each expert, so it finds where its
// own slots of each expert begin without another pass; a warp then ranks its slots in
// order, 32 at a time.  Bound by the chain of its phases: 32 slots take 6 us in one block,
// 524288 slots of 256 experts 4 us of counting and 13 here, of which their 8 MB would take
// 1.2.
__global__ void __launch_bounds__(SORT_THREADS) flp_expert_place_kernel(const SortParams p) {
    extern __shared__ int hist[];
    __shared__ int total[SORT_MAX_E + 1], before[SORT_MAX_E + 1], sums[SORT_WARPS];
    const int n = p.E + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    sort_count(p, hist);
    if (p.blocks > 1) {
        griddep_wait();  // every block's counts
        for (int e = warp; e < n; e += SORT_WARPS) {
            const int4 v = *reinterpret_cast<const int4*>(p.part + static_cast<long long>(e) * SORT_BLOCKS + 4 * lane);
            const int c[4] = {v.x, v.y, v.z, v.w};
            int all = 0, mine = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int b = 4 * lane + i;
                all += b < p.blocks ? c[i] : 0;
                mine += b < static_cast<int>(blockIdx.x) ? c[i] : 0;
            }
            all = __reduce_add_sync(0xffffffffu, all);
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0) total[e] = all, before[e] = mine;
        }
    } else {
        for (int e = threadIdx.x; e < n; e += SORT_THREADS) {
            int sum = 0;
            for (int w = 0; w < SORT_WARPS; ++w) sum += hist[w * n + e];
            total[e] = sum, before[e] = 0;
        }
    }
    __syncthreads();
    // where each expert begins: an exclusive sum over the experts, one per thread
    const int e = threadIdx.x, mine = e < p.E ? total[e] : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int v = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        sums[lane] = v;
    }
    __syncthreads();
    const int begin = upto - mine + (warp ? sums[warp - 1] : 0);
    const int kept = sums[SORT_WARPS - 1];
    if (blockIdx.x == 0) {
        if (e < p.E) p.counts[e] = mine, p.offsets[e] = begin;
        if (e == 0) p.offsets[p.E] = kept;
    }
    if (e < n) {
        int at = (e < p.E ? begin : kept) + before[e];
        for (int w = 0; w < SORT_WARPS; ++w) {
            const int c = hist[w * n + e];
            hist[w * n + e] = at;
            at += c;
        }
    }
    if (e == 0 && n > SORT_THREADS) {  // 1024 experts: one thread more than there are
        int at = kept + before[p.E];
        for (int w = 0; w < SORT_WARPS; ++w) {
            const int c = hist[w * n + p.E];
            hist[w * n + p.E] = at;
            at += c;
        }
    }
    __syncthreads();
    const SortRun run(p);
    int* next = hist + warp * n;
    for (long long s0 = run.lo; s0 < run.hi; s0 += 32) {
        const long long s = s0 + lane;
        const bool on = s < run.hi;
        const int key = on ? sort_key(p, s) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, key), below = same & ((1u << lane) - 1);
        int pos = 0;
        if (on) pos = next[key] + __popc(below);
        __syncwarp();
        if (on && below == 0) next[key] += __popc(same);
        __syncwarp();
        if (on && static_cast<unsigned>(pos) < p.S) {  // beyond it only if the choices change under the call
            p.rows[s] = pos;
            p.slots[pos] = static_cast<int>(s);
        }
    }
}

// ----------------------------------------------------------------------- rows

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_WARPS = MOVE_THREADS / 32;

struct MoveParams {
    void* one;  // [T, H]: x, y or dy
    long long ld_one;
    void* many;  // [S, H]: xs, ys or dxs
    long long ld_many;
    void* out;  // [S, H]: dys
    long long ld_out;
    const void* weights;  // [T, k], or null: 1
    bool weights_f32;
    float* dweights;  // [T, k], or null
    const int* rows;  // [T, k]; what is no position is passed over
    const long long* total;
    long long T;
    int k, H;
    int chunks;  // of a row, each a warp's
};

__device__ __forceinline__ float move_weight(const MoveParams& p, long long slot) {
    if (!p.weights) return 1.f;
    return p.weights_f32 ? static_cast<const float*>(p.weights)[slot]
                         : __bfloat162float(static_cast<const bf16*>(p.weights)[slot]);
}

// A warp's token and chunk of its row.
template <typename T, int NV>
struct MoveUnit {
    static constexpr int V = wide_v<T>();
    long long t;
    int col, left;  // this lane's first column, and the columns from there on
    __device__ __forceinline__ MoveUnit(const MoveParams& p, long long token, int chunk) : t(token) {
        col = (chunk * 32 * NV + (threadIdx.x & 31)) * V;
        left = p.H - col;
    }
};

// Shared memory a warp moves loose vectors through.
template <bool LOOSE>
__device__ __forceinline__ uint32_t move_stage() {
    if constexpr (LOOSE) {
        __shared__ __align__(16) uint8_t words[MOVE_WARPS * WARP_WORDS_BYTES];
        return smem_addr(words) + (threadIdx.x >> 5) * WARP_WORDS_BYTES;
    }
    return 0;
}

constexpr int GATHER_NV = 4;
template <typename T, bool LOOSE>
__global__ void __launch_bounds__(MOVE_THREADS) flp_expert_gather_kernel(const MoveParams p) {
    constexpr int NV = GATHER_NV, V = wide_v<T>();
    const unsigned unit = blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    const unsigned token = unit / static_cast<unsigned>(p.chunks);
    const int lane = threadIdx.x & 31;
    const uint32_t stage = move_stage<LOOSE>();
    if (token >= p.T) return;
    const MoveUnit<T, NV> u(p, token, static_cast<int>(unit - token * p.chunks));
    const T* src = static_cast<const T*>(p.one) + u.t * p.ld_one + u.col;
    RowVecs<T, LOOSE, NV> x;
    x.load(src, u.left, true, u.t == 0 || u.t == p.T - 1, extent_of<T>(p.one, p.T, p.ld_one, p.H));
    const long long total = *p.total, S = p.T * p.k;
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = x.get(i, src, u.left, stage);
    for (int j0 = 0; j0 < p.k; j0 += 32) {
        const int rows = min(32, p.k - j0);
        const int mine = lane < rows ? p.rows[u.t * p.k + j0 + lane] : 0;
        for (int j = 0; j < rows; ++j) {
            const int pos = __shfl_sync(0xffffffffu, mine, j);
            if (static_cast<unsigned>(pos) >= S) continue;  // not a position
            T* dst = static_cast<T*>(p.many) + pos * p.ld_many + u.col;
            const bool on = pos < total;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                store_row_vec<T, LOOSE>(dst + i * 32 * V, on ? v[i] : make_uint4(0, 0, 0, 0), u.left - i * 32 * V, stage);
        }
    }
}

// Vectors a lane, and rows under way at a time (loose bf16 rows, 20000 x 2 x 1001: four rows
// 54 us, two 38; aligned ones, 8192 x 8 x 2048: 58 and 63, 32768 x 4 x 5120: 251 and 263).
constexpr int COMBINE_NV = 2;
template <typename T, bool LOOSE>
__global__ void __launch_bounds__(MOVE_THREADS) flp_expert_combine_kernel(const MoveParams p) {
    constexpr int NV = COMBINE_NV, J = LOOSE ? 2 : 4, V = wide_v<T>(), P = V / 2;
    const unsigned unit = blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    const unsigned token = unit / static_cast<unsigned>(p.chunks);
    const int lane = threadIdx.x & 31;
    const uint32_t stage = move_stage<LOOSE>();
    if (token >= p.T) return;
    const MoveUnit<T, NV> u(p, token, static_cast<int>(unit - token * p.chunks));
    const long long total = *p.total, S = p.T * p.k;
    const T* many = static_cast<const T*>(p.many) + u.col;
    const Extent all = extent_of<T>(p.many, S, p.ld_many, p.H);
    uint64_t sum[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) sum[i][q] = 0;
    for (int j0 = 0; j0 < p.k; j0 += 32) {
        const int rows = min(32, p.k - j0);
        const long long slot = u.t * p.k + j0 + lane;
        const int mine = lane < rows ? p.rows[slot] : 0;
        float w = lane < rows ? move_weight(p, slot) : 0.f;
        for (int j = 0; j < rows; j += J) {
            RowVecs<T, LOOSE, NV> x[J];
            const T* src[J];
            bool on[J];
#pragma unroll
            for (int c = 0; c < J; ++c) {
                const int pos = __shfl_sync(0xffffffffu, mine, min(j + c, rows - 1));
                src[c] = many + pos * p.ld_many;
                on[c] = j + c < rows && pos < total && static_cast<unsigned>(pos) < S;
                x[c].load(src[c], u.left, on[c], pos == 0 || pos == S - 1, all);
            }
#pragma unroll
            for (int c = 0; c < J; ++c) {
                const float wc = __shfl_sync(0xffffffffu, w, min(j + c, rows - 1));
                if (!on[c]) continue;  // the whole warp
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const uint4 v = x[c].get(i, src[c], u.left, stage);
#pragma unroll
                    for (int q = 0; q < P; ++q) sum[i][q] = f2_fma(Pairs<T>::get(v, q), f2_splat(wc), sum[i][q]);
                }
            }
        }
    }
    T* dst = static_cast<T*>(p.one) + u.t * p.ld_one + u.col;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        store_row_vec<T, LOOSE>(dst + i * 32 * V, Pairs<T>::put(sum[i]), u.left - i * 32 * V, stage);
}

// A token per block, or per warp (WARP): its k products with dy need the whole row.  Three
// blocks an SM of aligned rows (65536 x 8 x 512 takes 175 us, with the registers of two
// 197), two of loose ones (4096 x 4 x 2047 takes 53 us, three spill: 113).
constexpr int CBWD_NV = 2, CBWD_J = 4;
template <typename T, bool LOOSE, bool WARP>
__global__ void __launch_bounds__(MOVE_THREADS, LOOSE ? 2 : 3) flp_expert_combine_bwd_kernel(const MoveParams p) {
    constexpr int NV = CBWD_NV, J = CBWD_J, V = wide_v<T>(), P = V / 2;
    __shared__ float red[J][MOVE_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t = WARP ? static_cast<long long>(blockIdx.x) * MOVE_WARPS + warp : blockIdx.x;
    const uint32_t stage = move_stage<LOOSE>();
    if (WARP && t >= p.T) return;
    const long long total = *p.total, S = p.T * p.k;
    const Extent all_dy = extent_of<T>(p.one, p.T, p.ld_one, p.H), all_ys = extent_of<T>(p.many, S, p.ld_many, p.H);
    const bool dots = p.dweights != nullptr;
    for (int j0 = 0; j0 < p.k; j0 += J) {
        int pos[J];
        float w[J];
        bool here[J], on[J];
        uint64_t dot[J];
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const long long slot = t * p.k + j0 + c;
            pos[c] = j0 + c < p.k ? p.rows[slot] : -1;
            here[c] = static_cast<unsigned>(pos[c]) < S;
            on[c] = here[c] && pos[c] < total;
            w[c] = on[c] ? move_weight(p, slot) : 0.f;
            dot[c] = 0;
        }
        for (int chunk = WARP ? 0 : warp; chunk < p.chunks; chunk += WARP ? 1 : MOVE_WARPS) {
            const MoveUnit<T, NV> u(p, t, chunk);
            const T* from = static_cast<const T*>(p.one) + t * p.ld_one + u.col;
            RowVecs<T, LOOSE, NV> d, x[J];
            d.load(from, u.left, true, t == 0 || t == p.T - 1, all_dy);
            const T* src[J];
#pragma unroll
            for (int c = 0; c < J; ++c) {
                src[c] = static_cast<const T*>(p.many) + pos[c] * p.ld_many + u.col;
                x[c].load(src[c], u.left, dots && on[c], pos[c] == 0 || pos[c] == S - 1, all_ys);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint4 dv = d.get(i, from, u.left, stage);
                uint64_t dp[P];
#pragma unroll
                for (int q = 0; q < P; ++q) dp[q] = Pairs<T>::get(dv, q);
#pragma unroll
                for (int c = 0; c < J; ++c) {
                    if (!here[c]) continue;  // the whole group
                    if (dots && on[c]) {
                        const uint4 v = x[c].get(i, src[c], u.left, stage);
#pragma unroll
                        for (int q = 0; q < P; ++q) dot[c] = f2_fma(Pairs<T>::get(v, q), dp[q], dot[c]);
                    }
                    uint64_t g[P];
#pragma unroll
                    for (int q = 0; q < P; ++q) g[q] = on[c] ? f2_mul(dp[q], f2_splat(w[c])) : 0ull;
                    T* dst = static_cast<T*>(p.out) + pos[c] * p.ld_out + u.col;
                    store_row_vec<T, LOOSE>(dst + i * 32 * V, Pairs<T>::put(g), u.left - i * 32 * V, stage);
                }
            }
        }
        if (dots) {
#pragma unroll
            for (int c = 0; c < J; ++c) {
                const float s = warp_sum(f2_sum(dot[c]));
                if (WARP) {
                    if (lane == 0 && j0 + c < p.k) p.dweights[t * p.k + j0 + c] = on[c] ? s : 0.f;
                } else if (lane == 0) {
                    red[c][warp] = s;
                }
            }
            if (!WARP) {
                __syncthreads();
                if (threadIdx.x < J && j0 + threadIdx.x < p.k) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < MOVE_WARPS; ++i) s += red[threadIdx.x][i];
                    p.dweights[t * p.k + j0 + threadIdx.x] = s;  // 0 for a slot without an expert
                }
                __syncthreads();
            }
        }
    }
}

// ------------------------------------------------------------- short rows
//
// Aligned rows of up to 32 vectors would leave lanes of the warp a token has idle, or give it
// less than the latency of its rows is worth: a thread takes one vector of one token instead,
// and in the backward `lanes` of a warp (a power of two that holds a row) a token.  Bound by
// latency and issue.  Gather, combine and its backward, long way -> short way (graph replay,
// some 5 us of each an empty one): 65536 x 8 x 64 bf16 37 -> 17, 56 -> 23, 113 -> 37 us (the
// bytes 11, 11, 21); 65536 x 4 x 256 bf16, 32 vectors, 33 -> 31, 46 -> 42, 76 -> 66; at 48
// vectors, 40000 x 2 x 384, it would be 21 -> 21, 29 -> 30, 46 -> 62.

constexpr int SHORT_VECS = 32;

template <typename T>
__global__ void __launch_bounds__(MOVE_THREADS) flp_expert_gather_short_kernel(const MoveParams p) {
    constexpr int V = wide_v<T>();
    const unsigned vecs = static_cast<unsigned>(p.H / V), i = blockIdx.x * MOVE_THREADS + threadIdx.x, token = i / vecs;
    if (token >= p.T) return;
    const int col = static_cast<int>(i - token * vecs) * V;
    const long long total = *p.total, S = p.T * p.k;
    const uint4 v = ld_global_16(static_cast<const T*>(p.one) + token * p.ld_one + col, true);
    const int* rows = p.rows + static_cast<long long>(token) * p.k;
    for (int j = 0; j < p.k; ++j) {
        const int pos = rows[j];
        if (static_cast<unsigned>(pos) >= S) continue;  // not a position
        st_global_16(static_cast<T*>(p.many) + pos * p.ld_many + col, pos < total ? v : make_uint4(0, 0, 0, 0), true);
    }
}

template <typename T>
__global__ void __launch_bounds__(MOVE_THREADS) flp_expert_combine_short_kernel(const MoveParams p) {
    constexpr int V = wide_v<T>(), P = V / 2, J = 4;
    const unsigned vecs = static_cast<unsigned>(p.H / V), i = blockIdx.x * MOVE_THREADS + threadIdx.x, token = i / vecs;
    if (token >= p.T) return;
    const int col = static_cast<int>(i - token * vecs) * V;
    const long long total = *p.total, S = p.T * p.k, slot = static_cast<long long>(token) * p.k;
    uint64_t sum[P];
#pragma unroll
    for (int q = 0; q < P; ++q) sum[q] = 0;
    for (int j = 0; j < p.k; j += J) {
        uint4 v[J];
        float w[J];
        bool on[J];
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const int pos = j + c < p.k ? p.rows[slot + j + c] : -1;
            on[c] = static_cast<unsigned>(pos) < S && pos < total;
            w[c] = on[c] ? move_weight(p, slot + j + c) : 0.f;
            v[c] = ld_global_16(static_cast<const T*>(p.many) + pos * p.ld_many + col, on[c]);
        }
#pragma unroll
        for (int c = 0; c < J; ++c) {
            if (!on[c]) continue;
#pragma unroll
            for (int q = 0; q < P; ++q) sum[q] = f2_fma(Pairs<T>::get(v[c], q), f2_splat(w[c]), sum[q]);
        }
    }
    st_global_16(static_cast<T*>(p.one) + token * p.ld_one + col, Pairs<T>::put(sum), true);
}

template <typename T>
__global__ void __launch_bounds__(MOVE_THREADS) flp_expert_combine_bwd_short_kernel(const MoveParams p, int lanes) {
    constexpr int V = wide_v<T>(), P = V / 2, J = 4;
    const unsigned i = blockIdx.x * MOVE_THREADS + threadIdx.x, at = i / static_cast<unsigned>(lanes);
    const bool here = at < p.T;
    const long long token = here ? at : p.T - 1;  // the lanes past the last token help its warp's sums
    const int col = (threadIdx.x & (lanes - 1)) * V;
    const bool mine = here && col < p.H;
    const long long total = *p.total, S = p.T * p.k, slot = token * p.k;
    const uint4 dv = ld_global_16(static_cast<const T*>(p.one) + token * p.ld_one + col, mine);
    uint64_t d[P];
#pragma unroll
    for (int q = 0; q < P; ++q) d[q] = Pairs<T>::get(dv, q);
    const bool dots = p.dweights != nullptr;
    for (int j = 0; j < p.k; j += J) {
        uint4 v[J];
        int pos[J];
        float w[J];
        bool on[J];
#pragma unroll
        for (int c = 0; c < J; ++c) {
            pos[c] = j + c < p.k ? p.rows[slot + j + c] : -1;
            on[c] = static_cast<unsigned>(pos[c]) < S && pos[c] < total;
            w[c] = on[c] ? move_weight(p, slot + j + c) : 0.f;
            v[c] = ld_global_16(static_cast<const T*>(p.many) + pos[c] * p.ld_many + col, dots && mine && on[c]);
        }
#pragma unroll
        for (int c = 0; c < J; ++c) {
            uint64_t g[P], dot = 0;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                dot = f2_fma(Pairs<T>::get(v[c], q), d[q], dot);
                g[q] = on[c] ? f2_mul(d[q], f2_splat(w[c])) : 0ull;
            }
            st_global_16(static_cast<T*>(p.out) + pos[c] * p.ld_out + col, Pairs<T>::put(g),
                         mine && static_cast<unsigned>(pos[c]) < S);
            if (dots) {  // the whole grid
                float s = on[c] && mine ? f2_sum(dot) : 0.f;
                for (int o = lanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (here && col == 0 && j + c < p.k) p.dweights[slot + j + c] = s;
            }
        }
    }
}

}  // namespace flp

// logits.cuh - log-probabilities of given tokens from logits that are in memory, with
// the entropy and the top alternatives, and the gradient by the logits.
//
// With z = s x for a row x of logits (s > 0), M = max x and c = s log2 e:
//     S = sum_j 2^((x_j - M) c),   A = sum_j 2^((x_j - M) c) (x_j - M) c
//     lse = s M + ln S,   logprob = s (x_y - M) - ln S,   entropy = ln S - ln 2 A / S
// (lse and z_y, both large, are not subtracted: the log-probability keeps its digits).
// One pass: a thread holds (M, S, A) of what it has read and rescales S and A when its
// maximum grows; threads, warps and the blocks of a row (a cluster, joined through
// distributed shared memory) are merged at the end.
//
// The alternatives come out of the same pass.  The largest element that a group of threads
// has read is an element of the row, so the k-th largest of such maxima, over groups that
// read different elements, is a bound that at least k elements reach; elements below it
// are not among the k largest.  With 16 or 32 groups little more than k elements of what
// was read pass it, and it is taken again whenever the amount has doubled, from what the
// warps have left in shared memory by then (an older maximum is still an element: no
// barrier).  Until k groups have read anything above -inf (a masked beginning) it is taken
// after every chunk, by the whole block.  A vector whose largest element passes goes to a
// list in shared memory; at the end the listed vectors are read again (from the L2), and
// what of them passes the last bound is ranked by value and column, so that equal logits
// come out in the order of their columns.  When a list overflows under bounds that came too
// late (rising logits), the block reads its part again and lists it by the last one.  When
// more pass that than the list holds (many equal logits), it reads its part once more,
// taking the largest left of each chunk in turn.
//
// Bound by memory and, close behind it, by instructions: 8192 rows of 131072 bf16 logits
// (317 us at the measured copy rate) take 328 us without alternatives, 388 with 8, 416 with
// 20: what they add is each row's end, which its block's loads do not overlap.  Four blocks
// of 256 threads an SM (two of 512: 371 and 490 with 8; three of 256: 349 and 424); 4
// vectors a thread at a time (2: 388 and 461).  Rows taken by resident blocks in turn, the
// next ones copied ahead through shared memory, took 396 and 468.
#pragma once
#include <cfloat>
#include "vec.cuh"

namespace flp {

constexpr int TLP_MAX_TOP = 32;
// vectors, and then elements, that a block can list
template <int THREADS>
constexpr int TLP_LIST = THREADS == 32 ? 256 : 512;
constexpr int TLP_CLUSTER = 8;     // blocks of a row at most
constexpr int TLP_NV = 4;          // vectors that a thread takes at a time

struct TlpParams {
    const void* x;
    long long ld;
    const long long* y;
    long long M;
    int V;
    int per;      // vectors of a row that one block of its cluster reads, a multiple of 32
    int cluster;  // blocks of a row
    int top;
    long long ignore_index;
    float scale, c;  // s, s log2 e
    float* logprob;
    float* lse;
    float* entropy;    // or null
    float* top_value;  // [M, top]
    long long* top_index;
};

struct TlpStats {
    float m, s, a;
};

// A key orders by value, then by column, lower ones first; 0 is no key.
__device__ __forceinline__ unsigned long long tlp_key(float x, int col) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are equal
    const uint32_t o = b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
    return static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ float tlp_key_value(unsigned long long key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(o >> 31 ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int tlp_key_col(unsigned long long key) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}

// Element i of a vector's words.
template <typename T>
__device__ __forceinline__ float tlp_elem(const uint32_t* w, int i) {
    if constexpr (sizeof(T) == 2)
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
        return __uint_as_float(w[i]);
}

// The largest element of a vector; NaN are passed over.
template <typename T>
__device__ __forceinline__ float tlp_max(const uint32_t* w) {
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        return fmaxf(fmax3(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2])), __uint_as_float(w[3]));
    }
}

__device__ __forceinline__ float redux_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// A row as the 16-byte vectors of memory that hold it, counted from the one with its first
// element; `head` elements of that one lie before the row.  A row needs no alignment: the
// vectors at its ends are read element by element.
template <typename T>
struct TlpRow {
    static constexpr int V = wide_v<T>();
    const T* x;
    int cols, head;
    __device__ __forceinline__ TlpRow(const T* row, int n)
        : x(row), cols(n), head(static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T))) {}
    __device__ __forceinline__ int vecs() const { return (head + cols + V - 1) / V; }
    __device__ __forceinline__ int col(int v) const { return v * V - head; }
    // vector v (if `on`) as words, -inf in the places past the row's ends
    __device__ __forceinline__ void load(uint32_t* w, int v, bool on) const {
        constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        const int c = col(v);
        const bool inner = c >= 0 && c + V <= cols;
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, %6;\n\tmov.b32 %1, %6;\n\tmov.b32 %2, %6;\n\t"
            "mov.b32 %3, %6;\n\t@p ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3])
            : "l"(x + c), "r"(static_cast<int>(on && inner)), "n"(none));
        if (on && !inner) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if (c + q < 0 || c + q >= cols) continue;
                if constexpr (sizeof(T) == 2) {
                    const uint32_t e = reinterpret_cast<const unsigned short*>(x)[c + q];
                    w[q / 2] = q & 1 ? (w[q / 2] & 0xffffu) | e << 16 : (w[q / 2] & 0xffff0000u) | e;
                } else {
                    w[q] = __float_as_uint(x[c + q]);
                }
            }
        }
    }
};

// A of a chunk some of whose elements are masked, or lie past the row's end (the last chunk
// of a row that does not fill it): a term whose exponential is 0 is 0.  Out of line, from
// the chunk read once more, so that the loop need not keep it: 8192 x 131072 bf16 with every
// other logit masked takes 720 us, without a mask 333.
template <typename T, int NV, int THREADS>
__device__ __noinline__ float tlp_masked(const TlpRow<T> row, int v0, int v1, float base, float c) {
    float a = 0.f;
    for (int i = 0; i < NV; ++i) {
        uint32_t w[4];
        row.load(w, v0 + i * THREADS, v0 + i * THREADS < v1);
#pragma unroll
        for (int q = 0; q < TlpRow<T>::V; ++q) {
            const float t = (tlp_elem<T>(w, q) - base) * c, e = ex2_approx(t);
            a += e > 0.f ? e * t : 0.f;
        }
    }
    return a;
}

template <int THREADS>
struct TlpShared {
    static constexpr int WARPS = THREADS / 32;
    unsigned long long list[TLP_LIST<THREADS>];
    unsigned long long best[TLP_MAX_TOP];  // this block's, in order; 0: none
    unsigned long long warp_key[WARPS];
    __align__(16) float group[32];         // the largest that each group of threads has read
    TlpStats warp_stats[WARPS];
    TlpStats stats;                        // this block's
    int vecs[TLP_LIST<THREADS>];
    int n_vecs, n;                         // vectors and elements listed
    float bound, first;                    // the latest, and the first that meant something
};

// Leaves the largest that each group of `lanes` threads has read, and returns it.
template <int THREADS>
__device__ __forceinline__ float tlp_put_maxima(TlpShared<THREADS>& sh, float m, int lanes) {
    volatile float* group = sh.group;
    for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (threadIdx.x % lanes == 0) group[threadIdx.x / lanes] = m;
    return m;
}

// The k-th largest of the groups' maxima: the largest that k of them reach; above -inf.
template <int THREADS>
__device__ __forceinline__ float tlp_bound(const TlpShared<THREADS>& sh, int k, int lanes) {
    const int lane = threadIdx.x & 31, groups = THREADS / lanes;
    const volatile float* group = sh.group;
    const float mine = lane < groups ? group[lane] : -INFINITY;
    int reach = 0;
    for (int i0 = 0; i0 < groups; i0 += 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) reach += __shfl_sync(0xffffffffu, mine, i0 + i) >= mine ? 1 : 0;
    return redux_max(reach >= k ? fmaxf(mine, -FLT_MAX) : -FLT_MAX);
}

// A warp's statistics in one, in every lane.
__device__ __forceinline__ TlpStats tlp_warp(TlpStats u, float c) {
    TlpStats r;
    r.m = redux_max(u.m);
    // a part that holds nothing above -inf brings nothing (or the NaN that it met), and one
    // so far below that its factor is 0 nothing, however large d is
    const float d = u.m == -INFINITY ? 0.f : (u.m - r.m) * c, f = ex2_approx(d);
    r.s = warp_sum(u.s * f);
    r.a = warp_sum(f > 0.f ? f * (u.a + d * u.s) : 0.f);
    return r;
}

// best[] from the n keys of the list: a key's place is how many are above it.
template <int THREADS>
__device__ __forceinline__ void tlp_rank(TlpShared<THREADS>& sh, int n, int k) {
    if (threadIdx.x < TLP_MAX_TOP) sh.best[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const unsigned long long key = sh.list[i];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) above += sh.list[j] > key ? 1 : 0;
        if (above < k && key) sh.best[above] = key;
    }
    __syncthreads();
}

// The block's k largest, one after another, chunk by chunk (the list has overflowed).
template <typename T, int THREADS>
__device__ __noinline__ void tlp_again(TlpShared<THREADS>& sh, const TlpRow<T> row, int v0, int v1, int k) {
    constexpr int V = TlpRow<T>::V, NV = 2;
    if (threadIdx.x < TLP_MAX_TOP) sh.best[threadIdx.x] = 0;
    __syncthreads();
    for (int v = v0; v < v1; v += THREADS * NV) {
        uint32_t w[4 * NV];
        const int mine = v + threadIdx.x;
#pragma unroll
        for (int i = 0; i < NV; ++i) row.load(w + 4 * i, mine + i * THREADS, mine + i * THREADS < v1);
        unsigned long long last = ~0ull;
        for (int round = 0; round < k; ++round) {
            unsigned long long top = sh.best[k - 1];  // none at or below it is wanted
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float x = tlp_elem<T>(w + 4 * i, q);
                    if (!(x > -INFINITY)) continue;
                    const unsigned long long key = tlp_key(x, row.col(mine + i * THREADS) + q);
                    if (key < last && key > top) top = key;
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const unsigned long long u = __shfl_xor_sync(0xffffffffu, top, o);
                top = u > top ? u : top;
            }
            if ((threadIdx.x & 31) == 0) sh.warp_key[threadIdx.x >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < THREADS / 32; ++i) top = sh.warp_key[i] > top ? sh.warp_key[i] : top;
            const bool none = top == sh.best[k - 1];
            __syncthreads();
            if (none) break;
            last = top;
            if (threadIdx.x == 0) {
                int at = k - 1;
                for (; at > 0 && sh.best[at - 1] < top; --at) sh.best[at] = sh.best[at - 1];
                sh.best[at] = top;
            }
            __syncthreads();
        }
    }
}

// Lists the block's vectors that reach `bound` (its last), when the list that was built under
// the bounds of the way has overflowed.  Returns how many there are.
template <typename T, int THREADS>
__device__ __noinline__ int tlp_relist(TlpShared<THREADS>& sh, const TlpRow<T> row, int v0, int v1, float bound) {
    constexpr int NV = 2;
    __syncthreads();
    if (threadIdx.x == 0) sh.n_vecs = 0;
    __syncthreads();
    for (int v = v0 + threadIdx.x; v < v1; v += THREADS * NV) {
        uint32_t w[4 * NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) row.load(w + 4 * i, v + i * THREADS, v + i * THREADS < v1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!(tlp_max<T>(w + 4 * i) >= bound)) continue;
            const int n = atomicAdd(&sh.n_vecs, 1);
            if (n < TLP_LIST<THREADS>) sh.vecs[n] = v + i * THREADS;
        }
    }
    __syncthreads();
    return sh.n_vecs;
}

__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) flp_token_logprob_kernel(const TlpParams p) {
    constexpr int V = wide_v<T>(), NV = TLP_NV, P = Pairs<T>::N, WARPS = THREADS / 32;
    __shared__ TlpShared<THREADS> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const long long at = blockIdx.x / p.cluster;
    const TlpRow<T> row(static_cast<const T*>(p.x) + at * p.ld, p.V);
    const int vecs = row.vecs();
    const int v0 = min(vecs, rank * p.per), v1 = min(vecs, v0 + p.per);
    const int lanes = THREADS / (p.top <= 16 ? 16 : 32);  // of a group: more groups than alternatives
    if (threadIdx.x == 0) sh.n = sh.n_vecs = 0, sh.bound = -FLT_MAX;
    long long y = 0;
    float xy = 0.f;
    if (rank == 0 && threadIdx.x == 0) {
        y = p.y[at];
        if (y >= 0 && y < p.V) xy = static_cast<float>(row.x[y]);
    }
    __syncthreads();

    TlpStats st{-INFINITY, 0.f, 0.f};
    float bound = -INFINITY;
    bool late = true;  // the whole block's: fewer groups than alternatives have read anything
    uint32_t next[4 * NV];
    auto load = [&](int v) {
#pragma unroll
        for (int i = 0; i < NV; ++i) row.load(next + 4 * i, v + i * THREADS, v + i * THREADS < v1);
    };
    load(v0 + threadIdx.x);
    unsigned chunk = 0;
    for (int v = v0; v < v1; v += THREADS * NV, ++chunk) {
        const int mine = v + threadIdx.x;
        uint32_t w[4 * NV];
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) w[i] = next[i];
        if (v + THREADS * NV < v1) load(mine + THREADS * NV);
        float tops[NV], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) tops[i] = tlp_max<T>(w + 4 * i), top = fmaxf(top, tops[i]);
        const float m = fmaxf(st.m, top);
        const float base = m == -INFINITY ? 0.f : m;  // nothing above -inf yet: every term is 0
        const uint64_t minus = f2_splat(-base), c2 = f2_splat(p.c);
        uint64_t s2 = 0, a2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4 u = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const uint64_t t = f2_mul(f2_add(Pairs<T>::get(u, q), minus), c2), e = f2_ex2(t);
                s2 = f2_add(s2, e);
                a2 = f2_fma(e, t, a2);
            }
        }
        TlpStats now{m, f2_sum(s2), f2_sum(a2)};
        // an infinite exponent times its 0
        if (__any_sync(0xffffffffu, now.a != now.a && now.s == now.s))
            now.a = tlp_masked<T, NV, THREADS>(row, mine, v1, base, p.c);
        if (m > st.m) {
            const float d = st.m == -INFINITY ? 0.f : (st.m - m) * p.c, f = ex2_approx(d);
            now.a += f > 0.f ? f * (st.a + d * st.s) : 0.f;
            now.s += f * st.s;
            st = now;
        } else {
            st.s += now.s, st.a += now.a;
        }
        if (p.top > 0) {
            if (late || (chunk & (chunk + 1)) == 0) {  // 1, 2, 4, ... chunks read
                const float m = tlp_put_maxima(sh, st.m, lanes);
                // the first bound is everybody's, and so is every one until it means something (a
                // masked beginning); then one warp takes the new one, the others when they come by
                const bool all = late;
                if (late) late = __syncthreads_count(threadIdx.x % lanes == 0 && m > -FLT_MAX) < p.top;
                if (all || chunk % WARPS == warp) {
                    __syncwarp();
                    bound = tlp_bound(sh, p.top, lanes);
                    if (lane == 0) *static_cast<volatile float*>(&sh.bound) = bound;
                    if (all && threadIdx.x == 0) sh.first = bound;
                }
            }
            bound = fmaxf(bound, *static_cast<volatile float*>(&sh.bound));
            if (top >= bound) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (tops[i] >= bound) {
                        const int n = atomicAdd(&sh.n_vecs, 1);
                        if (n < TLP_LIST<THREADS>) sh.vecs[n] = mine + i * THREADS;
                    }
                }
            }
        }
    }

    // the threads' sums in one, then the warps', then the blocks'
    const float thread_max = st.m;
    st = tlp_warp(st, p.c);
    if (lane == 0) sh.warp_stats[warp] = st;
    if (p.top > 0) tlp_put_maxima(sh, thread_max, lanes);
    __syncthreads();
    const TlpStats nothing{-INFINITY, 0.f, 0.f};
    if (warp == 0) {
        st = tlp_warp(lane < WARPS ? sh.warp_stats[lane] : nothing, p.c);
        if (lane == 0) sh.stats = st;
    }
    if (p.top > 0) {
        bound = tlp_bound(sh, p.top, lanes);
        int listed = sh.n_vecs;
        if (listed > TLP_LIST<THREADS> && bound > sh.first) listed = tlp_relist(sh, row, v0, v1, bound);
        for (int i = threadIdx.x; i < min(listed, TLP_LIST<THREADS>); i += THREADS) {
            const int col = row.col(sh.vecs[i]);
            uint32_t w[4];
            row.load(w, sh.vecs[i], true);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float x = tlp_elem<T>(w, q);
                if (x >= bound) {
                    const int n = atomicAdd(&sh.n, 1);
                    if (n < TLP_LIST<THREADS>) sh.list[n] = tlp_key(x, col + q);
                }
            }
        }
        __syncthreads();
        const int n = sh.n;
        if (listed > TLP_LIST<THREADS> || n > TLP_LIST<THREADS>)
            tlp_again(sh, row, v0, v1, p.top);
        else
            tlp_rank(sh, n, p.top);
    }
    if (p.cluster > 1) {
        __syncthreads();
        cluster_sync();
        if (rank == 0) {
            if (warp == 0) {
                TlpStats u = nothing;
                if (lane < p.cluster) {
                    const uint32_t from = mapa_shared(smem_addr(&sh.stats), lane);
                    u = TlpStats{ld_cluster_f32(from), ld_cluster_f32(from + 4), ld_cluster_f32(from + 8)};
                }
                st = tlp_warp(u, p.c);
            }
            if (p.top > 0) {
                const int n = p.cluster * p.top;
                for (int i = threadIdx.x; i < n; i += THREADS)
                    sh.list[i] = ld_cluster_u64(mapa_shared(smem_addr(&sh.best[i % p.top]), i / p.top));
                __syncthreads();
                tlp_rank(sh, n, p.top);
            }
        }
        __syncthreads();
        cluster_sync();  // no block leaves while its results are read
        if (rank != 0) return;
    }
    // warp 0 writes the row: its lanes hold the sums, and what it ranked lies in best[]
    if (warp != 0) return;
    const bool empty = st.m == -INFINITY && st.s == 0.f;  // a row with nothing above -inf
    const bool nan = st.s != st.s;                        // one with a NaN or +inf
    const float ln_s = empty ? 0.f : logf(st.s);
    if (lane == 0) {
        const bool skip = y == p.ignore_index, bad = y < 0 || y >= p.V;
        p.lse[at] = empty ? -INFINITY : fmaf(p.scale, st.m, ln_s);
        const float lp = empty ? -INFINITY : nan ? st.s : p.scale * (xy - st.m) - ln_s;
        p.logprob[at] = skip ? 0.f : bad ? __uint_as_float(0x7fc00000u) : lp;
        const float h = ln_s - LN2 * (st.a / st.s);
        if (p.entropy) p.entropy[at] = skip || empty ? 0.f : h < 0.f ? 0.f : h;
    }
    if (lane < p.top) {
        const unsigned long long key = nan ? 0 : sh.best[lane];
        p.top_value[at * p.top + lane] = key ? p.scale * (tlp_key_value(key) - st.m) - ln_s : nan ? st.s : -INFINITY;
        p.top_index[at * p.top + lane] = key ? tlp_key_col(key) : -1;
    }
}

// ------------------------------------------------------------------- gradient
//
// With a_j = z_j - lse = ln p_j and H the entropy,
//     d z_j = s [ 1[j = y] g_lp - p_j (g_lp + g_ent (a_j + H)) ]:
// one product per element on top of the exponential.

struct TlpBwdParams {
    const void* x;
    long long ld;
    const long long* y;
    long long M;
    int V;
    int chunks;  // of a row, each a warp's
    long long ignore_index;
    float scale;
    const float* lse;
    const float* entropy;  // or null: no gradient of it
    const float* g_lp;     // or null: 0
    const float* g_ent;
    void* dx;
    long long lddx;
};

constexpr int TLPB_THREADS = 256;
constexpr int TLPB_NV = 4;

template <typename T, bool LOOSE>
__global__ void __launch_bounds__(TLPB_THREADS) flp_token_logprob_bwd_kernel(const TlpBwdParams p) {
    constexpr int V = wide_v<T>(), NV = TLPB_NV, P = Pairs<T>::N;
    __shared__ __align__(16) uint8_t words[LOOSE ? TLPB_THREADS / 32 * WARP_WORDS_BYTES : 16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage = smem_addr(words) + (LOOSE ? warp * WARP_WORDS_BYTES : 0);
    const unsigned unit = blockIdx.x * (TLPB_THREADS / 32) + warp, in_row = unit / static_cast<unsigned>(p.chunks);
    const long long at = in_row;
    if (at >= p.M) return;
    const int v0 = static_cast<int>(unit - in_row * p.chunks) * 32 * NV + lane;
    const T* row = static_cast<const T*>(p.x) + at * p.ld;
    T* out = static_cast<T*>(p.dx) + at * p.lddx;
    const long long y = p.y[at];
    const float lse = p.lse[at];
    const bool zero = y == p.ignore_index || lse == -INFINITY;
    const T* src = row + v0 * V;
    RowVecs<T, LOOSE, NV> x;
    x.load(src, p.V - v0 * V, !zero, at == 0 || at == p.M - 1, extent_of<T>(p.x, p.M, p.ld, p.V));
    const float g_lp = p.g_lp ? p.g_lp[at] : 0.f;
    const float g_ent = p.entropy && p.g_ent ? p.g_ent[at] : 0.f, h = p.entropy ? p.entropy[at] : 0.f;
    const uint64_t s2 = f2_splat(p.scale), off = f2_splat(-lse), log2e = f2_splat(LOG2E);
    const uint64_t k0 = f2_splat(-p.scale * (g_lp + g_ent * h)), k1 = f2_splat(-p.scale * g_ent);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (v0 + 32 * i) * V;
        uint64_t g[P];
        if (zero) {
#pragma unroll
            for (int q = 0; q < P; ++q) g[q] = 0;
        } else {
            const uint4 u = x.get(i, src, p.V - v0 * V, stage);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float lo, hi;
                f2_unpack(f2_fma(Pairs<T>::get(u, q), s2, off), lo, hi);
                // p is 0 from -150 on; a finite exponent keeps it so in the product below
                const uint64_t a = f2_pack(max_nan(lo, -1000.f), max_nan(hi, -1000.f));
                f2_unpack(f2_mul(a, log2e), lo, hi);
                g[q] = f2_mul(f2_pack(ex2_approx(lo), ex2_approx(hi)), f2_fma(a, k1, k0));
            }
            const long long hit = y - col;
            if (hit >= 0 && hit < V) {
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const float one = p.scale * g_lp;
                    if (hit >> 1 == q) g[q] = f2_add(g[q], f2_pack(hit & 1 ? 0.f : one, hit & 1 ? one : 0.f));
                }
            }
        }
        store_row_vec<T, LOOSE>(out + col, Pairs<T>::put(g), p.V - col, stage);
    }
}

}  // namespace flp

// balance.cuh - the load-balance loss of a mixture-of-experts router, its
// gradient and the per-expert counts.
//
//   live rows : the mask keeps them and some logit is above -inf; N of them
//   p         = softmax(logits of a live row)
//   chosen    : the top_k largest logits (equal ones: lowest index first; -inf
//               never; none in a row that holds NaN or +inf), or the caller's
//   c_e       = times e is chosen, C = sum c_e
//   loss      = coef E sum_e (c_e / C) (1/N) sum_t p_te        (0 if N or C is 0)
//   d loss / d z_tj = coef / N  p_tj (a_j - sum_e p_te a_e),  a_e = (E c_e - C) / C
// (a_e is centred: subtracting a constant changes nothing because sum p = 1,
// and keeps the difference free of cancellation when the load is near even.)
//
// Three launches: statistics of the rows (softmax, choice) with each block's
// sums per expert, the join of the blocks' sums into counts, loss and a_e, and
// the gradient, which reads the logits again (from L2 when they fit).
#pragma once
#include "vec.cuh"

namespace flp {

constexpr int BAL_MAX_E = 1024;
constexpr int BAL_THREADS = 256;
constexpr int BAL_JOIN_THREADS = 1024;

struct BalParams {
    const void* z;
    long long ld;
    const uint8_t* mask;       // NULL: every row
    const long long* experts;  // NULL: the top_k largest
    long long T;
    int E, k;
    double coef;
    void* grad;  // [T, E] in the logits' type; NULL: not wanted
    float* loss;
    long long* counts;  // [E]
    float2* stat;       // [T]: row maximum and 1 / sum of exponentials (0: not live)
    float* part_p;      // [blocks][E]
    int* part_c;        // [blocks][E]
    int* part_n;        // [blocks]
    float* load;        // [E]: a_e; [E]: coef / N
    int blocks;
};

// An integer that orders floats: larger float, larger key (NaN excluded; the
// two zeros are equal); 0 is below every float's key.
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);  // -0 -> +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ uint32_t group_umin(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_min_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ bool group_any(bool b) {
    return group_umax<L>(b ? 1u : 0u) != 0u;
}

__device__ __forceinline__ float load_logit(const bf16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}
__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }

// L lanes per row; lane l holds experts l, l + L, ..., NE of them.
template <typename T, int L, int NE>
__global__ void __launch_bounds__(BAL_THREADS) flp_balance_rows_kernel(const BalParams p) {
    extern __shared__ uint32_t dyn[];  // [E] float sums, [E] counts, one live count
    float* bp = reinterpret_cast<float*>(dyn);
    int* bc = reinterpret_cast<int*>(dyn + p.E);
    int* bn = bc + p.E;
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) bc[e] = 0;
    if (threadIdx.x == 0) *bn = 0;
    __syncthreads();
    constexpr int RPB = BAL_THREADS / L;
    const int l = threadIdx.x % L, sub = threadIdx.x / L;
    float psum[NE] = {};
    int cnt[NE] = {};
    int live_rows = 0;
    const long long stride = static_cast<long long>(gridDim.x) * RPB;
    // every lane of a warp makes the same trips: the row groups of a warp move together
    const long long first = static_cast<long long>(blockIdx.x) * RPB;
    for (long long base = first; base < p.T; base += stride) {
        const long long row = base + sub;
        const bool in = row < p.T;
        const T* z = static_cast<const T*>(p.z) + row * p.ld;
        float v[NE];
        float m = -INFINITY;
        bool odd = false;  // NaN or +inf
        const bool kept = in && (!p.mask || p.mask[row]);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = l + i * L;
            v[i] = kept && e < p.E ? load_logit(z + e) : -INFINITY;
            odd |= !(v[i] < INFINITY);
            m = fmaxf(m, v[i]);
        }
        odd = group_any<L>(odd);
        m = group_max<L>(m);
        const bool live = odd || m > -INFINITY;
        float s = 0.f;
        float ex[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            ex[i] = live ? expf(v[i] - m) : 0.f;
            s += ex[i];
        }
        s = group_sum<L>(s);
        const float inv = odd ? __uint_as_float(0x7fc00000u) : live ? 1.f / s : 0.f;
        if (live) {
#pragma unroll
            for (int i = 0; i < NE; ++i) psum[i] = fmaf(ex[i], inv, psum[i]);
        }
        if (l == 0 && in) {
            p.stat[row] = make_float2(m, inv);
            live_rows += live;
        }
        if (p.experts) {
            if (live)
                for (int j = l; j < p.k; j += L) {
                    const long long e = p.experts[row * p.k + j];
                    if (e >= 0 && e < p.E) atomicAdd(&bc[e], 1);  // integers: any order gives the same sum
                }
        } else {
            uint32_t key[NE];
#pragma unroll
            for (int i = 0; i < NE; ++i) key[i] = !odd && v[i] > -INFINITY ? order_key(v[i]) : 0u;
            for (int j = 0; j < p.k; ++j) {
                uint32_t top = key[0];
#pragma unroll
                for (int i = 1; i < NE; ++i) top = max(top, key[i]);
                top = group_umax<L>(top);
                uint32_t at = 0xffffffffu;  // the lowest expert that holds it
#pragma unroll
                for (int i = NE - 1; i >= 0; --i)
                    if (key[i] == top) at = static_cast<uint32_t>(l + i * L);
                at = group_umin<L>(at);
                if (top == 0u) at = 0xffffffffu;  // nothing left to choose
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    if (static_cast<uint32_t>(l + i * L) == at) {
                        ++cnt[i];
                        key[i] = 0u;
                    }
            }
        }
    }
    griddep_launch_dependents();
    // this block's sums: counts in any order, the fp32 sums row group by row group
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = l + i * L;
        if (e < p.E && cnt[i]) atomicAdd(&bc[e], cnt[i]);
    }
    if (l == 0 && live_rows) atomicAdd(bn, live_rows);
    // lanes of a warp that hold the same experts first
#pragma unroll
    for (int i = 0; i < NE; ++i)
#pragma unroll
        for (int o = L; o < 32; o <<= 1) psum[i] += __shfl_xor_sync(0xffffffffu, psum[i], o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = 0; w < BAL_THREADS / 32; ++w) {
        if (warp == w && lane < L) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = l + i * L;
                if (e < p.E) bp[e] = (w ? bp[e] : 0.f) + psum[i];
            }
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
        p.part_p[static_cast<long long>(blockIdx.x) * p.E + e] = bp[e];
        p.part_c[static_cast<long long>(blockIdx.x) * p.E + e] = bc[e];
    }
    if (threadIdx.x == 0) p.part_n[blockIdx.x] = *bn;
}

// One block: counts, loss and the centred loads from the blocks' sums, in 64
// bits and a fixed order.
__global__ void __launch_bounds__(BAL_JOIN_THREADS) flp_balance_join_kernel(const BalParams p) {
    __shared__ double dsum[32], tot_p[BAL_MAX_E];
    __shared__ long long isum[32], tot_c[BAL_MAX_E];
    __shared__ double sh_d;
    __shared__ long long sh_i[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    // a warp takes 32 experts at a time and, when there are few experts, a
    // share of the blocks
    const int groups = (p.E + 31) / 32;
    for (int e = threadIdx.x; e < p.E; e += BAL_JOIN_THREADS) tot_p[e] = 0., tot_c[e] = 0;
    __shared__ double wp[32][32];
    __shared__ long long wc[32][32];
    const int ways = max(1, 32 / groups);  // warps per group of experts
    for (int g0 = 0; g0 < groups; g0 += 32 / ways) {
        const int g = g0 + warp / ways, way = warp % ways;
        double a = 0.;
        long long c = 0;
        const int e = g * 32 + lane;
        const bool on = warp / ways < 32 / ways && g < groups && e < p.E;
        if (on)
            for (int b = way; b < p.blocks; b += ways) {
                a += p.part_p[static_cast<long long>(b) * p.E + e];
                c += p.part_c[static_cast<long long>(b) * p.E + e];
            }
        wp[warp][lane] = a;
        wc[warp][lane] = c;
        __syncthreads();
        if (on && way == 0) {
            for (int w = 1; w < ways; ++w) a += wp[warp + w][lane], c += wc[warp + w][lane];
            tot_p[e] = a;
            tot_c[e] = c;
        }
        __syncthreads();
    }
    // N and C
    long long n = 0, c = 0;
    for (int b = threadIdx.x; b < p.blocks; b += BAL_JOIN_THREADS) n += p.part_n[b];
    for (int e = threadIdx.x; e < p.E; e += BAL_JOIN_THREADS) c += tot_c[e];
    for (int which = 0; which < 2; ++which) {
        long long x = which ? c : n;
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) isum[warp] = x;
        __syncthreads();
        if (threadIdx.x == 0) {
            long long y = 0;
            for (int w = 0; w < 32; ++w) y += isum[w];
            sh_i[which] = y;
        }
        __syncthreads();
    }
    const long long N = sh_i[0], C = sh_i[1];
    const bool any = N > 0 && C > 0;
    // loss = coef (1 + sum_e a_e p_e / N)
    double part = 0.;
    for (int e = threadIdx.x; e < p.E; e += BAL_JOIN_THREADS) {
        const double a = any ? (static_cast<double>(p.E) * static_cast<double>(tot_c[e]) - static_cast<double>(C)) /
                                   static_cast<double>(C)
                             : 0.;
        p.load[e] = static_cast<float>(a);
        p.counts[e] = tot_c[e];
        part += a * tot_p[e];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) dsum[warp] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
        sh_d = 0.;
        for (int w = 0; w < 32; ++w) sh_d += dsum[w];
        *p.loss = any ? static_cast<float>(p.coef * (1. + sh_d / static_cast<double>(N))) : 0.f;
        p.load[p.E] = any ? static_cast<float>(p.coef / static_cast<double>(N)) : 0.f;
    }
    griddep_launch_dependents();
}

template <typename T, int L, int NE>
__global__ void __launch_bounds__(BAL_THREADS) flp_balance_grad_kernel(const BalParams p) {
    constexpr int RPB = BAL_THREADS / L;
    const int l = threadIdx.x % L, sub = threadIdx.x / L;
    griddep_wait();
    float a[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) a[i] = l + i * L < p.E ? p.load[l + i * L] : 0.f;
    const float scale = p.load[p.E];
    const long long stride = static_cast<long long>(gridDim.x) * RPB;
    for (long long base = static_cast<long long>(blockIdx.x) * RPB; base < p.T; base += stride) {
        const long long row = base + sub;
        const bool in = row < p.T;
        const float2 st = in ? p.stat[row] : make_float2(0.f, 0.f);
        const bool live = !(st.y == 0.f);  // NaN counts
        const T* z = static_cast<const T*>(p.z) + row * p.ld;
        float pr[NE];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = l + i * L;
            pr[i] = live && e < p.E ? expf(load_logit(z + e) - st.x) * st.y : 0.f;
            dot = fmaf(pr[i], a[i], dot);
        }
        dot = group_sum<L>(dot);
        T* g = static_cast<T*>(p.grad) + row * p.E;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = l + i * L;
            const float o[1] = {live ? pr[i] * (a[i] - dot) * scale : 0.f};
            if (in && e < p.E) store_vec<1>(g + e, o);
        }
    }
}

}  // namespace flp

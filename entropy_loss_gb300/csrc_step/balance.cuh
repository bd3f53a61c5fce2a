// balance.cuh - the load-balance loss of a mixture-of-experts router, its
// gradient and the per-expert counts.
//
//   live rows : the mask keeps them and some logit is above -inf; N of them
//   p         = softmax(logits of a live row)
//   chosen    : the top_k largest logits (equal ones: lowest index first; -inf
//               never; none in a row that holds NaN or +inf), or the caller's
//   c_e       = times e is chosen, C = sum c_e
//   loss      = coef E sum_e (c_e / C) (1/N) sum_t p_te        (0 if N or C is 0, but NaN
//               whenever a live row holds a NaN or +inf)
//   d loss / d z_tj = coef / N  p_tj (a_j - sum_e p_te a_e),  a_e = (E c_e - C) / C
// (a_e is centred: subtracting a constant changes nothing because sum p = 1,
// and keeps the difference free of cancellation when the load is near even.)
//
// Three launches: the rows' statistics (softmax, choice) with each block's sums
// per expert; the join of the blocks' sums; and the gradient, whose blocks turn
// the counts into the loads a_e and which reads the logits again (from L2 when
// they fit).  Few rows take one launch instead: a cluster of blocks joins its
// sums through distributed shared memory between the two passes.
//
// A row belongs to L lanes of a warp, lane l holding vectors l, l + L, ... of V
// experts: the sums per expert then stay in the same registers from row to row.
// The next row's logits are loaded before this row's are worked on.
//
// The floor is one read of the logits and one write of the gradient.  Few tokens are
// bound by the launch and the cluster's exchange (64 x 8: 8 us), many by the rows'
// pass, whose choice of experts takes most of the instructions: 65536 x 256 fp32, top
// 8, takes 48 us, 26 of them in the rows' pass (66 % of the issue slots; its 67 MB would
// take 10), the rest in the join and the gradient's, against a floor of 20 us; bf16, half
// the bytes, 49 us against 10; top 24 takes 132 us.  The gradient needs the counts of all rows, and so a second read of the
// logits (of which an SM's share, 441 KB in that case, does not fit its shared memory).
#pragma once
#include "vec.cuh"

namespace flp {

constexpr int BAL_MAX_E = 1024;
constexpr int BAL_THREADS = 512;
constexpr int BAL_BOUND_K = 24;  // experts of a row up to which they are chosen by a bound
constexpr int BAL_CLUSTER = 8;  // blocks of the one-launch form
constexpr int BAL_CLUSTER_TRIPS = 4;  // trips of its row loop up to which it is the faster one

struct BalParams {
    const void* z;
    long long ld;
    const uint8_t* mask;       // NULL: every row
    const long long* experts;  // NULL: the top_k largest
    long long T;
    int E, k;
    double coef;
    void* grad;      // [T, E] in the logits' type, or fp32; NULL: not wanted
    bool grad_f32;
    float* loss;
    long long* counts;  // [E]
    float2* stat;       // [T]
    float* part_p;      // [blocks][E]
    int* part_c;        // [blocks][E]; 2^31 of one block would need 5 TB of given experts
    int* part_n;        // [blocks]
    double* tot_p;      // [E]
    long long* tot_c;   // [E]
    long long* tot_n;   // [1]
    int blocks;
};

// An integer that orders floats: larger float, larger key (NaN excluded; the
// two zeros are equal).  The lowest finite value's is BAL_LOWEST, -inf's the one below.
constexpr uint32_t BAL_LOWEST = 0x00800000u;
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);  // -0 -> +0
    return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The larger of two, NaN if either is; and the largest over a row's lanes.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
template <int L>
__device__ __forceinline__ float group_max_nan(float v) {
    if constexpr (L == 32) {
        float m;
        asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
        return m;
    } else {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
// Largest and smallest over a warp (no NaN).
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
__device__ __forceinline__ float warp_min(float v) {
    float m;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Expert i of lane l.
template <int L, int V>
__device__ __forceinline__ int expert(int l, int i) {
    return i / V * (L * V) + l * V + i % V;
}

// A lane's logits as loaded (V per access), or -inf, and in fp32.
template <typename T, int V>
struct Logits;
template <>
struct Logits<float, 1> {
    float u;
    __device__ __forceinline__ void none() { u = -INFINITY; }
    __device__ __forceinline__ void load(const float* p) { u = __ldg(p); }
    __device__ __forceinline__ void to(float* v) const { v[0] = u; }
};
template <>
struct Logits<float, 2> {
    float2 u;
    __device__ __forceinline__ void none() { u = make_float2(-INFINITY, -INFINITY); }
    __device__ __forceinline__ void load(const float* p) { u = __ldg(reinterpret_cast<const float2*>(p)); }
    __device__ __forceinline__ void to(float* v) const { v[0] = u.x, v[1] = u.y; }
};
template <>
struct Logits<float, 4> {
    float4 u;
    __device__ __forceinline__ void none() { u = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ void load(const float* p) { u = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void to(float* v) const { v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w; }
};
template <>
struct Logits<bf16, 1> {
    unsigned short u;
    __device__ __forceinline__ void none() { u = 0xff80; }
    __device__ __forceinline__ void load(const bf16* p) { u = __ldg(reinterpret_cast<const unsigned short*>(p)); }
    __device__ __forceinline__ void to(float* v) const { v[0] = __uint_as_float(static_cast<uint32_t>(u) << 16); }
};
template <>
struct Logits<bf16, 2> {
    uint32_t u;
    __device__ __forceinline__ void none() { u = 0xff80ff80u; }
    __device__ __forceinline__ void load(const bf16* p) { u = __ldg(reinterpret_cast<const uint32_t*>(p)); }
    __device__ __forceinline__ void to(float* v) const {
        v[0] = __uint_as_float(u << 16), v[1] = __uint_as_float(u & 0xffff0000u);
    }
};
template <>
struct Logits<bf16, 4> {
    uint2 u;
    __device__ __forceinline__ void none() { u = make_uint2(0xff80ff80u, 0xff80ff80u); }
    __device__ __forceinline__ void load(const bf16* p) { u = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void to(float* v) const {
        v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
};

template <int V>
__device__ __forceinline__ void store_grad(float* p, const float* v) {
    if constexpr (V == 4)
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    else if constexpr (V == 2)
        __stcs(reinterpret_cast<float2*>(p), make_float2(v[0], v[1]));
    else
        __stcs(p, v[0]);
}
template <int V>
__device__ __forceinline__ void store_grad(bf16* p, const float* v) {
    if constexpr (V == 4)
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
    else if constexpr (V == 2)
        __stcs(reinterpret_cast<uint32_t*>(p), pack_bf16x2(v[0], v[1]));
    else
        *p = __float2bfloat16_rn(v[0]);
}

// Whether this lane's expert is among its row's k largest keys, ties to the lowest
// expert.  One expert per lane, L lanes: a lane's rank is the number of lanes before it.
template <int L>
__device__ __forceinline__ bool chosen_by_rank(uint32_t key, int l, int k) {
    int before = 0;
#pragma unroll
    for (int o = 1; o < L; ++o) {
        const int from = (l + o) % L;
        const uint32_t other = __shfl_sync(0xffffffffu, key, from, L);
        before += (other > key || (other == key && from < l)) ? 1 : 0;
    }
    return key >= BAL_LOWEST && before < k;
}

// The same for a warp with NE experts per lane (no NaN, no +inf): a lane's chosen
// experts are marked in fields of 4 bits, eight to a word, so that adding the word
// counts them all at once (and its set bits are their number).
//
// The k-th largest of the lanes' maxima bounds the k-th largest logit from below: those
// at or above the bound are candidates, and the smallest are dropped until k are left
// (about one for 256 experts and k = 8).  Above BAL_BOUND_K the experts are taken one at
// a time, which drops nothing when many of the largest share a lane (65536 x 256 fp32:
// k = 20 takes 95 us by the bound, 125 one at a time, k = 24 132 and 143, k = 28 199 and
// 163; bf16 102 and 124, 146 and 142, 288 and 160).
// `top`: the lane's largest logit, `most`: the row's.
template <int NE>
__host__ __device__ constexpr int bal_words() { return (NE + 7) / 8; }

template <int NE, int V>
__device__ __forceinline__ void choose(const float (&v)[NE], float top, float most, int l, int k,
                                       uint32_t (&marks)[bal_words<NE>()]) {
    constexpr uint32_t ALL = 0xffffffffu;
    constexpr float LOWEST = -3.402823466e38f;
    int left = k;  // experts still to take: all, or among the logits equal to `tie`
    float tie = 0.f;
#pragma unroll
    for (int w = 0; w < bal_words<NE>(); ++w) marks[w] = 0;
    if (k <= BAL_BOUND_K) {
        float bound = most;
        for (int j = 1; j < k; ++j) {
            if (top == bound) top = -INFINITY;
            bound = warp_max(top);
        }
        bound = fmaxf(bound, LOWEST);
        auto mark = [&]() {  // logits at or above the bound
            int mine = 0;
#pragma unroll
            for (int w = 0; w < bal_words<NE>(); ++w) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 8 * w; i < NE && i < 8 * w + 8; ++i) m += v[i] >= bound ? 1u << (4 * (i % 8)) : 0u;
                marks[w] = m;
                mine += __popc(m);
            }
            return __reduce_add_sync(ALL, mine);
        };
        int total = mark();
        left = 0;
        while (total > k) {
            float low = INFINITY;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (v[i] >= bound) low = fminf(low, v[i]);
            low = warp_min(low);
            bound = key_value(order_key(low) + 1);
            total = mark();
            if (total < k) {  // only some of the smallest fit
                tie = low;
                left = k - total;
            }
        }
        if (left == 0) return;
    }
    // one at a time: the lowest expert of the ties, or the largest that is left
    uint32_t rest[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) rest[i] = k > BAL_BOUND_K || v[i] == tie ? order_key(v[i]) : 0u;
    for (int j = 0; j < left; ++j) {
        uint32_t m = rest[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) m = max(m, rest[i]);
        m = __reduce_max_sync(ALL, m);
        if (m < BAL_LOWEST) break;
        uint32_t at = ALL;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
            if (rest[i] == m) at = static_cast<uint32_t>(expert<32, V>(l, i));
        at = __reduce_min_sync(ALL, at);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (static_cast<uint32_t>(expert<32, V>(l, i)) == at) {
                marks[i / 8] += 1u << (4 * (i % 8));
                rest[i] = 0;
            }
    }
}

// This block's sums per expert in shared memory: [4][E] fp32 probabilities (the
// first row ends up with the sums), [E] counts, one count of live rows.
constexpr int BAL_SHARES = 4;
struct BalSums {
    float* p;
    int* c;
    int* n;
};
inline size_t bal_smem(int64_t E) { return ((BAL_SHARES + 1) * static_cast<size_t>(E) + 1) * 4; }
__device__ __forceinline__ BalSums bal_sums(uint32_t* dyn, int E) {
    BalSums s;
    s.p = reinterpret_cast<float*>(dyn);
    s.c = reinterpret_cast<int*>(dyn + BAL_SHARES * E);
    s.n = s.c + E;
    return s;
}

// Whether the next row's logits are loaded before this row is worked on: not with 1024
// experts, whose rows spill as it is (fp32 177 -> 196 us; bf16 161 -> 154).
template <int NE>
constexpr bool BAL_AHEAD = NE <= 16;

// The lane's logits of a row; -inf where there is no expert.
template <typename T, int L, int NE, int V>
struct RowLogits {
    Logits<T, V> u[NE / V];
    __device__ __forceinline__ RowLogits() {
#pragma unroll
        for (int i = 0; i < NE / V; ++i) u[i].none();
    }
    // `z`: the row's logits from this lane's first on
    __device__ __forceinline__ void load(const BalParams& p, const T* z, bool on, int l) {
#pragma unroll
        for (int i = 0; i < NE; i += V)
            if (on && expert<L, V>(l, i) < p.E) u[i / V].load(z + i * L);
    }
    __device__ __forceinline__ void to(bool wanted, float (&v)[NE]) const {
#pragma unroll
        for (int i = 0; i < NE; i += V) {
            u[i / V].to(v + i);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i + j] = wanted ? v[i + j] : -INFINITY;
        }
    }
};

// The first pass over rows `block`, `block + blocks`, ... (times the rows a
// block holds).  Ends with a block barrier behind the sums.
// `stat` gets each row's maximum and 1 / sum of exponentials (0: not live), by
// row, or (kLocal) by the block's own count of rows.
template <typename T, int L, int NE, int V, bool kLocal>
__device__ __forceinline__ void balance_rows(const BalParams& p, const BalSums& sums, float2* stat, int block, int blocks) {
    constexpr int RPB = BAL_THREADS / L;
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) sums.c[e] = 0;
    if (threadIdx.x == 0) *sums.n = 0;
    __syncthreads();
    const int l = threadIdx.x % L, sub = threadIdx.x / L;
    float psum[NE] = {};
    // experts chosen in up to 15 rows (fewer than 32 lanes a row: in all rows)
    uint32_t cnt[bal_words<NE>()] = {};
    int since = 0;
    auto count = [&]() {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = expert<L, V>(l, i);
            const int c = NE == 1 ? cnt[0] : (cnt[i / 8] >> (4 * (i % 8))) & 15u;
            if (c && e < p.E) atomicAdd(&sums.c[e], c);  // integers: any order gives the same sum
        }
    };
    int live_rows = 0;
    const long long stride = static_cast<long long>(blocks) * RPB;
    const long long stride_z = stride * p.ld;
    // every lane of a warp makes the same trips: the row groups of a warp move together
    long long base = static_cast<long long>(block) * RPB;
    const T* z = static_cast<const T*>(p.z) + (base + sub) * p.ld + l * V;
    RowLogits<T, L, NE, V> next;
    if (BAL_AHEAD<NE>) next.load(p, z, base + sub < p.T, l);
    bool kept_next = base + sub < p.T && (!p.mask || p.mask[base + sub]);
    for (int own = sub; base < p.T; base += stride, own += RPB) {
        const long long row = base + sub;
        const bool kept = kept_next;
        float v[NE];
        if (!BAL_AHEAD<NE>) next.load(p, z, kept, l);
        next.to(L == 32 || kept, v);
        z += stride_z;
        const bool more = row + stride < p.T;
        if (BAL_AHEAD<NE>) next.load(p, z, more, l);
        kept_next = more && (!p.mask || p.mask[row + stride]);
        if (L == 32 && !kept) {  // the whole warp's row
            if (l == 0 && row < p.T) stat[kLocal ? own : row] = make_float2(0.f, 0.f);
            continue;
        }
        float top = v[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) top = max_nan(top, v[i]);
        const float most = group_max_nan<L>(top);
        // a row without any logit gets maximum 0: all its exponentials are 0; with a NaN
        // or +inf in a row some are NaN
        const bool live = !(most == -INFINITY), whole = most < INFINITY;
        const float m = live ? most : 0.f;
        auto choice = [&]() {
            if (p.experts) {
                if (live)
                    for (int j = l; j < p.k; j += L) {
                        const long long e = p.experts[row * p.k + j];
                        if (e >= 0 && e < p.E) atomicAdd(&sums.c[e], 1);
                    }
            } else if constexpr (L < 32) {
                cnt[0] += chosen_by_rank<L>(whole ? order_key(v[0]) : 0u, l, p.k) ? 1u : 0u;
            } else if (live && whole) {  // the same in the whole warp
                uint32_t marks[bal_words<NE>()];
                choose<NE, V>(v, top, most, l, p.k, marks);
#pragma unroll
                for (int w = 0; w < bal_words<NE>(); ++w) cnt[w] += marks[w];
                if (++since == 15) {
                    count();
#pragma unroll
                    for (int w = 0; w < bal_words<NE>(); ++w) cnt[w] = 0;
                    since = 0;
                }
            }
        };
        // 16 or more experts a lane: first, while their logits are all that is held (1024
        // bf16 experts 164 -> 161 us; 256 stay at 49)
        if constexpr (NE >= 16) choice();
        // the difference is formed first: its error grows with its own size alone
        float ex[NE], s = 0.f;
        if constexpr (NE == 1) {
            s = ex[0] = ex2_approx((v[0] - m) * LOG2E);
        } else {
            const uint64_t minus = f2_splat(-m), log2e = f2_splat(LOG2E);
#pragma unroll
            for (int i = 0; i < NE; i += 2) {
                f2_unpack(f2_mul(f2_add(f2_pack(v[i], v[i + 1]), minus), log2e), ex[i], ex[i + 1]);
                ex[i] = ex2_approx(ex[i]);
                ex[i + 1] = ex2_approx(ex[i + 1]);
                s += ex[i] + ex[i + 1];
            }
        }
        s = group_sum<L>(s);
        const float inv = live ? rcp_approx(s) : 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) psum[i] = fmaf(ex[i], inv, psum[i]);
        if (l == 0 && row < p.T) {
            stat[kLocal ? own : row] = make_float2(m, inv);
            live_rows += live;
        }
        if constexpr (NE < 16) choice();
    }
    // the fp32 sums in a fixed order: lanes of a warp that hold the same experts, then
    // the warps
    count();
    if (l == 0 && live_rows) atomicAdd(sums.n, live_rows);
#pragma unroll
    for (int i = 0; i < NE; ++i)
#pragma unroll
        for (int o = L; o < 32; o <<= 1) psum[i] += __shfl_xor_sync(0xffffffffu, psum[i], o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 0; w < BAL_THREADS / 32; w += BAL_SHARES) {
        if (warp >= w && warp < w + BAL_SHARES && lane < L) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = expert<L, V>(l, i);
                float* at = sums.p + (warp - w) * p.E + e;
                if (e < p.E) *at = (w ? *at : 0.f) + psum[i];
            }
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
        float t = sums.p[e];
#pragma unroll
        for (int w = 1; w < BAL_SHARES; ++w) t += sums.p[w * p.E + e];
        sums.p[e] = t;
    }
    __syncthreads();
}

// The centred load a_e = (E c - C) / C: the numerator is exact in 64-bit integers.
__device__ __forceinline__ float bal_load(int E, long long c, long long C) {
    return static_cast<float>(E * c - C) / static_cast<float>(C);
}

// hi + lo += x with the rounding of the sum kept in lo (a 64-bit sum's accuracy
// without 64-bit arithmetic, of which the chip has very little).
__device__ __forceinline__ void sum_exactly(float& hi, float& lo, float x) {
    const float s = hi + x;
    const float t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
}

// Sum over the block of 64-bit values, the same in every thread; `red` holds one per warp.
template <typename V>
__device__ __forceinline__ V bal_block_sum(V x, V* red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    V y = red[0];
    for (int w = 1; w < BAL_THREADS / 32; ++w) y += red[w];
    return y;
}

// From the totals (tot_c(e), tot_p(e), N): this lane's loads and the factor of
// the gradient; `first` (one block) also writes counts and loss.
template <int L, int NE, int V, typename FC, typename FP>
__device__ __forceinline__ float balance_loads(const BalParams& p, bool first, long long N, FC&& tot_c, FP&& tot_p,
                                               float (&a)[NE]) {
    __shared__ long long red_i[BAL_THREADS / 32];
    __shared__ double red_d[BAL_THREADS / 32];
    long long c = 0;
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) c += tot_c(e);
    const long long C = bal_block_sum(c, red_i);
    const bool any = N > 0 && C > 0;
    const int l = threadIdx.x % L;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = expert<L, V>(l, i);
        a[i] = any && e < p.E ? bal_load(p.E, tot_c(e), C) : 0.f;
    }
    if (first) {
        // loss = coef (1 + sum_e a_e p_e / N)
        double part = 0.;
        for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
            p.counts[e] = tot_c(e);
            part += static_cast<double>(p.E * tot_c(e) - C) * tot_p(e);
        }
        part = bal_block_sum(part, red_d);
        // nothing chosen: every factor of `part` is 0, and 0 times a row's NaN is NaN (rows
        // that all hold one choose nothing).  The reciprocal is formed beside the reduction
        // (65536 x 64 28 us; a division behind a branch on `any` 33, whichever block is last
        // waits for it).
        const double each = 1. / (any ? static_cast<double>(N) * static_cast<double>(C) : 1.);
        if (threadIdx.x == 0) *p.loss = static_cast<float>(p.coef * fma(part, each, any ? 1. : 0.));
    }
    return any ? static_cast<float>(p.coef / static_cast<double>(N)) : 0.f;
}

// The second pass.
template <typename T, int L, int NE, int V, bool kLocal>
__device__ __forceinline__ void balance_grad(const BalParams& p, const float2* stat, const float (&a)[NE], float scale,
                                             int block, int blocks) {
    constexpr int RPB = BAL_THREADS / L;
    const int l = threadIdx.x % L, sub = threadIdx.x / L;
    const long long stride = static_cast<long long>(blocks) * RPB;
    long long base = static_cast<long long>(block) * RPB;
    const long long stride_z = stride * p.ld;
    const T* z = static_cast<const T*>(p.z) + (base + sub) * p.ld + l * V;
    RowLogits<T, L, NE, V> next;
    if (BAL_AHEAD<NE>) next.load(p, z, base + sub < p.T, l);
    float2 st_next = base + sub < p.T ? stat[kLocal ? sub : base + sub] : make_float2(0.f, 0.f);
    for (int own = sub; base < p.T; base += stride, own += RPB) {
        const long long row = base + sub;
        const float2 st = st_next;
        float pr[NE];
        // a row that is not live (1 / sum = 0) has exponentials of 0 whatever it holds
        if (!BAL_AHEAD<NE>) next.load(p, z, row < p.T, l);
        next.to(!(st.y == 0.f), pr);
        z += stride_z;
        if (BAL_AHEAD<NE>) next.load(p, z, row + stride < p.T, l);
        if (row + stride < p.T) st_next = stat[kLocal ? own + RPB : row + stride];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            pr[i] = ex2_approx((pr[i] - st.x) * LOG2E) * st.y;
            dot = fmaf(pr[i], a[i], dot);
        }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < NE; ++i) pr[i] *= (a[i] - dot) * scale;
        auto store = [&](auto* g) {
#pragma unroll
            for (int i = 0; i < NE; i += V)
                if (row < p.T && expert<L, V>(l, i) < p.E) store_grad<V>(g + row * p.E + expert<L, V>(l, i), pr + i);
        };
        if (sizeof(T) == 4 || p.grad_f32)
            store(static_cast<float*>(p.grad));
        else
            store(static_cast<T*>(p.grad));
    }
}

template <typename T, int L, int NE, int V>
__global__ void __launch_bounds__(BAL_THREADS) flp_balance_rows_kernel(const BalParams p) {
    extern __shared__ uint32_t dyn[];
    const BalSums sums = bal_sums(dyn, p.E);
    balance_rows<T, L, NE, V, false>(p, sums, p.stat, blockIdx.x, gridDim.x);
    griddep_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
        p.part_p[static_cast<long long>(blockIdx.x) * p.E + e] = sums.p[e];
        p.part_c[static_cast<long long>(blockIdx.x) * p.E + e] = sums.c[e];
    }
    if (threadIdx.x == 0) p.part_n[blockIdx.x] = *sums.n;
}

// The blocks' sums per expert in a fixed order: 32 experts per block, a warp per
// share of the partials.
__global__ void __launch_bounds__(1024) flp_balance_join_kernel(const BalParams p) {
    __shared__ float wp[2][32][33];
    __shared__ long long wc[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * 32 + lane;
    griddep_wait();
    griddep_launch_dependents();
    float hi = 0.f, lo = 0.f;
    long long c = 0;  // up to T top_k where the given experts of a row repeat
    if (e < p.E) {
#pragma unroll 4
        for (int b = warp; b < p.blocks; b += 32) {
            sum_exactly(hi, lo, p.part_p[static_cast<long long>(b) * p.E + e]);
            c += p.part_c[static_cast<long long>(b) * p.E + e];
        }
    }
    wp[0][warp][lane] = hi;
    wp[1][warp][lane] = lo;
    wc[warp][lane] = c;
    __syncthreads();
    hi = wp[0][lane][warp];
    lo = wp[1][lane][warp];
    c = wc[lane][warp];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, hi, o);
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        sum_exactly(hi, lo, other);
        c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    const int f = blockIdx.x * 32 + warp;
    if (lane == 0 && f < p.E) {
        p.tot_p[f] = static_cast<double>(hi) + static_cast<double>(lo);
        p.tot_c[f] = c;
    }
    if (blockIdx.x == 0 && warp == 0) {
        int n = 0;
        for (int b = lane; b < p.blocks; b += 32) n += p.part_n[b];
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) *p.tot_n = n;
    }
}

// Loss, counts and (unless there is none to write) the gradient.
template <typename T, int L, int NE, int V>
__global__ void __launch_bounds__(BAL_THREADS) flp_balance_grad_kernel(const BalParams p) {
    griddep_wait();
    float a[NE];
    const float scale = balance_loads<L, NE, V>(
        p, blockIdx.x == 0, *p.tot_n, [&](int e) { return p.tot_c[e]; }, [&](int e) { return p.tot_p[e]; }, a);
    if (p.grad) balance_grad<T, L, NE, V, false>(p, p.stat, a, scale, blockIdx.x, gridDim.x);
}

// Both passes in one launch of one cluster.
template <typename T, int L, int NE, int V>
__global__ void __launch_bounds__(BAL_THREADS) __cluster_dims__(BAL_CLUSTER, 1, 1)
    flp_balance_cluster_kernel(const BalParams p) {
    extern __shared__ uint32_t dyn[];
    __shared__ double tot_p[BAL_MAX_E];
    __shared__ int tot_c[BAL_MAX_E];
    __shared__ float2 stat[BAL_CLUSTER_TRIPS * BAL_THREADS / L];
    const int rank = static_cast<int>(cluster_ctarank());
    const BalSums sums = bal_sums(dyn, p.E);
    balance_rows<T, L, NE, V, true>(p, sums, stat, rank, BAL_CLUSTER);
    cluster_sync();
    auto peer = [](const void* at, int r) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_addr(at), r)) : "memory");
        return v;
    };
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
        float hi = 0.f, lo = 0.f;
        int c = 0;
#pragma unroll
        for (int r = 0; r < BAL_CLUSTER; ++r) {
            sum_exactly(hi, lo, __uint_as_float(peer(sums.p + e, r)));
            c += static_cast<int>(peer(sums.c + e, r));
        }
        tot_p[e] = static_cast<double>(hi) + static_cast<double>(lo);
        tot_c[e] = c;
    }
    long long n = 0;
    for (int r = 0; r < BAL_CLUSTER; ++r) n += static_cast<int>(peer(sums.n, r));
    cluster_sync();  // the peers' sums have been read: blocks may go their own ways
    float a[NE];
    const float scale = balance_loads<L, NE, V>(
        p, rank == 0, n, [&](int e) -> long long { return tot_c[e]; }, [&](int e) { return tot_p[e]; }, a);
    if (p.grad) balance_grad<T, L, NE, V, true>(p, stat, a, scale, rank, BAL_CLUSTER);
}

}  // namespace flp

// checkpoint.cuh - 8-bit checkpoints of activations: written from bf16 or fp32
// rows, and read back.  vec.cuh has the block arithmetic.
#pragma once
#include "vec.cuh"

namespace flp {

struct CkParams {
    void* x;  // read by pack, written by unpack
    long long ldx;
    uint8_t* q;      // [M, Hp]
    uint8_t* scale;  // [M, Hp / 32]
    long long M;
    int H, Hp;
    unsigned per_row;            // vectors of a padded row (loose rows: a multiple of a warp's 32)
    unsigned long long inverse;  // 2^64 / per_row, rounded up: row = hi(vector * inverse)
    int* clear;                  // a word that unpack zeroes (NULL: none)
};

constexpr int CK_THREADS = 256;
// Vectors in flight per thread: writing a checkpoint 4 (32768 x 4096 bf16 62 us; 2:
// 68, 8: 66), reading one, which stores twice what it loads, 2 (67 us; 1:
// 72, 4: 75, 8: 94).
constexpr int CK_PACK_N = 4;
constexpr int CK_UNPACK_N = 2;

// Row and first column of vector j.
template <int V>
__device__ __forceinline__ long long ck_place(const CkParams& p, long long j, int& col) {
    const long long row = static_cast<long long>(__umul64hi(static_cast<unsigned long long>(j), p.inverse));
    col = static_cast<int>(j - row * p.per_row) * V;
    return row;
}

// A thread's vectors.  Loose rows: a warp's 32 vectors are consecutive in one row
// (lanes past the row's end idle), so that they can move as words.
template <typename T, int N>
struct CkPlaces {
    static constexpr int V = wide_v<T>();
    long long row[N];
    int col[N];
    int valid[N];  // elements of the row from there on; at most 0: nothing of x
    bool on[N];    // the checkpoint has the vector
    __device__ __forceinline__ explicit CkPlaces(const CkParams& p) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const long long j = static_cast<long long>(blockIdx.x) * (CK_THREADS * N) + k * CK_THREADS + threadIdx.x;
            row[k] = ck_place<V>(p, j, col[k]);
            on[k] = row[k] < p.M && col[k] < p.Hp;
            valid[k] = row[k] < p.M ? p.H - col[k] : -32 * V;
        }
    }
};

template <typename T, bool LOOSE>
__global__ void __launch_bounds__(CK_THREADS) flp_ck_pack_kernel(const CkParams p) {
    constexpr int P = Pairs<T>::N, N = LOOSE ? WarpWords<T>::N : 4;
    __shared__ __align__(16) uint8_t words[LOOSE ? Stage<T, true>::bytes(CK_THREADS) : 16];
    const CkPlaces<T, CK_PACK_N> at(p);
    const T* src[CK_PACK_N];
    uint32_t r[CK_PACK_N][N];
#pragma unroll
    for (int k = 0; k < CK_PACK_N; ++k) {
        src[k] = static_cast<const T*>(p.x) + at.row[k] * p.ldx + at.col[k];
        if constexpr (LOOSE) {
            const Extent all = extent_of<T>(p.x, p.M, p.ldx, p.H);
            const WarpWords<T> w(src[k], at.valid[k]);
            if (sizeof(T) == 4 || (at.row[k] > 0 && at.row[k] < p.M - 1)) {
                r[k][0] = ld_global_4_at<0>(w.mine, w.has(0));
                r[k][1] = ld_global_4_at<128>(w.mine, w.has(1));
                r[k][2] = ld_global_4_at<256>(w.mine, w.has(2));
                r[k][3] = ld_global_4_at<384>(w.mine, w.has(3));
                if (N == 5) r[k][N - 1] = ld_global_4_at<512>(w.mine, w.has(4));
            } else {  // the first or last row, of which a word may reach out of the matrix
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const char* a = w.mine + 128 * i;
                    r[k][i] = 0;
                    if (w.has(i))
                        r[k][i] = a >= all.lo && a + 4 <= all.hi ? *reinterpret_cast<const uint32_t*>(a) : outer_word(a, all);
                }
            }
        } else {
            const uint4 u = at.valid[k] > 0 ? __ldcs(reinterpret_cast<const uint4*>(src[k])) : make_uint4(0, 0, 0, 0);
            r[k][0] = u.x, r[k][1] = u.y, r[k][2] = u.z, r[k][3] = u.w;
        }
    }
#pragma unroll
    for (int k = 0; k < CK_PACK_N; ++k) {
        uint4 u = make_uint4(r[k][0], r[k][1], r[k][2], r[k][3]);
        if constexpr (LOOSE) {
            const uint32_t base = smem_addr(words) + threadIdx.x / 32 * WARP_WORDS_BYTES, lane = threadIdx.x & 31;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < 4 || lane == 0)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + (lane + 32 * i) * 4), "r"(r[k][i]) : "memory");
            __syncwarp();
            u = vec_of_words<T>(base, at.valid[k], sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(src[k]) & 2));
            __syncwarp();
        }
        uint32_t w[P / 2];
        uint64_t v[P];
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = Pairs<T>::get(u, i);
        const uint32_t byte = ck_quantise_pairs<T>(u, v, w);
        ck_store_words(p.q + at.row[k] * p.Hp + at.col[k], w, at.on[k]);
        st_global_1(p.scale + at.row[k] * (static_cast<unsigned>(p.Hp) / CK_BLOCK) + static_cast<unsigned>(at.col[k]) / CK_BLOCK,
                    byte, at.on[k] && at.col[k] % CK_BLOCK == 0);
    }
}

template <typename T, bool LOOSE>
__global__ void __launch_bounds__(CK_THREADS) flp_ck_unpack_kernel(const CkParams p) {
    constexpr int P = Pairs<T>::N, V = 2 * P;
    __shared__ __align__(16) uint8_t words[LOOSE ? Stage<T, true>::bytes(CK_THREADS) : 16];
    const uint32_t stage = smem_addr(words) + (LOOSE ? threadIdx.x / 32 * WARP_WORDS_BYTES : 0);
    const CkPlaces<T, CK_UNPACK_N> at(p);
    uint32_t w[CK_UNPACK_N][P / 2];
    uint32_t byte[CK_UNPACK_N];
    griddep_launch_dependents();  // the weight gradient's contraction may set up meanwhile
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.clear = 0;
#pragma unroll
    for (int k = 0; k < CK_UNPACK_N; ++k) {
        byte[k] = 0;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) w[k][i] = 0;
        if (at.on[k]) {
            const uint8_t* q = p.q + at.row[k] * p.Hp + at.col[k];
            if constexpr (V == 8) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q));
                w[k][0] = u.x, w[k][1] = u.y;
            } else {
                w[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(q));
            }
            byte[k] = __ldcs(p.scale + at.row[k] * (static_cast<unsigned>(p.Hp) / CK_BLOCK) +
                             static_cast<unsigned>(at.col[k]) / CK_BLOCK);
        }
    }
#pragma unroll
    for (int k = 0; k < CK_UNPACK_N; ++k) {
        uint64_t v[P];
        ck_pairs<V>(w[k], ck_step(byte[k]), v);
        store_row_vec<T, LOOSE>(static_cast<T*>(p.x) + at.row[k] * p.ldx + at.col[k], Pairs<T>::put(v), at.valid[k], stage);
    }
}

}  // namespace flp

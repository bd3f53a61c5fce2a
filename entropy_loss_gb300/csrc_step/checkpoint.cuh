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
    int H, Hp;
    unsigned per_row;            // vectors of a padded row
    unsigned long long inverse;  // 2^64 / per_row, rounded up: row = hi(vector * inverse)
    long long total;             // vectors in all
    int* clear;                  // a word that unpack zeroes (NULL: none)
};

constexpr int CK_THREADS = 256;
constexpr int CK_PER_THREAD = 4;  // vectors in flight per thread

// Row and first column of vector j.
template <int V>
__device__ __forceinline__ long long ck_place(const CkParams& p, long long j, int& col) {
    const long long row = static_cast<long long>(__umul64hi(static_cast<unsigned long long>(j), p.inverse));
    col = static_cast<int>(j - row * p.per_row) * V;
    return row;
}

// V elements per access: 16 bytes (V > 1), or one where rows are not 16-byte
// aligned or not whole vectors.
template <typename T, int V>
__global__ void __launch_bounds__(CK_THREADS) flp_ck_pack_kernel(const CkParams p) {
    const long long first = static_cast<long long>(blockIdx.x) * (CK_THREADS * CK_PER_THREAD) + threadIdx.x;
    Raw<T, V> r[CK_PER_THREAD];
    long long row[CK_PER_THREAD];
    int col[CK_PER_THREAD];
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        const long long j = first + k * CK_THREADS;
        row[k] = ck_place<V>(p, j, col[k]);
        if (j < p.total && col[k] < p.H)
            r[k].load(static_cast<const T*>(p.x) + row[k] * p.ldx + col[k]);
        else
            r[k].zero();
    }
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        uint32_t byte;
        uint32_t w[V > 4 ? 2 : 1];
        if constexpr (V > 1) {
            uint64_t v[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) v[i] = Pairs<T>::get(r[k].bits(), i);
            byte = ck_quantise_pairs<T>(r[k].bits(), v, w);
        } else {
            float v[V];
            r[k].to(v);
            byte = ck_quantise<V>(v, w);
        }
        if (first + k * CK_THREADS < p.total) {
            ck_store<V>(p.q + row[k] * p.Hp + col[k], w);
            if (col[k] % CK_BLOCK == 0) p.scale[row[k] * (p.Hp / CK_BLOCK) + col[k] / CK_BLOCK] = static_cast<uint8_t>(byte);
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(CK_THREADS) flp_ck_unpack_kernel(const CkParams p) {
    const long long first = static_cast<long long>(blockIdx.x) * (CK_THREADS * CK_PER_THREAD) + threadIdx.x;
    RawCk<V> r[CK_PER_THREAD];
    long long row[CK_PER_THREAD];
    int col[CK_PER_THREAD];
    griddep_launch_dependents();  // the weight gradient's contraction may set up meanwhile
    if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.clear = 0;
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        const long long j = first + k * CK_THREADS;
        row[k] = ck_place<V>(p, j, col[k]);
        if (j < p.total)
            r[k].load(p.q + row[k] * p.Hp, p.scale + row[k] * (p.Hp / CK_BLOCK), col[k]);
        else
            r[k].zero();
    }
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        if (first + k * CK_THREADS < p.total && col[k] < p.H) {
            T* x = static_cast<T*>(p.x) + row[k] * p.ldx + col[k];
            if constexpr (V > 1) {
                uint64_t v[V / 2];
                ck_pairs<V>(r[k].w, ck_step(r[k].byte), v);
                Pairs<T>::store(x, v);
            } else {
                float v[V];
                r[k].to(v);
                store_vec<V>(x, v);
            }
        }
    }
}

}  // namespace flp

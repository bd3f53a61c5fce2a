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
    unsigned per_row;  // vectors of a padded row
    long long total;   // vectors in all
};

constexpr int CK_THREADS = 256;
constexpr int CK_PER_THREAD = 4;  // vectors in flight per thread

template <typename T, int V>
__global__ void __launch_bounds__(CK_THREADS) flp_ck_pack_kernel(const CkParams p) {
    const long long first = static_cast<long long>(blockIdx.x) * (CK_THREADS * CK_PER_THREAD) + threadIdx.x;
    Raw<T, V> r[CK_PER_THREAD];
    long long row[CK_PER_THREAD];
    int col[CK_PER_THREAD];
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        const long long j = first + k * CK_THREADS;
        row[k] = j / p.per_row;
        col[k] = static_cast<int>(j - row[k] * p.per_row) * V;
        if (j < p.total && col[k] < p.H)
            r[k].load(static_cast<const T*>(p.x) + row[k] * p.ldx + col[k]);
        else
            r[k].zero();
    }
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        float v[V];
        uint32_t w[V > 4 ? 2 : 1];
        r[k].to(v);
        const uint32_t byte = ck_quantise<V>(v, w);
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
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        const long long j = first + k * CK_THREADS;
        row[k] = j / p.per_row;
        col[k] = static_cast<int>(j - row[k] * p.per_row) * V;
        if (j < p.total)
            r[k].load(p.q + row[k] * p.Hp, p.scale + row[k] * (p.Hp / CK_BLOCK), col[k]);
        else
            r[k].zero();
    }
#pragma unroll
    for (int k = 0; k < CK_PER_THREAD; ++k) {
        if (first + k * CK_THREADS < p.total && col[k] < p.H) {
            float v[V];
            r[k].to(v);
            store_vec<V>(static_cast<T*>(p.x) + row[k] * p.ldx + col[k], v);
        }
    }
}

}  // namespace flp

// checkpoint.cuh - 8-bit checkpoints of activations: written from bf16 or fp32
// rows, and read back.  vec.cuh has the block arithmetic.
//
// One pass, bound by the bytes: 32768 x 4096 bf16 is written in 62 us (97 % of the
// measured copy rate) and read back in 60 us (100 %).  A thread takes a vector, so a
// block of 32 columns is four (bf16) or eight (fp32) neighbouring lanes, whose largest
// magnitude is exchanged by shuffles; no shared memory and nothing read twice.
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
// Vectors in flight per thread: writing a checkpoint 4 (32768 x 4096 bf16 62 us; 2: 67, 8
// spill), reading one, which stores twice what it loads, 2 (60 us; 1: 72, 4: 63).
constexpr int CK_PACK_N = 4;
constexpr int CK_UNPACK_N = 2;
// Blocks an SM must hold of the writing kernel: 5 bound the registers of aligned rows
// (bf16 65 -> 62 us, fp32 110 -> 101 us); loose ones need more (0: no bound).
constexpr int ck_pack_blocks(bool loose) { return loose ? 0 : 5; }

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
__global__ void __launch_bounds__(CK_THREADS, ck_pack_blocks(LOOSE)) flp_ck_pack_kernel(const CkParams p) {
    constexpr int P = Pairs<T>::N, N = LOOSE ? WarpWords<T>::N : 4;
    __shared__ __align__(16) uint8_t words[LOOSE ? Stage<T, true>::bytes(CK_THREADS) : 16];
    const CkPlaces<T, CK_PACK_N> at(p);
    const T* src[CK_PACK_N];
    uint32_t r[CK_PACK_N][N];
#pragma unroll
    for (int k = 0; k < CK_PACK_N; ++k) {
        src[k] = static_cast<const T*>(p.x) + at.row[k] * p.ldx + at.col[k];
        if constexpr (LOOSE) {
            load_words<T>(r[k], src[k], at.valid[k], at.row[k] == 0 || at.row[k] >= p.M - 1,
                          extent_of<T>(p.x, p.M, p.ldx, p.H));
        } else {
            const uint4 u = at.valid[k] > 0 ? __ldcs(reinterpret_cast<const uint4*>(src[k])) : make_uint4(0, 0, 0, 0);
            r[k][0] = u.x, r[k][1] = u.y, r[k][2] = u.z, r[k][3] = u.w;
        }
    }
#pragma unroll
    for (int k = 0; k < CK_PACK_N; ++k) {
        uint4 u;
        if constexpr (LOOSE)
            u = settle_words<T>(r[k], src[k], at.valid[k], smem_addr(words) + threadIdx.x / 32 * WARP_WORDS_BYTES);
        else
            u = make_uint4(r[k][0], r[k][1], r[k][2], r[k][3]);
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

// Loose bf16 rows copied to rows of Hp elements at `q`, 16-byte aligned, zeros behind
// each row's H elements: TMA reads the weight gradient's dY from there.  Bound by the
// words' loads as in the kernels above (loose rows of 4095 are packed at 64 % of the
// copy rate), a few percent of the contraction that follows.
__global__ void __launch_bounds__(CK_THREADS) flp_align_rows_kernel(const CkParams p) {
    __shared__ __align__(16) uint8_t words[Stage<bf16, true>::bytes(CK_THREADS)];
    const CkPlaces<bf16, CK_PACK_N> at(p);
    const bf16* src[CK_PACK_N];
    uint32_t r[CK_PACK_N][WarpWords<bf16>::N];
#pragma unroll
    for (int k = 0; k < CK_PACK_N; ++k) {
        src[k] = static_cast<const bf16*>(p.x) + at.row[k] * p.ldx + at.col[k];
        load_words<bf16>(r[k], src[k], at.valid[k], at.row[k] == 0 || at.row[k] >= p.M - 1,
                         extent_of<bf16>(p.x, p.M, p.ldx, p.H));
    }
#pragma unroll
    for (int k = 0; k < CK_PACK_N; ++k) {
        const uint4 u = settle_words<bf16>(r[k], src[k], at.valid[k], smem_addr(words) + threadIdx.x / 32 * WARP_WORDS_BYTES);
        st_global_16(reinterpret_cast<bf16*>(p.q) + at.row[k] * p.Hp + at.col[k], u, at.on[k]);
    }
}

}  // namespace flp

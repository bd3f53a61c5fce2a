// vec.cuh - what the training-step kernels share: rows as 16-byte vectors (for
// aligned rows and for any others), row reductions, and the 8-bit checkpoint's
// block arithmetic.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace flp {

using bf16 = __nv_bfloat16;

// Elements of a 16-byte vector.
template <typename T>
__host__ __device__ constexpr int wide_v() { return 16 / static_cast<int>(sizeof(T)); }

// --------------------------------------------------------------- packed pairs

__device__ __forceinline__ uint64_t f2_splat(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return lo + hi;
}

// A vector as packed fp32 pairs (two lanes per instruction), and pairs rounded
// once to a vector (nearest, ties to even).
template <typename T>
struct Pairs;
template <>
struct Pairs<bf16> {
    static constexpr int N = 4;  // pairs of a vector
    __device__ __forceinline__ static uint64_t get(const uint4& u, int i) {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ static uint4 put(const uint64_t (&v)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(v[i], lo, hi);
            w[i] = pack_bf16x2(lo, hi);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Pairs<float> {
    static constexpr int N = 2;
    __device__ __forceinline__ static uint64_t get(const uint4& u, int i) {
        return i == 0 ? f2_pack(__uint_as_float(u.x), __uint_as_float(u.y))
                      : f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    __device__ __forceinline__ static uint4 put(const uint64_t (&v)[2]) {
        float a, b, c, d;
        f2_unpack(v[0], a, b);
        f2_unpack(v[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
};

// V parameter values (norm weight or bias, of either type) from `col` on as
// pairs, `none` where there are none.
template <int V, bool LOOSE>
__device__ __forceinline__ void param_pairs(const void* base, bool f32, int col, int cols, float none,
                                            uint64_t (&v)[V / 2]) {
    float w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = none;
    if (base && col < cols) {
        if constexpr (LOOSE) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (col + i < cols)
                    w[i] = f32 ? __ldg(static_cast<const float*>(base) + col + i)
                               : __bfloat162float(static_cast<const bf16*>(base)[col + i]);
            }
        } else if (f32) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + col + i));
                w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const bf16*>(base) + col + i));
                w[i] = __uint_as_float(u.x << 16), w[i + 1] = __uint_as_float(u.x & 0xffff0000u);
                w[i + 2] = __uint_as_float(u.y << 16), w[i + 3] = __uint_as_float(u.y & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = f2_pack(w[2 * i], w[2 * i + 1]);
}

// ------------------------------------------------------------------- accesses

// Accesses with a predicate of their own instead of a branch around them.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on) {
    if constexpr (BYTES == 16)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
                     "l"(src), "r"(static_cast<int>(on))
                     : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], %2;\n\t}" ::"r"(dst),
            "l"(src), "n"(BYTES), "r"(static_cast<int>(on))
            : "memory");
}
// 4 bytes from src + OFF to dst + OFF.
template <int OFF>
__device__ __forceinline__ void cp_async_4_at(uint32_t dst, const void* src, bool on) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p cp.async.ca.shared.global [%0 + %2], [%1 + %2], 4;\n\t}" ::"r"(dst),
        "l"(src), "n"(OFF), "r"(static_cast<int>(on))
        : "memory");
}
// The word at p + OFF, or 0.
template <int OFF>
__device__ __forceinline__ uint32_t ld_global_4_at(const void* p, bool on) {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.cs.b32 %0, [%1 + %2];\n\t}"
                 : "=&r"(x)
                 : "l"(p), "n"(OFF), "r"(static_cast<int>(on)));
    return x;
}
__device__ __forceinline__ void st_global_16(void* p, uint4 u, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(p),
                 "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w), "r"(static_cast<int>(on))
                 : "memory");
}
__device__ __forceinline__ void st_global_8(void* p, uint32_t x, uint32_t y, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p st.global.v2.b32 [%0], {%1, %2};\n\t}" ::"l"(p), "r"(x), "r"(y),
                 "r"(static_cast<int>(on))
                 : "memory");
}
__device__ __forceinline__ void st_global_4(void* p, uint32_t x, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b32 [%0], %1;\n\t}" ::"l"(p), "r"(x),
                 "r"(static_cast<int>(on))
                 : "memory");
}
__device__ __forceinline__ void st_global_1(void* p, uint32_t x, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.u8 [%0], %1;\n\t}" ::"l"(p), "r"(x),
                 "r"(static_cast<int>(on))
                 : "memory");
}
__device__ __forceinline__ void st_shared_zero_16(uint32_t a) { st_shared_v4(a, 0, 0, 0, 0); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_16(uint32_t a) {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(a) : "memory");
    return u;
}
__device__ __forceinline__ uint2 ld_shared_8(uint32_t a) {
    uint2 u;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(a) : "memory");
    return u;
}
__device__ __forceinline__ uint32_t ld_shared_4(uint32_t a) {
    uint32_t u;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(a) : "memory");
    return u;
}

// ------------------------------------------- vectors on their way through smem
//
// Rows S ahead are copied into shared memory, so that the bytes in flight are not
// limited by registers.  Aligned rows (16-byte base and pitch, whole vectors) move
// 16 bytes at a time, and a thread copies exactly the vectors that it will itself
// read: its completed cp.async group is all the synchronisation there is.
//
// Loose rows (any others) move 4-byte words: a warp copies the words that hold its
// 32 consecutive vectors, lane by lane, which coalesces at any address, and reads
// vectors from them after a warp barrier.  A bf16 row may start at an odd element;
// then the vectors straddle words and are shifted out (one word more).

// First and one past the last byte of a matrix: no word that reaches out of it is
// accessed; its one element inside is then accessed alone.
struct Extent {
    const char* lo;
    const char* hi;
};

template <typename T>
__device__ __forceinline__ Extent extent_of(const void* base, long long rows, long long pitch, int cols) {
    const char* b = static_cast<const char*>(base);
    return {b, b + ((rows - 1) * pitch + cols) * static_cast<long long>(sizeof(T))};
}

// A warp's 32 consecutive vectors in a loose row, of which lane `lane` moves words
// lane, lane + 32, ... counted from the one that holds the first element.
template <typename T>
struct WarpWords {
    static constexpr int V = wide_v<T>();
    static constexpr int N = sizeof(T) == 2 ? 5 : 4;  // words per lane, the last of five lane 0's alone
    const char* mine;  // this lane's first word
    int bytes;         // from there to the end of what the row holds of the vectors
    bool odd;          // the first word starts with an element that is not the warp's
    // `src`: this lane's vector, of which and beyond the row holds `valid` elements
    __device__ __forceinline__ WarpWords(const T* src, int valid) {
        const int lane = threadIdx.x & 31;
        const uintptr_t at = reinterpret_cast<uintptr_t>(src);
        odd = sizeof(T) == 2 && (at & 2);
        // the vectors of two lanes are 16 bytes apart, their words 4
        mine = reinterpret_cast<const char*>(at & ~static_cast<uintptr_t>(3)) - 12 * lane;
        const int left = min(32 * V, valid + lane * V);
        bytes = (left > 0 ? left * static_cast<int>(sizeof(T)) - 4 * lane : -512) + (odd ? 2 : 0);
    }
    // whether word i holds an element of the row, and whether it holds nothing else behind it
    __device__ __forceinline__ bool has(int i) const { return bytes > 128 * i; }
    __device__ __forceinline__ bool whole(int i) const { return bytes >= 128 * i + 4; }
};

// The one element inside the matrix of a bf16 word that reaches out of it, in its place.
__device__ __forceinline__ uint32_t outer_word(const char* w, const Extent& all) {
    const int half = w < all.lo ? 2 : 0;
    return static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(w + half)) << (8 * half);
}

// This lane's vector from the warp's words at `base` (`odd`: the first
// word starts with an element that is not the warp's); elements past `valid` zero.
template <typename T>
__device__ __forceinline__ uint4 vec_of_words(uint32_t base, int valid, bool odd) {
    const uint32_t at = base + (threadIdx.x & 31) * 16;
    uint4 u = ld_shared_16(at);
    if constexpr (sizeof(T) == 2) {
        const uint32_t next = ld_shared_4(at + 16), shift = odd ? 16u : 0u;
        u = make_uint4(__funnelshift_r(u.x, u.y, shift), __funnelshift_r(u.y, u.z, shift),
                       __funnelshift_r(u.z, u.w, shift), __funnelshift_r(u.w, next, shift));
        if (valid < 8) {
            uint32_t o[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = 2 * i + 1 < valid ? o[i] : 2 * i < valid ? (o[i] & 0xffffu) : 0u;
            u = make_uint4(o[0], o[1], o[2], o[3]);
        }
    } else if (valid < 4) {
        u = make_uint4(valid > 0 ? u.x : 0u, valid > 1 ? u.y : 0u, valid > 2 ? u.z : 0u, 0u);
    }
    return u;
}

// The words of the matrix's first or last row, of which one may reach out of it
// (out of line: two rows need it).
template <typename T>
__device__ __noinline__ void fetch_edge_words(uint32_t at, const T* src, int valid, const char* lo, const char* hi) {
    const WarpWords<T> w(src, valid);
#pragma unroll
    for (int i = 0; i < WarpWords<T>::N; ++i) {
        const char* p = w.mine + 128 * i;
        const bool inside = p >= lo && p + 4 <= hi;
        cp_async<4>(at + i * 128, p, w.has(i) && inside);
        if (sizeof(T) == 2 && w.has(i) && !inside)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + i * 128), "r"(outer_word(p, Extent{lo, hi})) : "memory");
    }
}

constexpr int WARP_WORDS_BYTES = 544;  // 129 words, and 16 bytes before them for a store

// A warp's 32 vectors in a loose row straight into registers: first the words (so that
// several loads can be under way), then this lane's vector, through the warp's shared
// memory at `base`.
template <typename T>
__device__ __forceinline__ void load_words(uint32_t (&r)[WarpWords<T>::N], const T* src, int valid, bool edge,
                                           const Extent& all) {
    const WarpWords<T> w(src, valid);
    if (sizeof(T) == 4 || !edge) {
        r[0] = ld_global_4_at<0>(w.mine, w.has(0));
        r[1] = ld_global_4_at<128>(w.mine, w.has(1));
        r[2] = ld_global_4_at<256>(w.mine, w.has(2));
        r[3] = ld_global_4_at<384>(w.mine, w.has(3));
        if (sizeof(T) == 2) r[WarpWords<T>::N - 1] = ld_global_4_at<512>(w.mine, w.has(4));
    } else {  // the matrix's first or last row, of which a word may reach out of it
#pragma unroll
        for (int i = 0; i < WarpWords<T>::N; ++i) {
            const char* a = w.mine + 128 * i;
            r[i] = 0;
            if (w.has(i)) r[i] = a >= all.lo && a + 4 <= all.hi ? *reinterpret_cast<const uint32_t*>(a) : outer_word(a, all);
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 settle_words(const uint32_t (&r)[WarpWords<T>::N], const T* src, int valid, uint32_t base) {
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < WarpWords<T>::N; ++i)
        if (i < 4 || lane == 0)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + (lane + 32 * i) * 4), "r"(r[i]) : "memory");
    __syncwarp();
    const uint4 u = vec_of_words<T>(base, valid, sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(src) & 2));
    __syncwarp();
    return u;
}

template <typename T, bool LOOSE>
struct Stage {
    static constexpr bool SHIFT = LOOSE && sizeof(T) == 2;
    // shared memory of one vector of every thread of `threads`
    __host__ __device__ static constexpr int bytes(int threads) {
        return LOOSE ? threads / 32 * WARP_WORDS_BYTES : threads * 16;
    }
    // this thread's (LOOSE: warp's) place in the first vector's memory
    __device__ __forceinline__ static uint32_t mine(uint32_t base) {
        return base + (LOOSE ? threadIdx.x / 32 * WARP_WORDS_BYTES : threadIdx.x * 16);
    }
    // starts the copy of a vector from src, of which and beyond the row holds `valid`
    // elements; `edge`: the row is the matrix's first or last
    __device__ __forceinline__ static void fetch(uint32_t slot, const T* src, int valid, bool edge, const Extent& all) {
        if constexpr (!LOOSE) {
            cp_async<16>(slot, src, valid > 0);
        } else {
            const uint32_t at = slot + (threadIdx.x & 31) * 4;
            if (edge) {
                fetch_edge_words<T>(at, src, valid, all.lo, all.hi);
            } else {
                const WarpWords<T> w(src, valid);
                cp_async_4_at<0>(at, w.mine, w.has(0));
                cp_async_4_at<128>(at, w.mine, w.has(1));
                cp_async_4_at<256>(at, w.mine, w.has(2));
                cp_async_4_at<384>(at, w.mine, w.has(3));
                if (SHIFT) cp_async_4_at<512>(at, w.mine, w.has(4));
            }
        }
    }
    // before the first read of a stage, after the wait for its copies
    __device__ __forceinline__ static void arrived() {
        if constexpr (LOOSE) __syncwarp();
    }
    __device__ __forceinline__ static uint4 read(uint32_t slot, int valid, bool odd) {
        if constexpr (!LOOSE)
            return ld_shared_16(slot);  // places past the row hold zeros (clear)
        else
            return vec_of_words<T>(slot, valid, odd);
    }
    // zeros where nothing is copied, which nothing overwrites
    __device__ __forceinline__ static void clear(uint32_t slot, int valid) {
        if constexpr (!LOOSE)
            if (valid <= 0) st_shared_zero_16(slot);
    }
};

// Stores a vector of a row whose warp holds 32 consecutive vectors, `dst` being
// this lane's and `valid` the elements of the row from there on.  Loose rows go
// through the warp's shared memory (WARP_WORDS_BYTES at `stage`) and are
// written word by word, lane by lane, with single elements at the ends.
template <typename T, bool LOOSE>
__device__ __forceinline__ void store_row_vec(T* dst, const uint4& u, int valid, uint32_t stage) {
    if constexpr (!LOOSE) {
        st_global_16(dst, u, valid > 0);
    } else {
        // the vectors lie 16 bytes into the warp's memory: the word before them may be read
        const int lane = threadIdx.x & 31;
        const uint32_t vecs = stage + 16;
        st_shared_v4(vecs + lane * 16, u.x, u.y, u.z, u.w);
        __syncwarp();
        const WarpWords<T> w(dst, valid);
        char* p = const_cast<char*>(w.mine);
        const uint32_t shift = w.odd ? 16u : 0u, from = vecs + lane * 4, before = from - (w.odd ? 4 : 0);
        const bool leads = w.odd && lane == 0;  // its first word starts with another's element
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x = ld_shared_4(from + 128 * i);
            if (sizeof(T) == 2) x = __funnelshift_r(ld_shared_4(before + 128 * i), x, shift);
            st_global_4(p + 128 * i, x, w.whole(i) && !(i == 0 && leads));
        }
        if (sizeof(T) == 2) {
            // single elements: the first, behind another's, and the last, before another's
            if (leads && w.bytes >= 4) *reinterpret_cast<unsigned short*>(p + 2) = static_cast<unsigned short>(ld_shared_4(from));
            if ((w.bytes & 127) == 2 && w.bytes > 0) {
                const int i = w.bytes >> 7;
                *reinterpret_cast<unsigned short*>(p + 128 * i) = static_cast<unsigned short>(
                    __funnelshift_r(ld_shared_4(before + 128 * i), ld_shared_4(from + 128 * i), shift));
            }
        }
        __syncwarp();
    }
}

// ----------------------------------------------------------------- reductions

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of one or two values over a warp (WARPS = 0) or over a block of at most
// WARPS warps; every thread gets them.  `red` holds 32 floats per value, zero
// beyond the block's warps, that no thread still reads (alternate two of them
// between calls).  Two values halve the shuffles: after the first exchange the
// lower lanes sum one of them and the upper lanes the other.  The warps' sums are
// read back four at a time by every thread, which takes less time than another
// five shuffles.
template <int WARPS>
__device__ __forceinline__ float sum_red(const float* red) {
    uint64_t a = 0;
#pragma unroll
    for (int w = 0; w < WARPS; w += 4) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(red + w);
        a = f2_add(a, f2_add(u.x, u.y));
    }
    return f2_sum(a);
}

template <int WARPS>
__device__ __forceinline__ void group_sum(float& v, float* red) {
    v = warp_sum(v);
    if constexpr (WARPS > 0) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = sum_red<WARPS>(red);
    }
}

template <int WARPS>
__device__ __forceinline__ void group_sum2(float& v0, float& v1, float* red) {
    const int lane = threadIdx.x & 31;
    const bool upper = lane & 16;
    float r = (upper ? v1 : v0) + __shfl_xor_sync(0xffffffffu, upper ? v0 : v1, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if constexpr (WARPS == 0) {
        v0 = __shfl_sync(0xffffffffu, r, 0);
        v1 = __shfl_sync(0xffffffffu, r, 16);
    } else {
        if ((lane & 15) == 0) red[2 * lane + (threadIdx.x >> 5)] = r;
        __syncthreads();
        v0 = sum_red<WARPS>(red);
        v1 = sum_red<WARPS>(red + 32);
    }
}

// ------------------------------------------------------------ 8-bit blocks
//
// A block is 32 consecutive columns of a row.  With a = max |x| over it and
// E = floor(log2 a), its step is 2^max(E - 6, -126) and
//     q = clamp(rint(x / step), -127, 127),   value = q * step.
// The step's biased exponent is the block's scale byte (1..249); |x| / step is
// below 128, so only values that round to 128 are clamped (by at most one
// step).  A block that holds a NaN or an infinity gets the byte 255 and reads
// back as NaN.  Dividing by a power of two is exact, and 7 bits of magnitude
// times a power of two are exact in bf16, so the values are the same however
// they are computed.

constexpr int CK_BLOCK = 32;
constexpr uint32_t CK_NAN = 255;

// 1 / step and step of a scale byte.
__device__ __forceinline__ float ck_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float ck_step(uint32_t byte) {
    return byte == CK_NAN ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// The low bytes of four words in one.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

// Quantises one vector, given as loaded (`raw`) and as pairs: lanes that are
// consecutive hold consecutive vectors, so CK_BLOCK / V of them share a block.
// `w` gets the V bytes; returns the block's scale byte.  Every lane of the warp
// takes part.  Adding 1.5 * 2^23 to x / step rounds to an integer (ties to even)
// that sits in the low mantissa bits as two's complement; the division is exact,
// so the fma rounds once.  Only a block
// whose largest value lies within half a step of 128 steps can round to 128, so
// the clamp runs for those blocks alone (about one in 130 of normal values).
template <typename T>
__device__ __forceinline__ uint32_t ck_quantise_pairs(const uint4& raw, const uint64_t (&v)[Pairs<T>::N],
                                                      uint32_t (&w)[Pairs<T>::N / 2]) {
    constexpr int V = 2 * Pairs<T>::N;
    uint32_t top;
    if constexpr (V == 8) {
        // bf16 magnitudes compare as 16-bit integers, two per instruction
        constexpr uint32_t mag = 0x7fff7fffu;
        const uint32_t m = max_u16x2(max_u16x2(raw.x & mag, raw.y & mag), max_u16x2(raw.z & mag, raw.w & mag));
        top = max(m << 16, m & 0xffff0000u);
    } else {
        top = max(max(raw.x & 0x7fffffffu, raw.y & 0x7fffffffu), max(raw.z & 0x7fffffffu, raw.w & 0x7fffffffu));
    }
#pragma unroll
    for (int o = 1; o < CK_BLOCK / V; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    uint32_t byte = static_cast<uint32_t>(max(1, static_cast<int>(top >> 23) - 6));
    const float magic = 12582912.f;
    const uint64_t inv = f2_splat(ck_inverse(byte)), add = f2_splat(magic);
    float r[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f2_unpack(f2_fma(v[i], inv, add), r[2 * i], r[2 * i + 1]);
    const bool bad = top >= 0x7f800000u;
    if ((top & 0x7f0000u) == 0x7f0000u || bad) {
        if (bad) byte = CK_NAN;
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = bad ? 0.f : fminf(fmaxf(r[i], magic - 127.f), magic + 127.f);
    }
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        w[i] = pack_bytes(__float_as_uint(r[4 * i]), __float_as_uint(r[4 * i + 1]), __float_as_uint(r[4 * i + 2]),
                          __float_as_uint(r[4 * i + 3]));
    return byte;
}

__device__ __forceinline__ void ck_store_words(uint8_t* q, const uint32_t (&w)[2], bool on) { st_global_8(q, w[0], w[1], on); }
__device__ __forceinline__ void ck_store_words(uint8_t* q, const uint32_t (&w)[1], bool on) { st_global_4(q, w[0], on); }

// Values of a vector's bytes as pairs: byte b + 128 placed in the mantissa of
// 2^23 gives 2^23 + 128 + q, from which q comes out exactly.
template <int V>
__device__ __forceinline__ void ck_pairs(const uint32_t* w, float step, uint64_t (&v)[V / 2]) {
    const uint64_t off = f2_splat(-8388736.f), s = f2_splat(step);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const uint32_t u = w[i] ^ 0x80808080u;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            v[2 * i + j] = f2_mul(f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 + 2 * j)),
                                                 __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541 + 2 * j))),
                                         off),
                                  s);
    }
}


}  // namespace flp

// vec.cuh - what the training-step kernels share: typed vector access, warp
// and row reductions, and the 8-bit checkpoint's block arithmetic.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace flp {

using bf16 = __nv_bfloat16;

// Elements per access: 16 bytes where rows are 16-byte aligned and hold a
// whole number of such vectors, else one element.
template <typename T>
__host__ __device__ constexpr int wide_v() { return 16 / static_cast<int>(sizeof(T)); }

// V elements as loaded, and their values in fp32.
template <typename T, int V>
struct Raw;
template <>
struct Raw<bf16, 8> {
    uint4 u;
    __device__ __forceinline__ void load(const bf16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void load_kept(const bf16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint4 bits() const { return u; }
    __device__ __forceinline__ void to(float (&v)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw<float, 4> {
    float4 u;
    __device__ __forceinline__ void load(const float* p) { u = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void load_kept(const float* p) { u = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ uint4 bits() const {
        return make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(u.z), __float_as_uint(u.w));
    }
    __device__ __forceinline__ void to(float (&v)[4]) const {
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    }
};
template <>
struct Raw<bf16, 1> {
    unsigned short u;
    __device__ __forceinline__ void load(const bf16* p) { u = __ldcs(reinterpret_cast<const unsigned short*>(p)); }
    __device__ __forceinline__ void load_kept(const bf16* p) { u = __ldg(reinterpret_cast<const unsigned short*>(p)); }
    __device__ __forceinline__ void zero() { u = 0; }
    __device__ __forceinline__ void to(float (&v)[1]) const { v[0] = __uint_as_float(static_cast<uint32_t>(u) << 16); }
};
template <>
struct Raw<float, 1> {
    float u;
    __device__ __forceinline__ void load(const float* p) { u = __ldcs(p); }
    __device__ __forceinline__ void load_kept(const float* p) { u = __ldg(p); }
    __device__ __forceinline__ void zero() { u = 0.f; }
    __device__ __forceinline__ void to(float (&v)[1]) const { v[0] = u; }
};

// Stores V values at p, rounded once to T (nearest, ties to even).
template <int V>
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    else
        *p = __float2bfloat16_rn(v[0]);
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
    if constexpr (V == 4)
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *p = v[0];
}

// Parameters (norm weight and bias): V values of either type, kept in cache.
template <int V>
__device__ __forceinline__ void load_param(const void* base, bool f32, int col, float (&v)[V]) {
    if (f32) {
        const float* p = static_cast<const float*>(base) + col;
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 u = __ldg(reinterpret_cast<const float4*>(p) + i);
                v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
            }
        } else {
            v[0] = __ldg(p);
        }
    } else {
        const unsigned short* p = static_cast<const unsigned short*>(base) + col;
        uint32_t w[(V + 1) / 2];
        if constexpr (V == 8) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (V == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = u.x, w[1] = u.y;
        } else {
            w[0] = __ldg(p);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    }
}

// ------------------------------------------- vectors on their way through smem
//
// A thread copies ahead the vectors that it will itself read, each into its own
// 16 bytes (or 8) of shared memory, so a completed cp.async group is all the
// synchronisation there is, and the bytes in flight are not limited by registers.

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

// A 16-byte vector as packed fp32 pairs (two lanes per instruction).
template <typename T>
struct Pairs;
template <>
struct Pairs<bf16> {
    static constexpr int N = 4;  // pairs of a vector
    __device__ __forceinline__ static uint64_t get(const uint4& u, int i) {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ static void store(bf16* p, const uint64_t (&v)[4], bool on = true) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(v[i], lo, hi);
            w[i] = pack_bf16x2(lo, hi);
        }
        st_global_16(p, make_uint4(w[0], w[1], w[2], w[3]), on);
    }
};
template <>
struct Pairs<float> {
    static constexpr int N = 2;
    __device__ __forceinline__ static uint64_t get(const uint4& u, int i) {
        return i == 0 ? f2_pack(__uint_as_float(u.x), __uint_as_float(u.y))
                      : f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    __device__ __forceinline__ static void store(float* p, const uint64_t (&v)[2], bool on = true) {
        float4 u;
        f2_unpack(v[0], u.x, u.y);
        f2_unpack(v[1], u.z, u.w);
        st_global_16(p, make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(u.z), __float_as_uint(u.w)), on);
    }
};

__device__ __forceinline__ uint64_t f2_splat(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return lo + hi;
}

// V parameter values from `col` on as pairs (1 or 0 where there are none).
template <int V>
__device__ __forceinline__ void param_pairs(const void* base, bool f32, int col, bool in, float none, uint64_t (&v)[V / 2]) {
    float w[V];
    if (base && in) {
        load_param<V>(base, f32, col, w);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = none;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = f2_pack(w[2 * i], w[2 * i + 1]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N values over the TPR threads of a row (a warp, or the whole block);
// every thread gets them, in the same order.  `red` holds 32 * N floats that
// no thread of the block still reads (alternate two of them between calls).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) red[n * 32 + warp] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.f;
            if constexpr (TPR <= 256) {
#pragma unroll
                for (int w = 0; w < TPR / 32; ++w) s += red[n * 32 + w];
            } else {
                s = warp_sum(lane < TPR / 32 ? red[n * 32 + lane] : 0.f);
            }
            v[n] = s;
        }
    }
}

// Sums of one or two values over a warp (kWarp) or over the whole block of up to
// 16 warps, known at run time; every thread gets them.  `red` holds 16 * N
// floats, zero beyond the block's warps, that no thread still reads (alternate
// two of them between calls).  Two values halve the shuffles: after the first
// exchange the lower lanes sum one of them and the upper lanes the other.  The
// warps' sums are read back four at a time by every thread, which takes less
// time than another five shuffles.
__device__ __forceinline__ float sum_red(const float* red, int warps) {
    uint64_t a = 0;
#pragma unroll 2
    for (int w = 0; w < warps; w += 4) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(red + w);
        a = f2_add(a, f2_add(u.x, u.y));
    }
    return f2_sum(a);
}

template <bool kWarp>
__device__ __forceinline__ void group_sum(float& v, float* red) {
    v = warp_sum(v);
    if constexpr (!kWarp) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = sum_red(red, blockDim.x >> 5);
    }
}

template <bool kWarp>
__device__ __forceinline__ void group_sum2(float& v0, float& v1, float* red) {
    const int lane = threadIdx.x & 31;
    const bool upper = lane & 16;
    float r = (upper ? v1 : v0) + __shfl_xor_sync(0xffffffffu, upper ? v0 : v1, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if constexpr (kWarp) {
        v0 = __shfl_sync(0xffffffffu, r, 0);
        v1 = __shfl_sync(0xffffffffu, r, 16);
    } else {
        if ((lane & 15) == 0) red[lane + (threadIdx.x >> 5)] = r;
        __syncthreads();
        v0 = sum_red(red, blockDim.x >> 5);
        v1 = sum_red(red + 16, blockDim.x >> 5);
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

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale byte of a block from the largest |x| bits in it (NaN > inf > finite).
__device__ __forceinline__ uint32_t ck_byte(uint32_t top) {
    return top >= 0x7f800000u ? CK_NAN : static_cast<uint32_t>(max(1, static_cast<int>(top >> 23) - 6));
}

// 1 / step and step of a scale byte.
__device__ __forceinline__ float ck_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float ck_step(uint32_t byte) {
    return byte == CK_NAN ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// rint(x * inverse) in [-127, 127] as the low byte of the result: adding
// 1.5 * 2^23 rounds to an integer (ties to even) that sits in the low mantissa
// bits as two's complement; the product is exact, so the fma rounds once.
__device__ __forceinline__ uint32_t ck_round(float x, float inverse) {
    const float magic = 12582912.f;
    return __float_as_uint(fminf(fmaxf(__fmaf_rn(x, inverse, magic), magic - 127.f), magic + 127.f));
}

// The low bytes of four words in one.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four values of a q word times the step: byte b + 128 placed in the mantissa
// of 2^23 gives 2^23 + 128 + q, from which q comes out exactly.
__device__ __forceinline__ void ck_values4(uint32_t q, float step, float* v) {
    const uint32_t u = q ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 + i)) - 8388736.f) * step;
}

// Quantises one vector of a row: lanes that are consecutive in `lane` order
// hold consecutive vectors, so CK_BLOCK / V of them share a block.  `w` gets
// the V bytes (one word for V <= 4); returns the block's scale byte.  Every
// lane of the warp takes part.
template <int V>
__device__ __forceinline__ uint32_t ck_quantise(const float (&v)[V], uint32_t (&w)[V > 4 ? 2 : 1]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, abs_bits(v[i]));
#pragma unroll
    for (int o = 1; o < CK_BLOCK / V; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = ck_byte(top);
    const float inv = byte == CK_NAN ? 0.f : ck_inverse(byte);
    uint32_t r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = ck_round(v[i], inv);
    if constexpr (V == 1) {
        w[0] = r[0] & 0xffu;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) w[i] = pack_bytes(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    }
    if (byte == CK_NAN) {
#pragma unroll
        for (int i = 0; i < (V > 4 ? 2 : 1); ++i) w[i] = 0;
    }
    return byte;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

// The same for a 16-byte vector as loaded (`raw`) and as pairs.  Only a block
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

// Values of a vector's bytes as pairs.
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

template <int V>
__device__ __forceinline__ void ck_store(uint8_t* q, const uint32_t (&w)[V > 4 ? 2 : 1]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else if constexpr (V == 4)
        *reinterpret_cast<uint32_t*>(q) = w[0];
    else
        *q = static_cast<uint8_t>(w[0]);
}

// V bytes of a checkpoint row and their block's scale byte.
template <int V>
struct RawCk {
    uint32_t w[V > 4 ? 2 : 1];
    uint32_t byte;
    __device__ __forceinline__ void load(const uint8_t* q, const uint8_t* scale, int col) {
        if constexpr (V == 8) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q + col));
            w[0] = u.x, w[1] = u.y;
        } else if constexpr (V == 4) {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(q + col));
        } else {
            w[0] = __ldcs(q + col);
        }
        byte = __ldcs(scale + col / CK_BLOCK);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (V > 4 ? 2 : 1); ++i) w[i] = 0;
        byte = 1;
    }
    __device__ __forceinline__ void to(float (&v)[V]) const {
        const float step = ck_step(byte);
        if constexpr (V == 1) {
            v[0] = (__uint_as_float(0x4b000000u | (w[0] ^ 0x80u)) - 8388736.f) * step;
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) ck_values4(w[i], step, v + 4 * i);
        }
    }
};

}  // namespace flp

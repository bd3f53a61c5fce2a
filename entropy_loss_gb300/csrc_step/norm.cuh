// norm.cuh - layer norm over the last dimension, forward and backward.
//
//   forward : mean = sum x / H, var = sum (x - mean)^2 / H, rstd = (var + eps)^-1/2,
//             y = (x - mean) rstd w + b
//   backward: xh = (x - mean) rstd, g = dy w,
//             dx = rstd (g - sum(g)/H - xh sum(g xh)/H),
//             dw = sum over rows of dy xh,  db = sum over rows of dy
// Everything is fp32 between one load and one store of each element; the
// variance is taken from the centred values in registers (a second pass there
// costs no memory traffic and cannot cancel as sum x^2 - H mean^2 does).
#pragma once
#include "vec.cuh"

namespace flp {

constexpr int NORM_MAX_H = 16384;

struct NormFwdParams {
    const void* x;
    long long ldx;
    const void* w;  // NULL: 1
    const void* b;  // NULL: 0
    bool param_f32;
    long long M;
    int H;
    float inv_h, eps;
    void* y;
    long long ldy;
    float* mean;  // NULL: not written
    float* rstd;
    uint8_t* q;  // the checkpoint of x (CK): [M, Hp], Hp = H rounded up to 32
    uint8_t* scale;
    int Hp;
    // from a group's row to its next (an even number of rows, if there is a next), in
    // elements: rows, x, y, q, scale
    long long step, step_x, step_y, step_q, step_s;
};

struct NormBwdParams {
    const void* dy;
    long long lddy;
    const void* x;  // the activations, or (CK) NULL
    long long ldx;
    const uint8_t* q;
    const uint8_t* scale;
    int Hp;
    const void* w;  // NULL: 1
    bool param_f32;
    const float* mean;
    const float* rstd;
    long long M;
    int H;
    float inv_h;
    void* dx;
    long long lddx;
    bool sums;     // dw or db is wanted
    float* part;   // [gridDim.x][2][H] fp32 partial sums of dw and db
    bool cluster;  // the blocks are one cluster and join their sums themselves, into
    float* dw;     // these (NULL: not written)
    float* db;
    // from a group's row to its next (an even number of rows, if there is a next), in
    // elements: rows, dy, x, dx, q, scale
    long long step, step_dy, step_x, step_dx, step_q, step_s;
};

// ---------------------------------------------------------------- streaming rows
//
// A group of threads (a warp for short rows, else the block) takes rows group by
// group through the matrix and holds each in registers, NV vectors a thread; S
// rows ahead are on their way through shared memory.  The parameters stay in
// registers from the first row to the last.  Arithmetic runs on packed pairs,
// which halves the instructions that bound these kernels once enough bytes are
// in flight.
//
// The floor is one read and one write of the rows.  What is left above it is issue
// slots (45 to 60 % of them are used) and the two row sums, each a block barrier.
// Forward at 32768 x 4096 bf16: 82 us, 96 % of the measured copy rate; with a
// checkpoint 106 us, 94 %; one row of 4096 6 us (launch, one read, two barriers).

template <typename T, int NV, int S, bool CK, bool LOOSE, bool WARP, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) flp_norm_fwd_stream_kernel(const NormFwdParams p) {
    using X = Stage<T, LOOSE>;
    constexpr int P = Pairs<T>::N, V = 2 * P;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float red[2][32];
    __shared__ __align__(16) uint8_t out_stage[LOOSE ? Stage<T, true>::bytes(MAXT) : 16];
    const int group = WARP ? 32 : blockDim.x;
    const int groups = WARP ? blockDim.x / 32 : 1;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const long long first = static_cast<long long>(blockIdx.x) * groups + (WARP ? threadIdx.x >> 5 : 0);
    const long long step = p.step;
    const uint32_t pitch = X::bytes(blockDim.x);  // from one vector to the next
    const uint32_t slot0 = X::mine(smem_addr(ring)), ring_end = slot0 + S * NV * pitch;
    const int apart = group * V;             // columns between this thread's vectors
    int valid[NV];                           // elements of the row from this thread's vectors on
#pragma unroll
    for (int k = 0; k < NV; ++k) valid[k] = p.H - t * V - k * apart;
    if (!WARP && threadIdx.x < 32) red[0][threadIdx.x] = red[1][threadIdx.x] = 0.f;
    const uint32_t stage = smem_addr(out_stage) + (LOOSE ? threadIdx.x / 32 * WARP_WORDS_BYTES : 0);
    const Extent all = extent_of<T>(p.x, p.M, p.ldx, p.H);

    const T* ahead = static_cast<const T*>(p.x) + first * p.ldx + t * V;  // of the next row to fetch
    int rows_left = first < p.M ? static_cast<int>((p.M - first + step - 1) / step) : 0, to_fetch = rows_left;
    long long fetch_row = first;
    // bf16 rows that start at an odd element (LOOSE): all of this group's, step being even
    const bool odd = X::SHIFT && (reinterpret_cast<uintptr_t>(ahead) & 2);
    auto fetch = [&](uint32_t slot) {
        if (to_fetch > 0) {
            const bool edge = LOOSE && (fetch_row == 0 || fetch_row == p.M - 1);
#pragma unroll
            for (int k = 0; k < NV; ++k) X::fetch(slot + k * pitch, ahead + k * apart, valid[k], edge, all);
        }
        --to_fetch;
        if (LOOSE) fetch_row += step;
        ahead += p.step_x;
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S * NV; ++k) X::clear(slot0 + k * pitch, valid[k % NV]);
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(slot0 + s * NV * pitch);
    uint64_t w[NV][P], b[NV][P];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        param_pairs<V, LOOSE>(p.w, p.param_f32, t * V + k * apart, p.H, 1.f, w[k]);
        param_pairs<V, LOOSE>(p.b, p.param_f32, t * V + k * apart, p.H, 0.f, b[k]);
    }
    T* y = static_cast<T*>(p.y) + first * p.ldy + t * V;
    float* mean_at = p.mean ? p.mean + first : nullptr;
    float* rstd_at = p.rstd ? p.rstd + first : nullptr;
    const unsigned blocks = static_cast<unsigned>(p.Hp) / CK_BLOCK;
    uint8_t* q = CK ? p.q + first * p.Hp + t * V : nullptr;
    uint8_t* scale = CK ? p.scale + first * blocks + static_cast<unsigned>(t * V) / CK_BLOCK : nullptr;
    const bool leads = (t * V) % CK_BLOCK == 0;  // and so for all of this thread's vectors
    uint32_t slot = slot0;
    if constexpr (!WARP) __syncthreads();
    for (; rows_left > 0; --rows_left) {
        cp_async_wait<S - 1>();
        X::arrived();
        uint4 raw[NV];
        uint64_t v[NV][P];
        uint64_t acc = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            raw[k] = X::read(slot + k * pitch, valid[k], odd);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                v[k][i] = Pairs<T>::get(raw[k], i);
                acc = f2_add(acc, v[k][i]);
            }
        }
        float mean = f2_sum(acc);
        group_sum<WARP ? 0 : MAXT / 32>(mean, red[0]);
        // the sum has taken every value of this stage: its slots are free
        fetch(slot);
        slot += NV * pitch;
        if (slot == ring_end) slot = slot0;
        mean *= p.inv_h;
        const uint64_t minus = f2_splat(-mean);
        acc = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (CK) {
                uint32_t w8[P / 2];
                const uint32_t byte = ck_quantise_pairs<T>(raw[k], v[k], w8);
                const bool on = t * V + k * apart < p.Hp;
                ck_store_words(q + k * apart, w8, on);
                st_global_1(scale + static_cast<unsigned>(k * apart) / CK_BLOCK, byte, on && leads);
            }
            // zeros past the row stay zeros
            const uint64_t off = valid[k] > 0 ? minus : 0;
#pragma unroll
            for (int i = 0; i < P; ++i) v[k][i] = f2_add(v[k][i], off);
            if (LOOSE && valid[k] < V) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float lo, hi;
                    f2_unpack(v[k][i], lo, hi);
                    v[k][i] = f2_pack(2 * i < valid[k] ? lo : 0.f, 2 * i + 1 < valid[k] ? hi : 0.f);
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) acc = f2_fma(v[k][i], v[k][i], acc);
        }
        float rstd = f2_sum(acc);
        group_sum<WARP ? 0 : MAXT / 32>(rstd, red[1]);
        rstd = rsqrtf(fmaf(rstd, p.inv_h, p.eps));
        if (t == 0) {
            if (mean_at) *mean_at = mean;
            if (rstd_at) *rstd_at = rstd;
        }
        if (mean_at) mean_at += step;
        if (rstd_at) rstd_at += step;
        const uint64_t r2 = f2_splat(rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            uint64_t o[P];
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = f2_fma(f2_mul(v[k][i], r2), w[k][i], b[k][i]);
            store_row_vec<T, LOOSE>(y + k * apart, Pairs<T>::put(o), valid[k], stage);
        }
        y += p.step_y;
        if constexpr (CK) {
            q += p.step_q;
            scale += p.step_s;
        }
    }
    cp_async_wait<0>();
}

// Whether a thread has more elements of a row than its registers hold sums for.
template <typename T, int NV>
__host__ __device__ constexpr bool norm_bwd_wide() { return NV * wide_v<T>() > 16; }

// Whether the sums of dy wait in shared memory: for such rows, and where a block has 320
// threads, of which two leave 96 registers (bf16, one stage less in flight: 32768 x 5120
// 186 -> 161 us, from a checkpoint 175 -> 166, 20000 x 5001 266 -> 191; fp32 from a
// checkpoint 16384 x 5120 128 -> 120 us; but fp32 16384 x 4608 135 -> 147 us, and loose
// rows from a checkpoint, 20000 x 5001, 212 -> 221).
template <typename T, int NV, int MAXT, bool CK, bool LOOSE>
__host__ __device__ constexpr bool norm_bwd_db_shared() {
    return norm_bwd_wide<T, NV>() || (MAXT == 320 && (sizeof(T) == 2 || (CK && !LOOSE)));
}

// Backward: both sums of a row in one exchange, so one barrier a row; the sums over
// rows stay in registers until the last row, then go to the block's row of `part`.
// 32768 x 4096 bf16 127 us, 94 % of the measured copy rate; from a checkpoint 120 us,
// 83 % (its bytes are turned into pairs, 54 % of the issue slots); 32768 x 5120 161 us,
// 93 %, from a checkpoint 166 us, 75 %.  Above 8192 columns the weights (bf16) and the sums of dy
// wait in shared memory, which leaves room for one row in flight: 8192 x 16384 bf16
// 158 us, 75 % (195 us with the sums in registers, 202 with the weights), from a
// checkpoint 181 us, 55 % (222); fp32 273 us, 87 % (320), although that form and the
// loose ones still spill a few values.
template <typename T, int NV, int S, bool CK, bool LOOSE, bool WARP, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) flp_norm_bwd_stream_kernel(const NormBwdParams p) {
    using X = Stage<T, LOOSE>;
    constexpr int P = Pairs<T>::N, V = 2 * P;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float red[2][64];
    __shared__ __align__(16) uint8_t out_stage[LOOSE ? Stage<T, true>::bytes(MAXT) : 16];
    const int group = WARP ? 32 : blockDim.x;
    const int groups = WARP ? blockDim.x / 32 : 1;
    const int sub = WARP ? threadIdx.x >> 5 : 0;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const long long first = static_cast<long long>(blockIdx.x) * groups + sub;
    const long long step = p.step;
    const uint32_t pitch_y = X::bytes(blockDim.x), pitch_x = CK ? blockDim.x * V : pitch_y;
    const uint32_t ring_x = smem_addr(ring) + S * NV * pitch_y;
    const uint32_t slot0 = X::mine(smem_addr(ring)), ring_end = slot0 + S * NV * pitch_y;
    const uint32_t slot_x0 = CK ? ring_x + threadIdx.x * V : X::mine(ring_x);
    const int apart = group * V;
    int valid[NV];  // elements of the row from this thread's vectors on
#pragma unroll
    for (int k = 0; k < NV; ++k) valid[k] = p.H - t * V - k * apart;
    if (!WARP && threadIdx.x < 64) (&red[0][0])[threadIdx.x] = (&red[1][0])[threadIdx.x] = 0.f;
    const uint32_t stage = smem_addr(out_stage) + (LOOSE ? threadIdx.x / 32 * WARP_WORDS_BYTES : 0);
    const Extent all_y = extent_of<T>(p.dy, p.M, p.lddy, p.H), all_x = extent_of<T>(p.x, p.M, p.ldx, p.H);

    // of the next row to fetch
    const T* ahead_y = static_cast<const T*>(p.dy) + first * p.lddy + t * V;
    const T* ahead_x = CK ? nullptr : static_cast<const T*>(p.x) + first * p.ldx + t * V;
    const uint8_t* ahead_q = CK ? p.q + first * p.Hp + t * V : nullptr;
    int rows_left = first < p.M ? static_cast<int>((p.M - first + step - 1) / step) : 0, to_fetch = rows_left;
    long long fetch_row = first;
    // bf16 rows that start at an odd element (LOOSE): all of this group's, step being even
    const bool odd_y = X::SHIFT && (reinterpret_cast<uintptr_t>(ahead_y) & 2);
    const bool odd_x = X::SHIFT && (reinterpret_cast<uintptr_t>(ahead_x) & 2);
    auto fetch = [&](uint32_t slot, uint32_t slot_x) {
        if (to_fetch > 0) {
            const bool edge = LOOSE && (fetch_row == 0 || fetch_row == p.M - 1);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                X::fetch(slot + k * pitch_y, ahead_y + k * apart, valid[k], edge, all_y);
                if constexpr (CK)
                    cp_async<V>(slot_x + k * pitch_x, ahead_q + k * apart, valid[k] > 0);
                else
                    X::fetch(slot_x + k * pitch_x, ahead_x + k * apart, valid[k], edge, all_x);
            }
        }
        --to_fetch;
        if (LOOSE) fetch_row += step;
        ahead_y += p.step_dy;
        if constexpr (CK)
            ahead_q += p.step_q;
        else
            ahead_x += p.step_x;
        cp_async_commit();
    };
    // what a row needs beside its vectors, AHEAD rows before it in registers: two where
    // rows are short or registers are left for it (a miss takes longer than a row), else
    // one (one instead of two: 32768 x 4096 bf16 139 -> 127 us, 16384 x 8192 162 -> 136,
    // 8192 x 16384 164 -> 158; from a checkpoint 32768 x 5120 171 -> 165, 8192 x 16384
    // 220 -> 181, but 32768 x 4096 120 -> 122 and loose bf16 rows of 12000 x 10001 324 -> 419)
    constexpr bool WIDE = norm_bwd_wide<T, NV>();
    constexpr int AHEAD = (LOOSE ? CK && WIDE && sizeof(T) == 2 : WARP || (CK && MAXT != 320 && !WIDE)) ? 2 : 1;
    struct Few {
        float mean, rstd;
        uint32_t byte[CK ? NV : 1];
    };
    const float* mean_at = p.mean + first;
    const float* rstd_at = p.rstd + first;
    const unsigned blocks = static_cast<unsigned>(p.Hp) / CK_BLOCK;
    const uint8_t* scale = CK ? p.scale + first * blocks + static_cast<unsigned>(t * V) / CK_BLOCK : nullptr;
    auto fetch_few = [&](Few& f, bool there) {
        if (there) {
            f.mean = __ldg(mean_at);
            f.rstd = __ldg(rstd_at);
            if constexpr (CK) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (valid[k] > 0) f.byte[k] = __ldg(scale + static_cast<unsigned>(k * apart) / CK_BLOCK);
            }
        }
        mean_at += step;
        rstd_at += step;
        if constexpr (CK) scale += p.step_s;
    };
    // columns past the row read as zeros: dY's (so that nothing of what is beside
    // the row enters a sum), and x's so that no NaN comes of it (a checkpoint's bytes
    // are multiplied by a step of 0 there, or are its own padding)
#pragma unroll
    for (int k = 0; k < S * NV; ++k) {
        X::clear(slot0 + k * pitch_y, valid[k % NV]);
        if constexpr (!CK) X::clear(slot_x0 + k * pitch_x, valid[k % NV]);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(slot0 + s * NV * pitch_y, slot_x0 + s * NV * pitch_x);
    Few even{}, other{};
    fetch_few(even, rows_left > 0);
    if (AHEAD == 2) fetch_few(other, rows_left > 1);
    // where registers are short the weights wait in shared memory, each thread's own
    // (from a checkpoint 32768 x 4096 bf16 149 -> 120 us, 32768 x 5120 173 -> 165, 16384 x
    // 8192 167 -> 128; 8192 x 16384 without one 202 -> 158; but fp32 16384 x 6144 without one
    // 175 -> 190), and the sums of dy as well (norm_bwd_db_shared)
    constexpr bool DB_SHARED = norm_bwd_db_shared<T, NV, MAXT, CK, LOOSE>();
    constexpr bool W_SHARED = !WARP && (CK || MAXT == 320 || (WIDE && sizeof(T) == 2));
    __shared__ ulonglong2 w_shared[W_SHARED ? NV * P / 2 : 1][W_SHARED ? MAXT : 1];
    __shared__ ulonglong2 db_shared[DB_SHARED ? NV * P / 2 : 1][DB_SHARED ? MAXT : 1];
    uint64_t w_kept[W_SHARED ? 1 : NV][P], dw[NV][P] = {}, db[DB_SHARED ? 1 : NV][P] = {};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        uint64_t w[P];
        param_pairs<V, LOOSE>(p.w, p.param_f32, t * V + k * apart, p.H, 1.f, w);
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            if constexpr (W_SHARED)
                w_shared[(k * P + i) / 2][threadIdx.x] = make_ulonglong2(w[i], w[i + 1]);
            else
                w_kept[k][i] = w[i], w_kept[k][i + 1] = w[i + 1];
            if constexpr (DB_SHARED) db_shared[(k * P + i) / 2][threadIdx.x] = make_ulonglong2(0, 0);
        }
    }
    auto weight = [&](int k, uint64_t (&w)[P]) {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            if constexpr (W_SHARED) {
                const ulonglong2 u = w_shared[(k * P + i) / 2][threadIdx.x];
                w[i] = u.x, w[i + 1] = u.y;
            } else {
                w[i] = w_kept[k][i], w[i + 1] = w_kept[k][i + 1];
            }
        }
    };
    T* dx = static_cast<T*>(p.dx) + first * p.lddx + t * V;
    uint32_t slot = slot0, slot_x = slot_x0;
    int buf = 0;
    if constexpr (!WARP) __syncthreads();
    auto one_row = [&](Few& few) {
        cp_async_wait<S - 1>();
        X::arrived();
        uint4 ry[NV];
        uint64_t xh[NV][P];
        uint64_t s0 = 0, s1 = 0;
        const uint64_t minus = f2_splat(-few.mean), r2 = f2_splat(few.rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            ry[k] = X::read(slot + k * pitch_y, valid[k], odd_y);
            if constexpr (CK) {
                uint32_t q[V / 4];
                if constexpr (V == 8) {
                    const uint2 u = ld_shared_8(slot_x + k * pitch_x);
                    q[0] = u.x, q[1] = u.y;
                } else {
                    q[0] = ld_shared_4(slot_x + k * pitch_x);
                }
                ck_pairs<V>(q, ck_step(few.byte[k]), xh[k]);
            } else {
                const uint4 rx = X::read(slot_x + k * pitch_x, valid[k], odd_x);
#pragma unroll
                for (int i = 0; i < P; ++i) xh[k][i] = Pairs<T>::get(rx, i);
            }
            uint64_t w[P];
            weight(k, w);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const uint64_t d = Pairs<T>::get(ry[k], i);
                xh[k][i] = f2_mul(f2_add(xh[k][i], minus), r2);
                dw[k][i] = f2_fma(d, xh[k][i], dw[k][i]);
                if constexpr (!DB_SHARED) db[k][i] = f2_add(db[k][i], d);
                const uint64_t g = f2_mul(d, w[i]);
                s0 = f2_add(s0, g);
                s1 = f2_fma(g, xh[k][i], s1);
            }
            if constexpr (DB_SHARED) {
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    ulonglong2& u = db_shared[(k * P + i) / 2][threadIdx.x];
                    u = make_ulonglong2(f2_add(u.x, Pairs<T>::get(ry[k], i)), f2_add(u.y, Pairs<T>::get(ry[k], i + 1)));
                }
            }
        }
        // before the row's exchange, or behind it in one block of 512 threads of aligned bf16
        // rows (16384 x 8192 140 -> 136 us, 8192 x 6144 65 -> 63; but 32768 x 4096 127 -> 162,
        // loose 16000 x 8001 254 -> 262)
        constexpr bool LATE = sizeof(T) == 2 && !CK && !LOOSE && MAXT == 512 && !WIDE;
        if constexpr (!LATE) fetch_few(few, rows_left > AHEAD);
        float m1 = f2_sum(s0), m2 = f2_sum(s1);
        group_sum2<WARP ? 0 : MAXT / 32>(m1, m2, red[buf]);
        buf ^= 1;
        if constexpr (LATE) fetch_few(few, rows_left > AHEAD);
        // the sums have taken every value of this stage: its slots are free
        fetch(slot, slot_x);
        slot += NV * pitch_y;
        slot_x += NV * pitch_x;
        if (slot == ring_end) slot = slot0, slot_x = slot_x0;
        const uint64_t n1 = f2_splat(-m1 * p.inv_h), n2 = f2_splat(-m2 * p.inv_h);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            uint64_t o[P], w[P];
            weight(k, w);
#pragma unroll
            for (int i = 0; i < P; ++i)
                o[i] = f2_mul(r2, f2_fma(xh[k][i], n2, f2_fma(Pairs<T>::get(ry[k], i), w[i], n1)));
            store_row_vec<T, LOOSE>(dx + k * apart, Pairs<T>::put(o), valid[k], stage);
        }
        dx += p.step_dx;
        --rows_left;
    };
    while (rows_left > 0) {
        one_row(even);
        if constexpr (AHEAD == 2) {
            if (rows_left > 0) one_row(other);
        }
    }
    cp_async_wait<0>();
    griddep_launch_dependents();
    if (!p.sums) return;
    // this block's sums; with a row per warp, the warps join first (the ring is free)
    float* join = reinterpret_cast<float*>(ring);
    float* sums = join + (WARP ? (MAXT / 32) * (NV * 32 * V) : 0);  // [2][H] of a cluster's block
    if (p.cluster) __syncthreads();  // every warp is done with the ring
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* out = p.cluster ? sums + which * p.H : p.part + (static_cast<long long>(blockIdx.x) * 2 + which) * p.H;
        if constexpr (WARP) __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = t * V + k * apart;
            float* at = WARP ? join + sub * (NV * 32 * V) + col : out + col;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                uint64_t of_dy;
                if constexpr (DB_SHARED) {
                    const ulonglong2 u = db_shared[(k * P + i) / 2][threadIdx.x];
                    of_dy = i % 2 ? u.y : u.x;
                } else {
                    of_dy = db[k][i];
                }
                float2 a;
                f2_unpack(which ? of_dy : dw[k][i], a.x, a.y);
                if (!LOOSE || WARP) {
                    if (WARP || valid[k] > 0) *reinterpret_cast<float2*>(at + 2 * i) = a;
                } else {
                    if (2 * i < valid[k]) at[2 * i] = a.x;
                    if (2 * i + 1 < valid[k]) at[2 * i + 1] = a.y;
                }
            }
        }
        if constexpr (WARP) {
            __syncthreads();
            for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
                float a = 0.f;
                for (int u = 0; u < groups; ++u) a += join[u * (NV * 32 * V) + c];
                out[c] = a;
            }
        }
    }
    if (p.cluster) {
        cluster_sync();
        const unsigned blocks_in = gridDim.x;
        for (unsigned c = blockIdx.x * blockDim.x + threadIdx.x; c < 2u * p.H; c += blocks_in * blockDim.x) {
            float a = 0.f;
            for (unsigned r = 0; r < blocks_in; ++r) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_addr(sums + c), r)) : "memory");
                a += v;
            }
            float* to = c < static_cast<unsigned>(p.H) ? p.dw : p.db;
            if (to) to[c < static_cast<unsigned>(p.H) ? c : c - p.H] = a;
        }
        cluster_sync();  // no block leaves while its sums are read
    }
}

struct NormJoinParams {
    const float* part;  // [P][2][H]
    int P, H;
    float* dw;  // NULL: not written
    float* db;
};

// dw and db from the blocks' partial sums: 32 columns per block, 32 threads
// down the partials of each column, joined in a fixed order.  304 partials of
// 4096 columns come from L2 in 7 us, most of it launch and one round of loads.
__global__ void __launch_bounds__(1024) flp_norm_join_kernel(const NormJoinParams p) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, down = threadIdx.x >> 5;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;  // column of [dw | db]
    const long long width = 2ll * p.H;
    griddep_wait();
    float a = 0.f;
    if (c < width)
        for (int r = down; r < p.P; r += 32) a += p.part[r * width + c];
    part[down][lane] = a;
    __syncthreads();
    // warp `down` sums column `down` of this block
    const float s = warp_sum(part[lane][down]);
    const long long col = static_cast<long long>(blockIdx.x) * 32 + down;
    if (lane == 0 && col < width) {
        float* out = col < p.H ? p.dw : p.db;
        if (out) out[col < p.H ? col : col - p.H] = s;
    }
}

}  // namespace flp

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
};

template <int TPR>
__host__ __device__ constexpr int norm_rows_per_block() { return TPR >= 128 ? 1 : 128 / TPR; }

// One row per TPR threads, held in registers (NV vectors of V elements each).
template <typename T, int V, int TPR, int NV, bool CK>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) flp_norm_fwd_kernel(const NormFwdParams p) {
    constexpr int RPB = norm_rows_per_block<TPR>();
    __shared__ float red[2][32];
    const long long row = static_cast<long long>(blockIdx.x) * RPB + (RPB > 1 ? threadIdx.x / TPR : 0);
    const int t = RPB > 1 ? threadIdx.x % TPR : threadIdx.x;
    if (row >= p.M) return;  // a whole warp
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float v[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = (t + k * TPR) * V;
        Raw<T, V> r;
        if (col < p.H)
            r.load(x + col);
        else
            r.zero();
        r.to(v[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += v[k][i];
    }
    row_sum<TPR>(s, red[0]);
    const float mean = s[0] * p.inv_h;
    float c[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if ((t + k * TPR) * V < p.H) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[k][i] - mean;
                c[0] = fmaf(d, d, c[0]);
            }
        }
    }
    row_sum<TPR>(c, red[1]);
    const float rstd = rsqrtf(fmaf(c[0], p.inv_h, p.eps));
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = (t + k * TPR) * V;
        if constexpr (CK) {
            uint32_t w[V > 4 ? 2 : 1];
            const uint32_t byte = ck_quantise<V>(v[k], w);
            if (col < p.Hp) {
                ck_store<V>(p.q + row * p.Hp + col, w);
                if ((col % CK_BLOCK) == 0) p.scale[row * (p.Hp / CK_BLOCK) + col / CK_BLOCK] = static_cast<uint8_t>(byte);
            }
        }
        if (col < p.H) {
            float w[V], b[V], o[V];
            if (p.w)
                load_param<V>(p.w, p.param_f32, col, w);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] = 1.f;
            if (p.b)
                load_param<V>(p.b, p.param_f32, col, b);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) b[i] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf((v[k][i] - mean) * rstd, w[i], b[i]);
            store_vec<V>(y + col, o);
        }
    }
}

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
    float* part;  // [gridDim.x][2][H] fp32 partial sums of dw and db
};

// Each block takes rows blockIdx.x, blockIdx.x + gridDim.x, ... (times the rows
// a block holds) and keeps its columns' share of dw and db in registers; the
// next row's vectors are loaded before the current row's sums are known.
template <typename T, int V, int TPR, int NV, bool CK>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) flp_norm_bwd_kernel(const NormBwdParams p) {
    constexpr int RPB = norm_rows_per_block<TPR>();
    __shared__ float red[2][2][32];
    __shared__ float join[RPB > 1 ? RPB * TPR * NV * V : 1];
    const int sub = RPB > 1 ? threadIdx.x / TPR : 0;
    const int t = RPB > 1 ? threadIdx.x % TPR : threadIdx.x;
    const long long step = static_cast<long long>(gridDim.x) * RPB;
    float dw[NV][V] = {}, db[NV][V] = {};
    Raw<T, V> rdy[NV], rx[NV];
    RawCk<V> rq[NV];
    float mean = 0.f, rstd = 0.f;

    auto fetch = [&](long long row) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (t + k * TPR) * V;
            if (row < p.M && col < p.H) {
                rdy[k].load(static_cast<const T*>(p.dy) + row * p.lddy + col);
                if constexpr (CK)
                    rq[k].load(p.q + row * p.Hp, p.scale + row * (p.Hp / CK_BLOCK), col);
                else
                    rx[k].load(static_cast<const T*>(p.x) + row * p.ldx + col);
            } else {
                rdy[k].zero();
                if constexpr (CK)
                    rq[k].zero();
                else
                    rx[k].zero();
            }
        }
        if (row < p.M) {
            mean = __ldg(p.mean + row);
            rstd = __ldg(p.rstd + row);
        }
    };

    long long row = static_cast<long long>(blockIdx.x) * RPB + sub;
    fetch(row);
    int buf = 0;
    for (; row < p.M; row += step) {
        float g[NV][V], xh[NV][V];
        const float r = rstd;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (t + k * TPR) * V;
            float d[V], w[V];
            rdy[k].to(d);
            if constexpr (CK)
                rq[k].to(xh[k]);
            else
                rx[k].to(xh[k]);
            if (p.w && col < p.H)
                load_param<V>(p.w, p.param_f32, col, w);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] = 1.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[k][i] = (xh[k][i] - mean) * r;
                dw[k][i] = fmaf(d[i], xh[k][i], dw[k][i]);
                db[k][i] += d[i];
                g[k][i] = d[i] * w[i];
                s[0] += g[k][i];
                s[1] = fmaf(g[k][i], xh[k][i], s[1]);
            }
        }
        fetch(row + step);
        row_sum<TPR>(s, &red[buf][0][0]);
        buf ^= 1;
        const float m1 = s[0] * p.inv_h, m2 = s[1] * p.inv_h;
        T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (t + k * TPR) * V;
            if (col < p.H) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = r * (g[k][i] - fmaf(xh[k][i], m2, m1));
                store_vec<V>(dx + col, o);
            }
        }
    }
    griddep_launch_dependents();
    // this block's sums; with several rows per block, the row groups join first
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* out = p.part + (static_cast<long long>(blockIdx.x) * 2 + which) * p.H;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (t + k * TPR) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float a = which ? db[k][i] : dw[k][i];
                if constexpr (RPB > 1)
                    join[sub * (TPR * NV * V) + col + i] = a;
                else if (col + i < p.H)
                    out[col + i] = a;
            }
        }
        if constexpr (RPB > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < p.H; c += RPB * TPR) {
                float a = 0.f;
#pragma unroll
                for (int u = 0; u < RPB; ++u) a += join[u * (TPR * NV * V) + c];
                out[c] = a;
            }
            __syncthreads();
        }
    }
}

struct NormJoinParams {
    const float* part;  // [P][2][H]
    int P, H;
    float* dw;  // NULL: not written
    float* db;
};

// dw and db from the blocks' partial sums: 32 columns per block, 32 threads
// down the partials of each column, joined in a fixed order.
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

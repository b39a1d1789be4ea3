// The norms on both sides of a block, fused with its gate and residual scale.
//
//   p = y rstd(y) g_post            (post-norm; p = y without one)
//   r' = alpha r + beta s p         (s = sigmoid(z) per token or per element, or 1)
//   x' = r' rstd(r') g_pre          (the next block's pre-norm)
//   rstd(v) = 1 / sqrt(mean(v^2) + eps)
//
// and its gradient, with D the gradient of r' (what arrives for r' itself plus
// what comes back through the pre-norm):
//   D = dr' + rstd(r') (t - xh mean(t xh)),  t = dx' g_pre, xh = r' rstd(r')
//   dr = alpha D,  dp = beta s D,  dz = beta p D s (1 - s) (summed over a token's row)
//   dy = rstd(y) (q - yh mean(q yh)),        q = dp g_post, yh = y rstd(y)
//   dg_post = sum_t dp yh,  dg_pre = sum_t dx' xh
//
// Both are one pass over the rows, bound by HBM: a workgroup takes a row at a
// time, holds it in registers (CH chunks of 8 elements per thread) through
// both reductions and writes it once; r' enters the pre-norm before it is
// rounded.  The backward recomputes r' from y, r and z rather than reading
// it, from the same bytes.  All arithmetic is fp32; every output is rounded
// once.  The next row's loads are issued before this row's reductions.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxChunks = 4;

struct NormArgs {
    const uint16_t *y;
    const void *r, *z;
    const float *g_post, *g_pre;
    void *r_out;
    uint16_t *xn;
    float *stats;  // [rows][2]: rstd(y), rstd(r'); 0 where that norm is absent
    int64_t rows;
    int H, gate;
    float alpha, beta, eps;
};

struct NormBwdArgs {
    NormArgs f;  // r_out, xn unused; stats read
    const void *dr_out;
    const uint16_t *dxn;
    uint16_t *dy;
    void *dr, *dz;
    float *part;  // [workgroups][2][H]: each workgroup's sums of dg_post and dg_pre
};

// Eight elements as they lie in memory.
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
    u32x4 v;
    __device__ __forceinline__ void load(const void *p, int64_t chunk) { v = __builtin_nontemporal_load(static_cast<const u32x4 *>(p) + chunk); }
    __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ float operator[](int i) const {
        return __uint_as_float((i & 1) ? (v[i >> 1] & 0xffff0000u) : (v[i >> 1] << 16));
    }
};
template <>
struct Raw8<true> {
    f32x4 v[2];
    __device__ __forceinline__ void load(const void *p, int64_t chunk) {
        v[0] = __builtin_nontemporal_load(static_cast<const f32x4 *>(p) + 2 * chunk);
        v[1] = __builtin_nontemporal_load(static_cast<const f32x4 *>(p) + 2 * chunk + 1);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ float operator[](int i) const { return v[i >> 2][i & 3]; }
};

__device__ __forceinline__ void store8(uint16_t *p, int64_t chunk, const float (&v)[8]) {
    reinterpret_cast<u32x4 *>(p)[chunk] =
        u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
}
__device__ __forceinline__ void store8(float *p, int64_t chunk, const float (&v)[8]) {
    f32x4 *o = reinterpret_cast<f32x4 *>(p) + 2 * chunk;
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
}
template <bool F32>
__device__ __forceinline__ void store_res(void *p, int64_t chunk, const float (&v)[8]) {
    if constexpr (F32)
        store8(static_cast<float *>(p), chunk, v);
    else
        store8(static_cast<uint16_t *>(p), chunk, v);
}

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// Sums of N values over the workgroup, in a fixed order, on every thread.  Two
// LDS buffers in turn: a buffer is written again only after the barrier of the
// sum in between, which every reader of it has passed.
template <int N>
struct RowSum {
    float *lds;  // [2][N][16]
    int turn = 0;
    __device__ __forceinline__ explicit RowSum(float *p) : lds(p) {}
    __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int o = kWave / 2; o >= 1; o >>= 1) v[n] += __shfl_xor(v[n], o, kWave);
        const int waves = blockDim.x / kWave;
        if (waves == 1) return;
        float *b = lds + turn * N * 16;
        turn ^= 1;
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) b[n * 16 + threadIdx.x / kWave] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.f;
            for (int w = 0; w < waves; ++w) s += b[n * 16 + w];
            v[n] = s;
        }
    }
};

template <bool F32, int CH>
__device__ __forceinline__ void norm_fwd_body(const NormArgs &a, float *lds) {
    const int t = threadIdx.x, nt = blockDim.x, chunks = a.H / 8;
    const bool post = a.g_post, pre = a.g_pre, elem = a.gate == MOE_GATE_ELEM, token = a.gate == MOE_GATE_TOKEN;
    const float inv_h = 1.0f / (float)a.H;
    RowSum<1> sum(lds);
    Raw8<false> y[CH], z[CH];
    Raw8<F32> r[CH];
    float zt = 0.f;
    auto fetch = [&](int64_t row) {
        const int64_t base = row * chunks;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            if (c < chunks) {
                r[i].load(a.r, base + c);
                if (a.y) y[i].load(a.y, base + c);
                if (elem) z[i].load(a.z, base + c);
            }
        }
        if (token) zt = static_cast<const float *>(a.z)[row];
    };
#pragma unroll
    for (int i = 0; i < CH; ++i) y[i].zero(), z[i].zero(), r[i].zero();
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * chunks;
        float v[CH][8], p[CH][8], s[1] = {0.f};
        float scale = a.beta;
        if (token) scale *= sigmoid(zt);
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float yv = y[i][e];
                s[0] = fmaf(yv, yv, s[0]);
                p[i][e] = elem ? scale * sigmoid(z[i][e]) * yv : scale * yv;
                v[i][e] = a.y ? a.alpha * r[i][e] : r[i][e];
            }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        float ystd = 0.f;
        if (post) {
            sum(s);
            ystd = __builtin_amdgcn_rsqf(fmaf(s[0], inv_h, a.eps));
        }
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            if (c >= chunks) continue;
            if (post) {
                Raw8<true> g;
                g.load(a.g_post, c);
#pragma unroll
                for (int e = 0; e < 8; ++e) p[i][e] *= ystd * g[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (a.y) v[i][e] += p[i][e];
                s[0] = fmaf(v[i][e], v[i][e], s[0]);
            }
            if (a.r_out) store_res<F32>(a.r_out, base + c, v[i]);
        }
        float rstd = 0.f;
        if (pre) {
            sum(s);
            rstd = __builtin_amdgcn_rsqf(fmaf(s[0], inv_h, a.eps));
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * nt + t;
                if (c >= chunks) continue;
                Raw8<true> g;
                g.load(a.g_pre, c);
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[i][e] * rstd * g[e];
                store8(a.xn, base + c, x);
            }
        }
        if (t == 0) reinterpret_cast<float2 *>(a.stats)[row] = make_float2(ystd, rstd);
    }
}

template <bool F32, int CH>
__device__ __forceinline__ void norm_bwd_body(const NormBwdArgs &b, float *lds) {
    const NormArgs &a = b.f;
    const int t = threadIdx.x, nt = blockDim.x, chunks = a.H / 8;
    const bool post = a.g_post, pre = a.g_pre, elem = a.gate == MOE_GATE_ELEM, token = a.gate == MOE_GATE_TOKEN;
    const float inv_h = 1.0f / (float)a.H;
    RowSum<2> sum(lds);
    Raw8<false> y[CH], z[CH], dx[CH];
    Raw8<F32> r[CH], up[CH];
    float2 st = make_float2(0.f, 0.f);
    float zt = 0.f;
    auto fetch = [&](int64_t row) {
        const int64_t base = row * chunks;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            if (c < chunks) {
                r[i].load(a.r, base + c);
                if (a.y) y[i].load(a.y, base + c);
                if (elem) z[i].load(a.z, base + c);
                if (b.dr_out) up[i].load(b.dr_out, base + c);
                if (pre) dx[i].load(b.dxn, base + c);
            }
        }
        st = reinterpret_cast<const float2 *>(a.stats)[row];
        if (token) zt = static_cast<const float *>(a.z)[row];
    };
    float acc_post[CH][8], acc_pre[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        y[i].zero(), z[i].zero(), dx[i].zero(), r[i].zero(), up[i].zero();
#pragma unroll
        for (int e = 0; e < 8; ++e) acc_post[i][e] = acc_pre[i][e] = 0.f;
    }
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * chunks;
        const float ystd = post ? st.x : 1.0f, rstd = st.y;
        const float gt = token ? sigmoid(zt) : 1.0f;
        // yh, the gate, D (first what arrives for r'), t and xh of the row
        float yh[CH][8], gv[CH][8], D[CH][8], tv[CH][8], xh[CH][8], s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            if (c >= chunks) continue;
            Raw8<true> go, gi;
            if (post) go.load(a.g_post, c);
            if (pre) gi.load(a.g_pre, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                yh[i][e] = y[i][e] * ystd;
                gv[i][e] = elem ? sigmoid(z[i][e]) : gt;
                D[i][e] = up[i][e];
                const float p = post ? yh[i][e] * go[e] : yh[i][e];
                const float rn = a.y ? fmaf(a.beta * gv[i][e], p, a.alpha * r[i][e]) : r[i][e];
                xh[i][e] = rn * rstd;
                const float d = dx[i][e];
                tv[i][e] = pre ? d * gi[e] : 0.f;
                acc_pre[i][e] = fmaf(d, xh[i][e], acc_pre[i][e]);
                s[0] = fmaf(tv[i][e], xh[i][e], s[0]);
            }
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        if (pre) {
            sum(s);
            const float c1 = s[0] * inv_h;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) D[i][e] = fmaf(rstd, fmaf(-xh[i][e], c1, tv[i][e]), D[i][e]);
        }
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            if (c >= chunks) continue;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = a.y ? a.alpha * D[i][e] : D[i][e];
            store_res<F32>(b.dr, base + c, o);
            if (!a.y) continue;
            Raw8<true> go;
            if (post) go.load(a.g_post, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = a.beta * D[i][e];
                const float p = post ? yh[i][e] * go[e] : yh[i][e];
                o[e] = d * p * gv[i][e] * (1.0f - gv[i][e]);
                s[1] = fmaf(d, p, s[1]);
                const float dp = d * gv[i][e];
                acc_post[i][e] = fmaf(dp, yh[i][e], acc_post[i][e]);
                D[i][e] = post ? dp * go[e] : dp;  // q
                s[0] = fmaf(D[i][e], yh[i][e], s[0]);
            }
            if (elem) store8(static_cast<uint16_t *>(b.dz), base + c, o);
        }
        if (post || token) sum(s);
        if (a.y) {
            const float c2 = post ? s[0] * inv_h : 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * nt + t;
                if (c >= chunks) continue;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = ystd * fmaf(-yh[i][e], c2, D[i][e]);
                store8(b.dy, base + c, o);
            }
        }
        if (token && t == 0) static_cast<float *>(b.dz)[row] = s[1] * gt * (1.0f - gt);
    }
    if (post || pre) {
        float *o = b.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            if (c >= chunks) continue;
            if (post) store8(o, c, acc_post[i]);
            if (pre) store8(o + a.H, c, acc_pre[i]);
        }
    }
}

// dg[c] = the sum over the backward's workgroups of their partial sums:
// 64 columns x 16 groups of workgroups, each group in ascending order, then
// the groups in a fixed tree.
__device__ __forceinline__ void norm_dg_body(const float *part, int groups, int H, float *dg_post, float *dg_pre, float *lds) {
    const int col = blockIdx.x * 64 + threadIdx.x % 64, g0 = threadIdx.x / 64;
    float *out = blockIdx.y ? dg_pre : dg_post;
    if (!out) return;  // the whole workgroup
    float s = 0.f;
    if (col < H)
        for (int g = g0; g < groups; g += 16) s += part[((int64_t)g * 2 + blockIdx.y) * H + col];
    lds[threadIdx.x] = s;
    __syncthreads();
    for (int o = 8; o >= 1; o >>= 1) {
        if (g0 < o) lds[threadIdx.x] += lds[threadIdx.x + o * 64];
        __syncthreads();
    }
    if (g0 == 0 && col < H) out[col] = lds[threadIdx.x];
}

}  // namespace moe

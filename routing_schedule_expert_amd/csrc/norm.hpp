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
// time, one thread per 8 elements (two or four such chunks past H = 8192), holds it
// in registers through both reductions and writes it once; r' enters the pre-norm
// before it is rounded.  The backward recomputes r' from y, r and z rather than
// reading it, from the same bytes.  All arithmetic is fp32; every output is
// rounded once.
//   - The next row's loads are issued before this row's reductions.  Loads return
//     in order, so nothing else may be loaded from memory in the loop: g_post and
//     g_pre lie in LDS.  (Both only while the registers last: up to H = 8192, the
//     forward's loads ahead up to 16384; the backward reads a longer row twice.)
//   - Rows are raw buffers: absent tensors are empty buffers and the last chunk's
//     spare lanes read zeros, so the loop has no branch around a memory access and
//     the compiler waits for exactly the loads it needs.
// Measured: 57,344 rows of 7,168 with a gate per element, forward 0.79 ms (5.2
// TB/s; 1.15 ms with the gains read from L2 in the loop); 16,384 rows, backward 0.36
// to 0.38 ms and 5 us for the column sums (5.0 to 5.1 TB/s); a copy of 4 GiB gets 4.9 to
// 5.4 TB/s.
#pragma once

#include "buffer.hpp"
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

// A row of a tensor: element size ES bytes, empty where the tensor is absent
// (or not `in` use).
template <int ES>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void *p, int64_t row, int H, bool in = true) {
    in = in && p;
    return raw_buffer(static_cast<const char *>(p) + (in ? row * H * ES : 0), in ? (uint32_t)(H * ES) : 0u);
}

// The word of a row (0 where the tensor is absent).
__device__ __forceinline__ float row_word(const void *p, int64_t i, bool in) {
    in = in && p;
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(raw_buffer(static_cast<const float *>(p) + (in ? i : 0), in ? 4u : 0u), 0, 0, 0));
}

// Eight elements (a chunk) as they lie in memory.  KEEP: they are read again.
template <bool KEEP>
__device__ __forceinline__ u32x4 load_chunk(__amdgpu_buffer_rsrc_t b, int off) {
    return KEEP ? buffer_load16(b, off) : buffer_load16_nt(b, off);
}
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
    u32x4 v;
    template <bool KEEP = false>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int chunk) {
        v = load_chunk<KEEP>(b, chunk * 16);
    }
    __device__ __forceinline__ float operator[](int i) const {
        return __uint_as_float((i & 1) ? (v[i >> 1] & 0xffff0000u) : (v[i >> 1] << 16));
    }
};
template <>
struct Raw8<true> {
    u32x4 v[2];
    template <bool KEEP = false>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int chunk) {
        v[0] = load_chunk<KEEP>(b, chunk * 32);
        v[1] = load_chunk<KEEP>(b, chunk * 32 + 16);
    }
    __device__ __forceinline__ float operator[](int i) const { return __uint_as_float(v[i >> 2][i & 3]); }
};

template <bool F32>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t b, int chunk, const float (&v)[8]) {
    if constexpr (F32) {
        buffer_store16(b, chunk * 32, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
        buffer_store16(b, chunk * 32 + 16, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
    } else {
        buffer_store16(b, chunk * 16, u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])});
    }
}

// g_post and g_pre in LDS (1 where absent) up to H = 8192; read from L2 above.
constexpr int kNormLdsH = 8192;
struct NormGains {
    const float *post, *pre;  // of global memory
    float *lds;               // [2][H] or null
    int H;
    // every thread its own chunk, which no other reads
    __device__ __forceinline__ void fill() const {
        const int c = threadIdx.x;
        if (!lds || c * 8 >= H) return;
        const f32x4 one = f32x4{1.f, 1.f, 1.f, 1.f};
        f32x4 *o = reinterpret_cast<f32x4 *>(lds) + 2 * c, *p = reinterpret_cast<f32x4 *>(lds + H) + 2 * c;
        const f32x4 *a = reinterpret_cast<const f32x4 *>(post) + 2 * c, *b = reinterpret_cast<const f32x4 *>(pre) + 2 * c;
        const f32x4 v[4] = {post ? a[0] : one, post ? a[1] : one, pre ? b[0] : one, pre ? b[1] : one};
        o[0] = v[0], o[1] = v[1], p[0] = v[2], p[1] = v[3];
    }
    // no branch around the loads from memory: what is absent comes from an empty buffer
    template <bool LDS>
    __device__ __forceinline__ void load(int which, int chunk, float (&g)[8]) const {
        f32x4 a, b;
        if constexpr (LDS) {
            const f32x4 *s = reinterpret_cast<const f32x4 *>(lds + which * H) + 2 * chunk;
            a = b = f32x4{1.f, 1.f, 1.f, 1.f};
            if (chunk * 8 < H) a = s[0], b = s[1];
        } else {
            const float *p = which ? pre : post;
            const __amdgpu_buffer_rsrc_t s = raw_buffer(p, p ? (uint32_t)H * 4 : 0);
            a = __builtin_bit_cast(f32x4, buffer_load16(s, chunk * 32));
            b = __builtin_bit_cast(f32x4, buffer_load16(s, chunk * 32 + 16));
            if (!p) a = b = f32x4{1.f, 1.f, 1.f, 1.f};
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = a[e], g[4 + e] = b[e];
    }
};

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
// s = sigmoid(z) and 1 - s, which the gate's gradient needs, in one register: the smaller
// of the two, its sign bit set where that is 1 - s.  The difference 1 - s itself would lose
// its bits as the gate opens (at z = 11 all but 8, from z = 17 on s is 1); exp(-z) s does not.
struct Gate {
    float k;
    __device__ __forceinline__ Gate() {}
    __device__ __forceinline__ Gate(float e, float s) : k(e < 1.0f ? -(e * s) : s) {}  // e = exp(-z)
    __device__ __forceinline__ bool rest_held() const { return (int)__float_as_uint(k) < 0; }
    __device__ __forceinline__ float open() const { return rest_held() ? 1.0f + k : k; }
    __device__ __forceinline__ float rest() const { return rest_held() ? -k : 1.0f - k; }
};

// The sum over a wave, on every lane: within rows of 16 lanes by rotations, then
// across the four rows.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x128>(v);  // row_ror:8
    v = dpp_add<0x124>(v);
    v = dpp_add<0x122>(v);
    v = dpp_add<0x121>(v);
    v += __shfl_xor(v, 16, kWave);
    v += __shfl_xor(v, 32, kWave);
    return v;
}

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
        for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
        float *b = lds + turn * N * 16;
        turn ^= 1;
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) b[n * 16 + threadIdx.x / kWave] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            // the 16 slots, those past the last wave zero (norm_clear)
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const f32x4 q = reinterpret_cast<const f32x4 *>(b + n * 16)[w];
                s += (q[0] + q[1]) + (q[2] + q[3]);
            }
            v[n] = s;
        }
    }
};
__device__ __forceinline__ void norm_clear(float *red, int words) {
    for (int i = threadIdx.x; i < words; i += blockDim.x) red[i] = 0.f;
}

// CH chunks per thread; lds: RowSum's words, then the gains.
template <bool F32, int CH>
__device__ __forceinline__ void norm_fwd_body(const NormArgs &a, float *lds) {
    constexpr bool in_lds = CH == 1, ahead = CH <= 2;  // gains in LDS; the next row's loads ahead
    constexpr int RS = F32 ? 4 : 2;
    const int t = threadIdx.x, nt = blockDim.x, H = a.H;
    const bool post = a.g_post, pre = a.g_pre, elem = a.gate == MOE_GATE_ELEM, token = a.gate == MOE_GATE_TOKEN;
    const float inv_h = 1.0f / (float)H, alpha = a.y ? a.alpha : 1.0f;
    const void *ze = elem ? a.z : nullptr;
    RowSum<1> sum(lds);
    const NormGains gains{a.g_post, a.g_pre, in_lds ? lds + 32 : nullptr, H};
    Raw8<false> y[CH], z[CH];
    Raw8<F32> r[CH];
    float zt;
    auto fetch = [&](int64_t row, bool in) {
        const __amdgpu_buffer_rsrc_t br = row_buffer<RS>(a.r, row, H, in), by = row_buffer<2>(a.y, row, H, in),
                                     bz = row_buffer<2>(ze, row, H, in);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            r[i].load(br, i * nt + t);
            y[i].load(by, i * nt + t);
            z[i].load(bz, i * nt + t);
        }
        zt = row_word(token ? a.z : nullptr, row, in);
    };
    int64_t row = blockIdx.x;
    if (row >= a.rows) return;
    if (ahead) fetch(row, true);
    norm_clear(lds, 32);
    gains.fill();
    __syncthreads();
    for (; row < a.rows; row += gridDim.x) {
        float v[CH][8], p[CH][8], s[1] = {0.f};
        if (!ahead) fetch(row, true);
        float scale = a.beta;
        if (token) scale *= sigmoid(zt);
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float yv = y[i][e];
                s[0] = fmaf(yv, yv, s[0]);
                p[i][e] = (elem ? scale * sigmoid(z[i][e]) : scale) * yv;
                v[i][e] = alpha * r[i][e];
            }
        if (ahead) fetch(row + gridDim.x, row + gridDim.x < a.rows);
        float ystd = 1.0f;
        if (post) {
            sum(s);
            ystd = __builtin_amdgcn_rsqf(fmaf(s[0], inv_h, a.eps));
        }
        s[0] = 0.f;
        const __amdgpu_buffer_rsrc_t br = row_buffer<RS>(a.r_out, row, H), bx = row_buffer<2>(a.xn, row, H);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float g[8];
            gains.load<in_lds>(0, i * nt + t, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = fmaf(p[i][e] * ystd, g[e], v[i][e]);
                s[0] = fmaf(v[i][e], v[i][e], s[0]);
            }
            store8<F32>(br, i * nt + t, v[i]);
        }
        float rstd = 0.f;
        if (pre) {
            sum(s);
            rstd = __builtin_amdgcn_rsqf(fmaf(s[0], inv_h, a.eps));
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float g[8], x[8];
            gains.load<in_lds>(1, i * nt + t, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = v[i][e] * rstd * g[e];
            store8<false>(bx, i * nt + t, x);
        }
        if (t == 0) reinterpret_cast<float2 *>(a.stats)[row] = make_float2(post ? ystd : 0.f, rstd);
    }
}

// A value that the compiler must hold as it is, not as others that it can be computed from.
template <class T>
__device__ __forceinline__ void keep(T &v) {
    asm volatile("" : "+v"(v));
}

// Up to H = 8192: one chunk per thread, the row and the next one's loads in registers,
// gains in LDS.  With an fp32 residual the registers are just enough: the gate is held in
// eight (Gate; with exp(-z) and s beside each other 15 are spilled) and y as it lies in
// memory, in four, not as yh: 20,000 rows of 4,096 take 353 us, 390 with yh held, which
// spills 4; with bf16, where nothing is, holding y costs 4,095 rows of 2,048 31.7 us for 30.2.
template <bool F32>
__device__ __forceinline__ void norm_bwd_body(const NormBwdArgs &b, float *lds) {
    constexpr int RS = F32 ? 4 : 2;
    const NormArgs &a = b.f;
    const int t = threadIdx.x, H = a.H;
    const bool post = a.g_post, pre = a.g_pre, elem = a.gate == MOE_GATE_ELEM, token = a.gate == MOE_GATE_TOKEN;
    const float inv_h = 1.0f / (float)H, alpha = a.y ? a.alpha : 1.0f, beta = a.y ? a.beta : 0.0f;
    const void *ze = elem ? a.z : nullptr;
    RowSum<2> sum(lds);
    const NormGains gains{a.g_post, a.g_pre, lds + 64, H};
    Raw8<false> y, z, dx;
    Raw8<F32> r, up;
    float st_y, st_r, zt;
    auto fetch = [&](int64_t row, bool in) {
        const __amdgpu_buffer_rsrc_t br = row_buffer<RS>(a.r, row, H, in), by = row_buffer<2>(a.y, row, H, in),
                                     bz = row_buffer<2>(ze, row, H, in), bu = row_buffer<RS>(b.dr_out, row, H, in),
                                     bd = row_buffer<2>(b.dxn, row, H, in);
        r.load(br, t);
        y.load(by, t);
        z.load(bz, t);
        up.load(bu, t);
        dx.load(bd, t);
        st_y = row_word(a.stats, 2 * row, in);
        st_r = row_word(a.stats, 2 * row + 1, in);
        zt = row_word(token ? a.z : nullptr, row, in);
    };
    float acc_post[8], acc_pre[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc_post[e] = acc_pre[e] = 0.f;
    int64_t row = blockIdx.x;
    if (row >= a.rows) return;
    fetch(row, true);
    norm_clear(lds, 64);
    gains.fill();
    __syncthreads();
    for (; row < a.rows; row += gridDim.x) {
        const float ystd = post ? st_y : 1.0f, rstd = st_r;
        const float et = token ? __expf(-zt) : 0.0f, gt = token ? __builtin_amdgcn_rcpf(1.0f + et) : 1.0f;
        // yh, the gate, D (first what arrives for r'), t and xh of the row
        float yh[8], D[8], tv[8], xh[8], s[2] = {0.f, 0.f};
        Gate gate[8];
        float go[8], gi[8];
        gains.load<true>(0, t, go);
        gains.load<true>(1, t, gi);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            yh[e] = y[e] * ystd;
            const float ez = elem ? __expf(-z[e]) : et, gv = elem ? __builtin_amdgcn_rcpf(1.0f + ez) : gt;
            gate[e] = Gate(ez, gv);
            keep(gate[e].k);
            D[e] = up[e];
            xh[e] = fmaf(beta * gv, yh[e] * go[e], alpha * r[e]) * rstd;
            const float d = dx[e];
            tv[e] = d * gi[e];
            acc_pre[e] = fmaf(d, xh[e], acc_pre[e]);
            s[0] = fmaf(tv[e], xh[e], s[0]);
        }
        Raw8<false> yk = y;
        if constexpr (F32) keep(yk.v);
        fetch(row + gridDim.x, row + gridDim.x < a.rows);
        if (pre) {
            sum(s);
            const float c1 = s[0] * inv_h;
#pragma unroll
            for (int e = 0; e < 8; ++e) D[e] = fmaf(rstd, fmaf(-xh[e], c1, tv[e]), D[e]);
        }
        s[0] = s[1] = 0.f;
        const __amdgpu_buffer_rsrc_t br = row_buffer<RS>(b.dr, row, H), by = row_buffer<2>(b.dy, row, H),
                                     bz = row_buffer<2>(elem ? b.dz : nullptr, row, H);
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = alpha * D[e];
        store8<F32>(br, t, o);
        gains.load<true>(0, t, go);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (F32) yh[e] = yk[e] * ystd;
            const float d = beta * D[e], p = yh[e] * go[e], gv = gate[e].open();
            o[e] = d * p * gv * gate[e].rest();
            s[1] = fmaf(d, p, s[1]);
            const float dp = d * gv;
            acc_post[e] = fmaf(dp, yh[e], acc_post[e]);
            D[e] = dp * go[e];  // q
            s[0] = fmaf(D[e], yh[e], s[0]);
        }
        store8<false>(bz, t, o);
        if (post || token) sum(s);
        const float c2 = post ? s[0] * inv_h : 0.f;
        // without a post-norm dy is q itself, whatever y holds (an infinity times c2 = 0 would be NaN)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = post ? ystd * fmaf(-yh[e], c2, D[e]) : D[e];
        store8<false>(by, t, o);
        if (token && t == 0) static_cast<float *>(b.dz)[row] = s[1] * gt * Gate(et, gt).rest();
    }
    if (post || pre) {
        const __amdgpu_buffer_rsrc_t bo = row_buffer<4>(post ? b.part : nullptr, 2 * (int64_t)blockIdx.x, H),
                                     bi = row_buffer<4>(pre ? b.part : nullptr, 2 * (int64_t)blockIdx.x + 1, H);
        store8<true>(bo, t, acc_post);
        store8<true>(bi, t, acc_pre);
    }
}

// A chunk of a row as the backward reads it, and what it makes of one element.
template <bool F32>
struct NormBwdChunk {
    Raw8<false> y, z, dx;
    Raw8<F32> r, up;
    template <bool KEEP>
    __device__ __forceinline__ void load(const NormBwdArgs &b, int64_t row, int c) {
        constexpr int RS = F32 ? 4 : 2;
        const NormArgs &a = b.f;
        r.template load<KEEP>(row_buffer<RS>(a.r, row, a.H), c);
        y.template load<KEEP>(row_buffer<2>(a.y, row, a.H), c);
        z.template load<KEEP>(row_buffer<2>(a.gate == MOE_GATE_ELEM ? a.z : nullptr, row, a.H), c);
        up.template load<KEEP>(row_buffer<RS>(b.dr_out, row, a.H), c);
        dx.template load<KEEP>(row_buffer<2>(b.dxn, row, a.H), c);
    }
};
struct NormBwdElem {
    float yh, e, gate, u, xh, t;  // e = exp(-z), gate = s; u = beta s p, the block's part of r'
};

// Past H = 8192 a row does not fit the registers beside the column sums (holding it
// spilled: 10,000 rows of 12,288 took 810 us against 490, 4,000 of 32,768 2,490 against
// 757): the row is read for its sums and read again, from the caches, for the outputs
// (617 and 832 us where the first reading is nontemporal too), with one reduction
// between: with u = beta s p, the three sums
//   S1 = sum t xh,  S2 = sum u (dr' + rstd(r') t),  S3 = sum u xh
// give both means, mean(t xh) = S1 / H and, because q yh = D u, mean(q yh) =
// (S2 - rstd(r') S1 S3 / H) / H.  (The same single reduction in the body above costs
// the registers that hold the next row: 4,095 rows of 2,056 in fp32 took 56 us for 44.)
template <bool F32, int CH>
__device__ __forceinline__ void norm_bwd_wide_body(const NormBwdArgs &b, float *lds) {
    constexpr int RS = F32 ? 4 : 2;
    const NormArgs &a = b.f;
    const int t = threadIdx.x, nt = blockDim.x, H = a.H;
    const bool post = a.g_post, pre = a.g_pre, elem = a.gate == MOE_GATE_ELEM, token = a.gate == MOE_GATE_TOKEN;
    const float inv_h = 1.0f / (float)H, alpha = a.y ? a.alpha : 1.0f, beta = a.y ? a.beta : 0.0f;
    RowSum<3> sum(lds);
    // gains and rows are read from memory as they are used
    const NormGains gains{a.g_post, a.g_pre, nullptr, H};
    using Chunk = NormBwdChunk<F32>;
    struct Row {
        float st_y, st_r, zt;
    };
    auto fetch_row = [&](Row &k, int64_t row, bool in) {
        k.st_y = row_word(a.stats, 2 * row, in);
        k.st_r = row_word(a.stats, 2 * row + 1, in);
        k.zt = row_word(token ? a.z : nullptr, row, in);
    };
    // the sums of dg_post in LDS, [half][chunk], a thread's own; those of dg_pre in registers
    float acc_pre[CH][8];
    f32x4 *post_lds = reinterpret_cast<f32x4 *>(lds + 96);
    const int half = CH * nt;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc_pre[i][e] = 0.f;
        post_lds[i * nt + t] = post_lds[half + i * nt + t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    int64_t row = blockIdx.x;
    if (row >= a.rows) return;
    Chunk cur;
    Row w, wnext;
    fetch_row(w, row, true);
    norm_clear(lds, 96);
    __syncthreads();
    for (; row < a.rows; row += gridDim.x) {
        const bool more = row + gridDim.x < a.rows;
        fetch_row(wnext, row + gridDim.x, more);
        const float ystd = post ? w.st_y : 1.0f, rstd = w.st_r, et = token ? __expf(-w.zt) : 0.0f,
                    gt = __builtin_amdgcn_rcpf(1.0f + et);  // 1 without a gate
        auto element = [&](const Chunk &k, int e, const float (&go)[8], const float (&gi)[8]) {
            NormBwdElem x;
            x.yh = k.y[e] * ystd;
            x.e = elem ? __expf(-k.z[e]) : et;
            x.gate = elem ? __builtin_amdgcn_rcpf(1.0f + x.e) : gt;
            x.u = beta * x.gate * (x.yh * go[e]);
            x.xh = pre ? fmaf(alpha, k.r[e], x.u) * rstd : 0.f;
            x.t = k.dx[e] * gi[e];
            return x;
        };
        float s[3] = {0.f, 0.f, 0.f};
        // the scheduling barriers keep one chunk's loads and values in registers at a time
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            float go[8], gi[8];
            cur.template load<true>(b, row, c);
            gains.load<false>(0, c, go);
            gains.load<false>(1, c, gi);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const NormBwdElem x = element(cur, e, go, gi);
                s[0] = fmaf(x.t, x.xh, s[0]);
                s[1] = fmaf(x.u, fmaf(rstd, x.t, cur.up[e]), s[1]);
                s[2] = fmaf(x.u, x.xh, s[2]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (pre || post || token) sum(s);
        const float c1 = s[0] * inv_h, du = pre ? fmaf(-rstd * c1, s[2], s[1]) : s[1], c2 = post ? du * inv_h : 0.f;
        const __amdgpu_buffer_rsrc_t br = row_buffer<RS>(b.dr, row, H), by = row_buffer<2>(b.dy, row, H),
                                     bz = row_buffer<2>(elem ? b.dz : nullptr, row, H);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            float go[8], gi[8], dr[8], dz[8], dy[8], dp_yh[8];
            cur.template load<false>(b, row, c);
            gains.load<false>(0, c, go);
            gains.load<false>(1, c, gi);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const NormBwdElem x = element(cur, e, go, gi);
                const float D = fmaf(rstd, fmaf(-x.xh, c1, x.t), cur.up[e]), dp = beta * D * x.gate;
                dr[e] = alpha * D;
                // 1 - s as e s, e finite: where e is infinite, u is 0.  (Gate's form, with a selection an
                // element, costs 8,000 rows of 16,384 532 us for 516.)
                dz[e] = D * x.u * (fminf(x.e, __FLT_MAX__) * x.gate);
                dy[e] = post ? ystd * fmaf(-x.yh, c2, dp * go[e]) : dp;  // as above: q itself, whatever y holds
                dp_yh[e] = dp * x.yh;
                acc_pre[i][e] = fmaf(cur.dx[e], x.xh, acc_pre[i][e]);
            }
            f32x4 lo = post_lds[c], hi = post_lds[half + c];
#pragma unroll
            for (int e = 0; e < 4; ++e) lo[e] += dp_yh[e], hi[e] += dp_yh[4 + e];
            post_lds[c] = lo, post_lds[half + c] = hi;
            store8<F32>(br, c, dr);
            store8<false>(bz, c, dz);
            store8<false>(by, c, dy);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (token && t == 0) static_cast<float *>(b.dz)[row] = du * Gate(et, gt).rest();
        w = wnext;
    }
    if (post || pre) {
        const __amdgpu_buffer_rsrc_t bo = row_buffer<4>(post ? b.part : nullptr, 2 * (int64_t)blockIdx.x, H),
                                     bi = row_buffer<4>(pre ? b.part : nullptr, 2 * (int64_t)blockIdx.x + 1, H);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * nt + t;
            const f32x4 lo = post_lds[c], hi = post_lds[half + c];
            const float acc_post[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            store8<true>(bo, c, acc_post);
            store8<true>(bi, c, acc_pre[i]);
        }
    }
}

// dg[c] = the sum over the backward's workgroups of their partial sums: COLS
// columns x 1024 / COLS groups of workgroups, each group in ascending order (eight
// loads at a time), then the groups in a fixed tree.
template <int COLS>
__device__ __forceinline__ void norm_dg_body(const float *part, int parts, int H, float *dg_post, float *dg_pre, float *lds) {
    constexpr int kGroups = 1024 / COLS;
    const int col = blockIdx.x * COLS + threadIdx.x % COLS, g0 = threadIdx.x / COLS;
    float *out = blockIdx.y ? dg_pre : dg_post;
    if (!out) return;  // the whole workgroup
    float s = 0.f;
    if (col < H)
        for (int g = g0; g < parts; g += kGroups * 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = g + kGroups * k < parts ? part[((int64_t)(g + kGroups * k) * 2 + blockIdx.y) * H + col] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    lds[threadIdx.x] = s;
    __syncthreads();
    for (int o = kGroups / 2; o >= 1; o >>= 1) {
        if (g0 < o) lds[threadIdx.x] += lds[threadIdx.x + o * COLS];
        __syncthreads();
    }
    if (g0 == 0 && col < H) out[col] = lds[threadIdx.x];
}

}  // namespace moe

// Activation checkpoints in 8 bits, and the backward that reads them.
//
// Format: 128 consecutive elements of a row share one fp32 scale
//   s = fl(amax / 127),  code = rint(fl(x fl(127 fl(1 / amax)))) in [-127, 127],
// every operation one IEEE fp32 operation, so the codes are the same wherever
// they are computed.  A block whose largest magnitude is below 2^-100 gets
// scale 0; one that holds an infinity or a NaN gets scale NaN (and codes 0),
// so all of it reads back as NaN.  At the same 8 bits a linear code with a
// block maximum keeps a Gaussian block to 0.6% rms, against 2.6% for an 8-bit
// float's relative step; the scale adds 3% to the bytes.
//
// Measured: 61,440 rows of I = 2048, pack 139 us (5.5 TB/s), SwiGLU backward 244 to
// 252 us (5.0 to 5.2 TB/s); a copy of 4 GiB gets 4.9 to 5.4 TB/s.  Both are bound by HBM.
//
// Of the three buffers the bf16 backward keeps per dispatched row (Xd, HU, A:
// H + 3 I elements of 2 bytes) only HU's codes remain (2 I bytes and their
// scales): A is silu(h) u again, and Xd is pulled again from X.
#pragma once

#include "common.hpp"
#include "layer.hpp"

namespace moe {

constexpr int kCkptBlock = 128;
constexpr float kCkptTiny = 0x1p-100f;
constexpr int kCkptThreads = 256;

// Sixteen codes of one block as values.
__device__ __forceinline__ void ckpt_values(const u32x4 &c, float s, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = (float)(int8_t)(c[i >> 2] >> (8 * (i & 3))) * s;
}

// Packs rows [0, min(rows, *nrows)) of a dense [rows][cols] bf16 matrix: the
// blocks of 128 are consecutive in memory, 8 lanes x 16 elements each.
__device__ __forceinline__ void ckpt_pack_body(const uint16_t *src, int64_t rows, int cols, const int32_t *nrows, int8_t *q,
                                               float *scales) {
    if (nrows) rows = min(rows, (int64_t)max(*nrows, 0));
    const int64_t n = rows * (cols / 16), step = (int64_t)gridDim.x * kCkptThreads;
    for (int64_t i = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x; i < n; i += step) {
        const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(src) + 2 * i);
        const u32x4 b = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(src) + 2 * i + 1);
        uint32_t m = 0;  // the largest magnitude's bits (a NaN's exceed an infinity's)
        float x[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t w = k < 4 ? a[k] : b[k - 4];
            const uint32_t lo = w << 16, hi = w & 0xffff0000u;
            m = max(m, max(lo & 0x7fffffffu, hi & 0x7fffffffu));
            x[2 * k] = __uint_as_float(lo);
            x[2 * k + 1] = __uint_as_float(hi);
        }
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
        const float amax = __uint_as_float(m);
        const bool finite = m < 0x7f800000u, tiny = amax < kCkptTiny;
        const float inv = finite && !tiny ? 127.0f * (1.0f / amax) : 0.0f;
        u32x4 c;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f = finite ? x[4 * k + e] * inv : 0.0f;
                w |= ((uint32_t)(int)rintf(f) & 0xffu) << (8 * e);
            }
            c[k] = w;
        }
        reinterpret_cast<u32x4 *>(q)[i] = c;
        if (threadIdx.x % 8 == 0) scales[i / 8] = !finite ? __uint_as_float(0x7fc00000u) : tiny ? 0.0f : amax / 127.0f;
    }
}

// The SwiGLU backward of one element: dA' the gradient of a before the router
// weight wr.  The operations and their order are epilogue_swiglu_bwd_w's, so
// equal h and u give equal bits in both backwards.
struct SwigluGrad {
    float a, dh, du;
};
__device__ __forceinline__ SwigluGrad swiglu_grad(float h, float u, float dap, float wr) {
    const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-h)), dA = wr * dap;
    return {h * sg * u, dA * u * sg * (1.0f + h * (1.0f - sg)), dA * h * sg};
}

// Rows [0, min(rows, *nrows)), LANES lanes per row, 16 columns of h and of u
// per lane and step: h, u from the codes, a, dh and du from dA' and the row's
// weight; the row's sum of dA' a through a fixed butterfly.
template <int LANES>
__device__ __forceinline__ void ckpt_swiglu_bwd_body(const int8_t *q, const float *scales, const uint16_t *dA, const float *wrow,
                                                     int64_t rows, int I, const int32_t *nrows, uint16_t *dHU, uint16_t *A,
                                                     float *dw) {
    if (nrows) rows = min(rows, (int64_t)max(*nrows, 0));
    constexpr int kRows = kCkptThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t step = (int64_t)gridDim.x * kRows;
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES; row < rows; row += step) {
        const float wr = wrow ? wrow[row] : 1.0f;
        const int8_t *qr = q + row * 2 * I;
        const float *sr = scales + row * (2 * I / kCkptBlock);
        float dot = 0.f;
        for (int c = lane * 16; c < I; c += LANES * 16) {
            const u32x4 hc = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(qr + c));
            const u32x4 uc = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(qr + I + c));
            const u32x4 d0 = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(dA + row * I + c));
            const u32x4 d1 = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(dA + row * I + c) + 1);
            float h[16], u[16];
            ckpt_values(hc, sr[c / kCkptBlock], h);
            ckpt_values(uc, sr[(I + c) / kCkptBlock], u);
            u32x4 oh[2], ou[2], oa[2];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t w = k < 4 ? d0[k] : d1[k - 4];
                const float da = __uint_as_float(w << 16), db = __uint_as_float(w & 0xffff0000u);
                const SwigluGrad x = swiglu_grad(h[2 * k], u[2 * k], da, wr), y = swiglu_grad(h[2 * k + 1], u[2 * k + 1], db, wr);
                dot = fmaf(da, x.a, dot);
                dot = fmaf(db, y.a, dot);
                oh[k >> 2][k & 3] = pack_bf2(x.dh, y.dh);
                ou[k >> 2][k & 3] = pack_bf2(x.du, y.du);
                oa[k >> 2][k & 3] = pack_bf2(x.a, y.a);
            }
            u32x4 *ph = reinterpret_cast<u32x4 *>(dHU + row * 2 * I + c), *pu = reinterpret_cast<u32x4 *>(dHU + row * 2 * I + I + c);
            ph[0] = oh[0], ph[1] = oh[1];
            pu[0] = ou[0], pu[1] = ou[1];
            if (A) {
                u32x4 *pa = reinterpret_cast<u32x4 *>(A + row * I + c);
                pa[0] = oa[0], pa[1] = oa[1];
            }
        }
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) dot += __shfl_xor(dot, o, kWave);
        if (dw && lane == 0) dw[row] = dot;
    }
}

// ---------------------------------------------------------------------------
// The layer backward's down dgrad on a checkpoint.
// ---------------------------------------------------------------------------

struct CkptBwdArgs {
    BwdArgs b;  // HU and A unused
    const int8_t *q;
    const float *scales;
    uint16_t *A;
};

// The epilogue of bwd_down_phase with h and u decoded from their codes and a
// computed again and written (the weight gradients read it): the fp32 tile dA'
// goes through LDS in two 128-row halves, then every thread takes 8 contiguous
// columns of one row; a row's partial dots meet in a fixed butterfly over its
// 32 threads.
__device__ __forceinline__ void epilogue_swiglu_bwd_ckpt(AccW<kBwdWM, kBwdWN> &acc, char *lds, const int8_t *q, const float *scales,
                                                         const float *wrow, uint16_t *dHU, uint16_t *A, float *part, int nparts,
                                                         int I, int n0) {
    constexpr int WM = kBwdWM, WN = kBwdWN;
    using WG = WaveGrid<WM, WN>;
    constexpr int NT = WG::THREADS;
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, wm = wave / WN, wn = wave % WN;
    float *st = reinterpret_cast<float *>(lds);  // [128][256]
    const int ncols = min(256, I - n0);          // a multiple of 128
    const int64_t ld2 = 2ll * I, lds2 = ld2 / kCkptBlock;
    constexpr int rows_per_wave = 256 / WM;
    static_assert(rows_per_wave <= 128 && 128 % rows_per_wave == 0, "a wave's rows stay in one half");
    const int my_half = (wm * rows_per_wave) / 128;
    float *base = st + ((wm * rows_per_wave) % 128 + 4 * (lane >> 5)) * 256 + wn * (WG::NI * 32) + (lane & 31);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncthreads();  // the main loop or the previous half is done with LDS
        if (my_half == half) {
#pragma unroll
            for (int mi = 0; mi < WG::MI; ++mi)
#pragma unroll
                for (int ni = 0; ni < WG::NI; ++ni)
#pragma unroll
                    for (int e = 0; e < 16; ++e) base[(mi * 32 + 8 * (e >> 2) + (e & 3)) * 256 + ni * 32] = acc[mi][ni][e];
        }
        __syncthreads();
        for (int c = t; c < 128 * 32; c += NT) {
            const int rl = c >> 5, cc = (c & 31) * 8;
            const int row = 128 * half + rl;
            float dot = 0.f;
            if (cc < ncols) {
                const float wr = wrow[row];
                const int col = n0 + cc;
                const float4 d0 = *reinterpret_cast<const float4 *>(st + rl * 256 + cc);
                const float4 d1 = *reinterpret_cast<const float4 *>(st + rl * 256 + cc + 4);
                const float dap[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
                const uint2 hc = *reinterpret_cast<const uint2 *>(q + row * ld2 + col);
                const uint2 uc = *reinterpret_cast<const uint2 *>(q + row * ld2 + I + col);
                const float hs = scales[row * lds2 + col / kCkptBlock], us = scales[row * lds2 + (I + col) / kCkptBlock];
                u32x4 dh, du, av;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    SwigluGrad g[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int e = 2 * k + j;
                        const float h = (float)(int8_t)((e < 4 ? hc.x : hc.y) >> (8 * (e & 3))) * hs;
                        const float u = (float)(int8_t)((e < 4 ? uc.x : uc.y) >> (8 * (e & 3))) * us;
                        g[j] = swiglu_grad(h, u, dap[e], wr);
                        dot = fmaf(dap[e], g[j].a, dot);
                    }
                    dh[k] = pack_bf2(g[0].dh, g[1].dh);
                    du[k] = pack_bf2(g[0].du, g[1].du);
                    av[k] = pack_bf2(g[0].a, g[1].a);
                }
                *reinterpret_cast<u32x4 *>(dHU + row * ld2 + col) = dh;
                *reinterpret_cast<u32x4 *>(dHU + row * ld2 + I + col) = du;
                *reinterpret_cast<u32x4 *>(A + (int64_t)row * I + col) = av;
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) dot += __shfl_xor(dot, off, 64);
            if ((c & 31) == 0) part[(int64_t)row * nparts + n0 / 256] = dot;
        }
    }
}

// B2 of the layer backward (bwd_down_phase) on a checkpoint.
__device__ __forceinline__ void bwd_down_ckpt_phase(const CkptBwdArgs &k, char *lds) {
    const BwdArgs &a = k.b;
    const int H = a.H, I = a.I;
    const int npad = a.seg_off[a.L];
    const int mtiles = npad / kBM, ntiles = (I + 255) / 256;
    const int64_t total = (int64_t)mtiles * ntiles;
    for (int64_t it = blockIdx.x; it - blockIdx.x < total; it += gridDim.x) {
        const int64_t lid = logical_tile(it);
        if (lid >= total) continue;
        int mt, nt;
        grouped_mn<4>(lid, mtiles, ntiles, mt, nt);
        const int64_t m0 = (int64_t)mt * kBM;
        const int l = expert_of(a.seg_off, a.L, (int)m0);
        const uint16_t *g = a.dOd + m0 * H;
        const KOp ak{g, g + 128ll * H, H};
        const TOp bk{a.W2 + (int64_t)l * H * I + nt * 256, I, min(256, I - nt * 256)};  // [k = h][i]
        AccW<kBwdWM, kBwdWN> acc;
        gemm_mainloop_x<kBwdWM, kBwdWN, false, true>(ak, bk, H / 64, false, lds, acc);
        epilogue_swiglu_bwd_ckpt(acc, lds, k.q + m0 * 2 * I, k.scales + m0 * (2 * I / kCkptBlock), a.wrow + m0, a.dHU + m0 * 2 * I,
                                 k.A + m0 * I, a.part + m0 * a.nparts, a.nparts, I, nt * 256);
    }
}

}  // namespace moe

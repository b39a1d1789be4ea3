// The whole expert layer for a few tokens, in two launches.
//
//   gate/up  a_r = silu(x_t Wg[e]^T) * (x_t Wu[e]^T) for every local route
//            r = (t, j), e its expert            -> act (bf16, one rounding)
//   down     out_t = sum_j w_tj (a_r W2[e]^T) (+ the shared expert's output),
//            ascending j, in fp32                -> out (bf16, one rounding)
//
// With a few routes per expert both products read each weight once and use it
// for at most a few dozen columns, so the time is the weights' HBM read: a
// 16 x 16 x 32 MFMA takes 1 KiB of weights in 16 cycles, some 25 times the
// rate at which a CU's share of HBM delivers them.  Everything here is laid
// out for that read:
//   - the weights are the MFMA's A operand, straight from HBM to registers
//     (16 bytes per lane, a whole row's consecutive 64 bytes per instruction);
//     nothing is staged, so no barrier stands in the stream;
//   - the tokens are the columns of the B operand, read from L2 (a column
//     past the expert's last route re-reads the last one, its result unused);
//   - the waves of a workgroup share one block of weight rows and split the
//     reduction dimension (gate/up) or the experts and the reduction dimension
//     (down); their partial sums meet in LDS in a fixed order;
//   - only experts that a route names are read: every gate/up workgroup builds
//     the list of them from the routes, so no schedule launch comes first.
// No atomics touch a float: the result does not depend on timing.
#pragma once

#include "common.hpp"
#include "gemm.hpp"

namespace moe {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;
constexpr int kFewMaxRoutes = 1024;  // routes of one call (P * Np * K)
constexpr int kFewTiles = 4;         // 16-column tiles of one pass over an expert's weights
constexpr int kFewRows = 16;         // activation columns (gate/up) or output columns (down) of a block

struct FewArgs {
    const int32_t *routes;
    const float *w;
    const uint16_t *X;
    const void *W13, *W2;        // bf16, or E4M3 codes
    const uint8_t *W13s, *W2s;   // E8M0 scale bytes of the codes
    const uint16_t *S13, *S2;    // the shared expert's weights (bf16)
    uint16_t *out, *act;
    int32_t *plan;
    int T, K, R, E, L, base, H, I, Is, ld;  // ld: elements of an activation row, max(I, Is)
    int S;                                  // down: parts of the reduction dimension
};

// The list of a call's local routes grouped by expert, in the workspace
// (written by the gate/up launch's first workgroup, read by the down launch).
//   [0] ids outside [0, E)  [1] experts with a route (A)  [2] local routes (n)
//   [kFewHead ...]       A expert ids, then A + 1 offsets
//   then n route numbers in expert order, then the place of each route (-1)
constexpr int kFewHead = 64;
__host__ __device__ inline int few_max_experts(int L, int R) { return L < R ? L : R; }
__host__ __device__ inline int few_plan_words(int L, int R) { return kFewHead + 2 * few_max_experts(L, R) + 1 + 2 * R; }

struct FewPlan {
    int *expert, *off, *route, *place;
    __host__ __device__ FewPlan(int *p, int L, int R) {
        const int m = few_max_experts(L, R);
        expert = p;
        off = expert + m;
        route = off + m + 1;
        place = route + R;
    }
};

// Words of LDS of the gate/up launch: the waves' sums, one count per local
// expert, 4 words for the head, and the list; and of the down launch: the
// routes' sums and the list.
constexpr int kFewRedLd = 36;  // 32 sums of a column and 4 words that spread the columns over the banks
constexpr int kFewRedWords = kFewWaves * 2 * 16 * kFewRedLd;
__host__ __device__ inline int few_gateup_words(int L, int R) {
    return kFewRedWords + L + 4 + few_plan_words(L, R) - kFewHead;
}
__host__ __device__ inline int few_down_words(int L, int R, int rows, int S) {
    return S * rows * 16 + few_plan_words(L, R) - kFewHead;
}

// Builds the list in LDS: count the routes of each expert (a route's rank is
// the order in which the LDS atomics answer: it only says which MFMA column
// computes the route, and columns are independent), take the experts with a
// route in ascending order and their offsets, place the routes.
// Returns A; head[0..2] as in the plan.
__device__ __forceinline__ int few_build(const FewArgs &a, int *cnt, const FewPlan &p, int *head) {
    const int t = threadIdx.x;
    constexpr int kPer = kFewMaxRoutes / kFewThreads;
    int lid[kPer], rank[kPer], bad = 0;
    for (int i = t; i < a.L; i += kFewThreads) cnt[i] = 0;
    if (t < 3) head[t] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = t + i * kFewThreads;
        lid[i] = -1;
        if (r < a.R) {
            const int e = a.routes[r];
            bad += e < 0 || e >= a.E;
            if (e >= a.base && e - a.base < a.L) {
                lid[i] = e - a.base;
                rank[i] = atomicAdd(&cnt[lid[i]], 1);
            }
        }
    }
    if (bad) atomicAdd(&head[0], bad);
    __syncthreads();
    if (t < kWave) {
        int na = 0, n = 0;
        for (int l0 = 0; l0 < a.L; l0 += kWave) {
            const int l = l0 + t, c = l < a.L ? cnt[l] : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const int v = __shfl_up(incl, o, kWave);
                if (t >= o) incl += v;
            }
            const uint64_t some = ballot(c > 0);
            if (c > 0) {
                const int k = na + lanes_below(some);
                p.expert[k] = l;
                p.off[k] = n + incl - c;
            }
            if (l < a.L) cnt[l] = n + incl - c;
            na += __popcll(some);
            n += __shfl(incl, kWave - 1, kWave);
        }
        if (t == 0) p.off[na] = n, head[1] = na, head[2] = n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = t + i * kFewThreads;
        if (r < a.R) {
            const int at = lid[i] >= 0 ? cnt[lid[i]] + rank[i] : -1;
            p.place[r] = at;
            if (at >= 0) p.route[at] = r;
        }
    }
    __syncthreads();
    return head[1];
}

// One MX lane chunk: 16 E4M3 codes under one scale as two bf16 fragments (the
// product code * 2^(b - 127) has 4 significant bits, so bf16 holds it exactly
// unless it is below bf16's range).
__device__ __forceinline__ void few_mx_frags(const u32x4 &c, uint32_t sbyte, bf16x8 &f0, bf16x8 &f1) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(sbyte ? sbyte << 23 : 0x00400000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true);
        bf16x8 &f = i < 2 ? f0 : f1;
        f[4 * (i & 1)] = lo[0];
        f[4 * (i & 1) + 1] = lo[1];
        f[4 * (i & 1) + 2] = hi[0];
        f[4 * (i & 1) + 3] = hi[1];
    }
}

// acc[m][t] += W rows . columns over `steps` chunks of the reduction dimension
// (32 elements bf16, 64 codes MX).  Lane (row or column r = lane & 15, group
// g = lane >> 4) holds elements 8 g .. 8 g + 7 of a chunk of 32 (bf16), or
// 16 g .. 16 g + 15 of a chunk of 64 (MX: the first MFMA takes each group's
// first 8, the second its last 8; both operands use the same order, so the
// sum is over the same elements).
// wp[m]: this lane's row of row block m, advanced to its group and first
// chunk; xp[t]: this lane's column of tile t, the same; ws[m]: the row's scale
// bytes, advanced to the first chunk.
template <bool MX, int M, int NT, int U>
__device__ __forceinline__ void few_chunks(const uint8_t *const (&wp)[M], const uint8_t *const (&ws)[M],
                                           const uint16_t *const (&xp)[NT], int k0, f32x4 (&acc)[M][NT]) {
    u32x4 wv[U][M];
    uint32_t sb[U][M];
    bf16x8 xv[U][NT][MX ? 2 : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            wv[u][m] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wp[m] + (int64_t)(k0 + u) * 64));
            if constexpr (MX) sb[u][m] = ws[m][2 * (k0 + u)];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            xv[u][t][0] = *reinterpret_cast<const bf16x8 *>(xp[t] + (int64_t)(k0 + u) * (MX ? 64 : 32));
            if constexpr (MX) xv[u][t][1] = *reinterpret_cast<const bf16x8 *>(xp[t] + (int64_t)(k0 + u) * 64 + 8);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if constexpr (MX) {
                bf16x8 f0, f1;
                few_mx_frags(wv[u][m], sb[u][m], f0, f1);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f0, xv[u][t][0], acc[m][t], 0, 0, 0);
                    acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f1, xv[u][t][1], acc[m][t], 0, 0, 0);
                }
            } else {
                const bf16x8 f = __builtin_bit_cast(bf16x8, wv[u][m]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, xv[u][t][0], acc[m][t], 0, 0, 0);
            }
        }
}

template <bool MX, int M, int NT>
__device__ __forceinline__ void few_product(const uint8_t *const (&wp)[M], const uint8_t *const (&ws)[M],
                                            const uint16_t *const (&xp)[NT], int k0, int k1, f32x4 (&acc)[M][NT]) {
    // chunks whose loads are in flight together: as many as 128 registers hold
    // beside the sums (four waves per SIMD, no spills)
    constexpr int per = 4 * M + (MX ? 8 : 4) * NT;
    constexpr int U = per * 4 + 4 * M * NT <= 84 ? 4 : per * 2 + 4 * M * NT <= 84 ? 2 : 1;
    int k = k0;
    for (; k + U <= k1; k += U) few_chunks<MX, M, NT, U>(wp, ws, xp, k, acc);
    for (; k < k1; ++k) few_chunks<MX, M, NT, 1>(wp, ws, xp, k, acc);
}

// A weight matrix of an expert: rows of `cols` elements, bf16 or MX.
struct FewMatrix {
    const uint8_t *p, *s;
    int cols;
};
template <bool MX>
__device__ __forceinline__ void few_row(const FewMatrix &m, int64_t row, int group, const uint8_t *&wp, const uint8_t *&ws) {
    if constexpr (MX) {
        wp = m.p + row * m.cols + group * 16;
        ws = m.s + row * (m.cols / 32) + (group >> 1);
    } else {
        wp = m.p + (row * m.cols + group * 8) * 2;
        ws = nullptr;
    }
}

// Gate/up of columns [i0, i0 + 16) of one expert for up to NT * 16 of its
// routes: the workgroup's waves split H; sums meet in LDS (red), two tiles at
// a time, added in wave order.  rows: the routes' X rows (token numbers) come
// from `route` (divided by K; null: the token is the route itself, shared
// expert), whose activations go to act + route * ld.
template <bool MX, int NT>
__device__ __forceinline__ void few_gateup_pass(const FewArgs &a, const FewMatrix &W, int inner, int i0, const int *route,
                                                int first, int n, float *red) {
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, c = lane & 15, g = lane >> 4;
    const uint8_t *wp[2], *ws[2];
    const uint16_t *xp[NT];
    few_row<MX>(W, i0 + c, g, wp[0], ws[0]);
    few_row<MX>(W, (int64_t)inner + i0 + c, g, wp[1], ws[1]);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int k = min(first + q * 16 + c, n - 1);
        const int tok = route ? route[k] / a.K : k;
        xp[q] = a.X + (int64_t)tok * a.H + g * (MX ? 16 : 8);
    }
    f32x4 acc[2][NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int chunks = a.H / (MX ? 64 : 32);
    few_product<MX, 2, NT>(wp, ws, xp, wave * chunks / kFewWaves, (wave + 1) * chunks / kFewWaves, acc);
#pragma unroll
    for (int q0 = 0; q0 < NT; q0 += 2) {
        __syncthreads();  // the previous sums have been read
#pragma unroll
        for (int q = q0; q < (q0 + 2 < NT ? q0 + 2 : NT); ++q) {
            float *dst = red + ((wave * 2 + q - q0) * 16 + c) * kFewRedLd + 4 * g;
            *reinterpret_cast<f32x4 *>(dst) = acc[0][q];
            *reinterpret_cast<f32x4 *>(dst + 16) = acc[1][q];
        }
        __syncthreads();
        const int q = t >> 8, col = (t >> 4) & 15, i = t & 15, k = first + (q0 + q) * 16 + col;
        if (q0 + q < NT && k < n) {
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) {
                const float *src = red + ((v * 2 + q) * 16 + col) * kFewRedLd + i;
                gate += src[0];
                up += src[16];
            }
            const int row = route ? route[k] : a.R + k;
            a.act[(int64_t)row * a.ld + i0 + i] = f2bf(gate / (1.0f + __expf(-gate)) * up);
        }
    }
}

template <bool MX>
__device__ __forceinline__ void few_gateup_unit(const FewArgs &a, const FewMatrix &W, int inner, int i0, const int *route, int n,
                                                float *red) {
    for (int first = 0; first < n; first += 16 * kFewTiles) {
        const int left = n - first;
        if (left <= 16)
            few_gateup_pass<MX, 1>(a, W, inner, i0, route, first, n, red);
        else if (left <= 32)
            few_gateup_pass<MX, 2>(a, W, inner, i0, route, first, n, red);
        else
            few_gateup_pass<MX, kFewTiles>(a, W, inner, i0, route, first, n, red);
    }
}

// Persistent over (expert, block of 16 activation columns): the shared
// expert's blocks first (they have every token's column, so they are the
// longest), then those of the experts that have a route.
template <bool MX>
__device__ __forceinline__ void few_gateup_body(const FewArgs &a, int *lds) {
    float *red = reinterpret_cast<float *>(lds);
    int *cnt = lds + kFewRedWords, *head = cnt + a.L;
    const FewPlan p(head + 4, a.L, a.R);
    const int na = few_build(a, cnt, p, head);
    if (blockIdx.x == 0) {
        const FewPlan o(a.plan + kFewHead, a.L, a.R);
        if (threadIdx.x < 3) a.plan[threadIdx.x] = head[threadIdx.x];
        for (int i = threadIdx.x; i <= na; i += kFewThreads) {
            if (i < na) o.expert[i] = p.expert[i];
            o.off[i] = p.off[i];
        }
        for (int i = threadIdx.x; i < a.R; i += kFewThreads) {
            if (i < head[2]) o.route[i] = p.route[i];
            o.place[i] = p.place[i];
        }
    }
    const int blocks = a.I / kFewRows, shared = a.Is / kFewRows;
    const int64_t units = (int64_t)na * blocks + shared;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        if (u < shared) {
            const FewMatrix W{reinterpret_cast<const uint8_t *>(a.S13), nullptr, a.H};
            few_gateup_unit<false>(a, W, a.Is, (int)u * kFewRows, nullptr, a.T, red);
        } else {
            const int k = (int)((u - shared) / blocks), i0 = (int)((u - shared) % blocks) * kFewRows;
            const int64_t row = (int64_t)p.expert[k] * 2 * a.I;
            const FewMatrix W{static_cast<const uint8_t *>(a.W13) + row * a.H * (MX ? 1 : 2), MX ? a.W13s + row * (a.H / 32) : nullptr,
                              a.H};
            few_gateup_unit<MX>(a, W, a.I, i0, p.route + p.off[k], p.off[k + 1] - p.off[k], red);
        }
    }
}

// Down of output columns [h0, h0 + 16) for up to NT * 16 routes of one expert
// over one part of its activations: one wave, no barrier; the sums go to
// y[place][16].
template <bool MX, int NT>
__device__ __forceinline__ void few_down_pass(const FewArgs &a, const FewMatrix &W, int h0, const int *route, int first, int n,
                                              int part, float *y) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const uint8_t *wp[1], *ws[1];
    const uint16_t *xp[NT];
    few_row<MX>(W, h0 + c, g, wp[0], ws[0]);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int k = min(first + q * 16 + c, n - 1);
        xp[q] = a.act + (int64_t)(route ? route[k] : a.R + k) * a.ld + g * (MX ? 16 : 8);
    }
    f32x4 acc[1][NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[0][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int chunks = W.cols / (MX ? 64 : 32);
    few_product<MX, 1, NT>(wp, ws, xp, part * chunks / a.S, (part + 1) * chunks / a.S, acc);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int k = first + q * 16 + c;
        if (k < n) *reinterpret_cast<f32x4 *>(y + k * 16 + 4 * g) = acc[0][q];
    }
}

template <bool MX>
__device__ __forceinline__ void few_down_unit(const FewArgs &a, const FewMatrix &W, int h0, const int *route, int n, int part,
                                              float *y) {
    for (int first = 0; first < n; first += 16 * kFewTiles) {
        const int left = n - first;
        if (left <= 16)
            few_down_pass<MX, 1>(a, W, h0, route, first, n, part, y);
        else if (left <= 32)
            few_down_pass<MX, 2>(a, W, h0, route, first, n, part, y);
        else
            few_down_pass<MX, kFewTiles>(a, W, h0, route, first, n, part, y);
    }
}

// One workgroup per 16 output columns: its waves take (expert, part) pairs in
// turn, the shared expert's first, and leave every route's sums in LDS
// (y[part][place]); then every output element adds its token's routes in
// ascending slot order, the shared expert last, and is rounded once.
template <bool MX>
__device__ __forceinline__ void few_down_body(const FewArgs &a, int *lds) {
    const int t = threadIdx.x, wave = t >> 6, h0 = blockIdx.x * kFewRows;
    const int rows = a.R + (a.Is ? a.T : 0);  // y rows of a part: the routes, then the shared expert's tokens
    float *y = reinterpret_cast<float *>(lds);
    const FewPlan p(lds + a.S * rows * 16, a.L, a.R), src(a.plan + kFewHead, a.L, a.R);
    const int na = a.plan[1], n = a.plan[2];
    for (int i = t; i <= na; i += kFewThreads) {
        if (i < na) p.expert[i] = src.expert[i];
        p.off[i] = src.off[i];
    }
    for (int i = t; i < a.R; i += kFewThreads) {
        if (i < n) p.route[i] = src.route[i];
        p.place[i] = src.place[i];
    }
    __syncthreads();
    const int shared = a.Is ? a.S : 0, units = na * a.S + shared;
    for (int u = wave; u < units; u += kFewWaves) {
        if (u < shared) {
            const FewMatrix W{reinterpret_cast<const uint8_t *>(a.S2), nullptr, a.Is};
            few_down_unit<false>(a, W, h0, nullptr, a.T, u, y + ((int64_t)u * rows + a.R) * 16);
        } else {
            const int k = (u - shared) / a.S, part = (u - shared) % a.S;
            const int64_t row = (int64_t)p.expert[k] * a.H;
            const FewMatrix W{static_cast<const uint8_t *>(a.W2) + row * a.I * (MX ? 1 : 2), MX ? a.W2s + row * (a.I / 32) : nullptr, a.I};
            few_down_unit<MX>(a, W, h0, p.route + p.off[k], p.off[k + 1] - p.off[k], part, y + (part * rows + p.off[k]) * 16);
        }
    }
    __syncthreads();
    for (int i = t; i < a.T * 16; i += kFewThreads) {
        const int tok = i >> 4, h = i & 15;
        float sum = 0.f;
        for (int j = 0; j < a.K; ++j) {
            const int at = p.place[tok * a.K + j];
            if (at < 0) continue;
            float v = 0.f;
            for (int s = 0; s < a.S; ++s) v += y[(s * rows + at) * 16 + h];
            sum = fmaf(a.w[tok * a.K + j], v, sum);
        }
        if (a.Is) {
            float v = 0.f;
            for (int s = 0; s < a.S; ++s) v += y[(s * rows + a.R + tok) * 16 + h];
            sum += v;
        }
        a.out[(int64_t)tok * a.H + h0 + h] = f2bf(sum);
    }
}

}  // namespace moe

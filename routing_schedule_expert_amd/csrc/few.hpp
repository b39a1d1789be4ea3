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
//   - the weights are the MFMA's A operand, straight from HBM to registers in
//     whole 128-byte lines (FewLane); nothing is staged, so no barrier stands
//     in the stream, and steps are loaded ahead in registers;
//   - the tokens are the columns of the B operand, read from L2 (a column
//     past the expert's last route re-reads the last one, its result unused);
//   - the waves of a workgroup share one block of weight rows and split the
//     reduction dimension (down: small ones are split less, the waves then
//     take experts in turn); their partial sums meet in LDS in a fixed order;
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
constexpr int kFewRows = 16;         // activation columns of a gate/up unit

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
    int S, cap;                             // down: parts of the reduction dimension; places of a round
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
constexpr int kFewRedWords = kFewWaves * 32 * kFewRedLd;
__host__ __device__ inline int few_gateup_words(int L, int R) {
    return kFewRedWords + L + 4 + few_plan_words(L, R) - kFewHead;
}
__host__ __device__ inline int few_down_words(int L, int R, int rows, int S, int cap, int C) {
    return (rows + S * cap) * C + few_plan_words(L, R) - kFewHead;
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

// How a wave's 64 x 16 bytes of weights lie in one load (and in one MFMA, whose
// lane i + 16 g holds row or column i, group g of its operand):
//   dense  (V = 1)  16 rows x 64 consecutive bytes: lane i + 16 g reads group g
//                   of row i, a tile is 16 tokens;
//   halves (V = 2)  8 rows x 128 consecutive bytes: lane i + 16 g reads group
//                   4 (i & 1) + g of row i / 2, a tile is 8 tokens laid out
//                   alike.  MFMA row (r, p) times column (c, q) is then row r
//                   half p times token c half q: the wanted sum is the p = q
//                   entries of both halves, the other half of the products is
//                   dropped.
// Whole 128-byte lines are worth it: a kernel that only reads gets 7.1 TB/s
// with 128 (or 256) bytes of a row per load and 5.5 TB/s with 64.  The dropped
// products cost nothing while the matrix cores wait for HBM, but a tile holds
// half the tokens, so more than 16 routes of an expert take the dense form.
template <bool MX, int V>
struct FewLane {
    int row, group, token;  // of the weights' block; 16-byte group of a row; of a tile
    __device__ __forceinline__ FewLane() {
        const int lane = lane_id(), i = lane & 15, g = lane >> 4;
        row = token = i / V;
        group = V == 2 ? 4 * (i & 1) + g : g;
    }
    static constexpr int kTokens = 16 / V;
    static constexpr int kRows = 16 / V;                    // rows of a block
    static constexpr int kStep = V * (MX ? 64 : 32);        // elements of the reduction dimension per step
    static constexpr int kGroup = MX ? 16 : 8;              // elements of a group
};

// A weight matrix of an expert: rows of `cols` elements, bf16 or MX (codes p,
// scale bytes s).
struct FewMatrix {
    const uint8_t *p, *s;
    int cols;
};

// One step's operands: M blocks of weight rows and NT tiles of tokens.  With
// MX, the first MFMA takes each group's first 8 codes and the second its last
// 8; both operands use the same order, so the sum is over the same elements.
template <bool MX, int V, int M, int NT>
struct FewStep {
    u32x4 w[M];
    uint32_t sb[M];
    bf16x8 x[NT][MX ? 2 : 1];

    // wp[m], ws[m]: block m's first row at the step's first element (wave-
    // uniform), wo / so this lane's bytes from there; xb the tokens' matrix at
    // the step's first element, xo[t] this lane's bytes from there
    __device__ __forceinline__ void load(const uint8_t *const (&wp)[M], const uint8_t *const (&ws)[M], uint32_t wo, uint32_t so,
                                         const uint8_t *xb, const uint32_t (&xo)[NT], int k) {
        using L = FewLane<MX, V>;
        const uint8_t *xk = xb + (int64_t)k * L::kStep * 2;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            w[m] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wp[m] + (int64_t)k * V * 64 + wo));
            if constexpr (MX && V == 2) sb[m] = *reinterpret_cast<const uint32_t *>(ws[m] + (int64_t)k * 4 + so);
            if constexpr (MX && V == 1) sb[m] = *reinterpret_cast<const uint16_t *>(ws[m] + (int64_t)k * 2 + so);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < (MX ? 2 : 1); ++h) x[t][h] = *reinterpret_cast<const bf16x8 *>(xk + xo[t] + 16 * h);
    }
    __device__ __forceinline__ void mul(const FewLane<MX, V> &l, f32x4 (&acc)[M][NT]) const {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            bf16x8 f[2];
            if constexpr (MX)
                few_mx_frags(w[m], (sb[m] >> (8 * (l.group >> 1))) & 0xffu, f[0], f[1]);
            else
                f[0] = __builtin_bit_cast(bf16x8, w[m]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < (MX ? 2 : 1); ++h)
                    acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[h], x[t][h], acc[m][t], 0, 0, 0);
        }
    }
};

// acc[m][t] = block m's rows times tile t's tokens over the elements [e0, e1)
// of the reduction dimension (multiples of kStep from 0).  D steps are in
// flight: a step's registers are loaded again as soon as they are used.
template <bool MX, int V, int M, int NT>
__device__ __forceinline__ void few_product(const FewLane<MX, V> &l, const uint8_t *const (&wp)[M], const uint8_t *const (&ws)[M],
                                            int cols, const uint8_t *xb, const uint32_t (&xo)[NT], int k0, int k1,
                                            f32x4 (&acc)[M][NT]) {
    using Step = FewStep<MX, V, M, NT>;
    constexpr int per = (MX ? 5 : 4) * M + (MX ? 8 : 4) * NT, left = 92 - 4 * M * NT;  // registers of a step; for all steps
    constexpr int D = left >= 4 * per ? 4 : left >= 3 * per ? 3 : left >= 2 * per ? 2 : 1;
    const uint32_t wo = (uint32_t)(l.row * cols * (MX ? 1 : 2) + l.group * 16), so = (uint32_t)(l.row * (cols / 32));
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    Step st[D];
    int k = k0;
    if (k + D <= k1) {
#pragma unroll
        for (int j = 0; j < D; ++j) st[j].load(wp, ws, wo, so, xb, xo, k + j);
        for (; k + 2 * D <= k1; k += D)
#pragma unroll
            for (int j = 0; j < D; ++j) {
                st[j].mul(l, acc);
                st[j].load(wp, ws, wo, so, xb, xo, k + D + j);
            }
#pragma unroll
        for (int j = 0; j < D; ++j) st[j].mul(l, acc);
        k += D;
    }
    for (; k < k1; ++k) {
        st[0].load(wp, ws, wo, so, xb, xo, k);
        st[0].mul(l, acc);
    }
}

// The sums of a block and tile that this lane keeps: row r(i) of the block and
// the lane's token.  Dense: four rows 4 g + i.  Halves: both halves' entries
// meet (lane ^ 1), then the even lane keeps row 2 g and the odd lane 2 g + 1.
template <int V, class Put>
__device__ __forceinline__ void few_sums(const f32x4 &acc, Put put) {
    const int lane = lane_id(), g = lane >> 4;
    if constexpr (V == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) put(4 * g + i, acc[i]);
    } else {
        const bool odd = lane & 1;
        const float a = odd ? acc[1] : acc[0], b = odd ? acc[3] : acc[2];
        const float sa = a + __shfl_xor(a, 1, kWave), sb = b + __shfl_xor(b, 1, kWave);
        put(2 * g + (odd ? 1 : 0), odd ? sb : sa);
    }
}

__device__ __forceinline__ int wave_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Gate/up of activation columns [i0, i0 + 16) of one expert for up to
// NT tiles of its routes from `first` on: the workgroup's waves split H; their
// sums meet in LDS (red), 32 tokens at a time, added in wave order.  The
// routes' tokens are route[..] / K, their activations go to row route[..] of
// act; route null: the tokens themselves (shared expert), rows R + token.
template <bool MX, int V, int NT>
__device__ __forceinline__ void few_gateup_pass(const FewArgs &a, const FewMatrix &W, int inner, int i0, const int *route,
                                                int first, int n, float *red) {
    using L = FewLane<MX, V>;
    constexpr int M = 2 * V;  // gate blocks, then up blocks
    const L l;
    const int t = threadIdx.x, wave = wave_uniform(t >> 6);
    const uint8_t *wp[M], *ws[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int64_t row = (m < V ? 0 : inner) + i0 + (m % V) * L::kRows;
        wp[m] = W.p + row * W.cols * (MX ? 1 : 2);
        ws[m] = W.s + row * (W.cols / 32);
    }
    uint32_t xo[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int k = min(first + q * L::kTokens + l.token, n - 1);
        const int tok = route ? route[k] / a.K : k;
        xo[q] = (uint32_t)tok * (uint32_t)(a.H * 2) + l.group * (L::kGroup * 2);
    }
    f32x4 acc[M][NT];
    const int steps = a.H / L::kStep;
    few_product<MX, V, M, NT>(l, wp, ws, W.cols, reinterpret_cast<const uint8_t *>(a.X), xo, wave * steps / kFewWaves,
                              (wave + 1) * steps / kFewWaves, acc);
    constexpr int per = 32 / L::kTokens;  // tiles that meet at a time
#pragma unroll
    for (int q0 = 0; q0 < NT; q0 += per) {
        __syncthreads();  // the previous sums have been read
#pragma unroll
        for (int q = q0; q < (q0 + per < NT ? q0 + per : NT); ++q) {
            float *dst = red + (wave * 32 + (q - q0) * L::kTokens + l.token) * kFewRedLd;
#pragma unroll
            for (int m = 0; m < M; ++m) few_sums<V>(acc[m][q], [&](int r, float v) { dst[m * L::kRows + r] = v; });
        }
        __syncthreads();
        const int tok = t >> 4, i = t & 15, k = first + q0 * L::kTokens + tok;
        if (tok < (NT - q0) * L::kTokens && k < n) {
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) {
                const float *src = red + (v * 32 + tok) * kFewRedLd + i;
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
    if (n <= 8) return few_gateup_pass<MX, 2, 1>(a, W, inner, i0, route, 0, n, red);
    if (n <= 16) return few_gateup_pass<MX, 2, 2>(a, W, inner, i0, route, 0, n, red);
    for (int first = 0; first < n; first += 64) {
        if (n - first <= 32)
            few_gateup_pass<MX, 1, 2>(a, W, inner, i0, route, first, n, red);
        else
            few_gateup_pass<MX, 1, 4>(a, W, inner, i0, route, first, n, red);
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
    const int na = wave_uniform(few_build(a, cnt, p, head));
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
            const int64_t row = (int64_t)wave_uniform(p.expert[k]) * 2 * a.I;
            const int off = wave_uniform(p.off[k]), n = wave_uniform(p.off[k + 1]) - off;
            const FewMatrix W{static_cast<const uint8_t *>(a.W13) + row * a.H * (MX ? 1 : 2), MX ? a.W13s + row * (a.H / 32) : nullptr,
                              a.H};
            few_gateup_unit<MX>(a, W, a.I, i0, p.route + off, n, red);
        }
    }
}

// Down of output columns [h0, h0 + 8 B) for the routes [first, n) of one
// expert, at most NT tiles, over one part of its activations: one wave, no
// barrier; the sums go to y[.. - first][8 B].  act rows as in few_gateup_pass.
template <bool MX, int V, int B, int NT>
__device__ __forceinline__ void few_down_pass(const FewArgs &a, const FewMatrix &W, int h0, const int *route, int first, int n,
                                              int part, float *y) {
    using L = FewLane<MX, V>;
    constexpr int M = B * V / 2;
    const L l;
    const uint8_t *wp[M], *ws[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int64_t row = h0 + m * L::kRows;
        wp[m] = W.p + row * W.cols * (MX ? 1 : 2);
        ws[m] = W.s + row * (W.cols / 32);
    }
    uint32_t xo[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int k = min(first + q * L::kTokens + l.token, n - 1);
        xo[q] = (uint32_t)(route ? route[k] : a.R + k) * (uint32_t)(a.ld * 2) + l.group * (L::kGroup * 2);
    }
    f32x4 acc[M][NT];
    const int steps = W.cols / L::kStep;
    few_product<MX, V, M, NT>(l, wp, ws, W.cols, reinterpret_cast<const uint8_t *>(a.act), xo, part * steps / a.S,
                              (part + 1) * steps / a.S, acc);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int k = q * L::kTokens + l.token;
#pragma unroll
        for (int m = 0; m < M; ++m)
            few_sums<V>(acc[m][q], [&](int r, float v) {
                if (first + k < n) y[k * 8 * B + m * L::kRows + r] = v;
            });
    }
}

template <bool MX, int B>
__device__ __forceinline__ void few_down_unit(const FewArgs &a, const FewMatrix &W, int h0, const int *route, int first, int n, int part,
                                              float *y) {
    if (n - first <= 8) return few_down_pass<MX, 2, B, 1>(a, W, h0, route, first, n, part, y);
    if (n - first <= 16) return few_down_pass<MX, 2, B, 2>(a, W, h0, route, first, n, part, y);
    for (; first < n; first += 64, y += 64 * 8 * B) {
        if (n - first <= 32)
            few_down_pass<MX, 1, B, 2>(a, W, h0, route, first, n, part, y);
        else
            few_down_pass<MX, 1, B, 4>(a, W, h0, route, first, n, part, y);
    }
}

// One workgroup per 8 B output columns.  Its waves form S parts of the
// reduction dimension times 8 / S groups that take the experts in turn, so
// each wave has its share of every expert's bytes; the routes (in expert
// order, the shared expert's tokens after them) are taken `cap` places at a
// time: their parts' sums (part[S][cap][8 B]) are added in part order into
// y[place].  Then every output element adds its token's routes in ascending
// slot order, the shared expert last, and is rounded once.
template <bool MX, int B>
__device__ __forceinline__ void few_down_body(const FewArgs &a, int *lds) {
    constexpr int C = 8 * B;
    const int t = threadIdx.x, wave = wave_uniform(t >> 6), h0 = blockIdx.x * C;
    const int rows = a.R + (a.Is ? a.T : 0);
    float *y = reinterpret_cast<float *>(lds), *sums = y + rows * C;
    const FewPlan p(lds + rows * C + a.S * a.cap * C, a.L, a.R), src(a.plan + kFewHead, a.L, a.R);
    const int na = wave_uniform(a.plan[1]), n = wave_uniform(a.plan[2]);
    for (int i = t; i <= na; i += kFewThreads) {
        if (i < na) p.expert[i] = src.expert[i];
        p.off[i] = src.off[i];
    }
    for (int i = t; i < a.R; i += kFewThreads) {
        if (i < n) p.route[i] = src.route[i];
        p.place[i] = src.place[i];
    }
    __syncthreads();
    const int part = wave % a.S, group = wave / a.S, groups = kFewWaves / a.S, all = n + (a.Is ? a.T : 0);
    for (int base = 0; base < all; base += a.cap) {
        const int end = min(base + a.cap, all);
        for (int k = group; k < na + (a.Is ? 1 : 0); k += groups) {
            // places [lo, hi) of expert k in this round (na: the shared expert)
            const int off = k < na ? wave_uniform(p.off[k]) : n, past = k < na ? wave_uniform(p.off[k + 1]) : all;
            const int lo = max(off, base), hi = min(past, end);
            if (lo >= hi) continue;
            float *dst = sums + (part * a.cap + lo - base) * C;
            if (k < na) {
                const int64_t row = (int64_t)wave_uniform(p.expert[k]) * a.H;
                const FewMatrix W{static_cast<const uint8_t *>(a.W2) + row * a.I * (MX ? 1 : 2), MX ? a.W2s + row * (a.I / 32) : nullptr,
                                  a.I};
                few_down_unit<MX, B>(a, W, h0, p.route + off, lo - off, hi - off, part, dst);
            } else {
                const FewMatrix W{reinterpret_cast<const uint8_t *>(a.S2), nullptr, a.Is};
                few_down_unit<false, B>(a, W, h0, nullptr, lo - off, hi - off, part, dst);
            }
        }
        __syncthreads();
        for (int i = t; i < (end - base) * C; i += kFewThreads) {
            float v = 0.f;
            for (int s = 0; s < a.S; ++s) v += sums[s * a.cap * C + i];
            y[base * C + i] = v;
        }
        __syncthreads();
    }
    for (int i = t; i < a.T * C; i += kFewThreads) {
        const int tok = i / C, h = i % C;
        float sum = 0.f;
        for (int j = 0; j < a.K; ++j) {
            const int at = p.place[tok * a.K + j];
            if (at >= 0) sum = fmaf(a.w[tok * a.K + j], y[at * C + h], sum);
        }
        if (a.Is) sum += y[(n + tok) * C + h];
        a.out[(int64_t)tok * a.H + h0 + h] = f2bf(sum);
    }
}

}  // namespace moe

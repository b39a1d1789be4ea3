// The products of the gated feed-forward block for a few rows (a decode step): bound by
// the reading of the weights.
//
// A workgroup makes 16 weight rows' products with every row of X: 8 gate rows and the 8
// up rows that belong to them, or 16 rows of W2.  Its four waves share K between them, 64 at a
// time in turn, so that together they read whole runs of a weight row.  Each wave has a
// ring of LDS stages to itself, filled by buffer loads with the lds bit
// (128-byte lines of 8 rows to a load) and waited for by count: no wave waits for
// another until the sums of all are added, in ascending order, for the epilogue.
// v_mfma_f32_16x16x32: the weights are the 16 rows, X's rows the columns.
//
// H = 7168, I = 2048, weights from memory: 8 rows 12.4 + 9.3 us (4.7 and 3.2 TB/s, of which
// some 3.4 us of each launch pass before the first bytes are there), 64 rows 22.9 + 15.2, where each
// workgroup's reading of X from L2 is four times that of its weights.  Eight waves a workgroup, where
// there are no more workgroups than CUs, took 13.1 for 12.4, and H = 2048, I = 1024 5.9 for 5.2.
#pragma once

#include "dense.hpp"
#include "ffn.hpp"

namespace moe {

constexpr int kSkinnyWaves = 4;
// Stages of a wave's ring: as deep as leaves room for two workgroups on a CU (four stages of 17 to 32 rows 12.2 us in the
// down product for 10.2, of 33 to 64 rows 17.7 for 15.2).
constexpr int skinny_depth(int NT) { return NT == 1 ? 4 : NT == 2 ? 3 : 2; }
constexpr int skinny_stage_bytes(int NT) { return 2048 * (1 + NT); }
// dynamic LDS: the waves' rings, over which the sums go at the end
constexpr int skinny_lds(int NT) { return kSkinnyWaves * skinny_depth(NT) * skinny_stage_bytes(NT); }

struct SkinnyArgs {
    const uint16_t *X, *W;
    int64_t ldx, ldw;
    int M, N, K;       // rows of X; GLU: columns of a (W has 2 N rows), otherwise rows of W
    uint16_t *out;     // [M][ldo]
    int64_t ldo;
    uint16_t *HU;      // GLU: [M][2 N], nullable
    int act;
};

// 16 NT rows of X at most.
template <class T, int NT, bool GLU>
__device__ __forceinline__ void skinny_body(const SkinnyArgs &g, uint32_t lds) {
    constexpr int NW = kSkinnyWaves, DEPTH = skinny_depth(NT), ND = 2 + 2 * NT, STAGE = skinny_stage_bytes(NT), COLS = GLU ? 8 : 16;
    typedef typename T::v8 v8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * COLS;
    // a block of 8 rows: as LoadK
    uint32_t woff[2], xoff[4], wkc[2], xkc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int span = i * 4 + (lane >> 4), slot = (lane & 15) ^ (span & 15);
        const uint32_t r = (lane >> 4) * 2 + (slot >> 3), kc = (slot & 7) * 8;
        if (i < 2) woff[i] = r * (uint32_t)(2 * g.ldw) + kc * 2, wkc[i] = kc;
        xoff[i] = r * (uint32_t)(2 * g.ldx) + kc * 2, xkc[i] = kc;
    }
    const uint32_t xblock = (uint32_t)(16 * g.ldx), xbytes = (uint32_t)(2 * g.ldx) * (uint32_t)g.M;
    const uint32_t wblock = GLU ? 0 : (uint32_t)(16 * g.ldw), wbytes = (uint32_t)(2 * g.ldw) * (uint32_t)(GLU ? 8 : min(16, g.N - n0));
    const uint16_t *w0 = g.W + (int64_t)n0 * g.ldw, *w1 = GLU ? w0 + (int64_t)g.N * g.ldw : w0;
    const int steps = (g.K + kDenseK - 1) / kDenseK, left = g.K - (steps - 1) * kDenseK;
    const uint32_t ring = lds + wave * (DEPTH * STAGE);
    auto fill = [&](int step, uint32_t st) {
        const bool in = step < steps;
        if (step == steps - 1 && left < kDenseK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < 2 && (int)wkc[i] >= left) woff[i] = kPastEnd;
                if ((int)xkc[i] >= left) xoff[i] = kPastEnd;
            }
        }
        const uint32_t so = in ? (uint32_t)step * (kDenseK * 2) : 0u;
        const u32x4 r0 = dense_rsrc(w0, in ? wbytes : 0u), r1 = dense_rsrc(w1, in ? wbytes : 0u), rx = dense_rsrc(g.X, in ? xbytes : 0u);
        dense_dma(r0, st, woff[0] + so);
        dense_dma(r1, st + 1024, woff[1] + (so + wblock));
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) dense_dma(rx, st + 2048 + i * 1024, xoff[i & 3] + (so + i * xblock));
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fill(wave + d * NW, ring + d * STAGE);
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // lane l: row l % 16 of a block of 16, k 8 (l / 16) ... of 32
    const int row = lane & 15, span = row >> 1;
    const uint32_t at = span * 256;
    auto frag = [&](uint32_t tile, int blk, int s) {
        // windows go on counting from one block of 16 rows to the next
        const int slot = ((row & 1) * 8 | ((lane >> 4) + 4 * s)) ^ ((blk * 8 + span) & 15);
        return *(const __attribute__((address_space(3))) v8 *)(uintptr_t)(tile + blk * 2048 + at + slot * 16);
    };
    uint32_t slot = 0;
#pragma unroll 1
    for (int step = wave; step < steps; step += NW) {
        const uint32_t st = ring + slot * STAGE;
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((DEPTH - 1) * ND) : "memory");
        v8 w[2], x[2][NT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            w[s] = frag(st, 0, s);
#pragma unroll
            for (int t = 0; t < NT; ++t) x[s][t] = frag(st + 2048, t, s);
        }
        // the stage is in registers before it is filled again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        fill(step + DEPTH * NW, st);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = T::mfma16(w[s], x[s][t], acc[t]);
    }
    wait_loads_and_meet<0>();
    // [wave][16 weight rows][16 NT rows of X]
    typedef __attribute__((address_space(3))) float lds_float;
    lds_float *sum = (lds_float *)(uintptr_t)lds;
    constexpr int PLANE = 16 * 16 * NT;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[wave * PLANE + ((lane >> 4) * 4 + e) * (16 * NT) + t * 16 + row] = acc[t][e];
    __syncthreads();
    auto total = [&](int r, int m) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += sum[w * PLANE + r * (16 * NT) + m];
        return s;
    };
    for (int i = threadIdx.x; i < g.M * COLS; i += 64 * NW) {
        const int m = i / COLS, c = i % COLS;
        if (n0 + c >= g.N) continue;
        if constexpr (GLU) {
            const float h = total(c, m), u = total(8 + c, m);
            g.out[m * g.ldo + n0 + c] = T::down(activation1(g.act, h) * u);
            if (g.HU) {
                g.HU[(int64_t)m * 2 * g.N + n0 + c] = T::down(h);
                g.HU[(int64_t)m * 2 * g.N + g.N + n0 + c] = T::down(u);
            }
        } else {
            g.out[m * g.ldo + n0 + c] = T::down(total(c, m));
        }
    }
}

}  // namespace moe

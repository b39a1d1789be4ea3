// The whole expert layer for a few tokens, in two launches.
//
//   gate/up  a_r = silu(x_t Wg[e]^T) * (x_t Wu[e]^T) for every local route
//            r = (t, j), e its expert            -> act (bf16, one rounding)
//   down     out_t = sum_j w_tj (a_r W2[e]^T) (+ the shared expert's output),
//            ascending j, in fp32                -> out (bf16, one rounding)
//
// With a few routes per expert both products read each weight once and use it
// for at most a few dozen columns, so the time is the weights' HBM read: the
// MFMAs of a CU could take 1 KiB of weights every 4 cycles for 8 routes, some 20
// times the rate at which its share of HBM delivers them.  Everything here is
// laid out for that read:
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
//
// The activations' rounding to bf16 is the layer forward's own (and one of two
// roundings: the experts' sums stay fp32 to the output).  Keeping them as a high
// and a low bf16, which halves the output's error variance, doubles the down
// launch's token loads: 41.5 us against 39 for 8 tokens of the full-size share, 264
// against 241 for 128, 61 against 47 for 37 tokens of 64 experts, and 118 against 61
// for 32 tokens with MXFP8 weights (30 against 16 for 4).
//
// Measured (launches alone, rates of the weights of the experts that are hit; a
// read-only kernel gets 7.1 TB/s; each launch spends about 5 us before its stream
// flows and after it ends):
//   full-size share (H = 7168, I = 2048, 48 local experts, top-8 of 384)
//     8 tokens, 7 experts         gate/up 64 us (6.4 TB/s)   down 35 us (5.8 TB/s)
//     128 tokens, 46 and shared   gate/up 427 us (6.5 TB/s)  down 245 us (5.6 TB/s)
//     32 tokens, MXFP8, 17        gate/up 86 us (6.0 TB/s)   down 53 us (4.9 TB/s)
//   H = 2048, I = 1024, 37 tokens, 64 experts and the shared one
//                                 gate/up 93 us (5.8 TB/s)   down 48 us (5.7 TB/s)
#pragma once

#include "buffer.hpp"
#include "common.hpp"
#include "gemm.hpp"

namespace moe {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;
constexpr int kFewMaxRoutes = 1024;  // routes of one call (P * Np * K)
constexpr int kFewRows = 16;         // activation columns of a gate/up unit
constexpr int kFewGateupRegs = 200;  // registers for a wave's sums and steps in flight
// Down launch, B blocks of 8 output columns a workgroup: its waves, and the
// registers as above.  Two workgroups of four waves per CU with twice the loads
// in flight beat two of eight at 16 columns (MX down of 24 experts: 62 us against
// 100); at 8 columns there is one workgroup per CU, which takes eight waves (48 us
// against 62 for 64 experts of H = 2048, I = 1024).
constexpr int few_down_waves(int B) { return B == 1 ? 8 : 4; }
constexpr int few_down_threads(int B) { return 64 * few_down_waves(B); }
constexpr int few_down_regs(int B) { return B == 1 ? 72 : 104; }

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
    int words;                              // down: words of LDS for sums
};

// The list of a call's local routes grouped by expert, in the workspace
// (written by the gate/up launch's first workgroup, read by the down launch).
//   [0] ids outside [0, E)  [1] experts with a route (A)  [2] local routes (n)
//   [3], [4] of the A experts, how many have over 16 and over 8 routes
//   [kFewHead ...]       A expert ids, then A + 1 offsets
//   then n route numbers in expert order, then the place of each route (-1)
// The experts stand by their number of routes: over 16, 9 to 16, up to 8, by id
// within each kind.
constexpr int kFewHead = 64;
__host__ __device__ constexpr int few_max_experts(int L, int R) { return L < R ? L : R; }
__host__ __device__ constexpr int few_plan_words(int L, int R) { return kFewHead + 2 * few_max_experts(L, R) + 1 + 2 * R; }

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
// expert, 8 words for the head, and the list.
constexpr int kFewRedLd = 36;  // 32 sums of a column and 4 words that spread the columns over the banks
constexpr int kFewRedWords = kFewWaves * 32 * kFewRedLd;
__host__ __device__ constexpr int few_gateup_words(int L, int R) {
    return kFewRedWords + L + 8 + few_plan_words(L, R) - kFewHead;
}
// The list in the down launch's LDS: numbers of routes and places in 16 bits.
__host__ __device__ constexpr int few_list_words(int L, int R) { return 2 * few_max_experts(L, R) + 1 + R; }

// LDS words of the down launch for `rows` places of C columns and their parts' sums,
// one of each place for each wave, up to 32 KiB of parts, within `half` words beside the
// list where the places alone fit that (a call's routes are rarely all local: the parts
// then have the rows' unused space).
__host__ __device__ constexpr int few_sum_words(int rows, int C, int waves, int half) {
    const int sums = rows * C, parts = sums * waves < 8192 ? sums * waves : 8192;
    return (sums + parts <= half ? sums + parts : sums > half ? sums : half) / 4 * 4;
}
// The parts, of S that are wanted, for n places whose parts' sums have `room` places: every
// part of a round needs 16 places, or all of them.  A round reads the weights of its experts
// again: 1,000 routes of two experts of H = 7168, I = 2048 with a shared one took 985 us of 512
// tokens and 1,284 of 1,024 (MXFP8 1,108 and 1,410) in rounds of 12 places, and 846 and 1,213
// (854 and 1,220) with half the parts or one; with more places parts win (900 routes of 1,024
// tokens: 727 us with four parts and rounds of 31, 855 with two, 1,210 with one).
__host__ __device__ constexpr int few_fit_parts(int S, int n, int room) {
    while (S > 1 && room < (n < 16 ? n : 16) * S) S /= 2;
    return S;
}
constexpr bool few_small_calls_keep_their_parts() {
    for (int B = 1; B <= 2; ++B)
        for (int shared = 0; shared <= 1; ++shared)
            for (int K = 1; K <= 64; ++K)  // one token, any number of its slots local
                for (int n = 1; n <= K; ++n) {
                    const int C = 8 * B, S = few_down_waves(B), room = few_sum_words(K + shared, C, S, 16384) / C - n - shared;
                    if (few_fit_parts(S, n, room) != S || few_fit_parts(S, 1, room) != S) return false;
                    if (room / S < n) return false;  // in one round
                }
    return true;
}

// Builds the list in LDS: count the routes of each expert (a route's rank is
// the order in which the LDS atomics answer: it only says which MFMA column
// computes the route, and columns are independent), take the experts of each
// kind in ascending order and their offsets, place the routes.
// Returns A; head[0..4] as in the plan.
__device__ __forceinline__ int few_build(const FewArgs &a, int *cnt, const FewPlan &p, int *head) {
    const int t = threadIdx.x;
    constexpr int kPer = kFewMaxRoutes / kFewThreads;
    int lid[kPer], rank[kPer], bad = 0;
    for (int i = t; i < a.L; i += kFewThreads) cnt[i] = 0;
    if (t < 5) head[t] = 0;
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
        for (int kind = 0; kind < 3; ++kind) {
            const int least = kind == 0 ? 17 : kind == 1 ? 9 : 1, most = kind == 0 ? kFewMaxRoutes : kind == 1 ? 16 : 8;
            for (int l0 = 0; l0 < a.L; l0 += kWave) {
                const int l = l0 + t, all = l < a.L ? cnt[l] : 0;
                // an expert already placed holds -1 - its offset
                const int c = all >= least && all <= most ? all : 0;
                const uint64_t some = ballot(c > 0);
                if (!some) continue;
                int incl = c;
#pragma unroll
                for (int o = 1; o < kWave; o <<= 1) {
                    const int v = __shfl_up(incl, o, kWave);
                    if (t >= o) incl += v;
                }
                if (c > 0) {
                    const int k = na + lanes_below(some);
                    p.expert[k] = l;
                    p.off[k] = n + incl - c;
                    cnt[l] = -1 - (n + incl - c);
                }
                na += __popcll(some);
                n += __shfl(incl, kWave - 1, kWave);
            }
            if (t == 0 && kind < 2) head[3 + kind] = na;
        }
        if (t == 0) p.off[na] = n, head[1] = na, head[2] = n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = t + i * kFewThreads;
        if (r < a.R) {
            const int at = lid[i] >= 0 ? -1 - cnt[lid[i]] + rank[i] : -1;
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

// A step takes 128 consecutive bytes (64 bf16 elements or 128 codes of the
// reduction dimension) of each of a block's 8 weight rows, in one load: the
// MFMA's lane i + 16 g (row or column i, group g of its operand) reads 16-byte
// group 4 (i & 1) + g of row i / 2, and a tile is 8 tokens laid out alike.  MFMA
// row (r, p) times column (c, q) is then row r half p times token c half q: the
// wanted sum is the p = q entries of both halves, the other half of the products
// is dropped.  That costs nothing while the matrix cores wait for HBM, and whole
// 128-byte lines per load are worth it: a kernel that only reads gets 7.1 TB/s
// with 128 (or 256) bytes of a row per load and 5.5 TB/s with the 64 of a plain
// 16-row operand, and 64 tokens of 8 experts (H = 7168, I = 2048) took 179 + 161 us
// with plain operands against 130 + 107 us.
template <bool MX>
struct FewLane {
    static constexpr int kTokens = 8;                   // tokens of a tile
    static constexpr int kRows = 8;                     // rows of a block
    static constexpr int kStep = MX ? 128 : 64;         // elements of the reduction dimension per step
    static constexpr int kGroup = MX ? 16 : 8;          // elements of a group
    int row, group, token;                              // of the block; of the 128 bytes; of the tile
    __device__ __forceinline__ FewLane() {
        const int lane = lane_id(), i = lane & 15, g = lane >> 4;
        row = token = i / 2;
        group = 4 * (i & 1) + g;
    }
};

// A weight matrix of an expert: rows of `cols` elements, bf16 or MX (codes p,
// scale bytes s; the array that holds them ends at s_end).
struct FewMatrix {
    const uint8_t *p, *s, *s_end;
    int cols;
};

constexpr uint32_t kFewBytes = 0x7fffffffu;  // the host keeps every offset below; a buffer of 0 bytes reads as zeros

// Where an item's operands start: its M blocks of weight rows, G runs of
// consecutive blocks each from wp[.] / ws[.] (wave-uniform) on, and this lane's
// token of each tile (bytes from the tokens' matrix).
template <int G, int NT>
struct FewItem {
    const uint8_t *wp[G], *ws[G];
    uint32_t s_bytes[G];  // from ws[.] to the end of the scale bytes
    uint32_t xo[NT];
    template <bool MX>
    __device__ __forceinline__ void rows(int g, const FewMatrix &W, int64_t row) {
        wp[g] = W.p + row * W.cols * (MX ? 1 : 2);
        if constexpr (MX) {
            ws[g] = W.s + row * (W.cols / 32);
            s_bytes[g] = (uint32_t)min(W.s_end - ws[g], (ptrdiff_t)kFewBytes);
        }
    }
};

// What the steps of a run of items share: the tokens' matrix, bytes of a weight
// row and of its scale bytes, and this lane's bytes from a block's first row.
struct FewRun {
    const void *tokens;
    uint32_t row, srow, wo, so;
    template <bool MX>
    __device__ __forceinline__ static FewRun make(const FewLane<MX> &l, int cols, const void *tokens) {
        const uint32_t row = (uint32_t)cols * (MX ? 1 : 2), srow = (uint32_t)cols / 32;
        return {tokens, row, srow, l.row * row + l.group * 16, l.row * srow};
    }
};

// One step's operands: M blocks of weight rows and NT tiles of tokens.  With MX
// a load's 16 codes take two MFMAs, the first for each group's first 8 codes;
// both operands use the same order, so the sum is over the same elements.  OWN:
// the step loads its own scale bytes (MX; otherwise they come from FewScales).
template <bool MX, int M, int G, int NT, bool OWN>
struct FewStep {
    using L = FewLane<MX>;
    static constexpr int X = MX ? 2 : 1;  // 16-byte loads of 8 elements of a token's group
    u32x4 w[M];
    uint32_t sb[OWN ? M : 1];
    u32x4 x[NT][X];

    // step k's loads; all out of range unless `in` (which is wave-uniform)
    __device__ __forceinline__ void load(const FewRun &r, const FewItem<G, NT> &it, int k, bool in) {
        constexpr int per = M / G;
        if (!in) k = 0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            w[m] = buffer_load16_nt(raw_buffer(it.wp[m / per], in ? kFewBytes : 0), r.wo, in ? (m % per) * L::kRows * r.row + k * 128 : 0);
            if constexpr (OWN)
                sb[m] = __builtin_amdgcn_raw_buffer_load_b32(raw_buffer(it.ws[m / per], in ? it.s_bytes[m / per] : 0), r.so,
                                                             in ? (m % per) * L::kRows * r.srow + k * 4 : 0, 0);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < X; ++e)
                x[t][e] = buffer_load16(raw_buffer(r.tokens, in ? kFewBytes : 0), it.xo[t] + e * 16, k * (L::kStep * 2));
    }
    // scale(m): block m's four scale bytes of this step
    template <class Scale>
    __device__ __forceinline__ void mul(const L &l, Scale scale, f32x4 (&acc)[M][NT]) const {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            bf16x8 f[2];
            if constexpr (MX)
                few_mx_frags(w[m], (scale(m) >> (8 * (l.group >> 1))) & 0xffu, f[0], f[1]);
            else
                f[0] = __builtin_bit_cast(bf16x8, w[m]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < X; ++e)
                    acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[e], __builtin_bit_cast(bf16x8, x[t][e]), acc[m][t], 0,
                                                                        0, 0);
        }
    }
};

// The scale bytes of four steps (512 codes) in one load per block: a load of
// one step's four bytes per row costs as much address work as 128 bytes of the
// row's codes (gate/up of 24 experts took 124 us with one such load per step
// and block, 103 us without any).  A chunk may reach past its row, into bytes
// that no step uses, but not past the array: the buffer's size ends there.
template <int M, int G>
struct FewScales {
    u32x4 v[M];
    template <int NT>
    __device__ __forceinline__ void load(const FewRun &r, const FewItem<G, NT> &it, int k, bool in) {
        constexpr int per = M / G;
#pragma unroll
        for (int m = 0; m < M; ++m)
            v[m] = buffer_load16(raw_buffer(it.ws[m / per], in ? it.s_bytes[m / per] : 0), r.so,
                              in ? (m % per) * 8 * r.srow + k * 4 : 0);
    }
};

// Steps in flight that fit `regs` registers beside the sums; with MX four and
// the scale bytes of four steps where that fits.
template <bool MX, int M, int NT>
constexpr int few_step_regs() {
    return 4 * (M + (MX ? 2 : 1) * NT);
}
template <bool MX, int M, int NT>
constexpr bool few_chunked(int regs) {
    return MX && 4 * few_step_regs<MX, M, NT>() + 8 * M + 4 * M * NT <= regs;
}
template <bool MX, int M, int NT>
constexpr int few_depth(int regs) {
    if (few_chunked<MX, M, NT>(regs)) return 4;
    const int d = (regs - 4 * M * NT) / (few_step_regs<MX, M, NT>() + (MX ? M : 0));
    return d < 1 ? 1 : d > 8 ? 8 : d;
}

// Streams `items` products through one wave: for each, block m's rows times
// tile t's tokens over the steps [k0, k0 + n) of the reduction dimension go to
// emit(item, acc).  item(i) gives the operands' places.  D steps are in flight:
// a step's registers are loaded again as soon as they are used, the last ones of
// an item with the first steps of the next, so the wave's loads never run dry
// between items.  The scheduling barriers keep the loads where they are written:
// left alone, the compiler moves them next to their use.
//
// The compiler counts the loads in flight to wait for no more than a step needs,
// and loses count behind a branch around a load: it then waits for all D steps
// once every D.  EVEN has no such branch: every turn issues the same loads, those
// of steps that do not exist from an empty buffer.  That pays where a workgroup
// has a CU for itself and its waves never meet (down, 8 columns: 59 us to 47 for
// 64 experts of H = 2048, I = 1024) and not where few steps make many of the
// loads empty (gate/up of the same: 90 us to 100).
template <bool MX, int M, int G, int NT, int REGS, bool EVEN, class Item, class Emit>
__device__ __forceinline__ void few_stream(const FewLane<MX> &l, const FewRun &r, int k0, int n, int items, Item item, Emit emit) {
    if (items <= 0) return;
    constexpr bool chunks = few_chunked<MX, M, NT>(REGS), own = MX && !chunks;  // scale bytes: of four steps, of one
    constexpr int D = few_depth<MX, M, NT>(REGS);
    FewStep<MX, M, G, NT, own> st[D];
    FewScales<chunks ? M : G, G> now, then;
    FewItem<G, NT> cur, next;
    f32x4 acc[M][NT];
    auto mul = [&](int j) {
        st[j].mul(
            l,
            [&](int m) -> uint32_t {
                if constexpr (chunks) return now.v[m][j & 3];
                return st[j].sb[own ? m : 0];
            },
            acc);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto load = [&](int j, const FewItem<G, NT> &it, int step, bool in) {
        st[j].load(r, it, k0 + step, in);
        if constexpr (chunks)
            if (j == 0) then.load(r, it, k0 + step, in);
        __builtin_amdgcn_sched_barrier(0);
    };
    item(0, cur);
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (EVEN || j < n) load(j, cur, j, !EVEN || j < n);
    now = then;
    for (int it = 0; it < items; ++it) {
        const bool more = it + 1 < items;
        if (more) item(it + 1, next);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (EVEN) {
            const int turns = max(1, (n + D - 1) / D);
            for (int c = 0; c < turns; ++c) {
                const bool last = c + 1 == turns;
                if (last) cur = next;
                const int base = last ? 0 : (c + 1) * D, steps = last && !more ? 0 : n;
#pragma unroll
                for (int j = 0; j < D; ++j) {
                    if (c * D + j < n) mul(j);
                    load(j, cur, base + j, base + j < steps);
                }
                now = then;
            }
        } else {
            int k = 0;
            for (; k + 2 * D <= n; k += D) {
#pragma unroll
                for (int j = 0; j < D; ++j) {
                    mul(j);
                    load(j, cur, k + D + j, true);
                }
                now = then;
            }
            // fewer than 2 D steps are left, the first D of them in flight
#pragma unroll
            for (int j = 0; j < D; ++j)
                if (k + j < n) {
                    mul(j);
                    if (k + D + j < n)
                        load(j, cur, k + D + j, true);
                    else if (more)
                        load(j, next, j, true);
                }
            now = then;
            if (k + D < n) {
#pragma unroll
                for (int j = 0; j < D; ++j)
                    if (k + D + j < n) {
                        mul(j);
                        if (more) load(j, next, j, true);
                    }
                now = then;
            }
            cur = next;
        }
        emit(it, acc);
    }
}

// A block's and tile's sums: both halves' entries meet (lane ^ 1), then the even
// lane has row 2 g of the block and the odd lane row 2 g + 1, for the lane's token.
__device__ __forceinline__ int few_sum_row() { return 2 * (lane_id() >> 4) + (lane_id() & 1); }
__device__ __forceinline__ float few_sum(const f32x4 &acc) {
    const bool odd = lane_id() & 1;
    const float a = odd ? acc[1] : acc[0], b = odd ? acc[3] : acc[2];
    const float sa = a + __shfl_xor(a, 1, kWave), sb = b + __shfl_xor(b, 1, kWave);
    return odd ? sb : sa;
}

__device__ __forceinline__ int wave_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A unit of the gate/up launch: activation columns [i0, i0 + 4 M) of one expert
// (W, with `inner` activation columns) for its `n` routes.  The routes' tokens
// are route[..] / K, their activations go to row route[..] of act; route null:
// the tokens themselves (shared expert), rows R + token.
struct FewUnit {
    FewMatrix W;
    int inner, i0, n;
    const int *route;
};

__device__ __forceinline__ int few_token(const FewArgs &a, const int *route, int k) { return route ? route[k] / a.K : k; }
template <class T>
__device__ __forceinline__ int few_act_row(const FewArgs &a, const T *route, int k) { return route ? (int)route[k] : a.R + k; }

// Operands of a unit's routes from `first` on: M / 2 blocks of gate rows, M / 2 of
// up rows.
template <bool MX, int NT>
__device__ __forceinline__ void few_gateup_item(const FewArgs &a, const FewUnit &u, int first, const FewLane<MX> &l,
                                                FewItem<2, NT> &it) {
    using L = FewLane<MX>;
#pragma unroll
    for (int g = 0; g < 2; ++g) it.template rows<MX>(g, u.W, (int64_t)g * u.inner + u.i0);
#pragma unroll
    for (int q = 0; q < NT; ++q)
        it.xo[q] = (uint32_t)few_token(a, u.route, min(first + q * L::kTokens + l.token, u.n - 1)) * (uint32_t)(a.H * 2) +
                   l.group * (L::kGroup * 2);
}

// The waves' sums of a unit meet in LDS (red), 32 tokens at a time, and are
// added in wave order; then the activation, rounded once.
template <bool MX, int M, int NT>
__device__ __forceinline__ void few_gateup_join(const FewArgs &a, const FewUnit &u, int first, const FewLane<MX> &l,
                                                const f32x4 (&acc)[M][NT], float *red) {
    using L = FewLane<MX>;
    constexpr int per = 32 / L::kTokens;  // tiles that meet at a time
    const int t = threadIdx.x, wave = t >> 6;
#pragma unroll
    for (int q0 = 0; q0 < NT; q0 += per) {
        __syncthreads();  // the previous sums have been read
#pragma unroll
        for (int q = q0; q < (q0 + per < NT ? q0 + per : NT); ++q) {
            float *dst = red + (wave * 32 + (q - q0) * L::kTokens + l.token) * kFewRedLd + few_sum_row();
#pragma unroll
            for (int m = 0; m < M; ++m) dst[(m < M / 2 ? 0 : 16) + m % (M / 2) * L::kRows] = few_sum(acc[m][q]);
        }
        __syncthreads();
        const int tok = t >> 4, i = t & 15, k = first + q0 * L::kTokens + tok;
        if (i < 4 * M && tok < (NT - q0) * L::kTokens && k < u.n) {
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) {
                const float *src = red + (v * 32 + tok) * kFewRedLd + i;
                gate += src[0];
                up += src[16];
            }
            a.act[(int64_t)few_act_row(a, u.route, k) * a.ld + u.i0 + i] = f2bf(gate / (1.0f + __expf(-gate)) * up);
        }
    }
}

// `count` units (unit(i) for i in turn), all with at most NT tiles of routes
// from `first` on, the waves splitting H.
template <bool MX, int M, int NT, class Unit>
__device__ __forceinline__ void few_gateup_run(const FewArgs &a, int count, int first, Unit unit, float *red) {
    using L = FewLane<MX>;
    const L l;
    const int wave = wave_uniform(threadIdx.x >> 6), steps = a.H / L::kStep;
    const int k0 = wave * steps / kFewWaves, n = (wave + 1) * steps / kFewWaves - k0;
    few_stream<MX, M, 2, NT, kFewGateupRegs, false>(
        l, FewRun::make(l, a.H, a.X), k0, n, count, [&](int i, FewItem<2, NT> &it) { few_gateup_item<MX, NT>(a, unit(i), first, l, it); },
        [&](int i, const f32x4(&acc)[M][NT]) { few_gateup_join<MX, M, NT>(a, unit(i), first, l, acc, red); });
}

// The routes [first, min(n, first + 64)) of a unit.
template <bool MX>
__device__ __forceinline__ void few_gateup_pass(const FewArgs &a, const FewUnit &u, int first, float *red) {
    const int left = u.n - first;
    if (left <= 16)
        few_gateup_run<MX, 4, 2>(a, 1, first, [&](int) { return u; }, red);
    else if (left <= 32)
        few_gateup_run<MX, 4, 4>(a, 1, first, [&](int) { return u; }, red);
    else
        few_gateup_run<MX, 4, 8>(a, 1, first, [&](int) { return u; }, red);
}

// Persistent over the units in order, every workgroup taking each gridDim.x-th
// one (runs of neighbours instead read 256 far-apart places at a time: 520 us
// against 433 for 43 experts): the shared expert's blocks, 64 tokens at a time,
// the experts with over 16 routes, then in two streams those with up to 16 and
// up to 8.
template <bool MX>
__device__ __forceinline__ void few_gateup_body(const FewArgs &a, int *lds) {
    float *red = reinterpret_cast<float *>(lds);
    int *cnt = lds + kFewRedWords, *head = cnt + a.L;
    const FewPlan p(head + 8, a.L, a.R);
    const int na = wave_uniform(few_build(a, cnt, p, head));
    if (blockIdx.x == 0) {
        const FewPlan o(a.plan + kFewHead, a.L, a.R);
        if (threadIdx.x < 5) a.plan[threadIdx.x] = head[threadIdx.x];
        for (int i = threadIdx.x; i <= na; i += kFewThreads) {
            if (i < na) o.expert[i] = p.expert[i];
            o.off[i] = p.off[i];
        }
        for (int i = threadIdx.x; i < a.R; i += kFewThreads) {
            if (i < head[2]) o.route[i] = p.route[i];
            o.place[i] = p.place[i];
        }
    }
    const int blocks = a.I / kFewRows, sblocks = a.Is / kFewRows, shared = sblocks * ((a.T + 63) / 64), step = gridDim.x;
    const int wide = wave_uniform(head[3]) * blocks, mid = wave_uniform(head[4]) * blocks, all = na * blocks;
    int u = blockIdx.x;
    for (; u < shared; u += step) {
        const FewUnit s{{reinterpret_cast<const uint8_t *>(a.S13), nullptr, nullptr, a.H}, a.Is, u % sblocks * kFewRows, a.T, nullptr};
        if (a.T <= 8)
            few_gateup_run<false, 4, 1>(a, 1, 0, [&](int) { return s; }, red);
        else
            few_gateup_pass<false>(a, s, u / sblocks * 64, red);
    }
    auto routed = [&](int v) {  // unit v of the experts in the list's order
        const int k = v / blocks, off = wave_uniform(p.off[k]);
        const int64_t row = (int64_t)wave_uniform(p.expert[k]) * 2 * a.I;
        return FewUnit{{static_cast<const uint8_t *>(a.W13) + row * a.H * (MX ? 1 : 2), MX ? a.W13s + row * (a.H / 32) : nullptr,
                        MX ? a.W13s + (int64_t)a.L * 2 * a.I * (a.H / 32) : nullptr, a.H},
                       a.I, v % blocks * kFewRows, wave_uniform(p.off[k + 1]) - off, p.route + off};
    };
    for (u -= shared; u < wide; u += step) {
        const FewUnit r = routed(u);
        for (int first = 0; first < r.n; first += 64) few_gateup_pass<MX>(a, r, first, red);
    }
    const int nmid = u < mid ? (mid - u + step - 1) / step : 0;
    few_gateup_run<MX, 4, 2>(a, nmid, 0, [&](int i) { return routed(u + i * step); }, red);
    u += nmid * step;
    if (all - mid + shared >= 2 * step) {
        const int nlow = u < all ? (all - u + step - 1) / step : 0;
        few_gateup_run<MX, 4, 1>(a, nlow, 0, [&](int i) { return routed(u + i * step); }, red);
    } else {
        // fewer than two a workgroup: half as wide, so that every workgroup has its share (a token with one
        // local expert of the full-size share: the call takes 24.0 us, from 26.5; seven experts, 3.5 units a
        // workgroup, lose: 66 to 68 us)
        const int half = 2 * (all - mid), from = ((int)blockIdx.x + step - (2 * mid + shared) % step) % step;
        const int nlow = from < half ? (half - from + step - 1) / step : 0;
        few_gateup_run<MX, 2, 1>(
            a, nlow, 0,
            [&](int i) {
                const int v = from + i * step;
                FewUnit r = routed(mid + v / 2);
                r.i0 += v % 2 * 8;
                return r;
            },
            red);
    }
}

// Parts of a reduction dimension of `inner` elements, for n places: a power of two
// up to the waves, each part with at least 512 bytes of a row, or 2 KiB where the
// places are one tile or less: there the parts' join costs more than a shorter
// stream saves (down launch, one token, 4 experts and the shared one of H = 4096, I =
// 1024: 12.2 us with one part, 15.8 with four; 2 experts of H = 7168, I = 2048, MXFP8:
// 11.8 and 13.2, bf16 15.9 with one, 15.5 with two or four; one expert's 16 routes of H =
// 7168, I = 2048: 13.6 with one, 13.1 with four, its 64: 31.3 and 20.5).
template <bool MX>
__device__ __forceinline__ int few_parts(int inner, int n, int waves) {
    int S = waves;
    while (S > 1 && inner * (MX ? 1 : 2) < (n <= 8 ? 2048 : 512) * S) S /= 2;
    return S;
}

// An item of the down launch: output columns [h0, h0 + 8 B) of one expert for
// its routes [first, n), whose sums go to y[.. - first][8 B].
struct FewSlice {
    FewMatrix W;
    const uint16_t *route;
    int first, n;
    float *y;
};

// `count` items (slice(i) for i in turn) with at most NT tiles each, over part
// `part` of S of their activations: one wave, no barrier.
template <bool MX, int B, int NT, class Slice>
__device__ __forceinline__ void few_down_run(const FewArgs &a, int h0, int cols, int part, int S, int count, Slice slice) {
    using L = FewLane<MX>;
    const L l;
    const int steps = cols / L::kStep, k0 = part * steps / S, n = (part + 1) * steps / S - k0;
    few_stream<MX, B, 1, NT, few_down_regs(B), true>(
        l, FewRun::make(l, cols, a.act), k0, n, count,
        [&](int i, FewItem<1, NT> &it) {
            const FewSlice s = slice(i);
            it.template rows<MX>(0, s.W, h0);
#pragma unroll
            for (int q = 0; q < NT; ++q)
                it.xo[q] = (uint32_t)few_act_row(a, s.route, min(s.first + q * L::kTokens + l.token, s.n - 1)) * (uint32_t)(a.ld * 2) +
                           l.group * (L::kGroup * 2);
        },
        [&](int i, const f32x4(&acc)[B][NT]) {
            const FewSlice s = slice(i);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const int k = q * L::kTokens + l.token;
#pragma unroll
                for (int m = 0; m < B; ++m) {
                    const float v = few_sum(acc[m][q]);
                    if (s.first + k < s.n) s.y[k * 8 * B + m * L::kRows + few_sum_row()] = v;
                }
            }
        });
}

// An item with any number of routes: 64 at a time, 32 where the waves have
// fewer registers.
template <bool MX, int B>
__device__ __forceinline__ void few_down_wide(const FewArgs &a, int h0, int part, int S, FewSlice s) {
    constexpr int most = B == 1 ? 32 : 64;
    for (; s.first < s.n; s.first += most, s.y += most * 8 * B) {
        const int left = s.n - s.first;
        if (left <= 16)
            few_down_run<MX, B, 2>(a, h0, s.W.cols, part, S, 1, [&](int) { return s; });
        else if (B == 1 || left <= 32)
            few_down_run<MX, B, 4>(a, h0, s.W.cols, part, S, 1, [&](int) { return s; });
        else if constexpr (B > 1)
            few_down_run<MX, B, 8>(a, h0, s.W.cols, part, S, 1, [&](int) { return s; });
    }
}

// One workgroup per 8 B output columns.  Its waves form S parts of the
// reduction dimension times waves / S groups that take the experts in turn.
// One part is best (a wave then streams whole rows, and its sums go straight to
// y[place], the routes in expert order and the shared expert's tokens after
// them), as long as every wave gets at least four experts and none has over a
// sixteenth more than its share; otherwise as few parts as do.  Parts' sums meet
// in LDS, as many places a round as there is room for, and are added in part
// order into y.  At the end every output element adds its token's routes in
// ascending slot order, the shared expert last, and is rounded once.
template <bool MX, int B>
__device__ __forceinline__ void few_down_body(const FewArgs &a, int *lds) {
    constexpr int C = 8 * B, kWaves = few_down_waves(B), kThreads = few_down_threads(B);
    const int t = threadIdx.x, wave = wave_uniform(t >> 6), h0 = blockIdx.x * C;
    int *expert = lds + a.words, *offset = expert + few_max_experts(a.L, a.R);
    uint16_t *route = reinterpret_cast<uint16_t *>(offset + few_max_experts(a.L, a.R) + 1), *place = route + a.R;
    const FewPlan src(a.plan + kFewHead, a.L, a.R);
    // the whole list, entries past its counts too (never used), so that no load waits for the counts
    for (int i = t; i < 2 * few_max_experts(a.L, a.R) + 1; i += kThreads) expert[i] = src.expert[i];
    for (int i = t; i < 2 * a.R; i += kThreads) route[i] = (uint16_t)src.route[i];  // and the places: 65535 for none
    const int na = wave_uniform(a.plan[1]), n = wave_uniform(a.plan[2]), all = n + (a.Is ? a.T : 0);
    float *y = reinterpret_cast<float *>(lds), *sums = y + all * C;
    const int room = a.words / C - all;
    __syncthreads();
    auto join = [&](int base, int end, int S, int cap) {  // the sums of places [base, end)
        __syncthreads();
        for (int i = t; i < (end - base) * C; i += kThreads) {
            float v = 0.f;
            for (int s = 0; s < S; ++s) v += sums[s * cap * C + i];
            y[base * C + i] = v;
        }
        __syncthreads();
    };
    if (a.Is) {  // every token's column: all waves share it
        const int S = few_fit_parts(few_parts<false>(a.Is, a.T, kWaves), a.T, room);
        const int cap = S > 1 ? room / S : a.T;
        const FewMatrix W{reinterpret_cast<const uint8_t *>(a.S2), nullptr, nullptr, a.Is};
        for (int base = 0; base < a.T; base += cap) {
            const int end = min(base + cap, a.T);
            if (wave < S) {
                const FewSlice s{W, nullptr, base, end, S > 1 ? sums + wave * cap * C : y + n * C};
                if (end - base <= 8)
                    few_down_run<false, B, 1>(a, h0, a.Is, wave, S, 1, [&](int) { return s; });
                else
                    few_down_wide<false, B>(a, h0, wave, S, s);
            }
            if (S > 1) join(n + base, n + end, S, cap);
        }
    }
    const int most = few_parts<MX>(a.I, n, kWaves);
    int S = 1;
    while (S < most && (na * S < 4 * kWaves || 15 * ((na * S + kWaves - 1) / kWaves) * kWaves > 16 * na * S)) S *= 2;
    S = few_fit_parts(S, n, room);
    const int part = wave % S, group = wave / S, groups = kWaves / S, cap = S > 1 ? room / S : n;
    const int wide = wave_uniform(a.plan[3]), mid = wave_uniform(a.plan[4]);
    for (int base = 0, from = 0; base < n; base += cap) {
        // the experts [from, to) have places in [base, end); the first and the last may have others too
        const int end = min(base + cap, n);
        while (wave_uniform(offset[from + 1]) <= base) ++from;
        int to = na;
        if (end < n)
            for (to = from + 1; wave_uniform(offset[to]) < end;) ++to;
        auto slice = [&](int k) {
            const int off = wave_uniform(offset[k]), lo = max(off, base), hi = min(wave_uniform(offset[k + 1]), end);
            const int64_t row = (int64_t)wave_uniform(expert[k]) * a.H;
            return FewSlice{{static_cast<const uint8_t *>(a.W2) + row * a.I * (MX ? 1 : 2), MX ? a.W2s + row * (a.I / 32) : nullptr,
                             MX ? a.W2s + (int64_t)a.L * a.H * (a.I / 32) : nullptr, a.I},
                            route + off, lo - off, hi - off, S > 1 ? sums + (part * cap + lo - base) * C : y + lo * C};
        };
        int k = from + group;
        for (; k < min(wide, to); k += groups) few_down_wide<MX, B>(a, h0, part, S, slice(k));
        const int nmid = k < min(mid, to) ? (min(mid, to) - k + groups - 1) / groups : 0;
        few_down_run<MX, B, 2>(a, h0, a.I, part, S, nmid, [&](int i) { return slice(k + i * groups); });
        k += nmid * groups;
        const int nlow = k < to ? (to - k + groups - 1) / groups : 0;
        few_down_run<MX, B, 1>(a, h0, a.I, part, S, nlow, [&](int i) { return slice(k + i * groups); });
        if (S > 1) join(base, end, S, cap);
    }
    __syncthreads();
    for (int i = t; i < a.T * C; i += kThreads) {
        const int tok = i / C, h = i % C;
        float sum = 0.f;
        for (int j = 0; j < a.K; ++j) {
            const int at = place[tok * a.K + j];
            if (at != 0xffff) sum = fmaf(a.w[tok * a.K + j], y[at * C + h], sum);
        }
        if (a.Is) sum += y[(n + tok) * C + h];
        a.out[(int64_t)tok * a.H + h0 + h] = f2bf(sum);
    }
}

}  // namespace moe

// Dense 16-bit matrix products (bf16 or fp16 operands, fp32 accumulators) of any
// number of rows and columns: the products of the gated feed-forward block and of
// its gradient.
//
//   D[m][n] = sum_k A(m, k) B(n, k)
//
// Each operand lies either K-contiguous ([mn][k]) or MN-contiguous ([k][mn]), so no
// transposed copy is made for the gradient.  A workgroup of 4 waves (2 x 2) makes a
// tile of 64 MI x 64 NI outputs, each wave 32 MI x 32 NI of it in blocks of
// v_mfma_f32_32x32x16.  K steps of 64 go from memory to LDS by buffer loads with the
// lds bit, into a ring: of single operand tiles (dense_loop, large tiles) or of stages of
// both (dense_loop_deep, small ones).
//
// Edges cost the loop nothing.  Rows past the last one lie past the end of the raw
// buffer, which reads as zeros there; columns (of an MN-contiguous operand) and the
// k of the last step past K get an address past it.
//
// One wave per SIMD does not hide its own waits, so the loops do: the fragments of a
// 16-deep sub-step are read from LDS while the one before (in the deep loop, the two
// before) is multiplied, across the step's one barrier too, and the loads that fill the
// ring are spread over the MFMAs, one to four of them.
//
// Measured: 16,384 rows of H = 7168, I = 2048 forward 1,107 to 1,146 us, 1.30 to 1.26 PFLOP/s; the large tile's
// step takes 2,470 cycles of the 2,048 of its MFMAs, and 2,320 with no memory behind its
// loads.  The 128 x 128 tile reads its operands from LDS twice as often for its MFMAs: 900
// cycles a step of 512, bound by LDS.
//
// The loads are written as asm without outputs: known to the compiler as loads into
// LDS, each transposing LDS read would wait for all of them.  They are waited for by
// count (vector memory operations complete in order) before the barrier that
// publishes their stage; the compiler's own waits only become longer by them.
#pragma once

#include "buffer.hpp"
#include "common.hpp"

namespace moe {

struct Bf16 {
    static constexpr bool kNarrow = false;  // fp32 values may lie past its range
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) {
#if defined(__HIP_DEVICE_COMPILE__)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
#else
        return c;
#endif
    }
    static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
        return c;
#endif
    }
    static __device__ __forceinline__ uint16_t down(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
    static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
};
struct Fp16 {
    static constexpr bool kNarrow = true;
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x16 mfma(v8 a, v8 b, f32x16 c) {
#if defined(__HIP_DEVICE_COMPILE__)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
#else
        return c;
#endif
    }
    static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#else
        return c;
#endif
    }
    static __device__ __forceinline__ uint16_t down(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
    static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
};

struct F32 {};  // fp32 elements, where a call takes them too

template <class T>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (uint32_t)T::down(v[2 * i]) | (uint32_t)T::down(v[2 * i + 1]) << 16;
    return o;
}
template <class T>
__device__ __forceinline__ void unpack8(const u32x4 &p, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = T::up((uint16_t)p[i]), v[2 * i + 1] = T::up((uint16_t)(p[i] >> 16));
}

constexpr int kDenseThreads = 256;
constexpr int kDenseK = 64;          // k per step
constexpr uint32_t kPastEnd = 0x80000000u;  // a lane offset past every buffer's end

// 16 bytes per lane from a raw buffer to 1 KiB of LDS at byte address `lds`.  The whole
// offset is the lane's: the range check subtracts a wave-uniform one from the size,
// which must not go below zero.
__device__ __forceinline__ void dense_dma(u32x4 rsrc, uint32_t lds, uint32_t lane_off) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds), "v"(lane_off), "s"(rsrc));
#else
    (void)rsrc, (void)lds, (void)lane_off;
#endif
}
__device__ __forceinline__ u32x4 dense_rsrc(const void *base, uint32_t bytes) {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    return u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, bytes, 0x00020000u};
}

typedef __attribute__((address_space(3))) char lds_char;

// A K-contiguous operand's rows [0, valid) of a tile of R rows, row i at base + i ld.
// LDS: [R][64], rows of 128 bytes, two of them to a window of 256 bytes whose 16
// chunks of 16 bytes are permuted by XOR with the window's number: the 16 lanes of a
// ds_read_b128's phase, 16 rows at one k, then hit 16 different chunks of the window.
template <int R>
struct LoadK {
    static constexpr int BL = R / 8 / 4;  // 1 KiB blocks (8 rows) per wave and step
    static constexpr int P = BL < 4 ? BL : 4;
    const char *base;
    uint32_t bytes, block, first;  // bytes: of the valid rows; block: of 8 rows; first: this wave's first block's offset
    uint32_t off[P], kc[P];
    __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int valid, int wave, int lane, int row_blocks_before = 0) {
        base = reinterpret_cast<const char *>(p);
        block = (uint32_t)(16 * ld);
        first = (uint32_t)(wave * BL - row_blocks_before) * block;
        bytes = (uint32_t)(2 * ld) * (uint32_t)valid;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int span = ((wave * BL + i) & 3) * 4 + (lane >> 4), slot = (lane & 15) ^ (span & 15);
            kc[i] = (uint32_t)(slot & 7) * 8;
            off[i] = (uint32_t)((lane >> 4) * 2 + (slot >> 3)) * (uint32_t)(2 * ld) + kc[i] * 2;
        }
    }
    // the last step: k from `left` on read zeros
    __device__ __forceinline__ void cut(int left) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if ((int)kc[i] >= left) off[i] = kPastEnd;
    }
    __device__ __forceinline__ u32x4 stage(int64_t step, bool in) const { return dense_rsrc(base, in ? bytes : 0u); }
    __device__ __forceinline__ uint32_t step_off(int64_t step) const { return (uint32_t)(step * (kDenseK * 2)) + first; }
    __device__ __forceinline__ void load(const u32x4 &rsrc, uint32_t so, uint32_t lds, int wave, int i) const {
        dense_dma(rsrc, lds + (wave * BL + i) * 1024, off[i % P] + (so + i * block));
    }
};

// An MN-contiguous operand's columns [0, valid) of a tile of R columns, k row r at
// base + r ld.  LDS: [64][R], chunks of 16 bytes permuted so that the four k rows
// that 16 lanes of a transposing read take lie in four different quarters of a
// 256-byte window.
template <int R>
struct LoadMn {
    static constexpr int BL = R / 8 / 4, CPR = R / 8, RPB = 64 / CPR;  // blocks per wave; chunks per k row; k rows per block
    static constexpr int P = RPB < 4 ? 4 / RPB : 1;
    static_assert(BL % P == 0, "a wave's blocks start on a multiple of four k rows");
    const char *base;
    int64_t row;  // bytes
    int K;
    uint32_t off[P];
    static __device__ __forceinline__ int swz(int r) { return R == 64 ? 4 * ((r >> 1) & 1) : 4 * (r & 3); }
    __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int valid, int K_, int lane) {
        base = reinterpret_cast<const char *>(p);
        row = 2 * ld;
        K = K_;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int r = i * RPB + lane / CPR, c = (lane % CPR) ^ swz(r);
            off[i] = c * 8 < valid ? (uint32_t)(lane / CPR) * (uint32_t)row + c * 16 : kPastEnd;
        }
    }
    __device__ __forceinline__ void cut(int) {}
    __device__ __forceinline__ u32x4 stage(int64_t step, bool in) const {
        const int64_t left = K - step * kDenseK;
        return dense_rsrc(base + step * kDenseK * row, in ? (uint32_t)(left < kDenseK ? left : kDenseK) * (uint32_t)row : 0u);
    }
    __device__ __forceinline__ uint32_t step_off(int64_t) const { return 0; }
    __device__ __forceinline__ void load(const u32x4 &rsrc, uint32_t, uint32_t lds, int wave, int i) const {
        dense_dma(rsrc, lds + (wave * BL + i) * 1024, off[i % P] + (uint32_t)((wave * BL + i) * RPB) * (uint32_t)row);
    }
};

// Fragments: lane l of a block of 32 rows holds row l % 32, k 8 (l / 32) ... + 7 of the
// sub-step's 16.
template <class T, bool TR, int R>
struct Frags {
    typedef typename T::v8 v8;
    uint32_t at;  // K-contiguous: chunk of sub-step 0 in block 0; MN-contiguous: k row and columns of block 0
    __device__ __forceinline__ void init(int lane) {
        if constexpr (!TR) {
            const int row = lane & 31, span = row >> 1, slot = ((row & 1) * 8 | (lane >> 5)) ^ (span & 15);
            at = span * 256 + slot * 16;
        } else {
            const int g = (lane >> 4) & 1, q = lane & 15, j = q >> 2, cq = q & 3;
            at = (8 * (lane >> 5) + j) * (2 * R) + (((2 * g + (cq >> 1)) ^ LoadMn<R>::swz(j)) << 4) + (cq & 1) * 8;
        }
    }
    // block b (a wave's own first block included), sub-step s, of the tile at LDS address `tile`
    __device__ __forceinline__ v8 get(uint32_t tile, int b, int s) const {
        if constexpr (!TR) {
            return *(const __attribute__((address_space(3))) v8 *)(uintptr_t)(tile + b * 4096 + (at ^ (s << 5)));
        } else {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            struct Two {
                s16x4 lo, hi;
            };
            Two t{};
#if defined(__HIP_DEVICE_COMPILE__)
            const uint32_t p = tile + 16 * s * (2 * R) + (at ^ ((uint32_t)b << 6));
            t.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)p);
            t.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(p + 4 * (2 * R)));
#endif
            return __builtin_bit_cast(v8, t);
        }
    }
};

template <int MI, int NI>
using DenseAcc = f32x16[MI][NI];

template <bool TR, int R>
struct LoadOf {
    using type = LoadK<R>;
};
template <int R>
struct LoadOf<true, R> {
    using type = LoadMn<R>;
};

template <int N>
__device__ __forceinline__ void wait_loads_and_meet() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

constexpr int kDenseSlots = 5;  // of dense_loop's ring
constexpr int dense_stage_bytes(int MI, int NI) { return (MI + NI) * 64 * kDenseK * 2; }
// LDS of a tile: dense_loop's ring (STAGES 0), or that many stages of dense_loop_deep's
constexpr int dense_lds_bytes(int MI, int NI, int STAGES) {
    return STAGES ? STAGES * dense_stage_bytes(MI, NI) : kDenseSlots * (MI > NI ? MI : NI) * 64 * kDenseK * 2;
}

// The K loop over steps [k0, k1) (of the tile's K; `left`: k in the step k_last, the
// operand's last).  GLU: B's blocks are dealt to the waves so that a wave has NI / 2
// blocks of the tile's first half and the same of its second.  On return every load
// has landed and the workgroup has met.
//
// The ring of SLOTS operand tiles, an odd number, holds A and B of the step in hand and of the AHEAD - 1 that follow, and A of
// one more.  Past a step's barrier its two slots are free: B of step + AHEAD goes to A's,
// A of the step after to B's.  The loads are spread: a CU takes one of 1 KiB in 16
// cycles, so the 64 of a 256 x 256 step need half of its MFMAs' time, and issued in the
// quarter of it past the barrier they held up the waves' MFMAs (2,923 cycles a step
// with two slots of both operands, 2,661 with no memory behind them, 2,139 without loads).
template <class T, int MI, int NI, bool AT, bool BT, bool GLU, class LA, class LB>
__device__ __forceinline__ void dense_loop(LA &la, LB &lb, int k0, int k1, int k_last, int left, uint32_t lds, int wave, int lane,
                                           DenseAcc<MI, NI> &acc) {
    constexpr int SLOTS = kDenseSlots;
    static_assert(SLOTS % 2 == 1 && SLOTS >= 5, "A and B in turn");
    constexpr int SLOT = (MI > NI ? MI : NI) * 64 * kDenseK * 2, AHEAD = SLOTS / 2, NA = LA::BL, NB = LB::BL;
    constexpr int NQ = MI * NI, RPQ = (MI + NI + NQ - 1) / NQ;  // MFMAs per sub-step; fragment reads beside each of the first
    typedef typename T::v8 v8;
    const int wm = wave >> 1, wn = wave & 1;
    Frags<T, AT, 64 * MI> fa;
    Frags<T, BT, 64 * NI> fb;
    fa.init(lane);
    fb.init(lane);
    auto bblock = [&](int ni) { return GLU ? (ni < NI / 2 ? wn * (NI / 2) + ni : NI + wn * (NI / 2) + ni - NI / 2) : wn * NI + ni; };
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[mi][ni][e] = 0.f;
    u32x4 ra, rb;
    uint32_t sa, sb;
    auto open_a = [&](int step) {  // a step past the range is an empty buffer
        if (step == k_last && left < kDenseK) la.cut(left);
        ra = la.stage(step, step < k1), sa = la.step_off(step);
    };
    auto open_b = [&](int step) {
        if (step == k_last && left < kDenseK) lb.cut(left);
        rb = lb.stage(step, step < k1), sb = lb.step_off(step);
    };
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
        open_a(k0 + j), open_b(k0 + j);
#pragma unroll
        for (int i = 0; i < NA; ++i) la.load(ra, sa, lds + 2 * j * SLOT, wave, i);
#pragma unroll
        for (int i = 0; i < NB; ++i) lb.load(rb, sb, lds + (2 * j + 1) * SLOT, wave, i);
    }
    wait_loads_and_meet<(AHEAD - 1) * (NA + NB)>();
    v8 a[2][MI], b[2][NI];
    auto read = [&](int to, uint32_t sa_, uint32_t sb_, int s, int i) {  // i: 0 .. MI + NI - 1; what the first MFMAs take first
        if (i == 0 || i > MI)
            b[to][i == 0 ? 0 : i - MI] = fb.get(sb_, bblock(i == 0 ? 0 : i - MI), s);
        else
            a[to][i - 1] = fa.get(sa_, wm * MI + i - 1, s);
    };
    uint32_t slot = 0;  // of A of the step in hand
    auto after = [](uint32_t at, int n) { return at + n >= (uint32_t)SLOTS ? at + n - SLOTS : at + n; };
#pragma unroll
    for (int i = 0; i < MI + NI; ++i) read(0, lds, lds + SLOT, 0, i);
    int kt = k0;  // one step at least
#pragma unroll 1
    do {
        const uint32_t pa = lds + slot * SLOT, pb = lds + after(slot, 1) * SLOT;
        const uint32_t last = lds + after(slot, SLOTS - 1) * SLOT;  // B's slot of the step before
        slot = after(slot, 2);
        const uint32_t na = lds + slot * SLOT, nb = lds + after(slot, 1) * SLOT;
        open_a(kt + AHEAD);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int cur = s & 1;
            if (s == 3) {
                wait_loads_and_meet<(AHEAD - 1) * NA + (AHEAD - 2) * NB>();
                open_b(kt + AHEAD);
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                // what this sub-step issues beside its MFMAs, spread over them
#pragma unroll
                for (int i = q * RPQ; i < (q + 1) * RPQ && i < MI + NI; ++i) read(cur ^ 1, s == 3 ? na : pa, s == 3 ? nb : pb, s == 3 ? 0 : s + 1, i);
                if (s == 3) {
#pragma unroll
                    for (int i = q * NB / NQ; i < (q + 1) * NB / NQ; ++i) lb.load(rb, sb, pa, wave, i);
                }
                if (s < 2) {
#pragma unroll
                    for (int i = (s * NQ + q) * NA / (2 * NQ); i < (s * NQ + q + 1) * NA / (2 * NQ); ++i) la.load(ra, sa, last, wave, i);
                }
                // operands swapped: a lane then holds four consecutive columns of one row
                acc[q / NI][q % NI] = T::mfma(b[cur][q % NI], a[cur][q / NI], acc[q / NI][q % NI]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } while (++kt < k1);
    wait_loads_and_meet<0>();
}

// The same for small tiles, whose MFMAs of a sub-step (4 of a 128 x 128 tile's wave) end
// before a fragment read for the next has come back: fragments are read two sub-steps
// ahead, into four sets.  The barrier stands before the step's third sub-step, where the
// first reads of the next stage are; the stage of the step before is then free for the
// one STAGES - 1 further on, whose loads are spread over the step that follows.
template <class T, int MI, int NI, bool AT, bool BT, bool GLU, int STAGES, class LA, class LB>
__device__ __forceinline__ void dense_loop_deep(LA &la, LB &lb, int k0, int k1, int k_last, int left, uint32_t lds, int wave, int lane,
                                                DenseAcc<MI, NI> &acc) {
    static_assert(STAGES >= 4, "the stage before, the one in hand, the next and one that lands");
    constexpr int A_BYTES = MI * 64 * kDenseK * 2, STAGE = dense_stage_bytes(MI, NI), NA = LA::BL, ND = NA + LB::BL;
    constexpr int NQ = MI * NI, RPQ = (MI + NI + NQ - 1) / NQ;
    typedef typename T::v8 v8;
    const int wm = wave >> 1, wn = wave & 1;
    Frags<T, AT, 64 * MI> fa;
    Frags<T, BT, 64 * NI> fb;
    fa.init(lane);
    fb.init(lane);
    auto bblock = [&](int ni) { return GLU ? (ni < NI / 2 ? wn * (NI / 2) + ni : NI + wn * (NI / 2) + ni - NI / 2) : wn * NI + ni; };
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[mi][ni][e] = 0.f;
    u32x4 ra, rb;
    uint32_t sa, sb;
    auto open = [&](int step) {  // a step past the range is an empty buffer
        if (step == k_last && left < kDenseK) la.cut(left), lb.cut(left);
        const bool in = step < k1;
        ra = la.stage(step, in), rb = lb.stage(step, in);
        sa = la.step_off(step), sb = lb.step_off(step);
    };
    auto load = [&](uint32_t stage, int i) {
        if (i < NA)
            la.load(ra, sa, stage, wave, i);
        else
            lb.load(rb, sb, stage + A_BYTES, wave, i - NA);
    };
    // loads [0, ND) of a stage over the sub-steps 2, 3, 0, 1: the first of place p of 4 NQ
    auto first = [](int p) { return p * ND / (4 * NQ); };
#pragma unroll
    for (int j = 0; j < STAGES - 1; ++j) {
        open(k0 + j);
#pragma unroll
        for (int i = 0; i < (j < STAGES - 2 ? ND : first(2 * NQ)); ++i) load(lds + j * STAGE, i);
    }
    wait_loads_and_meet<(STAGES - 3) * ND + first(2 * NQ)>();
    v8 a[4][MI], b[4][NI];
    auto read = [&](int s, uint32_t stage, int i) {
        if (i == 0 || i > MI)
            b[s][i == 0 ? 0 : i - MI] = fb.get(stage + A_BYTES, bblock(i == 0 ? 0 : i - MI), s);
        else
            a[s][i - 1] = fa.get(stage, wm * MI + i - 1, s);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < MI + NI; ++i) read(s, lds, i);
        __builtin_amdgcn_sched_barrier(0);  // in the loop's order, or its first wait is for all of them
    }
    uint32_t slot = 0;
    auto after = [](uint32_t at, int n) { return at + n >= (uint32_t)STAGES ? at + n - STAGES : at + n; };
    int kt = k0;  // one step at least
#pragma unroll 1
    do {
        const uint32_t stage = lds + slot * STAGE, before = lds + after(slot, STAGES - 1) * STAGE, filling = lds + after(slot, STAGES - 2) * STAGE;
        slot = after(slot, 1);
        const uint32_t next = lds + slot * STAGE;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s == 2) {
                // every read of the stage before has been used; this one's are in flight
                asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((STAGES - 3) * ND) : "memory");
                open(kt + STAGES - 1);
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
#pragma unroll
                for (int i = q * RPQ; i < (q + 1) * RPQ && i < MI + NI; ++i) read((s + 2) & 3, s < 2 ? stage : next, i);
                const int p = ((s + 2) & 3) * NQ + q;
#pragma unroll
                for (int i = first(p); i < first(p + 1); ++i) load(s < 2 ? filling : before, i);
                acc[q / NI][q % NI] = T::mfma(b[s][q % NI], a[s][q / NI], acc[q / NI][q % NI]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } while (++kt < k1);
    wait_loads_and_meet<0>();
}

// Elements 4 q ... of an accumulator, where they are used: moved out of the accumulation
// registers all at once, ahead of the branches to the ways out, they would not fit.
__device__ __forceinline__ f32x4 dense_take(const f32x16 &c, int q) {
    float a = c[4 * q], b = c[4 * q + 1], d = c[4 * q + 2], e = c[4 * q + 3];
    asm volatile("" : "+v"(a), "+v"(b), "+v"(d), "+v"(e));
    return f32x4{a, b, d, e};
}

// The tile's values, 8 consecutive columns of a row at a time, through LDS that the
// wave has to itself (its own 32 rows x 32 NI columns of fp32): lane l of a block
// holds row l % 32, columns 8 q + 4 (l / 32) + 0..3 in elements 4 q ...  The chunks of
// a row are permuted by XOR with the row, so that 16 rows' writes of one column hit
// different chunks.  For each row and its 8 columns, of the tile: pre(row, column) loads
// what the output needs besides, some rows ahead; f(row, column, that, v) or, GLU,
// f(row, column, that, h, u).
template <int MI, int NI, bool GLU, class P, class F>
__device__ __forceinline__ void dense_rows(const DenseAcc<MI, NI> &acc, uint32_t lds, int wave, int lane, P &&pre, F &&f) {
    constexpr int ROW = NI * 128, MASK = NI * 8 < 16 ? NI * 8 - 1 : 15;
    constexpr int LPR = GLU ? NI * 2 : NI * 4, RPP = 64 / LPR, PASSES = 32 / RPP;  // lanes per row, rows per pass
    constexpr int AHEAD = PASSES < 4 ? PASSES : 4;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    const uint32_t st = lds + wave * 32 * ROW;
    const int wm = wave >> 1, wn = wave & 1, r = lane & 31, hi = lane >> 5;
    const int c8 = lane % LPR, col = wn * (GLU ? NI * 16 : NI * 32) + c8 * 8;
    auto get = [&](int row, int c, float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const f32x4 x = *(const lds_f32x4 *)(uintptr_t)(st + row * ROW + (((2 * c + k) ^ (row & MASK)) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * k + e] = x[e];
        }
    };
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = dense_take(acc[mi][ni], q);
                *(lds_f32x4 *)(uintptr_t)(st + r * ROW + (((ni * 8 + 2 * q + hi) ^ (r & MASK)) << 4)) = v;
            }
        const int row0 = wm * MI * 32 + mi * 32;
#pragma unroll 1
        for (int p0 = 0; p0 < PASSES; p0 += AHEAD) {
            decltype(pre(0, 0)) ahead[AHEAD];
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) ahead[p] = pre(row0 + (p0 + p) * RPP + lane / LPR, col);
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) {
                const int row = (p0 + p) * RPP + lane / LPR;
                float v[8];
                get(row, c8, v);
                if constexpr (GLU) {
                    float u[8];
                    get(row, LPR + c8, u);
                    f(row0 + row, col, ahead[p], v, u);
                } else {
                    f(row0 + row, col, ahead[p], v);
                }
            }
        }
    }
}

// The same for outputs that are 16-bit values of the tile's own: N matrices of COLS
// columns a wave (one of 32 NI, or GLU's a, h and u of 16 NI each), packed before they
// go through LDS.  value(m, x): matrix m's four values from the accumulators' four, x of
// a tile's columns or, GLU, x[0] of its first half and x[1] of its second.  put(m, row,
// column, 16 bytes).  Half the LDS traffic of dense_rows, and nothing but loads and
// stores past it.
template <class T, int MI, int NI, bool GLU, int N, class V, class P>
__device__ __forceinline__ void dense_rows16(const DenseAcc<MI, NI> &acc, uint32_t lds, int wave, int lane, V &&value, P &&put) {
    constexpr int NC = GLU ? NI / 2 : NI, RB = NC * 64, W = 256 / RB;   // blocks across; bytes of a row; rows of a window
    constexpr int G = N > 1 && MI > 2 ? MI / 2 : MI, PLANE = 32 * G * RB;  // blocks down at a time
    constexpr int LPR = RB / 16, RPP = 64 / LPR, PASSES = 32 * G / RPP, AHEAD = PASSES < 8 ? PASSES : 8;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    const uint32_t st = lds + wave * (N * PLANE);
    const int wm = wave >> 1, wn = wave & 1, hi = lane >> 5;
    // chunk c (16 bytes) of a row
    auto at = [&](int row, int c) { return (uint32_t)((row / W) * 256 + (((((row % W) * (16 / W)) | c) ^ ((row / W) & 15)) << 4)); };
#pragma unroll
    for (int g = 0; g < MI; g += G) {
#pragma unroll
        for (int mi = 0; mi < G; ++mi)
#pragma unroll
            for (int ni = 0; ni < NC; ++ni)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 c0 = dense_take(acc[g + mi][ni], q), c1 = GLU ? dense_take(acc[g + mi][GLU ? ni + NC : ni], q) : c0;
                    float x[2][4], o[N][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[0][e] = c0[e], x[1][e] = c1[e];
                    value(x, o);
#pragma unroll
                    for (int m = 0; m < N; ++m)
                        *(lds_u32x2 *)(uintptr_t)(st + m * PLANE + at(mi * 32 + (lane & 31), ni * 4 + q) + hi * 8) =
                            u32x2{(uint32_t)T::down(o[m][0]) | (uint32_t)T::down(o[m][1]) << 16, (uint32_t)T::down(o[m][2]) | (uint32_t)T::down(o[m][3]) << 16};
                    __builtin_amdgcn_sched_barrier(0);  // a few accumulators in registers at a time
                }
        const int c = lane % LPR, col = (wn * NC) * 32 + c * 8, row0 = wm * MI * 32 + g * 32;
#pragma unroll
        for (int m = 0; m < N; ++m)
#pragma unroll 1
            for (int p0 = 0; p0 < PASSES; p0 += AHEAD) {
                u32x4 v[AHEAD];
#pragma unroll
                for (int p = 0; p < AHEAD; ++p) v[p] = *(const lds_u32x4 *)(uintptr_t)(st + m * PLANE + at((p0 + p) * RPP + lane / LPR, c));
#pragma unroll
                for (int p = 0; p < AHEAD; ++p) put(m, row0 + (p0 + p) * RPP + lane / LPR, col, v[p]);
            }
    }
}

}  // namespace moe

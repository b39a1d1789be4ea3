// The gated feed-forward block of any number of rows, and its gradient.
//
//   h = X Wg^T, u = X Wu^T          (W13 = [Wg; Wu], one product of 2 I columns)
//   a = act(h) u                    (in the product's epilogue, in fp32, rounded once)
//   out = a W2^T
//
//   dA = dOut W2;  dh = dA u act'(h), du = dA act(h)   (epilogue; rounded once to 16 bits)
//   dX = [dh du] W13;  dW13 = [dh du]^T X;  dW2 = dOut^T a
//
// a and [dh du] are operands of matrix products, so they are 16-bit; every sum is fp32.
// A product with fewer tiles than the device has CUs may be cut along K: each part leaves
// its fp32 sums in the workspace, and a second pass adds them in ascending order and
// does the epilogue.
//
// Bound by the matrix cores from some hundred rows on (6 I H flop a row forward, 12 backward).
// H = 7168, I = 2048: 16,384 rows forward 722 + 385 us (1.30 PFLOP/s; a library's product of 8192^3
// reaches 1.25 here), 8,192 rows backward 205 for the activations and 917 for the three gradients in
// one launch, and up to 4% more where the clock is lower.  The backward's products have their operands as they lie, which costs
// transposing LDS reads and no copy.
#pragma once

#include "dense.hpp"

namespace moe {

// v = act(x), d = act'(x) (GRAD)
template <bool GRAD, int N>
__device__ __forceinline__ void activation(int kind, const float (&x)[N], float (&v)[N], float (&d)[N]) {
    if (kind == MOE_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-x[e]));
            v[e] = x[e] * s;
            if (GRAD) d[e] = s * fmaf(x[e], 1.0f - s, 1.0f);
        }
    } else if (kind == MOE_ACT_GELU) {
        // x Phi(x).  The tail Phi(-|x|) = e^{-x^2 / 2} / 2 times erfcx(z), z = |x| / sqrt(2): a polynomial of degree 9
        // in t = 1 / (1 + 0.45 z), times t, fitted to it for all z >= 0 (off by 3.2e-8 of its value; in fp32, with the
        // exponential, by 1.3e-6 to x = -6: relative to the tail, which a form of 1 - erf loses).  act' needs the
        // same exponential.  (With erfcf the gradient of 333 rows of I = 520 took 20.4 us for 13.)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float t = __builtin_amdgcn_rcpf(fmaf(0.31819805f, __builtin_fabsf(x[e]), 1.0f)), g = __expf(-0.5f * x[e] * x[e]);
            float r = -0.04140037f;
            r = fmaf(r, t, 0.19072819f);
            r = fmaf(r, t, -0.30065574f);
            r = fmaf(r, t, 0.14247319f);
            r = fmaf(r, t, -0.02239985f);
            r = fmaf(r, t, 0.11996497f);
            r = fmaf(r, t, 0.1752492f);
            r = fmaf(r, t, 0.22827196f);
            r = fmaf(r, t, 0.25388315f);
            r = fmaf(r, t, 0.25388532f);
            const float tail = 0.5f * g * (t * r), c = x[e] < 0.f ? tail : 1.0f - tail;
            v[e] = x[e] * c;
            if (GRAD) d[e] = fmaf(x[e] * 0.39894228f, g, c);
        }
    } else if (kind == MOE_ACT_GELU_TANH) {
        // (1 + tanh(w)) / 2 = sigmoid(2 w), w = sqrt(2 / pi) (x + 0.044715 x^3)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float x2 = x[e] * x[e], s = __builtin_amdgcn_rcpf(1.0f + __expf(-1.5957691f * x[e] * fmaf(0.044715f, x2, 1.0f)));
            v[e] = x[e] * s;
            if (GRAD) {
                const float g = s * (1.0f - s);  // 0 long before x^3 is infinite
                d[e] = g > 0.f ? fmaf(x[e] * g, 1.5957691f * fmaf(0.134145f, x2, 1.0f), s) : s;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            v[e] = x[e] > 0.f ? x[e] : x[e] == x[e] ? 0.f : x[e];
            if (GRAD) d[e] = x[e] > 0.f ? 1.0f : 0.f;
        }
    }
}

__device__ __forceinline__ float activation1(int kind, float h) {
    const float x[1] = {h};
    float v[1], none[1];
    activation<false>(kind, x, v, none);
    return v[0];
}

// One product: D[M][N] = A B^T over K.  For the gate / up product N counts the columns
// of a (I), B has 2 N rows.
struct DenseArgs {
    const uint16_t *A, *B;
    int64_t lda, ldb;
    int M, N, K;
    int mt, nt;        // tiles
    int splits, steps;  // parts of K, and steps of 64 k in each
    float *part;       // [splits][M][N (2 N)] fp32 sums of the parts (splits > 1)
};

// Tile `id` of a grid of workgroups: each XCD (workgroups go to the eight in turn) has
// a run of consecutive tiles, and those go down `kGroup` tiles of M for each of N, so
// the tiles that run at once on an XCD share operands in its L2.
constexpr int kGroup = 4;
__device__ __forceinline__ void dense_tile_of(int id, int mt, int nt, int &m, int &n) {
    const int per = kGroup * nt, g = id / per, in = id - g * per, gm = min(kGroup, mt - g * kGroup);
    m = g * kGroup + in % gm;
    n = in / gm;
}
__device__ __forceinline__ int dense_xcd_order(int block, int total) {
    const int x = block & 7, i = block >> 3, per = total >> 3, rest = total & 7;
    return x * per + min(x, rest) + i;
}

// ---------------------------------------------------------------------------
// What becomes of 8 consecutive columns of a row.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void store16(void *p, const u32x4 &v) { *reinterpret_cast<u32x4 *>(p) = v; }
__device__ __forceinline__ void store_f32x8(float *p, const float (&v)[8]) {
    reinterpret_cast<f32x4 *>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4 *>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}

struct Nothing {};

// a = act(h) u, and h, u themselves (HU nullable)
template <class T>
struct GluOut {
    uint16_t *HU, *A;
    int I, act;
    static constexpr int kPacked = 3;  // a, h, u
    static constexpr bool kAlwaysPacked = true;
    __device__ __forceinline__ bool packed() const { return true; }
    __device__ __forceinline__ void values(const float (&x)[2][4], float (&o)[3][4]) const {
        float none[4];
        activation<false>(act, x[0], o[0], none);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][e] *= x[1][e], o[1][e] = x[0][e], o[2][e] = x[1][e];
    }
    __device__ __forceinline__ void put(int m, int64_t r, int c, const u32x4 &v) const {
        if (m == 0)
            store16(A + r * I + c, v);
        else if (HU)
            store16(HU + r * 2 * I + (m - 1) * I + c, v);
    }
    __device__ __forceinline__ Nothing pre(int64_t, int) const { return {}; }
    __device__ __forceinline__ void operator()(int64_t r, int c, Nothing, const float (&h)[8], const float (&u)[8]) const {
        float a[8], none[8];
        activation<false>(act, h, a, none);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] *= u[e];
        store16(A + r * I + c, pack8<T>(a));
        if (HU) {
            store16(HU + r * 2 * I + c, pack8<T>(h));
            store16(HU + r * 2 * I + I + c, pack8<T>(u));
        }
    }
};

// v = dA: [dh du] from the h and u kept; a again for dW2 where it was not kept.
// In fp16, h and u past 65504 were kept as infinities, which stand for numbers.  In the place of h goes one that the activation
// takes to its limits and that makes every product but one with 0 infinite in fp16; in the place of u, where it meets a 0, a 0.
// (Branches, not selects: those took the gradient of 333 rows of I = 520 31.6 us for 27.3.  The branches' bodies
// are short, or the unrolled epilogue of the 256 x 256 tile gives up its registers for scratch memory.)
template <class T>
struct GluBwdOut {
    const uint16_t *HU;
    uint16_t *dHU, *A;  // A nullable
    int I, act;
    static constexpr int kPacked = 0;
    static constexpr bool kAlwaysPacked = false;
    struct Kept {
        u32x4 h, u;
    };
    __device__ __forceinline__ Kept pre(int64_t r, int c) const {
        const uint16_t *p = HU + r * 2 * I + c;
        return Kept{*reinterpret_cast<const u32x4 *>(p), *reinterpret_cast<const u32x4 *>(p + I)};
    }
    __device__ __forceinline__ void operator()(int64_t r, int c, const Kept &k, const float (&v)[8]) const {
        float h[8], u[8], a[8], d[8];
        unpack8<T>(k.h, h);
        unpack8<T>(k.u, u);
        bool far = false;
        if constexpr (T::kNarrow) {
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(fmaxf(most, __builtin_fabsf(h[e])), __builtin_fabsf(u[e]));
            far = most > 65504.f;
        }
        if (far) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = __builtin_isinf(h[e]) ? copysignf(0x1p70f, h[e]) : h[e];
        }
        activation<true>(act, h, a, d);
        float w[8];  // u where it meets a
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = u[e];
        if (far) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = __builtin_isinf(u[e]) && a[e] == 0.f ? 0.f : u[e];
                u[e] = __builtin_isinf(u[e]) && (d[e] == 0.f || v[e] == 0.f) ? 0.f : u[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            d[e] *= v[e] * u[e];
            h[e] = v[e] * a[e];
            a[e] *= w[e];
        }
        uint16_t *o = dHU + r * 2 * I + c;
        store16(o, pack8<T>(d));
        store16(o + I, pack8<T>(h));
        if (A) store16(A + r * I + c, pack8<T>(a));
    }
};

// rows of 16-bit or fp32 values; fp32 may be added to
template <class T>
struct MatOut {
    void *p;
    int64_t ld;
    int f32, add;
    static constexpr int kPacked = 1;
    static constexpr bool kAlwaysPacked = false;
    __device__ __forceinline__ bool packed() const { return !f32; }
    __device__ __forceinline__ void values(const float (&x)[2][4], float (&o)[1][4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][e] = x[0][e];
    }
    __device__ __forceinline__ void put(int, int64_t r, int c, const u32x4 &v) const { store16(static_cast<uint16_t *>(p) + r * ld + c, v); }
    struct Old {
        f32x4 v[2];
    };
    __device__ __forceinline__ Old pre(int64_t r, int c) const {
        Old o{};
        if (add) {
            const f32x4 *q = reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + r * ld + c);
            o.v[0] = q[0], o.v[1] = q[1];
        }
        return o;
    }
    __device__ __forceinline__ void operator()(int64_t r, int c, const Old &old, const float (&v)[8]) const {
        if (!f32) {
            store16(static_cast<uint16_t *>(p) + r * ld + c, pack8<T>(v));
            return;
        }
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = add ? v[e] + old.v[e >> 2][e & 3] : v[e];
        store_f32x8(static_cast<float *>(p) + r * ld + c, s);
    }
};

// the sums of one part of K
struct PartOut {
    float *p;
    int64_t ld;
    int N;
    __device__ __forceinline__ Nothing pre(int64_t, int) const { return {}; }
    __device__ __forceinline__ void operator()(int64_t r, int c, Nothing, const float (&v)[8]) const { store_f32x8(p + r * ld + c, v); }
    __device__ __forceinline__ void operator()(int64_t r, int c, Nothing, const float (&h)[8], const float (&u)[8]) const {
        store_f32x8(p + r * ld + c, h);
        store_f32x8(p + r * ld + N + c, u);
    }
};

// Workgroup's share of a product: one tile and one part of K, tiles of a part together.
template <class T, int MI, int NI, bool AT, bool BT, bool GLU, int STAGES, class F>
__device__ __forceinline__ void dense_body(const DenseArgs &g, const F &f, uint32_t lds, int block, int blocks) {
    const int id = dense_xcd_order(block, blocks), tiles = g.mt * g.nt, split = id / tiles, tile = id - split * tiles;
    constexpr int BM = 64 * MI, BN = GLU ? 32 * NI : 64 * NI;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    dense_tile_of(tile, g.mt, g.nt, mt, nt);
    const int m0 = mt * BM, n0 = nt * BN;
    typename LoadOf<AT, 64 * MI>::type la;
    typename LoadOf<BT, 64 * NI>::type lb;
    if constexpr (AT)
        la.init(g.A + m0, g.lda, min(BM, g.M - m0), g.K, lane);
    else
        la.init(g.A + (int64_t)m0 * g.lda, g.lda, min(BM, g.M - m0), wave, lane);
    if constexpr (BT) {
        lb.init(g.B + n0, g.ldb, min(BN, g.N - n0), g.K, lane);
    } else if constexpr (GLU) {  // the tile's first half gate rows, the second up rows: two waves each
        const bool up = wave >= 2;
        lb.init(g.B + ((int64_t)n0 + (up ? g.N : 0)) * g.ldb, g.ldb, min(BN, g.N - n0), wave, lane, up ? 2 * LoadK<64 * NI>::BL : 0);
    } else {
        lb.init(g.B + (int64_t)n0 * g.ldb, g.ldb, min(BN, g.N - n0), wave, lane);
    }
    const int total = (g.K + kDenseK - 1) / kDenseK, k0 = split * g.steps, k1 = min(total, k0 + g.steps);
    DenseAcc<MI, NI> acc;
    const int left = g.K - (total - 1) * kDenseK;
    if constexpr (STAGES > 0)
        dense_loop_deep<T, MI, NI, AT, BT, GLU, STAGES>(la, lb, k0, k1, total - 1, left, lds, wave, lane, acc);
    else
        dense_loop<T, MI, NI, AT, BT, GLU>(la, lb, k0, k1, total - 1, left, lds, wave, lane, acc);
    auto in = [&](int r, int c) { return m0 + r < g.M && n0 + c < g.N; };
    auto rows = [&](const auto &o) {
        typedef decltype(o.pre(0, 0)) Pre;
        dense_rows<MI, NI, GLU>(
            acc, lds, wave, lane, [&](int r, int c) { return in(r, c) ? o.pre(m0 + r, n0 + c) : Pre{}; },
            [&](int r, int c, const Pre &p, auto &...v) {
                if (in(r, c)) o(m0 + r, n0 + c, p, v...);
            });
    };
    if (g.splits > 1) {
        const int64_t ld = GLU ? 2 * (int64_t)g.N : g.N;
        rows(PartOut{g.part + split * (g.M * ld), ld, g.N});
        return;
    }
    // outputs that are 16-bit values of the tile alone have a way of their own
    if constexpr (F::kPacked > 0) {
        if (f.packed()) {
            dense_rows16<T, MI, NI, GLU, F::kPacked>(
                acc, lds, wave, lane, [&](const float (&x)[2][4], auto &o) { f.values(x, o); },
                [&](int m, int r, int c, const u32x4 &v) {
                    if (in(r, c)) f.put(m, m0 + r, n0 + c, v);
                });
            return;
        }
    }
    if constexpr (!F::kAlwaysPacked) rows(f);
}

// The parts' sums in ascending order, and the epilogue: 8 columns a thread.
template <bool GLU, class Out>
__device__ __forceinline__ void dense_join_body(const DenseArgs &g, const Out &out) {
    const int per = g.N / 8;
    const int64_t ld = GLU ? 2 * (int64_t)g.N : g.N, plane = g.M * ld, n = (int64_t)g.M * per;
    auto sum = [&](int64_t o, float (&v)[8]) {
        f32x4 a = f32x4{0.f, 0.f, 0.f, 0.f}, b = a;
        for (int s = 0; s < g.splits; ++s) {
            const f32x4 *p = reinterpret_cast<const f32x4 *>(g.part + s * plane + o);
            a += p[0], b += p[1];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    };
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per) * 8;
        float v[8];
        sum(r * ld + c, v);
        if constexpr (GLU) {
            float u[8];
            sum(r * ld + g.N + c, u);
            out(r, c, out.pre(r, c), v, u);
        } else {
            out(r, c, out.pre(r, c), v);
        }
    }
}

}  // namespace moe

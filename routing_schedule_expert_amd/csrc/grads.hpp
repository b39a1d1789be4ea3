// The norm of many gradients together, and the gradients scaled to it.
//
//   norm = |s| sqrt(sum of squares)  or  |s| max,   c = min(1, max_norm / (norm + eps)),   out = (s c) g
//
// Two passes over the gradients, bound by memory: 480 fp32 tensors of 2.5 GB take 1,360 us, the sums
// 432 (5.7 TB/s), the scaling 922 (5.4 TB/s read and written).  Squares are summed in 64 bits (no
// square of an fp32 number overflows or vanishes there), each workgroup's sum in a slot
// of its own, and the second pass's workgroups each add the slots in one fixed order,
// so no launch stands between the passes (past 2048 slots one workgroup does it: 4,096 slots, read
// by each of 2048 workgroups, are no longer little).  A maximum is that of the magnitudes' bits,
// where NaN is above infinity.
//
// The tensors of a launch come as its arguments (their addresses may be others in the
// next call).  They are cut into pieces, dealt to the workgroups in turn;
// loads are of 16 bytes: the sums' from a tensor's own start, the scaling's of whole aligned words, the
// neighbours' elements in a tensor's first and last word left out.
#pragma once

#include "dense.hpp"

namespace moe {

constexpr int kGradThreads = 512;
// Elements of a piece: 16384 stream best (2.5 GB), but leave most CUs without one where there
// are few (5 tensors of 100,000 elements: 9 pieces of 16384, 51 of 2048).
constexpr int kGradShift = 14, kGradShiftFew = 11;  // a piece has 2^shift elements
constexpr int kGradParts = 2048;    // workgroups of a launch of the first pass at most
// Tensors per launch: arguments below 4 KiB.  Where each is scaled in its own place the second pass needs no more of
// them than the first.
constexpr int kGradTensors = 248, kGradTensorsOut = 160;

// A tensor in 12 bytes: address (48 bits), elements (44) and type (2, above).
struct GradTensor {
    uint32_t w[3];
};
inline GradTensor grad_tensor(const void *g, int64_t n, int type) {
    const uint64_t p = (uint64_t)(uintptr_t)g;
    return GradTensor{{(uint32_t)p, (uint32_t)(p >> 32) | (uint32_t)n << 16, (uint32_t)((uint64_t)n >> 16) | (uint32_t)type << 28}};
}
template <class K>  // of an argument, which lies in an address space of its own
__device__ __forceinline__ const void *grad_address(const K &t) { return (const void *)(uintptr_t)((uint64_t)t.w[0] | (uint64_t)(t.w[1] & 0xffffu) << 32); }
template <class K>
__device__ __forceinline__ int64_t grad_numel(const K &t) { return (int64_t)((uint64_t)(t.w[1] >> 16) | (uint64_t)(t.w[2] & 0x0fffffffu) << 16); }

template <bool OUT>
struct GradLaunch {
    static constexpr int N = OUT ? kGradTensorsOut : kGradTensors;
    GradTensor t[N];
    int32_t start[N];        // each tensor's first piece
    void *out[OUT ? N : 1];  // without OUT: the tensors themselves
    int32_t count, pieces;
    int32_t shift;
};
struct GradScalars {
    double *parts;
    moe_grad_result *result;
    const float *coef;  // given: no norm is formed
    int32_t nparts, kind;
    float scale, max_norm, eps;
};

template <class T>
struct GradVec;  // 16 bytes of elements
template <>
struct GradVec<F32> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float get(const u32x4 &v, int i) { return __uint_as_float(v[i]); }
};
template <class T>
struct GradVec {
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(const u32x4 &v, int i) { return T::up((uint16_t)(v[i >> 1] >> (16 * (i & 1)))); }
};

// MAX: the largest magnitude's bits, otherwise the sum of squares.
template <bool MAX>
struct GradSum {
    double s = 0.0;
    uint32_t m = 0;
    __device__ __forceinline__ void add(float v) {
        if constexpr (MAX)
            m = max(m, __float_as_uint(v) & 0x7fffffffu);
        else
            s = fma((double)v, (double)v, s);
    }
};
// What the arguments point at is global memory; the compiler, which sees a pointer
// loaded from memory, cannot know.
typedef __attribute__((address_space(1))) u32x4 global_u32x4;
__device__ __forceinline__ const global_u32x4 *grad_words(const void *g) { return (const global_u32x4 *)((uintptr_t)g & ~(uintptr_t)15); }

// 16 bytes of a tensor's elements, wherever it starts.
struct __attribute__((packed, aligned(2))) GradLoose {
    u32x4 v;
};
typedef __attribute__((address_space(1))) GradLoose global_loose;

// Elements [e0, e1) of the tensor at g; e0 is a piece's first.  Words are counted from the tensor's own start, so that which
// thread adds which elements, and with it the sum's last bits, does not hang on the address.
template <class T, bool MAX>
__device__ __forceinline__ void grad_sum_piece(const void *g, int64_t e0, int64_t e1, GradSum<MAX> &acc) {
    constexpr int N = GradVec<T>::N, ES = 16 / N;
    const global_loose *p = (const global_loose *)(uintptr_t)g;
    const int64_t w0 = e0 / N, w1 = e1 / N;  // whole words
    auto whole = [&](u32x4 v) {
#pragma unroll
        for (int i = 0; i < N; ++i) acc.add(GradVec<T>::get(v, i));
    };
    constexpr int U = 4;
    int64_t w = w0 + threadIdx.x;
    for (; w + (U - 1) * kGradThreads < w1; w += U * kGradThreads) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = p[w + u * kGradThreads].v;
#pragma unroll
        for (int u = 0; u < U; ++u) whole(v[u]);
    }
    for (; w < w1; w += kGradThreads) whole(p[w].v);
    if (threadIdx.x == 64) {  // what is left of the tensor's last word
        for (int64_t e = w1 * N; e < e1; ++e) {
            if constexpr (ES == 4)
                acc.add(((const __attribute__((address_space(1))) float *)(uintptr_t)g)[e]);
            else
                acc.add(T::up(((const __attribute__((address_space(1))) uint16_t *)(uintptr_t)g)[e]));
        }
    }
}

// A workgroup's sum, on thread 0.
template <bool MAX>
__device__ __forceinline__ double grad_join(const GradSum<MAX> &acc, double *lds) {
    double s = acc.s;
    uint32_t m = acc.m;
    for (int o = 32; o >= 1; o >>= 1) {
        s += __shfl_xor(s, o, 64);
        m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    }
    const int wave = threadIdx.x / 64, waves = blockDim.x / 64;
    if ((threadIdx.x & 63) == 0) lds[wave] = MAX ? (double)__uint_as_float(m) : s;
    __syncthreads();
    double r = lds[0];
    for (int w = 1; w < waves; ++w) {
        const double v = lds[w];
        r = MAX ? (v > r || v != v ? v : r) : r + v;
    }
    return r;
}

// f(tensor, address, type, from, to) of the workgroup's pieces: every gridDim.x-th.  Each lane holds the starts of
// some tensors, and a piece's tensor, the last one that starts at or before it, is a count of ballots.  (A walk
// along the starts, one load after the other, took 405 tensors of 3.7 M elements 70 us for 24.)
template <class L, class F>
__device__ __forceinline__ void grad_pieces(const L &l, bool backwards, F &&f) {
    constexpr int N = (L::N + 63) / 64;
    const int lane = threadIdx.x & 63, all = l.pieces;
    int start[N];
#pragma unroll
    for (int k = 0; k < N; ++k) start[k] = k * 64 + lane < l.count ? l.start[k * 64 + lane] : 0x7fffffff;
    for (int i = blockIdx.x; i < all; i += gridDim.x) {
        const int c = backwards ? all - 1 - i : i;
        int t = -1, first = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int n = __popcll(__ballot(start[k] <= c));
            if (n) first = __builtin_amdgcn_readlane(start[k], n - 1);
            t += n;
        }
        const auto &g = l.t[t];
        const int64_t e0 = (int64_t)(c - first) << l.shift;
        f(t, grad_address(g), (int)(g.w[2] >> 28), e0, min(grad_numel(g), e0 + (1ll << l.shift)));
    }
}

template <bool MAX, class L>
__device__ __forceinline__ void grad_sums_body(const L &l, const GradScalars &k, double *lds) {
    GradSum<MAX> acc;
    grad_pieces(l, false, [&](int, const void *g, int type, int64_t e0, int64_t e1) {
        if (type == MOE_TYPE_FP32)
            grad_sum_piece<F32>(g, e0, e1, acc);
        else if (type == MOE_TYPE_BF16)
            grad_sum_piece<Bf16>(g, e0, e1, acc);
        else
            grad_sum_piece<Fp16>(g, e0, e1, acc);
    });
    const double s = grad_join(acc, lds);
    if (threadIdx.x == 0) k.parts[blockIdx.x] = s;
}

// The norm's sum, and what it makes of the gradients, from the first pass's parts: on
// every thread of any workgroup the same.
__device__ __forceinline__ moe_grad_result grad_result(const GradScalars &k, double *lds) {
    const bool max_of = k.kind == MOE_NORM_MAX;
    double s = 0.0;
    for (int i = threadIdx.x; i < k.nparts; i += blockDim.x) {
        const double v = k.parts[i];
        s = max_of ? (v > s || v != v ? v : s) : s + v;
    }
    for (int o = 32; o >= 1; o >>= 1) {
        const double v = __shfl_xor(s, o, 64);
        s = max_of ? (v > s || v != v ? v : s) : s + v;
    }
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = s;
    __syncthreads();
    s = lds[0];
    for (int w = 1; w < (int)blockDim.x / 64; ++w) {
        const double v = lds[w];
        s = max_of ? (v > s || v != v ? v : s) : s + v;
    }
    const double scale = k.scale < 0.f ? -(double)k.scale : (double)k.scale;
    moe_grad_result r;
    r.sum = max_of ? s * scale : s * scale * scale;
    const double norm = max_of ? r.sum : sqrt(s) * scale, below = norm + (double)k.eps;
    const double c = below == 0.0 ? 1.0 : __builtin_isinf(below) ? 0.0 : (double)k.max_norm / below;  // 0 for an infinite max_norm too
    r.norm = (float)norm;
    r.coef = (float)(c >= 1.0 ? 1.0 : c);  // NaN stays
    return r;
}

template <class T>
__device__ __forceinline__ void grad_scale_piece(const void *g, void *out, int64_t e0, int64_t e1, float f) {
    constexpr int N = GradVec<T>::N, ES = 16 / N;
    const int lead = (int)(((uintptr_t)g & 15) / ES);
    const global_u32x4 *p = grad_words(g);
    typedef __attribute__((address_space(1))) char global_char;
    global_char *o = (global_char *)out;
    const int64_t a = e0 + lead, b = e1 + lead, w0 = a / N, w1 = (b + N - 1) / N, in0 = (a + N - 1) / N, in1 = b / N;
    auto scaled = [&](u32x4 v) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (N == 4)
                r[i] = __float_as_uint(GradVec<T>::get(v, i) * f);
            else
                r[i] = (uint32_t)T::down(GradVec<T>::get(v, 2 * i) * f) | (uint32_t)T::down(GradVec<T>::get(v, 2 * i + 1) * f) << 16;
        }
        return r;
    };
    // whole words of g are words of out where both start alike, and 16 bytes of any alignment otherwise
    auto put = [&](int64_t w, u32x4 v) { ((global_loose *)(o + (w * N - lead) * ES))->v = v; };
    constexpr int U = 4;
    int64_t w = in0 + threadIdx.x;
    for (; w + (U - 1) * kGradThreads < in1; w += U * kGradThreads) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = p[w + u * kGradThreads];
#pragma unroll
        for (int u = 0; u < U; ++u) put(w + u * kGradThreads, scaled(v[u]));
    }
    for (; w < in1; w += kGradThreads) put(w, scaled(p[w]));
    auto part = [&](int64_t k) {
        const u32x4 v = scaled(p[k]);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (k * N + i >= a && k * N + i < b) {
                if constexpr (N == 4)
                    ((__attribute__((address_space(1))) uint32_t *)o)[k * N + i - lead] = v[i];
                else
                    ((__attribute__((address_space(1))) uint16_t *)o)[k * N + i - lead] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
            }
    };
    if (threadIdx.x == 0 && w0 < in0) part(w0);
    if (threadIdx.x == 64 && in1 < w1 && (in1 > w0 || w0 >= in0)) part(in1);
}

// Backwards: what the first pass read last is what the cache still holds.
template <bool OUT, class L>
__device__ __forceinline__ void grad_scale_body(const L &l, const GradScalars &k, double *lds) {
    float f;
    if (k.coef) {
        f = k.scale * *k.coef;
    } else {
        const moe_grad_result r = grad_result(k, lds);
        if (blockIdx.x == 0 && threadIdx.x == 0) *k.result = r;
        f = k.scale * r.coef;
    }
    if (!OUT && f == 1.0f) return;
    grad_pieces(l, true, [&](int t, const void *g, int type, int64_t e0, int64_t e1) {
        void *out = OUT ? l.out[t] : const_cast<void *>(g);
        if (OUT && f == 1.0f && g == out) return;
        if (type == MOE_TYPE_FP32)
            grad_scale_piece<F32>(g, out, e0, e1, f);
        else if (type == MOE_TYPE_BF16)
            grad_scale_piece<Bf16>(g, out, e0, e1, f);
        else
            grad_scale_piece<Fp16>(g, out, e0, e1, f);
    });
}

}  // namespace moe

// Layer norm and its gradient.
//
//   m = mean(x), s = 1 / sqrt(mean((x - m)^2) + eps), xh = (x - m) s
//   y = xh g + b
//   dx = s (t - mean(t) - xh mean(t xh)) + dres,  t = dy g
//   dg = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: a row is read once, held in registers through its sums (the
// variance is that of the differences from the mean, a second sum in registers) and
// written once.  A thread keeps the same columns for every row it takes, 8 at a time,
// so gains and biases and the column sums of the gradient stay in its registers.
// Rows up to 512 elements are taken by a wave or a part of one (64, 32, 16 or 8
// lanes: no barrier), longer ones by a workgroup, with one, two (past 8192 elements) or
// four chunks a thread (past 16384).  The loads of the next row (forward, up to two chunks: of the
// two next) are in flight during this row's sums, and gains and biases stay in
// registers; of four chunks the gains come with each row, and the backward loads its
// rows as they come.  Past 8192 elements the column sums have no registers: a second
// reading makes them.
//
// Measured: 57,344 rows of 7168 in bf16 forward 329 us (5.0 TB/s), 16,384 of 7168 backward
// 132 and 5 for the sums of the column sums (5.2 TB/s); 8,192 of 12,288 forward 67 (190 without the loads ahead and
// the gains in registers), backward 95, 93 for its column sums and 5; 4,096 of 32,768 forward 237 (2.3 TB/s, the gains'
// L2 traffic twice the row's), backward 265, 116 and 7.  Rows without 16-byte alignment: 16,384 of 7,171
// forward 108, of 7168 83.
//
// Any row length and stride: where H or a stride is not a multiple of 8, or a pointer
// not of 16 bytes, the last 8 columns of a row start at H - 8 and overlap those before
// them (ODD: they are counted once), and loads are of elements' alignment.
#pragma once

#include "dense.hpp"
#include "norm.hpp"

namespace moe {

// 8 consecutive elements as they lie in memory.
template <class T>
struct Chunk {
    u32x4 v;
    static constexpr int ES = 2;
    template <bool ODD>
    __device__ __forceinline__ void load(const char *p) {
        if constexpr (ODD)
            __builtin_memcpy(&v, p, 16);
        else
            v = *reinterpret_cast<const u32x4 *>(p);
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int elem) { v = buffer_load16_nt(b, elem * 2); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t b, int elem, const float (&o)[8]) { buffer_store16(b, elem * 2, pack8<T>(o)); }
    __device__ __forceinline__ void load_some(const char *p, int n) {
        v = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) v[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[e] << (16 * (e & 1));
    }
    __device__ __forceinline__ void get(float (&o)[8]) const { unpack8<T>(v, o); }
    template <bool ODD>
    static __device__ __forceinline__ void store(char *p, const float (&o)[8]) {
        const u32x4 w = pack8<T>(o);
        if constexpr (ODD)
            __builtin_memcpy(p, &w, 16);
        else
            *reinterpret_cast<u32x4 *>(p) = w;
    }
    static __device__ __forceinline__ void store_some(char *p, const float (&o)[8], int from, int to) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= from && e < to) reinterpret_cast<uint16_t *>(p)[e] = T::down(o[e]);
    }
};
template <>
struct Chunk<F32> {
    f32x4 v[2];
    static constexpr int ES = 4;
    template <bool ODD>
    __device__ __forceinline__ void load(const char *p) {
        if constexpr (ODD) {
            __builtin_memcpy(v, p, 32);
        } else {
            v[0] = reinterpret_cast<const f32x4 *>(p)[0];
            v[1] = reinterpret_cast<const f32x4 *>(p)[1];
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, int elem) {
        v[0] = __builtin_bit_cast(f32x4, buffer_load16_nt(b, elem * 4));
        v[1] = __builtin_bit_cast(f32x4, buffer_load16_nt(b, elem * 4 + 16));
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t b, int elem, const float (&o)[8]) {
        buffer_store16(b, elem * 4, __builtin_bit_cast(u32x4, f32x4{o[0], o[1], o[2], o[3]}));
        buffer_store16(b, elem * 4 + 16, __builtin_bit_cast(u32x4, f32x4{o[4], o[5], o[6], o[7]}));
    }
    __device__ __forceinline__ void load_some(const char *p, int n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = e < n ? reinterpret_cast<const float *>(p)[e] : 0.f;
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v[e >> 2][e & 3];
    }
    template <bool ODD>
    static __device__ __forceinline__ void store(char *p, const float (&o)[8]) {
        const f32x4 a = f32x4{o[0], o[1], o[2], o[3]}, b = f32x4{o[4], o[5], o[6], o[7]};
        if constexpr (ODD) {
            __builtin_memcpy(p, &a, 16);
            __builtin_memcpy(p + 16, &b, 16);
        } else {
            reinterpret_cast<f32x4 *>(p)[0] = a;
            reinterpret_cast<f32x4 *>(p)[1] = b;
        }
    }
    static __device__ __forceinline__ void store_some(char *p, const float (&o)[8], int from, int to) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= from && e < to) reinterpret_cast<float *>(p)[e] = o[e];
    }
};

struct LnArgs {
    const void *x;
    const float *g, *b;  // b nullable (1 and 0 where null: g too)
    void *y;
    float *stats;  // [rows][2]: mean, 1 / std; nullable
    int64_t rows, ldx, ldy;
    int H;
    float eps;
};
struct LnBwdArgs {
    LnArgs f;  // y, b unused; stats read
    const void *dy, *dres;
    void *dx;
    float *part;  // [workgroups][2][H]: sums of dg and of db (null: not wanted)
};

// The lanes that share a row: `lanes` of a wave (a power of two from 8 on), or the
// workgroup.
template <bool WAVE>
struct Team {
    int lanes, t, teams, team;  // threads per row, this one's place, teams per workgroup, this one's
    __device__ __forceinline__ explicit Team(int lanes_) {
        lanes = WAVE ? lanes_ : blockDim.x;
        t = WAVE ? threadIdx.x & (lanes - 1) : threadIdx.x;
        teams = WAVE ? blockDim.x / lanes : 1;
        team = WAVE ? threadIdx.x / lanes : 0;
    }
};

// Sums over a team, on all of its threads, in a fixed order.
template <bool WAVE, int N>
struct TeamSum {
    RowSum<N> sum;
    int lanes;
    __device__ __forceinline__ TeamSum(float *lds, int lanes_) : sum(lds), lanes(lanes_) {}
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        if constexpr (!WAVE) {
            sum(v);
        } else if (lanes == 64) {
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
        } else {
            for (int o = lanes / 2; o >= 1; o >>= 1)
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], o, 64);
        }
    }
};

// A thread's columns: chunk i of CH starts at column at[i], of which the elements from
// skip[i] on count (8: none).  BUF: the row is the workgroup's and even, and a raw buffer, so that neither a
// row past the last one nor a thread without columns needs a branch around its loads
// and stores: with one, the compiler could not count which of them it waits for.
template <int CH, bool ODD, bool BUF>
struct Columns {
    static_assert(!BUF || !ODD, "raw buffers are of whole chunks");
    static constexpr bool SHORT = ODD && CH == 1;  // a row may be shorter than a chunk
    int at[CH], skip[CH], H;
    __device__ __forceinline__ Columns(int t, int lanes, int H_) : H(H_) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (i * lanes + t) * 8;
            at[i] = BUF ? c : max(0, min(c, H - 8));  // past a buffer's end: zeros
            skip[i] = c < H ? c - at[i] : 8;
        }
    }
    __device__ __forceinline__ bool in(int i) const { return skip[i] < 8; }
    // whether element e of chunk i counts; without ODD a chunk counts as a whole
    __device__ __forceinline__ bool counts(int i, int e) const { return ODD ? e >= skip[i] && e < H : in(i); }
    // of the row that starts at element `elem` (none: nothing is loaded that counts)
    template <class C>
    __device__ __forceinline__ void load(C (&c)[CH], const void *p, int64_t elem, bool some = true) const {
        if constexpr (BUF) {
            some = some && p;
            const __amdgpu_buffer_rsrc_t b = raw_buffer(static_cast<const char *>(p) + (some ? elem * C::ES : 0), some ? (uint32_t)(H * C::ES) : 0u);
#pragma unroll
            for (int i = 0; i < CH; ++i) c[i].load(b, at[i]);
            return;
        }
        if (!some || !p) return;
        const char *q = static_cast<const char *>(p) + elem * C::ES;
        if (SHORT && H < 8) {  // one chunk, which is the row
            c[0].load_some(q, in(0) ? H : 0);
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) c[i].template load<ODD>(q + (int64_t)at[i] * C::ES);
        }
    }
    // ONCE: what overlaps is written by the chunk before alone, otherwise twice with the same value
    template <class C, bool ONCE = false>
    __device__ __forceinline__ void store(int i, void *p, int64_t elem, const float (&v)[8]) const {
        if constexpr (BUF) {
            C::store(raw_buffer(static_cast<char *>(p) + elem * C::ES, (uint32_t)(H * C::ES)), at[i], v);
            return;
        }
        if (!in(i)) return;
        char *q = static_cast<char *>(p) + (elem + at[i]) * C::ES;
        if ((SHORT && H < 8) || (ODD && ONCE && skip[i]))
            C::store_some(q, v, ONCE ? skip[i] : 0, H);
        else
            C::template store<ODD>(q, v);
    }
    // fp32 values of chunk i's columns, `none` where p is null
    __device__ __forceinline__ void vec(int i, float (&v)[8], const float *p, float none) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = none;
        if (!p) return;
        Chunk<F32> c;
        const char *q = reinterpret_cast<const char *>(p);
        if constexpr (BUF)
            c.load(raw_buffer(p, (uint32_t)H * 4), at[i]);
        else if (SHORT && H < 8)
            c.load_some(q, in(i) ? H : 0);
        else
            c.template load<ODD>(q + (int64_t)at[i] * 4);
        c.get(v);
    }
};

template <class TI, class TO, int CH, bool WAVE, bool ODD>
__device__ __forceinline__ void ln_fwd_body(const LnArgs &a, int lanes, float *lds) {
    const Team<WAVE> team(lanes);
    const Columns<CH, ODD, !WAVE && !ODD> col(team.t, team.lanes, a.H);
    TeamSum<WAVE, 1> sum1(lds, team.lanes);
    TeamSum<WAVE, 2> sum2(lds + 32, team.lanes);
    const float inv_h = 1.0f / (float)a.H;
    int64_t row = (int64_t)blockIdx.x * team.teams + team.team;
    const int64_t step = (int64_t)gridDim.x * team.teams;
    if (row >= a.rows) return;  // the whole team, and the whole workgroup where teams meet
    constexpr int AHEAD = CH <= 2 ? 2 : 1;
    constexpr bool BUF = !WAVE && !ODD, GAINS = CH <= 2;  // GAINS: they stay in registers
    Chunk<TI> c[AHEAD][CH];
    auto fetch = [&](Chunk<TI> (&to)[CH], int64_t r) { col.load(to, a.x, r * a.ldx, r < a.rows); };
    // the stores of a row: y's, and mean and 1 / std by its first thread
    auto put = [&](int64_t r, bool some, int i, const float (&o)[8]) {
        if (!BUF || some) col.template store<Chunk<TO>>(i, a.y, r * a.ldy, o);
        else Chunk<TO>::store(raw_buffer(a.y, 0), 0, o);
    };
    auto put_stats = [&](int64_t r, bool some, float m, float rstd) {
        if constexpr (BUF) {
            some = some && a.stats;
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(m), __float_as_uint(rstd)}, raw_buffer(a.stats + (some ? 2 * r : 0), some ? 8u : 0u),
                                                  team.t * 8, 0, 0);
        } else if (some && a.stats && team.t == 0) {
            reinterpret_cast<float2 *>(a.stats)[r] = make_float2(m, rstd);
        }
    };
    // As many stores that go nowhere stand between the first rows' loads as between the
    // later ones', so that the compiler may count on them: it waits for a row's loads and
    // not for the next row's.
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
        fetch(c[k], row + k * step);
        if constexpr (BUF) {
            const float nothing[8] = {};
            put_stats(0, false, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < CH; ++i) put(0, false, i, nothing);
        }
    }
    float g[GAINS ? CH : 1][8], b[GAINS ? CH : 1][8];
#pragma unroll
    for (int i = 0; i < (GAINS ? CH : 0); ++i) col.vec(i, g[i], a.g, 1.0f), col.vec(i, b[i], a.b, 0.0f);
    if constexpr (!WAVE) {
        norm_clear(lds, 96);
        __syncthreads();
    }
    auto one = [&](Chunk<TI> (&cur)[CH]) {
        float x[CH][8], s[1] = {0.f}, s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            cur[i].get(x[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += col.counts(i, e) ? x[i][e] : 0.f;
        }
        fetch(cur, row + AHEAD * step);
        sum1(s);
        const float m = s[0] * inv_h;
        // the differences' own mean is what the mean of the values lost to rounding
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[i][e] -= m;
                const float d = col.counts(i, e) ? x[i][e] : 0.f;
                s2[0] += d;
                s2[1] = fmaf(d, d, s2[1]);
            }
        sum2(s2);
        const float dm = s2[0] * inv_h, var = fmaxf(fmaf(-dm, dm, s2[1] * inv_h), 0.f);
        const float rstd = __builtin_amdgcn_rsqf(s2[1] == s2[1] ? var + a.eps : s2[1]);  // fmaxf would drop a NaN
        put_stats(row, true, m + dm, rstd);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = GAINS ? i : 0;
            if (!GAINS) col.vec(i, g[k], a.g, 1.0f), col.vec(i, b[k], a.b, 0.0f);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf((x[i][e] - dm) * rstd, g[k][e], b[k][e]);
            put(row, true, i, o);
            if (!GAINS) __builtin_amdgcn_sched_barrier(0);  // one chunk's gains in registers at a time
        }
        row += step;
    };
    // the buffers in turn, by name: copied, a load would be waited for
    while (row < a.rows) {
        one(c[0]);
        if (AHEAD > 1 && row < a.rows) one(c[AHEAD - 1]);
    }
}

// SUMS: with the column sums of dg and db (CH = 1).  lds: 64 words for the rows' sums,
// then, for the waves' column sums, 16 words for each lane of a team.
template <class TI, class TO, int CH, bool WAVE, bool ODD, bool SUMS>
__device__ __forceinline__ void ln_bwd_body(const LnBwdArgs &k, int lanes, float *lds) {
    static_assert(CH == 1 || !SUMS, "the column sums take one chunk's registers");
    const LnArgs &a = k.f;
    const Team<WAVE> team(lanes);
    const Columns<CH, ODD, !WAVE && !ODD> col(team.t, team.lanes, a.H);
    TeamSum<WAVE, 2> sum(lds, team.lanes);
    const float inv_h = 1.0f / (float)a.H;
    int64_t row = (int64_t)blockIdx.x * team.teams + team.team;
    const int64_t step = (int64_t)gridDim.x * team.teams;
    // KEEP: a row's values stay unpacked through its sums, so that the next row's loads may take the chunks' registers
    constexpr bool KEEP = CH <= 2;
    Chunk<TI> cx[CH], cr[KEEP ? CH : 1];
    Chunk<TO> cy[CH];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t r) {
        const bool some = r < a.rows;
        col.load(cx, a.x, r * a.ldx, some);
        col.load(cy, k.dy, r * a.ldy, some);
        if constexpr (KEEP) col.load(cr, k.dres, r * a.ldx, some);
        const float2 st = reinterpret_cast<const float2 *>(a.stats)[min(r, a.rows - 1)];
        mean = st.x, rstd = st.y;
    };
    if (KEEP) fetch(row);
    float g[KEEP ? CH : 1][8], dg[8], db[8];
#pragma unroll
    for (int i = 0; i < (KEEP ? CH : 0); ++i) col.vec(i, g[i], a.g, 1.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[e] = db[e] = 0.f;
    if constexpr (!WAVE) {
        norm_clear(lds, 64);
        __syncthreads();
    }
    for (; row < a.rows; row += step) {
        if (!KEEP) fetch(row);
        float xh[KEEP ? CH : 1][8], t[KEEP ? CH : 1][8], res[KEEP ? CH : 1][8], s[2] = {0.f, 0.f};
        const float m = mean, rs = rstd;
        // xh and dy g of a chunk; not kept, they are made again for the output
        auto make = [&](int i) {
            const int k = KEEP ? i : 0;
            if (!KEEP) col.vec(i, g[k], a.g, 1.0f);
            cx[i].get(xh[k]);
            cy[i].get(t[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[k][e] = (xh[k][e] - m) * rs;
                if constexpr (SUMS) {
                    dg[e] = fmaf(t[k][e], xh[k][e], dg[e]);
                    db[e] += t[k][e];
                }
                t[k][e] *= g[k][e];
            }
        };
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = KEEP ? i : 0;
            make(i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col.counts(i, e)) {
                    s[0] += t[k][e];
                    s[1] = fmaf(t[k][e], xh[k][e], s[1]);
                }
            if (KEEP) cr[k].get(res[k]);
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
        if (KEEP) fetch(row + step);
        sum(s);
        const float c0 = s[0] * inv_h, c1 = s[1] * inv_h;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int q = KEEP ? i : 0;
            if (!KEEP) {
                make(i);
                if (k.dres && col.in(i)) cr[0].template load<ODD>(static_cast<const char *>(k.dres) + (row * a.ldx + col.at[i]) * Chunk<TI>::ES);
                cr[0].get(res[q]);
            }
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = rs * (t[q][e] - fmaf(xh[q][e], c1, c0));
                if (k.dres) o[e] += res[q][e];
            }
            // dx may take the place of dres, which the thread of the chunk before may have still to read
            col.template store<Chunk<TI>, !KEEP>(i, k.dx, row * a.ldx, o);
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (SUMS) {
        if (!k.part) return;
        float *out = k.part + (int64_t)blockIdx.x * 2 * a.H;
        auto store = [&]() {
            col.template store<Chunk<F32>>(0, out, 0, dg);
            col.template store<Chunk<F32>>(0, out, a.H, db);
        };
        if constexpr (!WAVE) {
            store();
        } else {
            // the teams of a wave, then its waves in turn
            for (int o = team.lanes; o < 64; o <<= 1)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dg[e] += __shfl_xor(dg[e], o, 64);
                    db[e] += __shfl_xor(db[e], o, 64);
                }
            const int waves = blockDim.x / 64, wave = threadIdx.x / 64;
            const bool mine = (int)(threadIdx.x & 63) < team.lanes;
            float *p = lds + 64 + team.t;
            for (int w = 0; w < waves; ++w) {
                if (wave == w && mine) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float *q = p + e * team.lanes, *r = q + 8 * team.lanes;
                        if (w) dg[e] += *q, db[e] += *r;
                        if (w + 1 < waves) *q = dg[e], *r = db[e];
                    }
                    if (w + 1 == waves) store();
                }
                __syncthreads();
            }
        }
    }
}

// dg and db of long rows, from a second reading: a workgroup of 4 waves takes 512
// columns and every 4 gridDim.y-th row, 8 columns a lane.
template <class TI, class TO, bool ODD>
__device__ __forceinline__ void ln_columns_body(const LnBwdArgs &k, float *lds) {
    const LnArgs &a = k.f;
    const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    const Columns<1, ODD, false> col(blockIdx.x * 64 + lane, 0, a.H);
    float dg[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[e] = db[e] = 0.f;
    for (int64_t row = (int64_t)blockIdx.y * 4 + wave; row < a.rows; row += 4 * (int64_t)gridDim.y) {
        Chunk<TI> cx[1];
        Chunk<TO> cy[1];
        col.load(cx, a.x, row * a.ldx);
        col.load(cy, k.dy, row * a.ldy);
        const float2 st = reinterpret_cast<const float2 *>(a.stats)[row];
        float x[8], d[8];
        cx[0].get(x);
        cy[0].get(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dg[e] = fmaf(d[e], (x[e] - st.x) * st.y, dg[e]);
            db[e] += d[e];
        }
    }
    float *out = k.part + (int64_t)blockIdx.y * 2 * a.H;
    for (int w = 0; w < 4; ++w) {
        if (wave == w) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float *q = lds + e * 64 + lane, *r = q + 512;
                if (w) dg[e] += *q, db[e] += *r;
                if (w < 3) *q = dg[e], *r = db[e];
            }
            if (w == 3) {
                col.template store<Chunk<F32>>(0, out, 0, dg);
                col.template store<Chunk<F32>>(0, out, a.H, db);
            }
        }
        __syncthreads();
    }
}

}  // namespace moe

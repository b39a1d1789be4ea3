// C-ABI entry points and kernels of a dense block's operators (gfx950): the gated
// feed-forward block, layer norm, and the clipping of gradients.  Their arguments and
// errors are documented in include/moe.h; the device code lives in dense.hpp, ffn.hpp,
// skinny.hpp, lnorm.hpp and grads.hpp.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "dense.hpp"
#include "ffn.hpp"
#include "grads.hpp"
#include "host.hpp"
#include "lnorm.hpp"
#include "skinny.hpp"

using namespace moe;

// ---------------------------------------------------------------------------
// Kernels.
// ---------------------------------------------------------------------------

namespace {

extern __shared__ char block_lds[];
__device__ __forceinline__ uint32_t block_lds_address() { return (uint32_t)(uintptr_t)(lds_char *)block_lds; }

template <class T, int MI, int NI, bool AT, bool BT, bool GLU, int STAGES, class Out>
__global__ __launch_bounds__(kDenseThreads, 1) void k_dense(DenseArgs g, Out out) {
    dense_body<T, MI, NI, AT, BT, GLU, STAGES>(g, out, block_lds_address(), blockIdx.x, gridDim.x);
}

// The gradients of both weights and of the input in one launch: none needs another, and
// shorter tiles (of fewer steps along K), which come last, fill the CUs that the last
// round of the longer ones leaves.
template <class T, int MI, int NI, int STAGES>
__global__ __launch_bounds__(kDenseThreads, 1) void k_grads(DenseArgs g1, MatOut<T> o1, int blocks1, DenseArgs g2, MatOut<T> o2, int blocks2,
                                                            DenseArgs g3, MatOut<T> o3, int blocks3, int third_first) {
    const int b = blockIdx.x - (third_first ? blocks3 : 0), c = b - blocks1, d = third_first ? (int)blockIdx.x : c - blocks2;
    if (d >= 0 && d < blocks3)
        dense_body<T, MI, NI, false, true, false, STAGES>(g3, o3, block_lds_address(), d, blocks3);
    else if (b < blocks1)
        dense_body<T, MI, NI, true, true, false, STAGES>(g1, o1, block_lds_address(), b, blocks1);
    else
        dense_body<T, MI, NI, true, true, false, STAGES>(g2, o2, block_lds_address(), c, blocks2);
}

template <class T, int NT, bool GLU>
__global__ __launch_bounds__(64 * kSkinnyWaves, 1) void k_skinny(SkinnyArgs g) {
    skinny_body<T, NT, GLU>(g, block_lds_address());
}

template <bool GLU, class Out>
__global__ __launch_bounds__(256) void k_dense_join(DenseArgs g, Out out) {
    dense_join_body<GLU>(g, out);
}

template <class TI, class TO, int CH, bool WAVE, bool ODD>
__global__ __launch_bounds__(WAVE ? 256 : 1024, !WAVE && CH == 1 && sizeof(Chunk<TI>) == 16 ? 8 : 4) void k_ln_fwd(LnArgs a, int lanes) {
    ln_fwd_body<TI, TO, CH, WAVE, ODD>(a, lanes, reinterpret_cast<float *>(block_lds));
}

template <class TI, class TO, int CH, bool WAVE, bool ODD, bool SUMS>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_ln_bwd(LnBwdArgs a, int lanes) {
    ln_bwd_body<TI, TO, CH, WAVE, ODD, SUMS>(a, lanes, reinterpret_cast<float *>(block_lds));
}

template <class TI, class TO, bool ODD>
__global__ __launch_bounds__(256) void k_ln_columns(LnBwdArgs a) {
    __shared__ float lds[1024];
    ln_columns_body<TI, TO, ODD>(a, lds);
}

template <int COLS>
__global__ __launch_bounds__(1024) void k_ln_dg(const float *part, int parts, int H, float *dg, float *db) {
    __shared__ float lds[1024];
    norm_dg_body<COLS>(part, parts, H, dg, db, lds);
}

// The launch's tensors are read where the arguments lie: indexed at run time, a copy
// would go through scratch memory.
template <class L>
__device__ __forceinline__ const __attribute__((address_space(4))) L &first_argument() {
    return *(const __attribute__((address_space(4))) L *)__builtin_amdgcn_kernarg_segment_ptr();
}

__global__ __launch_bounds__(kGradThreads) void k_grad_sums(GradLaunch<false>, GradScalars k) {
    __shared__ double lds[kGradThreads / 64];
    if (k.kind == MOE_NORM_MAX)
        grad_sums_body<true>(first_argument<GradLaunch<false>>(), k, lds);
    else
        grad_sums_body<false>(first_argument<GradLaunch<false>>(), k, lds);
}

template <bool OUT>
__global__ __launch_bounds__(kGradThreads) void k_grad_scale(GradLaunch<OUT>, GradScalars k) {
    __shared__ double lds[kGradThreads / 64];
    grad_scale_body<OUT>(first_argument<GradLaunch<OUT>>(), k, lds);
}

__global__ __launch_bounds__(kGradThreads) void k_grad_result(GradScalars k) {
    __shared__ double lds[kGradThreads / 64];
    const moe_grad_result r = grad_result(k, lds);
    if (threadIdx.x == 0) *k.result = r;
}

__global__ void k_zero_f32(float *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) p[i] = 0.f;
}

int launch_zero(float *p, int64_t words, hipStream_t s) {
    TraceScope tr("zero", s);
    hipLaunchKernelGGL(k_zero_f32, dim3((int)std::min<int64_t>((words + 255) / 256, 2048)), dim3(256), 0, s, p, words);
    return launch_status();
}

// ---------------------------------------------------------------------------
// Gated feed-forward block.
// ---------------------------------------------------------------------------

int up_to(int64_t n, int d) { return (int)((n + d - 1) / d); }

// The tiles: 64 MI x 64 NI outputs, stages of dense_loop_deep (0: dense_loop).  The 128 x 128
// tile has a short ring, so that two workgroups share a CU, and a deep one for when there
// is one at most.
enum DenseTile { kTileL, kTileS2, kTileS, kTileX, kTiles };
struct DenseShape {
    int mi, ni, stages, per_cu;
    // us: a step of 64 k with every CU at work and what a tile takes besides: of one product, and among the gradients'
    // (whose transposing reads cost small tiles more, while their ends lie beside other tiles' steps)
    float step[2], ends[2];
};
constexpr DenseShape kShape[kTiles] = {{4, 4, 0, 1, {1.4f, 1.4f}, {9.f, 8.5f}},
                                        {2, 2, 0, 2, {0.85f, 0.85f}, {6.f, 3.7f}},
                                        {2, 2, 5, 1, {0.42f, 0.5f}, {6.f, 3.6f}},
                                        {1, 2, 6, 1, {0.3f, 0.35f}, {5.f, 2.7f}}};

// A product: its sizes (GLU: N of a, B has 2 N rows), its tiles and its cut along K.
struct DensePlan {
    int M, N, K;
    bool glu;
    int mt, nt, splits, steps;
    int blocks() const { return mt * nt * splits; }
    int64_t part_bytes() const { return splits > 1 ? align256((int64_t)splits * M * N * (glu ? 2 : 1) * 4) : 0; }
    int all_steps() const { return std::max(1, up_to(K, kDenseK)); }
};
DensePlan dense_product(int M, int N, int K, bool glu = false) { return DensePlan{M, N, K, glu, 0, 0, 1, 0}; }

// The tile for the products of one launch, and their cuts along K: the least of the times
// estimated from a step's and a tile's measured ones (kShape) for each choice.  One product
// goes in rounds of the tiles that the CUs hold, where a CU with one of its two tiles
// takes 0.6 of the time; several, by the sum of their tiles' times and part of the
// longest's.  A cut costs the second pass (kJoin and the parts' bytes); one product's stays within one round, of
// several a long one (X's gradient of few rows) is cut among the others' many short tiles.  Measured against the
// others forced, us, 256 x 256 / 128 x 128 shared / alone / 64 x 128, taken in brackets:
// up of 333 rows (H 1032, I 520) 30 / 13 / 13 / [10], of 1,021 (2056, 1032) 55 / 27 / [25] / 36, of 600
// (4096, 4096) 87 / [56] / 69 / 75, of 3,000 (2048, 1024) 54 / [34] / 40 / 46, of 8,192 (7168, 2048) [366] / 460; of 128
// rows (7168, 2048) uncut 125 / 60 / 48 / 37, in four parts of K [16 + 5]; gradients of 256 rows (4096, 4096) uncut
// 170 / 121 / 99 / 121, in four parts 70 / [66] / 85 / 124 and 6 for the join, of 1,024 (7168, 2048) [149] / 155 / 185 / 280,
// of 8,192 (2048, 1024) 179 / [163] / 191 / 282.  A 128 x 256 tile was
// never ahead of the better of its neighbours by more than 6%.
DenseTile dense_plan(DensePlan *p, int n) {
    constexpr float kJoin = 5.f, kPerMiB = 0.4f;
    constexpr int kCus = 256;  // of every gfx950; also where a workspace is sized without one
    DenseTile best = kTileL;
    float least = 1e30f;
    DensePlan chosen[3];
    for (int t = 0; t < kTiles; ++t) {
        const DenseShape &k = kShape[t];
        for (int cut = 1; cut <= 16; cut *= 2) {
            DensePlan q[3];
            float sum = 0.f, most = 0.f, join = 0.f;
            int blocks = 0;
            bool useful = cut == 1;
            for (int i = 0; i < n; ++i) {
                q[i] = p[i];
                q[i].mt = up_to(q[i].M, 64 * k.mi);
                q[i].nt = up_to(q[i].N, (q[i].glu ? 32 : 64) * k.ni);
                const int all = q[i].all_steps();
                q[i].steps = std::max(4, up_to(all, cut));
                q[i].splits = up_to(all, q[i].steps);
                if (q[i].splits == 1) q[i].steps = all;
                useful |= q[i].splits > 1;
                const float one = q[i].steps * k.step[n > 1] + k.ends[n > 1];
                sum += one * q[i].blocks();
                most = std::max(most, one);
                blocks += q[i].blocks();
                if (q[i].splits > 1) join += kJoin + kPerMiB * (float)(q[i].part_bytes() >> 20);
            }
            if (!useful || (n == 1 && cut > 1 && blocks > kCus * k.per_cu)) break;
            const int room = kCus * k.per_cu;
            const int rest = blocks % room;
            float time = join;
            if (n > 1)
                time += std::max(most, sum / room + 0.3f * most);
            else
                time += most * ((float)(blocks / room) + (rest == 0 ? 0.f : rest <= kCus && k.per_cu > 1 ? 0.6f : 1.f));
            if (time < least) {
                least = time;
                best = (DenseTile)t;
                std::copy(q, q + n, chosen);
            }
        }
    }
    std::copy(chosen, chosen + n, p);
    return best;
}

DenseArgs dense_args(const DensePlan &p, const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, void *part) {
    return DenseArgs{A, B, lda, ldb, p.M, p.N, p.K, p.mt, p.nt, p.splits, p.steps, static_cast<float *>(part)};
}

size_t dense_lds(DenseTile t) { return dense_lds_bytes(kShape[t].mi, kShape[t].ni, kShape[t].stages); }

template <class T, bool AT, bool BT, bool GLU, class Out>
auto *dense_kernel(DenseTile t) {
    return t == kTileL    ? k_dense<T, 4, 4, AT, BT, GLU, kShape[kTileL].stages, Out>
           : t == kTileS2 ? k_dense<T, 2, 2, AT, BT, GLU, kShape[kTileS2].stages, Out>
           : t == kTileS  ? k_dense<T, 2, 2, AT, BT, GLU, kShape[kTileS].stages, Out>
                          : k_dense<T, 1, 2, AT, BT, GLU, kShape[kTileX].stages, Out>;
}
template <class T>
auto *grads_kernel(DenseTile t) {
    return t == kTileL    ? k_grads<T, 4, 4, kShape[kTileL].stages>
           : t == kTileS2 ? k_grads<T, 2, 2, kShape[kTileS2].stages>
           : t == kTileS  ? k_grads<T, 2, 2, kShape[kTileS].stages>
                          : k_grads<T, 1, 2, kShape[kTileX].stages>;
}

template <bool GLU, class Out>
int launch_join(const DensePlan &p, const DenseArgs &g, const Out &out, hipStream_t s) {
    if (p.splits == 1) return MOE_OK;
    TraceScope tr("dense_join", s);
    auto *join = k_dense_join<GLU, Out>;
    const int64_t n = (int64_t)g.M * (g.N / 8);
    hipLaunchKernelGGL(join, dim3((int)std::min<int64_t>((n + 255) / 256, 2048)), dim3(256), 0, s, g, out);
    return launch_status();
}

template <class T, bool AT, bool BT, bool GLU, class Out>
int launch_dense(DenseTile t, const DensePlan &p, const DenseArgs &g, const Out &out, hipStream_t s, const char *name) {
    {
        TraceScope tr(name, s);
        auto *fn = dense_kernel<T, AT, BT, GLU, Out>(t);
        hipLaunchKernelGGL(fn, dim3(p.blocks()), dim3(kDenseThreads), dense_lds(t), s, g, out);
    }
    const int rc = launch_status();
    return rc != MOE_OK ? rc : launch_join<GLU>(p, g, out, s);
}

int64_t ffn_ldx(const moe_ffn_desc *n) { return n->ldx ? n->ldx : n->H; }
int64_t ffn_ldo(const moe_ffn_desc *n) { return n->ldo ? n->ldo : n->H; }

int ffn_check(const moe_ffn_desc *n) {
    if (!n || n->rows < 0 || n->H < 1 || n->I < 1 || n->act < MOE_ACT_SILU || n->act > MOE_ACT_RELU ||
        (n->type != MOE_TYPE_BF16 && n->type != MOE_TYPE_FP16) || n->ldx < 0 || n->ldo < 0 || ffn_ldx(n) < n->H || ffn_ldo(n) < n->H)
        return MOE_EINVAL;
    // a tile's rows, and 64 rows of an MN-contiguous operand, are raw buffers below 2 GiB; a grid has less than 2^32
    // threads, 2^24 tiles (of 128 x 128, 64 columns of a, where there are that many)
    constexpr int64_t kLd = 1 << 20;
    if (n->H % 8 || n->I % 8 || n->H > 65536 || n->I > 65536 || n->ldx % 8 || n->ldo % 8 || ffn_ldx(n) > kLd || ffn_ldo(n) > kLd ||
        (int64_t)n->H * n->I >= (1ll << 30) || n->rows >= (1ll << 30) || n->rows * std::max(n->H, 2 * n->I) >= (1ll << 36))
        return MOE_EUNSUPPORTED;
    return MOE_OK;
}

// A few rows go by the weights' stream.  Both products, us, by it / by dense_plan's tiles cut along K: H = 7168, I = 2048,
// 8 rows 22 / 36, 32 rows 29 / 37, 64 rows 38 / 40; H = 2048, I = 1024, 8 rows 10 / 23, 64 rows 15 / 27.
constexpr int kSkinnyRows = 64;
bool ffn_skinny(const moe_ffn_desc *n) { return n->rows <= kSkinnyRows; }

// dHU and a (where it was not kept), then the parts of a launch's products
int64_t ffn_bwd_base(const moe_ffn_desc *n) { return align256(n->rows * 4 * n->I) + align256(n->rows * 2 * n->I); }

// Forward: gate / up, down.  Backward: activations; then the gradients of W13, W2 and X in one launch.
struct FfnFwdPlan {
    DensePlan up, down;
    DenseTile tup, tdown;
    explicit FfnFwdPlan(const moe_ffn_desc *n)
        : up(dense_product((int)n->rows, n->I, n->H, true)), down(dense_product((int)n->rows, n->H, n->I)), tup(dense_plan(&up, 1)),
          tdown(dense_plan(&down, 1)) {}
    int64_t ws_bytes() const { return std::max(up.part_bytes(), down.part_bytes()); }
};
struct FfnBwdPlan {
    DensePlan act, g[3];
    DenseTile tact, tg;
    explicit FfnBwdPlan(const moe_ffn_desc *n)
        : act(dense_product((int)n->rows, n->I, n->H)),
          g{dense_product(2 * n->I, n->H, (int)n->rows), dense_product(n->H, n->I, (int)n->rows), dense_product((int)n->rows, n->H, 2 * n->I)},
          tact(dense_plan(&act, 1)), tg(dense_plan(g, 3)) {}
    int64_t ws_bytes() const { return std::max(act.part_bytes(), g[0].part_bytes() + g[1].part_bytes() + g[2].part_bytes()); }
};
int64_t ffn_ws_bytes(const moe_ffn_desc *n, bool bwd) {
    if (n->rows == 0) return 0;
    if (bwd) return ffn_bwd_base(n) + FfnBwdPlan(n).ws_bytes();
    return ffn_skinny(n) ? 0 : FfnFwdPlan(n).ws_bytes();
}

// Whether no output starts where an input or another output does (NULL: not there).
bool ffn_apart(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o)
        if (*o && (std::find(ins.begin(), ins.end(), *o) != ins.end() || std::find(o + 1, outs.end(), *o) != outs.end())) return false;
    return true;
}

template <class T, bool GLU>
int launch_skinny(const SkinnyArgs &g, hipStream_t s, const char *name) {
    const int units = up_to(g.N, GLU ? 8 : 16);
    const int nt = g.M <= 16 ? 1 : g.M <= 32 ? 2 : 4;
    TraceScope tr(name, s);
    auto *fn = nt == 1 ? k_skinny<T, 1, GLU> : nt == 2 ? k_skinny<T, 2, GLU> : k_skinny<T, 4, GLU>;
    hipLaunchKernelGGL(fn, dim3(units), dim3(64 * kSkinnyWaves), skinny_lds(nt), s, g);
    return launch_status();
}

template <class T>
int ffn_fwd(const moe_ffn_desc *n, const uint16_t *X, const uint16_t *W13, const uint16_t *W2, uint16_t *HU, uint16_t *A,
            uint16_t *out, void *ws, hipStream_t s) {
    const int R = (int)n->rows, H = n->H, I = n->I;
    if (ffn_skinny(n)) {
        const int rc = launch_skinny<T, true>(SkinnyArgs{X, W13, ffn_ldx(n), H, R, I, H, A, I, HU, n->act}, s, "ffn_up");
        if (rc != MOE_OK) return rc;
        return launch_skinny<T, false>(SkinnyArgs{A, W2, I, I, R, H, I, out, ffn_ldo(n), nullptr, 0}, s, "ffn_down");
    }
    const FfnFwdPlan p(n);
    const DenseArgs up = dense_args(p.up, X, ffn_ldx(n), W13, H, ws);
    const int rc = launch_dense<T, false, false, true>(p.tup, p.up, up, GluOut<T>{HU, A, I, n->act}, s, "ffn_up");
    if (rc != MOE_OK) return rc;
    const DenseArgs down = dense_args(p.down, A, I, W2, I, ws);
    return launch_dense<T, false, false, false>(p.tdown, p.down, down, MatOut<T>{out, ffn_ldo(n), 0, 0}, s, "ffn_down");
}

template <class T>
int ffn_bwd(const moe_ffn_desc *n, const uint16_t *dOut, const uint16_t *X, const uint16_t *HU, const uint16_t *A, const uint16_t *W13,
            const uint16_t *W2, uint16_t *dX, void *dW13, void *dW2, int f32, int add, void *ws, hipStream_t s) {
    FfnBwdPlan p(n);
    const int H = n->H, I = n->I;
    const int64_t ldx = ffn_ldx(n), ldo = ffn_ldo(n);
    char *w = static_cast<char *>(ws);
    uint16_t *dHU = reinterpret_cast<uint16_t *>(w), *a = reinterpret_cast<uint16_t *>(w + align256(n->rows * 4 * n->I));
    char *part = w + ffn_bwd_base(n);
    const DenseArgs act = dense_args(p.act, dOut, ldo, W2, I, part);
    int rc = launch_dense<T, false, true, false>(p.tact, p.act, act, GluBwdOut<T>{HU, dHU, A || !dW2 ? nullptr : a, I, n->act}, s, "ffn_bwd_act");
    if (rc != MOE_OK) return rc;
    const DenseArgs g[3] = {dense_args(p.g[0], dHU, 2 * I, X, ldx, part), dense_args(p.g[1], dOut, ldo, A ? A : a, I, part + p.g[0].part_bytes()),
                            dense_args(p.g[2], dHU, 2 * I, W13, H, part + p.g[0].part_bytes() + p.g[1].part_bytes())};
    const MatOut<T> o[3] = {{dW13, H, f32, add}, {dW2, I, f32, add}, {dX, ldx, 0, 0}};
    int blocks[3];
    for (int i = 0; i < 3; ++i) blocks[i] = o[i].p ? p.g[i].blocks() : 0;
    {
        TraceScope tr("ffn_bwd_grads", s);
        auto *fn = grads_kernel<T>(p.tg);
        hipLaunchKernelGGL(fn, dim3(blocks[0] + blocks[1] + blocks[2]), dim3(kDenseThreads), dense_lds(p.tg), s, g[0], o[0], blocks[0], g[1], o[1],
                           blocks[1], g[2], o[2], blocks[2], (int)(p.g[2].steps > p.g[0].steps));
    }
    rc = launch_status();
    for (int i = 0; i < 3 && rc == MOE_OK; ++i)
        if (o[i].p) rc = launch_join<false>(p.g[i], g[i], o[i], s);
    return rc;
}

// ---------------------------------------------------------------------------
// Layer norm.
// ---------------------------------------------------------------------------

int64_t ln_ldx(const moe_ln_desc *n) { return n->ldx ? n->ldx : n->H; }
int64_t ln_ldy(const moe_ln_desc *n) { return n->ldy ? n->ldy : n->H; }
// Rows up to 512 elements are a wave's (8 columns a lane at most): us forward / backward against a workgroup for each,
// 100,000 rows of 128 13 / 17 against 33 / 147, 60,000 of 512 22 / 27 against 27 / 91.
constexpr int kLnWaveH = 512, kLnMaxH = 32768, kLnSumH = 8192;

int ln_check(const moe_ln_desc *n) {
    if (!n || n->rows < 0 || n->H < 1 || n->ldx < 0 || n->ldy < 0 || ln_ldx(n) < n->H || ln_ldy(n) < n->H || !(n->eps >= 0.0f) ||
        n->x_type < MOE_TYPE_BF16 || n->x_type > MOE_TYPE_FP32 || n->y_type < MOE_TYPE_BF16 || n->y_type > MOE_TYPE_FP32)
        return MOE_EINVAL;
    if (n->H > kLnMaxH || n->rows > (1ll << 40) || ln_ldx(n) > (1ll << 40) || ln_ldy(n) > (1ll << 40) ||
        (n->x_type != n->y_type && n->x_type != MOE_TYPE_FP32))
        return MOE_EUNSUPPORTED;
    return MOE_OK;
}

// Whether the rows of y's side may take the place of those of x's.
bool ln_same_rows(const moe_ln_desc *n) { return n->x_type == n->y_type && ln_ldx(n) == ln_ldy(n); }

// How a row is shared out.
struct LnPlan {
    bool wave;
    int chunks, lanes, threads, teams;  // 8-column chunks per thread, threads per row and per workgroup, rows per workgroup
};
LnPlan ln_plan(const moe_ln_desc *n) {
    LnPlan p;
    const int c = (n->H + 7) / 8;
    p.wave = n->H <= kLnWaveH;
    if (p.wave) {
        p.chunks = 1;
        p.lanes = 8;
        while (p.lanes < c) p.lanes *= 2;
        p.threads = 256;
        p.teams = p.threads / p.lanes;
    } else {
        p.chunks = n->H <= 8192 ? 1 : n->H <= 16384 ? 2 : 4;
        p.lanes = p.threads = (c + 64 * p.chunks - 1) / (64 * p.chunks) * 64;
        p.teams = 1;
    }
    return p;
}

// Workgroups of the backward: each leaves one row of column sums.
int ln_groups(const moe_ln_desc *n) {
    const LnPlan p = ln_plan(n);
    if (p.wave) return (int)std::max<int64_t>(1, std::min<int64_t>((n->rows + 4 * p.teams - 1) / (4 * p.teams), 1024));
    // Two on a CU, one of more than 512 threads (half as many: 16,384 rows of 7168 118 -> 218 us, twice: 124 and 2 more
    // for the pass over the sums).  Four of up to 256 threads with 16-bit rows, 16 each, which pay for their sums (us
    // with that pass, two / four: 16,384 rows of 2048 43 / 42, 20,000 of 1536 47 / 42, 30,000 of 1024 61 / 44, where
    // eight take 47; 1,000 rows of 2048 14 / 19; 30,000 of 1024 in fp32 83 / 88).
    const int64_t groups = p.threads > 512 ? 256 : p.threads <= 256 && n->x_type != MOE_TYPE_FP32 && n->rows >= 16 * 1024 ? 1024 : 512;
    return (int)std::max<int64_t>(1, std::min<int64_t>(n->rows, groups));
}
// rows of sums of the long rows' second reading
int ln_column_groups(const moe_ln_desc *n) { return (int)std::max<int64_t>(1, std::min<int64_t>((n->rows + 15) / 16, 64)); }
int ln_parts(const moe_ln_desc *n) { return n->H <= kLnSumH ? ln_groups(n) : ln_column_groups(n); }
int64_t ln_ws_bytes(const moe_ln_desc *n) { return n->rows ? align256((int64_t)ln_parts(n) * 2 * n->H * 4) : 0; }

// Whether every row of p starts on 16 bytes and ends on a whole chunk.
bool ln_even(const moe_ln_desc *n, const void *p, int64_t ld) { return !p || (n->H % 8 == 0 && ld % 8 == 0 && aligned16(p)); }
bool ln_aligned(const void *p, int type) { return ((uintptr_t)p & (type == MOE_TYPE_FP32 ? 3u : 1u)) == 0; }

template <class TI, class TO, bool ODD>
auto *ln_fwd_kernel(const LnPlan &p) {
    if (p.wave) return k_ln_fwd<TI, TO, 1, true, ODD>;
    return p.chunks == 1   ? k_ln_fwd<TI, TO, 1, false, ODD>
           : p.chunks == 2 ? k_ln_fwd<TI, TO, 2, false, ODD>
                           : k_ln_fwd<TI, TO, 4, false, ODD>;
}
template <class TI, class TO, bool ODD>
auto *ln_bwd_kernel(const LnPlan &p) {
    if (p.wave) return k_ln_bwd<TI, TO, 1, true, ODD, true>;
    return p.chunks == 1   ? k_ln_bwd<TI, TO, 1, false, ODD, true>
           : p.chunks == 2 ? k_ln_bwd<TI, TO, 2, false, ODD, false>
                           : k_ln_bwd<TI, TO, 4, false, ODD, false>;
}

// f of the types and whether the rows are odd
template <class F>
int ln_typed(const moe_ln_desc *n, bool odd, F &&f) {
    auto with = [&](auto ti, auto to) { return odd ? f(ti, to, std::true_type{}) : f(ti, to, std::false_type{}); };
    if (n->x_type == MOE_TYPE_BF16) return with(Bf16{}, Bf16{});
    if (n->x_type == MOE_TYPE_FP16) return with(Fp16{}, Fp16{});
    if (n->y_type == MOE_TYPE_BF16) return with(F32{}, Bf16{});
    if (n->y_type == MOE_TYPE_FP16) return with(F32{}, Fp16{});
    return with(F32{}, F32{});
}

// ---------------------------------------------------------------------------
// Gradients.
// ---------------------------------------------------------------------------

// few elements (up to what a launch's workgroups take in one small piece each): small pieces
int grad_shift(const moe_grad *t, int32_t n) {
    int64_t all = 0;
    for (int i = 0; i < n; ++i) all += t[i].numel;
    return all <= (int64_t)kGradParts << kGradShiftFew ? kGradShiftFew : kGradShift;
}

int grad_check(const moe_grad *t, int32_t n, bool out) {
    if (n < 0 || (n > 0 && !t)) return MOE_EINVAL;
    int64_t all = 0;
    for (int i = 0; i < n; ++i) {
        const moe_grad &k = t[i];
        if (k.numel < 0 || k.type < MOE_TYPE_BF16 || k.type > MOE_TYPE_FP32 || k.reserved) return MOE_EINVAL;
        if (k.numel >= (1ll << 44)) return MOE_EUNSUPPORTED;
        if (k.numel == 0) continue;
        if (!k.g || !ln_aligned(k.g, k.type) || (out && (!k.out || !ln_aligned(k.out, k.type)))) return MOE_EINVAL;
        if ((uint64_t)(uintptr_t)k.g >> 48) return MOE_EUNSUPPORTED;
        all += k.numel;
        if (all >= (1ll << 44)) return MOE_EUNSUPPORTED;
    }
    return MOE_OK;
}
bool grad_scalars_ok(int32_t kind, float scale, float max_norm, float eps) {
    return (kind == MOE_NORM_L2 || kind == MOE_NORM_MAX) && scale == scale && max_norm >= 0.f && eps >= 0.f;
}

// Tensors [*at, n) that a launch takes, as many as fit; false when none is left.
template <bool OUT>
bool grad_fill(GradLaunch<OUT> &l, const moe_grad *t, int32_t n, int32_t *at, int shift) {
    l.count = 0;
    l.shift = shift;
    int64_t pieces = 0;
    for (; *at < n && l.count < l.N; ++*at) {
        const moe_grad &k = t[*at];
        if (!k.numel) continue;
        if constexpr (OUT) l.out[l.count] = k.out;
        l.start[l.count] = (int32_t)pieces;
        l.t[l.count++] = grad_tensor(k.g, k.numel, k.type);
        pieces += (k.numel + (1ll << shift) - 1) >> shift;
    }
    l.pieces = (int32_t)pieces;
    return l.count > 0;
}

int grad_launches(int32_t n) { return (n + kGradTensors - 1) / kGradTensors; }
int64_t grad_ws_bytes(int32_t n) { return 8ll * kGradParts * std::max(1, grad_launches(n)); }

int launch_grad_sums(const moe_grad *t, int32_t n, GradScalars &k, hipStream_t s) {
    double *parts = k.parts;
    GradLaunch<false> l;
    const int shift = grad_shift(t, n);
    for (int32_t at = 0; grad_fill(l, t, n, &at, shift);) {
        const int grid = std::min(l.pieces, kGradParts);
        GradScalars a = k;
        a.parts = parts;
        {
            TraceScope tr("grad_sums", s);
            hipLaunchKernelGGL(k_grad_sums, dim3(grid), dim3(kGradThreads), 0, s, l, a);
        }
        if (launch_status() != MOE_OK) return MOE_EHIP;
        parts += grid;
    }
    k.nparts = (int32_t)(parts - k.parts);
    return MOE_OK;
}

int launch_grad_result(const GradScalars &k, hipStream_t s) {
    TraceScope tr("grad_result", s);
    hipLaunchKernelGGL(k_grad_result, dim3(1), dim3(kGradThreads), 0, s, k);
    return launch_status();
}

template <bool OUT>
int launch_grad_scale_as(const moe_grad *t, int32_t n, const GradScalars &k, hipStream_t s) {
    GradLaunch<OUT> l;
    const int shift = grad_shift(t, n);
    // from the last tensors to the first, as within a launch: the cache holds what was read last
    for (int32_t end = n; end > 0;) {
        int32_t begin = end, taken = 0;
        while (begin > 0 && taken < l.N) taken += t[--begin].numel > 0;
        int32_t at = begin;
        if (grad_fill(l, t, end, &at, shift)) {
            const int grid = std::min(l.pieces, 8 * device_cus());
            TraceScope tr("grad_scale", s);
            hipLaunchKernelGGL(k_grad_scale<OUT>, dim3(grid), dim3(kGradThreads), 0, s, l, k);
            if (launch_status() != MOE_OK) return MOE_EHIP;
        }
        end = begin;
    }
    return MOE_OK;
}
int launch_grad_scale(const moe_grad *t, int32_t n, const GradScalars &k, hipStream_t s) {
    bool own = true;
    for (int32_t i = 0; i < n; ++i) own &= t[i].numel == 0 || t[i].out == t[i].g;
    return own ? launch_grad_scale_as<false>(t, n, k, s) : launch_grad_scale_as<true>(t, n, k, s);
}

}  // namespace

extern "C" {

int64_t moe_gated_ffn_workspace_bytes(const moe_ffn_desc *n, int32_t bwd) {
    return ffn_check(n) == MOE_OK && (bwd == 0 || bwd == 1) ? ffn_ws_bytes(n, bwd) : -1;
}

int moe_gated_ffn_fwd(const moe_ffn_desc *n, const uint16_t *X, const uint16_t *W13, const uint16_t *W2, uint16_t *HU, uint16_t *A,
                      uint16_t *out, void *ws, size_t ws_bytes, void *stream) {
    const int rc = ffn_check(n);
    if (rc != MOE_OK) return rc;
    if (n->rows == 0) return MOE_OK;
    if (!X || !W13 || !W2 || !A || !out || !all_aligned({X, W13, W2, HU, A, out, ws})) return MOE_EINVAL;
    const int64_t need = ffn_ws_bytes(n, false);
    if (need && !ws) return MOE_EINVAL;
    // out may take the place of X, which its launch no longer reads
    if (!ffn_apart({HU, A, out, need ? ws : nullptr}, {W13, W2}) || !ffn_apart({HU, A, need ? ws : nullptr}, {X})) return MOE_EINVAL;
    if ((int64_t)ws_bytes < need) return MOE_ENOSPC;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return n->type == MOE_TYPE_BF16 ? ffn_fwd<Bf16>(n, X, W13, W2, HU, A, out, ws, s) : ffn_fwd<Fp16>(n, X, W13, W2, HU, A, out, ws, s);
}

int moe_gated_ffn_bwd(const moe_ffn_desc *n, const uint16_t *dOut, const uint16_t *X, const uint16_t *HU, const uint16_t *A,
                      const uint16_t *W13, const uint16_t *W2, uint16_t *dX, void *dW13, void *dW2, int32_t dw_type, int32_t accumulate,
                      void *ws, size_t ws_bytes, void *stream) {
    const int rc = ffn_check(n);
    if (rc != MOE_OK) return rc;
    if ((dw_type != MOE_TYPE_FP32 && dw_type != n->type) || (accumulate != 0 && accumulate != 1)) return MOE_EINVAL;
    if (accumulate && dw_type != MOE_TYPE_FP32) return MOE_EUNSUPPORTED;
    if (!all_aligned({dW13, dW2})) return MOE_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (n->rows == 0) {
        if (accumulate) return MOE_OK;
        const int64_t words = (int64_t)n->H * n->I / (dw_type == MOE_TYPE_FP32 ? 1 : 2);
        int r = dW13 ? launch_zero(static_cast<float *>(dW13), 2 * words, s) : MOE_OK;
        if (r == MOE_OK && dW2) r = launch_zero(static_cast<float *>(dW2), words, s);
        return r;
    }
    if (!dOut || !X || !HU || !W13 || !W2 || !ws || !all_aligned({dOut, X, HU, A, W13, W2, dX, ws})) return MOE_EINVAL;
    if (!dX && !dW13 && !dW2) return MOE_EINVAL;
    if (!ffn_apart({dX, dW13, dW2, ws}, {dOut, X, HU, A, W13, W2})) return MOE_EINVAL;  // one launch reads and writes them
    if ((int64_t)ws_bytes < ffn_ws_bytes(n, true)) return MOE_ENOSPC;
    const int f32 = dw_type == MOE_TYPE_FP32;
    return n->type == MOE_TYPE_BF16 ? ffn_bwd<Bf16>(n, dOut, X, HU, A, W13, W2, dX, dW13, dW2, f32, accumulate, ws, s)
                                    : ffn_bwd<Fp16>(n, dOut, X, HU, A, W13, W2, dX, dW13, dW2, f32, accumulate, ws, s);
}

int64_t moe_layer_norm_workspace_bytes(const moe_ln_desc *n) { return ln_check(n) == MOE_OK ? ln_ws_bytes(n) : -1; }

int moe_layer_norm_fwd(const moe_ln_desc *n, const void *x, const float *g, const float *b, void *y, float *stats, void *stream) {
    const int rc = ln_check(n);
    if (rc != MOE_OK) return rc;
    if (n->rows == 0) return MOE_OK;
    if (!x || !y || !ln_aligned(x, n->x_type) || !ln_aligned(y, n->y_type) || !aligned4(g) || !aligned4(b) || ((uintptr_t)stats & 7u) ||
        (y == x && !ln_same_rows(n)))
        return MOE_EINVAL;
    const LnPlan p = ln_plan(n);
    const LnArgs a{x, g, b, y, stats, n->rows, ln_ldx(n), ln_ldy(n), n->H, n->eps};
    const bool odd = !ln_even(n, x, a.ldx) || !ln_even(n, y, a.ldy) || !all_aligned({g, b});
    // all that a CU holds: with half of them 16,384 rows of 7168 take 92 us for 85, of 7,171 116 for 108
    const int64_t per_cu = p.wave ? 8 : std::max(1, (p.chunks == 1 && n->x_type != MOE_TYPE_FP32 ? 2048 : 1024) / p.threads);
    const int grid = (int)std::min<int64_t>((n->rows + p.teams - 1) / p.teams, per_cu * device_cus());
    hipStream_t s = static_cast<hipStream_t>(stream);
    return ln_typed(n, odd, [&](auto ti, auto to, auto is_odd) {
        TraceScope tr("layer_norm_fwd", s);
        auto *fn = ln_fwd_kernel<decltype(ti), decltype(to), decltype(is_odd)::value>(p);
        hipLaunchKernelGGL(fn, dim3(grid), dim3(p.threads), p.wave ? 0 : 384, s, a, p.lanes);
        return launch_status();
    });
}

int moe_layer_norm_bwd(const moe_ln_desc *n, const void *x, const float *g, const float *stats, const void *dy, const void *dres,
                       void *dx, float *dg, float *db, void *ws, size_t ws_bytes, void *stream) {
    const int rc = ln_check(n);
    if (rc != MOE_OK) return rc;
    if (!dg != !db || !aligned4(dg) || !aligned4(db)) return MOE_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (n->rows > 0) {
        if (!x || !stats || !dy || !dx || !ln_aligned(x, n->x_type) || !ln_aligned(dy, n->y_type) || !ln_aligned(dres, n->x_type) ||
            !ln_aligned(dx, n->x_type) || !aligned4(g) || ((uintptr_t)stats & 7u) || !aligned16(ws) ||
            (dx == dy && !ln_same_rows(n)))
            return MOE_EINVAL;
        if (dg && !ws) return MOE_EINVAL;
        if (dg && (int64_t)ws_bytes < ln_ws_bytes(n)) return MOE_ENOSPC;
        const LnPlan p = ln_plan(n);
        const bool long_rows = n->H > kLnSumH;
        LnBwdArgs a{LnArgs{x, g, nullptr, nullptr, const_cast<float *>(stats), n->rows, ln_ldx(n), ln_ldy(n), n->H, n->eps}, dy, dres, dx,
                    dg ? static_cast<float *>(ws) : nullptr};
        const bool odd = !ln_even(n, x, a.f.ldx) || !ln_even(n, dy, a.f.ldy) || !ln_even(n, dres, a.f.ldx) || !ln_even(n, dx, a.f.ldx) ||
                         !aligned16(g);
        const int grid = ln_groups(n);
        const size_t lds = 256 + (p.wave ? 64 * (size_t)p.lanes : 0);
        int r = ln_typed(n, odd, [&](auto ti, auto to, auto is_odd) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr bool ODD = decltype(is_odd)::value;
            if (long_rows && dg) {  // before dx, which may take the place of an input
                TraceScope tr("layer_norm_columns", s);
                auto *fn = k_ln_columns<TI, TO, ODD>;
                hipLaunchKernelGGL(fn, dim3((n->H + 511) / 512, ln_column_groups(n)), dim3(256), 0, s, a);
                if (launch_status() != MOE_OK) return (int)MOE_EHIP;
            }
            TraceScope tr("layer_norm_bwd", s);
            auto *fn = ln_bwd_kernel<TI, TO, ODD>(p);
            hipLaunchKernelGGL(fn, dim3(grid), dim3(p.threads), lds, s, a, p.lanes);
            return launch_status();
        });
        if (r != MOE_OK) return r;
    }
    if (!dg) return MOE_OK;
    TraceScope tr("layer_norm_dg", s);
    const int parts = n->rows ? ln_parts(n) : 0;
    auto *fn = n->H < 2048 ? k_ln_dg<16> : k_ln_dg<64>;
    const int cols = n->H < 2048 ? 16 : 64;
    hipLaunchKernelGGL(fn, dim3((n->H + cols - 1) / cols, 2), dim3(1024), 0, s, static_cast<const float *>(ws), parts, n->H, dg, db);
    return launch_status();
}

int64_t moe_grad_workspace_bytes(int32_t n) { return n >= 0 ? grad_ws_bytes(n) : -1; }

static int grad_norm_check(const moe_grad *t, int32_t n, int32_t kind, float scale, float max_norm, float eps, const void *result,
                           const void *ws, size_t ws_bytes, bool out) {
    const int rc = grad_check(t, n, out);
    if (rc != MOE_OK) return rc;
    if (!grad_scalars_ok(kind, scale, max_norm, eps) || !result || ((uintptr_t)result & 7u) || !ws || ((uintptr_t)ws & 7u)) return MOE_EINVAL;
    return (int64_t)ws_bytes < grad_ws_bytes(n) ? MOE_ENOSPC : MOE_OK;
}

int moe_grad_norm(const moe_grad *t, int32_t n, int32_t kind, float scale, float max_norm, float eps, moe_grad_result *result, void *ws,
                  size_t ws_bytes, void *stream) {
    int rc = grad_norm_check(t, n, kind, scale, max_norm, eps, result, ws, ws_bytes, false);
    if (rc != MOE_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    GradScalars k{static_cast<double *>(ws), result, nullptr, 0, kind, scale, max_norm, eps};
    rc = launch_grad_sums(t, n, k, s);
    return rc != MOE_OK ? rc : launch_grad_result(k, s);
}

int moe_grad_clip(const moe_grad *t, int32_t n, int32_t kind, float scale, float max_norm, float eps, moe_grad_result *result, void *ws,
                  size_t ws_bytes, void *stream) {
    int rc = grad_norm_check(t, n, kind, scale, max_norm, eps, result, ws, ws_bytes, true);
    if (rc != MOE_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    GradScalars k{static_cast<double *>(ws), result, nullptr, 0, kind, scale, max_norm, eps};
    rc = launch_grad_sums(t, n, k, s);
    if (rc != MOE_OK) return rc;
    // one launch's slots are added by every workgroup of the second pass; more than that, once
    const bool alone = k.nparts > kGradParts || k.nparts == 0;
    if (alone) {
        rc = launch_grad_result(k, s);
        if (rc != MOE_OK) return rc;
        k.coef = &result->coef;
    }
    return launch_grad_scale(t, n, k, s);
}

int moe_grad_scale(const moe_grad *t, int32_t n, const float *coef, float scale, void *stream) {
    const int rc = grad_check(t, n, true);
    if (rc != MOE_OK) return rc;
    if (!coef || !aligned4(coef) || scale != scale) return MOE_EINVAL;
    GradScalars k{nullptr, nullptr, coef, 0, MOE_NORM_L2, scale, 0.f, 0.f};
    return launch_grad_scale(t, n, k, static_cast<hipStream_t>(stream));
}

}  // extern "C"

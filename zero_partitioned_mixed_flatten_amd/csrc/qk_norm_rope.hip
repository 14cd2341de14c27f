// qk_norm_rope.hip -- the norms of queries and keys over each head, and the
// position rotation in the same pass, forward and backward.
//
//   rstd = 1 / sqrt(mean(x^2) + eps),  h = x rstd,  u = h w,  y = R u
//   backward: g' = R^T dy,  dw = sum over tokens and heads of g' h,  g = g' w,
//             dx = rstd (g - h mean(g h))
// R turns the first `rot` elements of a head in pairs by the token's position;
// cosines and sines come from a table.  The backward pass takes rstd from x
// again: a head's sum of squares is there before dy is.
//
// Bound by memory: one read and one write of everything, with both tensors in
// one launch.
#include "attention.hpp"

namespace zero {
namespace attention {
namespace {

constexpr int kQkBlock = 256;
constexpr uint32_t kMaxQkDim = 256;

template <typename T>
struct QkSide {                                    // one of the two tensors
    T* out;                                        // y, or dx
    const T* x;
    const T* dy;                                   // backward only
    const void* w;
    uint64_t ld_out, hs_out, ld_x, hs_x, ld_dy, hs_dy;
    uint32_t heads;
};

template <typename T>
struct QkArgs {
    QkSide<T> side[2];
    uint64_t tokens;
    uint32_t dim, rot;
    bool vec_f32, interleaved;
    float eps;
    const float* table;                            // table_rows x rot / 2 x (cos, sin)
    uint64_t table_rows, period;
    const int32_t* positions;
    float* partials;                               // backward: blocks of q, then of k, x dim
    uint32_t blocks[2];
};

// A thread holds 16 bytes at each of two places of a head, so that it has
// whole pairs: of a turned half-split head the same part of both halves.
// Elements past `rot` are taken alike, as two halves of what is left.
template <typename T>
struct Part2 {
    static constexpr int kPer = 16 / sizeof(T);
    typedef T V __attribute__((ext_vector_type(kPer)));
    typedef V VU __attribute__((aligned(sizeof(T))));
    uint32_t at[2];                                // first columns
    bool turned;

    __device__ __forceinline__ Part2(uint32_t t, uint32_t dim, uint32_t rot)
    {
        const uint32_t parts = rot / (2 * kPer);
        turned = t < parts;
        at[0] = turned ? t * kPer : rot + (t - parts) * kPer;
        at[1] = at[0] + (turned ? rot / 2 : (dim - rot) / 2);
    }
    template <bool PAST>
    __device__ __forceinline__ void load(const T* p, float (&v)[2][kPer]) const
    {
        V r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = PAST ? V(__builtin_nontemporal_load(reinterpret_cast<const VU*>(p + at[i]))) : V(*reinterpret_cast<const VU*>(p + at[i]));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                v[i][j] = float(r[i][j]);
    }
    __device__ __forceinline__ void store(T* p, const float (&v)[2][kPer]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            V r;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                r[j] = T(v[i][j]);
            __builtin_nontemporal_store(r, reinterpret_cast<VU*>(p + at[i]));
        }
    }
    __device__ __forceinline__ void weights(const void* w, bool f32, float (&v)[2][kPer]) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                v[i][j] = 1.0f;
        if (!w)
            return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (f32) {
                typedef float F __attribute__((ext_vector_type(kPer)));
                typedef F FU __attribute__((aligned(4)));
                const F r = *reinterpret_cast<const FU*>(static_cast<const float*>(w) + at[i]);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    v[i][j] = r[j];
            } else {
                const V r = *reinterpret_cast<const VU*>(static_cast<const T*>(w) + at[i]);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    v[i][j] = float(r[j]);
            }
    }
};

template <typename T>
__device__ __forceinline__ const float* turn_row(const QkArgs<T>& a, uint64_t token, bool& known)
{
    uint64_t pos;
    if (a.positions) {
        const int32_t p = a.positions[token];
        pos = p < 0 ? ~uint64_t(0) : uint64_t(p);
    } else {
        pos = a.period ? token % a.period : token;
    }
    known = pos < a.table_rows;
    return a.table + (known ? pos : 0) * a.rot;
}

// Turns v by the row's angles, or back.
template <typename T, int PER>
__device__ __forceinline__ void turn(float (&v)[2][PER], const float* row, bool known, const Part2<T>& at, bool interleaved, bool back)
{
    typedef float F0 __attribute__((ext_vector_type(2 * PER)));
    typedef float H0 __attribute__((ext_vector_type(PER)));
    typedef F0 F __attribute__((aligned(16)));
    typedef H0 H __attribute__((aligned(16)));
    if (!at.turned)
        return;
    float cs[2 * PER];                             // cosine and sine of the thread's PER pairs
    if (interleaved) {
        const H x = *reinterpret_cast<const H*>(row + at.at[0]), y = *reinterpret_cast<const H*>(row + at.at[1]);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            cs[j] = x[j];
            cs[PER + j] = y[j];
        }
    } else {
        const F x = *reinterpret_cast<const F*>(row + 2 * at.at[0]);
#pragma unroll
        for (int j = 0; j < 2 * PER; ++j)
            cs[j] = x[j];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const float c = known ? cs[2 * j] : __builtin_nanf(""), s = back ? -cs[2 * j + 1] : cs[2 * j + 1];
        float& x = interleaved ? v[2 * j / PER][2 * j % PER] : v[0][j];
        float& y = interleaved ? v[2 * j / PER][2 * j % PER + 1] : v[1][j];
        const float p = x, q = y;
        x = __builtin_fmaf(p, c, -(q * s));
        y = __builtin_fmaf(q, c, p * s);
    }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v)
{
    if (LANES >= 2) v += layer::dpp<0xB1>(v);      // lane ^ 1
    if (LANES >= 4) v += layer::dpp<0x4E>(v);      // lane ^ 2
    if (LANES >= 8) v += layer::dpp<0x141>(v);     // the other quad of 8
    if (LANES >= 16) v += layer::dpp<0x140>(v);    // the other 8 of 16
    if (LANES >= 32) v += __shfl_xor(v, 16);
    return v;
}

template <int PER>
__device__ __forceinline__ float dot(const float (&a)[2][PER], const float (&b)[2][PER])
{
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        s0 = __builtin_fmaf(a[0][j], b[0][j], s0);
        s1 = __builtin_fmaf(a[1][j], b[1][j], s1);
    }
    return s0 + s1;
}

// LANES threads a head; STYLE 0: pairs of halves, 1: neighbours.
template <typename T, int LANES, int STYLE, bool PAST>
__global__ __launch_bounds__(kQkBlock) void qk_fwd_kernel(QkArgs<T> a)
{
    constexpr int kPer = Part2<T>::kPer, kItems = kQkBlock / LANES;
    const uint32_t heads = a.side[0].heads + a.side[1].heads;
    const uint64_t base = uint64_t(blockIdx.x) * kItems, token0 = base / heads;
    const uint32_t local = uint32_t(base - token0 * heads) + threadIdx.x / LANES, skip = local / heads;
    const uint64_t token = token0 + skip;
    uint32_t head = local - skip * heads;
    const uint32_t t = threadIdx.x % LANES;
    const bool active = token < a.tokens && t * 2 * kPer < a.dim;
    const bool second = head >= a.side[0].heads;
    const QkSide<T> side = second ? a.side[1] : a.side[0];
    head -= second ? a.side[0].heads : 0;
    const Part2<T> at(t, a.dim, a.rot);
    float x[2][kPer] = {}, w[2][kPer];
    const float* row = nullptr;
    bool known = true;
    if (active) {
        at.template load<PAST>(side.x + token * side.ld_x + head * side.hs_x, x);
        if (a.rot)
            row = turn_row(a, token, known);
        at.weights(side.w, a.vec_f32, w);
    }
    const float mean = group_sum<LANES>(dot(x, x)) / float(a.dim);
    if (!active)
        return;
    const float rstd = 1.0f / sqrtf(mean + a.eps);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            x[i][j] = x[i][j] * rstd * w[i][j];
    turn(x, row, known, at, STYLE != 0, false);
    at.store(side.out + token * side.ld_out + head * side.hs_out, x);
}

template <typename T, int LANES, int STYLE, bool PAST>
__global__ __launch_bounds__(kQkBlock) void qk_bwd_kernel(QkArgs<T> a)
{
    constexpr int kPer = Part2<T>::kPer, kItems = kQkBlock / LANES;
    __shared__ float sums[kQkBlock / 64][64 * 2 * kPer];
    const bool second = blockIdx.x >= a.blocks[0];
    const QkSide<T> side = second ? a.side[1] : a.side[0];
    const uint32_t block = blockIdx.x - (second ? a.blocks[0] : 0), blocks = second ? a.blocks[1] : a.blocks[0];
    const uint32_t t = threadIdx.x % LANES;
    const bool inside = t * 2 * kPer < a.dim;
    const Part2<T> at(t, a.dim, a.rot);
    float w[2][kPer], dw[2][kPer] = {};
    if (inside)
        at.weights(side.w, a.vec_f32, w);
    const uint64_t stride = uint64_t(blocks) * kItems, start = uint64_t(block) * kItems + threadIdx.x / LANES;
    const uint64_t step_token = stride / side.heads;
    const uint32_t step_head = uint32_t(stride - step_token * side.heads);
    uint64_t token = start / side.heads;
    uint32_t head = uint32_t(start - token * side.heads);
    const float inv = 1.0f / float(a.dim);
    while (__any(token < a.tokens)) {
        const bool active = inside && token < a.tokens;
        float x[2][kPer] = {}, g[2][kPer] = {};
        if (active) {
            at.template load<PAST>(side.x + token * side.ld_x + head * side.hs_x, x);
            at.template load<PAST>(side.dy + token * side.ld_dy + head * side.hs_dy, g);
            if (a.rot) {
                bool known;
                const float* row = turn_row(a, token, known);
                turn(g, row, known, at, STYLE != 0, true);
            }
        }
        const float rstd = 1.0f / sqrtf(group_sum<LANES>(dot(x, x)) / float(a.dim) + a.eps);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                x[i][j] *= rstd;
                dw[i][j] = __builtin_fmaf(g[i][j], x[i][j], dw[i][j]);
                g[i][j] = active ? g[i][j] * w[i][j] : 0.0f;
            }
        const float mean = group_sum<LANES>(dot(g, x)) * inv;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                g[i][j] = rstd * __builtin_fmaf(-x[i][j], mean, g[i][j]);
        if (active)
            at.store(side.out + token * side.ld_out + head * side.hs_out, g);
        token += step_token;
        head += step_head;
        if (head >= side.heads) {
            head -= side.heads;
            ++token;
        }
    }
    if (!a.partials)
        return;
    // the wave's heads, then the waves
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            float v = dw[i][j];
#pragma unroll
            for (int lane = LANES; lane < 64; lane <<= 1)
                v += __shfl_xor(v, lane);
            dw[i][j] = v;
        }
    const uint32_t wave = threadIdx.x / 64;
    if (threadIdx.x % 64 < LANES && inside)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                sums[wave][at.at[i] + j] = dw[i][j];
    __syncthreads();
    if (threadIdx.x < a.dim)
        a.partials[uint64_t(blockIdx.x) * a.dim + threadIdx.x] =
            (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

// Any even dim and rot, by elements: 16 threads a head, each with every 16th
// pair.  Elements past rot go in neighbouring pairs that are not turned.
constexpr int kAnyLanes = 16, kAnyPairs = kMaxQkDim / 2 / kAnyLanes;

template <typename T, bool BWD>
__global__ __launch_bounds__(kQkBlock) void qk_any_kernel(QkArgs<T> a)
{
    constexpr int kItems = kQkBlock / kAnyLanes;
    __shared__ float sums[kQkBlock / 64][kMaxQkDim];
    const bool second = blockIdx.x >= a.blocks[0];
    const QkSide<T> side = second ? a.side[1] : a.side[0];
    const uint32_t block = blockIdx.x - (second ? a.blocks[0] : 0), blocks = second ? a.blocks[1] : a.blocks[0];
    const uint32_t t = threadIdx.x % kAnyLanes, half = a.rot / 2;
    uint32_t lo[kAnyPairs], hi[kAnyPairs];
    float w[kAnyPairs][2], dw[kAnyPairs][2] = {};
#pragma unroll
    for (int i = 0; i < kAnyPairs; ++i) {
        const uint32_t pair = t + i * kAnyLanes;
        const bool split = pair < half && !a.interleaved;
        lo[i] = split ? pair : 2 * pair;
        hi[i] = split ? pair + half : 2 * pair + 1;
        const bool in = pair < a.dim / 2;
        auto value = [&](uint32_t col) {
            return !in || !side.w ? 1.0f : a.vec_f32 ? static_cast<const float*>(side.w)[col] : float(static_cast<const T*>(side.w)[col]);
        };
        w[i][0] = value(lo[i]);
        w[i][1] = value(hi[i]);
    }
    const uint64_t items = a.tokens * side.heads;
    const float n = float(a.dim);
    for (uint64_t item = uint64_t(block) * kItems + threadIdx.x / kAnyLanes; __any(item < items); item += uint64_t(blocks) * kItems) {
        const bool live = item < items;
        const uint64_t token = live ? item / side.heads : 0;
        const uint32_t head = live ? uint32_t(item - token * side.heads) : 0;
        const T* src = side.x + token * side.ld_x + head * side.hs_x;
        float x[kAnyPairs][2], g[kAnyPairs][2], s = 0.0f;
        bool known = true;
        const float* row = a.rot ? turn_row(a, token, known) : nullptr;
#pragma unroll
        for (int i = 0; i < kAnyPairs; ++i) {
            const bool in = live && t + i * kAnyLanes < a.dim / 2;
            x[i][0] = in ? float(src[lo[i]]) : 0.0f;
            x[i][1] = in ? float(src[hi[i]]) : 0.0f;
            s = __builtin_fmaf(x[i][0], x[i][0], s);
            s = __builtin_fmaf(x[i][1], x[i][1], s);
        }
        const float rstd = 1.0f / sqrtf(group_sum<kAnyLanes>(s) / n + a.eps);
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < kAnyPairs; ++i) {
            const uint32_t pair = t + i * kAnyLanes;
            const bool in = live && pair < a.dim / 2, turned = in && pair < half;
            float c = 1.0f, sn = 0.0f;
            if (turned) {
                c = known ? row[2 * pair] : __builtin_nanf("");
                sn = row[2 * pair + 1];
            }
            x[i][0] *= rstd;
            x[i][1] *= rstd;
            float p, q;
            if (BWD) {
                const T* dy = side.dy + token * side.ld_dy + head * side.hs_dy;
                p = in ? float(dy[lo[i]]) : 0.0f;
                q = in ? float(dy[hi[i]]) : 0.0f;
                sn = -sn;
            } else {
                p = x[i][0] * w[i][0];
                q = x[i][1] * w[i][1];
            }
            g[i][0] = turned ? __builtin_fmaf(p, c, -(q * sn)) : p;
            g[i][1] = turned ? __builtin_fmaf(q, c, p * sn) : q;
            if (BWD)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    dw[i][e] = __builtin_fmaf(g[i][e], x[i][e], dw[i][e]);
                    g[i][e] *= w[i][e];
                    mean = __builtin_fmaf(g[i][e], x[i][e], mean);
                }
        }
        if (BWD)
            mean = group_sum<kAnyLanes>(mean) / n;
        T* dst = side.out + token * side.ld_out + head * side.hs_out;
#pragma unroll
        for (int i = 0; i < kAnyPairs; ++i) {
            if (!(live && t + i * kAnyLanes < a.dim / 2))
                continue;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                dst[e ? hi[i] : lo[i]] = T(BWD ? rstd * __builtin_fmaf(-x[i][e], mean, g[i][e]) : g[i][e]);
        }
    }
    if (!BWD || !a.partials)
        return;
#pragma unroll
    for (int i = 0; i < kAnyPairs; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = dw[i][e];
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            if (threadIdx.x % 64 < kAnyLanes && t + i * kAnyLanes < a.dim / 2)
                sums[threadIdx.x / 64][e ? hi[i] : lo[i]] = v;
        }
    __syncthreads();
    if (threadIdx.x < a.dim)
        a.partials[uint64_t(blockIdx.x) * a.dim + threadIdx.x] =
            (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

// The weights' gradients: the workgroups' partials added up in their order.
constexpr int kQkFoldCols = 8, kQkFoldRows = 128;

template <typename T>
__global__ __launch_bounds__(kQkFoldCols* kQkFoldRows) void qk_fold_kernel(void* dwq, void* dwk, bool f32, bool accumulate,
                                                                         const float* partials, uint32_t blocks_q, uint32_t blocks_k,
                                                                         uint32_t dim)
{
    __shared__ float part[kQkFoldRows][kQkFoldCols];
    void* dst = blockIdx.y ? dwk : dwq;
    if (!dst)
        return;
    const uint32_t c = threadIdx.x % kQkFoldCols, r = threadIdx.x / kQkFoldCols, col = blockIdx.x * kQkFoldCols + c;
    const uint32_t first = blockIdx.y ? blocks_q : 0, n = blockIdx.y ? blocks_k : blocks_q;
    float v = 0.0f;
    if (col < dim)
        for (uint32_t i = r; i < n; i += kQkFoldRows)
            v += partials[uint64_t(first + i) * dim + col];
    part[r][c] = v;
    for (int rows = kQkFoldRows / 2; rows; rows >>= 1) {
        __syncthreads();
        if (int(r) < rows)
            part[r][c] += part[r + rows][c];
    }
    if (r || col >= dim)
        return;
    v = part[0][c];
    if (f32) {
        float* d = static_cast<float*>(dst) + col;
        *d = accumulate ? *d + v : v;
    } else {
        T* d = static_cast<T*>(dst) + col;
        *d = T(accumulate ? float(*d) + v : v);
    }
}

__global__ __launch_bounds__(256) void rope_table_kernel(float* table, uint64_t entries, uint32_t half, double log2_base)
{
    const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= entries)
        return;
    const uint64_t pos = i / half;
    const uint32_t p = uint32_t(i - pos * half);
    double s, c;
    sincos(double(pos) * exp2(-log2_base * p / half), &s, &c);
    table[2 * i] = float(c);
    table[2 * i + 1] = float(s);
}

// ---- host side --------------------------------------------------------------------------
struct QkTensor {
    void* out;
    uint64_t ld_out, hs_out;
    const void* x;
    uint64_t ld_x, hs_x;
    const void* dy;
    uint64_t ld_dy, hs_dy;
    const void* w;
    uint32_t heads;
};

struct QkCall {
    QkTensor side[2];
    int vec_dtype;
    uint64_t tokens;
    uint32_t dim;
    int dtype;
    double eps;
    const float* table;
    uint64_t table_rows;
    uint32_t rot;
    bool interleaved;
    const int32_t* positions;
    uint64_t period;
    // backward
    void* dw[2];
    int grad_dtype;
    bool accumulate;
    void* workspace;
    size_t workspace_bytes;
};

// Workgroups of a backward pass for one tensor: each has a partial sum of the
// weights' gradient, so no more than keep the card busy.
constexpr uint64_t kQkBlocks = 2048;

uint32_t bwd_blocks(uint64_t tokens, uint32_t heads, uint32_t all, uint32_t items)
{
    if (!heads)
        return 0;
    const uint64_t need = (tokens * heads + items - 1) / items;
    uint64_t most = (kQkBlocks * heads + all - 1) / all;
    return uint32_t(need < most ? need : most);
}

uint64_t qk_workspace(uint64_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim)
{
    // the fewest heads that any form gives a workgroup
    const uint64_t q = bwd_blocks(tokens, heads, heads + kv_heads, kQkBlock / 32), k = bwd_blocks(tokens, kv_heads, heads + kv_heads, kQkBlock / 32);
    return (q + k) * dim * 4;
}

template <typename T, bool BWD, int LANES, int STYLE>
void launch_part(const QkArgs<T>& a, uint64_t blocks, bool past, hipStream_t s)
{
    if constexpr (BWD) {
        if (past)
            hipLaunchKernelGGL((qk_bwd_kernel<T, LANES, STYLE, true>), dim3(uint32_t(blocks)), dim3(kQkBlock), 0, s, a);
        else
            hipLaunchKernelGGL((qk_bwd_kernel<T, LANES, STYLE, false>), dim3(uint32_t(blocks)), dim3(kQkBlock), 0, s, a);
    } else {
        if (past)
            hipLaunchKernelGGL((qk_fwd_kernel<T, LANES, STYLE, true>), dim3(uint32_t(blocks)), dim3(kQkBlock), 0, s, a);
        else
            hipLaunchKernelGGL((qk_fwd_kernel<T, LANES, STYLE, false>), dim3(uint32_t(blocks)), dim3(kQkBlock), 0, s, a);
    }
}

template <typename T, bool BWD>
int run_qk(const QkCall& c, hipStream_t s)
{
    QkArgs<T> a{};
    const uint32_t all = c.side[0].heads + c.side[1].heads;
    for (int i = 0; i < 2; ++i) {
        const QkTensor& t = c.side[i];
        a.side[i] = QkSide<T>{static_cast<T*>(t.out), static_cast<const T*>(t.x), static_cast<const T*>(t.dy), t.w, t.ld_out, t.hs_out,
                              t.ld_x, t.hs_x, t.ld_dy, t.hs_dy, t.heads};
    }
    a.tokens = c.tokens;
    a.dim = c.dim;
    a.rot = c.rot;
    a.vec_f32 = c.vec_dtype == ZERO_F32;
    a.interleaved = c.interleaved;
    a.eps = float(c.eps);
    a.table = c.table;
    a.table_rows = c.table_rows;
    a.period = c.period;
    a.positions = c.positions;
    a.partials = c.dw[0] || c.dw[1] ? static_cast<float*>(c.workspace) : nullptr;
    constexpr uint32_t kSpan = 2 * Part2<T>::kPer;
    const uint32_t threads = c.dim / kSpan;
    const bool parts = c.dim % kSpan == 0 && c.rot % kSpan == 0;
    uint32_t lanes = parts ? 1 : kAnyLanes;
    while (parts && lanes < threads)
        lanes *= 2;
    const uint32_t items = kQkBlock / lanes;
    uint64_t blocks;
    if (BWD || !parts) {
        for (int i = 0; i < 2; ++i)
            a.blocks[i] = bwd_blocks(c.tokens, c.side[i].heads, all, items);
        blocks = uint64_t(a.blocks[0]) + a.blocks[1];
    } else {
        blocks = (c.tokens * all + items - 1) / items;
    }
    // what is read once goes past the caches where it does not fit them anyway
    const bool past = c.tokens * all * c.dim * sizeof(T) * (BWD ? 3 : 2) > layer::kStreamBytes;
    if (c.tokens) {
        if (!parts) {
            hipLaunchKernelGGL((qk_any_kernel<T, BWD>), dim3(uint32_t(blocks)), dim3(kQkBlock), 0, s, a);
        } else {
            auto go = [&](auto style) {
                constexpr int kStyle = decltype(style)::value;
                switch (lanes) {
                case 1: launch_part<T, BWD, 1, kStyle>(a, blocks, past, s); break;
                case 2: launch_part<T, BWD, 2, kStyle>(a, blocks, past, s); break;
                case 4: launch_part<T, BWD, 4, kStyle>(a, blocks, past, s); break;
                case 8: launch_part<T, BWD, 8, kStyle>(a, blocks, past, s); break;
                case 16: launch_part<T, BWD, 16, kStyle>(a, blocks, past, s); break;
                default: launch_part<T, BWD, 32, kStyle>(a, blocks, past, s); break;
                }
            };
            if (c.interleaved)
                go(std::integral_constant<int, 1>{});
            else
                go(std::integral_constant<int, 0>{});
        }
        const int rc = launch_status();
        if (rc)
            return rc;
    }
    if (!BWD || !(c.dw[0] || c.dw[1]))
        return ZERO_OK;
    hipLaunchKernelGGL(qk_fold_kernel<T>, dim3((c.dim + kQkFoldCols - 1) / kQkFoldCols, 2), dim3(kQkFoldCols * kQkFoldRows), 0, s, c.dw[0],
                       c.dw[1], c.grad_dtype == ZERO_F32, c.accumulate, a.partials, a.blocks[0], a.blocks[1], c.dim);
    return launch_status();
}

template <bool BWD>
int dispatch_qk(const QkCall& c, void* stream)
{
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (c.dtype) {
    case ZERO_F16: return run_qk<_Float16, BWD>(c, s);
    case ZERO_BF16: return run_qk<bf16, BWD>(c, s);
    default: return run_qk<float, BWD>(c, s);
    }
}

int check_qk(const QkCall& c, bool bwd)
{
    if (!layer::dtype_ok(c.dtype) || !c.side[0].heads || !c.dim || c.dim % 2 || c.rot % 2 || c.rot > c.dim)
        return ZERO_EINVAL;
    const float eps = float(c.eps);
    if (!(eps > 0.0f) || !isfinite(eps))
        return ZERO_EINVAL;
    if (c.dim > kMaxQkDim || c.tokens > kMaxTokens || c.side[0].heads > kMaxHeads || c.side[1].heads > kMaxHeads || c.table_rows > kMaxTokens)
        return ZERO_ERANGE;
    // a forward pass gives a workgroup at least 8 heads
    if (c.tokens * (c.side[0].heads + uint64_t(c.side[1].heads)) > uint64_t(0x7fffffff) * 8)
        return ZERO_ERANGE;
    for (const QkTensor& t : c.side) {
        if (!t.heads) {
            if (t.out || t.x || t.dy || t.w)
                return ZERO_EINVAL;
            continue;
        }
        int rc = check_heads(t.out, t.ld_out, t.hs_out, c.tokens, t.heads, c.dim, c.dtype);
        if (!rc) rc = check_heads(t.x, t.ld_x, t.hs_x, c.tokens, t.heads, c.dim, c.dtype);
        if (!rc && bwd) rc = check_heads(t.dy, t.ld_dy, t.hs_dy, c.tokens, t.heads, c.dim, c.dtype);
        if (!rc) rc = layer::check_vector(t.w, c.vec_dtype, c.dtype);
        if (rc)
            return rc;
    }
    if (c.tokens && c.side[0].out == c.side[1].out)
        return ZERO_EINVAL;
    if (c.rot && (!c.table || !c.table_rows))
        return ZERO_EINVAL;
    // entries are read up to 16 at a time
    if (!is_aligned(c.table, 16) || !is_aligned(c.positions, 4))
        return ZERO_EALIGN;
    if (!bwd)
        return ZERO_OK;
    for (int i = 0; i < 2; ++i) {
        const int rc = layer::check_vector(c.dw[i], c.grad_dtype, c.dtype);
        if (rc)
            return rc;
    }
    if ((c.dw[0] && c.dw[0] == c.dw[1]) || (c.dw[1] && !c.side[1].heads))
        return ZERO_EINVAL;
    if (c.tokens && (c.dw[0] || c.dw[1])) {
        if (!c.workspace)
            return ZERO_EINVAL;
        if (!is_aligned(c.workspace, 16))
            return ZERO_EALIGN;
        if (c.workspace_bytes < qk_workspace(c.tokens, c.side[0].heads, c.side[1].heads, c.dim))
            return ZERO_ERANGE;
    }
    return ZERO_OK;
}

}  // namespace
}  // namespace attention
}  // namespace zero

using namespace zero;
using namespace zero::attention;

extern "C" int zero_rope_table(float* table, uint64_t positions, uint32_t rot, double base, void* stream)
{
    if (!(base > 0.0) || !isfinite(base) || rot % 2 || (positions && rot && !table))
        return ZERO_EINVAL;
    if (!is_aligned(table, 16))
        return ZERO_EALIGN;
    if (positions > kMaxTokens || rot > kMaxQkDim)
        return ZERO_ERANGE;
    const uint64_t entries = positions * (rot / 2);
    if (!entries)
        return ZERO_OK;
    hipLaunchKernelGGL(rope_table_kernel, dim3(uint32_t((entries + 255) / 256)), dim3(256), 0, static_cast<hipStream_t>(stream), table, entries,
                       rot / 2, log2(base));
    return launch_status();
}

extern "C" size_t zero_qk_workspace_bytes(uint64_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim)
{
    if (tokens > kMaxTokens || heads > kMaxHeads || kv_heads > kMaxHeads || dim > kMaxQkDim)
        return 0;
    return size_t(qk_workspace(tokens, heads, kv_heads, dim));
}

extern "C" int zero_qk_norm_rope_fwd(void* q_out, uint64_t ld_q_out, uint64_t hs_q_out, void* k_out, uint64_t ld_k_out, uint64_t hs_k_out,
                                     const void* q, uint64_t ld_q, uint64_t hs_q, const void* k, uint64_t ld_k, uint64_t hs_k,
                                     const void* wq, const void* wk, int vec_dtype, uint64_t tokens, uint32_t heads, uint32_t kv_heads,
                                     uint32_t dim, int dtype, double eps, const float* table, uint64_t table_rows, uint32_t rot,
                                     int interleaved, const int32_t* dev_positions, uint64_t period, void* stream)
{
    const QkCall c{{{q_out, ld_q_out, hs_q_out, q, ld_q, hs_q, nullptr, 0, 0, wq, heads}, {k_out, ld_k_out, hs_k_out, k, ld_k, hs_k, nullptr, 0, 0, wk, kv_heads}},
                   vec_dtype, tokens, dim, dtype, eps, table, table_rows, rot, interleaved != 0, dev_positions, period, {nullptr, nullptr}, 0,
                   false, nullptr, 0};
    const int rc = check_qk(c, false);
    return rc || !tokens ? rc : dispatch_qk<false>(c, stream);
}

extern "C" int zero_qk_norm_rope_bwd(void* dq, uint64_t ld_dq, uint64_t hs_dq, void* dk, uint64_t ld_dk, uint64_t hs_dk, void* dwq, void* dwk,
                                     int grad_dtype, int accumulate, const void* dq_out, uint64_t ld_dq_out, uint64_t hs_dq_out,
                                     const void* dk_out, uint64_t ld_dk_out, uint64_t hs_dk_out, const void* q, uint64_t ld_q,
                                     uint64_t hs_q, const void* k, uint64_t ld_k, uint64_t hs_k, const void* wq, const void* wk,
                                     int vec_dtype, uint64_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, int dtype, double eps,
                                     const float* table, uint64_t table_rows, uint32_t rot, int interleaved, const int32_t* dev_positions,
                                     uint64_t period, void* workspace, size_t workspace_bytes, void* stream)
{
    const QkCall c{{{dq, ld_dq, hs_dq, q, ld_q, hs_q, dq_out, ld_dq_out, hs_dq_out, wq, heads},
                    {dk, ld_dk, hs_dk, k, ld_k, hs_k, dk_out, ld_dk_out, hs_dk_out, wk, kv_heads}},
                   vec_dtype, tokens, dim, dtype, eps, table, table_rows, rot, interleaved != 0, dev_positions, period, {dwq, dwk}, grad_dtype,
                   accumulate != 0, workspace, workspace_bytes};
    const int rc = check_qk(c, true);
    if (rc)
        return rc;
    if (!tokens && (c.accumulate || !(dwq || dwk)))
        return ZERO_OK;
    return dispatch_qk<true>(c, stream);
}

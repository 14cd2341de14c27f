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
// One read and one write of everything, with both tensors in one launch.  8192
// tokens of 2 x 25 heads of 64, binary16: 22.6 us forward, 38.2 backward with the
// fold of the weights' gradients (34 and 4), 4.7 and 4.2 TB/s; a plain copy of
// the forward pass's bytes takes 17-19.  What is above the copy is a wave's
// start (weights, position, angles: loads that wait for one another) and vector
// instructions, 60% of the issue slots.  16384 tokens of 72 heads of 128, bfloat16,
// backward: 168-172 us, 5.3 TB/s.
#include <type_traits>

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
    float* partials;                               // backward: blocks x dim (qk_token_kernel: for each q, then k)
    uint32_t blocks[2];
    uint32_t split;
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

// A dimension of a launch holds fewer than 2^32 threads: more workgroups than
// 2^22 are dealt out over two.
dim3 flat_grid(uint64_t blocks)
{
    const uint64_t x = blocks < (uint64_t(1) << 22) ? blocks : uint64_t(1) << 22;
    return dim3(uint32_t(x), uint32_t((blocks + x - 1) / x));
}
__device__ __forceinline__ uint64_t flat_block() { return uint64_t(blockIdx.y) * gridDim.x + blockIdx.x; }

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

// 1 / sqrt(v), one step off at most; v below the normal numbers (a tiny eps and a head of zeros) by the long way.
__device__ __forceinline__ float inverse_root(float v)
{
    return v >= 0x1p-126f ? __builtin_amdgcn_rsqf(v) : 1.0f / sqrtf(v);
}

// ---- heads that turn wholly or not at all --------------------------------------------
// A wave has a token (or one of `split` parts of its heads): its angles are in
// registers for all heads, and addresses are a scalar base plus a lane's
// constant.  LANES lanes have a head, 16 bytes each, so that an access takes
// whole 128-byte lines.  The halves of a pair of a half-split head are then in
// different lanes: the upper half's pieces are taken in reverse, so that a
// piece's partner is in the mirrored lane, and the product with the partner is
// one instruction (DPP).  What it is against is vector instructions: 275 for 16
// binary16 elements of a lane with both halves of a head in a thread (an access
// of which leaves half of each line to the next), 23 us forward and 43 backward
// at 8192 tokens of 2 x 25 heads of 64.
template <typename T>
struct Piece16 {
    static constexpr int kPer = 16 / sizeof(T);
    typedef T V __attribute__((ext_vector_type(kPer)));
    typedef V VU __attribute__((aligned(sizeof(T))));
};

template <int LANES>
__device__ __forceinline__ float mirrored(float v)
{
    if (LANES == 2) return layer::dpp<0xB1>(v);
    if (LANES == 4) return layer::dpp<0x1B>(v);
    if (LANES == 8) return layer::dpp<0x141>(v);
    return layer::dpp<0x140>(v);
}

// STYLE 0: not turned, 1: pairs of halves, 2: neighbours.
template <typename T, int LANES, int STYLE, bool PAST, bool BWD>
__global__ __launch_bounds__(kQkBlock) void qk_token_kernel(QkArgs<T> a)
{
    typedef Piece16<T> P;
    typedef typename P::V V;
    typedef typename P::VU VU;
    constexpr int kPer = P::kPer, kHeads = 64 / LANES;             // heads of an access
    constexpr int kBatch = BWD ? 2 : 4;
    __shared__ float sums[BWD ? kQkBlock / 64 : 1][2][BWD ? LANES * kPer : 1];
    const uint32_t lane = threadIdx.x % 64, i = lane % LANES, sub = lane / LANES;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const bool high = STYLE == 1 && i >= LANES / 2;
    const uint32_t piece = high ? 3 * LANES / 2 - 1 - i : i;
    float w[2][kPer], dw[2][kPer] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const void* p = a.side[n].w;
        if (p && a.vec_f32) {
            typedef float F __attribute__((ext_vector_type(kPer)));
            typedef F FU __attribute__((aligned(4)));
            const F r = *reinterpret_cast<const FU*>(static_cast<const float*>(p) + piece * kPer);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                w[n][j] = r[j];
        } else if (p) {
            const V r = *reinterpret_cast<const VU*>(static_cast<const T*>(p) + piece * kPer);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                w[n][j] = float(r[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                w[n][j] = 1.0f;
        }
    }
    const float inv = 1.0f / float(LANES * kPer);
    const uint64_t units = a.tokens * a.split;
    for (uint64_t u = uint64_t(blockIdx.x) * (kQkBlock / 64) + wave; u < units; u += uint64_t(gridDim.x) * (kQkBlock / 64)) {
        const uint64_t token = a.split == 1 ? u : u / a.split;
        const uint32_t part = uint32_t(u - token * a.split);
        float c[kPer], s[kPer];                    // of each element's pair, the sine as it comes with the partner
        if (STYLE != 0) {
            bool known;
            const float* row = turn_row(a, token, known);
            if (STYLE == 1) {
                const uint32_t first = (high ? piece - LANES / 2 : piece) * kPer;
#pragma unroll
                for (int j = 0; j < kPer; j += 2) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(row + 2 * (first + j));
                    c[j] = v[0];
                    s[j] = high != BWD ? v[1] : -v[1];
                    c[j + 1] = v[2];
                    s[j + 1] = high != BWD ? v[3] : -v[3];
                }
            } else {
#pragma unroll
                for (int j = 0; j < kPer; j += 4) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(row + piece * kPer + j);
                    c[j] = c[j + 1] = v[0];
                    s[j] = BWD ? v[1] : -v[1];
                    s[j + 1] = -s[j];
                    c[j + 2] = c[j + 3] = v[2];
                    s[j + 2] = BWD ? v[3] : -v[3];
                    s[j + 3] = -s[j + 2];
                }
            }
            if (!known)
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    c[j] = __builtin_nanf("");
        }
        auto turned = [&](float (&v)[kPer]) {
            if (STYLE == 0)
                return;
            float p[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                p[j] = (STYLE == 1 ? mirrored<LANES>(v[j]) : v[j ^ 1]) * s[j];
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                v[j] = __builtin_fmaf(v[j], c[j], p[j]);
        };
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const QkSide<T>& side = a.side[n];
            const uint32_t accesses = (side.heads + kHeads - 1) / kHeads;
            uint32_t k = a.split == 1 ? 0 : accesses * part / a.split;
            const uint32_t end = a.split == 1 ? accesses : accesses * (part + 1) / a.split;
            auto at = [&](uint64_t hs, uint32_t access) {          // the lane's element, from the token's; heads past the last read that
                const uint32_t head = access * kHeads + sub;
                return (head < side.heads ? head : side.heads - 1) * uint32_t(hs) + piece * kPer;
            };
            auto read = [&](const T* p, uint64_t ld, uint64_t hs, uint32_t access) {
                const VU* from = reinterpret_cast<const VU*>(p + token * ld + at(hs, access));
                return PAST ? V(__builtin_nontemporal_load(from)) : V(*from);
            };
            for (; k < end; k += kBatch) {
                V raw[kBatch], grad[kBatch];       // a batch of accesses in flight together
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    raw[e] = read(side.x, side.ld_x, side.hs_x, k + e < end ? k + e : end - 1);
                    if (BWD)
                        grad[e] = read(side.dy, side.ld_dy, side.hs_dy, k + e < end ? k + e : end - 1);
                }
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    if (k + e >= end)
                        break;
                    const V rx = raw[e], rg = BWD ? grad[e] : raw[e];
                    const bool live = (k + e) * kHeads + sub < side.heads;
                    float x[kPer], g[kPer], q = 0.0f;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        x[j] = float(rx[j]);
                        q = __builtin_fmaf(x[j], x[j], q);
                    }
                    const float rstd = inverse_root(__builtin_fmaf(group_sum<LANES>(q), inv, a.eps));
                    if (!BWD) {
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            x[j] = x[j] * rstd * w[n][j];
                        turned(x);
                    } else {
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            g[j] = float(rg[j]);
                        turned(g);
                        float mean = 0.0f;
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            x[j] = live ? x[j] * rstd : 0.0f;
                            dw[n][j] = live ? __builtin_fmaf(g[j], x[j], dw[n][j]) : dw[n][j];
                            g[j] *= w[n][j];
                            mean = __builtin_fmaf(g[j], x[j], mean);
                        }
                        mean = group_sum<LANES>(mean) * inv;
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            x[j] = rstd * __builtin_fmaf(-x[j], mean, g[j]);
                    }
                    V out;
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        out[j] = T(x[j]);
                    if (live)
                        __builtin_nontemporal_store(out, reinterpret_cast<VU*>(side.out + token * side.ld_out + at(side.hs_out, k + e)));
                }
            }
        }
    }
    if (!BWD || !a.partials)
        return;
    // the wave's heads, then the waves
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            float v = dw[n][j];
#pragma unroll
            for (int d = LANES; d < 64; d <<= 1)
                v += __shfl_xor(v, d);
            if (lane < LANES)
                sums[wave][n][piece * kPer + j] = v;
        }
    __syncthreads();
    constexpr int kWavesOf = BWD ? kQkBlock / 64 : 1;
    for (uint32_t x = threadIdx.x; x < 2 * LANES * kPer; x += kQkBlock) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWavesOf; ++k)
            v += sums[k][x / (LANES * kPer)][x % (LANES * kPer)];
        a.partials[uint64_t(blockIdx.x) * (2 * LANES * kPer) + x] = v;
    }
}

// ---- other forms -------------------------------------------------------------------------
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
    const uint64_t base = flat_block() * kItems, token0 = base / heads;
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
                                                                         uint32_t dim, bool both)
{
    __shared__ float part[kQkFoldRows][kQkFoldCols];
    void* dst = blockIdx.y ? dwk : dwq;
    if (!dst)
        return;
    const uint32_t c = threadIdx.x % kQkFoldCols, r = threadIdx.x / kQkFoldCols, col = blockIdx.x * kQkFoldCols + c;
    // both: each workgroup has a partial for q, then one for k
    const uint32_t first = !blockIdx.y ? 0 : both ? 1 : blocks_q, n = blockIdx.y ? blocks_k : blocks_q, apart = both ? 2 : 1;
    float v = 0.0f;
    if (col < dim)
        for (uint32_t i = r; i < n; i += kQkFoldRows)
            v += partials[(uint64_t(first) + uint64_t(i) * apart) * dim + col];
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
    const uint64_t i = flat_block() * 256 + threadIdx.x;
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

// Of qk_token_kernel: a wave a token, or where that leaves most of the card idle a part of its heads, and no more
// workgroups than are resident, which go on to further tokens: a wave's start (its weights, the position, then the
// angles) is a chain of loads.  8192 tokens of 2 x 25 heads of 64, forward: 24 us with 1024 workgroups, 26 with 1536 or
// 2048, 29 in two parts a token; backward 40, 45, 47 and 42.
constexpr uint64_t kTokenWaves = 4096, kTokenBlocks = 1024;

uint32_t token_split(uint64_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t each)
{
    const uint64_t accesses = (heads + each - 1) / each, more = (kv_heads + each - 1) / each, most = accesses > more ? accesses : more;
    uint64_t n = tokens ? (kTokenWaves + tokens - 1) / tokens : 1;
    return uint32_t(n < most ? n : most);
}

uint64_t token_blocks(uint64_t tokens, uint32_t split, bool bwd)
{
    const uint64_t n = (tokens * split + kQkBlock / 64 - 1) / (kQkBlock / 64);
    return n > kTokenBlocks ? kTokenBlocks : n;
}

uint64_t qk_workspace(uint64_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim)
{
    // the fewest heads that any form gives a workgroup
    const uint64_t q = bwd_blocks(tokens, heads, heads + kv_heads, kQkBlock / 32), k = bwd_blocks(tokens, kv_heads, heads + kv_heads, kQkBlock / 32);
    const uint64_t by_token = 2 * token_blocks(tokens, token_split(tokens, heads, kv_heads, 1), true);
    return (q + k > by_token ? q + k : by_token) * dim * 4;
}

// Lanes a head of qk_token_kernel, or 0 where it does not take the call.
template <typename T>
uint32_t token_lanes(const QkCall& c)
{
    constexpr uint32_t kPer = 16 / sizeof(T);
    const uint32_t lanes = c.dim / kPer;
    if (c.dim % kPer || (c.rot && c.rot != c.dim) || lanes < 2 || lanes > 16 || (lanes & (lanes - 1)))
        return 0;
    // a lane's place in a token is 32 bits
    for (const QkTensor& t : c.side)
        for (uint64_t hs : {t.hs_out, t.hs_x, t.hs_dy})
            if (t.heads && hs * t.heads >= (uint64_t(1) << 30))
                return 0;
    return lanes;
}

template <typename T, bool BWD>
void launch_token(const QkArgs<T>& a, uint32_t lanes, uint64_t blocks, bool past, hipStream_t s)
{
    auto go = [&](auto n, auto style, auto p) {
        hipLaunchKernelGGL((qk_token_kernel<T, decltype(n)::value, decltype(style)::value, decltype(p)::value, BWD>), dim3(uint32_t(blocks)),
                           dim3(kQkBlock), 0, s, a);
    };
    auto with_past = [&](auto n, auto style) { past ? go(n, style, std::true_type{}) : go(n, style, std::false_type{}); };
    auto with_style = [&](auto n) {
        if (!a.rot) with_past(n, std::integral_constant<int, 0>{});
        else if (!a.interleaved) with_past(n, std::integral_constant<int, 1>{});
        else with_past(n, std::integral_constant<int, 2>{});
    };
    switch (lanes) {
    case 2: with_style(std::integral_constant<int, 2>{}); break;
    case 4: with_style(std::integral_constant<int, 4>{}); break;
    case 8: with_style(std::integral_constant<int, 8>{}); break;
    default: with_style(std::integral_constant<int, 16>{}); break;
    }
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
            hipLaunchKernelGGL((qk_fwd_kernel<T, LANES, STYLE, true>), flat_grid(blocks), dim3(kQkBlock), 0, s, a);
        else
            hipLaunchKernelGGL((qk_fwd_kernel<T, LANES, STYLE, false>), flat_grid(blocks), dim3(kQkBlock), 0, s, a);
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
    const uint32_t token_way = token_lanes<T>(c);
    const bool by_token = token_way != 0;
    if (c.tokens && by_token) {
        a.split = token_split(c.tokens, c.side[0].heads, c.side[1].heads, 64 / token_way);
        const uint64_t n = token_blocks(c.tokens, a.split, BWD);
        a.blocks[0] = uint32_t(n);
        a.blocks[1] = uint32_t(n);
        launch_token<T, BWD>(a, token_way, n, past, s);
        const int rc = launch_status();
        if (rc)
            return rc;
    } else if (c.tokens) {
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
                       c.dw[1], c.grad_dtype == ZERO_F32, c.accumulate, a.partials, a.blocks[0], a.blocks[1], c.dim, by_token);
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
    hipLaunchKernelGGL(rope_table_kernel, flat_grid((entries + 255) / 256), dim3(256), 0, static_cast<hipStream_t>(stream), table, entries,
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

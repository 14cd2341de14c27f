// dropout.hip -- dropout with a mask that is never stored (Srivastava et al.
// 2014; the mask comes from a counter-based generator, layer.hpp), fused with
// the bias before it and the residual sum after it, and the generator's state.
#include "layer.hpp"

namespace zero {
namespace layer {

int make_drop(double p, const zero_rng_t* rng, uint32_t site, Drop* d)
{
    if (!(p >= 0.0 && p <= 1.0))
        return ZERO_EINVAL;
    d->rng = rng;
    d->site = site;
    d->threshold = uint32_t(floor(p * 65536.0 + 0.5));
    d->scale = d->threshold < 65536 ? float(65536.0 / double(65536 - d->threshold)) : 0.0f;
    if (!d->threshold)
        return ZERO_OK;
    if (!rng)
        return ZERO_EINVAL;
    return is_aligned(rng, 8) ? ZERO_OK : ZERO_EALIGN;
}

namespace {

__global__ void rng_init_kernel(zero_rng_t* r, uint64_t seed) { *r = zero_rng_t{seed, 0, 0}; }

__global__ void rng_advance_kernel(zero_rng_t* r) { r->step += 1; }

// Division of 32-bit numbers by a number that is fixed for the launch, exact
// for every dividend (Granlund and Montgomery 1994).
struct Quotient {
    uint32_t multiplier, shift1, shift2;
    __device__ uint32_t operator()(uint32_t n) const
    {
        const uint32_t t = __umulhi(multiplier, n);
        return (t + ((n - t) >> shift1)) >> shift2;
    }
};

Quotient quotient_by(uint32_t d)
{
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d)
        ++l;
    const uint64_t m = ((uint64_t(1) << l) - d) * (uint64_t(1) << 32) / d + 1;
    return Quotient{uint32_t(m), l < 1 ? l : 1, l > 0 ? l - 1 : 0};
}

template <typename T>
struct DropoutArgs {
    T* out;
    const T* x;
    const T* residual;
    const void* bias;
    uint64_t ld_out, ld_x, ld_res;
    uint64_t rows, groups;                         // groups of 8 columns in a row
    Quotient by_groups;
    uint32_t cols;
    bool bias_f32;
    Drop drop;
};

constexpr int kDropBlock = 256;

// A short last group of 16-bit elements, loaded from the row's last 8 columns.
template <typename T>
__device__ __forceinline__ typename Raw<T>::type settle16(typename Raw<T>::type v, uint32_t shift)
{
    struct Words {
        uint32_t d[sizeof(v) / 4];
    };
    Words x = __builtin_bit_cast(Words, v);
    shift_down<int(sizeof(v) / 4), 8 * int(sizeof(T))>(x.d, shift);
    return __builtin_bit_cast(typename Raw<T>::type, x);
}

// out = residual + D(x + bias), one group of 8 elements per thread: every
// element is read once and written once, and the pass is bound by HBM.  A
// workgroup lives for one load and one store, so what comes before its loads
// counts: they come first, without a branch, after one multiplication in place
// of a division and before the generator's state is waited for (16384 x 8192
// fp16, no residual: 84.5 us = 6.35 TB/s; with a 64-bit division and the state
// first 97.0 us; a copy 81.2 us).  NARROW: rows of fewer than 8 columns, loaded
// by elements.  FAR: more than 2^22 workgroups' worth, 2^30 groups; the grid is
// then 2^22 workgroups that go around, and positions are counted in 64 bits
// (below it, a launch's threads and all group numbers are well inside the 32
// bits that they have).  Binary32 goes by the traded pieces of layer.hpp, over
// the 64 consecutive groups of a wave whatever rows they are in.
template <typename T, int HINT, bool NARROW, bool FAR>
__global__ __launch_bounds__(kDropBlock) void dropout_kernel(DropoutArgs<T> a)
{
    typedef typename Raw<T>::type V;
    constexpr bool PIECES = sizeof(T) == 4 && !NARROW;
    const bool ragged = a.cols % 8 != 0;
    const float one = opaque_one();
    const uint32_t groups = uint32_t(a.groups), lane = threadIdx.x & 63;
    const uint64_t total = FAR ? a.rows * a.groups : uint32_t(a.rows) * uint32_t(a.groups);
    const uint64_t stride = uint64_t(gridDim.x) * kDropBlock;
    uint64_t base = uint64_t(blockIdx.x) * kDropBlock;
    do {
        // the workgroup's first row and column, the thread's from there
        const uint64_t row0 = FAR ? base / a.groups : a.by_groups(uint32_t(base));
        const uint32_t c0 = uint32_t(base - row0 * a.groups);
        auto locate = [&](uint32_t offset, uint64_t& row, uint32_t& c) {   // the group `offset` after the first
            row = row0;
            c = c0 + offset;
            if (groups >= kDropBlock) {            // at most one row's end among the workgroup's threads
                const bool wrap = c >= groups;
                row += wrap;
                c -= wrap ? groups : 0;
            } else {
                const uint32_t wrap = a.by_groups(c);
                row += wrap;
                c -= wrap * groups;
            }
        };
        uint32_t mine = threadIdx.x;               // the thread's group, counted from the workgroup's first
        if (PIECES)
            mine = mine - lane + lane / 2 + (lane & 1) * 32;
        uint64_t row;
        uint32_t c;
        V x, res;
        if constexpr (PIECES) {
            uint64_t rows[2];
            uint32_t col[2], at[2];
            f32x4 xp[2], rp[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t group = threadIdx.x - lane + lane / 2 + p * 32;
                const bool in = base + group < total;
                locate(in ? group : 0, rows[p], col[p]);
                col[p] = col[p] * 8 + (lane & 1) * 4;
                at[p] = col[p] < a.cols - 4 ? col[p] : a.cols - 4;
                xp[p] = load4_full<HINT>(a.x + rows[p] * a.ld_x + at[p]);
                if (a.residual)
                    rp[p] = load4_full<HINT>(a.residual + rows[p] * a.ld_res + at[p]);
            }
            locate(base + mine < total ? mine : 0, row, c);
            struct Words {
                uint32_t d[2][4];
            };
            auto settle = [&](const f32x4 (&v)[2]) {
                Words w;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t (&d)[4] = w.d[p];
                    __builtin_memcpy(d, &v[p], 16);
                    if (ragged)
                        shift_down<4, 32>(d, col[p] - at[p]);
                }
                Part<float, 64>::trade(w.d[0], w.d[1]);
                return __builtin_bit_cast(f32x8, w);
            };
            f32x8 v = splat(-0.0f);                // x + -0 is x, -0 too
            if (a.bias)
                v = load8_vector<T>(a.bias, a.bias_f32, c * 8, int(a.cols) - int(c * 8), -0.0f);
            v = dropped(settle(xp) + v, a.drop, mask_bits(a.drop, rng_key(a.drop), base + mine));
            if (a.residual)
                v = settle(rp) + v;
            Words w = __builtin_bit_cast(Words, v);
            Part<float, 64>::trade(w.d[0], w.d[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t group = threadIdx.x - lane + lane / 2 + p * 32;
                f32x4 o;
                __builtin_memcpy(&o, w.d[p], 16);
                store4<HINT>(a.out + rows[p] * a.ld_out + col[p], o, base + group < total ? int(a.cols) - int(col[p]) : 0);
            }
        } else {
            if (base + mine >= total)
                continue;
            locate(mine, row, c);
            const Group at = NARROW ? Group{0, 0, int(a.cols)} : group_at(c * 8, a.cols);
            if (NARROW) {
                x = load8(a.x + row * a.ld_x, at.k);
                if (a.residual)
                    res = load8(a.residual + row * a.ld_res, at.k);
            } else {
                x = load8_full<HINT>(a.x + row * a.ld_x + at.at);
                if (a.residual)
                    res = load8_full<HINT>(a.residual + row * a.ld_res + at.at);
            }
            f32x8 v = splat(-0.0f);
            if (a.bias)
                v = load8_vector<T>(a.bias, a.bias_f32, c * 8, at.k, -0.0f);
            if (!NARROW && ragged) {
                x = settle16<T>(x, at.shift);
                if (a.residual)
                    res = settle16<T>(res, at.shift);
            }
            v = dropped(raw_plus<T>(x, v, one), a.drop, mask_bits(a.drop, rng_key(a.drop), base + mine));
            if (a.residual)
                v = raw_plus<T>(res, v, one);
            store8<HINT>(a.out + row * a.ld_out + c * 8, narrow<T>(v), at.k);
        }
    } while (FAR && (base += stride) < total);
}

template <typename T>
int launch(void* out, uint64_t ld_out, const void* x, uint64_t ld_x, const void* residual, uint64_t ld_res,
           const void* bias, int bias_dtype, uint64_t rows, uint64_t cols, const Drop& d, hipStream_t s)
{
    DropoutArgs<T> a{static_cast<T*>(out), static_cast<const T*>(x), static_cast<const T*>(residual), bias,
                     ld_out, ld_x, ld_res, rows, (cols + 7) / 8, quotient_by(uint32_t((cols + 7) / 8)), uint32_t(cols),
                     bias_dtype == ZERO_F32, d};
    const uint64_t grid = (rows * a.groups + kDropBlock - 1) / kDropBlock;
    const uint64_t bytes = rows * cols * sizeof(T) * (residual ? 3 : 2);
    constexpr uint64_t kMost = 1u << 22;           // past it: FAR
    const dim3 block(kDropBlock);
    if (grid > kMost) {
        if (cols < 8)
            hipLaunchKernelGGL((dropout_kernel<T, kStreamed, true, true>), dim3(kMost), block, 0, s, a);
        else
            hipLaunchKernelGGL((dropout_kernel<T, kStreamed, false, true>), dim3(kMost), block, 0, s, a);
    } else if (cols < 8)
        hipLaunchKernelGGL((dropout_kernel<T, kCached, true, false>), dim3(uint32_t(grid)), block, 0, s, a);
    else if (bytes <= kStreamBytes)
        hipLaunchKernelGGL((dropout_kernel<T, kCached, false, false>), dim3(uint32_t(grid)), block, 0, s, a);
    else
        hipLaunchKernelGGL((dropout_kernel<T, kStreamed, false, false>), dim3(uint32_t(grid)), block, 0, s, a);
    return launch_status();
}

}  // namespace
}  // namespace layer
}  // namespace zero

using namespace zero;
using namespace zero::layer;

extern "C" int zero_rng_init(zero_rng_t* dev_rng, uint64_t seed, void* stream)
{
    if (!dev_rng)
        return ZERO_EINVAL;
    if (!is_aligned(dev_rng, 8))
        return ZERO_EALIGN;
    hipLaunchKernelGGL(rng_init_kernel, dim3(1), dim3(1), 0, (hipStream_t)stream, dev_rng, seed);
    return launch_status();
}

extern "C" int zero_rng_advance(zero_rng_t* dev_rng, void* stream)
{
    if (!dev_rng)
        return ZERO_EINVAL;
    if (!is_aligned(dev_rng, 8))
        return ZERO_EALIGN;
    hipLaunchKernelGGL(rng_advance_kernel, dim3(1), dim3(1), 0, (hipStream_t)stream, dev_rng);
    return launch_status();
}

extern "C" int zero_dropout_fwd(void* out, uint64_t ld_out, const void* x, uint64_t ld_x, const void* residual,
                                uint64_t ld_residual, const void* bias, int bias_dtype, uint64_t rows, uint64_t cols,
                                int dtype, double p, const zero_rng_t* dev_rng, uint32_t site, void* stream)
{
    int rc = check_shape(rows, cols, dtype);
    Drop d;
    if (!rc) rc = make_drop(p, dev_rng, site, &d);
    if (!rc) rc = check_matrix(out, ld_out, rows, cols, dtype, true);
    if (!rc) rc = check_matrix(x, ld_x, rows, cols, dtype, true);
    if (!rc) rc = check_matrix(residual, ld_residual, rows, cols, dtype, false);
    if (!rc) rc = check_vector(bias, bias_dtype, dtype);
    if (rc || !rows || !cols)
        return rc;
    hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
    case ZERO_F16: return launch<_Float16>(out, ld_out, x, ld_x, residual, ld_residual, bias, bias_dtype, rows, cols, d, s);
    case ZERO_BF16: return launch<bf16>(out, ld_out, x, ld_x, residual, ld_residual, bias, bias_dtype, rows, cols, d, s);
    default: return launch<float>(out, ld_out, x, ld_x, residual, ld_residual, bias, bias_dtype, rows, cols, d, s);
    }
}

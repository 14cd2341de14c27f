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

template <typename T>
struct DropoutArgs {
    T* out;
    const T* x;
    const T* residual;
    const void* bias;
    uint64_t ld_out, ld_x, ld_res;
    uint64_t rows, groups;                         // groups of 8 columns in a row
    uint32_t cols;
    bool bias_f32;
    Drop drop;
};

constexpr int kDropBlock = 256;

// out = residual + D(x + bias), one group of 8 elements per thread: every
// element is read once and written once, and the pass is bound by HBM.  The
// loads come first, without a branch, so that they are in flight together.
// NARROW: rows of fewer than 8 columns, loaded by elements.
template <typename T, int HINT, bool NARROW>
__global__ __launch_bounds__(kDropBlock) void dropout_kernel(DropoutArgs<T> a)
{
    typedef typename Raw<T>::type V;
    const RngKey key = rng_key(a.drop);
    const bool ragged = a.cols % 8 != 0;
    const float one = opaque_one();
    const uint32_t groups = uint32_t(a.groups);
    const uint64_t total = a.rows * a.groups, stride = uint64_t(gridDim.x) * kDropBlock;
    for (uint64_t base = uint64_t(blockIdx.x) * kDropBlock; base < total; base += stride) {
        const uint64_t g = base + threadIdx.x;
        if (g >= total)
            return;
        // the workgroup's first row and column by one scalar division, the
        // thread's from there in 32 bits
        uint64_t row = base / a.groups;
        uint32_t c = uint32_t(base - row * a.groups) + threadIdx.x;
        if (groups >= kDropBlock) {                // at most one row's end among the workgroup's threads
            const bool wrap = c >= groups;
            row += wrap;
            c -= wrap ? groups : 0;
        } else {
            const uint32_t wrap = c / groups;
            row += wrap;
            c -= wrap * groups;
        }
        const Group at = NARROW ? Group{0, 0, int(a.cols)} : group_at(c * 8, a.cols);
        V x, res;
        if (NARROW) {
            x = load8(a.x + row * a.ld_x, at.k);
            if (a.residual)
                res = load8(a.residual + row * a.ld_res, at.k);
        } else {
            x = load8_full<HINT>(a.x + row * a.ld_x + at.at);
            if (a.residual)
                res = load8_full<HINT>(a.residual + row * a.ld_res + at.at);
        }
        f32x8 v = splat(-0.0f);                    // x + -0 is x, -0 too
        if (a.bias)
            v = load8_vector<T>(a.bias, a.bias_f32, c * 8, at.k, -0.0f);
        if (!NARROW && ragged) {
            x = settle<T>(x, at.shift, true);
            if (a.residual)
                res = settle<T>(res, at.shift, true);
        }
        v = dropped(raw_plus<T>(x, v, one), a.drop, key, g);
        if (a.residual)
            v = raw_plus<T>(res, v, one);
        store8<HINT>(a.out + row * a.ld_out + c * 8, narrow<T>(v), at.k);
    }
}

template <typename T>
int launch(void* out, uint64_t ld_out, const void* x, uint64_t ld_x, const void* residual, uint64_t ld_res,
           const void* bias, int bias_dtype, uint64_t rows, uint64_t cols, const Drop& d, hipStream_t s)
{
    DropoutArgs<T> a{static_cast<T*>(out), static_cast<const T*>(x), static_cast<const T*>(residual), bias,
                     ld_out, ld_x, ld_res, rows, (cols + 7) / 8, uint32_t(cols), bias_dtype == ZERO_F32, d};
    uint64_t grid = (a.rows * a.groups + kDropBlock - 1) / kDropBlock;
    if (grid > (1u << 22))
        grid = 1u << 22;
    const uint64_t bytes = rows * cols * sizeof(T) * (residual ? 3 : 2);
    if (cols < 8)
        hipLaunchKernelGGL((dropout_kernel<T, kCached, true>), dim3(uint32_t(grid)), dim3(kDropBlock), 0, s, a);
    else if (bytes <= kStreamBytes)
        hipLaunchKernelGGL((dropout_kernel<T, kCached, false>), dim3(uint32_t(grid)), dim3(kDropBlock), 0, s, a);
    else
        hipLaunchKernelGGL((dropout_kernel<T, kStreamed, false>), dim3(uint32_t(grid)), dim3(kDropBlock), 0, s, a);
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

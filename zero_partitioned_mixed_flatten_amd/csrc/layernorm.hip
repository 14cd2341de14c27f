// layernorm.hip -- layer norm (Ba, Kiros and Hinton 2016) forward, and the
// same fused behind the bias, dropout and residual sum that precede it in a
// transformer block.
//
//   r = residual + D(x + bias)           (the joined form; else r = x)
//   mean = sum(r) / n, var = sum((r - mean)^2) / n, rstd = 1/sqrt(var + eps)
//   y = (r - mean) * rstd * w + b
//
// The variance is summed from the deviations, after the mean, so a row far
// from zero loses nothing.  The joined form rounds r to the element type
// once, where it stores it, and normalises the stored value: what the backward
// pass reads again.
#include "layer.hpp"

namespace zero {
namespace layer {
namespace {

template <typename T>
struct FwdArgs {
    T* r;
    T* y;
    float* mean;
    float* rstd;
    const T* x;
    const T* residual;
    const void* bias;
    const void* w;
    const void* b;
    uint64_t ld_r, ld_y, ld_x, ld_res;
    uint64_t rows;
    uint32_t cols;
    bool vec_f32;
    float eps;
    Drop drop;
};

// Rows that fit the registers of TPR threads, VPT groups of 8 columns each:
// one pass over memory, the row kept as it was loaded.
template <typename T, bool JOIN, int BLOCK, int TPR, int VPT>
__global__ __launch_bounds__(BLOCK) void norm_fwd_kernel(FwdArgs<T> a)
{
    typedef typename Raw<T>::type V;
    constexpr int kRows = BLOCK / TPR;
    __shared__ alignas(16) float scratch[2 * BLOCK / 64];
    uint32_t parity = 0;
    const RngKey key = rng_key(a.drop);
    const uint32_t groups = (a.cols + 7) / 8;
    const float n = float(a.cols);
    uint32_t slot = threadIdx.x / TPR;
    if (TPR >= 64)
        slot = __builtin_amdgcn_readfirstlane(slot);
    const uint32_t t = threadIdx.x % TPR;
    for (uint64_t first = uint64_t(blockIdx.x) * kRows; first < a.rows; first += uint64_t(gridDim.x) * kRows) {
        const uint64_t row = first + slot;
        const bool live = row < a.rows;
        V raw[VPT];
        f32x8 w[VPT], b[VPT];
        float s[1] = {0.0f}, q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t g = i * TPR + t, col = g * 8;
            const int k = live ? int(a.cols) - int(col) : 0;
            raw[i] = load8(a.x + row * a.ld_x + col, k);
            if (JOIN) {
                V res;
                if (a.residual)
                    res = load8(a.residual + row * a.ld_res + col, k);
                f32x8 v = widen<T>(raw[i]);
                if (a.bias)
                    v = v + load8_vector<T>(a.bias, a.vec_f32, col, k, 0.0f);
                v = dropped(v, a.drop, key, row * groups + g);
                if (a.residual)
                    v = widen<T>(res) + v;
                raw[i] = narrow<T>(v);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t col = (i * TPR + t) * 8;
            const int k = live ? int(a.cols) - int(col) : 0;
            w[i] = load8_vector<T>(a.w, a.vec_f32, col, k, 1.0f);
            b[i] = load8_vector<T>(a.b, a.vec_f32, col, k, 0.0f);
            if (JOIN)
                store8(a.r + row * a.ld_r + col, raw[i], k);
            f32x8 v = widen<T>(raw[i]);
            if (k < 8)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = j < k ? v[j] : 0.0f;
            s[0] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        row_sum<BLOCK, TPR>(s, scratch, parity);
        const float mean = s[0] / n;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = int(a.cols) - int((i * TPR + t) * 8);
            f32x8 v = widen<T>(raw[i]) - mean;
            if (k < 8)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = j < k ? v[j] : 0.0f;
            v = v * v;
            q[0] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        row_sum<BLOCK, TPR>(q, scratch, parity);
        const float rstd = 1.0f / sqrtf(q[0] / n + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t col = (i * TPR + t) * 8;
            const int k = live ? int(a.cols) - int(col) : 0;
            f32x8 v = widen<T>(raw[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[i][j], b[i][j]);
            store8(a.y + row * a.ld_y + col, narrow<T>(v), k);
        }
        if (t == 0 && live) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Any width: a workgroup takes a row and goes over it three times.
constexpr int kWideBlock = 256;

template <typename T, bool JOIN>
__global__ __launch_bounds__(kWideBlock) void norm_fwd_wide_kernel(FwdArgs<T> a)
{
    __shared__ alignas(16) float scratch[2 * kWideBlock / 64];
    uint32_t parity = 0;
    const RngKey key = rng_key(a.drop);
    const uint32_t groups = (a.cols + 7) / 8;
    const float n = float(a.cols);
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* src = a.x + row * a.ld_x;
        float s[1] = {0.0f}, q[1] = {0.0f};
        for (uint32_t g = threadIdx.x; g < groups; g += kWideBlock) {
            const uint32_t col = g * 8;
            const int k = int(a.cols) - int(col);
            typename Raw<T>::type raw = load8(src + col, k);
            if (JOIN) {
                f32x8 v = widen<T>(raw);
                if (a.bias)
                    v = v + load8_vector<T>(a.bias, a.vec_f32, col, k, 0.0f);
                v = dropped(v, a.drop, key, row * groups + g);
                if (a.residual)
                    v = widen<T>(load8(a.residual + row * a.ld_res + col, k)) + v;
                raw = narrow<T>(v);
                store8(a.r + row * a.ld_r + col, raw, k);
            }
            const f32x8 v = widen<T>(raw);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[0] += j < k ? v[j] : 0.0f;
        }
        row_sum<kWideBlock, kWideBlock>(s, scratch, parity);
        const float mean = s[0] / n;
        if (JOIN)
            src = a.r + row * a.ld_r;
        for (uint32_t g = threadIdx.x; g < groups; g += kWideBlock) {
            const uint32_t col = g * 8;
            const int k = int(a.cols) - int(col);
            const f32x8 v = widen<T>(load8(src + col, k));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = j < k ? v[j] - mean : 0.0f;
                q[0] = __builtin_fmaf(d, d, q[0]);
            }
        }
        row_sum<kWideBlock, kWideBlock>(q, scratch, parity);
        const float rstd = 1.0f / sqrtf(q[0] / n + a.eps);
        for (uint32_t g = threadIdx.x; g < groups; g += kWideBlock) {
            const uint32_t col = g * 8;
            const int k = int(a.cols) - int(col);
            f32x8 v = widen<T>(load8(src + col, k));
            const f32x8 w = load8_vector<T>(a.w, a.vec_f32, col, k, 1.0f);
            const f32x8 b = load8_vector<T>(a.b, a.vec_f32, col, k, 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]);
            store8(a.y + row * a.ld_y + col, narrow<T>(v), k);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <typename T, bool JOIN, int TPR, int VPT>
int launch_rows(const FwdArgs<T>& a, hipStream_t s)
{
    constexpr int kBlock = TPR < 256 ? 256 : TPR;
    uint64_t grid = (a.rows + kBlock / TPR - 1) / (kBlock / TPR);
    if (grid > (1u << 20))
        grid = 1u << 20;
    hipLaunchKernelGGL((norm_fwd_kernel<T, JOIN, kBlock, TPR, VPT>), dim3(uint32_t(grid)), dim3(kBlock), 0, s, a);
    return launch_status();
}

template <typename T, bool JOIN>
int launch_fwd(const FwdArgs<T>& a, hipStream_t s)
{
    if (a.cols <= 64) return launch_rows<T, JOIN, 8, 1>(a, s);
    if (a.cols <= 128) return launch_rows<T, JOIN, 16, 1>(a, s);
    if (a.cols <= 256) return launch_rows<T, JOIN, 32, 1>(a, s);
    if (a.cols <= 512) return launch_rows<T, JOIN, 64, 1>(a, s);
    if (a.cols <= 1024) return launch_rows<T, JOIN, 128, 1>(a, s);
    if (a.cols <= 2048) return launch_rows<T, JOIN, 256, 1>(a, s);
    if (a.cols <= 4096) return launch_rows<T, JOIN, 512, 1>(a, s);
    if (a.cols <= 8192) return launch_rows<T, JOIN, 512, 2>(a, s);
    if (a.cols <= 16384) return launch_rows<T, JOIN, 1024, 2>(a, s);
    const uint64_t grid = a.rows < (1u << 20) ? a.rows : (1u << 20);
    hipLaunchKernelGGL((norm_fwd_wide_kernel<T, JOIN>), dim3(uint32_t(grid)), dim3(kWideBlock), 0, s, a);
    return launch_status();
}

struct FwdCall {
    void *r, *y;
    float *mean, *rstd;
    const void *x, *residual, *bias, *w, *b;
    uint64_t ld_r, ld_y, ld_x, ld_res, rows, cols;
    int dtype, vec_dtype;
    double eps;
    Drop drop;
};

template <typename T, bool JOIN>
int run_fwd(const FwdCall& c, hipStream_t s)
{
    FwdArgs<T> a{static_cast<T*>(c.r), static_cast<T*>(c.y), c.mean, c.rstd, static_cast<const T*>(c.x),
                 static_cast<const T*>(c.residual), c.bias, c.w, c.b, c.ld_r, c.ld_y, c.ld_x, c.ld_res, c.rows,
                 uint32_t(c.cols), c.vec_dtype == ZERO_F32, float(c.eps), c.drop};
    return launch_fwd<T, JOIN>(a, s);
}

// What both forward entry points check, in the order the header lists.
int check_fwd(const FwdCall& c, bool join)
{
    int rc = check_shape(c.rows, c.cols, c.dtype);
    if (rc)
        return rc;
    if (!(c.eps > 0.0) || !isfinite(c.eps) || !(float(c.eps) > 0.0f))
        return ZERO_EINVAL;
    if (!c.cols)
        return ZERO_ERANGE;
    if (join) rc = check_matrix(c.r, c.ld_r, c.rows, c.cols, c.dtype, true);
    if (!rc) rc = check_matrix(c.y, c.ld_y, c.rows, c.cols, c.dtype, true);
    if (!rc) rc = check_matrix(c.x, c.ld_x, c.rows, c.cols, c.dtype, true);
    if (!rc) rc = check_matrix(c.residual, c.ld_res, c.rows, c.cols, c.dtype, false);
    if (!rc) rc = check_vector(c.bias, c.vec_dtype, c.dtype);
    if (!rc) rc = check_vector(c.w, c.vec_dtype, c.dtype);
    if (!rc) rc = check_vector(c.b, c.vec_dtype, c.dtype);
    if (rc)
        return rc;
    if ((c.mean && !is_aligned(c.mean, 4)) || (c.rstd && !is_aligned(c.rstd, 4)))
        return ZERO_EALIGN;
    if (join && c.rows && c.r == c.y)
        return ZERO_EINVAL;
    return ZERO_OK;
}

}  // namespace
}  // namespace layer
}  // namespace zero

using namespace zero;
using namespace zero::layer;

extern "C" int zero_layernorm_fwd(void* y, uint64_t ld_y, float* mean, float* rstd, const void* x, uint64_t ld_x,
                                  const void* w, const void* b, int vec_dtype, uint64_t rows, uint64_t cols, int dtype,
                                  double eps, void* stream)
{
    const FwdCall c{nullptr, y, mean, rstd, x, nullptr, nullptr, w, b, 0, ld_y, ld_x, 0, rows, cols, dtype, vec_dtype,
                    eps, Drop{nullptr, 0, 0, 1.0f}};
    const int rc = check_fwd(c, false);
    if (rc || !rows)
        return rc;
    hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
    case ZERO_F16: return run_fwd<_Float16, false>(c, s);
    case ZERO_BF16: return run_fwd<bf16, false>(c, s);
    default: return run_fwd<float, false>(c, s);
    }
}

extern "C" int zero_dropout_layernorm_fwd(void* r, uint64_t ld_r, void* y, uint64_t ld_y, float* mean, float* rstd,
                                          const void* x, uint64_t ld_x, const void* residual, uint64_t ld_residual,
                                          const void* bias, const void* w, const void* b, int vec_dtype, uint64_t rows,
                                          uint64_t cols, int dtype, double eps, double p, const zero_rng_t* dev_rng,
                                          uint32_t site, void* stream)
{
    FwdCall c{r, y, mean, rstd, x, residual, bias, w, b, ld_r, ld_y, ld_x, ld_residual, rows, cols, dtype, vec_dtype,
              eps, Drop{}};
    int rc = make_drop(p, dev_rng, site, &c.drop);
    if (!rc) rc = check_fwd(c, true);
    if (rc || !rows)
        return rc;
    hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
    case ZERO_F16: return run_fwd<_Float16, true>(c, s);
    case ZERO_BF16: return run_fwd<bf16, true>(c, s);
    default: return run_fwd<float, true>(c, s);
    }
}

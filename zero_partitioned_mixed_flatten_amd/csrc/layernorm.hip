// layernorm.hip -- layer norm (Ba, Kiros and Hinton 2016) forward, and the
// same fused behind the bias, dropout and residual sum that precede it in a
// transformer block.
//
//   r = residual + D(x + bias)           (the joined form; else r = x)
//   mean = sum(r) / n, var = sum((r - mean)^2) / n, rstd = 1/sqrt(var + eps)
//   y = (r - mean) * rstd * w + b
//
// The variance is summed from the deviations, after the mean, so a row far
// from zero loses only what its mean does, summed and rounded in binary32.  The
// joined form rounds r to the element type once, where it stores it, and
// normalises the stored value: what the backward pass reads again.
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
// one pass over memory, the row kept as it was loaded.  A persistent workgroup
// takes every gridDim.x-th block of BLOCK / TPR rows, the next rows' loads in
// flight while it works on the present ones, w, b and bias in registers (but
// see kLate).
template <typename T, bool JOIN, int BLOCK, int TPR, int VPT, int HINT>
__global__ __launch_bounds__(BLOCK) void norm_fwd_kernel(FwdArgs<T> a)
{
    typedef typename Raw<T>::type V;
    typedef Part<T, TPR> P;
    constexpr int kRows = BLOCK / TPR;
    // r of a joined 16-bit row is made 0 past the row's end once, when it is
    // rounded, instead of x and residual
    constexpr bool kZero = !JOIN || sizeof(T) == 4;
    // 1024 threads have 128 registers each, too few for two joined binary32
    // groups with the next row's and the vectors: the next row is fetched when
    // this one is summed up, into the same registers, and the vectors are read
    // again from the caches (1000 x 16384 49 us, 300 x 16384 20; with the rest's
    // way and 38 registers spilt 76 and 34, and three passes 70 and 28; 3000 x
    // 10240, 640 threads, 99 so and 91 the rest's way).  No vector register is
    // spilt so, but 140 scalars are, to lanes of vector registers (the other
    // joined forms spill up to 32 of them)
    constexpr bool kLate = JOIN && sizeof(T) == 4 && BLOCK == 1024;
    __shared__ alignas(16) float scratch[2 * BLOCK / 64];
    uint32_t parity = 0;
    const RngKey key = rng_key(a.drop);
    const uint32_t groups = (a.cols + 7) / 8;
    const bool ragged = a.cols % 8 != 0;
    const float n = float(a.cols), inv = 1.0f / n, one = opaque_one();
    uint32_t slot = threadIdx.x / TPR;
    if (TPR >= 64)
        slot = __builtin_amdgcn_readfirstlane(slot);
    const uint32_t t = threadIdx.x % TPR;
    auto part = [&](int i) { return P(i, t, a.cols); };

    struct Row {
        V x[VPT], res[VPT];
    };
    auto fetch = [&](uint64_t row, Row& f) {
        row = row < a.rows ? row : a.rows - 1;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            f.x[i] = part(i).template load<HINT>(a.x + row * a.ld_x);
            if (JOIN && a.residual)
                f.res[i] = part(i).template load<HINT>(a.residual + row * a.ld_res);
        }
    };
    const uint64_t stride = uint64_t(gridDim.x) * kRows;
    uint64_t first = uint64_t(blockIdx.x) * kRows;
    Row cur, next;
    fetch(first + slot, cur);
    f32x8 w[VPT], b[VPT], bias[VPT];
    auto load_w = [&](int i) {
        const P at = part(i);
        w[i] = load8_vector<T>(a.w, a.vec_f32, at.group * 8, at.k, 1.0f);
        b[i] = load8_vector<T>(a.b, a.vec_f32, at.group * 8, at.k, 0.0f);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const P at = part(i);
        if (!kLate)
            load_w(i);
        if (JOIN && !kLate)
            bias[i] = load8_vector<T>(a.bias, a.vec_f32, at.group * 8, at.k, -0.0f);   // x + -0 is x, -0 too
    }
    for (; first < a.rows; first += stride) {
        const uint64_t row = first + slot;
        if (!kLate && first + stride < a.rows)
            fetch(row + stride, next);
        const bool live = row < a.rows;
        u32x4 bits[VPT];
        if (JOIN)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                bits[i] = mask_bits(a.drop, key, row * groups + part(i).group);
        V raw[VPT];                                // 0 past the row's end, the sum needs no test
        f32x8 x[VPT], s8;
        float s[1] = {0.0f}, q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const P at = part(i);
            raw[i] = at.template settle<kZero>(cur.x[i], ragged);
            if (JOIN) {
                if (kLate)
                    bias[i] = load8_vector<T>(a.bias, a.vec_f32, at.group * 8, at.k, -0.0f);
                f32x8 v = raw_plus<T>(raw[i], bias[i], one);
                v = dropped(v, a.drop, bits[i]);
                if (a.residual)
                    v = raw_plus<T>(at.template settle<kZero>(cur.res[i], ragged), v, one);
                raw[i] = narrow<T>(v);
                if (!kZero && at.k < 8)            // a short or absent group: 0 past the row's end
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        raw[i][j] = j < at.k ? raw[i][j] : T(0.0f);
                at.template store<HINT>(a.r + row * a.ld_r, raw[i], live);
            }
            s8 = i ? raw_plus<T>(raw[i], s8, one) : widen<T>(raw[i]);
        }
        if (kLate && first + stride < a.rows)
            fetch(row + stride, cur);
        s[0] = ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
        row_sum<BLOCK, TPR>(s, scratch, parity);
        const float mean = over(s[0], n, inv);
        float qb = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = part(i).k;
            x[i] = raw_plus<T>(raw[i], splat(-mean), one);
            if (k < 8)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[i][j] = j < k ? x[i][j] : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                q[0] = __builtin_fmaf(x[i][j], x[i][j], q[0]);
                qb = __builtin_fmaf(x[i][j + 1], x[i][j + 1], qb);
            }
        }
        q[0] += qb;
        row_sum<BLOCK, TPR>(q, scratch, parity);
        const float rstd = 1.0f / sqrtf(over(q[0], n, inv) + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            f32x8 v;
            if (kLate)
                load_w(i);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_fmaf(x[i][j] * rstd, w[i][j], b[i][j]);
            part(i).template store<HINT>(a.y + row * a.ld_y, narrow<T>(v), live);
        }
        if (t == 0 && live) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (!kLate)
            cur = next;
    }
}

// Wider rows: a workgroup takes a row and goes over it three times, the second
// and third time from the caches.
constexpr int kWideBlock = 1024;

template <typename T, bool JOIN>
__global__ __launch_bounds__(kWideBlock) void norm_fwd_wide_kernel(FwdArgs<T> a)
{
    typedef typename Raw<T>::type V;
    typedef Part<T, kWideBlock> P;
    __shared__ alignas(16) float scratch[2 * kWideBlock / 64];
    uint32_t parity = 0;
    const RngKey key = rng_key(a.drop);
    const uint32_t groups = (a.cols + 7) / 8, rounds = (groups + kWideBlock - 1) / kWideBlock;
    const bool ragged = a.cols % 8 != 0;
    const float n = float(a.cols), inv = 1.0f / n, one = opaque_one();
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* src = a.x + row * a.ld_x;
        float s[1] = {0.0f}, q[1] = {0.0f};
        for (uint32_t i = 0; i < rounds; ++i) {
            const P at(i, threadIdx.x, a.cols);
            V raw = at.template load<kCached>(src), res;
            if (JOIN && a.residual)
                res = at.template load<kCached>(a.residual + row * a.ld_res);
            raw = at.settle(raw, ragged);
            if (JOIN) {
                const Group g = group_at(at.group * 8, a.cols);
                f32x8 v = raw_plus<T>(raw, load8_vector_at<T>(a.bias, a.vec_f32, g, ragged, -0.0f), one);
                v = dropped(v, a.drop, mask_bits(a.drop, key, row * groups + at.group));
                if (a.residual)
                    v = raw_plus<T>(at.settle(res, ragged), v, one);
                if (at.k <= 0)
                    v = splat(0.0f);               // past the row: not the bias either
                raw = narrow<T>(v);
                at.template store<0>(a.r + row * a.ld_r, raw, true);
            }
            const f32x8 v = widen<T>(raw);
            s[0] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        row_sum<kWideBlock, kWideBlock>(s, scratch, parity);
        const float mean = over(s[0], n, inv);
        if (JOIN)
            src = a.r + row * a.ld_r;              // each thread uses what it stored there itself
        for (uint32_t i = 0; i < rounds; ++i) {
            const P at(i, threadIdx.x, a.cols);
            const f32x8 d = raw_plus<T>(at.settle(at.template load<kCached>(src), ragged), splat(-mean), one);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[0] = j < at.k ? __builtin_fmaf(d[j], d[j], q[0]) : q[0];
        }
        row_sum<kWideBlock, kWideBlock>(q, scratch, parity);
        const float rstd = 1.0f / sqrtf(over(q[0], n, inv) + a.eps);
        for (uint32_t i = 0; i < rounds; ++i) {
            const P at(i, threadIdx.x, a.cols);
            const Group g = group_at(at.group * 8, a.cols);
            f32x8 v = raw_plus<T>(at.settle(at.template load<kCached>(src), ragged), splat(-mean), one);
            const f32x8 w = load8_vector_at<T>(a.w, a.vec_f32, g, ragged, 1.0f);
            const f32x8 b = load8_vector_at<T>(a.b, a.vec_f32, g, ragged, 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_fmaf(v[j] * rstd, w[j], b[j]);
            at.template store<kStreamed>(a.y + row * a.ld_y, narrow<T>(v), true);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// The threads of a row: one below 8 columns; as few powers of two as hold its
// groups one each up to a wave; wider rows take two groups a thread and whole
// waves, at least two.  The workgroup is one row, or as many as make 256
// threads.  Measured at 13.1 M fp16 elements (layer norm / joined, us; a copy
// and two copies of the same bytes take 10.6 / 21.1): 512 columns 12.8 / 22.7,
// 64 threads x 1, against 13.1 / 23.6 with 32 x 2; 1600 columns 13.7 / 24.2,
// 128 x 2, against 14.6 / 25.6 with 256 x 1 and 14.9 / 29.2 with 64 x 4; 8192
// columns 13.1 / 23.8, 512 x 2, against 14.5 / 27.0 with 1024 x 1 and 15.1 / 26.8
// with 256 x 4.
//
// The grid: what is resident at once with the registers each form takes, and
// no more than there are blocks of rows; workgroups that wait for a place
// leave the last ones running alone.  Threads a CU, layer norm, plain loads:
// 512 columns 2048 10.5 us, 1536 11.1, 1024 11.4; 1600 columns 1536 10.8, 1024
// 11.7, 768 12.0; joined, 1600 columns: 1024 24.2, 768 24.7, 2048 26.5.  Past
// the cache two groups a thread do better with 1024 (16384 x 8192: 92 us, 1536
// 101).
constexpr uint64_t kCus = 256;

template <typename T, bool JOIN, int TPR, int VPT, int HINT>
void launch_hinted(const FwdArgs<T>& a, hipStream_t s)
{
    constexpr int kBlock = TPR < 192 ? 256 : TPR;
    constexpr int kThreads = VPT == 1 ? (JOIN ? 1536 : 2048) : JOIN || sizeof(T) == 4 || HINT == kStreamed ? 1024 : 1536;
    constexpr uint64_t kMost = kCus * (kThreads / kBlock);
    const uint64_t blocks = (a.rows + kBlock / TPR - 1) / (kBlock / TPR);
    hipLaunchKernelGGL((norm_fwd_kernel<T, JOIN, kBlock, TPR, VPT, HINT>), dim3(uint32_t(blocks < kMost ? blocks : kMost)),
                       dim3(kBlock), 0, s, a);
}

template <typename T, bool JOIN, int TPR, int VPT>
int launch_rows(const FwdArgs<T>& a, hipStream_t s)
{
    const uint64_t bytes = a.rows * a.cols * sizeof(T) * (JOIN ? (a.residual ? 4 : 3) : 2);
    if (bytes <= kStreamBytes)
        launch_hinted<T, JOIN, TPR, VPT, kCached>(a, s);
    else
        launch_hinted<T, JOIN, TPR, VPT, kStreamed>(a, s);
    return launch_status();
}

template <typename T, bool JOIN>
int launch_fwd(const FwdArgs<T>& a, hipStream_t s)
{
    if (a.cols < 8) return launch_rows<T, JOIN, 1, 1>(a, s);
    if (a.cols <= 64) return launch_rows<T, JOIN, 8, 1>(a, s);
    if (a.cols <= 128) return launch_rows<T, JOIN, 16, 1>(a, s);
    if (a.cols <= 256) return launch_rows<T, JOIN, 32, 1>(a, s);
    if (a.cols <= 512) return launch_rows<T, JOIN, 64, 1>(a, s);
    if (a.cols <= 1024) return launch_rows<T, JOIN, 64, 2>(a, s);
    switch ((a.cols + 1023) / 1024) {              // whole waves of 1024 columns
    case 2: return launch_rows<T, JOIN, 128, 2>(a, s);
    case 3: return launch_rows<T, JOIN, 192, 2>(a, s);
    case 4: return launch_rows<T, JOIN, 256, 2>(a, s);
    case 5: return launch_rows<T, JOIN, 320, 2>(a, s);
    case 6: return launch_rows<T, JOIN, 384, 2>(a, s);
    case 7: return launch_rows<T, JOIN, 448, 2>(a, s);
    case 8: return launch_rows<T, JOIN, 512, 2>(a, s);
    case 9: case 10: return launch_rows<T, JOIN, 640, 2>(a, s);
    case 11: case 12: return launch_rows<T, JOIN, 768, 2>(a, s);
    case 13: case 14: case 15: case 16: return launch_rows<T, JOIN, 1024, 2>(a, s);
    }
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
    const float eps = float(c.eps);                // what the kernels add: a binary64 value may round to 0 or inf
    if (!(eps > 0.0f) || !isfinite(eps))
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
    if (c.rows && ((join && c.r == c.y) || (c.mean && c.mean == c.rstd)))
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

// layernorm_bwd.hip -- the backward passes of layer norm, of dropout with a
// bias, and of the two joined, with the sums over the rows that are the
// gradients of the weights and biases.
//
//   h = (r - mean) * rstd, g = dy * w, c1 = sum(g) / n, c2 = sum(g h) / n
//   e = rstd * (g - c1 - h * c2) + dres       (dropout alone: e = dout)
//   dr = e, dx = D(e)                         (layer norm alone: dx = e)
//   dw = sum_rows dy * h, db = sum_rows dy, dbias = sum_rows D(e)
//
// h is recomputed from the saved mean and rstd.  The masks of D come from the
// generator's counters again.  Sums are binary32.
#include "layer.hpp"

namespace zero {
namespace layer {
namespace {

template <typename T>
struct BwdArgs {
    T* dx;
    T* dr;
    const T* dy;
    const T* dres;
    const T* r;
    const float* mean;
    const float* rstd;
    const void* w;
    uint64_t ld_dx, ld_dr, ld_dy, ld_dres, ld_r;
    uint64_t rows, rows_per_chunk;
    uint32_t cols, chunks;
    bool vec_f32;
    Drop drop;
    float* row_sums;                               // c1, c2 of each row
    float* partials;                               // [chunk][3][cols]
    bool want[3];                                  // dw, db, dbias
};

// The pass in two kernels, for any width: c1 and c2 of each row, then strips
// of columns going down a chunk of rows.
constexpr int kWideBlock = 256;
constexpr uint64_t kStrip = kWideBlock * 8;
constexpr uint64_t kWideTarget = 1024;             // workgroups the strips are cut into rows for

uint64_t wide_chunks(uint64_t rows, uint64_t cols)
{
    const uint64_t strips = (cols + kStrip - 1) / kStrip;
    uint64_t c = kWideTarget / strips;
    if (c < 1) c = 1;
    return c < rows ? c : rows;
}

template <typename T>
__global__ __launch_bounds__(kWideBlock) void row_sums_kernel(BwdArgs<T> a)
{
    __shared__ float scratch[2][kWideBlock / 64];
    const uint32_t groups = (a.cols + 7) / 8;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (uint32_t g = threadIdx.x; g < groups; g += kWideBlock) {
            const uint32_t col = g * 8, k = a.cols - col;
            const f32x8 dy = widen<T>(load8(a.dy + row * a.ld_dy + col, k));
            const f32x8 r = widen<T>(load8(a.r + row * a.ld_r + col, k));
            const f32x8 w = load8_vector<T>(a.w, a.vec_f32, col, k, 1.0f);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const float gj = dy[j] * w[j], h = (r[j] - mean) * rstd;
                if (j < k) {
                    s1 += gj;
                    s2 = __builtin_fmaf(gj, h, s2);
                }
            }
        }
        s1 = block_sum<kWideBlock>(s1, scratch[0]);
        s2 = block_sum<kWideBlock>(s2, scratch[1]);
        if (threadIdx.x == 0) {
            a.row_sums[2 * row] = s1 / float(a.cols);
            a.row_sums[2 * row + 1] = s2 / float(a.cols);
        }
        __syncthreads();
    }
}

template <typename T, bool NORM, bool DROP>
__global__ __launch_bounds__(kWideBlock) void strips_kernel(BwdArgs<T> a)
{
    const uint32_t groups = (a.cols + 7) / 8;
    const uint32_t g = blockIdx.x * kWideBlock + threadIdx.x;
    if (g >= groups)
        return;
    const RngKey key = rng_key(a.drop);
    const uint32_t col = g * 8, k = a.cols - col;
    f32x8 w, sum[3];
    if (NORM)
        w = load8_vector<T>(a.w, a.vec_f32, col, k, 1.0f);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[i][j] = 0.0f;
    const uint64_t first = uint64_t(blockIdx.y) * a.rows_per_chunk;
    const uint64_t last = first + a.rows_per_chunk < a.rows ? first + a.rows_per_chunk : a.rows;
    for (uint64_t row = first; row < last; ++row) {
        f32x8 e = widen<T>(load8(a.dy + row * a.ld_dy + col, k));
        if (NORM) {
            const float mean = a.mean[row], rstd = a.rstd[row];
            const float c1 = a.row_sums[2 * row], c2 = a.row_sums[2 * row + 1];
            f32x8 r = widen<T>(load8(a.r + row * a.ld_r + col, k));
            f32x8 t;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float h = (r[j] - mean) * rstd;
                sum[0][j] = __builtin_fmaf(e[j], h, sum[0][j]);
                sum[1][j] += e[j];
                t[j] = rstd * __builtin_fmaf(-h, c2, e[j] * w[j] - c1);
            }
            e = t;
            if (a.dres)
                e = e + widen<T>(load8(a.dres + row * a.ld_dres + col, k));
        }
        if (DROP) {
            if (NORM)
                store8(a.dr + row * a.ld_dr + col, narrow<T>(e), k);
            e = dropped(e, a.drop, key, row * groups + g);
            sum[2] = sum[2] + e;
        }
        store8(a.dx + row * a.ld_dx + col, narrow<T>(e), k);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (a.want[i]) {
            float* p = a.partials + (uint64_t(blockIdx.y) * 3 + i) * a.cols + col;
            for (uint32_t j = 0; j < 8; ++j)
                if (j < k)
                    p[j] = sum[i][j];
        }
}

// Adds the chunks' partials of each column in their order and stores the sum,
// or adds it to what is there, rounded once to the gradient's type.
constexpr int kFoldBlock = 256;

template <typename T>
__global__ __launch_bounds__(kFoldBlock) void fold_kernel(SumOut out, const float* partials, uint32_t chunks,
                                                          uint32_t cols)
{
    const uint64_t col = uint64_t(blockIdx.x) * kFoldBlock + threadIdx.x;
    const int i = blockIdx.y;
    if (col >= cols || !out.dst[i])
        return;
    float s = 0.0f;
    for (uint32_t c = 0; c < chunks; ++c)
        s += partials[(uint64_t(c) * 3 + i) * cols + col];
    if (out.f32) {
        float* d = static_cast<float*>(out.dst[i]) + col;
        *d = out.accumulate ? *d + s : s;
    } else {
        T* d = static_cast<T*>(out.dst[i]) + col;
        *d = T(out.accumulate ? float(*d) + s : s);
    }
}

struct BwdCall {
    void *dx, *dr;
    const void *dy, *dres, *r;
    const float *mean, *rstd;
    const void* w;
    int vec_dtype;
    uint64_t ld_dx, ld_dr, ld_dy, ld_dres, ld_r, rows, cols;
    int dtype;
    Drop drop;
    void *dw, *db, *dbias;
    int grad_dtype;
    bool accumulate;
    void* workspace;
    size_t workspace_bytes;
};

uint64_t row_sums_bytes(uint64_t rows) { return (rows * 8 + 15) / 16 * 16; }

uint64_t workspace_need(uint64_t rows, uint64_t cols)
{
    return row_sums_bytes(rows) + wide_chunks(rows, cols) * 3 * cols * 4;
}

template <typename T, bool NORM, bool DROP>
int run_bwd(const BwdCall& c, hipStream_t s)
{
    BwdArgs<T> a{};
    a.dx = static_cast<T*>(c.dx);
    a.dr = static_cast<T*>(c.dr);
    a.dy = static_cast<const T*>(c.dy);
    a.dres = static_cast<const T*>(c.dres);
    a.r = static_cast<const T*>(c.r);
    a.mean = c.mean;
    a.rstd = c.rstd;
    a.w = c.w;
    a.ld_dx = c.ld_dx;
    a.ld_dr = c.ld_dr;
    a.ld_dy = c.ld_dy;
    a.ld_dres = c.ld_dres;
    a.ld_r = c.ld_r;
    a.rows = c.rows;
    a.cols = uint32_t(c.cols);
    a.vec_f32 = c.vec_dtype == ZERO_F32;
    a.drop = c.drop;
    a.row_sums = static_cast<float*>(c.workspace);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(c.workspace) + row_sums_bytes(c.rows));
    a.want[0] = c.dw;
    a.want[1] = c.db;
    a.want[2] = c.dbias;
    uint64_t chunks = 0;
    if (c.rows) {
        chunks = wide_chunks(c.rows, c.cols);
        a.rows_per_chunk = (c.rows + chunks - 1) / chunks;
        chunks = (c.rows + a.rows_per_chunk - 1) / a.rows_per_chunk;
        if (NORM) {
            const uint64_t grid = c.rows < (1u << 20) ? c.rows : (1u << 20);
            hipLaunchKernelGGL(row_sums_kernel<T>, dim3(uint32_t(grid)), dim3(kWideBlock), 0, s, a);
        }
        const uint64_t strips = (c.cols + kStrip - 1) / kStrip;
        hipLaunchKernelGGL((strips_kernel<T, NORM, DROP>), dim3(uint32_t(strips), uint32_t(chunks)), dim3(kWideBlock),
                           0, s, a);
        const int rc = launch_status();
        if (rc)
            return rc;
    }
    if (!c.dw && !c.db && !c.dbias)
        return ZERO_OK;
    const SumOut out{{c.dw, c.db, c.dbias}, c.grad_dtype == ZERO_F32, c.accumulate};
    hipLaunchKernelGGL(fold_kernel<T>, dim3(uint32_t((c.cols + kFoldBlock - 1) / kFoldBlock), 3), dim3(kFoldBlock), 0, s,
                       out, a.partials, uint32_t(chunks), uint32_t(c.cols));
    return launch_status();
}

int check_bwd(const BwdCall& c, bool norm, bool join)
{
    int rc = check_shape(c.rows, c.cols, c.dtype);
    if (rc)
        return rc;
    if (norm && !c.cols)
        return ZERO_ERANGE;
    rc = check_matrix(c.dx, c.ld_dx, c.rows, c.cols, c.dtype, true);
    if (!rc && join) rc = check_matrix(c.dr, c.ld_dr, c.rows, c.cols, c.dtype, true);
    if (!rc) rc = check_matrix(c.dy, c.ld_dy, c.rows, c.cols, c.dtype, true);
    if (!rc) rc = check_matrix(c.dres, c.ld_dres, c.rows, c.cols, c.dtype, false);
    if (!rc && norm) rc = check_matrix(c.r, c.ld_r, c.rows, c.cols, c.dtype, true);
    if (!rc) rc = check_vector(c.w, c.vec_dtype, c.dtype);
    if (!rc) rc = check_vector(c.dw, c.grad_dtype, c.dtype);
    if (!rc) rc = check_vector(c.db, c.grad_dtype, c.dtype);
    if (!rc) rc = check_vector(c.dbias, c.grad_dtype, c.dtype);
    if (rc)
        return rc;
    if (norm && c.rows && (!c.mean || !c.rstd))
        return ZERO_EINVAL;
    if (norm && (!is_aligned(c.mean, 4) || !is_aligned(c.rstd, 4)))
        return ZERO_EALIGN;
    if (join && c.rows && c.dx == c.dr)
        return ZERO_EINVAL;
    const void* g[3] = {c.dw, c.db, c.dbias};
    for (int i = 0; i < 3; ++i)
        if (g[i] && g[i] == g[(i + 1) % 3])
            return ZERO_EINVAL;
    if (!c.rows || !c.cols)
        return ZERO_OK;
    if (norm || c.dbias) {
        if (!c.workspace)
            return ZERO_EINVAL;
        if (!is_aligned(c.workspace, 16))
            return ZERO_EALIGN;
        if (c.workspace_bytes < workspace_need(c.rows, c.cols))
            return ZERO_ERANGE;
    }
    return ZERO_OK;
}

template <bool NORM, bool DROP>
int dispatch(const BwdCall& c, void* stream)
{
    hipStream_t s = (hipStream_t)stream;
    switch (c.dtype) {
    case ZERO_F16: return run_bwd<_Float16, NORM, DROP>(c, s);
    case ZERO_BF16: return run_bwd<bf16, NORM, DROP>(c, s);
    default: return run_bwd<float, NORM, DROP>(c, s);
    }
}

}  // namespace
}  // namespace layer
}  // namespace zero

using namespace zero;
using namespace zero::layer;

extern "C" size_t zero_layer_workspace_bytes(uint64_t rows, uint64_t cols)
{
    if (rows > kMaxRows || cols > kMaxCols || !cols || !rows)
        return 0;
    return size_t(workspace_need(rows, cols));
}

extern "C" int zero_layernorm_bwd(void* dx, uint64_t ld_dx, void* dw, void* db, int grad_dtype, int accumulate,
                                  const void* dy, uint64_t ld_dy, const void* dres, uint64_t ld_dres, const void* x,
                                  uint64_t ld_x, const float* mean, const float* rstd, const void* w, int vec_dtype,
                                  uint64_t rows, uint64_t cols, int dtype, void* workspace, size_t workspace_bytes,
                                  void* stream)
{
    const BwdCall c{dx, nullptr, dy, dres, x, mean, rstd, w, vec_dtype, ld_dx, 0, ld_dy, ld_dres, ld_x, rows, cols,
                    dtype, Drop{nullptr, 0, 0, 1.0f}, dw, db, nullptr, grad_dtype, accumulate != 0, workspace,
                    workspace_bytes};
    const int rc = check_bwd(c, true, false);
    return rc ? rc : dispatch<true, false>(c, stream);
}

extern "C" int zero_dropout_bwd(void* dx, uint64_t ld_dx, void* dbias, int grad_dtype, int accumulate,
                                const void* dout, uint64_t ld_dout, uint64_t rows, uint64_t cols, int dtype, double p,
                                const zero_rng_t* dev_rng, uint32_t site, void* workspace, size_t workspace_bytes,
                                void* stream)
{
    BwdCall c{dx, nullptr, dout, nullptr, nullptr, nullptr, nullptr, nullptr, ZERO_F32, ld_dx, 0, ld_dout, 0, 0, rows,
              cols, dtype, Drop{}, nullptr, nullptr, dbias, grad_dtype, accumulate != 0, workspace, workspace_bytes};
    int rc = make_drop(p, dev_rng, site, &c.drop);
    if (!rc) rc = check_bwd(c, false, false);
    if (rc || !cols)
        return rc;
    // without a bias gradient the backward pass is the forward's map
    if (!dbias)
        return zero_dropout_fwd(dx, ld_dx, dout, ld_dout, nullptr, 0, nullptr, 0, rows, cols, dtype, p, dev_rng, site,
                                stream);
    return dispatch<false, true>(c, stream);
}

extern "C" int zero_dropout_layernorm_bwd(void* dx, uint64_t ld_dx, void* dr, uint64_t ld_dr, void* dw, void* db,
                                          void* dbias, int grad_dtype, int accumulate, const void* dy, uint64_t ld_dy,
                                          const void* dres, uint64_t ld_dres, const void* r, uint64_t ld_r,
                                          const float* mean, const float* rstd, const void* w, int vec_dtype,
                                          uint64_t rows, uint64_t cols, int dtype, double p, const zero_rng_t* dev_rng,
                                          uint32_t site, void* workspace, size_t workspace_bytes, void* stream)
{
    BwdCall c{dx, dr, dy, dres, r, mean, rstd, w, vec_dtype, ld_dx, ld_dr, ld_dy, ld_dres, ld_r, rows, cols, dtype,
              Drop{}, dw, db, dbias, grad_dtype, accumulate != 0, workspace, workspace_bytes};
    int rc = make_drop(p, dev_rng, site, &c.drop);
    if (!rc) rc = check_bwd(c, true, true);
    return rc ? rc : dispatch<true, true>(c, stream);
}

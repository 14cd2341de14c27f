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

// Rows that fit the registers of TPR threads, VPT groups of 8 columns each,
// in one pass: a persistent workgroup takes every gridDim.x-th block of
// BLOCK / TPR rows, the next rows' loads in flight while it works on the
// present ones, and keeps its columns' sums in registers to the end, where
// it stores one partial.
template <typename T, bool NORM, bool DROP, int BLOCK, int TPR, int VPT, int NBUF, int HINT>
__global__ __launch_bounds__(BLOCK) void rows_bwd_kernel(BwdArgs<T> a)
{
    typedef typename Raw<T>::type V;
    constexpr int kRows = BLOCK / TPR;
    constexpr int kSums = (NORM ? 2 : 0) + (DROP ? 1 : 0);
    __shared__ alignas(16) float scratch[NORM ? 4 * BLOCK / 64 : 1];
    uint32_t parity = 0;
    const RngKey key = rng_key(a.drop);
    const uint32_t groups = (a.cols + 7) / 8;
    const bool ragged = a.cols % 8 != 0;
    const float n = float(a.cols), inv = 1.0f / n, one = opaque_one();
    uint32_t slot = threadIdx.x / TPR;
    if (TPR >= 64)
        slot = __builtin_amdgcn_readfirstlane(slot);
    const uint32_t t = threadIdx.x % TPR;

    Group at[VPT];
    f32x8 w[VPT], sum[kSums][VPT];
    struct Row {
        V dy[VPT], r[VPT], dres[VPT];
        float mean, rstd;
    };
    auto fetch = [&](uint64_t row, Row& f) {
        row = row < a.rows ? row : a.rows - 1;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            f.dy[i] = load8_full<HINT>(a.dy + row * a.ld_dy + at[i].at);
            if (NORM) {
                f.r[i] = load8_full<HINT>(a.r + row * a.ld_r + at[i].at);
                if (a.dres)
                    f.dres[i] = load8_full<HINT>(a.dres + row * a.ld_dres + at[i].at);
            }
        }
        if (NORM) {
            f.mean = a.mean[row];
            f.rstd = a.rstd[row];
        }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        at[i] = group_at((i * TPR + t) * 8, a.cols);
    const uint64_t stride = uint64_t(gridDim.x) * kRows;
    uint64_t first = uint64_t(blockIdx.x) * kRows;
    Row buf[NBUF];
#pragma unroll
    for (int i = 0; i < NBUF - 1; ++i)
        fetch(first + i * stride + slot, buf[i]);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (NORM)
            w[i] = load8_vector<T>(a.w, a.vec_f32, (i * TPR + t) * 8, at[i].k, 1.0f);
#pragma unroll
        for (int q = 0; q < kSums; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[q][i][j] = 0.0f;
    }
    auto work = [&](uint64_t row, Row& cur) {
        const bool live = row < a.rows;
        // with d = dy * rstd and x = r - mean: g rstd = d w, h rstd = x rstd^2
        f32x8 x[VPT], g[VPT];
        float c[2] = {0.0f, 0.0f};
        if (NORM) {
            float c0b = 0.0f, c1b = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                cur.dy[i] = settle<T>(cur.dy[i], at[i].shift, ragged);   // 0 past the row's end
                const f32x8 d = raw_times<T>(cur.dy[i], cur.rstd);
                x[i] = raw_plus<T>(settle<T, false>(cur.r[i], at[i].shift, ragged), splat(-cur.mean), one);
                g[i] = d * w[i];
                if (live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[0][i][j] = __builtin_fmaf(d[j], x[i][j], sum[0][i][j]);
                    sum[1][i] = raw_plus<T>(cur.dy[i], sum[1][i], one);
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    c[0] += g[i][j];
                    c0b += g[i][j + 1];
                    c[1] = __builtin_fmaf(g[i][j], x[i][j], c[1]);
                    c1b = __builtin_fmaf(g[i][j + 1], x[i][j + 1], c1b);
                }
            }
            c[0] += c0b;
            c[1] += c1b;
            row_sum<BLOCK, TPR>(c, scratch, parity);
            c[0] = -over(c[0], n, inv);
            c[1] = -(over(c[1], n, inv) * cur.rstd * cur.rstd);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t g8 = i * TPR + t, col = g8 * 8;
            const int k = live ? at[i].k : 0;
            f32x8 e;
            if (NORM) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    e[j] = __builtin_fmaf(x[i][j], c[1], g[i][j] + c[0]);
                if (a.dres)
                    e = raw_plus<T>(settle<T, false>(cur.dres[i], at[i].shift, ragged), e, one);
            } else {
                e = widen<T>(settle<T>(cur.dy[i], at[i].shift, ragged));
            }
            if (DROP) {
                if (NORM)
                    store8<HINT>(a.dr + row * a.ld_dr + col, narrow<T>(e), k);
                e = dropped(e, a.drop, key, row * groups + g8);
                if (live)
                    sum[kSums - 1][i] = sum[kSums - 1][i] + e;
            }
            store8<HINT>(a.dx + row * a.ld_dx + col, narrow<T>(e), k);
        }
    };
    for (bool more = true; more;) {
#pragma unroll
        for (int i = 0; i < NBUF; ++i) {           // the buffers in turn: a copy would wait for its loads
            if (more) {
                fetch(first + (NBUF - 1) * stride + slot, buf[(i + NBUF - 1) % NBUF]);
                work(first + slot, buf[i]);
                first += stride;
                more = first < a.rows;
            }
        }
    }

    // one partial of the workgroup: the upper half of its rows' threads hands
    // its sums to the lower half, until one row's are left
    if (kRows > 1) {
        __shared__ f32x4 hand[kRows > 1 ? kSums * VPT * BLOCK : 1];
#pragma unroll
        for (int half = kRows / 2; half >= 1; half /= 2) {
            const int lanes = half * TPR;
            if (int(slot) >= half && int(slot) < 2 * half)
#pragma unroll
                for (int q = 0; q < kSums * VPT; ++q)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const f32x8 v = sum[q / VPT][q % VPT];
                        hand[(2 * q + p) * lanes + (int(threadIdx.x) - lanes)] = f32x4{v[4 * p], v[4 * p + 1], v[4 * p + 2],
                                                                                       v[4 * p + 3]};
                    }
            __syncthreads();
            if (int(slot) < half)
#pragma unroll
                for (int q = 0; q < kSums * VPT; ++q)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const f32x4 o = hand[(2 * q + p) * lanes + int(threadIdx.x)];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sum[q / VPT][q % VPT][4 * p + j] += o[j];
                    }
            __syncthreads();
        }
    }
    if (slot != 0)
        return;
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
        const int which = NORM ? q : 2;
        if (!a.want[which])
            continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t col = (i * TPR + t) * 8;
            store8_f32(a.partials + (uint64_t(blockIdx.x) * 3 + which) * a.cols + col, sum[q][i], int(a.cols) - int(col));
        }
    }
}

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
    __shared__ alignas(16) float scratch[4 * kWideBlock / 64];
    uint32_t parity = 0;
    const uint32_t groups = (a.cols + 7) / 8;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.0f, 0.0f};
        for (uint32_t g = threadIdx.x; g < groups; g += kWideBlock) {
            const uint32_t col = g * 8;
            const int k = int(a.cols) - int(col);
            const f32x8 dy = widen<T>(load8(a.dy + row * a.ld_dy + col, k));
            const f32x8 r = widen<T>(load8(a.r + row * a.ld_r + col, k));
            const f32x8 w = load8_vector<T>(a.w, a.vec_f32, col, k, 1.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gj = dy[j] * w[j], h = (r[j] - mean) * rstd;
                if (j < k) {
                    s[0] += gj;
                    s[1] = __builtin_fmaf(gj, h, s[1]);
                }
            }
        }
        row_sum<kWideBlock, kWideBlock>(s, scratch, parity);
        if (threadIdx.x == 0) {
            a.row_sums[2 * row] = s[0] / float(a.cols);
            a.row_sums[2 * row + 1] = s[1] / float(a.cols);
        }
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
    const uint32_t col = g * 8;
    const int k = int(a.cols) - int(col);
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
        if (a.want[i])
            store8_f32(a.partials + (uint64_t(blockIdx.y) * 3 + i) * a.cols + col, sum[i], k);
}

// Adds the partials of each column in their order and stores the sum, or adds
// it to what is there, rounded once to the gradient's type.  A workgroup
// takes 64 columns; each of its 16 waves adds every 16th partial, its loads in
// flight together, and the waves' sums are added in order.
constexpr int kFoldBlock = 1024;
constexpr uint32_t kFoldCols = 64;

template <typename T>
__global__ __launch_bounds__(kFoldBlock) void fold_kernel(SumOut out, const float* __restrict__ partials, uint32_t chunks,
                                                          uint32_t cols)
{
    __shared__ float part[kFoldBlock / 64][kFoldCols];
    const int i = blockIdx.y;
    if (!out.dst[i])
        return;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t col = blockIdx.x * kFoldCols + lane;
    float s = 0.0f;
    if (col < cols) {
        const float* p = partials + uint64_t(i) * cols + col;
        const uint64_t step = uint64_t(3) * cols;
        for (uint32_t c = wave; c < chunks; c += 8 * 16) {
            float v[8];
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u)
                v[u] = c + 16 * u < chunks ? p[(c + 16 * u) * step] : 0.0f;
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u)
                s += v[u];
        }
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave || col >= cols)
        return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kFoldBlock / 64; ++k)
        s += part[k][lane];
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

// The one-pass kernel: rows up to 8192 columns, one workgroup of 1024 threads
// a CU, one group of 8 columns a thread.  Every workgroup costs a partial
// (written and read again: as much as 2.4 joined rows of fp16), so there are no
// more than 256, and only 128 where 256 would get no more than 1.5 blocks of
// rows each.  Measured (kernel and fold, us, fp16): joined 8192 x 1600, 256 x
// 4 rows of 256 threads 33.4, 512 workgroups of 512 threads 34.7, 128 threads
// with two groups each 44.0; joined 16384 x 8192, 1024 threads x 1 group 237,
// 512 x 2 254.  Layer norm, 128 against 256 workgroups at most: 200 x 8192
// 12.7 and 15.1, 400 x 8192 15.0 and 17.6, 1000 x 1600 9.2 and 9.7, 800 x 8192
// 18.4 and 17.4, 2000 x 1600 11.7 and 11.0.
constexpr uint64_t kRowsMaxCols = 8192;
constexpr int kRowsBlock = 1024;

uint64_t rows_tpr(uint64_t cols)
{
    uint64_t tpr = 8;
    while (tpr * 8 < cols)
        tpr *= 2;
    return tpr;
}

bool one_pass(uint64_t cols) { return cols >= 8 && cols <= kRowsMaxCols; }

uint64_t rows_chunks(uint64_t rows, uint64_t cols)
{
    const uint64_t per = kRowsBlock / rows_tpr(cols), blocks = (rows + per - 1) / per;
    const uint64_t most = blocks <= 400 ? 128 : 256;
    return blocks < most ? blocks : most;
}

uint64_t row_sums_bytes(uint64_t rows, uint64_t cols) { return one_pass(cols) ? 0 : (rows * 8 + 15) / 16 * 16; }

uint64_t workspace_need(uint64_t rows, uint64_t cols)
{
    const uint64_t chunks = one_pass(cols) ? rows_chunks(rows, cols) : wide_chunks(rows, cols);
    return row_sums_bytes(rows, cols) + chunks * 3 * cols * 4;
}

// Two rows in flight ahead of the present one where the registers hold them
// (layer norm alone, 16-bit elements: 8192 x 1600 21.8 us against 22.1 with one,
// 1600 x 8192 28.5 against 29.3), else one.
template <typename T, bool NORM, bool DROP, int TPR>
void launch_rows(const BwdArgs<T>& a, uint64_t chunks, hipStream_t s)
{
    constexpr int kBuffers = DROP || sizeof(T) == 4 ? 2 : 3;
    const uint64_t arrays = (NORM ? 3 + (a.dres != nullptr) : 2) + (NORM && DROP);
    if (a.rows * a.cols * sizeof(T) * arrays <= kStreamBytes)
        hipLaunchKernelGGL((rows_bwd_kernel<T, NORM, DROP, kRowsBlock, TPR, 1, kBuffers, kCached>), dim3(uint32_t(chunks)),
                           dim3(kRowsBlock), 0, s, a);
    else
        hipLaunchKernelGGL((rows_bwd_kernel<T, NORM, DROP, kRowsBlock, TPR, 1, kBuffers, kStreamed>),
                           dim3(uint32_t(chunks)), dim3(kRowsBlock), 0, s, a);
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
    a.partials = reinterpret_cast<float*>(static_cast<char*>(c.workspace) + row_sums_bytes(c.rows, c.cols));
    a.want[0] = c.dw;
    a.want[1] = c.db;
    a.want[2] = c.dbias;
    uint64_t chunks = 0;
    if (c.rows && one_pass(c.cols)) {
        chunks = rows_chunks(c.rows, c.cols);
        switch (rows_tpr(c.cols)) {
        case 8: launch_rows<T, NORM, DROP, 8>(a, chunks, s); break;
        case 16: launch_rows<T, NORM, DROP, 16>(a, chunks, s); break;
        case 32: launch_rows<T, NORM, DROP, 32>(a, chunks, s); break;
        case 64: launch_rows<T, NORM, DROP, 64>(a, chunks, s); break;
        case 128: launch_rows<T, NORM, DROP, 128>(a, chunks, s); break;
        case 256: launch_rows<T, NORM, DROP, 256>(a, chunks, s); break;
        case 512: launch_rows<T, NORM, DROP, 512>(a, chunks, s); break;
        default: launch_rows<T, NORM, DROP, 1024>(a, chunks, s); break;
        }
    } else if (c.rows) {
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
    }
    if (c.rows) {
        const int rc = launch_status();
        if (rc)
            return rc;
    }
    if (!c.dw && !c.db && !c.dbias)
        return ZERO_OK;
    const SumOut out{{c.dw, c.db, c.dbias}, c.grad_dtype == ZERO_F32, c.accumulate};
    hipLaunchKernelGGL(fold_kernel<T>, dim3(uint32_t((c.cols + kFoldCols - 1) / kFoldCols), 3), dim3(kFoldBlock), 0, s,
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

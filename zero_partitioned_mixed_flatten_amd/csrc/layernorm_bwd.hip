// layernorm_bwd.hip -- the backward passes of layer norm, of dropout with a
// bias, and of the two joined, with the sums over the rows that are the
// gradients of the weights and biases.
//
//   h = (r - mean) * rstd, g = dy * w, c1 = sum(g) / n, c2 = sum(g h) / n
//   e = rstd * (g - c1 - h * c2) + dres       (dropout alone: e = dout)
//   dr = e, dx = D(e)                         (layer norm alone: dx = e)
//   dw = sum_rows dy * h, db = sum_rows dy, dbias = sum_rows D(e)
//
// h is recomputed from the saved mean and rstd, and only it, dy and w enter the
// sums: rstd alone, squared or times dy, may leave binary32's range where the
// gradients do not.  The masks of D come from the generator's counters again.
// Sums are binary32.
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
    float* row_sums;                               // -c1, -c2 of each row
    float* partials;                               // [chunk][3][cols]
    bool want[3];                                  // dw, db, dbias
};

// h = (r - mean) * rstd of a group.
template <typename T>
__device__ __forceinline__ f32x8 normalised(typename Raw<T>::type r, float mean, float rstd, float one)
{
    return raw_plus<T>(r, splat(-mean), one) * rstd;
}

// Rows that fit the registers of TPR threads, a group of 8 columns each, in
// one pass: a persistent workgroup takes every gridDim.x-th block of
// BLOCK / TPR rows, the loads of the next NBUF - 1 in flight while it works on
// the present one, and keeps its columns' sums in registers to the end, where
// it stores one partial.
template <typename T, bool NORM, bool DROP, int BLOCK, int TPR, int NBUF, int HINT>
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
    const Part<T, TPR> at(0, threadIdx.x % TPR, a.cols);

    struct Row {
        V dy, r, dres;
        float mean, rstd;
    };
    auto fetch = [&](uint64_t row, Row& f) {
        row = row < a.rows ? row : a.rows - 1;
        f.dy = at.template load<HINT>(a.dy + row * a.ld_dy);
        if (NORM) {
            f.r = at.template load<HINT>(a.r + row * a.ld_r);
            if (a.dres)
                f.dres = at.template load<HINT>(a.dres + row * a.ld_dres);
            f.mean = a.mean[row];
            f.rstd = a.rstd[row];
        }
    };
    const uint64_t stride = uint64_t(gridDim.x) * kRows;
    uint64_t first = uint64_t(blockIdx.x) * kRows;
    Row buf[NBUF];
#pragma unroll
    for (int i = 0; i < NBUF - 1; ++i)
        fetch(first + i * stride + slot, buf[i]);
    f32x8 w, sum[kSums];
    if (NORM)
        w = load8_vector<T>(a.w, a.vec_f32, at.group * 8, at.k, 1.0f);
#pragma unroll
    for (int q = 0; q < kSums; ++q)
        sum[q] = splat(0.0f);
    auto work = [&](uint64_t row, Row& cur) {
        const bool live = row < a.rows;
        // the mask ahead of the loads' use; binary32 rows leave no registers to
        // keep it (8192 x 1600 joined 58.4 us so, 56.2 with it drawn at the end)
        constexpr bool kEarly = sizeof(T) == 2;
        u32x4 bits;
        if (DROP && kEarly)
            bits = mask_bits(a.drop, key, row * groups + at.group);
        const V dy = at.settle(cur.dy, ragged);    // 0 past the row's end
        f32x8 e;
        if (NORM) {
            const f32x8 h = normalised<T>(at.template settle<false>(cur.r, ragged), cur.mean, cur.rstd, one);
            const f32x8 g = raw_times<T>(dy, w);
            if (live) {
                sum[0] = raw_fma<T>(dy, h, sum[0]);
                sum[1] = raw_plus<T>(dy, sum[1], one);
            }
            float c[2] = {0.0f, 0.0f}, c0b = 0.0f, c1b = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                c[0] += g[j];
                c0b += g[j + 1];
                c[1] = __builtin_fmaf(g[j], h[j], c[1]);
                c1b = __builtin_fmaf(g[j + 1], h[j + 1], c1b);
            }
            c[0] += c0b;
            c[1] += c1b;
            row_sum<BLOCK, TPR>(c, scratch, parity);
            c[0] = -over(c[0], n, inv);
            c[1] = -over(c[1], n, inv);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = __builtin_fmaf(h[j], c[1], g[j] + c[0]);
            if (a.dres)
                e = fma_raw<T>(e, cur.rstd, at.template settle<false>(cur.dres, ragged));
            else
                e = e * cur.rstd;
        } else {
            e = widen<T>(dy);
        }
        if (DROP) {
            if (NORM)
                at.template store<HINT>(a.dr + row * a.ld_dr, narrow<T>(e), live);
            if (!kEarly)
                bits = mask_bits(a.drop, key, row * groups + at.group);
            e = dropped(e, a.drop, bits);
            if (live)
                sum[kSums - 1] = sum[kSums - 1] + e;
        }
        at.template store<HINT>(a.dx + row * a.ld_dx, narrow<T>(e), live);
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
        __shared__ f32x4 hand[kRows > 1 ? kSums * BLOCK : 1];
        for (int half = kRows / 2; half >= 1; half /= 2) {
            const int lanes = half * TPR;
            if (int(slot) >= half && int(slot) < 2 * half)
#pragma unroll
                for (int q = 0; q < kSums; ++q)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        hand[(2 * q + p) * lanes + (int(threadIdx.x) - lanes)] =
                            f32x4{sum[q][4 * p], sum[q][4 * p + 1], sum[q][4 * p + 2], sum[q][4 * p + 3]};
            __syncthreads();
            if (int(slot) < half)
#pragma unroll
                for (int q = 0; q < kSums; ++q)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const f32x4 o = hand[(2 * q + p) * lanes + int(threadIdx.x)];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sum[q][4 * p + j] += o[j];
                    }
            __syncthreads();
        }
    }
    if (slot != 0)
        return;
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
        const int which = NORM ? q : 2;
        if (a.want[which])
            store8_f32(a.partials + (uint64_t(blockIdx.x) * 3 + which) * a.cols + at.group * 8, sum[q], at.k);
    }
}

// Wider rows, in two kernels: c1 and c2 of each row, then strips of columns
// going down a chunk of rows, reading dy and r again (as far as they are still
// there from the 256 MB cache).
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
    typedef Part<T, kWideBlock> P;
    __shared__ alignas(16) float scratch[4 * kWideBlock / 64];
    uint32_t parity = 0;
    const uint32_t groups = (a.cols + 7) / 8, rounds = (groups + kWideBlock - 1) / kWideBlock;
    const bool ragged = a.cols % 8 != 0;
    const float n = float(a.cols), inv = 1.0f / n, one = opaque_one();
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float c[2] = {0.0f, 0.0f};
        for (uint32_t i = 0; i < rounds; ++i) {
            const P at(i, threadIdx.x, a.cols);
            const typename Raw<T>::type dy = at.template load<kCached>(a.dy + row * a.ld_dy);
            const typename Raw<T>::type r = at.template load<kCached>(a.r + row * a.ld_r);
            const f32x8 w = load8_vector_at<T>(a.w, a.vec_f32, group_at(at.group * 8, a.cols), ragged, 1.0f);
            const f32x8 g = raw_times<T>(at.settle(dy, ragged), w);              // 0 past the row's end
            const f32x8 h = normalised<T>(at.settle(r, ragged), mean, rstd, one);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[0] += g[j];
                c[1] = __builtin_fmaf(g[j], h[j], c[1]);
            }
        }
        row_sum<kWideBlock, kWideBlock>(c, scratch, parity);
        if (threadIdx.x == 0) {
            a.row_sums[2 * row] = -over(c[0], n, inv);
            a.row_sums[2 * row + 1] = -over(c[1], n, inv);
        }
    }
}

template <typename T, bool NORM, bool DROP>
__global__ __launch_bounds__(kWideBlock) void strips_kernel(BwdArgs<T> a)
{
    typedef typename Raw<T>::type V;
    constexpr int kSums = (NORM ? 2 : 0) + (DROP ? 1 : 0);
    const RngKey key = rng_key(a.drop);
    const uint32_t groups = (a.cols + 7) / 8;
    const bool ragged = a.cols % 8 != 0;
    const float one = opaque_one();
    const Part<T, kWideBlock> at(blockIdx.x, threadIdx.x, a.cols);
    struct Row {
        V dy, r, dres;
    };
    auto fetch = [&](uint64_t row, Row& f) {
        row = row < a.rows ? row : a.rows - 1;
        f.dy = at.template load<kStreamed>(a.dy + row * a.ld_dy);
        if (NORM) {
            f.r = at.template load<kStreamed>(a.r + row * a.ld_r);
            if (a.dres)
                f.dres = at.template load<kStreamed>(a.dres + row * a.ld_dres);
        }
    };
    const uint64_t first = uint64_t(blockIdx.y) * a.rows_per_chunk;
    const uint64_t last = first + a.rows_per_chunk < a.rows ? first + a.rows_per_chunk : a.rows;
    Row buf[2];
    fetch(first, buf[0]);
    f32x8 w, sum[kSums];
    if (NORM)
        w = load8_vector<T>(a.w, a.vec_f32, at.group * 8, at.k, 1.0f);
#pragma unroll
    for (int q = 0; q < kSums; ++q)
        sum[q] = splat(0.0f);
    auto work = [&](uint64_t row, Row& cur) {
        u32x4 bits;
        if (DROP)
            bits = mask_bits(a.drop, key, row * groups + at.group);
        const V dy = at.settle(cur.dy, ragged);
        f32x8 e;
        if (NORM) {
            const float mean = a.mean[row], rstd = a.rstd[row];
            const float c0 = a.row_sums[2 * row], c1 = a.row_sums[2 * row + 1];
            const f32x8 h = normalised<T>(at.template settle<false>(cur.r, ragged), mean, rstd, one);
            const f32x8 g = raw_times<T>(dy, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = __builtin_fmaf(h[j], c1, g[j] + c0);
            sum[0] = raw_fma<T>(dy, h, sum[0]);
            sum[1] = raw_plus<T>(dy, sum[1], one);
            if (a.dres)
                e = fma_raw<T>(e, rstd, at.template settle<false>(cur.dres, ragged));
            else
                e = e * rstd;
        } else {
            e = widen<T>(dy);
        }
        if (DROP) {
            if (NORM)
                at.template store<kStreamed>(a.dr + row * a.ld_dr, narrow<T>(e), true);
            e = dropped(e, a.drop, bits);
            sum[kSums - 1] = sum[kSums - 1] + e;
        }
        at.template store<kStreamed>(a.dx + row * a.ld_dx, narrow<T>(e), true);
    };
    for (uint64_t row = first; row < last;) {
        fetch(row + 1, buf[1]);
        work(row, buf[0]);
        if (++row >= last)
            break;
        fetch(row + 1, buf[0]);
        work(row, buf[1]);
        ++row;
    }
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
        const int which = NORM ? q : 2;
        if (a.want[which])
            store8_f32(a.partials + (uint64_t(blockIdx.y) * 3 + which) * a.cols + at.group * 8, sum[q], at.k);
    }
}

// Adds the partials of each column in a fixed order and stores the sum, or adds
// it to what is there, rounded once to the gradient's type.  A workgroup takes
// 32 columns; each of its 32 half waves adds every 32nd partial, its loads in
// flight together (all of them up to 256 partials), and the half waves' sums
// are added in order.
constexpr int kFoldBlock = 1024;
constexpr uint32_t kFoldCols = 32;

template <typename T>
__global__ __launch_bounds__(kFoldBlock) void fold_kernel(SumOut out, const float* __restrict__ partials, uint32_t chunks,
                                                          uint32_t cols)
{
    constexpr uint32_t kParts = kFoldBlock / kFoldCols;
    __shared__ float part[kParts][kFoldCols];
    const int i = blockIdx.y;
    if (!out.dst[i])
        return;
    const uint32_t lane = threadIdx.x % kFoldCols, first = threadIdx.x / kFoldCols;
    for (uint32_t block = blockIdx.x; block * kFoldCols < cols; block += gridDim.x) {
        const uint32_t col = block * kFoldCols + lane;
        float s = 0.0f;
        if (col < cols) {
            const float* p = partials + uint64_t(i) * cols + col;
            const uint64_t step = uint64_t(3) * cols;
            for (uint32_t c = first; c < chunks; c += 8 * kParts) {
                float v[8];
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u)
                    v[u] = c + kParts * u < chunks ? p[(c + kParts * u) * step] : 0.0f;
                s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
        }
        part[first][lane] = s;
        __syncthreads();
        if (first == 0 && col < cols) {
            s = 0.0f;
#pragma unroll
            for (uint32_t k = 0; k < kParts; ++k)
                s += part[k][lane];
            if (out.f32) {
                float* d = static_cast<float*>(out.dst[i]) + col;
                *d = out.accumulate ? *d + s : s;
            } else {
                T* d = static_cast<T*>(out.dst[i]) + col;
                *d = T(out.accumulate ? float(*d) + s : s);
            }
        }
        __syncthreads();                           // part is free for the next columns
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
// a CU, one group of 8 columns a thread (with two a thread, rows up to 16384
// columns spill the sums: layer norm 2048 x 12288 72 us and joined 175, against
// 58 and 82 in two kernels).  Every workgroup costs a partial (written and read again: as much as 2.4 joined rows
// of fp16), so there are no more than 256, and only 128 where 256 would get no
// more than 1.5 blocks of rows each.  Measured (kernel and fold, us, fp16):
// joined 8192 x 1600, 256 x 4 rows of 256 threads 33.4, 512 workgroups of 512
// threads 34.7, 128 threads with two groups each 44.0; joined 16384 x 8192, 1024
// threads x 1 group 237, 512 x 2 254.  Layer norm, 128 against 256 workgroups
// at most: 200 x 8192 12.7 and 15.1, 400 x 8192 15.0 and 17.6, 1000 x 1600 9.2
// and 9.7, 800 x 8192 18.4 and 17.4, 2000 x 1600 11.7 and 11.0.
constexpr uint64_t kRowsMaxCols = 8192;
constexpr int kRowsBlock = 1024;

uint64_t rows_tpr(uint64_t cols)
{
    if (cols < 8)
        return 1;
    uint64_t tpr = 8;
    while (tpr * 8 < cols)
        tpr *= 2;
    return tpr;
}

bool one_pass(uint64_t cols) { return cols <= kRowsMaxCols; }

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

// Rows in flight ahead of the present one: as many as the registers hold
// (layer norm alone, 16-bit elements, two: 8192 x 1600 21.8 us against 22.1 with
// one, 1600 x 8192 28.5 against 29.3).  The binary32 joined form has one and
// still spills vector registers at some widths: 9 with 8 or 16 threads a row,
// 12 with 32, 2 with 128 to 512, none with 1, 64 or 1024.
template <typename T, bool NORM, bool DROP, int TPR>
void launch_rows(const BwdArgs<T>& a, uint64_t chunks, hipStream_t s)
{
    constexpr int kBuffers = !NORM ? 4 : DROP || sizeof(T) == 4 ? 2 : 3;
    const uint64_t arrays = (NORM ? 3 + (a.dres != nullptr) : 2) + (NORM && DROP);
    if (a.rows * a.cols * sizeof(T) * arrays <= kStreamBytes)
        hipLaunchKernelGGL((rows_bwd_kernel<T, NORM, DROP, kRowsBlock, TPR, kBuffers, kCached>),
                           dim3(uint32_t(chunks)), dim3(kRowsBlock), 0, s, a);
    else
        hipLaunchKernelGGL((rows_bwd_kernel<T, NORM, DROP, kRowsBlock, TPR, kBuffers, kStreamed>),
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
        case 1: launch_rows<T, NORM, DROP, 1>(a, chunks, s); break;
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
    const uint64_t blocks = (c.cols + kFoldCols - 1) / kFoldCols;
    hipLaunchKernelGGL(fold_kernel<T>, dim3(uint32_t(blocks < 65536 ? blocks : 65536), 3), dim3(kFoldBlock), 0, s, out,
                       a.partials, uint32_t(chunks), uint32_t(c.cols));
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

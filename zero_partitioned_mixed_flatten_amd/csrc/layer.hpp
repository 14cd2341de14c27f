// layer.hpp -- what the layer operators share (dropout.hip, layernorm.hip,
// layernorm_bwd.hip): element types, vectors of 8 elements at any element
// alignment, the counter-based generator behind dropout, and sums over a
// workgroup.
#pragma once

#include <math.h>

#include "zero_internal.hpp"

namespace zero {
namespace layer {

typedef __bf16 bf16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// ---- vectors of 8 elements -----------------------------------------------------
// Every operator works on groups of 8 columns, the unit of the generator.  A
// group is loaded and stored with 16-byte instructions whatever its address:
// the declared alignment is the element's, which the target's unaligned
// global access serves in one instruction (rows of an odd width start
// anywhere).  Only a row's last group, when it is short, goes by elements.

template <typename T>
struct Raw;                                        // 8 elements as loaded
template <>
struct Raw<_Float16> {
    typedef f16x8 type;
};
template <>
struct Raw<bf16> {
    typedef bf16x8 type;
};
template <>
struct Raw<float> {
    typedef f32x8 type;
};

// The first k elements of a group (k <= 0: none), the others 0.
template <typename T>
__device__ __forceinline__ typename Raw<T>::type load8(const T* p, int k)
{
    typedef typename Raw<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    if (k >= 8)
        return __builtin_nontemporal_load(reinterpret_cast<const VU*>(p));
    V v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = T(0.0f);
    if (k > 0)
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < k)
                v[j] = p[j];
    return v;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, typename Raw<T>::type v, int k)
{
    typedef typename Raw<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    if (k >= 8)
        __builtin_nontemporal_store(v, reinterpret_cast<VU*>(p));
    else if (k > 0)
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < k)
                p[j] = v[j];
}

// 8 sums into a partial's row, which the fold reads back soon: kept in the caches.
__device__ __forceinline__ void store8_f32(float* p, f32x8 v, int k)
{
    typedef f32x8 __attribute__((aligned(4))) VU;
    if (k >= 8)
        *reinterpret_cast<VU*>(p) = v;
    else if (k > 0)
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < k)
                p[j] = v[j];
}

template <typename T>
__device__ __forceinline__ f32x8 widen(typename Raw<T>::type v)
{
    return __builtin_convertvector(v, f32x8);
}

template <typename T>
__device__ __forceinline__ typename Raw<T>::type narrow(f32x8 v)   // round to nearest even
{
    return __builtin_convertvector(v, typename Raw<T>::type);
}

// The vectors over the columns (weights, biases) have a type of their own:
// the matrices' or binary32.  An absent one (NULL) reads as `absent`.
template <typename T>
__device__ __forceinline__ f32x8 load8_vector(const void* p, bool f32, uint64_t col, int k, float absent)
{
    f32x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = absent;
    if (!p || k <= 0)
        return v;
    if (f32) {
        typedef f32x8 __attribute__((aligned(4))) VU;
        const float* q = static_cast<const float*>(p) + col;
        if (k >= 8)
            return *reinterpret_cast<const VU*>(q);
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < k)
                v[j] = q[j];
        return v;
    }
    typedef typename Raw<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    const T* q = static_cast<const T*>(p) + col;
    if (k >= 8)
        return widen<T>(*reinterpret_cast<const VU*>(q));
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < k)
            v[j] = float(q[j]);
    return v;
}

// ---- the generator ---------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw 2011): ten rounds of two
// 32 x 32 -> 64-bit products over a 128-bit counter under a 64-bit key.
// A group of 8 elements takes one block: 16 bits each, so the drop
// probability is a whole number of 2^-16.  Nothing is stored: the backward
// pass and a recomputed forward pass give the same counters again.  The ten
// rounds hide under the memory traffic of the pass around them (a 1 GiB
// fp16 pass measured 327.8 us with 10 rounds, 326.6 us with 7 and 330.3 us
// with none).
struct Drop {
    const zero_rng_t* rng;
    uint32_t site;
    uint32_t threshold;                            // dropped when the 16-bit word is below it; 0: nothing is
    float scale;                                   // 65536 / (65536 - threshold), rounded once; 0 when all is dropped
};

struct RngKey {
    uint32_t k0, k1, step;
};

__device__ __forceinline__ RngKey rng_key(const Drop& d)
{
    if (!d.threshold)
        return RngKey{0, 0, 0};
    const uint64_t seed = d.rng->seed;
    return RngKey{uint32_t(seed), uint32_t(seed >> 32), d.rng->step};
}

__device__ __forceinline__ u32x4 philox(RngKey key, uint32_t site, uint64_t group)
{
    uint32_t c0 = uint32_t(group), c1 = uint32_t(group >> 32), c2 = site, c3 = key.step;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ k0;
        c2 = uint32_t(a >> 32) ^ c3 ^ k1;
        c1 = uint32_t(b);
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// D(v): a dropped element is 0 whatever it holds (a select, not a product, so
// an inf or NaN there does not come through).
__device__ __forceinline__ f32x8 dropped(f32x8 v, const Drop& d, RngKey key, uint64_t group)
{
    if (!d.threshold)
        return v;
    const u32x4 bits = philox(key, d.site, group);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t word = (bits[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        v[j] = word >= d.threshold ? v[j] * d.scale : 0.0f;
    }
    return v;
}

// ---- sums over the threads of a row ------------------------------------------------------
// A row is shared by TPR threads.  Within a wave the sum goes through lane
// permutes of the vector ALU (DPP), each step a pairwise addition that both
// lanes do alike, so every thread of the row ends with the same bits.
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    v += dpp<0xB1>(v);                             // quad_perm 1,0,3,2: lane ^ 1
    v += dpp<0x4E>(v);                             // quad_perm 2,3,0,1: lane ^ 2
    v += dpp<0x141>(v);                            // row_half_mirror: the other quad of 8
    if (LANES >= 16)
        v += dpp<0x140>(v);                        // row_mirror: the other 8 of 16
    if (LANES >= 32)
        v += __shfl_xor(v, 16);
    if (LANES >= 64)
        v += __shfl_xor(v, 32);
    return v;
}

// The sums of N values over the TPR threads of each row of the workgroup, in
// every thread of the row.  Rows wider than a wave meet in LDS, one barrier
// a call: `scratch` is [2][N][BLOCK / 64] floats, its halves used in turn
// (`parity`), so a call's reads are over before the same half is written
// again.  Every thread of the workgroup calls it.
template <int BLOCK, int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* scratch, uint32_t& parity)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = lanes_sum<(TPR < 64 ? TPR : 64)>(v[i]);
    if (TPR <= 64)
        return;
    constexpr int kWaves = BLOCK / 64, kPerRow = TPR / 64;
    float* buf = scratch + parity * (N * kWaves);
    parity ^= 1;
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            buf[i * kWaves + wave] = v[i];
    __syncthreads();
    const uint32_t first = wave / kPerRow * kPerRow;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kPerRow; ++j)
            s += buf[i * kWaves + first + j];
        v[i] = s;
    }
}

// ---- host side ------------------------------------------------------------------------
inline bool dtype_ok(int t) { return t == ZERO_F16 || t == ZERO_BF16 || t == ZERO_F32; }
inline uint64_t dtype_size(int t) { return t == ZERO_F32 ? 4 : 2; }

// Sizes every operator accepts: rows and row strides whose offsets stay well
// inside 64 bits, columns whose groups fit 32.
constexpr uint64_t kMaxRows = uint64_t(1) << 40;
constexpr uint64_t kMaxCols = uint64_t(1) << 30;

inline int check_shape(uint64_t rows, uint64_t cols, int dtype)
{
    if (!dtype_ok(dtype))
        return ZERO_EINVAL;
    return rows > kMaxRows || cols > kMaxCols ? ZERO_ERANGE : ZERO_OK;
}

// A rows x cols matrix argument; `need`: NULL is an error.
inline int check_matrix(const void* p, uint64_t ld, uint64_t rows, uint64_t cols, int dtype, bool need)
{
    if (!p)
        return need && rows && cols ? ZERO_EINVAL : ZERO_OK;
    if (!is_aligned(p, dtype_size(dtype)))
        return ZERO_EALIGN;
    if (rows > 1 && (ld < cols || ld > (uint64_t(1) << 50) || (unsigned __int128)rows * ld > (uint64_t(1) << 56)))
        return ZERO_ERANGE;
    return ZERO_OK;
}

// A vector argument over the columns: the matrices' type or binary32.
inline int check_vector(const void* p, int vtype, int dtype)
{
    if (!p)
        return ZERO_OK;
    if (vtype != dtype && vtype != ZERO_F32)
        return ZERO_EINVAL;
    return is_aligned(p, dtype_size(vtype)) ? ZERO_OK : ZERO_EALIGN;
}

// Checks p and the generator and fills d.
int make_drop(double p, const zero_rng_t* rng, uint32_t site, Drop* d);

// ---- sums over the rows (layernorm_bwd.hip) ------------------------------------------
// The backward passes sum over the rows for up to three vectors at once (the
// gradients of w, b and the bias), each in binary32: a workgroup adds up the
// rows it owns in registers and stores one partial, and fold_kernel adds the
// partials in their order, so the result does not depend on timing.
struct SumOut {
    void* dst[3];                                  // w, b, bias gradients; NULL: not wanted
    bool f32;                                      // their type: binary32, or the matrices'
    bool accumulate;
};

}  // namespace layer
}  // namespace zero

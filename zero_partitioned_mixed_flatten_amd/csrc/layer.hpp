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
// anywhere).

// Cache hints of a pass: bit 0, loads nontemporal; bit 1, stores.  The passes
// that read each element once store so always and load so in a call that moves
// more than kStreamBytes: what a smaller one reads, the operator before it has
// mostly left in the 256 MB cache, while a larger one runs a little better past
// it.  What does not follow this: rows too wide for the registers are loaded
// plainly in the forward passes and the first time of a backward pass (the
// joined form's r is stored plainly too, it is read again), nontemporally the
// second time; what goes by elements (rows of fewer than 8 columns, a row's
// short last group when stored) and partial sums are plain.  Measured, plain
// against nontemporal loads: layer norm forward 1600 x 8192 fp16 (52 MB) 11.0
// and 13.3 us, backward 800 x 8192 (39 MB) 17.4 and 22.6 us, joined forward
// 1600 x 8192 (105 MB) 23.7 and 22.7 us, 16384 x 8192 (1.07 GB) 203 and 183 us.
constexpr int kCached = 2, kStreamed = 3;
constexpr uint64_t kStreamBytes = 96000000;

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

template <int HINT = kStreamed, typename T>
__device__ __forceinline__ typename Raw<T>::type load8_full(const T* p)
{
    typedef typename Raw<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    if (HINT & 1)
        return __builtin_nontemporal_load(reinterpret_cast<const VU*>(p));
    return *reinterpret_cast<const VU*>(p);
}

template <int HINT>
__device__ __forceinline__ f32x4 load4_full(const float* p)
{
    typedef f32x4 __attribute__((aligned(4))) VU;
    if (HINT & 1)
        return __builtin_nontemporal_load(reinterpret_cast<const VU*>(p));
    return *reinterpret_cast<const VU*>(p);
}

template <int HINT>
__device__ __forceinline__ void store4(float* p, f32x4 v, int k)
{
    typedef f32x4 __attribute__((aligned(4))) VU;
    if (k >= 4 && (HINT & 2))
        __builtin_nontemporal_store(v, reinterpret_cast<VU*>(p));
    else if (k >= 4)
        *reinterpret_cast<VU*>(p) = v;
    else if (k > 0)
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < k)
                p[j] = v[j];
}

// The first k elements of a group (k <= 0: none), the others 0.
template <typename T>
__device__ __forceinline__ typename Raw<T>::type load8(const T* p, int k)
{
    if (k >= 8)
        return load8_full<kStreamed>(p);
    typename Raw<T>::type v;
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

template <int HINT = kStreamed, typename T>
__device__ __forceinline__ void store8(T* p, typename Raw<T>::type v, int k)
{
    typedef typename Raw<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    if (k >= 8 && (HINT & 2))
        __builtin_nontemporal_store(v, reinterpret_cast<VU*>(p));
    else if (k >= 8)
        *reinterpret_cast<VU*>(p) = v;
    else if (k > 0)
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < k)
                p[j] = v[j];
}

// Where a group of 8 columns is loaded without a branch (a branch around a load
// makes the next load wait for it), in a row of at least 8 columns: a group
// past the row's last 8 columns reads those 8 instead (memory of the row), and
// settling moves the elements to their places and puts 0 in the others.
struct Group {
    uint32_t at;                                   // first column loaded
    uint32_t shift;                                // the group's column - at; 8 and more: no columns in the row
    int k;                                         // columns in the row: 8, less in the last group, <= 0 past it
};

__device__ __forceinline__ Group group_at(uint32_t col, uint32_t cols)
{
    const uint32_t at = col < cols - 8 ? col : cols - 8;
    return Group{at, col - at, int(cols) - int(col)};
}

// Moves WORDS words down by `shift` elements of BITS bits, 0 from above.
template <int WORDS, int BITS>
__device__ __forceinline__ void shift_down(uint32_t (&d)[WORDS], uint32_t shift)
{
#pragma unroll
    for (int bit = BITS == 16 ? 2 : 1; bit >= 0; --bit) {
        const bool on = (shift >> bit) & 1;
        const int words = (1 << bit) * BITS / 32;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            uint32_t moved;
            if (words)
                moved = i + words < WORDS ? d[i + words < WORDS ? i + words : 0] : 0;
            else
                moved = (d[i] >> 16) | (i + 1 < WORDS ? d[i + 1 < WORDS ? i + 1 : 0] << 16 : 0);
            d[i] = on ? moved : d[i];
        }
    }
}

// The part of a row that one of its TPR threads holds in pass i, and how it is
// loaded and stored.  16-bit elements: the thread's group, one 16-byte access.
// Binary32: a group is two 16-byte pieces, and threads that each accessed
// their own 32 bytes would leave every access of a wave with half of each line
// (a plain copy done so runs at 3.9 TB/s against 6.2).  So the threads of a
// wave access the pieces of 2 * 64 consecutive pieces in order, 64 at a time,
// and neighbours trade: an even thread ends with the group whose two pieces
// the pair has in the first access, an odd one with the second's.  TPR = 1:
// a row of fewer than 8 columns, by elements.
template <typename T, int TPR>
struct Part {
    static constexpr int kPieces = sizeof(T) == 4 ? 2 : 1;
    static constexpr uint32_t kPer = 8 / kPieces;  // elements of a piece
    uint32_t group;
    int k;                                         // the group's columns in the row
    uint32_t at[kPieces], shift[kPieces];          // the pieces as loaded
    int have[kPieces];                             // the pieces' columns in the row

    __device__ __forceinline__ Part(uint32_t i, uint32_t t, uint32_t cols)
    {
        if (TPR == 1) {
            group = 0;
            k = have[0] = int(cols);
            return;
        }
        if (kPieces == 1) {
            group = i * TPR + t;
            at[0] = group * 8;
        } else {
            constexpr uint32_t kSpan = TPR < 64 ? TPR : 64;
            const uint32_t lane = t % kSpan, base = i * TPR + (t - lane);
            group = base + lane / 2 + (lane & 1) * (kSpan / 2);
            at[0] = base * 8 + lane * 4;
            at[kPieces - 1] = at[0] + kSpan * 4;
        }
        k = int(cols) - int(group * 8);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const uint32_t col = at[p];
            have[p] = int(cols) - int(col);
            at[p] = col < cols - kPer ? col : cols - kPer;
            shift[p] = col - at[p];
        }
    }

    template <int HINT>
    __device__ __forceinline__ typename Raw<T>::type load(const T* row) const
    {
        if constexpr (TPR == 1) {
            return load8(row, k);
        } else if constexpr (kPieces == 1) {
            return load8_full<HINT>(row + at[0]);
        } else {
            const f32x4 a = load4_full<HINT>(row + at[0]), b = load4_full<HINT>(row + at[1]);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // What load() gave, as the thread's group.  `ragged`: cols is not a multiple
    // of 8 (the same for every thread).  ZERO false: groups with no columns in
    // the row may hold anything.
    template <bool ZERO = true>
    __device__ __forceinline__ typename Raw<T>::type settle(typename Raw<T>::type v, bool ragged) const
    {
        if constexpr (TPR == 1) {
            return v;
        } else {
            constexpr int kWords = 2 * int(sizeof(T)) / kPieces;
            struct Words {
                uint32_t d[kPieces][kWords];
            };
            Words x = __builtin_bit_cast(Words, v);
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (ragged) {
                    uint32_t by = shift[p];
                    asm volatile("" : "+v"(by));   // its tests stay in this branch
                    shift_down<kWords, 8 * int(sizeof(T))>(x.d[p], by);
                }
                if (ZERO)
#pragma unroll
                    for (int i = 0; i < kWords; ++i)
                        x.d[p][i] = shift[p] < kPer ? x.d[p][i] : 0;
            }
            if constexpr (kPieces == 2)
                trade(x.d[0], x.d[1]);
            return __builtin_bit_cast(typename Raw<T>::type, x);
        }
    }

    template <int HINT>
    __device__ __forceinline__ void store(T* row, typename Raw<T>::type v, bool live) const
    {
        if constexpr (kPieces == 1 || TPR == 1) {
            store8<HINT>(row + group * 8, v, live ? k : 0);
        } else {
            struct Words {
                uint32_t d[2][4];
            };
            Words x = __builtin_bit_cast(Words, v);
            trade(x.d[0], x.d[1]);
            store4<HINT>(row + at[0] + shift[0], __builtin_bit_cast(f32x4, x.d[0]), live ? have[0] : 0);
            store4<HINT>(row + at[1] + shift[1], __builtin_bit_cast(f32x4, x.d[1]), live ? have[1] : 0);
        }
    }

    // The even thread gives its second piece and takes the odd one's first: its own inverse.
    static __device__ __forceinline__ void trade(uint32_t (&lo)[4], uint32_t (&hi)[4])
    {
        const bool odd = threadIdx.x & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t give = odd ? lo[i] : hi[i];
            const uint32_t take = __builtin_amdgcn_update_dpp(0, give, 0xB1, 0xf, 0xf, true);   // lane ^ 1
            lo[i] = odd ? take : lo[i];
            hi[i] = odd ? hi[i] : take;
        }
    }
};

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

// raw + b, raw * a, raw * a + b and v * a + raw, elementwise, rounded once.
// binary16 elements are widened inside the instruction (v_fma_mix_f32), which
// the compiler forms only for a product: `one` is a 1 that it cannot see.
__device__ __forceinline__ float opaque_one()
{
    float one = 1.0f;
    asm("" : "+s"(one));
    return one;
}

template <typename T>
__device__ __forceinline__ f32x8 raw_plus(typename Raw<T>::type raw, f32x8 b, float one)
{
    f32x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __is_same(T, _Float16) ? __builtin_fmaf(float(raw[j]), one, b[j]) : float(raw[j]) + b[j];
    return v;
}

template <typename T>
__device__ __forceinline__ f32x8 raw_times(typename Raw<T>::type raw, f32x8 a)
{
    f32x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __is_same(T, _Float16) ? __builtin_fmaf(float(raw[j]), a[j], -0.0f) : float(raw[j]) * a[j];
    return v;
}

template <typename T>
__device__ __forceinline__ f32x8 raw_fma(typename Raw<T>::type raw, f32x8 a, f32x8 b)
{
    f32x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __builtin_fmaf(float(raw[j]), a[j], b[j]);
    return v;
}

template <typename T>
__device__ __forceinline__ f32x8 fma_raw(f32x8 v, float a, typename Raw<T>::type raw)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __builtin_fmaf(v[j], a, float(raw[j]));
    return v;
}

__device__ __forceinline__ f32x8 splat(float x) { return f32x8{x, x, x, x, x, x, x, x}; }

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

// The same without a branch on the thread (see Group), for loads inside a
// loop; groups with no columns in the row may hold anything.
template <typename T>
__device__ __forceinline__ f32x8 load8_vector_at(const void* p, bool f32, const Group& at, bool ragged, float absent)
{
    if (!p)
        return splat(absent);
    f32x8 v;
    if (f32) {
        typedef f32x8 __attribute__((aligned(4))) VU;
        v = *reinterpret_cast<const VU*>(static_cast<const float*>(p) + at.at);
    } else {
        typedef typename Raw<T>::type V;
        typedef V __attribute__((aligned(sizeof(T)))) VU;
        v = widen<T>(*reinterpret_cast<const VU*>(static_cast<const T*>(p) + at.at));
    }
    if (ragged) {
        struct Words {
            uint32_t d[8];
        };
        Words x = __builtin_bit_cast(Words, v);
#pragma unroll
        for (int bit = 2; bit >= 0; --bit)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int from = i + (1 << bit);
                x.d[i] = (at.shift >> bit) & 1 ? (from < 8 ? x.d[from < 8 ? from : 0] : 0) : x.d[i];
            }
        v = __builtin_bit_cast(f32x8, x);
    }
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
    uint32_t threshold;                            // dropped when the 16-bit word is below it; 0: nothing is, 65536: all
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
    uint32_t k0 = __builtin_amdgcn_readfirstlane(key.k0), k1 = __builtin_amdgcn_readfirstlane(key.k1);
    // the ten rounds' keys are scalar additions next to the vector work; kept
    // from one call to the next they would push other scalars out
    asm volatile("" : "+s"(k0), "+s"(k1));
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = __builtin_amdgcn_bitop3_b32(uint32_t(b >> 32), c1, k0, 0x96);   // the exclusive or of the three
        c2 = __builtin_amdgcn_bitop3_b32(uint32_t(a >> 32), c3, k1, 0x96);
        c1 = uint32_t(b);
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// The random bits of a group, which depend on nothing that is loaded: a pass
// draws them while its loads are on their way.
__device__ __forceinline__ u32x4 mask_bits(const Drop& d, RngKey key, uint64_t group)
{
    if (d.threshold - 1 > 0xfffeu)                 // none or all dropped
        return u32x4{0, 0, 0, 0};
    return philox(key, d.site, group);
}

// D(v): a dropped element is 0 whatever it holds (a select, not a product, so
// an inf or NaN there does not come through).  The 16-bit words are compared
// in the upper half of a register: the odd ones as they are, what is below
// them does not change the order.
__device__ __forceinline__ f32x8 dropped(f32x8 v, const Drop& d, u32x4 bits)
{
    if (!d.threshold)
        return v;
    if (d.threshold > 0xffffu)
        return splat(0.0f);
    const uint32_t limit = d.threshold << 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t word = j & 1 ? bits[j >> 1] : bits[j >> 1] << 16;
        v[j] = word >= limit ? v[j] * d.scale : 0.0f;
    }
    return v;
}

// ---- sums over the threads of a row ------------------------------------------------------
// A row is shared by TPR threads.  Within a wave the sum goes through lane
// permutes of the vector ALU (DPP): up to 16 lanes by pairwise additions that
// both lanes do alike, then by adding up the rows of 16; every thread of the
// row ends with the same bits.
// ROWS: the rows of 16 lanes that take part, the others get 0.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, ROWS == 0xf));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    static_assert(LANES == 1 || LANES == 8 || LANES == 16 || LANES == 32 || LANES == 64, "lanes of a row");
    if (LANES >= 8) {
        v += dpp<0xB1>(v);                         // quad_perm 1,0,3,2: lane ^ 1
        v += dpp<0x4E>(v);                         // quad_perm 2,3,0,1: lane ^ 2
        v += dpp<0x141>(v);                        // row_half_mirror: the other quad of 8
    }
    if (LANES >= 16)
        v += dpp<0x140>(v);                        // row_mirror: the other 8 of 16
    if (LANES == 32)
        v += __shfl_xor(v, 16);
    if (LANES >= 64) {                             // rows of 16 lanes: 1 += 0 and 3 += 2, then 3 += 1; lane 63 has it all
        v += dpp<0x142, 0xa>(v);                   // row_bcast 15
        v += dpp<0x143, 0xc>(v);                   // row_bcast 31
        v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    }
    return v;
}

// s / n for a whole number n and inv = fp32(1 / n): the product corrected by
// its remainder, which gives the rounded quotient at 5 instructions (an inf or
// NaN stays what the product makes of it).
__device__ __forceinline__ float over(float s, float n, float inv)
{
    const float q = s * inv, rest = __builtin_fmaf(-q, n, s);
    return rest == rest ? __builtin_fmaf(rest, inv, q) : q;
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
    // each wave adds up its row's waves in its first 8 or 16 lanes' order
    constexpr int kLanes = kPerRow <= 8 ? 8 : 16;
    const uint32_t j = threadIdx.x % kLanes, first = wave / kPerRow * kPerRow;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float part = buf[i * kWaves + first + (j < kPerRow ? j : 0)];
        v[i] = lanes_sum<kLanes>(j < kPerRow ? part : 0.0f);
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

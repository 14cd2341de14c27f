// attention.hip -- causal attention over packed sequences with a sliding
// window, first tokens that stay visible and a learned relative position bias
// by buckets, forward.
//
//   s_ij = scale q_i.k_j + bias[h][bucket(i - j)]   for visible (i, j)
//   o_i = sum_j exp(s_ij - lse_i) v_j,   lse_i = log sum_j exp(s_ij)
//
// One pass over the visible keys with a running maximum and sum of each row.  A
// workgroup owns 128 queries of a head, 32 a wave, and goes over tiles of 64 keys,
// two in LDS: one is fetched under the other's products.  Of a wave's 32 x 32
// scores each lane owns a query (attention.hpp), so a row's maximum and sum are
// the lane's own but for one exchange, and the weights go from the first product's
// registers to the second's operand.
//
// Bound by issue: the exponentials, masks and roundings of 32 x 32 scores (some
// 110 vector instructions at 64 columns, 150 at 128) and the products follow one
// another in a wave, and waves overlap little of them.  Left out in trials at
// 8 x 1024 positions: both products, 60% of the time stays; the tiles' fetches,
// 85%.  8 x 1024 positions, 25 heads of 64: 46-49 us, 549-582 TFLOP/s of the visible
// pairs.  2 x 4096 positions, 64 heads of 128 on 8 of keys, window 512: 204-217 us,
// 599-637 TFLOP/s.  Operands read further ahead, two tiles a turn of the loop and
// wave priorities gave nothing; no bank conflicts are counted.  64 columns take
// 124 registers, four waves a SIMD; with the bias' table 130, three.
#include <type_traits>
#include <vector>

#include "attention.hpp"

namespace zero {
namespace attention {
namespace {

template <typename T>
struct FwdArgs {
    Heads<T> o;
    float* lse;
    Heads<const T> q, k, v;
    Shape s;
    Buckets b;
    Order order;
};

// binary16 has no numbers below 2^-24, and a row may have many keys whose weights are below that beside the largest: the
// weights are formed in units of 2^-7, where the largest and the 2^8 that a maximum may lag behind leave room.
template <typename T>
constexpr float kLift = __is_same(T, _Float16) ? 7.0f : 0.0f;

// The output of one row by a wave, from its maximum and sum, over the keys that
// it sees and no others: 64 keys a time, a lane a key for their weights, then a
// lane a column.  Slow, a row after the other (all rows of 2 x 4096 positions, 64
// heads of 128, window 512: 38 ms for 0.2); for rows of a tile beside an inf or
// NaN value that they do not see.  Rows that do see one come this way too, unless
// their scores have one as well, and end where all their columns are NaN.
template <typename T, int DIM, int BIAS>
__device__ __forceinline__ void sum_row(const FwdArgs<T>& a, const Piece& at, uint32_t head, uint32_t i, float m, float sum)
{
    typedef typename Vec8<T>::type VU __attribute__((aligned(sizeof(T))));
    const Shape& s = a.s;
    const uint32_t lane = threadIdx.x & 63;
    const T* q = a.q.p + (uint64_t(at.start) + i) * a.q.ld + uint64_t(head) * a.q.hs;
    const T* kp = a.k.p + uint64_t(at.start) * a.k.ld + uint64_t(head / s.group) * a.k.hs;
    const T* vp = a.v.p + uint64_t(at.start) * a.v.ld + uint64_t(head / s.group) * a.v.hs;
    const float base = (m == -INFINITY ? 0.0f : m) - kLift<T>;
    float acc[DIM / 64] = {};
    const uint32_t near = i >= s.window ? (i - s.window + 1) & ~63u : 0;         // where the window's keys start
    for (uint32_t j0 = 0; j0 <= i; j0 = j0 + 64 >= s.sinks && j0 + 64 < near ? near : j0 + 64) {
        const uint32_t j = j0 + lane;
        const bool in = j <= i && (i - j < s.window || j < s.sinks);
        float p = 0.0f;
        if (in) {
            for (uint32_t d = 0; d < s.dim; d += 8) {
                const VU x = *reinterpret_cast<const VU*>(q + d), y = *reinterpret_cast<const VU*>(kp + j * a.k.ld + d);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p = __builtin_fmaf(float(x[e]), float(y[e]), p);
            }
            p *= s.scale2;
            if (BIAS != kNoBias)
                p += bias_value<T>(a.b, head, bucket_of(a.b.starts, a.b.count, i - j)) * kLog2e;
            p = __builtin_amdgcn_exp2f(p - base);
        }
        auto add = [&](uint32_t k) {
            const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, p), k));
#pragma unroll
            for (int n = 0; n < DIM / 64; ++n)
                if (lane + 64 * n < s.dim)
                    acc[n] = __builtin_fmaf(w, float(vp[(j0 + k) * a.v.ld + lane + 64 * n]), acc[n]);
        };
        uint64_t left = __ballot(in);
        if (left == ~0ull)                         // loads ahead of the sums
#pragma unroll 16
            for (uint32_t k = 0; k < 64; ++k)
                add(k);
        else
            for (; left; left &= left - 1)
                add(__builtin_ctzll(left));
        bool open = false;
#pragma unroll
        for (int n = 0; n < DIM / 64; ++n)
            open |= lane + 64 * n < s.dim && acc[n] == acc[n];
        if (!__ballot(open))
            break;
    }
#pragma unroll
    for (int n = 0; n < DIM / 64; ++n)
        if (lane + 64 * n < s.dim)
            a.o.p[(uint64_t(at.start) + i) * a.o.ld + uint64_t(head) * a.o.hs + lane + 64 * n] = T(acc[n] / sum);
}

template <typename T, int DIM, int BIAS, bool DIRECT>
__global__ __launch_bounds__(kBlock, DIM == 64 ? 3 : 2) void attention_fwd_kernel(FwdArgs<T> a)
{
    typedef Tile<DIM> L;
    __shared__ alignas(16) T keys[2][L::kElems];
    __shared__ alignas(16) T values[2][L::kElems];
    __shared__ typename std::conditional<BIAS == kLine, BiasLine, int>::type bias;
    extern __shared__ __attribute__((aligned(16))) float table[];               // BIAS == kTable: of table_size() distances

    const Shape& s = a.s;
    uint32_t head, slot;
    Piece at;
    if (!a.order.template find<true>(s, blockIdx.x, &head, &slot) || !find_piece(s, slot, kOwn, &at))
        return;
    const uint32_t lane = threadIdx.x & 63, c = lane % 32, h = lane / 32;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t first = at.first + 32 * wave, mine = first + c;       // the wave's queries, the lane's
    const uint32_t row = mine < at.len ? mine : at.len - 1;
    const T* kp = a.k.p + uint64_t(at.start) * a.k.ld + uint64_t(head / s.group) * a.k.hs;
    const T* vp = a.v.p + uint64_t(at.start) * a.v.ld + uint64_t(head / s.group) * a.v.hs;

    const KeyTiles tiles(s, at.first, kOwn, at.len);
    const Places<DIM> places;
    Carrier<T, DIM, DIRECT> nk, nv;
    uint32_t t = tiles.begin();
    clear<T, DIM, DIRECT>(keys[0], 2 * L::kElems, s.dim);
    clear<T, DIM, DIRECT>(values[0], 2 * L::kElems, s.dim);
    cleared<DIRECT, DIM>(s.dim);
    nk.fetch(keys[0], kp, a.k.ld, t * kTile, at.len, s.dim);
    nv.fetch(values[0], vp, a.v.ld, t * kTile, at.len, s.dim);
    Operand<T, DIM> q;
    load_operand<T, DIM>(q, a.q.p + uint64_t(at.start) * a.q.ld + uint64_t(head) * a.q.hs, a.q.ld, row, s.dim);
    float beyond = 0.0f;                           // kTable: the bias of the last bucket
    if constexpr (BIAS == kTable) {
        draw_table<T>(table, a.b, head);
        beyond = bias_value<T>(a.b, head, a.b.count - 1) * kLog2e;
    }
    if constexpr (BIAS == kLine) {
        load_line_values<T>(bias, a.b, head);
        __syncthreads();
    }
    auto draw_line = [&](uint32_t tile, int buf) {
        if constexpr (BIAS == kLine)
            bias.draw(buf, a.b.count, int(at.first + kOwn - 1) - int(tile * kTile), -1);
    };

    f32x16 acc[DIM / 32] = {};
    float m = -INFINITY, sum = 0.0f;               // in units of log2; the sum over this half of the keys, in the weights' units
    nk.put(keys[0]);
    nv.put(values[0]);
    draw_line(t, 0);
    int buf = 0;
    while (true) {
        const uint32_t next = tiles.next(t);
        const bool more = next < tiles.end;
        tiles_there<DIRECT>();
        if (more) {
            nk.fetch(keys[buf ^ 1], kp, a.k.ld, next * kTile, at.len, s.dim);
            nv.fetch(values[buf ^ 1], vp, a.v.ld, next * kTile, at.len, s.dim);
        }
        const uint32_t j0 = t * kTile;
        const Seen see = seen(s, first, 32, j0, kTile);
        if (see != kNone) {
            f32x16 x[2];
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
                x[sub] = rows_times<T, DIM>(keys[buf], places, sub, q);
            // the scores are scores * factor + shift: where the bias is of one bucket it is the shift, else it is in them
            float factor = s.scale2, shift = beyond;
            if (BIAS == kLine || (BIAS == kTable && nearest(first, j0, kTile) < a.b.starts[a.b.count - 1])) {
                const float* line = BIAS == kLine ? &bias_line(bias, buf)[kOwn - 1 - 32 * wave - c + 4 * h]
                                                  : table + (int(mine) - int(j0) - (kTile - 1) + kTableBefore - 4 * int(h));
#pragma unroll
                for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int j = 32 * sub + row_of(r, 0);
                        x[sub][r] = __builtin_fmaf(x[sub][r], s.scale2, line[BIAS == kLine ? j : kTile - 1 - j]);
                    }
                factor = 1.0f;
                shift = 0.0f;
            }
            if (see == kSome) {
                const Mask mask = Mask::keys(s, mine, j0 + 4 * h);
#pragma unroll
                for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        x[sub][r] = mask.seen_or(x[sub][r], 0xff800000u, sub, r);      // -inf
            }
            float top = x[0][0];
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    top = fmaxf(top, x[sub][r]);
            top = halves_max(top);
            top = __builtin_fmaf(top, factor, shift);
            // the sums go by the maximum so far until it has been passed by a factor of 2^8: they have the room, and most tiles
            // need not touch them
            if (__any(top > m + 8.0f)) {
                const float higher = fmaxf(top, m), fall = higher == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - higher);
                m = higher;
                sum *= fall;
#pragma unroll
                for (int n = 0; n < DIM / 32; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        acc[n][r] *= fall;
            }
            const float base = (m == -INFINITY ? 0.0f : m) - shift - kLift<T>;
            float part = 0.0f;                     // the tile's, so that small weights do not meet a large sum one by one
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    x[sub][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[sub][r], factor, -base));
                    part += x[sub][r];
                }
            sum += part;
            // the weights are rounded to the element type, as the matrix instruction takes them, where the binary32 sum they are
            // divided by is of the unrounded ones: half a step of each, in binary16 of those above 2^-21 of the row's largest;
            // below it 2^-32 of the largest at most
#pragma unroll
            for (int step = 0; step < 4; ++step)
                columns_times<T, DIM>(acc, values[buf], places, step, rounded<T>(x[step / 2], step % 2));
        }
        if (!more)
            break;
        t = next;
        buf ^= 1;
        nk.put(keys[buf]);
        nv.put(values[buf]);
        draw_line(t, buf);
    }
    sum = halves_sum(sum);
    const bool live = mine < at.len;
    // a weight of 0 times an inf or NaN value is a NaN: rows with one are summed again over the keys that they see
    float probe = 0.0f;
#pragma unroll
    for (int n = 0; n < DIM / 32; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            probe = __builtin_fmaf(acc[n][r], 0.0f, probe);
    const uint64_t marked = __ballot(probe != probe && sum < INFINITY);          // a NaN or inf among the scores stays what it is
    uint32_t again = uint32_t(marked) | uint32_t(marked >> 32);
    store_columns<T, DIM>(a.o.p + uint64_t(at.start) * a.o.ld + uint64_t(head) * a.o.hs, a.o.ld, mine, live && !(again >> c & 1), s.dim, acc, 1.0f / sum);
    if (a.lse && live && h == 0)
        a.lse[uint64_t(head) * s.tokens + at.start + mine] = (m + __builtin_amdgcn_logf(sum * __builtin_ldexpf(1.0f, -int(kLift<T>)))) * kLn2;
    for (; again; again &= again - 1) {
        const uint32_t i = __builtin_ctz(again);
        if (first + i < at.len)
            sum_row<T, DIM, BIAS>(a, at, head, first + i, __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, m), i)),
                                  __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sum), i)));
    }
}

template <typename T, int DIM, bool DIRECT>
int launch(const FwdArgs<T>& a, hipStream_t stream)
{
    const uint32_t blocks = uint32_t(a.order.blocks(a.s));
    if (!a.b.count)
        hipLaunchKernelGGL((attention_fwd_kernel<T, DIM, kNoBias, DIRECT>), dim3(blocks), dim3(kBlock), 0, stream, a);
    else if (table_fits(a.b))
        hipLaunchKernelGGL((attention_fwd_kernel<T, DIM, kTable, DIRECT>), dim3(blocks), dim3(kBlock), table_size(a.b) * 4, stream, a);
    else
        hipLaunchKernelGGL((attention_fwd_kernel<T, DIM, kLine, DIRECT>), dim3(blocks), dim3(kBlock), 0, stream, a);
    return launch_status();
}

}  // namespace

int make_shape(const zero_attention_t* a, uint64_t tokens, const int32_t* dev_offsets, uint64_t sequences, int dtype,
               const void* bias, int vec_dtype, Shape* s, Buckets* b)
{
    if (!a || (dtype != ZERO_F16 && dtype != ZERO_BF16))
        return ZERO_EINVAL;
    if (!a->heads || !a->kv_heads || a->heads % a->kv_heads || !a->dim || a->dim % 8)
        return ZERO_EINVAL;
    const float scale = float(a->scale), scale2 = float(a->scale * 1.4426950408889634);
    if (!(scale > 0.0f) || !isfinite(scale) || !(scale2 > 0.0f) || !isfinite(scale2))
        return ZERO_EINVAL;
    if (a->heads > kMaxHeads || a->dim > 128 || tokens > kMaxTokens || sequences > kMaxTokens || a->buckets > ZERO_MAX_BUCKETS)
        return ZERO_ERANGE;
    if (!!bias != !!a->buckets)
        return ZERO_EINVAL;
    if (tokens && (!sequences || (!dev_offsets && tokens % sequences)))
        return ZERO_EINVAL;
    if (dev_offsets && !is_aligned(dev_offsets, 4))
        return ZERO_EALIGN;
    for (uint32_t i = 0; i < a->buckets; ++i)
        if (i ? a->starts[i] <= a->starts[i - 1] : a->starts[i] != 0)
            return ZERO_EINVAL;
    const int rc = layer::check_vector(bias, vec_dtype, dtype);
    if (rc)
        return rc;
    s->offsets = dev_offsets;
    s->tokens = uint32_t(tokens);
    s->sequences = uint32_t(sequences);
    s->length = sequences ? uint32_t(tokens / sequences) : 0;
    s->heads = a->heads;
    s->group = a->heads / a->kv_heads;
    s->dim = a->dim;
    s->window = a->window && a->window < 0xffffffffu ? uint32_t(a->window) : 0xffffffffu;
    s->sinks = a->sinks;
    s->scale = scale;
    s->scale2 = scale2;
    b->table = bias;
    b->count = a->buckets;
    b->f32 = vec_dtype == ZERO_F32;
    for (uint32_t i = 0; i < ZERO_MAX_BUCKETS; ++i)
        b->starts[i] = i < a->buckets ? a->starts[i] : 0xffffffffu;
    if (tokens && slots_of(s->tokens, s->sequences, dev_offsets != nullptr, kOwn) * a->heads >= kMaxPieces)
        return ZERO_ERANGE;
    return ZERO_OK;
}

namespace {

template <typename T>
int run_fwd(void* o, uint64_t ld_o, uint64_t hs_o, float* lse, const void* q, uint64_t ld_q, uint64_t hs_q, const void* k, uint64_t ld_k,
            uint64_t hs_k, const void* v, uint64_t ld_v, uint64_t hs_v, const Shape& s, const Buckets& b, hipStream_t stream)
{
    const FwdArgs<T> a{{static_cast<T*>(o), ld_o, hs_o}, lse, {static_cast<const T*>(q), ld_q, hs_q}, {static_cast<const T*>(k), ld_k, hs_k},
                       {static_cast<const T*>(v), ld_v, hs_v}, s, b, Order(s, s.heads, slots_of(s.tokens, s.sequences, s.offsets != nullptr, kOwn))};
    if (direct(k, ld_k, hs_k) && direct(v, ld_v, hs_v))
        return s.dim <= 64 ? launch<T, 64, true>(a, stream) : launch<T, 128, true>(a, stream);
    return s.dim <= 64 ? launch<T, 64, false>(a, stream) : launch<T, 128, false>(a, stream);
}

// 0 in the rows before the first sequence and behind the last, 8 elements a
// thread: bound by the bytes of those rows, or where there are none by the launch.
template <typename T>
__global__ __launch_bounds__(kBlock) void clear_rows_kernel(Heads<T> x, uint64_t tokens, uint32_t heads, uint32_t dim, const int32_t* offsets,
                                                            uint64_t sequences)
{
    typedef T V0 __attribute__((ext_vector_type(8)));
    typedef V0 V __attribute__((aligned(sizeof(T))));
    auto offset = [&](uint64_t i) {
        const int32_t o = offsets[i];
        return o < 0 ? uint64_t(0) : uint64_t(o) < tokens ? uint64_t(o) : tokens;
    };
    const uint64_t first = offset(0), end = offset(sequences);
    const uint32_t pieces = dim / 8;
    const uint64_t row = uint64_t(heads) * pieces, items = (first + (end < tokens ? tokens - (end > first ? end : first) : 0)) * row;
    for (uint64_t i = uint64_t(blockIdx.x) * kBlock + threadIdx.x; i < items; i += uint64_t(gridDim.x) * kBlock) {
        const uint64_t r = i / row, token = r < first ? r : r - first + (end > first ? end : first);
        const uint32_t rest = uint32_t(i - r * row), head = rest / pieces;
        *reinterpret_cast<V*>(x.p + token * x.ld + head * x.hs + (rest - head * pieces) * 8) = V0{};
    }
}

// A natural number of any size, for comparing powers.
struct Natural {
    std::vector<uint32_t> d{1};
    void times(uint32_t f)
    {
        uint64_t carry = 0;
        for (uint32_t& x : d) {
            carry += uint64_t(x) * f;
            x = uint32_t(carry);
            carry >>= 32;
        }
        if (carry)
            d.push_back(uint32_t(carry));
    }
    bool below(const Natural& o) const
    {
        if (d.size() != o.d.size())
            return d.size() < o.d.size();
        for (size_t i = d.size(); i--;)
            if (d[i] != o.d[i])
                return d[i] < o.d[i];
        return false;
    }
};

}  // namespace
}  // namespace attention
}  // namespace zero

using namespace zero;
using namespace zero::attention;

extern "C" int zero_attention_buckets(uint32_t* starts, uint32_t buckets, uint32_t max_distance)
{
    if (!starts || !buckets)
        return ZERO_EINVAL;
    const uint32_t half = buckets / 2, n = buckets - half;
    if (buckets > ZERO_MAX_BUCKETS || max_distance > (1u << 30))
        return ZERO_ERANGE;
    if (buckets == 1) {
        starts[0] = 0;
        return ZERO_OK;
    }
    if (max_distance <= half)
        return ZERO_EINVAL;
    for (uint32_t b = 0; b < half; ++b)
        starts[b] = b;
    try {
        for (uint32_t b = 0; b < n; ++b) {
            // the smallest d with d^n half^b >= max_distance^b half^n: bisected in whole numbers
            Natural most;
            for (uint32_t i = 0; i < b; ++i) most.times(max_distance);
            for (uint32_t i = 0; i < n; ++i) most.times(half);
            uint32_t low = half, high = max_distance;          // high always reaches it
            while (low < high) {
                const uint32_t mid = low + (high - low) / 2;
                Natural x;
                for (uint32_t i = 0; i < n; ++i) x.times(mid);
                for (uint32_t i = 0; i < b; ++i) x.times(half);
                if (x.below(most)) low = mid + 1;
                else high = mid;
            }
            starts[half + b] = low > starts[half + b - 1] ? low : starts[half + b - 1] + 1;
        }
    } catch (const std::bad_alloc&) {
        return ZERO_ENOMEM;
    }
    return ZERO_OK;
}

extern "C" int zero_attention_clear_rows(void* x, uint64_t ld, uint64_t hs, uint64_t tokens, uint32_t heads, uint32_t dim, int dtype,
                                         const int32_t* dev_offsets, uint64_t sequences, void* stream)
{
    if (!layer::dtype_ok(dtype) || !heads || !dim || dim % 8 || !dev_offsets)
        return ZERO_EINVAL;
    if (!is_aligned(dev_offsets, 4))
        return ZERO_EALIGN;
    if (heads > kMaxHeads || dim > 128 || tokens > kMaxTokens || sequences > kMaxTokens)
        return ZERO_ERANGE;
    const int rc = check_heads(x, ld, hs, tokens, heads, dim, dtype);
    if (rc || !tokens)
        return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const uint64_t most = (tokens * heads * (dim / 8) + kBlock - 1) / kBlock;
    const dim3 grid(uint32_t(most < 1024 ? most : 1024));
    if (dtype == ZERO_F32)
        hipLaunchKernelGGL(clear_rows_kernel<float>, grid, dim3(kBlock), 0, s, Heads<float>{static_cast<float*>(x), ld, hs}, tokens, heads, dim,
                           dev_offsets, sequences);
    else                                           // the zeros of both 16-bit types are the same bits
        hipLaunchKernelGGL(clear_rows_kernel<_Float16>, grid, dim3(kBlock), 0, s, Heads<_Float16>{static_cast<_Float16*>(x), ld, hs}, tokens,
                           heads, dim, dev_offsets, sequences);
    return launch_status();
}

extern "C" int zero_attention_fwd(void* o, uint64_t ld_o, uint64_t hs_o, float* lse, const void* q, uint64_t ld_q, uint64_t hs_q,
                                  const void* k, uint64_t ld_k, uint64_t hs_k, const void* v, uint64_t ld_v, uint64_t hs_v,
                                  const void* bias, int vec_dtype, const zero_attention_t* params, uint64_t tokens,
                                  const int32_t* dev_offsets, uint64_t sequences, int dtype, void* stream)
{
    Shape s;
    Buckets b;
    int rc = make_shape(params, tokens, dev_offsets, sequences, dtype, bias, vec_dtype, &s, &b);
    if (!rc) rc = check_heads(o, ld_o, hs_o, tokens, params->heads, params->dim, dtype);
    if (!rc) rc = check_heads(q, ld_q, hs_q, tokens, params->heads, params->dim, dtype);
    if (!rc) rc = check_heads(k, ld_k, hs_k, tokens, params->kv_heads, params->dim, dtype);
    if (!rc) rc = check_heads(v, ld_v, hs_v, tokens, params->kv_heads, params->dim, dtype);
    if (!rc && lse && !is_aligned(lse, 4)) rc = ZERO_EALIGN;
    if (rc || !tokens)
        return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == ZERO_F16)
        return run_fwd<_Float16>(o, ld_o, hs_o, lse, q, ld_q, hs_q, k, ld_k, hs_k, v, ld_v, hs_v, s, b, st);
    return run_fwd<bf16>(o, ld_o, hs_o, lse, q, ld_q, hs_q, k, ld_k, hs_k, v, ld_v, hs_v, s, b, st);
}

// attention_bwd.hip -- the gradients of attention.hip's forward pass at the
// queries, keys, values and the bias table.
//
//   p_ij = exp(s_ij - lse_i),  delta_i = do_i.o_i,  ds_ij = p_ij (do_i.v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//   dbias[h][b] = sum of ds over the pairs whose distance is in bucket b
//
// Two passes over the visible pairs, so that every sum is one workgroup's own:
// one whose waves own queries (dq, the bias, and delta for the other), one
// whose waves own keys (dk and dv).  That is 7 products a pair of tiles where
// one pass would take 5, and no atomic sums, whose order would change the
// results, nor a binary32 copy of dq.
//
// p and ds are rounded to the element type as operands of the products, half a
// step each; the sums stay in binary32.  Where the keys share a common part, as
// keys with a mean other than 0 do, the exact sum of ds over a row is 0 and takes it
// out of dq, the roundings' is not: dq is then 1.5 times as far off as from unrounded
// ds (2-norm, relative: 2.5e-3 to 1.7e-3 in bfloat16, 3.1e-4 to 2.1e-4 in binary16).
//
// Bound by issue, as the forward pass, with more products a pair of tiles.
// 8 x 1024 positions, 25 heads of 64: dq 63-67 us, dk and dv 95-99, 408-427 TFLOP/s
// of the formula's five products; 8191 packed positions, 64 heads of 128 on 8 of
// keys, window 1024: 463-502 and 689-765 us under the profiler, 1062-1110 together
// without, 509-532 TFLOP/s.  The bias adds 15 us to dk and dv, and its gradient's
// sums by distance 50 to dq at 25 heads of 64.
#include <type_traits>

#include "attention.hpp"

namespace zero {
namespace attention {
namespace {

// binary16 has few exponents below a gradient's: ds is formed in units of
// 2^-(k + 4) where 2^k is about |do_i| (its 2-norm, a power of two, so the
// products are exact), for dk the largest of the rows so far, and p of the dv
// product in units of 2^-6.  bfloat16 needs neither.
// In units of 2^-k |do_i| is below 1 and ds below |v_j| + |o_i|, which may leave
// binary16 (2^20.6 for 128 columns of its largest values), and where a few keys
// have most of a row's weight, the ds of the many others are small beside it:
// the 4 makes room below, and above it the units also go by what of |o_i| is
// past 2^10, for dk by what of the wave's largest |v_j| is.  The dq pass has the
// values only as they come: rows whose ds leave binary16 there have sums of inf
// or NaN, and are summed again in binary32 (sum_dq_row).
template <typename T>
constexpr bool kUnits = __is_same(T, _Float16);
constexpr float kWeightUnits = 64.0f, kWeightShift = 6.0f;
constexpr int kBelow = 4, kRoom = 14 - kBelow;     // 2^kRoom: what |v_j| and |o_i| may come to each

// The power of two by which a vector of this squared 2-norm is too large, at most 1.
__device__ __forceinline__ float room(float norm)
{
    const int over = ((__builtin_amdgcn_frexp_expf(norm) + 1) >> 1) - kRoom;
    return __builtin_ldexpf(1.0f, over > 0 ? -over : 0);
}

// The units by |do_i|, from its square.  A row of zeros gets a large one, so that it does not set that of the rows beside it.
__device__ __forceinline__ float unit_of(float norm)
{
    return norm > 0.0f ? __builtin_ldexpf(1.0f, kBelow - ((__builtin_amdgcn_frexp_expf(norm) + 1) >> 1)) : 0x1p60f;
}

// The lane's part of the sum of squares of its operand's column.
template <typename T, int DIM>
__device__ __forceinline__ float squares(const Operand<T, DIM>& x)
{
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum = __builtin_fmaf(float(x.v[k][j]), float(x.v[k][j]), sum);
    return sum;
}

template <typename T>
struct BwdArgs {
    Heads<T> dq, dk, dv;
    Heads<const T> dout, o, q, k, v;
    const float* lse;
    f32x2* stats;                                  // heads x tokens: lse in units of log2 (binary16: less the weights' units), delta
    float* units;                                  // heads x slots x waves: the smallest units of 32 rows (binary16)
    float* partials;                               // heads x slots x buckets
    float* near;                                   // parts of dk and dv (see dkv_items)
    float* far;
    Shape s;
    Buckets b;
    uint32_t slots, splits, far_slots, near_slots, long_from, apart;             // see Deal
    Order queries, keys;                           // of the two passes
};

template <int BIAS>
struct BinsLds {
    float bins[kWaves][BIAS == kLine ? ZERO_MAX_BUCKETS : 1];      // kTable: of the last bucket
};

__device__ __forceinline__ float lane_value(float v, uint32_t from)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(int(from * 4), __builtin_bit_cast(int, v)));
}

// The sums by distance of a wave (kTable), up to where the last bucket begins.
// They are formed from kSkewRows rows (keys) of a product at a time, written so
// that the elements of one distance are neighbours: element (row, c) at
// (c - row + kSkewRows - 1) * kSkewPitch + row, what no element goes to stays 0.
// Then a lane takes a distance.  Atomic additions in LDS, a distance a lane,
// took longer than the products (bias_bwd at 8 x 1024, 25 heads: 313 us against
// 196 for lane permutes of each register; so 111 for the pass, 64 without a bias).
template <int DIM>
constexpr int kSkewRows = DIM == 64 ? 32 : 8;      // 36 KB a workgroup, or 7.5: LDS for two workgroups a CU
template <int DIM>
constexpr int kSkewPitch = kSkewRows<DIM> + 4;
template <int DIM>
constexpr int kSkewSize = (31 + kSkewRows<DIM>) * kSkewPitch<DIM>;

// Where the first wave's begin behind the table: 16-byte aligned.
__host__ __device__ inline uint32_t sums_at(const Buckets& b) { return (table_size(b) + 3) / 4 * 4; }

// ds[r] of lane (c, h): the pair at distance base + c - row_of(r, h).  Returns
// the lane's part of the sum over the distances from `last` on.
template <int DIM>
__device__ __forceinline__ float add_distances(float* skew, float* sums, int last, int base, f32x16 ds, float back)
{
    float beyond = 0.0f;
    constexpr int kR = kSkewRows<DIM>, kP = kSkewPitch<DIM>, kLast = kR - 5;
    const int lane = threadIdx.x & 63, c = lane % 32, h = lane / 32;
    float* to = skew + (c + kR - 1) * kP - (kLast + 4 * h) * (kP - 1);
#pragma unroll
    for (int pass = 0; pass < 32 / kR; ++pass) {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int r = 0; r < kR / 2; ++r)
            to[(kLast - row_of(r, 0)) * (kP - 1)] = ds[kR / 2 * pass + r] * back;
        // the wave's LDS operations are done in order: its writes are there
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (lane < 31 + kR) {
            f32x4 v = *reinterpret_cast<const f32x4*>(skew + lane * kP);
#pragma unroll
            for (int i = 1; i < kR / 4; ++i)
                v += *reinterpret_cast<const f32x4*>(skew + lane * kP + 4 * i);
            const float sum = (v[0] + v[1]) + (v[2] + v[3]);
            const int d = base - kR * pass + lane - (kR - 1);      // below 0 there is nothing
            if (d >= last)
                beyond += sum;
            else if (d >= 0)
                sums[d] += sum;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    return beyond;
}

// bins[bucket] += the sums of ds along the distances of a 32 x 32 product
// whose rows are keys: ds[r] of lane (c, h) is the pair at distance base + c - row_of(r, h).
__device__ __forceinline__ void add_diagonals(float* bins, const BiasLine& bias, uint32_t count, int base, const float (&ds)[16])
{
    const uint32_t lane = threadIdx.x & 63;        // takes the distance base + lane - 31
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c = int(lane) - 31 + row_of(r, half);
            const float v = lane_value(ds[r], (c & 31) + 32 * half);
            sum += c >= 0 && c < 32 ? v : 0.0f;
        }
    const int d = base + int(lane) - 31;
    const uint32_t bucket = bucket_of(bias.starts, count, d > 0 ? d : 0);
    // equal buckets are neighbours: their sum ends up in the last lane of each
#pragma unroll
    for (uint32_t step = 1; step < 64; step <<= 1) {
        const uint32_t from = lane >= step ? lane - step : lane;
        const float v = lane_value(sum, from);
        const uint32_t b = __builtin_amdgcn_ds_bpermute(int(from * 4), int(bucket));
        sum += lane >= step && b == bucket ? v : 0.0f;
    }
    const uint32_t after = __builtin_amdgcn_ds_bpermute(int((lane + 1) % 64 * 4), int(bucket));
    if (lane == 63 || after != bucket)
        bins[bucket] += sum;
}
__device__ __forceinline__ void add_diagonals_of(const BiasLine& bias, float* bins, uint32_t count, int base, const float (&ds)[16])
{
    add_diagonals(bins, bias, count, base, ds);
}
__device__ __forceinline__ void add_diagonals_of(int, float*, uint32_t, int, const float (&)[16]) {}

// dq of one row by a wave, all in binary32 but the store: 64 keys a time, a lane
// a key for their ds, then a lane a column.  Slow, as the forward pass's rows
// beside an inf (attention.hip).  lse is in units of log2.
template <typename T, int DIM, int BIAS>
__device__ __forceinline__ void sum_dq_row(const BwdArgs<T>& a, const Piece& at, uint32_t head, uint32_t i, float lse, float delta)
{
    typedef typename Vec8<T>::type VU __attribute__((aligned(sizeof(T))));
    const Shape& s = a.s;
    const uint32_t lane = threadIdx.x & 63;
    const T* q = a.q.p + (uint64_t(at.start) + i) * a.q.ld + uint64_t(head) * a.q.hs;
    const T* dout = a.dout.p + (uint64_t(at.start) + i) * a.dout.ld + uint64_t(head) * a.dout.hs;
    const T* kp = a.k.p + uint64_t(at.start) * a.k.ld + uint64_t(head / s.group) * a.k.hs;
    const T* vp = a.v.p + uint64_t(at.start) * a.v.ld + uint64_t(head / s.group) * a.v.hs;
    float acc[DIM / 64] = {};
    const uint32_t near = i >= s.window ? (i - s.window + 1) & ~63u : 0;         // where the window's keys start
    for (uint32_t j0 = 0; j0 <= i; j0 = j0 + 64 >= s.sinks && j0 + 64 < near ? near : j0 + 64) {
        const uint32_t j = j0 + lane;
        const bool in = j <= i && (i - j < s.window || j < s.sinks);
        float ds = 0.0f;
        if (in) {
            float x = 0.0f, dp = 0.0f;
            for (uint32_t d = 0; d < s.dim; d += 8) {
                const VU qx = *reinterpret_cast<const VU*>(q + d), kx = *reinterpret_cast<const VU*>(kp + j * a.k.ld + d);
                const VU ox = *reinterpret_cast<const VU*>(dout + d), vx = *reinterpret_cast<const VU*>(vp + j * a.v.ld + d);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x = __builtin_fmaf(float(qx[e]), float(kx[e]), x);
                    dp = __builtin_fmaf(float(ox[e]), float(vx[e]), dp);
                }
            }
            float shift = -lse;
            if (BIAS != kNoBias)
                shift += bias_value<T>(a.b, head, bucket_of(a.b.starts, a.b.count, i - j)) * kLog2e;
            ds = __builtin_amdgcn_exp2f(__builtin_fmaf(x, s.scale2, shift)) * (dp - delta);
        }
        for (uint64_t left = __ballot(in); left; left &= left - 1) {
            const uint32_t k = __builtin_ctzll(left);
            const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ds), k));
#pragma unroll
            for (int n = 0; n < DIM / 64; ++n)
                if (lane + 64 * n < s.dim)
                    acc[n] = __builtin_fmaf(w, float(kp[(j0 + k) * a.k.ld + lane + 64 * n]), acc[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < DIM / 64; ++n)
        if (lane + 64 * n < s.dim)
            a.dq.p[(uint64_t(at.start) + i) * a.dq.ld + uint64_t(head) * a.dq.hs + lane + 64 * n] = T(acc[n] * s.scale);
}

// Without a bias 64 columns leave registers for three waves a SIMD: 63-66 us at 8 x 1024 positions, 25 heads, where two take 79.
template <typename T, int DIM, int BIAS, bool DIRECT>
__global__ __launch_bounds__(kBlock, DIM == 64 && BIAS == kNoBias ? 3 : 2) void attention_dq_kernel(BwdArgs<T> a)
{
    typedef Tile<DIM> L;
    __shared__ alignas(16) T keys[2][L::kElems];
    __shared__ alignas(16) T values[2][L::kElems];
    __shared__ typename std::conditional<BIAS == kLine, BiasLine, int>::type bias;
    __shared__ typename std::conditional<BIAS != kNoBias, BinsLds<BIAS>, int>::type sums;
    extern __shared__ __attribute__((aligned(16))) float table[];               // BIAS == kTable: the table; with a gradient the waves' skewed rows and sums by distance

    const Shape& s = a.s;
    uint32_t head, slot;
    Piece at;
    if (!a.queries.template find<true>(s, blockIdx.x, &head, &slot))
        return;
    if (!find_piece(s, slot, kOwn, &at)) {
        if (BIAS != kNoBias && a.partials && threadIdx.x < a.b.count)
            a.partials[(uint64_t(head) * a.slots + slot) * a.b.count + threadIdx.x] = 0.0f;
        return;
    }
    const uint32_t lane = threadIdx.x & 63, c = lane % 32, h = lane / 32;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t first = at.first + 32 * wave, mine = first + c;
    const uint32_t row = mine < at.len ? mine : at.len - 1;
    const bool live = mine < at.len;
    const T* kp = a.k.p + uint64_t(at.start) * a.k.ld + uint64_t(head / s.group) * a.k.hs;
    const T* vp = a.v.p + uint64_t(at.start) * a.v.ld + uint64_t(head / s.group) * a.v.hs;

    const KeyTiles tiles(s, at.first, kOwn, at.len);
    Places<DIM> places;
    Carrier<T, DIM, DIRECT> nk, nv;
    uint32_t t = tiles.begin();
    clear<T, DIM, DIRECT>(keys[0], 2 * L::kElems, s.dim);
    clear<T, DIM, DIRECT>(values[0], 2 * L::kElems, s.dim);
    cleared<DIRECT, DIM>(s.dim);
    nk.fetch(keys[0], kp, a.k.ld, t * kTile, at.len, s.dim);
    nv.fetch(values[0], vp, a.v.ld, t * kTile, at.len, s.dim);
    Operand<T, DIM> q, dout;
    load_operand<T, DIM>(q, a.q.p + uint64_t(at.start) * a.q.ld + uint64_t(head) * a.q.hs, a.q.ld, row, s.dim);
    load_operand<T, DIM>(dout, a.dout.p + uint64_t(at.start) * a.dout.ld + uint64_t(head) * a.dout.hs, a.dout.ld, row, s.dim);
    float delta = 0.0f, unit = 1.0f;
    {
        Operand<T, DIM> o;
        load_operand<T, DIM>(o, a.o.p + uint64_t(at.start) * a.o.ld + uint64_t(head) * a.o.hs, a.o.ld, row, s.dim);
#pragma unroll
        for (int k = 0; k < DIM / 16; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                delta = __builtin_fmaf(float(dout.v[k][j]), float(o.v[k][j]), delta);
        delta = halves_sum(delta);
        if (kUnits<T>)
            unit = unit_of(halves_sum(squares<T, DIM>(dout))) * room(halves_sum(squares<T, DIM>(o)));
    }
    const uint64_t stat = uint64_t(head) * s.tokens + at.start + row;
    // Lanes past the sequence's end have its last row, but distances that none of its pairs has, and so any bias: their weights
    // are 0 (a factor of 0 behind them would not do: exp of a bias far above the row's own scores is inf).
    const float lse = live ? a.lse[stat] * kLog2e : INFINITY;
    if (kUnits<T>) {
        float least = unit;
#pragma unroll
        for (int step = 16; step; step >>= 1)
            least = fminf(least, __shfl_xor(least, step));
        if (lane == 0)
            a.units[(uint64_t(head) * a.slots + slot) * kWaves + wave] = least;
    }
    if (live && h == 0)
        a.stats[stat] = f32x2{lse - (kUnits<T> ? kWeightShift : 0.0f), delta};
    delta *= unit;

    float beyond = 0.0f;                           // kTable: the bias of the last bucket
    const uint32_t last_start = BIAS == kTable ? a.b.starts[a.b.count - 1] : 0;
    float* const skews = table + (BIAS == kTable ? sums_at(a.b) : 0);           // where a.partials, from here on
    float* const skew = skews + wave * kSkewSize<DIM>, * const by_distance = skews + kWaves * kSkewSize<DIM> + wave * last_start;
    if constexpr (BIAS == kTable) {
        draw_table<T>(table, a.b, head);
        beyond = bias_value<T>(a.b, head, a.b.count - 1) * kLog2e;
        if (a.partials) {
            for (uint32_t x = lane; x < last_start; x += 64)
                by_distance[x] = 0.0f;
            for (uint32_t x = lane; x < kSkewSize<DIM>; x += 64)
                skew[x] = 0.0f;
        }
    }
    if constexpr (BIAS == kLine) {
        load_line_values<T>(bias, a.b, head);
        for (uint32_t i = threadIdx.x; i < kWaves * ZERO_MAX_BUCKETS; i += kBlock)
            sums.bins[i / ZERO_MAX_BUCKETS][i % ZERO_MAX_BUCKETS] = 0.0f;
        __syncthreads();
    }
    auto draw_line = [&](uint32_t tile, int buf) {
        if constexpr (BIAS == kLine)
            bias.draw(buf, a.b.count, int(at.first + kOwn - 1) - int(tile * kTile), -1);
    };
    float far_sum = 0.0f;                          // ds of tiles whose distances are all in the last bucket
    const float back = 1.0f / unit;                // a power of two: exact

    f32x16 acc[DIM / 32] = {};
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
            const bool apart = BIAS == kLine || (BIAS == kTable && nearest(first, j0, kTile) < last_start);
            const float row_shift = apart ? lse : lse - beyond;
            const int line_at = int(mine) - int(j0) - (kTile - 1) + kTableBefore - 4 * int(h);
#pragma unroll DIM == 64 ? 2 : 1
            for (int sub = 0; sub < 2; ++sub) {
                // half a tile beyond the window's edge: 2% of dq, dk and dv of 2 x 4096 positions, 64 heads of 128; none of heads of 64
                if (DIM == 128 && see == kSome && seen(s, first, 32, j0 + 32 * sub, 32) == kNone)
                    continue;
                if (DIM == 128)
                    places.anew();
                const f32x16 x = rows_times<T, DIM>(keys[buf], places, sub, q);
                const f32x16 dp = rows_times<T, DIM>(values[buf], places, sub, dout);
                f32x16 ds;
                if (apart) {
                    const float* b = BIAS == kLine ? &bias_line(bias, buf)[kOwn - 1 - 32 * wave - c + 4 * h + 32 * sub]
                                                   : table + line_at - 32 * sub;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        ds[r] = __builtin_fmaf(x[r], s.scale2, b[BIAS == kLine ? row_of(r, 0) : kTile - 1 - row_of(r, 0)] - row_shift);
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        ds[r] = __builtin_fmaf(x[r], s.scale2, -row_shift);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    ds[r] = __builtin_amdgcn_exp2f(ds[r]) * __builtin_fmaf(dp[r], unit, -delta);
                if (see == kSome) {
                    const Mask mask = Mask::keys(s, mine, j0 + 4 * h);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        ds[r] = mask.seen_or_0(ds[r], sub, r);
                }
                if constexpr (BIAS != kNoBias)
                    if (a.partials) {
                        if (BIAS == kLine) {
                            float w[16];
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                w[r] = ds[r] * back;
                            add_diagonals_of(bias, sums.bins[wave], a.b.count, int(first) - int(j0) - 32 * sub, w);
                        } else if (apart) {
                            far_sum += add_distances<DIM>(skew, by_distance, int(last_start), int(first) - int(j0) - 32 * sub, ds, back);
                        } else {
                            float v = 0.0f;
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                v += ds[r];
                            far_sum = __builtin_fmaf(v, back, far_sum);
                        }
                    }
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    columns_times<T, DIM>(acc, keys[buf], places, 2 * sub + half, rounded<T>(ds, half));
            }
        }
        if (!more)
            break;
        t = next;
        buf ^= 1;
        nk.put(keys[buf]);
        nv.put(values[buf]);
        draw_line(t, buf);
    }
    uint32_t again = 0;                            // rows whose ds were too large for binary16 (not those with an inf or NaN of their own)
    if (kUnits<T>) {
        float probe = 0.0f;
#pragma unroll
        for (int n = 0; n < DIM / 32; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                probe = __builtin_fmaf(acc[n][r], 0.0f, probe);
        const uint64_t marked = __ballot(live && probe != probe && fabsf(lse) < INFINITY && fabsf(delta) < INFINITY);
        again = uint32_t(marked) | uint32_t(marked >> 32);
    }
    store_columns<T, DIM>(a.dq.p + uint64_t(at.start) * a.dq.ld + uint64_t(head) * a.dq.hs, a.dq.ld, mine, live && !(again >> c & 1), s.dim,
                          acc, s.scale / unit);
    if (kUnits<T>) {
        delta /= unit;
        for (; again; again &= again - 1) {
            const uint32_t i = __builtin_ctz(again);
            sum_dq_row<T, DIM, BIAS>(a, at, head, first + i, __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, lse), i)),
                                     __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, delta), i)));
        }
    }
    if constexpr (BIAS == kLine)
        if (a.partials) {
            __syncthreads();
            if (threadIdx.x < a.b.count) {
                float v = 0.0f;
                for (int w = 0; w < kWaves; ++w)
                    v += sums.bins[w][threadIdx.x];
                a.partials[(uint64_t(head) * a.slots + slot) * a.b.count + threadIdx.x] = v;
            }
        }
    if constexpr (BIAS == kTable)
        if (a.partials) {
            far_sum = layer::lanes_sum<64>(far_sum);
            if (lane == 0)
                sums.bins[wave][0] = far_sum;
            __syncthreads();
            // the waves' sums of each distance, then each bucket's distances: a wave a bucket
            float* all = skews + kWaves * kSkewSize<DIM>;
            for (uint32_t x = threadIdx.x; x < last_start; x += kBlock) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
                    v += all[w * last_start + x];
                all[x] = v;
            }
            __syncthreads();
            for (uint32_t b = wave; b < a.b.count; b += kWaves) {
                float v = 0.0f;
                if (b + 1 < a.b.count) {
                    for (uint32_t x = a.b.starts[b] + lane; x < a.b.starts[b + 1]; x += 64)
                        v += all[x];
                    v = layer::lanes_sum<64>(v);
                } else
                    v = (sums.bins[0][0] + sums.bins[1][0]) + (sums.bins[2][0] + sums.bins[3][0]);
                if (lane == 0)
                    a.partials[(uint64_t(head) * a.slots + slot) * a.b.count + b] = v;
            }
        }
}

// ---- dk and dv ----------------------------------------------------------------------
// A workgroup goes over the tiles of queries that see its keys, for each query
// head that shares the key head: a list of (head, tile) steps.  Two things
// would leave a few workgroups with most of the work:
//   - few keys in all: the list is then cut into `splits` parts, whose binary32
//     sums go to the workspace and are added up by dkv_sum_kernel;
//   - a window with first tokens that stay visible: the piece of keys that holds
//     them is seen by every query of the sequence.  Where there are queries
//     behind the window, in sequences of at least long_from tokens, its list
//     ends with the window, and the queries behind are taken kFar at a time by
//     workgroups of their own, whose sums are added likewise.
constexpr uint32_t kFar = 1024;

// Rows of the tiles of queries.  A wave has its keys, and 64 columns take 32
// registers of each of dk and dv, 128 columns 64: then the values are read from
// LDS instead (two workgroups a CU have 80 KB each, so tiles are half as long).
template <int DIM>
constexpr int kRows = DIM == 64 ? kTile : 32;

template <int DIM>
struct RowStats {
    float lse[kRows<DIM>], delta[kRows<DIM>];
};

// Whether the queries behind the window are taken apart: where the first tokens are in one piece.
__host__ __device__ inline bool far_apart(const Shape& s) { return s.sinks && s.sinks <= kOwn && s.window != 0xffffffffu; }

// The queries below this are in the list of the piece of keys at `first`.
__device__ __forceinline__ uint32_t near_end(const Shape& s, uint32_t first, uint32_t len)
{
    const bool bounded = s.window != 0xffffffffu && (first >= s.sinks || far_apart(s));
    return bounded && len - first > kOwn - 1 && len - first - (kOwn - 1) > s.window ? first + (kOwn - 1) + s.window : len;
}

template <typename T, int DIM, int BIAS, bool DIRECT>
__global__ __launch_bounds__(kBlock, 2) void attention_dkv_kernel(BwdArgs<T> a)
{
    constexpr int kQ = kRows<DIM>;
    constexpr bool kValuesInLds = DIM == 128;
    typedef Tile<DIM, kQ> L;
    __shared__ alignas(16) T queries[2][L::kElems];
    __shared__ alignas(16) T douts[2][L::kElems];
    __shared__ alignas(16) T values[kValuesInLds ? Tile<DIM, kOwn>::kElems : 8];
    __shared__ alignas(16) RowStats<DIM> stats[2];
    __shared__ typename std::conditional<BIAS == kLine, BiasLine, int>::type bias;
    extern __shared__ __attribute__((aligned(16))) float table[];               // BIAS == kTable: of table_size() distances

    const Shape& s = a.s;
    const uint32_t kv_heads = s.heads / s.group;
    // the far items first, then the pieces' lists (of one part), or their parts
    const uint32_t far_items = a.far_slots * kv_heads, block = blockIdx.x - far_items;
    const bool is_far = blockIdx.x < far_items;
    Piece at;
    uint32_t kv, slot, part = 0, begin, end, first_key;
    float* out = nullptr;                          // binary32 sums: dk of the piece's rows, then dv; NULL: dk and dv themselves
    if (is_far) {
        kv = blockIdx.x / a.far_slots;
        if (!find_piece(s, blockIdx.x - kv * a.far_slots, kFar, &at, a.apart) || at.len < a.long_from)
            return;
        first_key = 0;
        begin = (near_end(s, 0, at.len) + kQ - 1) / kQ;
        const uint32_t stop = at.first + kFar < at.len ? at.first + kFar : at.len;
        begin = begin > at.first / kQ ? begin : at.first / kQ;
        end = (stop + kQ - 1) / kQ;
        if (begin >= end)
            return;
        out = a.far + uint64_t(blockIdx.x) * (2 * kOwn * DIM);
    } else {
        if (a.splits > 1) {
            part = block % a.splits;
            kv = block / a.splits / a.slots;
            slot = block / a.splits - kv * a.slots;
        } else if (!a.keys.template find<false>(s, block, &kv, &slot)) {
            return;
        }
        if (!find_piece(s, slot, kOwn, &at))
            return;
        first_key = at.first;
        begin = at.first / kQ;
        end = (near_end(s, at.first, at.len) + kQ - 1) / kQ;
        if (a.splits > 1)
            out = a.near + uint64_t(block) * (2 * kOwn * DIM);
        else if (a.far_slots && at.first == 0 && at.len >= a.long_from)
            out = a.near + (uint64_t(kv) * a.near_slots + (a.apart ? at.start / a.apart : at.seq)) * (2 * kOwn * DIM);
    }
    const uint32_t lane = threadIdx.x & 63, c = lane % 32, h = lane / 32;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t first = first_key + 32 * wave, mine = first + c;
    const uint32_t row = mine < at.len ? mine : at.len - 1;
    Places<DIM> places;
    Operand<T, DIM> k, v;
    load_operand<T, DIM>(k, a.k.p + uint64_t(at.start) * a.k.ld + uint64_t(kv) * a.k.hs, a.k.ld, row, s.dim);
    const T* vp = a.v.p + uint64_t(at.start) * a.v.ld + uint64_t(kv) * a.v.hs;
    clear<T, DIM, DIRECT>(queries[0], 2 * L::kElems, s.dim);
    clear<T, DIM, DIRECT>(douts[0], 2 * L::kElems, s.dim);
    if (kValuesInLds)
        clear<T, DIM, DIRECT>(values, Tile<DIM, kOwn>::kElems, s.dim);
    cleared<DIRECT, DIM>(s.dim);
    if (kValuesInLds) {
        Carrier<T, DIM, DIRECT, kOwn> nv;
        nv.fetch(values, vp, a.v.ld, first_key, at.len, s.dim);
        nv.put(values);
    } else {
        load_operand<T, DIM>(v, vp, a.v.ld, row, s.dim);
    }

    const uint32_t tiles = end - begin, steps = tiles * s.group;
    uint32_t step = is_far ? 0 : uint32_t(uint64_t(steps) * part / a.splits);
    const uint32_t step_end = is_far ? steps : uint32_t(uint64_t(steps) * (part + 1) / a.splits);
    uint32_t head = step / tiles, t = begin + step - head * tiles;
    head += kv * s.group;

    Carrier<T, DIM, DIRECT, kQ> nq, ndo;
    f32x2 nstat = {};
    float nunit = 0.0f, tile_unit = 0.0f;
    // the sequence's first slot among the dq kernel's, which wrote the units
    const uint32_t unit_slots = s.offsets ? at.start / kOwn + at.seq : at.seq * ((s.length + kOwn - 1) / kOwn);
    auto ask = [&](int buf, uint32_t hd, uint32_t tile) {
        if (threadIdx.x < kQ) {
            const uint32_t i = tile * kQ + threadIdx.x;
            nstat = a.stats[uint64_t(hd) * s.tokens + at.start + (i < at.len ? i : at.len - 1)];
        }
        if (kUnits<T>) {
            const float* u = a.units + (uint64_t(hd) * a.slots + unit_slots) * kWaves + kQ / 32 * tile;
            nunit = kQ == 64 ? fminf(u[0], u[1]) : u[0];
        }
        nq.fetch(queries[buf], a.q.p + uint64_t(at.start) * a.q.ld + uint64_t(hd) * a.q.hs, a.q.ld, tile * kQ, at.len, s.dim);
        ndo.fetch(douts[buf], a.dout.p + uint64_t(at.start) * a.dout.ld + uint64_t(hd) * a.dout.hs, a.dout.ld, tile * kQ, at.len, s.dim);
    };
    float beyond = 0.0f;                           // kTable: the bias of the last bucket
    auto load_bias = [&](uint32_t hd) {
        if constexpr (BIAS == kLine)
            load_line_values<T>(bias, a.b, hd);
        if constexpr (BIAS == kTable) {
            draw_table<T>(table, a.b, hd);
            beyond = bias_value<T>(a.b, hd, a.b.count - 1) * kLog2e;
        }
    };
    // whether every pair of the piece's keys and a tile's queries is in the last bucket
    auto all_beyond = [&](uint32_t tile) { return BIAS == kTable && nearest(tile * kQ, first_key, kOwn) >= a.b.starts[a.b.count - 1]; };
    auto place = [&](int buf, uint32_t tile) {
        nq.put(queries[buf]);
        ndo.put(douts[buf]);
        if (threadIdx.x < kQ) {
            stats[buf].lse[threadIdx.x] = all_beyond(tile) ? nstat[0] - beyond : nstat[0];
            stats[buf].delta[threadIdx.x] = nstat[1];
        }
        tile_unit = nunit;
        if constexpr (BIAS == kLine)
            bias.draw(buf, a.b.count, int(tile * kQ) - int(first_key + kOwn - 1), 1);
    };
    if constexpr (BIAS != kNoBias) {
        load_bias(head);
        __syncthreads();
    }
    f32x16 dk[DIM / 32] = {}, dv[DIM / 32] = {};
    float unit = 0x1p60f;                          // of dk's sums, but for v_room
    int buf = 0;
    if (step < step_end) {
        ask(0, head, t);
        place(0, t);
    }
    float v_room = 1.0f;                           // the wave's
    if (kUnits<T>) {
        if (kValuesInLds)
            load_operand<T, DIM>(v, vp, a.v.ld, row, s.dim);
        float norm = halves_sum(squares<T, DIM>(v));
#pragma unroll
        for (int step = 16; step; step >>= 1)
            norm = fmaxf(norm, __shfl_xor(norm, step));
        v_room = room(norm);
    }
    while (step < step_end) {
        uint32_t next = t + 1, next_head = head;
        if (next >= end) {
            next = begin;
            ++next_head;
        }
        const bool more = ++step < step_end;
        tiles_there<DIRECT>();
        if (more)
            ask(buf ^ 1, next_head, next);
        const uint32_t i0 = t * kQ;
        const Seen see = seen(s, i0, kQ, first, 32);
        if (see != kNone) {
            const bool whole = see == kAll && i0 + kQ <= at.len;
            if (kUnits<T> && tile_unit < unit) {   // the same for every lane
                const float by = tile_unit / unit;
                unit = tile_unit;
#pragma unroll
                for (int n = 0; n < DIM / 32; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        dk[n][r] *= by;
            }
            const float ds_unit = unit * (v_room / kWeightUnits);
            const bool apart = BIAS == kLine || (BIAS == kTable && !all_beyond(t));
            const float* line = BIAS == kLine ? bias_line(bias, buf) + kOwn - 1 - 32 * wave - c + 4 * h
                                              : table + (int(i0) - int(mine) + kTableBefore + 4 * int(h));
#pragma unroll
            for (int sub = 0; sub < kQ / 32; ++sub) {
                if (DIM == 128)
                    places.anew();
                const f32x16 x = rows_times<T, DIM>(queries[buf], places, sub, k);
                const f32x16 dp = kValuesInLds ? rows_times_rows<T, DIM>(douts[buf], values + 32 * DIM * wave, places)
                                               : rows_times<T, DIM>(douts[buf], places, sub, v);
                if (DIM == 128 && BIAS == kTable)
                    __builtin_amdgcn_sched_barrier(0);             // no loads ahead: the registers are full
                f32x16 p, ds;
                if (apart) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        p[r] = line[32 * sub + row_of(r, 0)];
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        p[r] = 0.0f;
                }
#pragma unroll
                for (int quad = 0; quad < 4; ++quad) {
                    const uint32_t i = 32 * sub + 8 * quad + 4 * h;
                    const f32x4 lse = *reinterpret_cast<const f32x4*>(&stats[buf].lse[i]);
                    const f32x4 delta = *reinterpret_cast<const f32x4*>(&stats[buf].delta[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 4 * quad + e;
                        p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r], s.scale2, BIAS == kNoBias ? -lse[e] : p[r] - lse[e]));
                        ds[r] = dp[r] - delta[e];
                        if (kUnits<T>)
                            ds[r] *= ds_unit;
                        ds[r] *= p[r];
                    }
                }
                if (!whole) {
                    const Mask mask = Mask::queries(s, mine, i0 + 4 * h, at.len);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        p[r] = mask.seen_or_0(p[r], sub, r);
                        ds[r] = mask.seen_or_0(ds[r], sub, r);
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    columns_times<T, DIM>(dv, douts[buf], places, 2 * sub + half, rounded<T>(p, half));
                    columns_times<T, DIM>(dk, queries[buf], places, 2 * sub + half, rounded<T>(ds, half));
                }
            }
        }
        if (!more)
            break;
        if constexpr (BIAS != kNoBias)
            if (next_head != head) {
                __syncthreads();                   // the bias before is read no more
                load_bias(next_head);
                __syncthreads();
            }
        head = next_head;
        t = next;
        buf ^= 1;
        place(buf, t);
    }
    const bool live = mine < at.len;
    const float k_unit = kUnits<T> ? s.scale / (unit * v_room) : s.scale, v_unit = kUnits<T> ? 1.0f / kWeightUnits : 1.0f;
    if (!out) {
        store_columns<T, DIM>(a.dk.p + uint64_t(at.start) * a.dk.ld + uint64_t(kv) * a.dk.hs, a.dk.ld, mine, live, s.dim, dk, k_unit);
        store_columns<T, DIM>(a.dv.p + uint64_t(at.start) * a.dv.ld + uint64_t(kv) * a.dv.hs, a.dv.ld, mine, live, s.dim, dv, v_unit);
        return;
    }
    float* mine_out = out + (32 * wave + c) * DIM + 4 * h;
#pragma unroll
    for (int n = 0; n < DIM / 32; ++n)
#pragma unroll
        for (int quad = 0; quad < 4; ++quad) {
            f32x4 x, y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = dk[n][4 * quad + e] * k_unit;
                y[e] = dv[n][4 * quad + e] * v_unit;
            }
            *reinterpret_cast<f32x4*>(mine_out + 32 * n + 8 * quad) = x;
            *reinterpret_cast<f32x4*>(mine_out + kOwn * DIM + 32 * n + 8 * quad) = y;
        }
}

// dk and dv of a piece of keys from its parts, in their order.  16 rows a workgroup.
constexpr int kSumRows = 16;

template <typename T, int DIM>
__global__ __launch_bounds__(kSumRows* DIM / 8) void dkv_sum_kernel(BwdArgs<T> a)
{
    typedef typename Vec8<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    const Shape& s = a.s;
    const uint32_t kv = blockIdx.y;
    const uint32_t slot = blockIdx.x / (kOwn / kSumRows);          // of the pieces, or of the long sequences' first ones
    Piece at;
    if (a.splits > 1 ? !find_piece(s, slot, kOwn, &at) : !find_piece(s, slot, 1u << 31, &at, a.apart) || at.len < a.long_from)
        return;
    const uint32_t local = blockIdx.x % (kOwn / kSumRows) * kSumRows + threadIdx.x / (DIM / 8), col = threadIdx.x % (DIM / 8) * 8;
    const uint32_t row = at.first + local;
    if (row >= at.len || col >= s.dim)
        return;
    constexpr uint64_t kPart = 2 * kOwn * DIM;
    const float* near = a.near + (a.splits > 1 ? (uint64_t(kv) * a.slots + slot) * a.splits : uint64_t(kv) * a.near_slots + slot) * kPart;
    uint32_t far_begin = 0, far_end = 0;
    if (a.far_slots && at.first == 0 && at.len >= a.long_from) {
        const uint32_t slots = s.offsets ? at.start / kFar + (a.apart ? at.start / a.apart : at.seq) : at.seq * ((s.length + kFar - 1) / kFar);
        constexpr uint32_t kQ = kRows<DIM>;
        const uint32_t behind = (near_end(s, 0, at.len) + kQ - 1) / kQ * kQ;
        if (behind < at.len) {
            far_begin = slots + behind / kFar;
            far_end = slots + (at.len + kFar - 1) / kFar;
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const uint64_t place = (which * kOwn + local) * DIM + col;
        layer::f32x8 sum = {};
        for (uint32_t p = 0; p < a.splits; ++p)
            sum += *reinterpret_cast<const layer::f32x8*>(near + p * kPart + place);
        for (uint32_t p = far_begin; p < far_end; ++p)
            sum += *reinterpret_cast<const layer::f32x8*>(a.far + (uint64_t(kv) * a.far_slots + p) * kPart + place);
        const Heads<T>& to = which ? a.dv : a.dk;
        *reinterpret_cast<VU*>(to.p + (uint64_t(at.start) + row) * to.ld + uint64_t(kv) * to.hs + col) = __builtin_convertvector(sum, V);
    }
}

// A head's bias gradient: its partials added up in their order.
template <typename T>
__global__ __launch_bounds__(kBlock) void fold_bias_kernel(void* dst, bool f32, bool accumulate, const float* partials, uint32_t slots,
                                                           uint32_t count)
{
    __shared__ float part[kWaves][ZERO_MAX_BUCKETS];
    const uint32_t i = threadIdx.x % 64, w = threadIdx.x / 64;
    float v = 0.0f;
    if (i < count)
        for (uint32_t slot = w; slot < slots; slot += kWaves)
            v += partials[(uint64_t(blockIdx.x) * slots + slot) * count + i];
    part[w][i] = v;
    __syncthreads();
    if (w || i >= count)
        return;
    v = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
    const uint64_t to = uint64_t(blockIdx.x) * count + i;
    if (f32) {
        float* d = static_cast<float*>(dst) + to;
        *d = accumulate ? *d + v : v;
    } else {
        T* d = static_cast<T*>(dst) + to;
        *d = T(accumulate ? float(*d) + v : v);
    }
}

// ---- host side --------------------------------------------------------------------------
// How the work on dk and dv is dealt out (see attention_dkv_kernel).
struct Deal {
    uint64_t slots, splits;
    uint64_t far_slots, near_slots, long_from;     // of the queries behind the window, and of the pieces of keys that they see, in
                                                   // sequences of at least long_from tokens
    uint64_t apart;                                // of find_piece() for these: long_from where that gives fewer slots, else 0
    uint64_t parts;                                // of dk and dv, of 128 keys, that go to the workspace
};

constexpr uint64_t kItems = 512;

// Parts with the fewest steps that one may have, where a sequence has `length` positions.
uint64_t most_splits(const Shape& s, uint64_t length)
{
    const uint64_t keys = s.window < length / 2 ? s.window : length / 2, splits = s.group * (keys / kTile + 2) / 4;
    return splits ? splits : 1;
}

Deal deal(const Shape& s, bool ragged)
{
    Deal d{slots_of(s.tokens, s.sequences, ragged, kOwn), 1, 0, 0, 0, 0, 0};
    const uint64_t behind = uint64_t(s.window) + kOwn;             // near_end() is before the end from here on
    if (far_apart(s) && (ragged ? s.tokens : s.length) >= behind) {
        d.long_from = behind;
        const uint64_t most = s.tokens / behind;                   // such sequences
        d.apart = ragged && most < s.sequences ? behind : 0;
        d.far_slots = d.apart ? s.tokens / kFar + most : slots_of(s.tokens, s.sequences, ragged, kFar);
        d.near_slots = d.apart ? most : s.sequences;
    }
    // enough parts for two workgroups a CU, but none with fewer than four steps where a sequence has the mean length:
    // a part costs a workgroup's start and 128 rows of binary32 sums written and read.  4099 positions in 5, 3 key heads
    // of 80, window 700: 99 pieces in 111 slots, five parts each: 74 us and 12 for the sums
    const uint64_t kv = s.heads / s.group, items = d.slots * kv;
    const uint64_t wanted = (kItems + items - 1) / items, most = most_splits(s, s.tokens / s.sequences + 1);
    d.splits = wanted < most ? wanted : most;
    d.parts = d.splits > 1 ? items * d.splits : kv * d.near_slots;
    return d;
}

// The workspace, each part from a multiple of 256 bytes: the rows' statistics,
// the units, the bias' partial sums, the parts of dk and dv.
struct Space {
    uint64_t stats, units, partials, near, far, bytes;
};

Space space(const Shape& s, const Deal& d, uint32_t buckets, int dim)
{
    const uint64_t kv = s.heads / s.group, part = 2 * kOwn * uint64_t(dim) * 4;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t from = at;
        at = (at + bytes + 255) / 256 * 256;
        return from;
    };
    Space p;
    p.stats = take(uint64_t(s.heads) * s.tokens * 8);
    p.units = take(uint64_t(s.heads) * d.slots * kWaves * 4);
    p.partials = take(uint64_t(s.heads) * d.slots * buckets * 4);
    p.near = take(d.parts * part);
    p.far = take(kv * d.far_slots * part);
    p.bytes = at;
    return p;
}

// Of a call with or without offsets, and of every smaller one: no more tokens in
// no more sequences.  The slots of sequences of equal length are no more than
// those with offsets (which hold for any lengths); fewer items may be cut into
// more parts, of which i items have at most i + kItems - 1, and i times what the
// longest sequence allows.
uint64_t workspace_need(const Shape& s, uint32_t buckets)
{
    Deal d = deal(s, true);
    const uint64_t kv = s.heads / s.group, items = d.slots * kv, cut = items < kItems ? items : kItems - 1;
    const uint64_t most = most_splits(s, s.tokens + 1);
    if (most > 1) {
        const uint64_t parts = cut * most < cut + kItems - 1 ? cut * most : cut + kItems - 1;
        d.parts = parts > d.parts ? parts : d.parts;
    }
    if (kv * d.near_slots > d.parts)
        d.parts = kv * d.near_slots;
    return space(s, d, buckets, s.dim <= 64 ? 64 : 128).bytes;
}

// Workgroups of attention_dkv_kernel but for the far ones.
template <typename T>
uint64_t near_blocks(const BwdArgs<T>& a)
{
    return a.splits > 1 ? uint64_t(a.slots) * a.splits * (a.s.heads / a.s.group) : a.keys.blocks(a.s);
}

// Whether the launches after the first fit theirs, too (dkv_sum_kernel has kBlock threads or half as many).
template <typename T>
bool launches_fit(const BwdArgs<T>& a)
{
    return near_blocks(a) + uint64_t(a.far_slots) * (a.s.heads / a.s.group) < kMostBlocks &&
           uint64_t(a.splits > 1 ? a.slots : a.near_slots) * (kOwn / kSumRows) < kMostBlocks;
}

template <typename T, int DIM, int BIAS, bool DIRECT>
int launch(const BwdArgs<T>& a, hipStream_t stream)
{
    const uint64_t near = near_blocks(a);
    const uint32_t kv = a.s.heads / a.s.group, table = BIAS == kTable ? table_size(a.b) * 4 : 0;
    const uint32_t sums = BIAS == kTable && a.partials ? (sums_at(a.b) + kWaves * (a.b.starts[a.b.count - 1] + kSkewSize<DIM>)) * 4 : 0;
    hipLaunchKernelGGL((attention_dq_kernel<T, DIM, BIAS, DIRECT>), dim3(uint32_t(a.queries.blocks(a.s))), dim3(kBlock),
                       sums ? sums : table, stream, a);
    int rc = launch_status();
    if (rc)
        return rc;
    hipLaunchKernelGGL((attention_dkv_kernel<T, DIM, BIAS, DIRECT>), dim3(uint32_t(near + uint64_t(a.far_slots) * kv)), dim3(kBlock),
                       table, stream, a);
    rc = launch_status();
    if (rc || (a.splits == 1 && !a.far_slots))
        return rc;
    hipLaunchKernelGGL((dkv_sum_kernel<T, DIM>), dim3((a.splits > 1 ? a.slots : a.near_slots) * (kOwn / kSumRows), kv),
                       dim3(kSumRows * DIM / 8), 0, stream, a);
    return launch_status();
}

template <typename T>
int run(Heads<void> dq, Heads<void> dk, Heads<void> dv, Heads<const void> dout, Heads<const void> o, Heads<const void> q, Heads<const void> k,
        Heads<const void> v, const float* lse, const Shape& s, const Buckets& b, void* dbias, int grad_dtype, bool accumulate,
        char* workspace, hipStream_t stream)
{
    auto out = [](Heads<void> x) { return Heads<T>{static_cast<T*>(x.p), x.ld, x.hs}; };
    auto in = [](Heads<const void> x) { return Heads<const T>{static_cast<const T*>(x.p), x.ld, x.hs}; };
    const Deal d = deal(s, s.offsets != nullptr);
    const Space p = space(s, d, b.count, s.dim <= 64 ? 64 : 128);
    auto part = [&](uint64_t at) { return reinterpret_cast<float*>(workspace + at); };
    const BwdArgs<T> a{out(dq), out(dk), out(dv), in(dout), in(o), in(q), in(k), in(v), lse, reinterpret_cast<f32x2*>(workspace + p.stats),
                       part(p.units), dbias ? part(p.partials) : nullptr, part(p.near), part(p.far), s, b, uint32_t(d.slots), uint32_t(d.splits),
                       uint32_t(d.far_slots), uint32_t(d.near_slots), uint32_t(d.long_from), uint32_t(d.apart), Order(s, s.heads, d.slots),
                       Order(s, s.heads / s.group, d.slots)};
    if (!launches_fit(a))
        return ZERO_ERANGE;
    auto go = [&](auto dim, auto way) {
        constexpr int kDim = decltype(dim)::value;
        constexpr bool kDirect = decltype(way)::value;
        if (!b.count)
            return launch<T, kDim, kNoBias, kDirect>(a, stream);
        // with sums for more than some 512 distances (384 at 128 columns) LDS has one workgroup a CU.  25 heads of 64, the
        // last bucket from 1000 on: table and line take 328 and 264 us at 8 x 1024 positions, where most tiles need the
        // table, 919 and 1108 at 2 x 4096.  64 heads of 128 on 8, window 1024: 1863 and 1958
        const uint32_t last = b.starts[b.count - 1];
        const bool line = kDim == 64 && dbias && last > 512 && s.tokens / s.sequences < 2 * last;
        return table_fits(b) && !line ? launch<T, kDim, kTable, kDirect>(a, stream) : launch<T, kDim, kLine, kDirect>(a, stream);
    };
    const std::integral_constant<int, 64> d64;
    const std::integral_constant<int, 128> d128;
    int rc;
    if (direct(q.p, q.ld, q.hs) && direct(k.p, k.ld, k.hs) && direct(v.p, v.ld, v.hs) && direct(dout.p, dout.ld, dout.hs))
        rc = s.dim <= 64 ? go(d64, std::true_type{}) : go(d128, std::true_type{});
    else
        rc = s.dim <= 64 ? go(d64, std::false_type{}) : go(d128, std::false_type{});
    if (rc || !dbias)
        return rc;
    hipLaunchKernelGGL(fold_bias_kernel<T>, dim3(s.heads), dim3(kBlock), 0, stream, dbias, grad_dtype == ZERO_F32, accumulate, a.partials,
                       a.slots, b.count);
    return launch_status();
}

}  // namespace
}  // namespace attention
}  // namespace zero

using namespace zero;
using namespace zero::attention;

extern "C" size_t zero_attention_workspace_bytes(const zero_attention_t* params, uint64_t tokens, uint64_t sequences)
{
    Shape s;
    Buckets b;
    if (!tokens || !sequences || !params)
        return 0;
    // the larger of a call with offsets and one without, where they are not refused; the pointers are only tested for NULL
    const void* bias = params->buckets ? params : nullptr;
    const int32_t* offsets = reinterpret_cast<const int32_t*>(params);
    if (make_shape(params, tokens, offsets, sequences, ZERO_F16, bias, ZERO_F16, &s, &b) &&
        make_shape(params, tokens, nullptr, sequences, ZERO_F16, bias, ZERO_F16, &s, &b))
        return 0;
    return size_t(workspace_need(s, b.count));
}

extern "C" int zero_attention_bwd(void* dq, uint64_t ld_dq, uint64_t hs_dq, void* dk, uint64_t ld_dk, uint64_t hs_dk, void* dv,
                                  uint64_t ld_dv, uint64_t hs_dv, void* dbias, int grad_dtype, int accumulate, const void* dout,
                                  uint64_t ld_dout, uint64_t hs_dout, const void* o, uint64_t ld_o, uint64_t hs_o, const float* lse,
                                  const void* q, uint64_t ld_q, uint64_t hs_q, const void* k, uint64_t ld_k, uint64_t hs_k, const void* v,
                                  uint64_t ld_v, uint64_t hs_v, const void* bias, int vec_dtype, const zero_attention_t* params,
                                  uint64_t tokens, const int32_t* dev_offsets, uint64_t sequences, int dtype, void* workspace,
                                  size_t workspace_bytes, void* stream)
{
    Shape s;
    Buckets b;
    int rc = make_shape(params, tokens, dev_offsets, sequences, dtype, bias, vec_dtype, &s, &b);
    if (rc)
        return rc;
    const uint32_t hq = params->heads, hk = params->kv_heads, dim = params->dim;
    rc = check_heads(dq, ld_dq, hs_dq, tokens, hq, dim, dtype);
    if (!rc) rc = check_heads(dk, ld_dk, hs_dk, tokens, hk, dim, dtype);
    if (!rc) rc = check_heads(dv, ld_dv, hs_dv, tokens, hk, dim, dtype);
    if (!rc) rc = check_heads(dout, ld_dout, hs_dout, tokens, hq, dim, dtype);
    if (!rc) rc = check_heads(o, ld_o, hs_o, tokens, hq, dim, dtype);
    if (!rc) rc = check_heads(q, ld_q, hs_q, tokens, hq, dim, dtype);
    if (!rc) rc = check_heads(k, ld_k, hs_k, tokens, hk, dim, dtype);
    if (!rc) rc = check_heads(v, ld_v, hs_v, tokens, hk, dim, dtype);
    if (!rc) rc = layer::check_vector(dbias, grad_dtype, dtype);
    if (rc)
        return rc;
    if (dbias && !bias)
        return ZERO_EINVAL;
    if (tokens && (!lse || dq == dk || dq == dv || dk == dv))
        return ZERO_EINVAL;
    if (!is_aligned(lse, 4))
        return ZERO_EALIGN;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (!tokens) {
        if (!dbias || accumulate)
            return ZERO_OK;
        if (dtype == ZERO_F16)
            hipLaunchKernelGGL(fold_bias_kernel<_Float16>, dim3(hq), dim3(kBlock), 0, st, dbias, grad_dtype == ZERO_F32, false, nullptr, 0,
                               params->buckets);
        else
            hipLaunchKernelGGL(fold_bias_kernel<bf16>, dim3(hq), dim3(kBlock), 0, st, dbias, grad_dtype == ZERO_F32, false, nullptr, 0,
                               params->buckets);
        return launch_status();
    }
    if (!workspace)
        return ZERO_EINVAL;
    if (!is_aligned(workspace, 16))
        return ZERO_EALIGN;
    if (workspace_bytes < workspace_need(s, b.count))
        return ZERO_ERANGE;
    const auto go = dtype == ZERO_F16 ? run<_Float16> : run<bf16>;
    return go({dq, ld_dq, hs_dq}, {dk, ld_dk, hs_dk}, {dv, ld_dv, hs_dv}, {dout, ld_dout, hs_dout}, {o, ld_o, hs_o}, {q, ld_q, hs_q},
              {k, ld_k, hs_k}, {v, ld_v, hs_v}, lse, s, b, dbias, grad_dtype, accumulate != 0, static_cast<char*>(workspace), st);
}

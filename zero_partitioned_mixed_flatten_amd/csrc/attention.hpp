// attention.hpp -- what the attention kernels share (attention.hip,
// attention_bwd.hip): the arguments, the place of a workgroup's tile in the
// packed sequences, which keys a tile of queries sees, tiles in LDS and the
// matrix products on them.
//
// All products are 32 x 32 x 16 matrix instructions on binary16 or bfloat16
// operands with binary32 sums.  Lane l of a wave (c = l % 32, h = l / 32)
// holds of such a product
//   A (32 x 16):  row c, columns 8h .. 8h + 7
//   B (16 x 32):  column c, rows 8h .. 8h + 7
//   C (32 x 32):  column c, rows row_of(r, h), r = 0 .. 15
// so each lane owns one column of C: scores are formed with the operand that
// stays (a wave's 32 queries in the forward pass and for dq, its 32 keys for
// dk and dv) as the columns, a softmax row is then one lane pair's own, and
// registers 8n .. 8n + 7 of C, rounded, are a B operand whose 16 rows are the
// tile's rows 16n + {4h, .. 4h + 3, 8 + 4h, .. 8 + 4h + 3}: the order in which
// the other operand's rows are read is the same, and no lane exchange is needed.
#pragma once

#include "layer.hpp"

namespace zero {
namespace attention {

typedef layer::bf16 bf16;
typedef layer::bf16x8 bf16x8;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4;                          // waves of a workgroup
constexpr int kBlock = 64 * kWaves;
constexpr int kOwn = 32 * kWaves;                  // rows a workgroup owns: 32 a wave, the columns of its scores
constexpr int kTile = 64;                          // rows of the tiles it goes over
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

template <typename T>
struct Vec8;
template <>
struct Vec8<_Float16> {
    typedef f16x8 type;
    static __device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Vec8<bf16> {
    typedef bf16x8 type;
    static __device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// The row of C that register r of a lane of half h holds.
__device__ __forceinline__ constexpr int row_of(int r, int h) { return 8 * (r / 4) + 4 * h + r % 4; }

// tokens x heads x dim elements: (i, h, d) at i * ld + h * hs + d.
template <typename T>
struct Heads {
    T* p;
    uint64_t ld, hs;
};

// What the kernels need of the call's geometry.
struct Shape {
    const int32_t* offsets;                        // sequences + 1 token indices, or NULL: equal lengths
    uint32_t tokens, sequences, length;            // length: of each sequence where offsets is NULL
    uint32_t heads, group, dim;                    // group: query heads that share a key head
    uint32_t window, sinks;                        // window: 0xffffffff where there is no limit
    float scale, scale2;                           // scale2: scale * log2(e)
};

struct Buckets {
    const void* table;                             // heads x count, NULL: no bias
    uint32_t count;
    bool f32;                                      // type of the table: binary32, or the activations'
    uint32_t starts[ZERO_MAX_BUCKETS];
};

// ---- the tile of a workgroup --------------------------------------------------------
// The rows of all sequences are dealt out in pieces of `own` that do not cross a
// sequence.  Where the lengths are in device memory, sequence s gets the slots
// from offsets[s] / own + s on: at least as many as it has pieces, so a slot
// finds its sequence from the offsets alone, and some slots stay empty.
// Offsets out of order or out of range are clamped: they give wrong tiles, but
// none outside the tensors.
// Where only sequences of at least `apart` tokens matter, they get the slots
// from offsets[s] / own + offsets[s] / apart on: another such sequence begins at
// least `apart` tokens later, so these are as many as it has pieces, too, and
// tokens / own + tokens / apart in all.  A shorter one has slots that the long
// one after it may share: the last sequence is found that has a slot.
struct Piece {
    uint32_t seq, start, len;                      // the sequence: its index, first token, tokens
    uint32_t first;                                // the piece's first row in the sequence
    uint32_t slots;                                // the sequence's first slot
};

__host__ __device__ inline uint64_t slots_of(uint32_t tokens, uint32_t sequences, bool ragged, uint32_t own)
{
    if (ragged)
        return uint64_t(tokens) / own + sequences;
    return uint64_t(sequences) * ((tokens / sequences + own - 1) / own);
}

__device__ __forceinline__ bool find_piece(const Shape& s, uint32_t slot, uint32_t own, Piece* out, uint32_t apart = 0)
{
    if (!s.offsets) {
        const uint32_t per = (s.length + own - 1) / own;
        out->seq = slot / per;
        out->start = out->seq * s.length;
        out->len = s.length;
        out->slots = out->seq * per;
        out->first = (slot - out->slots) * own;
        return true;
    }
    const uint32_t lane = threadIdx.x & 63;
    auto offset = [&](uint32_t i) {
        const int32_t o = s.offsets[i];
        return o < 0 ? 0u : uint32_t(o) < s.tokens ? uint32_t(o) : s.tokens;
    };
    uint32_t seq = 0;                              // the number of sequences whose slots begin at or before this one
    for (uint32_t base = 0; base < s.sequences; base += 64) {
        const uint32_t i = base + lane;
        const uint32_t at = offset(i < s.sequences ? i : 0);
        const bool before = i < s.sequences && at / own + (apart ? at / apart : i) <= slot;
        const uint32_t n = __popcll(__ballot(before));
        seq += n;
        if (n < 64)
            break;
    }
    if (!seq)
        return false;
    --seq;
    const uint32_t start = __builtin_amdgcn_readfirstlane(offset(seq)), end = __builtin_amdgcn_readfirstlane(offset(seq + 1));
    out->seq = seq;
    out->start = start;
    out->len = end > start ? end - start : 0;
    out->slots = start / own + (apart ? start / apart : seq);
    out->first = (slot - out->slots) * own;
    return slot >= out->slots && uint64_t(slot - out->slots) * own < out->len;
}

// A dimension of a launch holds fewer than 2^32 threads: with kBlock a workgroup fewer workgroups than this.
constexpr uint64_t kMostBlocks = (uint64_t(1) << 32) / kBlock;

// Which head and piece a block takes.  Blocks go to the eight dies in turn;
// neighbours that share a head's keys belong on one, whose L2 then holds them.
// Sequences of equal length: each die has its own (sequence, head) pairs and
// takes all of their heaviest pieces first, so that light ones are left for
// the end; with fewer than 64 pairs that are no multiple of 8 some dies would
// have less to do.  Else a die takes a contiguous part of the list of heads and
// slots.
struct Order {
    uint32_t heads, slots, pairs;                  // pairs: of a die, or 0

    __host__ Order(const Shape& s, uint32_t h, uint64_t n) : heads(h), slots(uint32_t(n)), pairs(0)
    {
        const uint64_t all = uint64_t(h) * s.sequences;
        if (!s.offsets && (all >= 64 || all % 8 == 0) && (all + 7) / 8 * 8 * (n / s.sequences) < kMostBlocks)
            pairs = uint32_t((all + 7) / 8);
    }
    __host__ uint64_t blocks(const Shape& s) const
    {
        return pairs ? uint64_t(pairs) * 8 * (slots / s.sequences) : (uint64_t(heads) * slots + 7) / 8 * 8;
    }
    // LATE: the last rows of a sequence have the most work, else the first
    template <bool LATE>
    __device__ __forceinline__ bool find(const Shape& s, uint32_t block, uint32_t* head, uint32_t* slot) const
    {
        const uint32_t die = block % 8, i = block / 8;
        if (pairs) {
            const uint32_t per = (s.length + kOwn - 1) / kOwn, rank = i / pairs, pair = die * pairs + (i - rank * pairs), seq = pair / heads;
            *head = pair - seq * heads;
            *slot = seq * per + (LATE ? per - 1 - rank : rank);
            return rank < per && seq < s.sequences;
        }
        const uint32_t work = die * ((heads * slots + 7) / 8) + i;
        *head = work / slots;
        const uint32_t rest = work - *head * slots;
        *slot = LATE ? slots - 1 - rest : rest;
        return i < (heads * slots + 7) / 8 && work < heads * slots;
    }
};

// ---- visibility ------------------------------------------------------------------------
// Position j is visible to i where j <= i and (i - j < window or j < sinks).
enum Seen { kNone, kSome, kAll };

// Of the keys [j, j + nk) by the queries [i, i + nq).
__device__ __forceinline__ Seen seen(const Shape& s, uint32_t i, uint32_t nq, uint32_t j, uint32_t nk)
{
    if (j > i + nq - 1)
        return kNone;
    // the nearest pair is i - (j + nk - 1), at least 0; the farthest i + nq - 1 - j
    if (i > j + nk - 1 && i - (j + nk - 1) >= s.window && j >= s.sinks)
        return kNone;
    if (j + nk - 1 <= i && (i + nq - 1 - j < s.window || j + nk <= s.sinks))
        return kAll;
    return kSome;
}

// The same for single pairs: a bit for each of a lane's rows of a tile, two
// words of 32 rows.  A select by one is two vector instructions and takes no
// scalar registers, of which 32 comparisons would need 64.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

struct Mask {
    uint32_t word[2];

    // of the keys j0 + 4 h + row_of(r, 0), those that the query i sees
    static __device__ __forceinline__ Mask keys(const Shape& s, uint32_t i, uint32_t j0)
    {
        const int end = int(i) - int(j0) + 1;                      // keys below this are not behind the query
        const int far = s.window > i ? -int(j0) : int(i - s.window) + 1 - int(j0);         // keys from this on are in the window
        const int first = s.sinks > j0 ? int(s.sinks - j0 < uint32_t(kTile) ? s.sinks - j0 : uint32_t(kTile)) : 0;
        Mask m;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
            m.word[sub] = below(end - 32 * sub) & (~below(far - 32 * sub) | below(first - 32 * sub));
        return m;
    }
    // of the queries i0 + 4 h + row_of(r, 0), those that see the key j
    static __device__ __forceinline__ Mask queries(const Shape& s, uint32_t j, uint32_t i0, uint32_t len)
    {
        const uint32_t last = j < s.sinks || s.window > len || j + s.window > len ? len : j + s.window;
        Mask m;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
            m.word[sub] = below(int(last) - int(i0) - 32 * sub) & ~below(int(j) - int(i0) - 32 * sub);
        return m;
    }
    // all ones where register r of the product `sub` is seen
    __device__ __forceinline__ uint32_t bits(int sub, int r) const { return uint32_t(__builtin_amdgcn_sbfe(int(sub ? word[1] : word[0]), row_of(r, 0), 1)); }
    __device__ __forceinline__ float seen_or(float x, uint32_t other, int sub, int r) const
    {
        const uint32_t m = bits(sub, r);
        return __builtin_bit_cast(float, (m & __builtin_bit_cast(uint32_t, x)) | (~m & other));
    }
    __device__ __forceinline__ float seen_or_0(float x, int sub, int r) const
    {
        return __builtin_bit_cast(float, bits(sub, r) & __builtin_bit_cast(uint32_t, x));
    }
};

// The key tiles that some query of [i, i + nq) sees, in order: those of the
// first tokens, then those of the window.
struct KeyTiles {
    uint32_t sink_end, win_begin, end;             // in tiles

    __device__ __forceinline__ KeyTiles(const Shape& s, uint32_t i, uint32_t nq, uint32_t len)
    {
        const uint32_t last = i + nq < len ? i + nq : len;         // keys below this
        end = (last + kTile - 1) / kTile;
        win_begin = i >= s.window ? (i - s.window + 1) / kTile : 0;
        const uint32_t sinks = s.sinks < last ? s.sinks : last;
        sink_end = s.window == 0xffffffffu ? 0 : (sinks + kTile - 1) / kTile;
        if (sink_end >= win_begin)
            sink_end = win_begin = 0;
    }
    __device__ __forceinline__ uint32_t begin() const { return sink_end ? 0 : win_begin; }
    __device__ __forceinline__ uint32_t next(uint32_t t) const { return t + 1 == sink_end ? win_begin : t + 1; }
};

// ---- tiles in LDS ---------------------------------------------------------------------
// ROWS rows of DIM elements in 16-byte pieces.  The pieces of a row are
// permuted by the row, so that both ways to read a tile spread over the 64
// banks: 16 bytes of one column place in consecutive rows (operand A as rows),
// and 8-byte parts of 4 rows that the transposing read turns (operand A as
// columns).
template <int DIM, int ROWS = kTile>
struct Tile {
    static constexpr int kPieces = DIM / 8;        // a row
    static constexpr int kPerThread = ROWS * kPieces / kBlock;
    static constexpr int kElems = ROWS * DIM;

    static __device__ __forceinline__ uint32_t twist(uint32_t row)
    {
        return DIM == 128 ? (row & 3) << 2 | ((row >> 2) & 3) : ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ uint32_t place(uint32_t row, uint32_t piece)   // in elements
    {
        return row * DIM + ((piece ^ twist(row)) * 8);
    }
};

// A tile's way there.  DIRECT: straight into LDS, 16 bytes a lane to consecutive
// addresses of a wave, so a lane takes the piece that belongs at its address;
// it needs rows at 16-byte aligned places.  Else through registers.  Rows past
// the sequence's end repeat its last one (what they give is masked); columns
// past `dim` are 0 (DIRECT: left as clear() made them).
template <typename T, int DIM, bool DIRECT, int ROWS = kTile>
class Carrier;

template <typename T, int DIM, int ROWS>
class Carrier<T, DIM, false, ROWS> {
    typedef typename Vec8<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    typedef Tile<DIM, ROWS> L;
    V v[L::kPerThread];

public:
    __device__ __forceinline__ void fetch(T*, const T* head, uint64_t ld, uint32_t row0, uint32_t len, uint32_t dim)
    {
#pragma unroll
        for (int i = 0; i < L::kPerThread; ++i) {
            const uint32_t id = threadIdx.x + i * kBlock, row = id / L::kPieces, col = id % L::kPieces * 8;
            const uint32_t at = row0 + row < len ? row0 + row : len - 1;
            const bool in = col < dim;
            const V x = *reinterpret_cast<const VU*>(head + at * ld + (in ? col : 0));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = in ? x[j] : T(0.0f);
        }
    }
    __device__ __forceinline__ void put(T* tile)
    {
#pragma unroll
        for (int i = 0; i < L::kPerThread; ++i) {
            const uint32_t id = threadIdx.x + i * kBlock;
            *reinterpret_cast<V*>(tile + L::place(id / L::kPieces, id % L::kPieces)) = v[i];
        }
    }
};

template <typename T, int DIM, int ROWS>
class Carrier<T, DIM, true, ROWS> {
    typedef Tile<DIM, ROWS> L;
    static constexpr uint32_t kRows = kBlock / L::kPieces;         // of one round; the permutation of a row repeats after it
    static_assert(kRows % 16 == 0, "rows of a round");

public:
    // The compiler waits for such a load before any read of LDS that it cannot tell apart from it, the other buffer's too: in
    // assembly it does not, and tiles_there() waits.
    __device__ __forceinline__ void fetch(T* tile, const T* head, uint64_t ld, uint32_t row0, uint32_t len, uint32_t dim)
    {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        const uint32_t row = threadIdx.x / L::kPieces, col = (threadIdx.x % L::kPieces ^ L::twist(row)) * 8;
        const uint32_t to = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) T*)tile)) + wave * 1024;
        const T* from = head + row0 * ld;
        if (col >= dim)
            return;
        const uint32_t step = uint32_t(ld) * sizeof(T), last = len - 1 - row0;      // ld is below 2^24
        if (last >= uint32_t(ROWS) - 1) {
            const uint32_t at = row * step + col * uint32_t(sizeof(T));
#pragma unroll
            for (int i = 0; i < L::kPerThread; ++i)
                load(to + i * 16 * kBlock, at, from + i * kRows * ld);
        } else {
#pragma unroll
            for (int i = 0; i < L::kPerThread; ++i) {
                const uint32_t r = row + i * kRows;
                load(to + i * 16 * kBlock, (r < last ? r : last) * step + col * uint32_t(sizeof(T)), from);
            }
        }
    }
    __device__ __forceinline__ void put(T*) {}

private:
    static __device__ __forceinline__ void load(uint32_t to, uint32_t at, const T* base)
    {
        const uint64_t b = reinterpret_cast<uintptr_t>(base);      // the same in every lane
        const uint64_t from = uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(b >> 32)))) << 32 |
                              uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(b)));
        to = __builtin_amdgcn_readfirstlane(to);
        // m0 is a register that the compiler reserves, of which it warns; the clobber keeps it from taking over a value of its own
        // that it set there before
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(to), "v"(at), "s"(from) : "memory", "m0");
#pragma clang diagnostic pop
    }
};

// Before the first fetch into `elems` elements of LDS: 0 in the columns that no fetch writes.
template <typename T, int DIM, bool DIRECT>
__device__ __forceinline__ void clear(T* tiles, uint32_t elems, uint32_t dim)
{
    if (!DIRECT || dim == DIM)
        return;
    typename Vec8<T>::type zero = {};
    for (uint32_t i = threadIdx.x * 8; i < elems; i += kBlock * 8)
        *reinterpret_cast<typename Vec8<T>::type*>(tiles + i) = zero;
}
template <bool DIRECT, int DIM>
__device__ __forceinline__ void cleared(uint32_t dim)
{
    if (DIRECT && dim != DIM)
        __syncthreads();
}

// What was fetched is in LDS for every wave, and what the waves read before may be written over.
template <bool DIRECT>
__device__ __forceinline__ void tiles_there()
{
    if (DIRECT)
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    __syncthreads();
}

// The operand that stays: a wave's 32 rows as columns of B.
template <typename T, int DIM>
struct Operand {
    typename Vec8<T>::type v[DIM / 16];
};

template <typename T, int DIM>
__device__ __forceinline__ void load_operand(Operand<T, DIM>& o, const T* head, uint64_t ld, uint32_t row, uint32_t dim)
{
    typedef typename Vec8<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    const uint32_t h = (threadIdx.x & 63) / 32;
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k) {
        const uint32_t col = 16 * k + 8 * h;
        const bool in = col < dim;
        const V v = *reinterpret_cast<const VU*>(head + row * ld + (in ? col : 0));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o.v[k][j] = in ? v[j] : T(0.0f);
    }
}

// Where a lane reads a tile, in elements from its start: the reads of one way
// differ from the first by an exclusive or (the piece) and by a constant (the
// row), since the rows' permutation repeats every 16 rows.
template <int DIM>
struct Places {
    uint32_t row, col, col8;

    __device__ __forceinline__ Places()
    {
        const uint32_t lane = threadIdx.x & 63, h = lane / 32, i = lane % 16, g = lane / 16 % 2, r = 4 * h + i / 4;
        row = Tile<DIM>::place(lane % 32, h);
        col = Tile<DIM>::place(r, 2 * g + i % 4 / 2) + i % 2 * 4;
        col8 = Tile<DIM>::place(r + 8, 2 * g + i % 4 / 2) + i % 2 * 4;
    }
    // In a loop that is short of registers: the places are formed anew from these three instead of kept.
    __device__ __forceinline__ void anew() { asm volatile("" : "+v"(row), "+v"(col), "+v"(col8)); }
};

// C = (rows 32 sub .. of the tile) x operand.
template <typename T, int DIM>
__device__ __forceinline__ f32x16 rows_times(const T* tile, const Places<DIM>& at, int sub, const Operand<T, DIM>& b)
{
    f32x16 c = {};
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k)
        c = Vec8<T>::mfma(*reinterpret_cast<const typename Vec8<T>::type*>(tile + 32 * DIM * sub + (at.row ^ (16 * k))), b.v[k], c);
    return c;
}

// The same with 32 rows of another tile as the operand.
template <typename T, int DIM>
__device__ __forceinline__ f32x16 rows_times_rows(const T* tile, const T* other, const Places<DIM>& at)
{
    typedef typename Vec8<T>::type V;
    f32x16 c = {};
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k)
        c = Vec8<T>::mfma(*reinterpret_cast<const V*>(tile + (at.row ^ (16 * k))), *reinterpret_cast<const V*>(other + (at.row ^ (16 * k))), c);
    return c;
}

template <typename T>
__device__ __forceinline__ typename Vec8<T>::type column_pair(const T* a, const T* b)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* P;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(a)), y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(b));
    return __builtin_bit_cast(typename Vec8<T>::type, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Operands A for 16 rows of the tile (from 16 step on) as columns: their
// elements 32 n .. 32 n + 31 each, the rows in the order that a score's
// registers give them as an operand B.
template <typename T, int DIM>
struct Columns {
    typename Vec8<T>::type v[DIM / 32];
};

template <typename T, int DIM>
__device__ __forceinline__ void read_columns(Columns<T, DIM>& a, const T* tile, const Places<DIM>& at, int step)
{
    const T* rows = tile + 16 * DIM * step;
#pragma unroll
    for (int n = 0; n < DIM / 32; ++n)
        a.v[n] = column_pair<T>(rows + (at.col ^ (32 * n)), rows + (at.col8 ^ (32 * n)));
}

// acc[n] += (columns of those rows)^T x p
template <typename T, int DIM>
__device__ __forceinline__ void columns_times(f32x16 (&acc)[DIM / 32], const Columns<T, DIM>& a, typename Vec8<T>::type p)
{
#pragma unroll
    for (int n = 0; n < DIM / 32; ++n)
        acc[n] = Vec8<T>::mfma(a.v[n], p, acc[n]);
}

template <typename T, int DIM>
__device__ __forceinline__ void columns_times(f32x16 (&acc)[DIM / 32], const T* tile, const Places<DIM>& at, int step,
                                              typename Vec8<T>::type p)
{
    Columns<T, DIM> a;
    read_columns<T, DIM>(a, tile, at, step);
    columns_times<T, DIM>(acc, a, p);
}

// Registers 8 half .. 8 half + 7, rounded to nearest even.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::type rounded(f32x16 c, int half)
{
    layer::f32x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = c[8 * half + j];
    return __builtin_convertvector(v, typename Vec8<T>::type);
}

// x of the lane and of the one 32 lanes away, which hold the two halves of a column.
struct Pair {
    float low, high;
};
__device__ __forceinline__ Pair both_halves(float x)
{
    const uint32_t bits = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
    const uint32_t low = r[0], high = r[1];        // a bit cast of an element itself would take the first
    return Pair{__builtin_bit_cast(float, low), __builtin_bit_cast(float, high)};
}
__device__ __forceinline__ float halves_sum(float x)
{
    const Pair p = both_halves(x);
    return p.low + p.high;
}
__device__ __forceinline__ float halves_max(float x)
{
    const Pair p = both_halves(x);
    return fmaxf(p.low, p.high);
}

// Stores acc^T * factor (column c of acc is row `row` of the output) with
// 16-byte stores: the halves of a wave trade 4-element parts first.
template <typename T, int DIM>
__device__ __forceinline__ void store_columns(T* head, uint64_t ld, uint32_t row, bool live, uint32_t dim, const f32x16 (&acc)[DIM / 32],
                                              float factor)
{
    typedef typename Vec8<T>::type V;
    typedef V __attribute__((aligned(sizeof(T)))) VU;
    const uint32_t h = (threadIdx.x & 63) / 32;
#pragma unroll
    for (int n = 0; n < DIM / 32; ++n)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            layer::f32x8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = acc[n][8 * half + j] * factor;
            struct Words {
                uint32_t d[4];
            };
            const Words w = __builtin_bit_cast(Words, __builtin_convertvector(v, V));
            Words out;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const auto r = __builtin_amdgcn_permlane32_swap(w.d[j], w.d[j + 2], false, false);
                out.d[j] = r[0];
                out.d[j + 2] = r[1];
            }
            const uint32_t col = 32 * n + 16 * half + 8 * h;
            if (live && col < dim)
                *reinterpret_cast<VU*>(head + row * ld + col) = __builtin_bit_cast(V, out);
        }
}

// ---- the bias -------------------------------------------------------------------------
// bucket(d): the last b with starts[b] <= d.
__device__ __forceinline__ uint32_t bucket_of(const uint32_t* starts, uint32_t count, uint32_t d)
{
    uint32_t b = 0;
#pragma unroll
    for (uint32_t step = ZERO_MAX_BUCKETS / 2; step; step >>= 1)
        if (b + step < count && starts[b + step] <= d)
            b += step;
    return b;
}

template <typename T>
__device__ __forceinline__ float bias_value(const Buckets& b, uint32_t head, uint32_t i)
{
    const uint64_t at = uint64_t(head) * b.count + i;
    return b.f32 ? static_cast<const float*>(b.table)[at] : float(static_cast<const T*>(b.table)[at]);
}

// How a kernel has the bias (template parameter).  kTable: a value for each
// distance in LDS, up to where every pair of a tile is in the last bucket, whose
// bias is then one number.  kLine: where the last bucket begins too far out for
// that, a line of values for each tile, searched for in the buckets.  Table and
// line, 25 heads of 64, the last bucket from 128 on: 51 and 57 us forward at 8 x
// 1024 positions, 203 and 264 backward; 190 and 231, 653 and 1110 at 2 x 4096; from
// 1000 on: 60 and 57 forward, 197 and 232.
enum { kNoBias, kTable, kLine };

// The table: the distance d at d + kTableBefore.  A tile that is not wholly in
// the last bucket reaches from 94 before distance 0 to 190 past where that begins.
constexpr int kTableBefore = 96, kTableBeyond = 192;
constexpr uint32_t kTableMost = 1024;              // LDS for two workgroups a CU beside tiles of 64 columns, one of 128

__host__ __device__ inline bool table_fits(const Buckets& b) { return b.starts[b.count - 1] <= kTableMost; }
__host__ __device__ inline uint32_t table_size(const Buckets& b) { return b.starts[b.count - 1] + kTableBefore + kTableBeyond; }

// The least distance between the rows from i on and nk keys from j on.
__device__ __forceinline__ uint32_t nearest(uint32_t i, uint32_t j, uint32_t nk) { return i > j + nk - 1 ? i - (j + nk - 1) : 0; }

template <typename T>
__device__ __forceinline__ void draw_table(float* table, const Buckets& b, uint32_t head)
{
    for (uint32_t x = threadIdx.x; x < table_size(b); x += kBlock) {
        const int d = int(x) - kTableBefore;
        table[x] = bias_value<T>(b, head, bucket_of(b.starts, b.count, d > 0 ? d : 0)) * kLog2e;
    }
}

struct BiasLine {
    float value[ZERO_MAX_BUCKETS];                 // the head's bias times log2(e)
    uint32_t starts[ZERO_MAX_BUCKETS];
    float line[2][kOwn + kTile];

    // line[x]: the distance `from` + x step
    __device__ __forceinline__ void draw(int buf, uint32_t count, int from, int step)
    {
        if (threadIdx.x < kOwn + kTile - 1) {
            const int d = from + step * int(threadIdx.x);
            line[buf][threadIdx.x] = value[bucket_of(starts, count, d > 0 ? d : 0)];
        }
    }
};
__device__ __forceinline__ const float* bias_line(const BiasLine& b, int buf) { return b.line[buf]; }
__device__ __forceinline__ const float* bias_line(int, int) { return nullptr; }

template <typename T>
__device__ __forceinline__ void load_line_values(BiasLine& line, const Buckets& b, uint32_t head)
{
    if (threadIdx.x < b.count) {
        line.value[threadIdx.x] = bias_value<T>(b, head, threadIdx.x) * kLog2e;
        line.starts[threadIdx.x] = b.starts[threadIdx.x];
    }
}

// ---- host side --------------------------------------------------------------------------
constexpr uint64_t kMaxTokens = uint64_t(1) << 30;
constexpr uint32_t kMaxHeads = 65535;
constexpr uint64_t kMaxPieces = kMostBlocks - 8;   // of all heads; Order rounds up to the dies

// Rows that go straight into LDS: at 16-byte aligned places.
inline bool direct(const void* p, uint64_t ld, uint64_t hs)
{
    return is_aligned(p, 16) && ld % 8 == 0 && hs % 8 == 0 && ld < (1u << 24);
}

inline int check_heads(const void* p, uint64_t ld, uint64_t hs, uint64_t tokens, uint32_t heads, uint32_t dim, int dtype)
{
    if (!p)
        return tokens ? ZERO_EINVAL : ZERO_OK;
    if (!is_aligned(p, layer::dtype_size(dtype)))
        return ZERO_EALIGN;
    if ((tokens > 1 && ld < dim) || (heads > 1 && hs < dim))
        return ZERO_ERANGE;
    if (ld > (uint64_t(1) << 50) || hs > (uint64_t(1) << 50) ||
        (unsigned __int128)tokens * ld + (unsigned __int128)heads * hs > (uint64_t(1) << 56))
        return ZERO_ERANGE;
    return ZERO_OK;
}

// Checks what the calls share and fills the kernels' arguments.
int make_shape(const zero_attention_t* a, uint64_t tokens, const int32_t* dev_offsets, uint64_t sequences, int dtype,
               const void* bias, int vec_dtype, Shape* s, Buckets* b);

}  // namespace attention
}  // namespace zero

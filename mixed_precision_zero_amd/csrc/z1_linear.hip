// z1_linear.hip -- the products of z1_linear and z1_linear_grad.
//
// All three are C[q][p] = sum_k P(p, k) Q(q, k) with p along C's rows' elements:
//   x W'   (forward)   P = W [out, in],        Q = x [rows, in]     both deep in memory
//   dz W   (input)     P = W, depth its rows,  Q = dz [rows, out]
//   dz' x  (weight)    P = x, depth its rows,  Q = dz, likewise
// "Deep" operands are contiguous along k, the others along their own index.
// P takes the matrix instruction's rows and Q its columns, so that a lane ends
// up with runs of p and writes C's rows in 16-byte pieces.
#include "z1_layers_internal.h"

namespace z1 {
namespace ops {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
// LDS as an address space of its own.  The kernels' loops take the ring as two
// restrict pointers, one that copies write and one that fragments are read from:
// else the compiler waits for every copy under way before a transposing read.  What
// orders the two is the kernels' own waits and barriers, each beside a fence that is
// given both pointers (one that is not is no fence for them: the compiler takes
// restrict memory that it cannot see passed on for untouched).  The pointers are passed
// on by value alone, as what a closure holds by reference loses its restrict, and the
// second one's value is hidden, as a constant argument does too.
typedef __attribute__((address_space(3))) char lds_char;
[[maybe_unused]] __device__ __forceinline__ const lds_char *hidden(const lds_char *p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm("" : "+s"(p));
#endif
    return p;
}

// The workgroup's barrier, with no access to the ring moved across it.
[[maybe_unused]] __device__ __forceinline__ void ring_barrier(lds_char *to, const lds_char *from)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : : "s"(to), "s"(from) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : "s"(to), "s"(from) : "memory");
#endif
}

// acc += A B for the 16 bytes of depth that a lane holds of either operand: one
// instruction of depth 16 in 16 bits, four of depth 2 in fp32 (there, the k of
// an instruction's two halves are 4 apart, alike in both operands).
[[maybe_unused]] __device__ __forceinline__ void mma(BF16, float16v &acc, uint4v a, uint4v b)
{
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
[[maybe_unused]] __device__ __forceinline__ void mma(F16, float16v &acc, uint4v a, uint4v b)
{
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), acc, 0, 0, 0);
}
[[maybe_unused]] __device__ __forceinline__ void mma(F32, float16v &acc, uint4v a, uint4v b)
{
    const float4v x = __builtin_bit_cast(float4v, a), y = __builtin_bit_cast(float4v, b);
#pragma unroll
    for (int s = 0; s < 4; ++s)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[s], y[s], acc, 0, 0, 0);
}

constexpr uint32_t kRange = 0x7ffffff0u, kOutside = 0x80000000u;

// One operand's share of a panel (DB bytes of depth, 64 or 128) in LDS, TILE * DB
// bytes, copied there directly, 1 KiB a wave and instruction; and the fragments of 32
// indexes x 32 bytes of depth (16 a lane) read from it.
//
// Deep operands: a row of DB bytes for each index, its 16-byte chunks permuted by the
// row's number, so that the 16 rows that share a cycle of a fragment read touch all 64
// banks once: four rows of 64 bytes span the banks, or two of 128.
//
// The others: a row for each k, the tile's indexes along it.  In 16 bits the
// fragments are read with the transposing LDS read: 16 lanes take 16 indexes x
// 4 k.  The 32 lanes that share a cycle take 64 bytes of 4 rows; row k's chunks
// are moved by 64 bytes times (k mod 4) (two positions of a 128-byte row), which
// puts them on different banks.  In fp32 a lane reads its elements one by one;
// the rows of the upper half of the lanes are moved by 128 bytes.
//
// The permutations are applied to the global address, as the LDS side of the
// copy is fixed in lane order.  Chunks behind the operand's end (its depth, or
// the contiguous extent) get an offset outside the descriptor's range and
// arrive as zeros; rows of a deep operand behind its extent repeat the last one
// and end up in rows or columns of C that nobody writes.
template <typename E, bool DEEP, int TILE, int NW, int DB>
struct Side {
    static constexpr int kSize = (int)sizeof(typename E::store);
    static constexpr int kPanel = DB / kSize;             // depth of a panel
    static constexpr int kParts = DB / 32;                // fragments along it
    static constexpr int kBytes = TILE * DB;              // of a panel's share
    static constexpr int kLoads = kBytes / 1024 / NW;     // copies per wave and panel
    static constexpr int kReads = (DEEP || kSize == 4) ? (DEEP ? 1 : 4) : 2;   // LDS reads of a fragment
    static constexpr int kRow = TILE * kSize;             // bytes of a row in LDS, if not deep
    static constexpr int kChunks = DEEP ? DB / 16 : kRow / 16;   // of a row
    static_assert(kLoads >= 1 && (DEEP || kChunks >= 8) && (DB == 64 || DB == 128), "tile");

    const char *base;        // of the next panel
    int64_t step;
    int32_t left;            // depth from there on: bytes if deep, else rows
    uint32_t at[kLoads];     // offsets of this lane's copies
    int32_t limit[kLoads];   // copied while limit < left

    // what the chunks of row r are xored with
    static __device__ __forceinline__ int turn(int r)
    {
        if (DEEP)
            return DB == 64 ? (r >> 2) & 3 : (r >> 1) & 7;
        if (kSize == 4)
            return ((r >> 2) & 1) << 3;
        return kChunks >= 16 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
    }

    __device__ __forceinline__ void start(const Operand &o, int32_t tile, int32_t panel, int wave, int lane)
    {
        const int32_t i0 = tile * TILE;
        base = static_cast<const char *>(o.base);
        if (DEEP) {
            base += (int64_t)i0 * o.ld + (int64_t)panel * DB;
            step = DB;
            left = o.depth * kSize - panel * DB;
        } else {
            base += (int64_t)panel * kPanel * o.ld + (int64_t)i0 * kSize;
            step = kPanel * o.ld;
            left = o.depth - panel * kPanel;
        }
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int c = (wave * kLoads + q) * 64 + lane;
            const int row = c / kChunks, chunk = (c % kChunks) ^ turn(row);
            if (DEEP) {
                at[q] = (uint32_t)min(row, o.extent - 1 - i0) * (uint32_t)o.ld + chunk * 16;
                limit[q] = chunk * 16;
            } else {
                at[q] = (uint32_t)row * (uint32_t)o.ld + chunk * 16;
                // behind the row's end: never copied
                limit[q] = (i0 * (int64_t)kSize + chunk * 16 < (int64_t)o.extent * kSize) ? row : INT32_MAX;
            }
        }
    }

    // Copies FROM .. TO - 1 of the wave's share of the next panel; the last one
    // goes on to the panel behind it.
    template <int FROM = 0, int TO = kLoads>
    __device__ __forceinline__ void load(lds_char *to, int wave)
    {
        const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, kRange, 0x00020000);
#pragma unroll
        for (int q = FROM; q < TO; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(to + (wave * kLoads + q) * 1024), 16,
                                                     limit[q] < left ? at[q] : kOutside, 0, 0, 0);
        if (TO == kLoads) {
            base += step;
            left -= DEEP ? DB : kPanel;
        }
    }

    // Where fragments of the 32 indexes from i0 are read, for frag().
    static __device__ __forceinline__ int place(int i0, int lane)
    {
        const int half = lane >> 5, low = lane & 31;
        if (DEEP)
            return (i0 + low) * DB + ((half ^ turn(low)) * 16);
        if (kSize == 4) {
            const int k = 4 * half, col = i0 + low;
            return k * kRow + (((col >> 2) ^ turn(k)) << 4) + (col & 3) * 4;
        }
        const int k = 8 * half + ((lane >> 2) & 3), col = i0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        return k * kRow + (((col >> 3) ^ turn(k)) << 4) + (col & 7) * 2;
    }

    // The fragment of part kk of the panel's depth.
    static __device__ __forceinline__ uint4v frag(const lds_char *lds, int place, int kk)
    {
        if (DEEP)
            return *(const __attribute__((address_space(3))) uint4v *)(lds + (place ^ (kk * 32)));
        if (kSize == 4) {
            uint4v v;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                v[s] = *(const __attribute__((address_space(3))) uint32_t *)(lds + place + (8 * kk + s) * kRow);
            return v;
        }
        union {
            short4v h[2];
            uint4v v;
        } u;
        typedef __attribute__((address_space(3))) short4v lds4;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(lds + place + (16 * kk) * kRow));
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(lds + place + (16 * kk + 4) * kRow));
        return u.v;
    }
};

template <int N>
__device__ __forceinline__ void wait_copies()
{
    // at most N copies of this wave outstanding, no LDS read outstanding
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
}

// --------------------------------------------------------------------------
// Epilogues: eight elements (row, col ..) of C, of which n are inside it.  What they
// read of the row (In) is fetched apart, so that it can be on its way early; the bias
// goes by the column alone.
// --------------------------------------------------------------------------

template <typename E>
__device__ __forceinline__ void get_row(const void *p, int64_t at, typename Eight<E>::Raw &raw)
{
    Eight<E>::fetch(static_cast<const typename E::store *>(p) + at, raw);
}
// The eight values of a fetched row, or those of the row's end.
template <typename E>
__device__ __forceinline__ void row_values(const typename Eight<E>::Raw &raw, const void *p, int64_t at, int n, float (&v)[8])
{
    if (n >= 8)
        Eight<E>::up(raw, v);
    else
        Eight<E>::load_some(static_cast<const typename E::store *>(p) + at, v, n);
}
template <typename E>
__device__ __forceinline__ void put_row(void *p, int64_t at, int n, const float (&v)[8])
{
    typename E::store *to = static_cast<typename E::store *>(p) + at;
    if (n >= 8)
        Eight<E>::store(to, v);
    else
        Eight<E>::store_some(to, v, n);
}

// A fetched row's words to a lane's own places in LDS, 64 lanes of 16 bytes apart, and
// from there.
template <typename RAW>
__device__ __forceinline__ void park_words(char *to, const RAW &raw)
{
#pragma unroll
    for (int w = 0; w < (int)(sizeof(RAW) / 16); ++w)
        *reinterpret_cast<uint4v *>(to + w * 1024) = raw[w];
}
template <typename RAW>
__device__ __forceinline__ void take_words(const char *from, RAW &raw)
{
#pragma unroll
    for (int w = 0; w < (int)(sizeof(RAW) / 16); ++w)
        raw[w] = *reinterpret_cast<const uint4v *>(from + w * 1024);
}

template <typename O>
struct PlainOut {
    static constexpr bool kDrops = false;
    struct In {
        typename Eight<O>::Raw add;
    };
    static __device__ __forceinline__ void park(const Epilogue &e, char *to, const In &in)
    {
        if (e.add)
            park_words(to, in.add);
    }
    static __device__ __forceinline__ void take(const Epilogue &e, const char *from, In &in)
    {
        if (e.add)
            take_words(from, in.add);
    }
    static __device__ __forceinline__ void bias(const Epilogue &, int32_t, int, float (&)[8]) {}
    static __device__ __forceinline__ void fetch(const Epilogue &e, int64_t row, int32_t col, In &in)
    {
        if (e.add)
            get_row<O>(e.add, row * e.ld_add + col, in.add);
    }
    static __device__ __forceinline__ void put(const Epilogue &e, const DropKey &, int64_t row, int32_t col, int n, const In &in,
                                               const float (&)[8], float (&v)[8])
    {
        if (e.add) {
            float a[8];
            row_values<O>(in.add, e.add, row * e.ld_add + col, n, a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += a[j];
        }
        put_row<O>(e.out, row * e.ld_out + col, n, v);
    }
};

template <typename E, bool ACT>
struct FullOut {
    static constexpr bool kDrops = true;
    struct In {
        typename Eight<E>::Raw mul, add;
    };
    static __device__ __forceinline__ void park(const Epilogue &e, char *to, const In &in)
    {
        if (e.mul)
            park_words(to, in.mul);
        if (e.add)
            park_words(to + sizeof(in.mul) * 64, in.add);
    }
    static __device__ __forceinline__ void take(const Epilogue &e, const char *from, In &in)
    {
        if (e.mul)
            take_words(from, in.mul);
        if (e.add)
            take_words(from + sizeof(in.mul) * 64, in.add);
    }
    static __device__ __forceinline__ void bias(const Epilogue &e, int32_t col, int n, float (&b)[8])
    {
        const typename E::store *from = static_cast<const typename E::store *>(e.bias) + col;
        if (e.bias && n >= 8)
            Eight<E>::load(from, b);
        else if (e.bias && n > 0)
            Eight<E>::load_some(from, b, n);
    }
    static __device__ __forceinline__ void fetch(const Epilogue &e, int64_t row, int32_t col, In &in)
    {
        if (e.mul)
            get_row<E>(e.mul, row * e.ld_mul + col, in.mul);
        if (e.add)
            get_row<E>(e.add, row * e.ld_add + col, in.add);
    }
    static __device__ __forceinline__ void put(const Epilogue &e, const DropKey &key, int64_t row, int32_t col, int n, const In &in,
                                               const float (&b)[8], float (&v)[8])
    {
        float a[8];
        if (e.bias)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += b[j];
        if (e.pre)
            put_row<E>(e.pre, row * e.ld_pre + col, n, v);
        if (ACT)
            act_values(e.act, v);
        if (e.mul) {
            row_values<E>(in.mul, e.mul, row * e.ld_mul + col, n, a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] *= a[j];
        }
        if (key.on)
            drop8(key, (uint32_t)col >> 3, (uint32_t)row, v);
        if (e.add) {
            row_values<E>(in.add, e.add, row * e.ld_add + col, n, a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += a[j];
        }
        put_row<E>(e.out, row * e.ld_out + col, n, v);
    }
};

// Eight elements at once, from what is fetched here.
template <typename OUT>
__device__ __forceinline__ void put_now(const Epilogue &e, const DropKey &key, int64_t row, int32_t col, int n, float (&v)[8])
{
    typename OUT::In in;
    float b[8];
    OUT::bias(e, col, n, b);
    if (n >= 8)
        OUT::fetch(e, row, col, in);
    OUT::put(e, key, row, col, n, in, b, v);
}

// The 32 x 32 block at (q0, p0) of C as the matrix instruction leaves it: column
// `low`, rows 8 g + 4 half + r.  Swapping the halves' registers of two g gives
// every lane eight consecutive p of its q.
template <typename OUT>
__device__ __forceinline__ void put_block(const Product &g, const DropKey &key, int64_t q0, int64_t p0, int lane,
                                          const float4v (&acc)[4])
{
    const int half = lane >> 5, low = lane & 31;
    const int64_t q = q0 + low;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        float v[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[2 * s][r]), __float_as_uint(acc[2 * s + 1][r]),
                                                            false, false);
            v[r] = __uint_as_float(x[0]);
            v[4 + r] = __uint_as_float(x[1]);
        }
        const int64_t p = p0 + 16 * s + 8 * half;
        if (q < g.Q && p < g.P)
            put_now<OUT>(g.e, key, q, (int32_t)p, (int)(g.P - p), v);
    }
}

// Workgroup b's place: workgroup b runs on XCD b mod 8, so XCD x takes the
// x-th eighth of the order below, and tiles that share operand panels share an
// L2.  The order walks columns of kGroup tiles of Q.
constexpr int kGroup = 8;
[[maybe_unused]] __device__ __forceinline__ void tile_of(const Product &g, uint32_t b, uint32_t n, int32_t &tp, int32_t &tq, int32_t &piece)
{
    const uint32_t x = b & 7, per = n >> 3, more = n & 7;
    uint32_t id = x * per + min(x, more) + (b >> 3);
    const uint32_t tiles = (uint32_t)g.tiles_p * (uint32_t)g.tiles_q;
    piece = (int32_t)(id / tiles);
    id %= tiles;
    const uint32_t band = (uint32_t)g.tiles_p * kGroup;
    const uint32_t first = id / band * kGroup, high = min((uint32_t)kGroup, (uint32_t)g.tiles_q - first);
    id %= band;
    tp = (int32_t)(id / high);
    tq = (int32_t)(first + id % high);
}

// The fragments of part kk of a panel.
template <typename SP, typename SQ, int TP, int TQ>
__device__ __forceinline__ void read_part(const lds_char *p, const lds_char *q, const int (&pat)[TP], const int (&qat)[TQ],
                                          int kk, uint4v (&a)[TP], uint4v (&b)[TQ])
{
#pragma unroll
    for (int j = 0; j < TQ; ++j)
        b[j] = SQ::frag(q, qat[j], kk);
#pragma unroll
    for (int i = 0; i < TP; ++i)
        a[i] = SP::frag(p, pat[i], kk);
}

template <typename E, int TP, int TQ>
__device__ __forceinline__ void multiply(float16v (&acc)[TP][TQ], const uint4v (&a)[TP], const uint4v (&b)[TQ])
{
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j)
            mma(E(), acc[i][j], a[i], b[j]);
}

// What a product's kernel sets up: its tile, its operands' sides, and the places of its
// wave's fragments; and what it does with its sums.
template <typename SP, typename SQ, int TILE, int TP, int TQ>
struct Setup {
    SP sp;
    SQ sq;
    int32_t tp, tq, piece, panels;
    int lane, wave, wp, wq;
    int pat[TP], qat[TQ];

    __device__ __forceinline__ void start(const Product &g)
    {
        constexpr int DB = SP::kParts * 32;
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wp = wave >> 1;
        wq = wave & 1;
        tile_of(g, blockIdx.x, gridDim.x, tp, tq, piece);
        const int32_t per = g.piece / DB, first = piece * per;
        sp.start(g.p, tp, first, wave, lane);
        sq.start(g.q, tq, first, wave, lane);
        panels = min(per, (g.p.depth + SP::kPanel - 1) / SP::kPanel - first);
#pragma unroll
        for (int i = 0; i < TP; ++i)
            pat[i] = SP::place((wp * TP + i) * 32, lane);
#pragma unroll
        for (int j = 0; j < TQ; ++j)
            qat[j] = SQ::place((wq * TQ + j) * 32, lane);
    }
};

template <int TP, int TQ>
__device__ __forceinline__ void clear(float16v (&acc)[TP][TQ])
{
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.f;
}

// The sums of one piece of a split product, for k_product_join: 16 bytes a lane.
template <int TILE, int TP, int TQ>
__device__ __forceinline__ void put_parts(const Product &g, int32_t tp, int32_t tq, int32_t piece, int wave, int lane,
                                          const float16v (&acc)[TP][TQ])
{
    float *to = g.parts + ((int64_t)piece * g.tiles_p * g.tiles_q + (int64_t)tq * g.tiles_p + tp) * TILE * TILE +
                wave * TP * TQ * 1024 + lane * 4;
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<float4v *>(to + (i * TQ + j) * 1024 + r * 256) =
                    float4v{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
}

// A wave's sums into C, a strip of 32 or 64 rows of C at a time through its own part of
// the LDS, so that TP * 4 lanes write TP * 32 elements of a row together.  Rows are 16
// bytes longer than their data, which spreads both accesses over the banks.
//
// READS: the epilogue reads rows of its own (add, mul).  Those of a strip are fetched a
// strip early, all at once, as nothing else hides the wait for them: 8192 x 2048 -> 8192
// with a residual 332 us with two accesses of a lane under way, 265 so, 236 without a
// residual (now 250 and 221, in a form of their own).  They are parked in LDS too, so that the loop over the rows, with its
// activations, need not be unrolled for the sake of the registers' names; strips are 32
// rows then, as 64 with what is parked do not fit.  Without, 64 are faster (236 and 249).
template <typename OUT, int TP, int TQ, bool READS>
struct Strip {
    static constexpr int kTall = READS || TQ < 2 ? 1 : 2;   // blocks of 32 rows
    static constexpr int kRowBytes = TP * 128 + 16, kLanes = TP * 4, kRows = 64 / kLanes, kTurns = kTall * 32 / kRows;
    static constexpr int kIn = (int)sizeof(typename OUT::In), kSums = kTall * 32 * kRowBytes;
    static constexpr int kBytes = kSums + (READS ? kTurns * 64 * kIn : 0);   // of a wave
};

template <typename OUT, int TILE, bool READS, int TP, int TQ>
__device__ __forceinline__ void put_strips_of(const Product &g, const Epilogue &e, int32_t tp, int32_t tq, int wp, int wq, int wave,
                                              int lane, char *lds, const float16v (&acc)[TP][TQ])
{
    typedef Strip<OUT, TP, TQ, READS> S;
    const DropKey key = OUT::kDrops ? drop_key(e.drop) : DropKey{};
    char *own = lds + wave * S::kBytes, *parked = own + S::kSums + lane * 16;
    const int half = lane >> 5, low = lane & 31, at = lane % S::kLanes, row = lane / S::kLanes;
    const int64_t p0 = (int64_t)tp * TILE + wp * TP * 32 + at * 8, q0 = (int64_t)tq * TILE + wq * TQ * 32 + row;
    const int n = (int)min((int64_t)8, g.P - p0);
    float b[8];
    OUT::bias(e, (int32_t)p0, n, b);
    typename OUT::In in[S::kTurns];
    const auto fetch = [&](int j) {
#pragma unroll
        for (int f = 0; f < S::kTurns; ++f)
            if (n >= 8 && q0 + j * 32 + f * S::kRows < g.Q)
                OUT::fetch(e, q0 + j * 32 + f * S::kRows, (int32_t)p0, in[f]);
    };
    if (READS)
        fetch(0);
#pragma unroll
    for (int j = 0; j < TQ; j += S::kTall) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int k = 0; k < S::kTall; ++k)
#pragma unroll
            for (int i = 0; i < TP; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<float4v *>(own + (k * 32 + low) * S::kRowBytes + (i * 32 + 8 * r + 4 * half) * 4) =
                        float4v{acc[i][j + k][4 * r], acc[i][j + k][4 * r + 1], acc[i][j + k][4 * r + 2],
                                acc[i][j + k][4 * r + 3]};
        if (READS) {
#pragma unroll
            for (int f = 0; f < S::kTurns; ++f)
                OUT::park(e, parked + f * 64 * S::kIn, in[f]);
            if (j + S::kTall < TQ)
                fetch(j + S::kTall);
        }
        asm volatile("" ::: "memory");   // a wave's LDS accesses take place in order
        // the next two turns' are read while two are worked on
        float4v x[2][2];
        typename OUT::In here[2];
        const auto read = [&](int f, int u) {
            const char *from = own + (row + f * S::kRows) * S::kRowBytes + at * 32;
            x[u][0] = reinterpret_cast<const float4v *>(from)[0];
            x[u][1] = reinterpret_cast<const float4v *>(from)[1];
            if (READS)
                OUT::take(e, parked + f * 64 * S::kIn, here[u]);
        };
        read(0, 0);
        read(1, 1);
#pragma unroll 1
        for (int f = 0; f < S::kTurns; f += 2)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t q = q0 + j * 32 + (f + u) * S::kRows;
                float v[8] = {x[u][0][0], x[u][0][1], x[u][0][2], x[u][0][3], x[u][1][0], x[u][1][1], x[u][1][2], x[u][1][3]};
                if (n > 0 && q < g.Q)
                    OUT::put(e, key, q, (int32_t)p0, n, here[u], b, v);
                if (f + 2 < S::kTurns)
                    read(f + 2 + u, u);
            }
    }
}

template <typename OUT, int TILE, int TP, int TQ>
__device__ __forceinline__ void put_strips(const Product &g, int32_t tp, int32_t tq, int wp, int wq, int wave, int lane,
                                           char *lds, const float16v (&acc)[TP][TQ])
{
    if (g.e.add || g.e.mul)
        return put_strips_of<OUT, TILE, true>(g, g.e, tp, tq, wp, wq, wave, lane, lds, acc);
    Epilogue e = g.e;
    e.add = e.mul = nullptr;
    put_strips_of<OUT, TILE, false>(g, e, tp, tq, wp, wq, wave, lane, lds, acc);
}

// The LDS of a kernel's four waves: its ring, then the epilogue's strips.
template <typename OUT, int TP, int TQ>
constexpr int lds_of(int ring)
{
    const int a = 4 * Strip<OUT, TP, TQ, true>::kBytes, b = 4 * Strip<OUT, TP, TQ, false>::kBytes;
    return ring > a ? (ring > b ? ring : b) : a > b ? a : b;
}

// A quarter of a panel of k_product_64 and k_product_128: multiplies a0 b0, reads the
// fragments of part kk of the panel at `at`, and makes the F-th quarter of the wave's
// copies of a panel on its way to `to`; on 128 tiles in the order P's reads, P's copy,
// Q's reads, Q's copy, spread between the matrix instructions.  (Reads and copies stay in
// the order written, as the compiler does not tell a transposing read from what a copy
// writes.)
template <typename E, typename SP, typename SQ, int T, int F>
__device__ __forceinline__ void small_quarter(const lds_char *at, const int (&pat)[T], const int (&qat)[T], int kk,
                                              uint4v (&a)[T], uint4v (&b)[T], lds_char *to, SP &sp, SQ &sq, int wave,
                                              float16v (&acc)[T][T], const uint4v (&a0)[T], const uint4v (&b0)[T])
{
    static_assert(SP::kLoads == 2 * T && SQ::kLoads == 2 * T && SP::kParts == 4, "the copies of a quarter");
    constexpr int kMma = sizeof(typename E::store) == 4 ? 4 : 1;   // instructions of an mma
#pragma unroll
    for (int i = 0; i < T; ++i)
        a[i] = SP::frag(at, pat[i], kk);
    if constexpr (T == 2)
        sp.template load<F, F + 1>(to, wave);
    else if constexpr (F < 2)
        sp.template load<F, F + 1>(to, wave);
    else
        sq.template load<F - 2, F - 1>(to + SP::kBytes, wave);
#pragma unroll
    for (int j = 0; j < T; ++j)
        b[j] = SQ::frag(at + SP::kBytes, qat[j], kk);
    if constexpr (T == 2)
        sq.template load<F, F + 1>(to + SP::kBytes, wave);
    multiply<E>(acc, a0, b0);
    if constexpr (T == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, SP::kReads, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, kMma, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, SQ::kReads, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, kMma, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// One panel after another in a ring of RING: the fragments of one quarter of a panel's
// depth are read while the one before is multiplied.  One barrier a panel, in front of
// its last quarter: behind it every wave has all of panel k in registers, so its slot
// takes panel k + RING, and panel k + 1 has arrived.  Copies past the last panel bring
// zeros and keep the count of outstanding ones even.
template <typename E, typename SP, typename SQ, int T, int RING>
__device__ __forceinline__ void ahead_loop(lds_char *__restrict__ to, const lds_char *__restrict__ from, SP &sp, SQ &sq,
                                           const int (&pat)[T], const int (&qat)[T], float16v (&acc)[T][T], int panels, int wave)
{
    constexpr int kBytes = SP::kBytes + SQ::kBytes, kCopies = SP::kLoads + SQ::kLoads;
    uint4v a[2][T], b[2][T];
    if (panels < RING) {   // all there is fits the ring
        for (int s = 0; s < panels; ++s) {
            sp.load(to + s * kBytes, wave);
            sq.load(to + s * kBytes + SP::kBytes, wave);
        }
        wait_copies<0>();
        ring_barrier(to, from);
        for (int s = 0; s < panels; ++s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                read_part<SP, SQ>(from + s * kBytes, from + s * kBytes + SP::kBytes, pat, qat, kk, a[0], b[0]);
                multiply<E>(acc, a[0], b[0]);
            }
        return;
    }
#pragma unroll
    for (int s = 0; s < RING - 1; ++s) {
        sp.load(to + s * kBytes, wave);
        sq.load(to + s * kBytes + SP::kBytes, wave);
    }
    sp.template load<0, 1>(to + (RING - 1) * kBytes, wave);
    if constexpr (T == 2)
        sq.template load<0, 1>(to + (RING - 1) * kBytes + SP::kBytes, wave);
    wait_copies<(RING - 2) * kCopies + T>();
    ring_barrier(to, from);
    read_part<SP, SQ>(from, from + SP::kBytes, pat, qat, 0, a[0], b[0]);
    for (int k = 0; k < panels; k += RING)
#pragma unroll
        for (int slot = 0; slot < RING; ++slot) {
            const lds_char *at = from + slot * kBytes;
            const int next = slot == RING - 1 ? 0 : slot + 1, before = slot == 0 ? RING - 1 : slot - 1;
            lds_char *const other = to + before * kBytes;
            if (k + slot < panels) {
                small_quarter<E, SP, SQ, T, 1>(at, pat, qat, 1, a[1], b[1], other, sp, sq, wave, acc, a[0], b[0]);
                small_quarter<E, SP, SQ, T, 2>(at, pat, qat, 2, a[0], b[0], other, sp, sq, wave, acc, a[1], b[1]);
                small_quarter<E, SP, SQ, T, 3>(at, pat, qat, 3, a[1], b[1], other, sp, sq, wave, acc, a[0], b[0]);
                __builtin_amdgcn_sched_barrier(0);
                wait_copies<(RING - 2) * kCopies>();
                ring_barrier(to, from);
                __builtin_amdgcn_sched_barrier(0);
                small_quarter<E, SP, SQ, T, 0>(from + next * kBytes, pat, qat, 0, a[0], b[0], to + slot * kBytes, sp, sq, wave,
                                               acc, a[1], b[1]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
}

// One 64 x 64 tile of C, or one piece of its depth; three workgroups a compute unit, or
// more where the depth is less than the ring, which is no longer than it has to be (16384 x
// 64 -> 4096: 56 us with three, 48 with four).
constexpr int kRing64 = 3;
template <typename E, bool PD, bool QD, typename OUT>
__global__ __launch_bounds__(256) void k_product_64(Product g)
{
#if defined(__HIP_DEVICE_COMPILE__)   // the host's pass does not know the matrix and LDS builtins
    constexpr int TILE = 64, RING = kRing64;
    typedef Side<E, PD, TILE, 4, 128> SP;
    typedef Side<E, QD, TILE, 4, 128> SQ;
    extern __shared__ __align__(1024) char lds[];
    Setup<SP, SQ, TILE, 1, 1> u;
    u.start(g);
    float16v acc[1][1];
    clear(acc);
    ahead_loop<E, SP, SQ, 1, RING>((lds_char *)&lds[0], hidden((const lds_char *)&lds[0]), u.sp, u.sq, u.pat, u.qat, acc,
                                   u.panels, u.wave);
    if (g.splits > 1) {
        wait_copies<0>();   // the LDS is not to be written behind the workgroup's end
        put_parts<TILE>(g, u.tp, u.tq, u.piece, u.wave, u.lane, acc);
        return;
    }
    wait_copies<0>();   // what still comes must not fall into what the LDS holds next
    ring_barrier((lds_char *)&lds[0], (const lds_char *)&lds[0]);
    put_strips<OUT, TILE>(g, u.tp, u.tq, u.wp, u.wq, u.wave, u.lane, &lds[0], acc);
#endif
}

// One 128 x 128 tile of C, or one piece of its depth, on four waves of 64 x 64.  A
// panel's fragment reads and copies keep the LDS busy half again as long as its matrix
// instructions take.  One workgroup a compute unit; a ring of three panels (four or five
// make no difference), its slots known to the compiler (2048^3: 22.0 us with slots kept
// in registers, 21.5 without; 25.3 where a wave reads all of a panel, then multiplies).
template <typename E, bool PD, bool QD, typename OUT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_product_128(Product g)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int TILE = 128, RING = 3;
    typedef Side<E, PD, TILE, 4, 128> SP;
    typedef Side<E, QD, TILE, 4, 128> SQ;
    __shared__ __align__(1024) char lds[lds_of<OUT, 2, 2>(RING * (SP::kBytes + SQ::kBytes))];
    Setup<SP, SQ, TILE, 2, 2> u;
    u.start(g);
    float16v acc[2][2];
    clear(acc);
    ahead_loop<E, SP, SQ, 2, RING>((lds_char *)&lds[0], hidden((const lds_char *)&lds[0]), u.sp, u.sq, u.pat, u.qat, acc,
                                   u.panels, u.wave);
    wait_copies<0>();   // what still comes must not fall into what the LDS holds next
    if (g.splits > 1) {
        put_parts<TILE>(g, u.tp, u.tq, u.piece, u.wave, u.lane, acc);
        return;
    }
    ring_barrier((lds_char *)&lds[0], (const lds_char *)&lds[0]);
    put_strips<OUT, TILE>(g, u.tp, u.tq, u.wp, u.wq, u.wave, u.lane, &lds[0], acc);
#endif
}

// READS LDS reads in front of each of four matrix instructions, then two copies with one
// behind each.
template <int READS>
__device__ __forceinline__ void half_order()
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
}

// A quarter of a panel of k_product_256: multiplies a0 b0, reads the fragments of part
// kk of the panel at p and q, and makes four of the wave's copies of side C's next
// panel, from copy FROM on.  The scheduler is given the order: P's reads between the
// first four of the 16 matrix instructions, two copies, Q's reads, two copies.  (Reads
// and copies stay in the order written, as the compiler does not tell a transposing
// read from what a copy writes.)
template <typename E, typename SP, typename SQ, int T, int FROM, typename SC>
__device__ __forceinline__ void quarter(const lds_char *p, const lds_char *q, const int (&pat)[T], const int (&qat)[T], int kk,
                                        uint4v (&a)[T], uint4v (&b)[T], lds_char *to, SC &side, int wave,
                                        float16v (&acc)[T][T], const uint4v (&a0)[T], const uint4v (&b0)[T])
{
#pragma unroll
    for (int i = 0; i < T; ++i)
        a[i] = SP::frag(p, pat[i], kk);
    side.template load<FROM, FROM + 2>(to, wave);
#pragma unroll
    for (int j = 0; j < T; ++j)
        b[j] = SQ::frag(q, qat[j], kk);
    side.template load<FROM + 2, FROM + 4>(to, wave);
    multiply<E>(acc, a0, b0);
    half_order<SP::kReads>();
    half_order<SQ::kReads>();
    __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
    __builtin_amdgcn_sched_barrier(0);
}

// The same on 256 x 256 tiles with four waves, one a SIMD, each of which holds 128 x
// 128 of C in 256 registers: 64 bytes of depth then take 64 KiB of LDS reads where
// eight waves of 128 x 64 take 96, and with the copies' 32 KiB the LDS is busy for
// three quarters of the time that the matrix instructions take, not for all of it.
// A wave has nobody to hide its waits, so it runs ahead of itself: the fragments of
// one quarter of a panel's depth (128 bytes) are read while the one before is
// multiplied, and the scheduler is told to spread reads and copies between the matrix
// instructions.
//
// One barrier a panel, in front of its last quarter: behind it every wave has all of
// panel k in registers, and panel k + 1 has arrived.  P has two slots, Q three (160
// KiB in all).  P of panel k + 1 is copied through the last quarter of panel k - 1 and
// the first of k, Q of panel k + 2 through the two quarters behind those, one copy to
// four matrix instructions: the address unit is busy for half of its time with them,
// and a wave that has to wait for it issues no matrix instruction either.  Copies past
// the last panel bring zeros and keep the count of outstanding ones even.
// 8192^3, us: with 64-byte panels, whose deep rows are half a cache line, and all of a
// panel's copies behind its barrier 904, spread over the panel 899; as it is 794 (1.38
// PFLOP/s).
template <typename E, typename SP, typename SQ, int T>
__device__ __forceinline__ void wide_loop(lds_char *__restrict__ to, const lds_char *__restrict__ from, SP &sp, SQ &sq,
                                          const int (&pat)[T], const int (&qat)[T], float16v (&acc)[T][T], int panels, int wave)
{
    constexpr int kQ = 2 * SP::kBytes;   // Q's slots lie behind P's two
    static_assert(SP::kLoads == 8 && SQ::kLoads == 8 && T == 4 && SP::kParts == 4, "the schedule below");
    uint4v a[2][T], b[2][T];
    sp.load(to, wave);
    sq.load(to + kQ, wave);
    sq.load(to + kQ + SQ::kBytes, wave);
    sp.template load<0, 4>(to + SP::kBytes, wave);
    wait_copies<12>();
    ring_barrier(to, from);
    read_part<SP, SQ>(from, from + kQ, pat, qat, 0, a[0], b[0]);
    int ps = 0, qs = 0;   // the panel's slots
    for (int k = 0; k < panels; ++k) {
        const lds_char *p = from + ps * SP::kBytes, *q = from + kQ + qs * SQ::kBytes;
        const int before = qs == 0 ? 2 : qs - 1, next = qs == 2 ? 0 : qs + 1;
        lds_char *const p_other = to + (ps ^ 1) * SP::kBytes, *const q_free = to + kQ + before * SQ::kBytes;
        quarter<E, SP, SQ, T, 4>(p, q, pat, qat, 1, a[1], b[1], p_other, sp, wave, acc, a[0], b[0]);
        quarter<E, SP, SQ, T, 0>(p, q, pat, qat, 2, a[0], b[0], q_free, sq, wave, acc, a[1], b[1]);
        quarter<E, SP, SQ, T, 4>(p, q, pat, qat, 3, a[1], b[1], q_free, sq, wave, acc, a[0], b[0]);
        wait_copies<8>();
        ring_barrier(to, from);
        __builtin_amdgcn_sched_barrier(0);
        quarter<E, SP, SQ, T, 0>(from + (ps ^ 1) * SP::kBytes, from + kQ + next * SQ::kBytes, pat, qat, 0, a[0], b[0],
                                 to + ps * SP::kBytes, sp, wave, acc, a[1], b[1]);
        ps ^= 1;
        qs = next;
    }
}

template <typename E, bool PD, bool QD, typename OUT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_product_256(Product g)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int TILE = 256;
    typedef Side<E, PD, TILE, 4, 128> SP;
    typedef Side<E, QD, TILE, 4, 128> SQ;
    __shared__ __align__(1024) char lds[2 * SP::kBytes + 3 * SQ::kBytes];
    static_assert(lds_of<OUT, 4, 4>(0) <= (int)sizeof(lds), "the epilogue's strips");
    Setup<SP, SQ, TILE, 4, 4> u;
    u.start(g);
    float16v acc[4][4];
    clear(acc);
    wide_loop<E, SP, SQ, 4>((lds_char *)&lds[0], hidden((const lds_char *)&lds[0]), u.sp, u.sq, u.pat, u.qat, acc, u.panels, u.wave);
    wait_copies<0>();   // what still comes must not fall into what the LDS holds next
    if (g.splits > 1) {
        put_parts<TILE>(g, u.tp, u.tq, u.piece, u.wave, u.lane, acc);
        return;
    }
    ring_barrier((lds_char *)&lds[0], (const lds_char *)&lds[0]);
    put_strips<OUT, TILE>(g, u.tp, u.tq, u.wp, u.wq, u.wave, u.lane, &lds[0], acc);
#endif
}

// C from the pieces' sums, added in order: a wave per 32 x 32 block of a tile, lanes as
// in the product.
template <int TILE, typename OUT>
__global__ __launch_bounds__(256) void k_product_join(Product g)
{
    constexpr int T = TILE / 64;   // blocks of a wave along either side
    const int lane = threadIdx.x & 63;
    const int64_t tiles = (int64_t)g.tiles_p * g.tiles_q;
    const int64_t block = blockIdx.x * 4ll + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tile = block / (4 * T * T);
    const int of = (int)(block % (4 * T * T)), wave = of / (T * T), i = of % (T * T) / T, j = of % T;
    const float *from = g.parts + block * 1024 + lane * 4;
    float4v s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        s[r] = *reinterpret_cast<const float4v *>(from + r * 256);
#pragma unroll 4
    for (int z = 1; z < g.splits; ++z)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            s[r] += *reinterpret_cast<const float4v *>(from + z * tiles * TILE * TILE + r * 256);
    const DropKey key = OUT::kDrops ? drop_key(g.e.drop) : DropKey{};
    const int64_t tq = tile / g.tiles_p, tp = tile % g.tiles_p;
    put_block<OUT>(g, key, tq * TILE + ((wave & 1) * T + j) * 32, tp * TILE + ((wave >> 1) * T + i) * 32, lane, s);
}

template <typename E, bool PD, bool QD, typename OUT>
hipError_t products(const Product &g, hipStream_t s)
{
    const uint32_t tiles = (uint32_t)g.tiles_p * (uint32_t)g.tiles_q, n = tiles * (uint32_t)g.splits;
    const bool join = g.splits > 1;
    if (g.tile == 256) {
        if constexpr (sizeof(typename E::store) == 2)
            k_product_256<E, PD, QD, OUT><<<n, 256, 0, s>>>(g);
        if (join)
            k_product_join<256, OUT><<<tiles * 16, 256, 0, s>>>(g);
    } else if (g.tile == 128) {
        k_product_128<E, PD, QD, OUT><<<n, 256, 0, s>>>(g);
        if (join)
            k_product_join<128, OUT><<<tiles * 4, 256, 0, s>>>(g);
    } else {
        const int panels = std::max(1, std::min(kRing64, g.piece / 128));
        const bool reads = g.e.add || g.e.mul;
        const int strips = 4 * (reads ? Strip<OUT, 1, 1, true>::kBytes : Strip<OUT, 1, 1, false>::kBytes);
        k_product_64<E, PD, QD, OUT><<<n, 256, std::max(panels * 2 * 64 * 128, strips), s>>>(g);
        if (join)
            k_product_join<64, OUT><<<tiles, 256, 0, s>>>(g);
    }
    return hipGetLastError();
}

template <typename E>
hipError_t product_of(Form form, int32_t out_dtype, const Product &g, hipStream_t s)
{
    if (form == kForward) {
        // The less an epilogue may have to do, the fewer registers and instructions: 16384 x
        // 64 -> 4096 without any of it 48 us in the form for all, 34 in its own, and 8192 x
        // 2048 -> 8192 239 and 222; that with residual dropout 288, 268 in a form without
        // activations.
        const Epilogue &e = g.e;
        if (e.act != Z1_ACT_NONE)
            return products<E, true, true, FullOut<E, true>>(g, s);
        if (e.pre || e.mul || e.bias || e.drop.rng)
            return products<E, true, true, FullOut<E, false>>(g, s);
        return products<E, true, true, PlainOut<E>>(g, s);
    }
    if (form == kInput)
        return products<E, false, true, PlainOut<E>>(g, s);
    if (out_dtype == Z1_F32)
        return products<E, false, false, PlainOut<F32>>(g, s);
    return products<E, false, false, PlainOut<E>>(g, s);
}

// z1_linear of up to R rows: the weight is read once and everything else is small, so a
// wave streams two rows of it past x, each lane its groups of eight elements, and the
// lanes' sums are added up; eight outputs a workgroup go through the epilogue together.
// Operands at any alignment.  1 x 2048 -> 2048 bf16: 4.4 us (split products of 64
// tiles and their join 10).  Memory bounds it: 1 x 4096 -> 11008 reads its weight at 4.4 TB/s.
template <typename E, int R, typename OUT>
__global__ __launch_bounds__(256) void k_linear_rows(Product g)
{
    typedef typename E::store store;
    __shared__ float sums[R][8];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t col = blockIdx.x * 8, K = g.p.depth;
    const store *w[2], *x[R];
#pragma unroll
    for (int o = 0; o < 2; ++o)
        w[o] = reinterpret_cast<const store *>(static_cast<const char *>(g.p.base) + min(col + wave * 2 + o, g.P - 1) * g.p.ld);
#pragma unroll
    for (int r = 0; r < R; ++r)
        x[r] = reinterpret_cast<const store *>(static_cast<const char *>(g.q.base) + min(r, g.Q - 1) * g.q.ld);
    float acc[2][R] = {};
    const auto add = [&](const float (&a)[2][8], const float (&b)[R][8]) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    acc[o][r] = fmaf(a[o][j], b[r][j], acc[o][r]);
    };
    int32_t k = lane * 8;
#pragma unroll 4
    for (; k + 8 <= K; k += 512) {
        float a[2][8], b[R][8];
#pragma unroll
        for (int o = 0; o < 2; ++o)
            Eight<E>::load(w[o] + k, a[o]);
#pragma unroll
        for (int r = 0; r < R; ++r)
            Eight<E>::load(x[r] + k, b[r]);
        add(a, b);
    }
    if (k < K) {
        float a[2][8], b[R][8];
#pragma unroll
        for (int o = 0; o < 2; ++o)
            Eight<E>::load_some(w[o] + k, a[o], K - k);
#pragma unroll
        for (int r = 0; r < R; ++r)
            Eight<E>::load_some(x[r] + k, b[r], K - k);
        add(a, b);
    }
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int d = 32; d > 0; d >>= 1)
                acc[o][r] += __shfl_xor(acc[o][r], d);
            if (lane == 0)
                sums[r][wave * 2 + o] = acc[o][r];
        }
    __syncthreads();
    const int r = threadIdx.x;
    if (r < g.Q) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = sums[r][j];
        put_now<OUT>(g.e, drop_key(g.e.drop), r, col, g.P - col, v);
    }
}

template <typename E>
hipError_t rows_of(const Product &g, hipStream_t s)
{
    const uint32_t n = (uint32_t)(g.P + 7) / 8;
    if (g.Q <= 1)
        k_linear_rows<E, 1, FullOut<E, true>><<<n, 256, 0, s>>>(g);
    else if (g.Q <= 2)
        k_linear_rows<E, 2, FullOut<E, true>><<<n, 256, 0, s>>>(g);
    else
        k_linear_rows<E, kRowsMost, FullOut<E, true>><<<n, 256, 0, s>>>(g);
    return hipGetLastError();
}

// Eight elements of a row each; rows start anywhere and end in zeros.  The first `first`
// workgroups make copy a, the others b: one launch for both operands of a product (777 x
// 333 in fp32 takes 3.5 us, most of it the launch).
template <typename T>
__global__ __launch_bounds__(256) void k_pack(Copy a, Copy b, uint32_t first)
{
    const bool second = blockIdx.x >= first;
    const Copy c = second ? b : a;
    const int64_t per = c.cols_to / 8, block = second ? blockIdx.x - first : blockIdx.x;
    const int64_t blocks = second ? gridDim.x - first : first;
    for (int64_t i = block * 256 + threadIdx.x; i < c.rows * per; i += blocks * 256) {
        const int64_t r = i / per, at = i % per * 8;
        float v[8];
        const typename T::store *p = static_cast<const typename T::store *>(c.from) + r * c.ld + at;
        if (at + 8 <= c.cols)
            Eight<T>::load(p, v);
        else
            Eight<T>::load_some(p, v, (int)(c.cols - at));
        Eight<T>::store(static_cast<typename T::store *>(c.to) + r * c.cols_to + at, v);
    }
}

}  // namespace

hipError_t launch_product(Form form, int32_t dtype, int32_t out_dtype, const Product &g, hipStream_t s)
{
    if (g.P == 0 || g.Q == 0)
        return hipSuccess;
    switch (dtype) {
    case Z1_F32: return product_of<F32>(form, out_dtype, g, s);
    case Z1_BF16: return product_of<BF16>(form, out_dtype, g, s);
    default: return product_of<F16>(form, out_dtype, g, s);
    }
}

hipError_t launch_rows(int32_t dtype, const Product &g, hipStream_t s)
{
    switch (dtype) {
    case Z1_F32: return rows_of<F32>(g, s);
    case Z1_BF16: return rows_of<BF16>(g, s);
    default: return rows_of<F16>(g, s);
    }
}

hipError_t launch_pack(int32_t dtype, const Copy &a, const Copy &b, hipStream_t s)
{
    const auto grid = [](const Copy &c) { return (uint32_t)std::min<int64_t>((c.rows * (c.cols_to / 8) + 255) / 256, 8192); };
    const uint32_t first = grid(a), all = first + grid(b);
    if (all == 0)
        return hipSuccess;
    switch (dtype) {
    case Z1_F32: k_pack<F32><<<all, 256, 0, s>>>(a, b, first); break;
    case Z1_BF16: k_pack<BF16><<<all, 256, 0, s>>>(a, b, first); break;
    default: k_pack<F16><<<all, 256, 0, s>>>(a, b, first); break;
    }
    return hipGetLastError();
}

}  // namespace ops
}  // namespace z1

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

// One operand's share of a panel (64 bytes of depth: 32 or 16 elements) in LDS,
// TILE * 64 bytes, copied there directly, 1 KiB a wave and instruction; and the
// fragments of 32 indexes x 16 bytes of depth read from it.
//
// Deep operands: a row of 64 bytes for each index.  Four rows span the 64 banks;
// the 16-byte chunks of row r sit permuted by (r / 4) mod 4, so that the lanes
// of a fragment read that share a cycle touch all banks once.
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
template <typename E, bool DEEP, int TILE, int NW>
struct Side {
    static constexpr int kSize = (int)sizeof(typename E::store);
    static constexpr int kPanel = 64 / kSize;             // depth of a panel
    static constexpr int kLoads = TILE / 16 / NW;         // copies per wave and panel
    static constexpr int kRow = TILE * kSize;             // bytes of a row in LDS, if not deep
    static constexpr int kChunks = kRow / 16;
    static_assert(kLoads >= 1 && kChunks >= 8, "tile");

    const char *base;        // of the next panel
    int64_t step;
    int32_t left;            // depth from there on: bytes if deep, else rows
    uint32_t at[kLoads];     // offsets of this lane's copies
    int32_t limit[kLoads];   // copied while limit < left

    static __device__ __forceinline__ int turn(int k)     // what row k's chunks are xored with
    {
        if (kSize == 4)
            return ((k >> 2) & 1) << 3;
        return kChunks >= 16 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
    }

    __device__ __forceinline__ void start(const Operand &o, int32_t tile, int32_t panel, int wave, int lane)
    {
        const int32_t i0 = tile * TILE;
        base = static_cast<const char *>(o.base);
        if (DEEP) {
            base += (int64_t)i0 * o.ld + (int64_t)panel * 64;
            step = 64;
            left = o.depth * kSize - panel * 64;
        } else {
            base += (int64_t)panel * kPanel * o.ld + (int64_t)i0 * kSize;
            step = kPanel * o.ld;
            left = o.depth - panel * kPanel;
        }
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int c = (wave * kLoads + q) * 64 + lane;
            if (DEEP) {
                const int row = c >> 2, chunk = (c & 3) ^ ((row >> 2) & 3);
                at[q] = (uint32_t)min(row, o.extent - 1 - i0) * (uint32_t)o.ld + chunk * 16;
                limit[q] = chunk * 16;
            } else {
                const int k = c / kChunks, chunk = (c % kChunks) ^ turn(k);
                at[q] = (uint32_t)k * (uint32_t)o.ld + chunk * 16;
                // behind the row's end: never copied
                limit[q] = (i0 * (int64_t)kSize + chunk * 16 < (int64_t)o.extent * kSize) ? k : INT32_MAX;
            }
        }
    }

    // Copies the next panel to `to` in LDS.
    __device__ __forceinline__ void load(char *to, int wave)
    {
        const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, kRange, 0x00020000);
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(to + (wave * kLoads + q) * 1024), 16,
                                                     limit[q] < left ? at[q] : kOutside, 0, 0, 0);
        base += step;
        left -= DEEP ? 64 : kPanel;
    }

    // Where fragments of the 32 indexes from i0 are read, for frag().
    static __device__ __forceinline__ int place(int i0, int lane)
    {
        const int half = lane >> 5, low = lane & 31;
        if (DEEP)
            return (i0 + low) * 64 + ((half ^ ((low >> 2) & 3)) * 16);
        if (kSize == 4) {
            const int k = 4 * half, col = i0 + low;
            return k * kRow + (((col >> 2) ^ turn(k)) << 4) + (col & 3) * 4;
        }
        const int k = 8 * half + ((lane >> 2) & 3), col = i0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        return k * kRow + (((col >> 3) ^ turn(k)) << 4) + (col & 7) * 2;
    }

    // The fragment of half kk of the panel's depth.
    static __device__ __forceinline__ uint4v frag(const char *lds, int place, int kk)
    {
        if (DEEP)
            return *reinterpret_cast<const uint4v *>(lds + (place ^ (kk * 32)));
        if (kSize == 4) {
            uint4v v;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                v[s] = *reinterpret_cast<const uint32_t *>(lds + place + (8 * kk + s) * kRow);
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
// Epilogues: eight elements (row, col ..) of C, of which n are inside it.
// --------------------------------------------------------------------------

template <typename O>
struct PlainOut {
    static constexpr bool kDrops = false;
    static __device__ __forceinline__ void put(const Epilogue &e, const DropKey &, int64_t row, int32_t col, int n,
                                               float (&v)[8])
    {
        typedef typename O::store store;
        store *out = static_cast<store *>(e.out) + row * e.ld_out + col;
        const store *add = static_cast<const store *>(e.add) + row * e.ld_add + col;
        float a[8];
        if (n >= 8) {
            if (e.add) {
                Eight<O>::load(add, a);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += a[j];
            }
            Eight<O>::store(out, v);
        } else {
            if (e.add) {
                Eight<O>::load_some(add, a, n);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += a[j];
            }
            Eight<O>::store_some(out, v, n);
        }
    }
};

template <typename E>
struct FullOut {
    static constexpr bool kDrops = true;
    static __device__ __forceinline__ void get(const void *p, int64_t at, int n, float (&v)[8])
    {
        const typename E::store *from = static_cast<const typename E::store *>(p) + at;
        if (n >= 8)
            Eight<E>::load(from, v);
        else
            Eight<E>::load_some(from, v, n);
    }
    static __device__ __forceinline__ void set(void *p, int64_t at, int n, const float (&v)[8])
    {
        typename E::store *to = static_cast<typename E::store *>(p) + at;
        if (n >= 8)
            Eight<E>::store(to, v);
        else
            Eight<E>::store_some(to, v, n);
    }
    static __device__ __forceinline__ void put(const Epilogue &e, const DropKey &key, int64_t row, int32_t col, int n,
                                               float (&v)[8])
    {
        float a[8];
        if (e.bias) {
            get(e.bias, col, n, a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += a[j];
        }
        if (e.pre)
            set(e.pre, row * e.ld_pre + col, n, v);
        if (e.act != Z1_ACT_NONE)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = act_value(e.act, v[j]);
        if (e.mul) {
            get(e.mul, row * e.ld_mul + col, n, a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] *= a[j];
        }
        if (key.on)
            drop8(key, (uint32_t)col >> 3, (uint32_t)row, v);
        if (e.add) {
            get(e.add, row * e.ld_add + col, n, a);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += a[j];
        }
        set(e.out, row * e.ld_out + col, n, v);
    }
};

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
            OUT::put(g.e, key, q, (int32_t)p, (int)(g.P - p), v);
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

// One TILE x TILE tile of C, one 64-byte deep panel after another, in a ring of
// RING panels, so that RING - 1 are on their way while one is multiplied.
// PAIRED (256 tiles, 8 waves, one workgroup a compute unit): waves w and w + 4
// share a SIMD, and the second four run half a step behind the first, so that
// one of the two multiplies while the other reads its fragments and issues
// copies; two barriers a panel keep them in step.
template <typename E, bool PD, bool QD, int TILE, int WP, int WQ, int PANELS, int RING, bool PAIRED, typename OUT>
__global__ __launch_bounds__(64 * WP * WQ) void k_product(Product g)
{
#if defined(__HIP_DEVICE_COMPILE__)   // the host's pass does not know the matrix and LDS builtins
    constexpr int NW = WP * WQ;
    constexpr int TP = TILE / WP / 32, TQ = TILE / WQ / 32;
    static_assert(!PAIRED || PANELS == 1, "one panel a phase");
    typedef Side<E, PD, TILE, NW> SP;
    typedef Side<E, QD, TILE, NW> SQ;
    constexpr int kShare = TILE * 64;
    constexpr int kAhead = (RING - 2) * PANELS * (SP::kLoads + SQ::kLoads);   // copies that may stay out at a wait
    __shared__ __align__(1024) char lds[RING][PANELS][2][kShare];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave / WQ, wq = wave % WQ;
    int32_t tp, tq, piece;
    tile_of(g, blockIdx.x, gridDim.x, tp, tq, piece);

    SP sp;
    SQ sq;
    const int32_t first = piece * g.piece;
    sp.start(g.p, tp, first, wave, lane);
    sq.start(g.q, tq, first, wave, lane);
    const int32_t panels = min(g.piece, (g.p.depth + SP::kPanel - 1) / SP::kPanel - first);
    const int steps = (panels + PANELS - 1) / PANELS;

    int pat[TP], qat[TQ];
#pragma unroll
    for (int i = 0; i < TP; ++i)
        pat[i] = SP::place((wp * TP + i) * 32, lane);
#pragma unroll
    for (int j = 0; j < TQ; ++j)
        qat[j] = SQ::place((wq * TQ + j) * 32, lane);

    const auto load = [&](int slot, int panel) {
        sp.load(lds[slot][panel][0], wave);
        sq.load(lds[slot][panel][1], wave);
    };

    float16v acc[TP][TQ];
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.f;

#pragma unroll
    for (int s = 0; s < RING - 1; ++s)
        if (s < steps)
#pragma unroll
            for (int p = 0; p < PANELS; ++p)
                load(s, p);
    if (PAIRED) {
        if (steps >= RING - 1)
            wait_copies<kAhead>();
        else
            wait_copies<0>();
        __builtin_amdgcn_s_barrier();
        if (wave >= NW / 2)
            __builtin_amdgcn_s_barrier();
    }
    int slot = 0;
    for (int k = 0; k < steps; ++k) {
        const int next = slot == 0 ? RING - 1 : slot - 1;   // the slot of step k + RING - 1
        const bool more = k + RING - 1 < steps;
        if (!PAIRED) {
            // panel k has arrived, and every wave has read panel k - 1, whose
            // slot the next copy overwrites
            if (k + RING - 2 < steps)
                wait_copies<kAhead>();
            else
                wait_copies<0>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (more)
#pragma unroll
                for (int p = 0; p < PANELS; ++p)
                    load(next, p);
        }
        uint4v a[2 * PANELS][TP], b[2 * PANELS][TQ];
        asm volatile("" ::: "memory");
#pragma unroll
        for (int kk = 0; kk < 2 * PANELS; ++kk) {
#pragma unroll
            for (int j = 0; j < TQ; ++j)
                b[kk][j] = SQ::frag(lds[slot][kk >> 1][1], qat[j], kk & 1);
#pragma unroll
            for (int i = 0; i < TP; ++i)
                a[kk][i] = SP::frag(lds[slot][kk >> 1][0], pat[i], kk & 1);
        }
        if (PAIRED) {
            // the slot being filled was last read in panel k - 1, by both
            // halves before the barrier that ended their reads of it
            if (more)
                load(next, 0);
            asm volatile("" ::: "memory");
            // panel k + 1 has arrived once every wave is past this barrier
            if (more)
                wait_copies<kAhead>();
            else
                wait_copies<0>();
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int kk = 0; kk < 2 * PANELS; ++kk)
#pragma unroll
            for (int i = 0; i < TP; ++i)
#pragma unroll
                for (int j = 0; j < TQ; ++j)
                    mma(E(), acc[i][j], a[kk][i], b[kk][j]);
        if (PAIRED) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" ::: "memory");
        slot = slot + 1 == RING ? 0 : slot + 1;
    }
    if (PAIRED && wave < NW / 2)
        __builtin_amdgcn_s_barrier();   // as many as the second four

    if (g.splits > 1) {
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
        return;
    }
    const DropKey key = OUT::kDrops ? drop_key(g.e.drop) : DropKey{};
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j) {
            float4v v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[r] = float4v{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
            put_block<OUT>(g, key, (int64_t)tq * TILE + (wq * TQ + j) * 32, (int64_t)tp * TILE + (wp * TP + i) * 32, lane, v);
        }
#endif
}

// C from the pieces' sums, added in order: a wave per 32 x 32 block of a 64 x 64
// tile, lanes as in the product.
template <typename OUT>
__global__ __launch_bounds__(256) void k_product_join(Product g)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles = (int64_t)g.tiles_p * g.tiles_q, tile = blockIdx.x;
    const float *from = g.parts + tile * 4096 + wave * 1024 + lane * 4;
    float4v s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        s[r] = *reinterpret_cast<const float4v *>(from + r * 256);
#pragma unroll 4
    for (int z = 1; z < g.splits; ++z)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            s[r] += *reinterpret_cast<const float4v *>(from + z * tiles * 4096 + r * 256);
    const DropKey key = OUT::kDrops ? drop_key(g.e.drop) : DropKey{};
    const int64_t tq = tile / g.tiles_p, tp = tile % g.tiles_p;
    put_block<OUT>(g, key, tq * 64 + (wave & 1) * 32, tp * 64 + (wave >> 1) * 32, lane, s);
}

template <typename E, bool PD, bool QD, typename OUT>
hipError_t products(const Product &g, hipStream_t s)
{
    const uint32_t tiles = (uint32_t)g.tiles_p * (uint32_t)g.tiles_q, n = tiles * (uint32_t)g.splits;
    if (g.tile == 256) {
        if constexpr (sizeof(typename E::store) == 2)
            k_product<E, PD, QD, 256, 2, 4, 1, 4, true, OUT><<<n, 512, 0, s>>>(g);
    } else if (g.tile == 128) {
        k_product<E, PD, QD, 128, 2, 2, 1, 3, false, OUT><<<n, 256, 0, s>>>(g);
    } else {
        k_product<E, PD, QD, 64, 2, 2, 2, 3, false, OUT><<<n, 256, 0, s>>>(g);
        if (g.splits > 1)
            k_product_join<OUT><<<tiles, 256, 0, s>>>(g);
    }
    return hipGetLastError();
}

template <typename E>
hipError_t product_of(Form form, int32_t out_dtype, const Product &g, hipStream_t s)
{
    if (form == kForward)
        return products<E, true, true, FullOut<E>>(g, s);
    if (form == kInput)
        return products<E, false, true, PlainOut<E>>(g, s);
    if (out_dtype == Z1_F32)
        return products<E, false, false, PlainOut<F32>>(g, s);
    return products<E, false, false, PlainOut<E>>(g, s);
}

// Eight elements of a row each; rows start anywhere and end in zeros.
template <typename T>
__global__ __launch_bounds__(256) void k_pack(const void *from, int64_t ld, void *to, int64_t cols_to, int64_t rows, int64_t cols)
{
    const int64_t per = cols_to / 8;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < rows * per; i += gridDim.x * 256ll) {
        const int64_t r = i / per, c = i % per * 8;
        float v[8];
        const typename T::store *p = static_cast<const typename T::store *>(from) + r * ld + c;
        if (c + 8 <= cols)
            Eight<T>::load(p, v);
        else
            Eight<T>::load_some(p, v, (int)(cols - c));
        Eight<T>::store(static_cast<typename T::store *>(to) + r * cols_to + c, v);
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

hipError_t launch_pack(int32_t dtype, const void *from, int64_t ld, void *to, int64_t cols_to, int64_t rows,
                       int64_t cols, hipStream_t s)
{
    const int64_t n = rows * (cols_to / 8);
    if (n == 0)
        return hipSuccess;
    const uint32_t grid = (uint32_t)std::min<int64_t>((n + 255) / 256, 8192);
    switch (dtype) {
    case Z1_F32: k_pack<F32><<<grid, 256, 0, s>>>(from, ld, to, cols_to, rows, cols); break;
    case Z1_BF16: k_pack<BF16><<<grid, 256, 0, s>>>(from, ld, to, cols_to, rows, cols); break;
    default: k_pack<F16><<<grid, 256, 0, s>>>(from, ld, to, cols_to, rows, cols); break;
    }
    return hipGetLastError();
}

}  // namespace ops
}  // namespace z1

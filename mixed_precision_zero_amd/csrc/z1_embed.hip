// z1_embed.hip -- embedding lookup with scaling, and its gradient.
//
//   out[t] = scale W[id_t]          dW[v] (+)= scale sum_{t: id_t = v} dout[t]
//
// Both are bound by bytes.  The gradient adds rows of equal ids without
// atomics, so that it gives the same bits every time: the positions are
// sorted by id (a stable radix sort), the sorted positions are cut into
// chunks of equal length, and every chunk walks its rows in order, keeping
// the running sum of the current id in registers.  An id whose run lies
// inside one chunk is written at once; a run that crosses chunks leaves one
// partial row per chunk, and the join adds those in order.  Chunks of equal
// length keep the sums' work even however often the commonest id occurs; the
// join's is not, for one workgroup adds a run's partial rows, four at a time
// (65536 equal ids: 252 us instead of 210 at 2048 columns, 348 instead of 66 at
// 64, where chunks are of 16).
//
// Lanes are laid over (chunk, 16-byte vector of the row) pairs in one flat
// order, so that rows of any length fill whole waves.
//
// Measured, bf16: 65536 x 2048 into 49152 rows of fp32 sums, 269 us in all:
// lookup 83 (4.7 TB/s), sort 27, sums 143 (5.4 TB/s), join 12.  8192 x 576,
// 44 us: lookup 5, sort of up to 8192 positions in one workgroup while the
// others clear dW 22 (5.1 TB/s of zeros), sums 10, join 5.
#include "z1_ops_internal.h"

namespace z1 {
namespace ops {
namespace {

__device__ __forceinline__ int64_t id_at(const EmbedShape &e, int64_t t)
{
    return e.id32 ? (int64_t) static_cast<const int32_t *>(e.ids)[t]
                  : static_cast<const int64_t *>(e.ids)[t];
}

// The sort key of a position: its id, or vocab for an id that has no row.
__device__ __forceinline__ uint32_t key_at(const EmbedShape &e, int64_t t)
{
    const int64_t id = id_at(e, t);
    return id < 0 || id >= e.vocab ? (uint32_t)e.vocab : (uint32_t)id;
}

// Flat lane index -> (row, vector) with `per` vectors a row.
struct Flat {
    int64_t row;
    int32_t vec;
    __device__ __forceinline__ Flat(int32_t per, int64_t row0)
    {
        const int64_t first = (int64_t)blockIdx.x * blockDim.x;
        const int64_t r0 = first / per;
        const uint32_t at = (uint32_t)(first - r0 * per) + threadIdx.x;
        const uint32_t up = at / (uint32_t)per;
        row = row0 + r0 + up;
        vec = (int32_t)(at - up * (uint32_t)per);
    }
};

// N elements of type T as fp32.
template <typename T, int N>
struct Vec {
    float f[N];
    template <bool STREAM = false>
    __device__ __forceinline__ void load(const void *base, int64_t i)
    {
        const typename T::store *p = static_cast<const typename T::store *>(base) + i;
        if (N == 1) {
            f[0] = T::up(p[0]);
        } else {
            Pack16<T> q;
            q.raw = STREAM ? __builtin_nontemporal_load(reinterpret_cast<const uint4v *>(p))
                           : *reinterpret_cast<const uint4v *>(p);
#pragma unroll
            for (int k = 0; k < N; ++k)
                f[k] = T::up(q.e[k]);
        }
    }
    // STREAM: more than the caches hold is being written
    template <bool STREAM>
    __device__ __forceinline__ void store(void *base, int64_t i) const
    {
        typename T::store *p = static_cast<typename T::store *>(base) + i;
        if (N == 1) {
            p[0] = T::down(f[0]);
        } else {
            Pack16<T> q;
#pragma unroll
            for (int k = 0; k < N; ++k)
                q.e[k] = T::down(f[k]);
            if (STREAM)
                __builtin_nontemporal_store(q.raw, reinterpret_cast<uint4v *>(p));
            else
                *reinterpret_cast<uint4v *>(p) = q.raw;
        }
    }
    // as fp32 rows
    __device__ __forceinline__ void load_f32(const float *p)
    {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            if (N == 1) {
                f[0] = p[0];
            } else {
                const float4v q = *reinterpret_cast<const float4v *>(p + k);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[(k + j) % N] = q[j];
            }
        }
    }
    __device__ __forceinline__ void store_f32(float *p) const
    {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            if (N == 1)
                p[0] = f[0];
            else
                *reinterpret_cast<float4v *>(p + k) =
                    float4v{f[k], f[(k + 1) % N], f[(k + 2) % N], f[(k + 3) % N]};
        }
    }
};

// R positions a lane, whose ids, rows and results are each in flight together.
template <typename T, int N, int R>
__global__ __launch_bounds__(256) void k_lookup(EmbedShape e, const void *w, int64_t ld_w, void *out,
                                                int64_t ld_out, int32_t per, int64_t row0, int64_t row1)
{
    const Flat at(per, row0);
    if (at.row >= row1)
        return;
    const int64_t first = at.row * R, col = (int64_t)at.vec * N;
    int64_t id[R];
    Vec<T, N> x[R];
#pragma unroll
    for (int q = 0; q < R; ++q)
        id[q] = first + q < e.n ? id_at(e, first + q) : -1;
#pragma unroll
    for (int q = 0; q < R; ++q) {
        if (id[q] >= 0 && id[q] < e.vocab) {
            x[q].load(w, id[q] * ld_w + col);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[q].f[k] = id[q] < 0 ? 0.f : __builtin_nanf("");
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
        if (first + q >= e.n)
            break;
#pragma unroll
        for (int k = 0; k < N; ++k)
            x[q].f[k] *= e.scale;
        x[q].template store<(R > 1)>(out, (first + q) * ld_out + col);
    }
}

// ------------------------------------------------------------------ sorting

// Rows of zeros, written by the workgroups that a sort kernel does not need:
// the sort's few workgroups and the gradient's zeros share the GPU.
__device__ __forceinline__ void fill_zero(float *p, int64_t n, int64_t block, int64_t blocks)
{
    const int64_t step = blocks * blockDim.x, first = block * blockDim.x + threadIdx.x;
    if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
        float4v *q = reinterpret_cast<float4v *>(p);
#pragma unroll 4
        for (int64_t i = first; i < n / 4; i += step)
            __builtin_nontemporal_store(float4v{0.f, 0.f, 0.f, 0.f}, q + i);
        for (int64_t i = n / 4 * 4 + first; i < n; i += step)
            p[i] = 0.f;
    } else {
        for (int64_t i = first; i < n; i += step)
            p[i] = 0.f;
    }
}

// Lanes of the wave whose 8-bit digit equals this lane's (among active ones).
__device__ __forceinline__ uint64_t match_digit(uint32_t digit, bool active)
{
    uint64_t m = __ballot(active);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint64_t set = __ballot(active && ((digit >> b) & 1u));
        m &= (digit >> b) & 1u ? set : ~set;
    }
    return m;
}

// Stable placement of one wave's `rounds` * 64 consecutive items by digit:
// `next[digit]` (this wave's own row in LDS) holds where the next one goes.
// place(i, position) is called for the items i below n.
template <typename K, typename F>
__device__ __forceinline__ void place_wave(volatile uint32_t *next, int64_t first, int rounds,
                                           int64_t n, K &&key_of, int shift, F &&place)
{
    const int lane = threadIdx.x & 63;
    for (int r = 0; r < rounds; ++r) {
        const int64_t i = first + r * 64 + lane;
        const bool live = i < n;
        const uint32_t key = live ? key_of(i) : 0u;
        const uint32_t d = (key >> shift) & 255u;
        const uint64_t same = match_digit(d, live);
        const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
        uint32_t at = 0;
        if (live)
            at = next[d];
        __builtin_amdgcn_wave_barrier();   // every lane has read before the first adds
        if (live && rank == 0)
            next[d] = at + (uint32_t)__popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (live)
            place(i, key, at + rank);
    }
}

// Exclusive prefix of one value a thread over the first 256 threads; every
// thread of the workgroup calls it.
__device__ __forceinline__ uint32_t prefix_256(uint32_t x, uint32_t *tmp)
{
    const int t = threadIdx.x, lane = t & 63;
    uint32_t up = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = __shfl_up(up, o);
        if (lane >= o)
            up += y;
    }
    if (t < 256 && lane == 63)
        tmp[t >> 6] = up;
    __syncthreads();
    uint32_t before = up - x;
    for (int w = 0; w < (t >> 6) && w < 4; ++w)
        before += tmp[w];
    return before;
}

// Exclusive prefix, over digits and then waves, of cnt[wave][256]: position of
// each wave's first item of each digit.
template <int WAVES>
__device__ __forceinline__ void prefix_counts(uint32_t (*cnt)[256], uint32_t *tmp)
{
    const int t = threadIdx.x;
    uint32_t total = 0;
    if (t < 256) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const uint32_t c = cnt[w][t];
            cnt[w][t] = total;
            total += c;
        }
    }
    const uint32_t before = prefix_256(total, tmp);
    if (t < 256) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            cnt[w][t] += before;
    }
    __syncthreads();
}

// The whole sort of up to kSortSmall ids in one workgroup's LDS; the other
// workgroups clear dW.
__global__ __launch_bounds__(1024) void k_sort_small(EmbedShape e, int passes, uint32_t *keys,
                                                     uint32_t *perm, float *dw, int64_t dw_elems)
{
    __shared__ uint32_t key[2][kSortSmall];
    __shared__ uint16_t pos[2][kSortSmall];
    __shared__ uint32_t cnt[16][256];
    __shared__ uint32_t tmp[4];
    if (blockIdx.x > 0) {
        fill_zero(dw, dw_elems, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    const int n = (int)e.n;
    const int rounds = (n + 1023) / 1024;          // per wave, 64 items each
    const int wave = threadIdx.x >> 6;
    const int first = wave * rounds * 64;
    for (int i = threadIdx.x; i < n; i += 1024) {
        key[0][i] = key_at(e, i);
        pos[0][i] = (uint16_t)i;
    }
    for (int p = 0; p < passes; ++p) {
        const int src = p & 1, shift = 8 * p;
        for (int i = threadIdx.x; i < 16 * 256; i += 1024)
            (&cnt[0][0])[i] = 0u;
        __syncthreads();
        for (int r = 0; r < rounds; ++r) {
            const int i = first + r * 64 + (threadIdx.x & 63);
            if (i < n)
                atomicAdd(&cnt[wave][(key[src][i] >> shift) & 255u], 1u);
        }
        __syncthreads();
        prefix_counts<16>(cnt, tmp);
        place_wave(cnt[wave], first, rounds, n, [&](int64_t i) { return key[src][i]; }, shift,
                   [&](int64_t i, uint32_t k, uint32_t at) {
                       key[src ^ 1][at] = k;
                       pos[src ^ 1][at] = pos[src][i];
                   });
        __syncthreads();
    }
    const int last = passes & 1;
    for (int i = threadIdx.x; i < n; i += 1024) {
        keys[i] = key[last][i];
        perm[i] = pos[last][i];
    }
}

// One 8-bit pass over many workgroups: hist[block][digit], then placement.  In
// the first pass the workgroups after the last block clear dW.
__global__ __launch_bounds__(256) void k_sort_count(EmbedShape e, const uint32_t *keys, int shift,
                                                    uint32_t *hist, int64_t n_blocks, float *dw,
                                                    int64_t dw_elems)
{
    __shared__ uint32_t cnt[256];
    if (blockIdx.x >= n_blocks) {
        fill_zero(dw, dw_elems, blockIdx.x - n_blocks, gridDim.x - n_blocks);
        return;
    }
    cnt[threadIdx.x] = 0u;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSortBlock;
#pragma unroll
    for (int r = 0; r < kSortBlock / 256; ++r) {
        const int64_t i = first + r * 256 + threadIdx.x;
        if (i < e.n)
            atomicAdd(&cnt[((keys ? keys[i] : key_at(e, i)) >> shift) & 255u], 1u);
    }
    __syncthreads();
    hist[(int64_t)blockIdx.x * 256 + threadIdx.x] = cnt[threadIdx.x];
}

// Many blocks: hist[block][digit] becomes the digit's count in the blocks
// before, and hist[n_blocks][digit] its count in all, by one workgroup whose
// four groups of 256 threads take a quarter of the blocks each.
__global__ __launch_bounds__(1024) void k_sort_prefix(uint32_t *hist, int64_t n_blocks)
{
    __shared__ uint32_t part[4][256];
    const int d = threadIdx.x & 255, group = threadIdx.x >> 8;
    const int64_t lo = n_blocks * group / 4, hi = n_blocks * (group + 1) / 4;
    uint32_t sum = 0;
#pragma unroll 16
    for (int64_t b = lo; b < hi; ++b)
        sum += hist[b * 256 + d];
    part[group][d] = sum;
    __syncthreads();
    uint32_t at = 0;
    for (int g = 0; g < group; ++g)
        at += part[g][d];
#pragma unroll 16
    for (int64_t b = lo; b < hi; ++b) {
        const uint32_t c = hist[b * 256 + d];
        hist[b * 256 + d] = at;
        at += c;
    }
    if (group == 3)
        hist[n_blocks * 256 + d] = at;
}

// Up to this many blocks, each workgroup of the placement adds up the counts
// of the others by itself: 64 blocks 3 us, where a kernel of its own took 11.
constexpr int64_t kSortInline = 128;

__global__ __launch_bounds__(256) void k_sort_place(EmbedShape e, const uint32_t *keys,
                                                    const uint32_t *perm, int shift,
                                                    const uint32_t *hist, int64_t n_blocks,
                                                    uint32_t *keys_out, uint32_t *perm_out)
{
    __shared__ uint32_t cnt[4][256];
    __shared__ uint32_t tmp[4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        cnt[w][threadIdx.x] = 0u;
    __syncthreads();
    constexpr int kRounds = kSortBlock / 256;
    const int64_t first = (int64_t)blockIdx.x * kSortBlock + wave * kRounds * 64;
    const auto key_of = [&](int64_t i) { return keys ? keys[i] : key_at(e, i); };
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t i = first + r * 64 + lane;
        if (i < e.n)
            atomicAdd(&cnt[wave][(key_of(i) >> shift) & 255u], 1u);
    }
    uint32_t all = 0, at = 0;
    if (n_blocks <= kSortInline) {
#pragma unroll 16
        for (int64_t b = 0; b < n_blocks; ++b) {
            const uint32_t c = hist[b * 256 + threadIdx.x];
            all += c;
            at += b < blockIdx.x ? c : 0u;
        }
    } else {
        all = hist[n_blocks * 256 + threadIdx.x];
        at = hist[(int64_t)blockIdx.x * 256 + threadIdx.x];
    }
    at += prefix_256(all, tmp);   // also ends the counting above
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t c = cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = at;
        at += c;
    }
    __syncthreads();
    place_wave(cnt[wave], first, kRounds, e.n, key_of, shift,
               [&](int64_t i, uint32_t k, uint32_t to) {
                   keys_out[to] = k;
                   perm_out[to] = perm ? perm[i] : (uint32_t)i;
               });
}

// --------------------------------------------------------------------- sums

struct SumArgs {
    const uint32_t *keys, *perm;
    int64_t n, vocab, dim, ld, chunk, n_chunks;
    const void *dout;
    float *dw, *parts;      // parts: [n_chunks][2][dim]
    float scale;
    int32_t per, accumulate;
};

template <typename T, int N>
__device__ __forceinline__ void put_row(const SumArgs &a, uint32_t key, int64_t col, Vec<T, N> &s)
{
    float *to = a.dw + (int64_t)key * a.dim + col;
#pragma unroll
    for (int k = 0; k < N; ++k)
        s.f[k] *= a.scale;
    if (a.accumulate) {
        Vec<T, N> old;
        old.load_f32(to);
#pragma unroll
        for (int k = 0; k < N; ++k)
            s.f[k] += old.f[k];
    }
    s.store_f32(to);
}

// Chunk c's walk over its sorted positions.  parts[c][0] gets the sum of a
// run that began before the chunk, parts[c][1] that of one that began in it
// and goes on after it.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_embed_sum(SumArgs a, int64_t row0, int64_t row1)
{
    const Flat at(a.per, row0);
    if (at.row >= row1)
        return;
    const int64_t c = at.row, col = (int64_t)at.vec * N;
    const int64_t lo = c * a.chunk, hi = lo + a.chunk < a.n ? lo + a.chunk : a.n;
    const uint32_t none = (uint32_t)a.vocab;
    const uint32_t before = lo > 0 ? a.keys[lo - 1] : none, after = hi < a.n ? a.keys[hi] : none;
    uint32_t cur = a.keys[lo];
    if (cur == none)
        return;   // nothing but positions without a row from here on
    bool inherited = before == cur;
    Vec<T, N> s;
#pragma unroll
    for (int k = 0; k < N; ++k)
        s.f[k] = 0.f;
    const auto flush = [&](bool goes_on) {
        if (inherited)
            s.store_f32(a.parts + (c * 2) * a.dim + col);
        else if (goes_on)
            s.store_f32(a.parts + (c * 2 + 1) * a.dim + col);
        else
            put_row<T, N>(a, cur, col, s);
    };
    constexpr int U = 8;
    for (int64_t i = lo; i < hi; i += U) {
        uint32_t key[U];
        Vec<T, N> x[U];
        if (i + U <= hi) {
            uint32_t row[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                key[q] = a.keys[i + q];
                row[q] = a.perm[i + q];
            }
#pragma unroll
            for (int q = 0; q < U; ++q)
                x[q].template load<true>(a.dout, (int64_t)row[q] * a.ld + col);
        } else {
#pragma unroll
            for (int q = 0; q < U; ++q) {
                key[q] = none;
                if (i + q < hi) {
                    key[q] = a.keys[i + q];
                    x[q].template load<true>(a.dout, (int64_t)a.perm[i + q] * a.ld + col);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (i + q >= hi || cur == none)
                continue;
            if (key[q] != cur) {
                flush(false);
                cur = key[q];
                inherited = false;
#pragma unroll
                for (int k = 0; k < N; ++k)
                    s.f[k] = x[q].f[k];
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    s.f[k] += x[q].f[k];
            }
        }
    }
    if (cur != none)
        flush(after == cur);
}

// The runs that cross chunks: the chunk in which such a run begins adds its
// own partial row and those of the following chunks, in order.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_embed_join(SumArgs a, int64_t row0, int64_t row1)
{
    const Flat at(a.per, row0);
    if (at.row >= row1 || at.row + 1 >= a.n_chunks)
        return;
    const int64_t c = at.row, col = (int64_t)at.vec * N;
    const int64_t lo = c * a.chunk, hi = lo + a.chunk;
    const uint32_t none = (uint32_t)a.vocab;
    const uint32_t key = a.keys[hi - 1];
    if (key == none || a.keys[hi] != key)
        return;                                     // no run leaves this chunk
    if (a.keys[lo] == key && lo > 0 && a.keys[lo - 1] == key)
        return;                                     // it began in an earlier one
    // the run's last chunk: in steps that double, then halving between the
    // last chunk seen to begin with the id and the first seen not to (a
    // sorted run: keys[first of q] == key for every chunk up to the last)
    int64_t last = c + 1, past = last + 1;
    for (int64_t step = 1; past < a.n_chunks && a.keys[past * a.chunk] == key; step *= 2) {
        last = past;
        past = last + step;
    }
    past = past < a.n_chunks ? past : a.n_chunks;
    while (past - last > 1) {
        const int64_t mid = (last + past) >> 1;
        if (a.keys[mid * a.chunk] == key)
            last = mid;
        else
            past = mid;
    }
    Vec<T, N> s;
    s.load_f32(a.parts + (c * 2 + 1) * a.dim + col);
    int64_t q = c + 1;
    for (; q + 3 <= last; q += 4) {
        Vec<T, N> x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k].load_f32(a.parts + ((q + k) * 2) * a.dim + col);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e)
                s.f[e] += x[k].f[e];
    }
    for (; q <= last; ++q) {
        Vec<T, N> x;
        x.load_f32(a.parts + (q * 2) * a.dim + col);
#pragma unroll
        for (int e = 0; e < N; ++e)
            s.f[e] += x.f[e];
    }
    put_row<T, N>(a, key, col, s);
}

template <typename F>
hipError_t by_type(int32_t dtype, F &&f)
{
    if (dtype == Z1_F32)
        f(F32());
    else if (dtype == Z1_BF16)
        f(BF16());
    else
        f(F16());
    return hipGetLastError();
}

bool at16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Launches f(blocks, first row, end row) over rows * per lanes, in pieces of fewer than
// 2^31 lanes (a launch takes no more than 2^32 - 1).
template <typename F>
void over_rows(int64_t rows, int32_t per, F &&f)
{
    const int64_t step = (INT64_C(1) << 31) / per;
    for (int64_t r = 0; r < rows; r += step)
        f((uint32_t)((std::min(step, rows - r) * per + 255) / 256), r, std::min(rows, r + step));
}

}  // namespace

EmbedWork embed_work(int64_t n, int64_t vocab, int64_t dim)
{
    (void)vocab;
    EmbedWork w{};
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    w.n_blocks = (n + kSortBlock - 1) / kSortBlock;
    // chunks long enough that their partial rows are little beside the rows
    // they sum, short enough to fill the GPU (65536 x 2048 with chunks of 128,
    // 64 and 32: 299, 286 and 289 us)
    w.chunk = 16;
    while (w.chunk < 128 && n * ((dim + 7) / 8) / (w.chunk * 2) >= 262144)
        w.chunk *= 2;
    w.n_chunks = (n + w.chunk - 1) / w.chunk;
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = take(n * 4);
        w.perm[k] = take(n * 4);
    }
    w.hist = take(n ? (w.n_blocks + 1) * 256 * 4 : 0);
    w.parts = take(w.n_chunks * 2 * dim * 4);
    w.bytes = at;
    return w;
}

hipError_t launch_lookup(int32_t dtype, const EmbedShape &e, const void *w, int64_t ld_w, void *out,
                         int64_t ld_out, hipStream_t s)
{
    if (e.n == 0)
        return hipSuccess;
    return by_type(dtype, [&](auto t) {
        typedef decltype(t) T;
        constexpr int N = Pack16<T>::N;
        const bool wide = e.dim % N == 0 && ld_w % N == 0 && ld_out % N == 0 && at16(w) && at16(out);
        const int32_t per = (int32_t)(wide ? e.dim / N : e.dim);
        // four positions a lane once that still fills the GPU (65536 x 2048:
        // 83 us against 108 with one)
        const bool four = wide && e.n * per >= (INT64_C(1) << 20);
        over_rows(four ? (e.n + 3) / 4 : e.n, per, [&](uint32_t nb, int64_t r, int64_t end) {
            if (four)
                k_lookup<T, N, 4><<<nb, 256, 0, s>>>(e, w, ld_w, out, ld_out, per, r, end);
            else if (wide)
                k_lookup<T, N, 1><<<nb, 256, 0, s>>>(e, w, ld_w, out, ld_out, per, r, end);
            else
                k_lookup<T, 1, 1><<<nb, 256, 0, s>>>(e, w, ld_w, out, ld_out, per, r, end);
        });
    });
}

hipError_t launch_embed_grad(int32_t dtype, const EmbedShape &e, const void *dout, int64_t ld,
                             float *dw, bool accumulate, void *work, hipStream_t s)
{
    const int64_t elems = e.vocab * e.dim;
    const int64_t clear = accumulate ? 0 : elems;
    // workgroups that clear dW beside a sort kernel's own
    const uint32_t fill = clear ? (uint32_t)std::min<int64_t>(2048, (clear + 4095) / 4096) : 0;
    const EmbedWork w = embed_work(e.n, e.vocab, e.dim);
    char *base = static_cast<char *>(work);
    uint32_t *keys[2], *perm[2];
    for (int k = 0; k < 2; ++k) {
        keys[k] = reinterpret_cast<uint32_t *>(base + w.keys[k]);
        perm[k] = reinterpret_cast<uint32_t *>(base + w.perm[k]);
    }
    uint32_t *hist = reinterpret_cast<uint32_t *>(base + w.hist);
    int passes = 1;
    while (passes < 4 && (e.vocab >> (8 * passes)) != 0)
        ++passes;
    int last = 0;
    if (e.n == 0) {
        if (fill)
            k_sort_count<<<fill, 256, 0, s>>>(e, nullptr, 0, hist, 0, dw, clear);
        return hipGetLastError();
    }
    if (e.n <= kSortSmall) {
        k_sort_small<<<1 + fill, 1024, 0, s>>>(e, passes, keys[0], perm[0], dw, clear);
    } else {
        const uint32_t nb = (uint32_t)w.n_blocks;
        for (int p = 0; p < passes; ++p) {
            const uint32_t *k = p ? keys[last] : nullptr, *i = p ? perm[last] : nullptr;
            const int to = p ? last ^ 1 : 0;
            k_sort_count<<<nb + (p ? 0 : fill), 256, 0, s>>>(e, k, 8 * p, hist, w.n_blocks, dw, clear);
            if (w.n_blocks > kSortInline)
                k_sort_prefix<<<1, 1024, 0, s>>>(hist, w.n_blocks);
            k_sort_place<<<nb, 256, 0, s>>>(e, k, i, 8 * p, hist, w.n_blocks, keys[to], perm[to]);
            last = to;
        }
    }
    SumArgs a{};
    a.keys = keys[last];
    a.perm = perm[last];
    a.n = e.n;
    a.vocab = e.vocab;
    a.dim = e.dim;
    a.ld = ld;
    a.chunk = w.chunk;
    a.n_chunks = w.n_chunks;
    a.dout = dout;
    a.dw = dw;
    a.parts = reinterpret_cast<float *>(base + w.parts);
    a.scale = e.scale;
    a.accumulate = accumulate;
    return by_type(dtype, [&](auto t) {
        typedef decltype(t) T;
        constexpr int N = Pack16<T>::N;
        const bool wide = e.dim % N == 0 && ld % N == 0 && at16(dout) && at16(dw);
        a.per = (int32_t)(wide ? e.dim / N : e.dim);
        over_rows(a.n_chunks, a.per, [&](uint32_t nb, int64_t r, int64_t end) {
            if (wide)
                k_embed_sum<T, N><<<nb, 256, 0, s>>>(a, r, end);
            else
                k_embed_sum<T, 1><<<nb, 256, 0, s>>>(a, r, end);
        });
        if (a.n_chunks > 1)
            over_rows(a.n_chunks, a.per, [&](uint32_t nb, int64_t r, int64_t end) {
                if (wide)
                    k_embed_join<T, N><<<nb, 256, 0, s>>>(a, r, end);
                else
                    k_embed_join<T, 1><<<nb, 256, 0, s>>>(a, r, end);
            });
    });
}

}  // namespace ops
}  // namespace z1

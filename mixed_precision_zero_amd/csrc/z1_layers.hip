// z1_layers.hip -- the elementwise layers: dropout, the gradient through
// z1_linear's epilogue, and norm and rotation of queries and keys with their
// gradients.
#include "z1_layers_internal.h"

namespace z1 {
namespace ops {
namespace {

// --------------------------------------------------------------------------
// Walks the blocks of eight columns of a matrix, row after row, a grid apart:
// one division at the start, then sums.
// --------------------------------------------------------------------------
struct Walk {
    int64_t row, rows;
    uint32_t block, blocks;
    int64_t row_step;
    uint32_t block_step;
    __device__ __forceinline__ Walk(int64_t rows_, int64_t cols)
        : rows(rows_), blocks((uint32_t)((cols + 7) / 8))
    {
        const uint64_t first = blockIdx.x * 256ull + threadIdx.x, step = gridDim.x * 256ull;
        row = (int64_t)(first / blocks);
        block = (uint32_t)(first % blocks);
        row_step = (int64_t)(step / blocks);
        block_step = (uint32_t)(step % blocks);
    }
    __device__ __forceinline__ bool here() const { return row < rows; }
    __device__ __forceinline__ void next()
    {
        row += row_step;
        block += block_step;
        if (block >= blocks) {
            block -= blocks;
            ++row;
        }
    }
};

template <typename T>
__device__ __forceinline__ void get8(const void *p, int64_t at, int64_t n, float (&v)[8])
{
    const typename T::store *from = static_cast<const typename T::store *>(p) + at;
    if (n >= 8)
        Eight<T>::load(from, v);
    else
        Eight<T>::load_some(from, v, (int)n);
}
template <typename T>
__device__ __forceinline__ void set8(void *p, int64_t at, int64_t n, const float (&v)[8])
{
    typename T::store *to = static_cast<typename T::store *>(p) + at;
    if (n >= 8)
        Eight<T>::store(to, v);
    else
        Eight<T>::store_some(to, v, (int)n);
}

template <typename T>
__global__ __launch_bounds__(256) void k_dropout(z1_dropout_args a, Drop d)
{
    const DropKey key = drop_key(d);
    for (Walk w(a.rows, a.cols); w.here(); w.next()) {
        const int64_t c = (int64_t)w.block * 8, n = a.cols - c;
        float v[8], r[8];
        get8<T>(a.x, w.row * a.ld_x + c, n, v);
        if (a.residual)
            get8<T>(a.residual, w.row * a.ld_residual + c, n, r);
        if (key.on)
            drop8(key, w.block, (uint32_t)w.row, v);
        if (a.residual)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] += r[j];
        set8<T>(a.y, w.row * a.ld_y + c, n, v);
    }
}

// --------------------------------------------------------------------------
// The gradient through the epilogue.  A workgroup takes a piece of the rows of 8 * LX
// columns: LX lanes of eight columns, 256 / LX of rows; the column sums of its piece go
// to a row of `parts`, which k_join adds up.  The pieces are as small as 1024 workgroups
// make them (2048 x 1536 with SILU and a product, bf16: 29 us in pieces of 64 rows, 192
// workgroups; 9.8 in pieces of 16: 31 MB at 3.2 TB/s, at which size the launch is half
// of it).
// --------------------------------------------------------------------------
template <typename T, int LX>
__global__ __launch_bounds__(256) void k_linear_dz(z1_linear_dz_args a, Drop d, float *parts, int64_t piece)
{
    constexpr int RX = 256 / LX;
    __shared__ float lds[RX][LX * 8];
    const int cx = threadIdx.x % LX, rx = threadIdx.x / LX;
    const int64_t c = blockIdx.x * (LX * 8ll) + cx * 8, n = a.out - c;
    const int64_t r0 = blockIdx.y * piece, end = min(a.rows, r0 + piece);
    const DropKey key = drop_key(d);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
        for (int64_t r = r0 + rx; r < end; r += RX) {
            float g[8], z[8] = {}, m[8] = {};
            get8<T>(a.dy, r * a.ld_dy + c, n, g);
            if (a.pre)
                get8<T>(a.pre, r * a.ld_pre + c, n, z);
            if (a.mul)
                get8<T>(a.mul, r * a.ld_mul + c, n, m);
            if (key.on) {
                // z and m too where dropped, as they may not be finite there
                uint32_t w[4];
                philox(key, (uint32_t)(c >> 3), (uint32_t)r, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool kept = drop_keeps(key, w, j);
                    g[j] = kept ? g[j] * key.scale : 0.f;
                    z[j] = kept ? z[j] : 0.f;
                    m[j] = kept ? m[j] : 0.f;
                }
            }
            float value[8], slope[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                value[j] = z[j];
                slope[j] = 1.f;
            }
            with_act(a.act, [&](auto k) {   // together: they share most of their work
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    value[j] = act_value<decltype(k)::value>(z[j], above_low(z[j]));
                    slope[j] = act_slope<decltype(k)::value>(z[j]);
                }
            });
            if (a.dmul) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    value[j] *= g[j];
                set8<T>(a.dmul, r * a.ld_dmul + c, n, value);
            }
            if (a.mul)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    g[j] *= m[j];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g[j] *= slope[j];
            if (a.dz)
                set8<T>(a.dz, r * a.ld_dz + c, n, g);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[j] += g[j];
        }
    }
    if (!a.dbias)
        return;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        lds[rx][cx * 8 + j] = sum[j];
    __syncthreads();
    const int64_t col = blockIdx.x * (LX * 8ll) + threadIdx.x;
    if (threadIdx.x < LX * 8 && col < a.out) {
        float s = lds[0][threadIdx.x];
#pragma unroll
        for (int q = 1; q < RX; ++q)
            s += lds[q][threadIdx.x];
        parts[blockIdx.y * a.out + col] = s;
    }
}

template <typename T>
void dz_run(const z1_linear_dz_args &a, const Drop &d, float *parts, hipStream_t s)
{
    const int64_t piece = dz_piece(a.rows, a.out);
    const int lanes = dz_lanes(a.out);
    const dim3 grid((uint32_t)((a.out + lanes * 8 - 1) / (lanes * 8)), (uint32_t)((a.rows + piece - 1) / piece));
    if (lanes == 8)
        k_linear_dz<T, 8><<<grid, 256, 0, s>>>(a, d, parts, piece);
    else if (lanes == 16)
        k_linear_dz<T, 16><<<grid, 256, 0, s>>>(a, d, parts, piece);
    else
        k_linear_dz<T, 32><<<grid, 256, 0, s>>>(a, d, parts, piece);
}

// out[c] (+)= the sum of rows of parts: 64 columns x 16 lanes of rows a
// workgroup, the lanes' sums added in order.
__global__ __launch_bounds__(1024) void k_join(const float *parts, int64_t rows, int64_t cols, int64_t ld, float *out,
                                               int32_t accumulate)
{
    __shared__ float lds[16][64];
    const int cx = threadIdx.x & 63, rx = threadIdx.x >> 6;
    const int64_t c = blockIdx.x * 64ll + cx;
    float s = 0.f;
    if (c < cols)
#pragma unroll 8
        for (int64_t r = rx; r < rows; r += 16)
            s += parts[r * ld + c];
    lds[rx][cx] = s;
    __syncthreads();
    if (rx == 0 && c < cols) {
#pragma unroll
        for (int q = 1; q < 16; ++q)
            s += lds[q][cx];
        out[c] = accumulate ? out[c] + s : s;
    }
}

// --------------------------------------------------------------------------
// Norm and rotation of queries and keys.
//
// `lanes` lanes hold a head, 2 V elements each: lane j the pairs j V .. of the
// rotated part (V first and V second elements), the lanes behind them the rest
// of the head, 2 V elements in a row, which are turned by no angle.  A wave
// takes 64 / lanes heads of one token at a time, and the sums over a head are
// over its lanes.  The token's cosines and sines are computed once, one
// frequency a lane, and passed through LDS to the lanes that need them.
//
// VEC: rows of 16-byte aligned chunks of V = 16 bytes; else V = 8 elements one
// by one, at any dim, alignment and distance.
// --------------------------------------------------------------------------
template <typename T, bool VEC, bool INTER>
struct Head {
    typedef typename T::store store;
    static constexpr int V = VEC ? 16 / (int)sizeof(store) : 8;

    int32_t a, b;        // first elements of the lane's two runs
    int32_t na, nb;      // how many of them there are
    int32_t j;           // the lane's chunk
    bool pairs;          // of the rotated part

    static __host__ __device__ int chunks(int32_t dim, int32_t n_freq)
    {
        return (n_freq + V - 1) / V + (dim - 2 * n_freq + 2 * V - 1) / (2 * V);
    }

    __device__ __forceinline__ Head(int32_t dim, int32_t n_freq, int j_) : j(j_)
    {
        const int cp = (n_freq + V - 1) / V;
        pairs = j < cp;
        if (pairs) {
            na = nb = min(V, n_freq - j * V);
            a = INTER ? 2 * V * j : V * j;
            b = INTER ? a + V : n_freq + V * j;
        } else {
            a = 2 * n_freq + 2 * V * (j - cp);
            b = a + V;
            na = max(0, min(V, dim - a));
            nb = max(0, min(V, dim - b));
        }
    }

    // Element i of the first (0) or second run, as the head numbers it, or -1.
    __device__ __forceinline__ int32_t index(int which, int i) const
    {
        if (pairs)
            return i < na ? (INTER ? a + 2 * i + which : (which ? b : a) + i) : -1;
        if (INTER) {
            const int m = 2 * i + which;
            return m < na + nb ? a + m : -1;
        }
        return i < (which ? nb : na) ? (which ? b : a) + i : -1;
    }

    // A lane's elements as they lie in memory, and as numbers: apart, so that the
    // next head's can be on their way while one is worked on.
    struct Raw {
        union {
            Pack16<T> run[2];           // VEC
            store e[2][V];
        };
    };
    __device__ __forceinline__ void fetch(const void *head, Raw &r) const
    {
        const store *p = static_cast<const store *>(head);
        if (VEC) {
            r.run[0].raw = r.run[1].raw = uint4v{0u, 0u, 0u, 0u};
            if (na > 0)
                r.run[0].raw = *reinterpret_cast<const uint4v *>(p + a);
            if (nb > 0)
                r.run[1].raw = *reinterpret_cast<const uint4v *>(p + b);
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int32_t e = index(w, i);
                    r.e[w][i] = e >= 0 ? p[e] : T::down(0.f);
                }
        }
    }
    static __device__ __forceinline__ void values(const Raw &r, float (&x)[2][V])
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int m = VEC && INTER ? 2 * i + w : w * V + i;
                x[w][i] = T::up(r.e[m / V][m % V]);
            }
    }

    __device__ __forceinline__ void store_to(void *head, const float (&x)[2][V]) const
    {
        store *p = static_cast<store *>(head);
        if (VEC) {
            Pack16<T> lo, hi;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int m = INTER ? 2 * i + w : w * V + i;
                    (m < V ? lo : hi).e[m % V] = T::down(x[w][i]);
                }
            if (na > 0)
                *reinterpret_cast<uint4v *>(p + a) = lo.raw;
            if (nb > 0)
                *reinterpret_cast<uint4v *>(p + b) = hi.raw;
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int32_t e = index(w, i);
                    if (e >= 0)
                        p[e] = T::down(x[w][i]);
                }
        }
    }
};

constexpr int kQkWaves = 4;
constexpr int kMostFreq = 256;

struct QkShape {
    int32_t lanes;           // of a head: a power of two
    int32_t groups[2];       // of heads that a wave takes at once: queries, keys
    int32_t parts[2];        // waves that share the groups of a token; forward: [0], of both kinds
    uint32_t blocks[2];      // workgroups; forward: [0]
};

__device__ __forceinline__ int64_t position_of(const z1_qk_args &a, int64_t t)
{
    return a.position_type == Z1_I32 ? (int64_t)static_cast<const int32_t *>(a.positions)[t]
                                     : static_cast<const int64_t *>(a.positions)[t];
}

// The token's (cos, sin) of every frequency into the wave's LDS.  The angle in binary64 is
// reduced to a part of a turn with 1 / (2 pi) in two parts and the product's own rounding,
// so that the part is exact to fp32 up to angles of 2^53.
__device__ __forceinline__ void put_turns(const z1_qk_args &a, int64_t t, float2 *lds, int lane)
{
    const double pos = (double)position_of(a, t);
    asm volatile("" ::: "memory");
    for (int f = lane; f < a.n_freq; f += 64) {
        const double angle = pos * a.inv_freq[f], turn = angle * 0.15915494309189535;
        const double rest = fma(angle, -9.839338337591243e-18, fma(angle, 0.15915494309189535, -turn));
        float s, c;
        sincospif((float)((turn - rint(turn)) + rest) * 2.f, &s, &c);
        lds[f] = make_float2(c, s);
    }
    // one wave's LDS accesses take place in order
    asm volatile("" ::: "memory");
}

// (cos, sin) of the lane's i-th pair.
template <int V>
__device__ __forceinline__ float2 turn_of(const z1_qk_args &a, const float2 *lds, int j, bool pairs, int i)
{
    return pairs && j * V + i < a.n_freq ? lds[j * V + i] : make_float2(1.f, 0.f);
}

template <int CTRL>
__device__ __forceinline__ float plus_lane(float x)
{
    return x + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// The sum over a head's lanes, in all of them: lanes 1 and 2 apart by permutations of
// four, then mirrors of 8 and 16.
__device__ __forceinline__ float lane_sum(float x, int lanes)
{
    if (lanes > 1)
        x = plus_lane<0xb1>(x);
    if (lanes > 2)
        x = plus_lane<0x4e>(x);
    if (lanes > 4)
        x = plus_lane<0x141>(x);
    if (lanes > 8)
        x = plus_lane<0x140>(x);
    if (lanes > 16)
        x += __shfl_xor(x, 16);
    if (lanes > 32)
        x += __shfl_xor(x, 32);
    return x;
}

// A wave's walk over (token, group of heads).
struct QkWalk {
    int64_t unit, units, step, t;
    int32_t parts, groups, g;
    bool fresh;              // of a token
    __device__ __forceinline__ QkWalk(int64_t first, int64_t step_, int64_t tokens, int32_t parts_, int32_t groups_)
        : unit(first), units(tokens * parts_), step(step_), parts(parts_), groups(groups_), fresh(true)
    {
        t = unit / parts;
        g = (int32_t)(unit % parts);
    }
    __device__ __forceinline__ bool here() const { return unit < units; }
    __device__ __forceinline__ void next()
    {
        g += parts;
        fresh = g >= groups;
        if (fresh) {
            unit += step;
            t = unit / parts;
            g = (int32_t)(unit % parts);
        }
    }
};

template <typename T>
__device__ __forceinline__ const typename T::store *head_at(const void *p, int64_t token, int64_t head, int64_t t, int64_t h)
{
    return static_cast<const typename T::store *>(p) + t * token + h * head;
}

// The next group's elements are on their way while one is worked on, and one token's turns
// stay in registers (8192 tokens of 32 + 32 heads of 128, bf16: 49 us, 5.4 TB/s; 52 without).
template <typename T, bool VEC, bool INTER>
__global__ __launch_bounds__(64 * kQkWaves) void k_qk(z1_qk_args a, QkShape sh)
{
    typedef Head<T, VEC, INTER> H;
    constexpr int V = H::V;
    __shared__ float2 lds[kQkWaves][kMostFreq];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane / sh.lanes, across = 64 / sh.lanes;
    const H h(a.dim, a.n_freq, lane % sh.lanes);
    const float per = 1.f / (float)a.dim, eps = (float)a.eps;
    typename H::Raw weight[2], raw{};
    if (a.q.weight)
        h.fetch(a.q.weight, weight[0]);
    if (a.k.weight)
        h.fetch(a.k.weight, weight[1]);
    QkWalk w((int64_t)blockIdx.x * kQkWaves + wave, (int64_t)gridDim.x * kQkWaves, a.tokens, sh.parts[0],
             sh.groups[0] + sh.groups[1]);
    const auto fetch = [&] {
        const bool is_k = w.g >= sh.groups[0];
        const z1_heads &k = is_k ? a.k : a.q;
        const int64_t head = (int64_t)(w.g - (is_k ? sh.groups[0] : 0)) * across + sub;
        if (head < k.heads)
            h.fetch(head_at<T>(k.x, k.x_token, k.x_head, w.t, head), raw);
        else
            raw = typename H::Raw{};
    };
    if (!w.here())
        return;
    fetch();
    float cs[V], sn[V];
    while (true) {
        if (w.fresh) {
            put_turns(a, w.t, lds[wave], lane);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 turn = turn_of<V>(a, lds[wave], h.j, h.pairs, i);
                cs[i] = turn.x;
                sn[i] = turn.y;
            }
        }
        float x[2][V];
        H::values(raw, x);
        const bool is_k = w.g >= sh.groups[0];
        const z1_heads &k = is_k ? a.k : a.q;
        const int64_t head = (int64_t)(w.g - (is_k ? sh.groups[0] : 0)) * across + sub, t = w.t;
        w.next();
        const bool more = w.here();
        if (more)
            fetch();
        if (k.weight) {
            float s = 0.f, m[2][V];
            H::values(is_k ? weight[1] : weight[0], m);
#pragma unroll
            for (int i = 0; i < V; ++i)
                s = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], s));
            const float inv = rsqrtf(fmaf(lane_sum(s, sh.lanes), per, eps));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[0][i] *= inv * m[0][i];
                x[1][i] *= inv * m[1][i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = x[0][i], q = x[1][i];
            x[0][i] = fmaf(p, cs[i], -(q * sn[i]));
            x[1][i] = fmaf(q, cs[i], p * sn[i]);
        }
        if (head < k.heads)
            h.store_to(const_cast<typename T::store *>(head_at<T>(k.out, k.out_token, k.out_head, t, head)), x);
        if (!more)
            return;
    }
}

// The gradient.  With g the output's gradient turned back, xh = x / norm:
//   dw = sum g xh,   dx = (g w - xh mean(g w xh)) / norm
// both means from one pass over the head.  A workgroup takes queries or keys alone, so
// that a wave holds one weight and one dw, and takes cosines and sines from LDS each
// time: four waves a SIMD, all 1024 workgroups at once.  8192 tokens of 32 + 32 heads of
// 128, bf16: 91 us, 50 without norm; with the turns in registers and the next heads'
// elements fetched ahead, three waves a SIMD, 91 and 59; with both weights in every wave,
// two a SIMD, 108 and 67.  Memory bounds it without norm (268 MB at 5.4 TB/s); with norm
// 402 MB at 4.5 TB/s, then the join, with the lanes' sums between.
template <typename T, bool VEC, bool INTER>
__global__ __launch_bounds__(64 * kQkWaves) void k_qk_grad(z1_qk_args a, QkShape sh, float *parts)
{
    typedef Head<T, VEC, INTER> H;
    constexpr int V = H::V;
    __shared__ float2 lds[kQkWaves][kMostFreq];
    __shared__ float sums[kQkWaves][512];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane / sh.lanes, across = 64 / sh.lanes;
    const int is_k = blockIdx.x >= sh.blocks[0];
    const z1_heads &k = is_k ? a.k : a.q;
    const uint32_t block = blockIdx.x - (is_k ? sh.blocks[0] : 0);
    const H h(a.dim, a.n_freq, lane % sh.lanes);
    const float per = 1.f / (float)a.dim, eps = (float)a.eps;
    float dw[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        dw[0][i] = dw[1][i] = 0.f;
    typename H::Raw weight{};
    const bool norm = k.weight != nullptr;
    if (norm)
        h.fetch(k.weight, weight);
    for (QkWalk w((int64_t)block * kQkWaves + wave, (int64_t)sh.blocks[is_k] * kQkWaves, a.tokens, sh.parts[is_k],
                  sh.groups[is_k]);
         w.here(); w.next()) {
        const int64_t head = (int64_t)w.g * across + sub;
        const bool there = head < k.heads;
        typename H::Raw rx{}, rd{};
        if (there) {
            h.fetch(head_at<T>(k.dout, k.dout_token, k.dout_head, w.t, head), rd);
            if (norm)
                h.fetch(head_at<T>(k.x, k.x_token, k.x_head, w.t, head), rx);
        }
        if (w.fresh)
            put_turns(a, w.t, lds[wave], lane);
        float x[2][V], d[2][V];
        H::values(rd, d);
        H::values(rx, x);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 turn = turn_of<V>(a, lds[wave], h.j, h.pairs, i);
            const float p = d[0][i], q = d[1][i];
            d[0][i] = fmaf(p, turn.x, q * turn.y);
            d[1][i] = fmaf(q, turn.x, -(p * turn.y));
        }
        if (norm) {
            float s = 0.f, m = 0.f, g[2][V];
            H::values(weight, g);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[q][i] *= d[q][i];
                    s = fmaf(x[q][i], x[q][i], s);
                    m = fmaf(g[q][i], x[q][i], m);
                }
            // a head that is not there has no norm either (eps may be 0)
            const float inv = there ? rsqrtf(fmaf(lane_sum(s, sh.lanes), per, eps)) : 0.f;
            const float pull = lane_sum(m, sh.lanes) * per * inv * inv * inv;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dw[q][i] = fmaf(d[q][i], x[q][i] * inv, dw[q][i]);
                    d[q][i] = fmaf(-x[q][i], pull, g[q][i] * inv);
                }
        }
        if (there)
            h.store_to(const_cast<typename T::store *>(head_at<T>(k.out, k.out_token, k.out_head, w.t, head)), d);
    }
    if (!parts)
        return;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float x = dw[q][i];
            for (int o = sh.lanes; o < 64; o <<= 1)
                x += __shfl_xor(x, o);
            const int32_t e = h.index(q, i);
            if (sub == 0 && e >= 0)
                sums[wave][e] = x;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < a.dim; e += 64 * kQkWaves) {
        float s = sums[0][e];
#pragma unroll
        for (int w2 = 1; w2 < kQkWaves; ++w2)
            s += sums[w2][e];
        parts[(int64_t)blockIdx.x * a.dim + e] = s;
    }
}

// Either dweight (+)= the sum of its workgroups' rows of parts: as k_join, blockIdx.y 0
// for queries and 1 for keys.
__global__ __launch_bounds__(1024) void k_qk_join(const float *parts, z1_qk_args a, QkShape sh)
{
    __shared__ float lds[16][64];
    const int cx = threadIdx.x & 63, rx = threadIdx.x >> 6, is_k = blockIdx.y;
    float *out = is_k ? a.k.dweight : a.q.dweight;
    if (!out)
        return;
    const float *from = parts + (is_k ? (int64_t)sh.blocks[0] * a.dim : 0);
    const int64_t c = blockIdx.x * 64ll + cx;
    float s = 0.f;
    if (c < a.dim)
#pragma unroll 8
        for (uint32_t r = rx; r < sh.blocks[is_k]; r += 16)
            s += from[(int64_t)r * a.dim + c];
    lds[rx][cx] = s;
    __syncthreads();
    if (rx == 0 && c < a.dim) {
#pragma unroll
        for (int q = 1; q < 16; ++q)
            s += lds[q][cx];
        out[c] = a.accumulate ? out[c] + s : s;
    }
}

uint32_t grid_for(int64_t items) { return (uint32_t)std::min<int64_t>((items + 255) / 256, 4096); }

bool mult16(const void *p, int64_t a, int64_t b, int64_t size)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a * size % 16 == 0 && b * size % 16 == 0;
}

template <typename T>
bool qk_vec(const z1_qk_args &a, bool grad)
{
    constexpr int64_t size = sizeof(typename T::store);
    constexpr int V = 16 / (int)size;
    if (a.dim % V || a.n_freq % V)
        return false;
    for (const z1_heads *k : {&a.q, &a.k}) {
        if (k->heads == 0)
            continue;
        if (!mult16(k->out, k->out_token, k->out_head, size) || reinterpret_cast<uintptr_t>(k->weight) % 16)
            return false;
        if ((!grad || k->weight) && !mult16(k->x, k->x_token, k->x_head, size))
            return false;
        if (grad && !mult16(k->dout, k->dout_token, k->dout_head, size))
            return false;
    }
    return true;
}

QkShape qk_shape(const z1_qk_args &a, int chunks, bool grad)
{
    QkShape s{};
    s.lanes = 1;
    while (s.lanes < chunks)
        s.lanes <<= 1;
    const int64_t across = 64 / s.lanes;
    const int64_t heads[2] = {a.q.heads, a.k.heads};
    for (int i = 0; i < 2; ++i)
        s.groups[i] = (int32_t)((heads[i] + across - 1) / across);
    // few tokens: several waves share one, down to one group of heads each
    const int64_t most = 2048 / std::max<int64_t>(1, a.tokens);
    const auto parts = [&](int64_t groups) { return (int32_t)std::max<int64_t>(1, std::min<int64_t>(groups, most)); };
    if (!grad) {
        s.parts[0] = parts(s.groups[0] + s.groups[1]);
        s.blocks[0] = (uint32_t)std::min<int64_t>(8192, (a.tokens * s.parts[0] + kQkWaves - 1) / kQkWaves);
        return s;
    }
    for (int i = 0; i < 2; ++i) {
        s.parts[i] = parts(s.groups[i]);
        s.blocks[i] = (uint32_t)qk_grad_groups(a.tokens, a.q.heads, a.k.heads, i);
    }
    return s;
}

template <typename T, bool VEC, bool INTER>
hipError_t qk_run(const z1_qk_args &a, float *parts, bool grad, hipStream_t s)
{
    const QkShape sh = qk_shape(a, Head<T, VEC, INTER>::chunks(a.dim, a.n_freq), grad);
    if (!grad) {
        k_qk<T, VEC, INTER><<<sh.blocks[0], 64 * kQkWaves, 0, s>>>(a, sh);
    } else {
        if (sh.blocks[0] + sh.blocks[1] > 0)
            k_qk_grad<T, VEC, INTER><<<sh.blocks[0] + sh.blocks[1], 64 * kQkWaves, 0, s>>>(a, sh, parts);
        if (a.q.dweight || a.k.dweight)   // of no tokens: written as zeros from no parts
            k_qk_join<<<dim3((uint32_t)((a.dim + 63) / 64), 2), 1024, 0, s>>>(parts, a, sh);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t qk_typed(const z1_qk_args &a, float *parts, bool grad, hipStream_t s)
{
    if (qk_vec<T>(a, grad))
        return a.interleaved ? qk_run<T, true, true>(a, parts, grad, s) : qk_run<T, true, false>(a, parts, grad, s);
    return a.interleaved ? qk_run<T, false, true>(a, parts, grad, s) : qk_run<T, false, false>(a, parts, grad, s);
}

hipError_t qk_any(const z1_qk_args &a, float *parts, bool grad, hipStream_t s)
{
    switch (a.dtype) {
    case Z1_F32: return qk_typed<F32>(a, parts, grad, s);
    case Z1_BF16: return qk_typed<BF16>(a, parts, grad, s);
    default: return qk_typed<F16>(a, parts, grad, s);
    }
}

}  // namespace

hipError_t launch_dropout(const z1_dropout_args &a, const Drop &d, hipStream_t s)
{
    const int64_t items = a.rows * ((a.cols + 7) / 8);
    if (items == 0)
        return hipSuccess;
    switch (a.dtype) {
    case Z1_F32: k_dropout<F32><<<grid_for(items), 256, 0, s>>>(a, d); break;
    case Z1_BF16: k_dropout<BF16><<<grid_for(items), 256, 0, s>>>(a, d); break;
    default: k_dropout<F16><<<grid_for(items), 256, 0, s>>>(a, d); break;
    }
    return hipGetLastError();
}

hipError_t launch_linear_dz(const z1_linear_dz_args &a, const Drop &d, float *parts, hipStream_t s)
{
    const int64_t piece = dz_piece(a.rows, a.out), pieces = (a.rows + piece - 1) / piece;
    if (pieces > 0) {
        switch (a.dtype) {
        case Z1_F32: dz_run<F32>(a, d, parts, s); break;
        case Z1_BF16: dz_run<BF16>(a, d, parts, s); break;
        default: dz_run<F16>(a, d, parts, s); break;
        }
    }
    if (a.dbias && (pieces > 0 || !a.accumulate))
        k_join<<<(uint32_t)((a.out + 63) / 64), 1024, 0, s>>>(parts, pieces, a.out, a.out, a.dbias, a.accumulate);
    return hipGetLastError();
}

int64_t qk_grad_groups(int64_t tokens, int64_t q_heads, int64_t k_heads, int kind)
{
    // enough waves for every token, and for few tokens' heads, up to four workgroups a
    // compute unit, shared out by the heads
    const int64_t heads = kind ? k_heads : q_heads, both = q_heads + k_heads;
    if (heads == 0 || tokens == 0)
        return 0;
    const int64_t wanted = (tokens * std::min<int64_t>(heads, 64) + kQkWaves - 1) / kQkWaves;
    return std::max<int64_t>(1, std::min<int64_t>(1024 * heads / both, wanted));
}

hipError_t launch_qk(const z1_qk_args &a, hipStream_t s)
{
    return a.tokens * (a.q.heads + a.k.heads) == 0 ? hipSuccess : qk_any(a, nullptr, false, s);
}

hipError_t launch_qk_grad(const z1_qk_args &a, float *parts, hipStream_t s) { return qk_any(a, parts, true, s); }

}  // namespace ops
}  // namespace z1

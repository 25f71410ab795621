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
// workgroups; X in pieces of 16).
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
            float g[8], z[8], m[8];
            get8<T>(a.dy, r * a.ld_dy + c, n, g);
            if (a.pre)
                get8<T>(a.pre, r * a.ld_pre + c, n, z);
            if (a.mul)
                get8<T>(a.mul, r * a.ld_mul + c, n, m);
            if (key.on)
                drop8(key, (uint32_t)(c >> 3), (uint32_t)r, g);
            if (a.dmul) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = z[j];
                act_values(a.act, o);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] *= g[j];
                set8<T>(a.dmul, r * a.ld_dmul + c, n, o);
            }
            if (a.mul)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    g[j] *= m[j];
            with_act(a.act, [&](auto k) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    g[j] *= act_slope<decltype(k)::value>(z[j]);
            });
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

    __device__ __forceinline__ void load(const void *head, float (&x)[2][V]) const
    {
        const store *p = static_cast<const store *>(head);
        if (VEC) {
            Pack16<T> lo, hi;
            lo.raw = hi.raw = uint4v{0u, 0u, 0u, 0u};
            if (na > 0)
                lo.raw = *reinterpret_cast<const uint4v *>(p + a);
            if (nb > 0)
                hi.raw = *reinterpret_cast<const uint4v *>(p + b);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int m = INTER ? 2 * i + w : w * V + i;
                    x[w][i] = T::up(m < V ? lo.e[m % V] : hi.e[m % V]);
                }
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int32_t e = index(w, i);
                    x[w][i] = e >= 0 ? T::up(p[e]) : 0.f;
                }
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
    int32_t lanes;        // of a head: a power of two
    int32_t parts;        // a token's heads are shared out over so many waves
    int64_t units;        // tokens * parts
};

__device__ __forceinline__ int64_t position_of(const z1_qk_args &a, int64_t t)
{
    return a.position_type == Z1_I32 ? (int64_t)static_cast<const int32_t *>(a.positions)[t]
                                     : static_cast<const int64_t *>(a.positions)[t];
}

// The token's (cos, sin) of every frequency into the wave's LDS, and this lane's
// V of them out of it.  The angle is reduced to a part of a turn in binary64.
template <int V>
__device__ __forceinline__ void turns(const z1_qk_args &a, int64_t t, float2 *lds, int lane, int j, bool pairs,
                                      float (&cs)[V], float (&sn)[V])
{
    const double pos = (double)position_of(a, t);
    asm volatile("" ::: "memory");
    for (int f = lane; f < a.n_freq; f += 64) {
        const double turn = pos * a.inv_freq[f] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(turn - rint(turn)) * 2.f, &s, &c);
        lds[f] = make_float2(c, s);
    }
    // one wave's LDS accesses take place in order
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool there = pairs && j * V + i < a.n_freq;
        const float2 v = there ? lds[j * V + i] : make_float2(1.f, 0.f);
        cs[i] = v.x;
        sn[i] = v.y;
    }
}

__device__ __forceinline__ float lane_sum(float x, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1)
        x += __shfl_xor(x, o);
    return x;
}

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
    float wq[2][V], wk[2][V];
    if (a.q.weight)
        h.load(a.q.weight, wq);
    if (a.k.weight)
        h.load(a.k.weight, wk);
    const int64_t q_groups = (a.q.heads + across - 1) / across;
    for (int64_t unit = (int64_t)blockIdx.x * kQkWaves + wave; unit < sh.units; unit += (int64_t)gridDim.x * kQkWaves) {
        const int64_t t = unit / sh.parts;
        const int part = (int)(unit % sh.parts);
        float cs[V], sn[V];
        turns<V>(a, t, lds[wave], lane, h.j, h.pairs, cs, sn);
        const auto kind = [&](const z1_heads &k, const float (&w)[2][V], int64_t first) {
            for (int64_t g = first; g * across < k.heads; g += sh.parts) {
                const int64_t head = g * across + sub;
                const bool there = head < k.heads;
                float x[2][V];
                if (there)
                    h.load(static_cast<const typename T::store *>(k.x) + t * k.x_token + head * k.x_head, x);
                else
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        x[0][i] = x[1][i] = 0.f;
                if (k.weight) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        s = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], s));
                    s = lane_sum(s, sh.lanes);
                    const float inv = rsqrtf(s / (float)a.dim + (float)a.eps);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        x[0][i] *= inv * w[0][i];
                        x[1][i] *= inv * w[1][i];
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float p = x[0][i], q = x[1][i];
                    x[0][i] = p * cs[i] - q * sn[i];
                    x[1][i] = q * cs[i] + p * sn[i];
                }
                if (there)
                    h.store_to(static_cast<typename T::store *>(k.out) + t * k.out_token + head * k.out_head, x);
            }
        };
        kind(a.q, wq, part);
        // the keys' groups go on where the queries' end
        kind(a.k, wk, (part + sh.parts - q_groups % sh.parts) % sh.parts);
    }
}

// The gradient.  With g the output's gradient turned back, xh = x / norm:
//   dw = sum g xh,   dx = (g w - xh mean(g w xh)) / norm
// both means from one pass over the head.  The waves walk the tokens a grid
// apart and keep dw in registers.
template <typename T, bool VEC, bool INTER>
__global__ __launch_bounds__(64 * kQkWaves) void k_qk_grad(z1_qk_args a, QkShape sh, float *parts)
{
    typedef Head<T, VEC, INTER> H;
    constexpr int V = H::V;
    __shared__ float2 lds[kQkWaves][kMostFreq];
    __shared__ float sums[kQkWaves][2][512];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane / sh.lanes, across = 64 / sh.lanes;
    const H h(a.dim, a.n_freq, lane % sh.lanes);
    float wq[2][V], wk[2][V], dq[2][V], dk[2][V];
    if (a.q.weight)
        h.load(a.q.weight, wq);
    if (a.k.weight)
        h.load(a.k.weight, wk);
#pragma unroll
    for (int i = 0; i < V; ++i)
        dq[0][i] = dq[1][i] = dk[0][i] = dk[1][i] = 0.f;
    const int64_t q_groups = (a.q.heads + across - 1) / across;
    for (int64_t unit = (int64_t)blockIdx.x * kQkWaves + wave; unit < sh.units; unit += (int64_t)gridDim.x * kQkWaves) {
        const int64_t t = unit / sh.parts;
        const int part = (int)(unit % sh.parts);
        float cs[V], sn[V];
        turns<V>(a, t, lds[wave], lane, h.j, h.pairs, cs, sn);
        const auto kind = [&](const z1_heads &k, const float (&w)[2][V], float (&dw)[2][V], int64_t first) {
            for (int64_t g = first; g * across < k.heads; g += sh.parts) {
                const int64_t head = g * across + sub;
                const bool there = head < k.heads;
                float x[2][V], d[2][V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    x[0][i] = x[1][i] = d[0][i] = d[1][i] = 0.f;
                if (there) {
                    h.load(static_cast<const typename T::store *>(k.dout) + t * k.dout_token + head * k.dout_head, d);
                    if (k.weight)
                        h.load(static_cast<const typename T::store *>(k.x) + t * k.x_token + head * k.x_head, x);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float p = d[0][i], q = d[1][i];
                    d[0][i] = p * cs[i] + q * sn[i];
                    d[1][i] = q * cs[i] - p * sn[i];
                }
                if (k.weight) {
                    float s = 0.f, m = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], s));
                        m = fmaf(d[0][i] * w[0][i], x[0][i], fmaf(d[1][i] * w[1][i], x[1][i], m));
                    }
                    s = lane_sum(s, sh.lanes);
                    m = lane_sum(m, sh.lanes);
                    const float inv = rsqrtf(s / (float)a.dim + (float)a.eps);
                    const float mean = m * inv / (float)a.dim;
                    const bool counts = there;   // a head that is not there has no norm either (eps may be 0)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float xh = x[q][i] * inv;
                            if (counts)
                                dw[q][i] = fmaf(d[q][i], xh, dw[q][i]);
                            d[q][i] = inv * fmaf(-xh, mean, d[q][i] * w[q][i]);
                        }
                }
                if (there)
                    h.store_to(static_cast<typename T::store *>(k.out) + t * k.out_token + head * k.out_head, d);
            }
        };
        kind(a.q, wq, dq, part);
        kind(a.k, wk, dk, (part + sh.parts - q_groups % sh.parts) % sh.parts);
    }
    if (!parts)
        return;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float x = dq[q][i], y = dk[q][i];
            for (int o = sh.lanes; o < 64; o <<= 1) {
                x += __shfl_xor(x, o);
                y += __shfl_xor(y, o);
            }
            const int32_t e = h.index(q, i);
            if (sub == 0 && e >= 0) {
                sums[wave][0][e] = x;
                sums[wave][1][e] = y;
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += 64 * kQkWaves) {
        const int q = i / a.dim, e = i % a.dim;
        float s = sums[0][q][e];
#pragma unroll
        for (int w = 1; w < kQkWaves; ++w)
            s += sums[w][q][e];
        parts[(int64_t)blockIdx.x * 2 * a.dim + i] = s;
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

QkShape qk_shape(const z1_qk_args &a, int chunks)
{
    QkShape s{};
    s.lanes = 1;
    while (s.lanes < chunks)
        s.lanes <<= 1;
    const int64_t across = 64 / s.lanes;
    const int64_t groups = (a.q.heads + across - 1) / across + (a.k.heads + across - 1) / across;
    // few tokens: several waves share one, down to one group of heads each
    s.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>(groups, 2048 / std::max<int64_t>(1, a.tokens)));
    s.units = a.tokens * s.parts;
    return s;
}

template <typename T, bool VEC, bool INTER>
hipError_t qk_run(const z1_qk_args &a, float *parts, bool grad, hipStream_t s)
{
    const QkShape sh = qk_shape(a, Head<T, VEC, INTER>::chunks(a.dim, a.n_freq));
    const int64_t groups = qk_grad_groups(a.tokens, a.q.heads + a.k.heads);
    if (!grad)
        k_qk<T, VEC, INTER><<<(uint32_t)std::min<int64_t>(8192, (sh.units + kQkWaves - 1) / kQkWaves), 64 * kQkWaves, 0, s>>>(a, sh);
    else
        k_qk_grad<T, VEC, INTER><<<(uint32_t)groups, 64 * kQkWaves, 0, s>>>(a, sh, parts);
    if (grad && parts) {
        const uint32_t grid = (uint32_t)((a.dim + 63) / 64);
        if (a.q.dweight)
            k_join<<<grid, 1024, 0, s>>>(parts, groups, a.dim, 2 * a.dim, a.q.dweight, a.accumulate);
        if (a.k.dweight)
            k_join<<<grid, 1024, 0, s>>>(parts + a.dim, groups, a.dim, 2 * a.dim, a.k.dweight, a.accumulate);
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

int64_t qk_grad_groups(int64_t tokens, int64_t heads)
{
    // enough waves for every token, and for few tokens' heads, up to four
    // workgroups a compute unit
    return std::max<int64_t>(1, std::min<int64_t>(1024, (tokens * std::min<int64_t>(heads, 64) + kQkWaves - 1) / kQkWaves));
}

hipError_t launch_qk(const z1_qk_args &a, hipStream_t s)
{
    return a.tokens * (a.q.heads + a.k.heads) == 0 ? hipSuccess : qk_any(a, nullptr, false, s);
}

hipError_t launch_qk_grad(const z1_qk_args &a, float *parts, hipStream_t s) { return qk_any(a, parts, true, s); }

}  // namespace ops
}  // namespace z1

// z1_loss.hip -- log-probabilities of target tokens, the clipped policy loss
// and the preference loss, with their gradients in the logits.
//
// For a row x and target y, lse = log sum_v exp x_v and logp = x_y - lse;
// d logp / d x_v = 1[v == y] - exp(x_v - lse).  All of it is bound by the
// bytes of the logits, so each kernel reads a row once, 16 bytes a lane:
//   - z1_token_logprob and z1_policy_loss load a whole row into registers, so
//     all of its loads are in flight at once; each lane takes the maximum m
//     and the sum of exp(x - m) of what it holds, and the lanes' pairs are
//     joined in a fixed order (6144 x 32000 bf16: 59 us, 6.6 TB/s; streamed
//     four vectors at a time, 100).  A row too long for that is streamed with
//     a running maximum and a sum rescaled when it grows;
//   - z1_policy_loss's gradient needs nothing but the row itself, so it is
//     taken from the registers, and the logits cross memory once in and once
//     out, the gradient's stores past the caches (4096 x 49152 bf16: 142 us,
//     5.7 TB/s both ways; 157 with ordinary stores, 173 with 1024 lanes a row,
//     152 with 256);
//   - z1_logprob_grad is one pass from logits to gradient (6144 x 32000 bf16:
//     114 us, 6.9 TB/s, part of it from cache), and two for rows far from zero.
// Maxima, sums, log-probabilities and losses are fp32 or wider; the gradient
// is rounded once, to the logits' type.
#include "z1_ops_internal.h"

namespace z1 {
namespace ops {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();

// exp(x) through the hardware's 2^x; results below 2^-126 become 0.  The
// argument is rounded once, so a result is off by |x| 2^-24 of itself: 2e-6 for a
// probability of e^-30, nothing beside the rest of a sum.  Two more operations an
// element would mend it, where one more costs z1_policy_loss 1.4%.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Running maximum and sum of exponentials.  A maximum of -inf stands for "only
// -inf so far": its exponentials are taken from 0, so they are 0 and a NaN
// still shows.
struct Stat {
    float m, s;
    __device__ __forceinline__ float base() const { return m == -kInf ? 0.f : m; }
    __device__ __forceinline__ void raise(float to)
    {
        if (to > m) {
            s *= fast_exp(m - to);
            m = to;
        }
    }
    __device__ __forceinline__ void join(float m2, float s2)
    {
        const float to = fmaxf(m, m2);
        const float b = to == -kInf ? 0.f : to;
        s = s * fast_exp(m - b) + s2 * fast_exp(m2 - b);
        m = to;
    }
};

template <int NT>
__device__ __forceinline__ Stat block_stat(Stat a, float *lds)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float m2 = __shfl_xor(a.m, o), s2 = __shfl_xor(a.s, o);
        a.join(m2, s2);
    }
    if (NT > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            lds[2 * wave] = a.m;
            lds[2 * wave + 1] = a.s;
        }
        __syncthreads();
        a = Stat{lds[0], lds[1]};
#pragma unroll
        for (int w = 1; w < NT / 64; ++w)
            a.join(lds[2 * w], lds[2 * w + 1]);
    }
    return a;
}

__device__ __forceinline__ int64_t target_of(const Rows &r, int64_t row)
{
    return r.y32 ? (int64_t) static_cast<const int32_t *>(r.y)[row]
                 : static_cast<const int64_t *>(r.y)[row];
}

// A row cut for 16-byte loads: `head` elements up to the first 16-byte
// boundary, nvec whole vectors, `tail` elements.
template <typename T>
struct Cut {
    typedef typename T::store E;
    const E *x;
    E *d;
    int head, tail;
    int64_t nvec;
    bool d_vec;
    __device__ __forceinline__ Cut(const Rows &r, int64_t row)
    {
        x = static_cast<const E *>(r.x) + row * r.ld;
        d = r.d ? static_cast<E *>(r.d) + row * r.ld_d : nullptr;
        constexpr int N = Pack16<T>::N;
        const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(E));
        head = off ? N - off : 0;
        if (head > r.vocab)
            head = (int)r.vocab;
        nvec = (r.vocab - head) / N;
        tail = (int)(r.vocab - head - nvec * N);
        d_vec = r.d_vec;
    }
    // LAST: nothing reads these logits again, so the caches need not keep them
    template <bool LAST>
    __device__ __forceinline__ Pack16<T> load(int64_t v) const
    {
        const uint4v *at = reinterpret_cast<const uint4v *>(x + head + v * Pack16<T>::N);
        Pack16<T> p;
        p.raw = LAST ? __builtin_nontemporal_load(at) : *at;
        return p;
    }
    __device__ __forceinline__ void store(int64_t v, const Pack16<T> &p) const
    {
        E *at = d + head + v * Pack16<T>::N;
        if (d_vec)
            __builtin_nontemporal_store(p.raw, reinterpret_cast<uint4v *>(at));
        else
#pragma unroll
            for (int k = 0; k < Pack16<T>::N; ++k)
                at[k] = p.e[k];
    }
    // element index of this thread's head or tail element, -1 for none
    __device__ __forceinline__ int64_t edge(bool last) const
    {
        if (!last)
            return (int)threadIdx.x < head ? (int64_t)threadIdx.x : -1;
        return (int)threadIdx.x < tail ? head + nvec * Pack16<T>::N + threadIdx.x : -1;
    }
};

template <typename T>
__device__ __forceinline__ void add_vec(Stat &a, const Pack16<T> &p)
{
    constexpr int N = Pack16<T>::N;
    float f[N], top = -kInf;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        f[k] = T::up(p.e[k]);
        top = fmaxf(top, f[k]);
    }
    a.raise(top);
    const float b = a.base();
#pragma unroll
    for (int k = 0; k < N; ++k)
        a.s += fast_exp(f[k] - b);
}

__device__ __forceinline__ void add_one(Stat &a, float x)
{
    a.raise(x);
    a.s += fast_exp(x - a.base());
}

// Statistics of a row by streaming it: 4 vectors a lane in flight.
template <typename T, int NT>
__device__ __forceinline__ Stat stream_stat(const Cut<T> &c, float *lds)
{
    Stat a{-kInf, 0.f};
    int64_t v = threadIdx.x;
    for (; v + 3 * NT < c.nvec; v += 4 * NT) {
        Pack16<T> p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            p[q] = c.template load<false>(v + q * NT);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            add_vec(a, p[q]);
    }
    for (; v < c.nvec; v += NT)
        add_vec(a, c.template load<false>(v));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t i = c.edge(e);
        if (i >= 0)
            add_one(a, T::up(c.x[i]));
    }
    return block_stat<NT>(a, lds);
}

// Statistics of a row, all of whose vectors (NV a lane) and edge elements stay
// in registers; NV == 0: of a row that is streamed.
template <typename T, int NT, int NV>
__device__ __forceinline__ Stat row_stat(const Cut<T> &c, float *lds, Pack16<T> (&v)[NV > 0 ? NV : 1],
                                         float (&edge)[2])
{
    if (NV == 0)
        return stream_stat<T, NT>(c, lds);
    constexpr int N = Pack16<T>::N;
    Stat a{-kInf, 0.f};
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int64_t at = threadIdx.x + q * NT;
        if (at < c.nvec)
            v[q] = c.template load<false>(at);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t i = c.edge(e);
        edge[e] = i >= 0 ? T::up(c.x[i]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < NV; ++q)
        if ((int64_t)threadIdx.x + q * NT < c.nvec)
#pragma unroll
            for (int e = 0; e < N; ++e)
                a.m = fmaxf(a.m, T::up(v[q].e[e]));
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (c.edge(e) >= 0)
            a.m = fmaxf(a.m, edge[e]);
    const float b = a.base();
#pragma unroll
    for (int q = 0; q < NV; ++q)
        if ((int64_t)threadIdx.x + q * NT < c.nvec)
#pragma unroll
            for (int e = 0; e < N; ++e)
                a.s += fast_exp(T::up(v[q].e[e]) - b);
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (c.edge(e) >= 0)
            a.s += fast_exp(edge[e] - b);
    return block_stat<NT>(a, lds);
}

// log sum_v exp x_v in two parts: the row's maximum, and the binary logarithm
// of what its exponentials sum to when taken from there.  x - top is rounded at
// the size of the row's spread, where x less a sum of both would be off by that
// sum's rounding, 5e-4 of every probability for logits around 1e4.
struct Lse {
    float top, log2s;
    // exp(x - lse)
    __device__ __forceinline__ float prob(float x) const
    {
        return __builtin_amdgcn_exp2f(fmaf(x - top, kLog2e, -log2s));
    }
};

// -d exp(x - lse), and d more at the target.
template <typename T>
__device__ __forceinline__ Pack16<T> grad_vec(const Pack16<T> &p, int64_t at, int64_t y, float d,
                                              Lse lse)
{
    Pack16<T> g;
    float f[Pack16<T>::N];
#pragma unroll
    for (int k = 0; k < Pack16<T>::N; ++k)
        f[k] = -d * lse.prob(T::up(p.e[k]));
    if (y >= at && y < at + Pack16<T>::N) {
#pragma unroll
        for (int k = 0; k < Pack16<T>::N; ++k)
            if (y == at + k)
                f[k] += d;
    }
#pragma unroll
    for (int k = 0; k < Pack16<T>::N; ++k)
        g.e[k] = T::down(f[k]);
    return g;
}

template <typename T, int NT>
__device__ __forceinline__ void grad_edges(const Cut<T> &c, int64_t y, float d, Lse lse)
{
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t i = c.edge(e);
        if (i >= 0) {
            float f = -d * lse.prob(T::up(c.x[i]));
            if (i == y)
                f += d;
            c.d[i] = T::down(f);
        }
    }
}

// Vectors first .. end - 1 of the row, and with the first of them its edges.
template <typename T, int NT>
__device__ __forceinline__ void stream_grad(const Cut<T> &c, int64_t y, float d, Lse lse,
                                            int64_t first, int64_t end)
{
    constexpr int N = Pack16<T>::N;
    int64_t v = first + threadIdx.x;
    for (; v + 3 * NT < end; v += 4 * NT) {
        Pack16<T> p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            p[q] = c.template load<true>(v + q * NT);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            c.store(v + q * NT, grad_vec(p[q], c.head + (v + q * NT) * N, y, d, lse));
    }
    for (; v < end; v += NT)
        c.store(v, grad_vec(c.template load<true>(v), c.head + v * N, y, d, lse));
    if (first == 0)
        grad_edges<T, NT>(c, y, d, lse);
}

template <typename T, int NT>
__device__ __forceinline__ void zero_row(const Cut<T> &c, int64_t first, int64_t end)
{
    Pack16<T> z;
    z.raw = uint4v{0, 0, 0, 0};
    for (int64_t v = first + threadIdx.x; v < end; v += NT)
        c.store(v, z);
    if (first > 0)
        return;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t i = c.edge(e);
        if (i >= 0)
            c.d[i] = T::down(0.f);
    }
}

template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT) void k_logprob(Rows r, int64_t row0, float *logp, float *lse)
{
    __shared__ float lds[2 * NT / 64];
    const int64_t row = row0 + blockIdx.x;
    const int64_t y = target_of(r, row);
    if (y < 0) {
        if (threadIdx.x == 0) {
            logp[row] = 0.f;
            if (lse)
                lse[row] = 0.f;
        }
        return;
    }
    const Cut<T> c(r, row);
    Pack16<T> v[NV > 0 ? NV : 1];
    float edge[2];
    const Stat a = row_stat<T, NT, NV>(c, lds, v, edge);
    if (threadIdx.x == 0) {
        const float xy = y < r.vocab ? T::up(c.x[y]) : __builtin_nanf("");
        const float logs = logf(a.s);
        logp[row] = (xy - a.base()) - logs;
        if (lse)
            lse[row] = y < r.vocab ? a.base() + logs : __builtin_nanf("");
    }
}

// From this |lse| on z1_logprob_grad takes a row's maximum and log-sum anew.
// Below it lse's own rounding is at most 2^-19 of a probability, no more than
// the exponent's for one of e^-22.
constexpr float kFarLse = 64.f;

// The last rows first: z1_token_logprob has just read the logits front to
// back, and the end of them is still in the 256 MB memory-side cache (6144 x
// 32000 bf16, both kernels and the pairs': 189 us, front to back 208).
template <typename T, int NT>
__global__ __launch_bounds__(NT) void k_logprob_grad(Rows r, int64_t row0, const float *lse,
                                                    const float *dlogp)
{
    __shared__ float lds[2 * NT / 64];
    const int64_t row = row0 + gridDim.x - 1 - blockIdx.x;
    const int64_t y = target_of(r, row);
    const Cut<T> c(r, row);
    int64_t first = c.nvec * blockIdx.y / gridDim.y, end = c.nvec * (blockIdx.y + 1) / gridDim.y;
    // a piece without vectors has nothing to do, unless it is the first
    if (blockIdx.y > 0 && first == 0)
        return;
    if (y < 0) {
        zero_row<T, NT>(c, first, end);
        return;
    }
    const float d = y < r.vocab ? dlogp[row] : __builtin_nanf("");
    Lse l{lse[row], 0.f};
    if (fabsf(l.top) >= kFarLse) {
        // a far row is one workgroup's, for it has to be read whole before any
        // of it is overwritten (dlogits may be the logits); an lse that is not
        // the row's own to a unit or two in its last place is taken as it is
        if (blockIdx.y > 0)
            return;
        first = 0;
        end = c.nvec;
        const Stat a = stream_stat<T, NT>(c, lds);
        const float logs = logf(a.s);
        if (fabsf((a.base() + logs) - l.top) < fabsf(l.top) * 0x1p-22f)
            l = Lse{a.base(), logs * kLog2e};
    }
    stream_grad<T, NT>(c, y, d, l, first, end);
}

// Loss of one counted row and its slope in logp.
__device__ __forceinline__ float policy_row(const PolicyPtrs &p, const PolicyScalars &k, int64_t row,
                                            float logp, float &slope)
{
    const float adv = p.adv[row];
    const float rho = expf(logp - p.old_logp[row]);
    const float near = rho < k.lo ? k.lo : rho > k.hi ? k.hi : rho;   // NaN stays
    const float free = rho * adv, held = near * adv;
    float l = -(held < free ? held : free);
    // the unclamped side carries the slope inside the clamp, and where it is
    // the smaller one
    slope = (near == rho || free < held || free != free) ? -free : 0.f;
    if (p.ref_logp) {
        const float gap = p.ref_logp[row] - logp;
        const float e = expm1f(gap);
        l += k.kl * (e - gap);
        slope -= k.kl * e;
    }
    return l;
}

// One row per workgroup.  NV > 0: the row sits in registers, NV vectors a
// lane, between its statistics and its gradient.  NV == 0: it is streamed,
// twice if there is a gradient.
template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT) void k_policy(Rows r, int64_t row0, PolicyPtrs p, PolicyScalars k)
{
    __shared__ float lds[2 * NT / 64];
    __shared__ float shared[3];
    const int64_t row = row0 + blockIdx.x;
    const int64_t y = target_of(r, row);
    const float w = p.w ? p.w[row] : 1.f;
    const Cut<T> c(r, row);
    if (y < 0 || w == 0.f) {
        if (threadIdx.x == 0) {
            p.token_loss[row] = 0.f;
            if (p.logp)
                p.logp[row] = 0.f;
        }
        if (c.d)
            zero_row<T, NT>(c, 0, c.nvec);
        return;
    }
    constexpr int N = Pack16<T>::N;
    // read before the barrier below: the gradient may overwrite the logits
    float xy = 0.f;
    if (threadIdx.x == 0)
        xy = y < r.vocab ? T::up(c.x[y]) : __builtin_nanf("");
    Pack16<T> v[NV > 0 ? NV : 1];
    float edge[2];
    const Stat a = row_stat<T, NT, NV>(c, lds, v, edge);
    if (threadIdx.x == 0) {
        const float logs = logf(a.s);
        const float logp = (xy - a.base()) - logs;
        float slope;
        p.token_loss[row] = policy_row(p, k, row, logp, slope);
        if (p.logp)
            p.logp[row] = logp;
        shared[0] = slope * w * k.scale;
        shared[1] = a.base();
        shared[2] = logs * kLog2e;
    }
    if (!c.d)
        return;
    __syncthreads();
    const float d = shared[0];
    const Lse lse{shared[1], shared[2]};
    if (NV > 0) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int64_t at = threadIdx.x + q * NT;
            if (at < c.nvec)
                c.store(at, grad_vec(v[q], c.head + at * N, y, d, lse));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t i = c.edge(e);
            if (i >= 0) {
                float f = -d * lse.prob(edge[e]);
                if (i == y)
                    f += d;
                c.d[i] = T::down(f);
            }
        }
    } else {
        stream_grad<T, NT>(c, y, d, lse, 0, c.nvec);
    }
}

// scale * sum_r w_r l_r in binary64, in a fixed order: one workgroup, for it
// reads 4 to 16 bytes for each row of logits.  A row that does not count (l is
// 0 there) is left out whatever its weight: 0 times an infinity or a NaN would
// be the whole loss.
__global__ __launch_bounds__(1024) void k_loss_sum(const float *l, const float *w, Rows r,
                                                   double scale, float *loss)
{
    __shared__ double lds[16];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < r.n; i += 1024) {
        const float wi = w ? w[i] : 1.f;
        if (wi != 0.f && !(w && target_of(r, i) < 0))
            s += (double)l[i] * (double)wi;
    }
    for (int o = 32; o > 0; o >>= 1)
        s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int q = 0; q < 16; ++q)
            t += lds[q];
        *loss = (float)(t * scale);
    }
}

__device__ __forceinline__ int64_t offset_of(const z1_preference_args &a, int64_t i)
{
    int64_t o = a.cu_type == Z1_I32 ? (int64_t) static_cast<const int32_t *>(a.cu_seqlens)[i]
                                    : static_cast<const int64_t *>(a.cu_seqlens)[i];
    return o < 0 ? 0 : o > a.n_rows ? a.n_rows : o;
}

__device__ __forceinline__ bool counted(const z1_preference_args &a, int64_t row)
{
    return a.target_type == Z1_I32 ? static_cast<const int32_t *>(a.targets)[row] >= 0
                                   : static_cast<const int64_t *>(a.targets)[row] >= 0;
}

// One pair per workgroup; the workgroup after the last pair clears the slopes
// of the rows outside every sequence.  The sequences' log-ratio sums and the
// logistic are taken in binary64.
__global__ __launch_bounds__(256) void k_preference(z1_preference_args a)
{
    __shared__ double lds[4];
    const int64_t p = blockIdx.x;
    if (p == a.n_pairs) {
        if (!a.dlogp)
            return;
        const int64_t lo = a.n_pairs ? offset_of(a, 0) : a.n_rows;
        const int64_t hi = a.n_pairs ? offset_of(a, 2 * a.n_pairs) : a.n_rows;
        for (int64_t i = threadIdx.x; i < lo; i += 256)
            a.dlogp[i] = 0.f;
        for (int64_t i = hi + threadIdx.x; i < a.n_rows; i += 256)
            a.dlogp[i] = 0.f;
        return;
    }
    const int64_t c0 = offset_of(a, 2 * p), c1 = offset_of(a, 2 * p + 1), c2 = offset_of(a, 2 * p + 2);
    double s = 0.0;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += 256)
        if (counted(a, i))
            s += (double)a.logp[i] - (double)a.ref_logp[i];
    for (int64_t i = c1 + threadIdx.x; i < c2; i += 256)
        if (counted(a, i))
            s -= (double)a.logp[i] - (double)a.ref_logp[i];
    for (int o = 32; o > 0; o >>= 1)
        s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = s;
    __syncthreads();
    const double z = a.beta * (lds[0] + lds[1] + lds[2] + lds[3]);
    const double t = exp(-fabs(z));
    const double e = a.label_smoothing;
    // sigmoid(-z) = the part of the loss's slope, from whichever side is exact
    const double sn = z >= 0.0 ? t / (1.0 + t) : 1.0 / (1.0 + t);
    const double sp = z >= 0.0 ? 1.0 / (1.0 + t) : t / (1.0 + t);
    if (threadIdx.x == 0) {
        const double soft = log1p(t);
        const double down = soft + (z < 0.0 ? -z : 0.0), up = soft + (z > 0.0 ? z : 0.0);
        // a side of weight 0 adds nothing, infinite or not
        a.pair_loss[p] = (float)((e != 1.0 ? (1.0 - e) * down : 0.0) + (e != 0.0 ? e * up : 0.0));
        if (a.margins)
            a.margins[p] = (float)z;
    }
    if (!a.dlogp)
        return;
    const float d = (float)(a.scale * a.beta * (e * sp - (1.0 - e) * sn));
    for (int64_t i = c0 + threadIdx.x; i < c1; i += 256)
        a.dlogp[i] = counted(a, i) ? d : 0.f;
    for (int64_t i = c1 + threadIdx.x; i < c2; i += 256)
        a.dlogp[i] = counted(a, i) ? -d : 0.f;
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

template <int V>
using Int = std::integral_constant<int, V>;

// One workgroup of NT lanes per row, in pieces of fewer than 2^32 lanes (the
// most one launch takes).
template <typename F>
void over_rows(int64_t n, int nt, F &&f)
{
    const int64_t step = (INT64_C(1) << 31) / nt;
    for (int64_t r = 0; r < n; r += step)
        f((uint32_t)std::min(step, n - r), r);
}

// Lanes and vectors a lane (0: streamed) of the kernels that hold a row in
// registers: the loads of a whole row are then in flight at once.  Each stair is
// the fewest registers that hold its rows, as they cost residency: with 16
// vectors a lane instead of 12, 6144 vectors take 102 us instead of 78
// (z1_token_logprob, 4096 x 49152 bf16), with 24 5000 take 99 instead of 62.
// Held / streamed, us, of z1_policy_loss and z1_token_logprob: 6144 vectors
// (4096 x 49152 bf16) 154 / 190 and 78 / 84; 8192 (4096 x 65536 bf16) 215 / 234
// and 118 / 87; 12288 (2048 x 98304 bf16) 176 / 167 and 82 / 69, (2048 x 49152
// fp32) 158 / 155 and 73 / 70; 16032 (2048 x 128256 bf16, 1024 lanes of 16) 216 /
// 229 and 140 / 88.  So holding a row pays for both up to 6144 vectors and for
// the policy loss, which reads it twice otherwise, to 8192; 12288 is where it has
// stopped paying.
template <typename T, typename F>
void by_row(int64_t vocab, F &&f)
{
    const int64_t nv = vocab / Pack16<T>::N;
    if (nv <= 256)
        f(Int<64>(), Int<4>());
    else if (nv <= 1024)
        f(Int<256>(), Int<4>());
    else if (nv <= 4096)
        f(Int<512>(), Int<8>());
    else if (nv <= 6144)
        f(Int<512>(), Int<12>());
    else if (nv <= 8192)
        f(Int<512>(), Int<16>());
    else if (nv <= 12288)
        f(Int<1024>(), Int<12>());
    else
        f(Int<1024>(), Int<0>());
}

}  // namespace

hipError_t launch_logprob(int32_t dtype, const Rows &r, float *logp, float *lse, hipStream_t s)
{
    if (r.n == 0)
        return hipSuccess;
    return by_type(dtype, [&](auto t) {
        typedef decltype(t) T;
        by_row<T>(r.vocab, [&](auto nt, auto nvec) {
            constexpr int NT = decltype(nt)::value, NV = decltype(nvec)::value;
            over_rows(r.n, NT, [&](uint32_t nb, int64_t row0) {
                k_logprob<T, NT, NV><<<nb, NT, 0, s>>>(r, row0, logp, lse);
            });
        });
    });
}

hipError_t launch_logprob_grad(int32_t dtype, const Rows &r, const float *lse, const float *dlogp,
                               hipStream_t s)
{
    if (r.n == 0)
        return hipSuccess;
    return by_type(dtype, [&](auto t) {
        typedef decltype(t) T;
        const int64_t nv = r.vocab / Pack16<T>::N;
        const auto go = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            // few long rows: in pieces of 1024 vectors at least, 2048
            // workgroups at most (348 x 32001 fp32: 18.4 us against 19.7)
            const int64_t most = std::min<int64_t>(nv / 1024, 2048 / r.n);
            const uint32_t pieces = (uint32_t)std::max<int64_t>(1, most);
            over_rows(r.n, NT, [&](uint32_t nb, int64_t row0) {
                k_logprob_grad<T, NT><<<dim3(nb, pieces), NT, 0, s>>>(r, row0, lse, dlogp);
            });
        };
        if (nv <= 128)
            go(Int<64>());
        else
            go(Int<256>());
    });
}

hipError_t launch_policy(int32_t dtype, const Rows &r, const PolicyPtrs &p, const PolicyScalars &k,
                         float *loss, double scale, hipStream_t s)
{
    hipError_t e = hipSuccess;
    if (r.n > 0)
        e = by_type(dtype, [&](auto t) {
            typedef decltype(t) T;
            by_row<T>(r.vocab, [&](auto nt, auto nvec) {
                constexpr int NT = decltype(nt)::value, NV = decltype(nvec)::value;
                over_rows(r.n, NT, [&](uint32_t nb, int64_t row0) {
                    k_policy<T, NT, NV><<<nb, NT, 0, s>>>(r, row0, p, k);
                });
            });
        });
    if (e != hipSuccess)
        return e;
    k_loss_sum<<<1, 1024, 0, s>>>(p.token_loss, p.w, r, scale, loss);
    return hipGetLastError();
}

hipError_t launch_preference(const z1_preference_args &a, hipStream_t s)
{
    k_preference<<<(uint32_t)(a.n_pairs + 1), 256, 0, s>>>(a);
    Rows pairs{};
    pairs.n = a.n_pairs;
    k_loss_sum<<<1, 1024, 0, s>>>(a.pair_loss, nullptr, pairs, a.scale, a.loss);
    return hipGetLastError();
}

}  // namespace ops
}  // namespace z1

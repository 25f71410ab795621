// z1_layers_internal.h -- what the host code of the layers (z1_layers_api.hip)
// and their kernels (z1_linear.hip, z1_layers.hip) share.  Not installed.
#pragma once

#include "z1_layers.h"
#include "z1_ops_internal.h"

namespace z1 {
namespace ops {

// z1_drop as the kernels take it; rng null: no dropout.
struct Drop {
    const uint64_t *rng;
    uint64_t offset;
    uint32_t threshold;   // 0 .. 65536
    float scale;
};

// The same with the device's seed and offset read.
struct DropKey {
    uint32_t seed[2], offset[2], threshold;
    float scale;
    bool on;
};

__device__ __forceinline__ DropKey drop_key(const Drop &d)
{
    DropKey k{};
    k.on = d.rng != nullptr;
    if (k.on) {
        const uint64_t seed = d.rng[0], offset = d.rng[1] + d.offset;
        k.seed[0] = (uint32_t)seed;
        k.seed[1] = (uint32_t)(seed >> 32);
        k.offset[0] = (uint32_t)offset;
        k.offset[1] = (uint32_t)(offset >> 32);
        k.threshold = d.threshold;
        k.scale = d.scale;
    }
    return k;
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): the four words of counter
// (block, row, offset).  The key schedule is the same for the whole launch and
// stays in scalar registers; a round is two 32 x 32 bit multiplies.
__device__ __forceinline__ void philox(const DropKey &k, uint32_t block, uint32_t row, uint32_t (&w)[4])
{
    uint32_t a = block, b = row, c = k.offset[0], d = k.offset[1], k0 = k.seed[0], k1 = k.seed[1];
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(q >> 32) ^ b ^ k0;
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ d ^ k1;
        d = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = a;
    w[1] = b;
    w[2] = c;
    w[3] = d;
}

// Whether the mask's words keep element j of eight.
__device__ __forceinline__ bool drop_keeps(const DropKey &k, const uint32_t (&w)[4], int j)
{
    return (j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu) >= k.threshold;
}

// Eight elements (row, 8 block ..) after dropout.
__device__ __forceinline__ void drop8(const DropKey &k, uint32_t block, uint32_t row, float (&v)[8])
{
    uint32_t w[4];
    philox(k, block, row, w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = drop_keeps(k, w, j) ? v[j] * k.scale : 0.f;
}

// Eight elements of type T at any alignment of T, in as few accesses as that
// takes (the hardware takes vector accesses at any address).
template <int ALIGN>
struct Words {
    typedef uint32_t four __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Words<4> {
    typedef uint32_t four __attribute__((ext_vector_type(4), aligned(4)));
};

template <typename T>
struct Eight {
    typedef typename Words<(int)sizeof(typename T::store)>::four word4;
    static constexpr int kWords = (int)sizeof(typename T::store) / 2;   // of 16 bytes
    typedef uint4v Raw[kWords];
    static __device__ __forceinline__ void fetch(const void *p, Raw &raw)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            raw[i] = static_cast<const word4 *>(p)[i];
    }
    static __device__ __forceinline__ void up(const Raw &raw, float (&v)[8])
    {
        union {
            Raw raw;
            typename T::store e[8];
        } u;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            u.raw[i] = raw[i];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = T::up(u.e[j]);
    }
    static __device__ __forceinline__ void load(const void *p, float (&v)[8])
    {
        Raw raw;
        fetch(p, raw);
        up(raw, v);
    }
    static __device__ __forceinline__ void store(void *p, const float (&v)[8])
    {
        union {
            Raw raw;
            typename T::store e[8];
        } u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            u.e[j] = T::down(v[j]);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            static_cast<word4 *>(p)[i] = u.raw[i];
    }
    // the first n of them, where there are so many; the others load as zeros
    static __device__ __forceinline__ void load_some(const void *p, float (&v)[8], int n)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = j < n ? T::up(static_cast<const typename T::store *>(p)[j]) : 0.f;
    }
    static __device__ __forceinline__ void store_some(void *p, const float (&v)[8], int n)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                static_cast<typename T::store *>(p)[j] = T::down(v[j]);
    }
};

// act(z) and act'(z).  Written so that they hold at both ends: the sigmoid
// underflows to 0 for z << 0, and Phi keeps its relative precision there.
//
// The gradient's pre may be infinite where z was not (one past fp16 is), so there both are
// their limits: act takes `above_low(z)` for its factor z, which is finite where the other
// factor is 0, and the slopes take their factor z between ends where theirs is.  NaN comes
// through the other factors.  (8192 x 8192 fp16: SILU without a product 88 -> 91 us.)
__device__ __forceinline__ float above_low(float z) { return __builtin_amdgcn_fmed3f(z, -1e30f, __builtin_inff()); }
__device__ __forceinline__ float between_ends(float z) { return __builtin_amdgcn_fmed3f(z, -1e15f, 1e15f); }
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + expf(-z)); }
__device__ __forceinline__ float gelu_tanh_arg(float z)
{
    return 1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f);   // 2 sqrt(2 / pi)
}

// exp(-z^2 / 2) and Phi(z), both to 1e-6 of themselves while they are normal numbers (|z| <
// 12.9).  For u = |z| / sqrt(2),
//   Phi(-|z|) = erfc(u) / 2 = exp(-z^2 / 2) t Q(t) / 2,   t = 1 / (1 + 0.3 u)
// with a Q of degree 8 fitted to exp(u^2) erfc(u) / t over u in [0, 11] by least squares,
// reweighted until its relative error was even: 2e-8.  z^2 is taken with its rounding, as
// the exponential multiplies that by z^2 / 2.  Behind |z| = 16 both are 0 in fp32; NaN
// is not behind it.  8192 x 2048 -> 8192 with bias and GELU: 314 us, 344 with the library's
// erfc; its gradient of 8192 x 8192, with a product: 143 and 230.
struct Normal {
    float bell, below;
};
__device__ __forceinline__ Normal normal_of(float z)
{
    const float s = fabsf(z) > 16.f ? 16.f : fabsf(z), square = s * s;
    const float e = expf(-0.5f * square), bell = fmaf(-0.5f * e, fmaf(s, s, -square), e);
    const float t = __builtin_amdgcn_rcpf(fmaf(s, 0.212132034f, 1.f));
    float q = -0.129556016f;
    q = fmaf(q, t, 0.485737081f);
    q = fmaf(q, t, -0.512669489f);
    q = fmaf(q, t, 0.548212623f);
    q = fmaf(q, t, -0.0950292301f);
    q = fmaf(q, t, 0.215107598f);
    q = fmaf(q, t, 0.148286179f);
    q = fmaf(q, t, 0.170723821f);
    q = fmaf(q, t, 0.169187413f);
    const float tail = 0.5f * bell * (t * q);
    return Normal{bell, z < 0.f ? tail : 1.f - tail};
}

// factor: z, or above_low(z)
template <int ACT>
__device__ __forceinline__ float act_value(float z, float factor)
{
    if constexpr (ACT == Z1_ACT_RELU)
        return z < 0.f ? 0.f : z;
    if constexpr (ACT == Z1_ACT_GELU)
        return factor * normal_of(z).below;
    if constexpr (ACT == Z1_ACT_GELU_TANH)
        return factor * sigmoid(gelu_tanh_arg(z));
    if constexpr (ACT == Z1_ACT_SILU)
        return factor * sigmoid(z);
    if constexpr (ACT == Z1_ACT_RELU2) {
        const float r = z < 0.f ? 0.f : z;
        return r * r;
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == Z1_ACT_RELU)
        return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == Z1_ACT_GELU) {
        const Normal n = normal_of(z);
        return fmaf(between_ends(z) * 0.39894228040143268f, n.bell, n.below);
    }
    if constexpr (ACT == Z1_ACT_GELU_TANH) {
        const float s = sigmoid(gelu_tanh_arg(z)), f = between_ends(z);
        return fmaf(f * s * (1.f - s), 1.5957691216057308f * fmaf(3.f * 0.044715f, f * f, 1.f), s);
    }
    if constexpr (ACT == Z1_ACT_SILU) {
        const float s = sigmoid(z);
        return s * fmaf(between_ends(z), 1.f - s, 1.f);
    }
    if constexpr (ACT == Z1_ACT_RELU2)
        return 2.f * (z < 0.f ? 0.f : z);
    return 1.f;
}

// f(a constant) for the activation of this number; nothing for none.
template <typename F>
__device__ __forceinline__ void with_act(int32_t act, F &&f)
{
    switch (act) {
    case Z1_ACT_RELU: f(std::integral_constant<int, Z1_ACT_RELU>()); break;
    case Z1_ACT_GELU: f(std::integral_constant<int, Z1_ACT_GELU>()); break;
    case Z1_ACT_GELU_TANH: f(std::integral_constant<int, Z1_ACT_GELU_TANH>()); break;
    case Z1_ACT_SILU: f(std::integral_constant<int, Z1_ACT_SILU>()); break;
    case Z1_ACT_RELU2: f(std::integral_constant<int, Z1_ACT_RELU2>()); break;
    default: break;
    }
}

__device__ __forceinline__ void act_values(int32_t act, float (&v)[8])
{
    with_act(act, [&](auto a) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = act_value<decltype(a)::value>(v[j], v[j]);
    });
}

// --------------------------------------------------------------------------
// Products.  C[q][p] = sum_k P(p, k) Q(q, k), p along C's rows' elements.
// --------------------------------------------------------------------------

// One operand.  Deep: element (i, k) at base + i * ld + k * size ("the depth is
// contiguous"); else at base + k * ld + i * size.  ld in bytes, a multiple of
// 16 as base is; the contiguous extent is whole 16-byte chunks.
struct Operand {
    const void *base;
    int64_t ld;
    int32_t extent;       // of i
    int32_t depth;        // of k
};

// What is done with C's elements.  Plain: out = c + add.  Full: z1_linear's
// epilogue.  Distances in elements.
struct Epilogue {
    void *out, *pre;
    const void *add, *mul, *bias;
    int64_t ld_out, ld_pre, ld_add, ld_mul;
    Drop drop;
    int32_t act;
};

struct Product {
    Operand p, q;
    int32_t P, Q;          // C's row length and rows
    Epilogue e;
    float *parts;          // partial sums of `splits` pieces of the depth
    int32_t splits;        // 1: not split
    int32_t piece;         // bytes of depth a piece takes, whole panels
    int32_t tiles_p, tiles_q;
    int32_t tile;          // side: 64, 128 or 256; 0: few rows
};

enum Form { kForward, kInput, kWeight };   // x W', dz W, dz' x: which operands are deep

hipError_t launch_product(Form form, int32_t dtype, int32_t out_dtype, const Product &g, hipStream_t s);

// x W' of at most kRowsMost rows (tile 0): no copies, no partial sums.
constexpr int64_t kRowsMost = 4;
hipError_t launch_rows(int32_t dtype, const Product &g, hipStream_t s);

// Rows of `cols` elements to be copied to rows of `cols_to`, a multiple of eight, zeros
// behind them.
struct Copy {
    const void *from;
    void *to;
    int64_t ld, rows, cols, cols_to;
};
// Both at once; rows 0: none.
hipError_t launch_pack(int32_t dtype, const Copy &a, const Copy &b, hipStream_t s);

// --------------------------------------------------------------------------
// Elementwise layers
// --------------------------------------------------------------------------

hipError_t launch_dropout(const z1_dropout_args &a, const Drop &d, hipStream_t s);

// z1_linear_dz: lanes of eight columns a workgroup has, and the rows of its piece, whole
// groups of 256 / lanes; each piece leaves one row of column sums.
inline int64_t dz_lanes(int64_t out) { return out <= 64 ? 8 : out <= 128 ? 16 : 32; }
inline int64_t dz_piece(int64_t rows, int64_t out)
{
    const int64_t lanes = dz_lanes(out), across = (out + lanes * 8 - 1) / (lanes * 8);
    return pad_to(std::max<int64_t>(1, rows * across / 1024), 256 / lanes);
}
hipError_t launch_linear_dz(const z1_linear_dz_args &a, const Drop &d, float *parts, hipStream_t s);

// Workgroups that z1_qk_norm_rope_grad gives to queries (kind 0) or keys (1), each of
// which leaves a row of sums.
int64_t qk_grad_groups(int64_t tokens, int64_t q_heads, int64_t k_heads, int kind);
hipError_t launch_qk(const z1_qk_args &a, hipStream_t s);
hipError_t launch_qk_grad(const z1_qk_args &a, float *parts, hipStream_t s);

}  // namespace ops
}  // namespace z1

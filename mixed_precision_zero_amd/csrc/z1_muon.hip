// z1_muon.hip -- the kernels of z1_muon_step and z1_muon_orthogonalize.
//
// Newton-Schulz: X <- a X + (b A + c A A) X with A = X X^T, ns_steps times,
// from X = U / (|U|_F + eps), X the m x n matrix with m <= n.  Three products
// a step: A (symmetric), A A (symmetric) and B X.  Only the tiles on and
// below the diagonal of the symmetric ones are computed and mirrored, so a
// step costs 2 (m^2 n / 2 + m^3 / 2 + m^2 n) multiply-adds' flops, not
// 2 (2 m^2 n + m^3).
//
// Every product is of the form C_ij = sum_k P_ik Q_jk with both operands
// contiguous along k: X X^T, A A^T, and B (X^T)^T from a kept transpose Y of
// X.  The update's epilogue writes X and Y, which costs 2 more bytes per
// element and lets one kernel feed all three with 16-byte rows.
//
// Numbers.  The products take fp16 operands and accumulate in fp32 on the
// matrix cores.  X, A and B are bounded (|X| <= 1.21, |A| <= 1.46,
// |B| <= 2.81 for the usual coefficients; z1_muon_create refuses others that
// leave 3.9), so they are stored times kScale = 2^14: nothing overflows, and
// values down to 2^-28 stay normal numbers, which matters because X starts
// with elements near 1 / sqrt(m n).  fp16 keeps 11 bits where bf16 keeps 8.
// X is carried from step to step in fp32 and only its operand copies are
// rounded: the step multiplies the small singular values by a = 3.44 each
// time, and with them every rounding of X, so with X itself rounded to fp16 a
// low-rank U plus 1% noise comes out 4% off (34% with bf16 throughout), and
// 0.04% with the fp32 carry (simulated in binary64 with these roundings,
// 1024 x 1024; a gaussian U: 0.13% against 0.12% and 0.9%).
#include "z1_ops_internal.h"

namespace z1 {
namespace ops {
namespace {

constexpr float kScale = 16384.0f;
constexpr float kUnscale = 1.0f / 16384.0f;

__device__ __forceinline__ double block_sum(double x, double *lds)
{
    for (int o = 32; o > 0; o >>= 1)
        x += __shfl_xor(x, o);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
        lds[wave] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w)
        s += lds[w];
    __syncthreads();
    return s;
}

// min(1, clip / (sqrt(S) + 1e-6)), as the AdamW step takes it: a NaN norm
// stays NaN.
__device__ __forceinline__ float clip_factor(const MuonUpdate &u)
{
    if (!(u.clip > 0.0))
        return 1.0f;
    const double c = u.clip / (sqrt(*u.d_S) + 1e-6);
    return (float)(c > 1.0 ? 1.0 : c);
}

template <bool BF>
__device__ __forceinline__ float load_grad(const MuonMat &t, int64_t i)
{
    return BF ? bf16_to_f32(static_cast<const uint16_t *>(t.grad)[i])
              : static_cast<const float *>(t.grad)[i];
}

// Elementwise pass: the momentum update and the partial sums of U's squares
// (binary64: squares of any finite fp32 values neither overflow nor vanish).
template <bool BF, bool STEP>
__global__ __launch_bounds__(256) void k_muon_momentum(const MuonMat *mats,
                                                       const MuonChunk *chunks, double *partials,
                                                       MuonUpdate u)
{
    __shared__ double lds[4];
    const MuonChunk ch = chunks[blockIdx.x];
    const MuonMat &t = mats[ch.mat];
    const float c = STEP ? clip_factor(u) : 1.0f;
    double s = 0.0;
    const auto one = [&](float grad, float &mom) {
        const float g = c * grad;
        float x = g;
        if (STEP) {
            mom = fmaf(u.mu, mom, g);
            x = u.nesterov ? fmaf(u.mu, mom, g) : mom;
        }
        s += (double)x * (double)x;
    };
    int done = 0;
    if (t.vec) {
        done = ch.count & ~3;
        for (int e = threadIdx.x * 4; e < done; e += 256 * 4) {
            const int64_t i = ch.start + e;
            float g[4];
            if (BF) {
                const uint2v p =
                    *reinterpret_cast<const uint2v *>(static_cast<const uint16_t *>(t.grad) + i);
                g[0] = __uint_as_float(p.x << 16);
                g[1] = __uint_as_float(p.x & 0xffff0000u);
                g[2] = __uint_as_float(p.y << 16);
                g[3] = __uint_as_float(p.y & 0xffff0000u);
            } else {
                const float4v p =
                    *reinterpret_cast<const float4v *>(static_cast<const float *>(t.grad) + i);
                for (int k = 0; k < 4; ++k)
                    g[k] = p[k];
            }
            float4v m = {0.f, 0.f, 0.f, 0.f};
            if (STEP)
                m = *reinterpret_cast<const float4v *>(t.mom + i);
            for (int k = 0; k < 4; ++k) {
                float mk = m[k];
                one(g[k], mk);
                m[k] = mk;
            }
            if (STEP)
                *reinterpret_cast<float4v *>(t.mom + i) = m;
        }
    }
    for (int e = done + threadIdx.x; e < ch.count; e += 256) {
        const int64_t i = ch.start + e;
        float m = STEP ? t.mom[i] : 0.f;
        one(load_grad<BF>(t, i), m);
        if (STEP)
            t.mom[i] = m;
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0)
        partials[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_muon_norm(const MuonMat *mats, const double *partials,
                                                   double *inv, double eps)
{
    __shared__ double lds[4];
    const MuonMat &t = mats[blockIdx.x];
    double s = 0.0;
    for (int64_t q = threadIdx.x; q < t.n_part; q += 256)
        s += partials[t.part0 + q];
    s = block_sum(s, lds);
    if (threadIdx.x == 0) {
        const double d = sqrt(s) + eps;
        inv[blockIdx.x] = d == 0.0 ? 0.0 : 1.0 / d;
    }
}

// X = U / (|U|_F + eps), as the fp16 operands X and Y = X^T and the fp32
// carry, one 64 x 64 tile of the padded X per workgroup through LDS.
template <bool BF, bool STEP>
__global__ __launch_bounds__(256) void k_muon_cast(const MuonMat *mats, const MuonTile *tiles,
                                                   const double *inv, MuonUpdate u)
{
    __shared__ float lds[kCastTile][kCastTile + 1];   // [X row][X column]
    const MuonTile tl = tiles[blockIdx.x];
    const MuonMat &t = mats[tl.mat];
    const float c = STEP ? clip_factor(u) : 1.0f;
    const double r = inv[tl.mat] * (double)kScale;
    const int i0 = tl.ti * kCastTile, j0 = tl.tj * kCastTile;
    const int r0 = t.flip ? j0 : i0, c0 = t.flip ? i0 : j0;
    const int cc = threadIdx.x & 63;
#pragma unroll 4
    for (int q = 0; q < 16; ++q) {
        const int rr = (threadIdx.x >> 6) + 4 * q;
        float x = 0.f;
        if (r0 + rr < t.rows && c0 + cc < t.cols) {
            const int64_t i = (int64_t)(r0 + rr) * t.cols + c0 + cc;
            const float g = c * load_grad<BF>(t, i);
            x = g;
            if (STEP)
                x = u.nesterov ? fmaf(u.mu, t.mom[i], g) : t.mom[i];
            x = (float)((double)x * r);
        }
        if (t.flip)
            lds[cc][rr] = x;
        else
            lds[rr][cc] = x;
    }
    __syncthreads();
    for (int q = threadIdx.x; q < 512; q += 256) {
        const int row = q >> 3, at = (q & 7) * 8;
        half8 x, y;
        for (int k = 0; k < 8; ++k) {
            x[k] = (_Float16)lds[row][at + k];
            y[k] = (_Float16)lds[at + k][row];
        }
        *reinterpret_cast<half8 *>(t.X + (int64_t)(i0 + row) * t.np + j0 + at) = x;
        *reinterpret_cast<half8 *>(t.Y[0] + (int64_t)(j0 + row) * t.mp + i0 + at) = y;
    }
    for (int q = threadIdx.x; q < 1024; q += 256) {
        const int row = q >> 4, at = (q & 15) * 4;
        float4v y;
        for (int k = 0; k < 4; ++k)
            y[k] = lds[at + k][row];
        *reinterpret_cast<float4v *>(t.C + (int64_t)(j0 + row) * t.mp + i0 + at) = y;
    }
}

enum Mode { kGram, kPoly, kUpdate, kOrtho, kStep };

// C_ij = sum_k P_ik Q_jk on one T x T tile, K in steps of 64: both operands'
// 64-wide panels come straight into LDS (16 bytes a lane, double buffered, so
// the next panel is in flight while this one is multiplied).  A panel row is
// 128 bytes, all 32 banks, so the 16-byte chunks of row r are stored permuted
// by r mod 8: the 8 rows a fragment read touches at once then lie on
// different banks.  The permutation is applied to the global address, as the
// LDS side of the copy is fixed at 16 bytes a lane in lane order.
template <int T, int WM, int WN, Mode MODE>
__global__ __launch_bounds__(64 * WM * WN) void k_muon_gemm(const MuonMat *mats,
                                                            const MuonTile *tiles, int src,
                                                            float ca, float cb, float cc,
                                                            MuonUpdate u)
{
    constexpr int NW = WM * WN;
    constexpr int TM = T / WM / 32, TN = T / WN / 32;
    constexpr int kLoads = T / 8 / NW;   // 1 KiB copies per wave, operand and step
    static_assert(kLoads >= 1 && TM >= 1 && TN >= 1, "tile and wave grid");
    __shared__ __align__(16) _Float16 lds[2][2 * T * 64];

    const MuonTile tl = tiles[blockIdx.x];
    const MuonMat &t = mats[tl.mat];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i0 = tl.ti * T, j0 = tl.tj * T;

    const _Float16 *P, *Q;
    int K;
    if (MODE == kGram) {
        P = Q = t.X;
        K = t.np;
    } else if (MODE == kPoly) {
        P = Q = t.A;
        K = t.mp;
    } else {
        P = t.B;
        Q = t.Y[src];
        K = t.mp;
    }
    // both operands' rows are K elements apart; a tile's panel rows span less
    // than 2^31 bytes (T * K * 2 with K <= 2^20 + 256)
    const int span = T * K * 2;
    const auto rp = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<_Float16 *>(P + (int64_t)i0 * K), 0, span, 0x00020000);
    const auto rq = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<_Float16 *>(Q + (int64_t)j0 * K), 0, span, 0x00020000);
    const int voff = ((lane >> 3) * K + ((lane & 7) ^ (lane >> 3)) * 8) * 2;

    typedef __attribute__((address_space(3))) void lds_void;
    const auto load = [&](int b, int k) {
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int at = wave * kLoads + q;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (lds_void *)&lds[b][at * 512], 16, voff,
                                                     (at * 8 * K + k) * 2, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_void *)&lds[b][T * 64 + at * 512],
                                                     16, voff, (at * 8 * K + k) * 2, 0, 0);
        }
    };

    float16v acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.f;

    const int half = lane >> 5, low = lane & 31;
    load(0, 0);
    const int steps = K / 64;
    for (int k = 0; k < steps; ++k) {
        // this panel has arrived (vmcnt 0) and every wave has read the one
        // before it (lgkmcnt 0), whose buffer the next copy overwrites
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (k + 1 < steps)
            load((k + 1) & 1, (k + 1) * 64);
        const _Float16 *pa = &lds[k & 1][0], *pb = &lds[k & 1][T * 64];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            half8 a[TM], b[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int r = (wm * TM + i) * 32 + low;
                a[i] = *reinterpret_cast<const half8 *>(pa + r * 64 + (((kk * 2 + half) ^ (r & 7)) * 8));
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int r = (wn * TN + j) * 32 + low;
                b[j] = *reinterpret_cast<const half8 *>(pb + r * 64 + (((kk * 2 + half) ^ (r & 7)) * 8));
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
        asm volatile("" ::: "memory");
    }

    // A lane holds, of each 32 x 32 block, column `low` and rows
    // 8 g + 4 half + (0..3) for g = 0..3.
    const double decay = 1.0 - u.lr * u.wd * t.wd_scale, step = u.lr * t.lr_scale;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int jj = j0 + (wn * TN + j) * 32 + low;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int ii = i0 + (wm * TM + i) * 32 + 8 * g + 4 * half;
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = acc[i][j][4 * g + k] * kUnscale;
                if (MODE == kGram || MODE == kPoly) {
                    _Float16 *D = MODE == kGram ? t.A : t.B;
                    if (MODE == kPoly) {
                        const half4 x = *reinterpret_cast<const half4 *>(t.A + (int64_t)jj * t.mp + ii);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = fmaf(cc, v[k], cb * (float)x[k]);
                    }
                    half4 h;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = (_Float16)v[k];
                    *reinterpret_cast<half4 *>(D + (int64_t)jj * t.mp + ii) = h;
                    if (tl.ti != tl.tj)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            D[(int64_t)(ii + k) * t.mp + jj] = h[k];
                } else {
                    float4v *cp = reinterpret_cast<float4v *>(t.C + (int64_t)jj * t.mp + ii);
                    const float4v x = *cp;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = fmaf(ca, x[k], v[k]);
                    if (MODE == kUpdate) {
                        float4v y;
                        half4 h;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            y[k] = v[k];
                            h[k] = (_Float16)v[k];
                            t.X[(int64_t)(ii + k) * t.np + jj] = h[k];
                        }
                        *cp = y;
                        *reinterpret_cast<half4 *>(t.Y[src ^ 1] + (int64_t)jj * t.mp + ii) = h;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (ii + k >= t.m || jj >= t.n)
                                continue;
                            const int64_t e = t.flip ? (int64_t)jj * t.cols + ii + k
                                                     : (int64_t)(ii + k) * t.cols + jj;
                            const float o = v[k] * kUnscale;
                            if (MODE == kOrtho) {
                                t.ortho[e] = f32_to_bf16(o);
                            } else {
                                const float w = (float)((double)t.master[e] * decay - step * (double)o);
                                t.master[e] = w;
                                t.weight[e] = f32_to_bf16(w);
                            }
                        }
                    }
                }
            }
        }
    }
}

template <int T, int WM, int WN>
void iterate(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s)
{
    constexpr int B = 64 * WM * WN;
    for (int k = 0; k < ns_steps; ++k) {
        const int src = k & 1;
        k_muon_gemm<T, WM, WN, kGram><<<(uint32_t)t.n_sym, B, 0, s>>>(t.mats, t.sym, src, t.a, t.b, t.c, u);
        k_muon_gemm<T, WM, WN, kPoly><<<(uint32_t)t.n_sym, B, 0, s>>>(t.mats, t.sym, src, t.a, t.b, t.c, u);
        if (k + 1 < ns_steps)
            k_muon_gemm<T, WM, WN, kUpdate><<<(uint32_t)t.n_full, B, 0, s>>>(t.mats, t.full, src, t.a, t.b, t.c, u);
        else if (u.step)
            k_muon_gemm<T, WM, WN, kStep><<<(uint32_t)t.n_full, B, 0, s>>>(t.mats, t.full, src, t.a, t.b, t.c, u);
        else
            k_muon_gemm<T, WM, WN, kOrtho><<<(uint32_t)t.n_full, B, 0, s>>>(t.mats, t.full, src, t.a, t.b, t.c, u);
    }
}

template <bool BF, bool STEP>
void first(const MuonTables &t, const MuonUpdate &u, hipStream_t s)
{
    k_muon_momentum<BF, STEP><<<(uint32_t)t.n_chunks, 256, 0, s>>>(t.mats, t.chunks, t.partials, u);
    k_muon_norm<<<(uint32_t)t.n, 256, 0, s>>>(t.mats, t.partials, t.inv, t.eps);
    k_muon_cast<BF, STEP><<<(uint32_t)t.n_cast, 256, 0, s>>>(t.mats, t.cast, t.inv, u);
}

}  // namespace

hipError_t launch_muon(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s)
{
    if (t.n == 0)
        return hipSuccess;
    if (t.grad_bf16)
        u.step ? first<true, true>(t, u, s) : first<true, false>(t, u, s);
    else
        u.step ? first<false, true>(t, u, s) : first<false, false>(t, u, s);
    if (t.tile == 256)
        iterate<256, 2, 4>(t, u, ns_steps, s);
    else if (t.tile == 128)
        iterate<128, 2, 2>(t, u, ns_steps, s);
    else
        iterate<64, 2, 2>(t, u, ns_steps, s);
    return hipGetLastError();
}

}  // namespace ops
}  // namespace z1

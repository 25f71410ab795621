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
// element and lets one kernel feed all three the same way.  With the
// remainder a step's epilogue moves 10 bytes an element (14 with an fp32
// carry), which is what bounds the update of small matrices.
//
// Numbers.  The products take fp16 operands and accumulate in fp32 on the
// matrix cores.  X, A and B are bounded (|X| <= 1.21, |A| <= 1.46,
// |B| <= 2.81 for the usual coefficients; z1_muon_create refuses others that
// leave 3.9), so they are stored times kScale = 2^14: nothing overflows, and
// values down to 2^-28 stay normal numbers, which matters because X starts
// with elements near 1 / sqrt(m n).  fp16 keeps 11 bits where bf16 keeps 8.
// X is carried from step to step in 22 bits, as its fp16 operand copy plus an
// fp16 remainder (fp32 registers in the one-workgroup kernel), and only the
// products see it rounded to 11: the step multiplies the small singular values
// by a = 3.44 each time, and with them every rounding of X.  Error of O,
// measured, and simulated in binary64 with these roundings and X carried in 32,
// 22 or 11 bits: 2048 x 2048 gaussian 1.2e-3; 1.2e-3, 1.2e-3, 1.1e-3, of rank 4
// plus 1% noise 8e-5; 8e-5, 8e-5, 4.2e-2, 64 x 64 gaussian 2e-3; 2e-3, 2e-3,
// 1.7e-3, noisy 5e-4; 5e-4, 5e-4, 3.6e-2.  With bf16 operands throughout it is
// 1% to 34%.
//
// Wide products (z1_muon_create_wide) take X, A and B in 22 bits and carry X in
// fp32: 1.4e-6 and 2.6e-5 for those 2048 x 2048, where fp32 products leave 3.6e-6
// and 7e-5.  Steps of 4 x 2048^2 2.71 ms against 1.04, 4096 x 11008 10.4 against
// 3.8, 8 x 1536 x 576 0.55 against 0.26, 2 x 64 x 256 85 us against 28.
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

// What fp16 leaves of x, itself in fp16: together 22 bits.
__device__ __forceinline__ _Float16 low_part(float x)
{
    return (_Float16)(x - (float)(_Float16)x);
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

// 1 / (|U|_F + eps) from a matrix's partial sums, in a fixed order; called by a
// workgroup of 256.
__device__ __forceinline__ double inverse_norm(const MuonMat &t, const double *partials, double eps,
                                               double *lds)
{
    double s = 0.0;
    for (int64_t q = threadIdx.x; q < t.n_part; q += 256)
        s += partials[t.part0 + q];
    const double d = sqrt(block_sum(s, lds)) + eps;
    return d == 0.0 ? 0.0 : 1.0 / d;
}

__global__ __launch_bounds__(256) void k_muon_norm(const MuonMat *mats, const double *partials,
                                                   double *inv, double eps)
{
    __shared__ double lds[4];
    const double r = inverse_norm(mats[blockIdx.x], partials, eps, lds);
    if (threadIdx.x == 0)
        inv[blockIdx.x] = r;
}

// X = U / (|U|_F + eps), as the fp16 operands X and Y = X^T and the
// remainder, one 64 x 64 tile of the padded X per workgroup through LDS.
template <bool BF, bool STEP, bool WIDE>
__global__ __launch_bounds__(256) void k_muon_cast(const MuonMat *mats, const MuonTile *tiles,
                                                   const double *inv, const double *partials,
                                                   double eps, MuonUpdate u)
{
    __shared__ float lds[kCastTile][kCastTile + 1];   // [X row][X column]
    __shared__ double red[4];
    const MuonTile tl = tiles[blockIdx.x];
    const MuonMat &t = mats[tl.mat];
    const float c = STEP ? clip_factor(u) : 1.0f;
    const double r = (inv ? inv[tl.mat] : inverse_norm(t, partials, eps, red)) * (double)kScale;
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
        *reinterpret_cast<half8 *>(t.X + panel_at(t.mp, i0 + row, j0 + at)) = x;
        *reinterpret_cast<half8 *>(t.Y[0] + panel_at(t.np, j0 + row, i0 + at)) = y;
        if (WIDE) {
            for (int k = 0; k < 8; ++k) {
                x[k] = low_part(lds[row][at + k]);
                y[k] = low_part(lds[at + k][row]);
            }
            *reinterpret_cast<half8 *>(t.Xl + panel_at(t.mp, i0 + row, j0 + at)) = x;
            *reinterpret_cast<half8 *>(t.Yl[0] + panel_at(t.np, j0 + row, i0 + at)) = y;
        }
    }
    for (int q = threadIdx.x; q < 1024; q += 256) {
        // 4 rows of one column, lanes in the remainder's order
        const int block = q >> 8, i = (block >> 1) * 32 + ((q >> 6) & 3) * 8 + ((q >> 5) & 1) * 4;
        const int j = (block & 1) * 32 + (q & 31);
        half4 y;
        float4v f;
        for (int k = 0; k < 4; ++k) {
            f[k] = lds[i + k][j];
            y[k] = low_part(f[k]);
        }
        if (WIDE)
            *reinterpret_cast<float4v *>(t.F + carry_at(t.np, i0 + i, j0 + j)) = f;
        else
            *reinterpret_cast<half4 *>(t.L + carry_at(t.np, i0 + i, j0 + j)) = y;
    }
}

enum Mode { kGram, kGramPart, kPoly, kUpdate, kOrtho, kStep };

// Transposes 4 x 4 halves across 4 lanes: lane q's column becomes row q.
__device__ __forceinline__ half4 quad_transpose(half4 h)
{
    union {
        half4 h;
        uint32_t d[2];
    } v;
    v.h = h;
    const bool odd = threadIdx.x & 1, upper = threadIdx.x & 2;
    // with lane ^ 1: even lanes keep elements 0 and 2, odd ones 1 and 3
    const uint32_t sel = odd ? 0x03020706u : 0x05040100u;   // bytes of {other, own}
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t other = __builtin_amdgcn_mov_dpp(v.d[k], 0xb1, 0xf, 0xf, true);
        v.d[k] = __builtin_amdgcn_perm(other, v.d[k], sel);
    }
    // with lane ^ 2: the lower two keep word 0, the upper two word 1
    const uint32_t send = upper ? v.d[0] : v.d[1];
    const uint32_t got = __builtin_amdgcn_mov_dpp(send, 0x4e, 0xf, 0xf, true);
    v.d[0] = upper ? got : v.d[0];
    v.d[1] = upper ? v.d[1] : got;
    return v.h;
}

template <int N>
__device__ __forceinline__ void wait_copies()
{
    // at most N copies of this wave outstanding, no LDS read outstanding
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
}

// The caller's outputs of one 32 x 32 block of the last X, held as the matrix
// instruction leaves it: column `low`, rows 8 g + 4 half + k.  Element (i, j)
// of X sits at i * si + j * sj of the caller's matrix.  A whole block is written
// without a test per element, 8 or 16 bytes a lane where its rows are 16-byte
// aligned (4 x 2048 x 2048: 274 us for this product with the tests, 86 for
// one that writes no outputs).
template <Mode MODE>
__device__ __forceinline__ void put_block(const MuonMat &t, const MuonUpdate &u, int64_t i0, int64_t j0,
                                          const float4v (&x)[4])
{
    const int lane = threadIdx.x & 63, half = lane >> 5, low = lane & 31;
    const double decay = 1.0 - u.lr * u.wd * t.wd_scale, step = u.lr * t.lr_scale;
    uint16_t *out = MODE == kOrtho ? t.ortho : t.weight;
    const auto fresh = [&](float o, float old) {
        return MODE == kOrtho ? o : (float)((double)old * decay - step * (double)o);
    };
    const int64_t ii = i0 + half * 4, jj = j0 + low;
    if (i0 + 32 <= t.m && j0 + 32 <= t.n && (t.vec4 || !t.flip)) {
        float4v w[4];
        if (t.flip) {
            const int64_t at = jj * t.cols + ii;
            if (MODE == kStep)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    w[g] = *reinterpret_cast<const float4v *>(t.master + at + 8 * g);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                half4 h;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[g][k] = fresh(x[g][k] * kUnscale, w[g][k]);
                    h[k] = __builtin_bit_cast(_Float16, f32_to_bf16(w[g][k]));
                }
                if (MODE == kStep)
                    *reinterpret_cast<float4v *>(t.master + at + 8 * g) = w[g];
                *reinterpret_cast<half4 *>(out + at + 8 * g) = h;
            }
        } else {
            float *m = t.master + ii * t.cols + jj;
            uint16_t *o = out + (ii + (t.vec4 ? lane & 3 : 0)) * t.cols + (t.vec4 ? jj & ~3 : jj);
            if (MODE == kStep)
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[g][k] = m[(int64_t)(8 * g + k) * t.cols];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                half4 h;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[g][k] = fresh(x[g][k] * kUnscale, w[g][k]);
                    h[k] = __builtin_bit_cast(_Float16, f32_to_bf16(w[g][k]));
                    if (MODE == kStep)
                        m[(int64_t)(8 * g + k) * t.cols] = w[g][k];
                }
                if (t.vec4)
                    *reinterpret_cast<half4 *>(o + (int64_t)(8 * g) * t.cols) = quad_transpose(h);
                else
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[(int64_t)(8 * g + k) * t.cols] = f32_to_bf16(w[g][k]);
            }
        }
        return;
    }
    const int64_t si = t.flip ? 1 : t.cols, sj = t.flip ? t.cols : 1;
    if (jj < t.n) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t r = ii + 8 * g + k, e = r * si + jj * sj;
                if (r < t.m) {
                    const float w = fresh(x[g][k] * kUnscale, MODE == kStep ? t.master[e] : 0.f);
                    if (MODE == kStep)
                        t.master[e] = w;
                    out[e] = f32_to_bf16(w);
                }
            }
    }
}

// C_ij = sum_k P_ik Q_jk on one T x T tile, one 32-deep panel after another.
//
// A panel's share of both operands (T x 32 halves each, contiguous) is copied
// straight into LDS, 1 KiB a wave and instruction, into a ring of RING panels,
// so RING - 1 panels are on their way while one is multiplied.  A row is 64
// bytes, so four rows span the 64 banks; the 16-byte chunks of row r sit
// permuted by (r / 4) mod 4, and the 16 lanes of a fragment read that share a
// cycle then touch all banks once (the counters show no conflict; permuted by
// (r / 2) mod 4, half the reads wait).  The permutation is applied to the
// global address, as the LDS side of the copy is fixed in lane order.
//
// PAIRED (256 tiles, 8 waves, one workgroup a compute unit): waves w and w + 4
// share a SIMD, and the second four run half a step behind the first, so that
// one of the two multiplies while the other reads its fragments and issues
// copies; two barriers a panel keep them in step.  4096 x 4096 x 4096: 110 us
// (1250 TFLOP/s) against 139 with all waves in phase; with row-major operands
// 121, with 64-deep panels 127.  Smaller tiles get the same effect from
// three workgroups a compute unit; 64 tiles take two panels a step, as a step
// of so few matrix instructions is mostly the wait for its fragments
// (333 x 1537: 112 us against 137).
//
// WIDE: P = Ph + Pl and Q = Qh + Ql, each half an operand of its own, and the
// product is Ph Ql + Pl Qh + Ph Qh (Pl Ql is below what 22 bits hold): the
// panels of three products one after another into the same accumulators.
template <int T, int WM, int WN, int PANELS, int RING, bool PAIRED, Mode MODE, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN) void k_muon_gemm(const MuonMat *mats,
                                                            const MuonTile *tiles, int src,
                                                            float ca, float cb, float cc,
                                                            MuonUpdate u, float *parts, int splits)
{
    constexpr int NW = WM * WN;
    constexpr int TM = T / WM / 32, TN = T / WN / 32;
    constexpr int kLoads = T / 16 / NW;   // copies per wave, operand and panel
    static_assert(kLoads >= 1 && TM >= 1 && TN >= 1, "tile and wave grid");
    static_assert(!PAIRED || PANELS == 1, "one panel a phase");
    __shared__ __align__(16) _Float16 lds[RING][PANELS][2][T * 32];

    const MuonTile tl = tiles[blockIdx.x];
    const MuonMat &t = mats[tl.mat];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i0 = tl.ti * T, j0 = tl.tj * T;

    const _Float16 *P, *Q, *Pl = nullptr, *Ql = nullptr;
    int64_t p_step, q_step;
    int K;
    if (MODE == kGram || MODE == kGramPart) {
        P = Q = t.X;
        Pl = Ql = t.Xl;
        K = t.np;
        p_step = q_step = (int64_t)t.mp * 32;
        if (MODE == kGramPart) {   // one of `splits` equal pieces of the depth
            const int piece = (t.np / 64 + splits - 1) / splits * 64;
            const int first = tl.part % splits * piece;
            P = Q = t.X + (int64_t)first * t.mp;
            Pl = Ql = t.Xl + (int64_t)first * t.mp;
            K = max(0, min(piece, t.np - first));
        }
    } else if (MODE == kPoly) {
        P = Q = t.A;
        Pl = Ql = t.Al;
        K = t.mp;
        p_step = q_step = (int64_t)t.mp * 32;
    } else {
        P = t.B;
        Q = t.Y[src];
        Pl = t.Bl;
        Ql = t.Yl[src];
        K = t.mp;
        p_step = (int64_t)t.mp * 32;
        q_step = (int64_t)t.np * 32;
    }
    P += (int64_t)i0 * 32;
    Q += (int64_t)j0 * 32;
    const _Float16 *const Ph = P, *const Qh = Q;
    int left = K / 32, pass = 0;   // panels before the next of the three products
    if (WIDE) {
        Pl += (int64_t)i0 * 32;
        Ql += (int64_t)j0 * 32;
        Q = Ql;
    }
    const int voff = ((lane >> 2) * 32 + ((lane & 3) ^ ((lane >> 4) & 3)) * 8) * 2;

    typedef __attribute__((address_space(3))) void lds_void;
    // copies the next panel; the descriptors end with the tile's share of it
    const auto load = [&](int slot, int panel) {
        const auto rp = __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16 *>(P), 0, T * 64, 0x00020000);
        const auto rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16 *>(Q), 0, T * 64, 0x00020000);
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int at = wave * kLoads + q;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (lds_void *)&lds[slot][panel][0][at * 512], 16, voff,
                                                     at * 1024, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_void *)&lds[slot][panel][1][at * 512], 16, voff,
                                                     at * 1024, 0, 0);
        }
        P += p_step;
        Q += q_step;
        if (WIDE && --left == 0) {
            left = K / 32;
            P = pass == 0 ? Pl : Ph;
            Q = Qh;
            ++pass;
        }
    };
    constexpr int kAhead = (RING - 2) * PANELS * 2 * kLoads;   // copies that may stay out at a wait

    float16v acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][j][r] = 0.f;

    const int half = lane >> 5, low = lane & 31;
    const auto frag = [&](const _Float16 *p, int row, int kk) {
        return *reinterpret_cast<const half8 *>(p + row * 32 + (((kk * 2 + half) ^ ((row >> 2) & 3)) * 8));
    };
    const int steps = (WIDE ? 3 : 1) * (K / (32 * PANELS));
    // Wide B X on the tiles of deep matrices: the sums of Ph Qh, whose many
    // roundings at the size of U's strong directions end up in its weak ones, go
    // to X every kFlush steps (2048^2 of rank 4 plus 1% noise: O 2.5e-5 off
    // without, 1.4e-5 with).  Smaller tiles would lose their second wave to it
    // (8 x 1536 x 576: 783 us against 573).
    constexpr bool kFlushes = WIDE && T == 256 && (MODE == kUpdate || MODE == kOrtho || MODE == kStep);
    constexpr int kFlush = 1024 / (32 * PANELS);
    int next_flush = steps / 3 * 2 + kFlush;
    float scale = ca;   // of the X in F
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
        half8 a[2 * PANELS][TM], b[2 * PANELS][TN];
        asm volatile("" ::: "memory");
#pragma unroll
        for (int kk = 0; kk < 2 * PANELS; ++kk) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
                b[kk][j] = frag(lds[slot][kk >> 1][1], (wn * TN + j) * 32 + low, kk & 1);
#pragma unroll
            for (int i = 0; i < TM; ++i)
                a[kk][i] = frag(lds[slot][kk >> 1][0], (wm * TM + i) * 32 + low, kk & 1);
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
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[kk][i], b[kk][j], acc[i][j], 0, 0, 0);
        if (PAIRED) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" ::: "memory");
        slot = slot + 1 == RING ? 0 : slot + 1;
        if (kFlushes && k + 1 == next_flush && k + 1 < steps) {
            float *F = t.F;
            const int64_t across = t.np >> 5;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int64_t bi = i0 / 32 + wm * TM + i, bj = j0 / 32 + wn * TN + j;
                        float4v *at = reinterpret_cast<float4v *>(
                            F + (bi * across + bj) * 1024 + lane * 4 + g * 256);
                        float4v x = *at;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = fmaf(scale, x[e], acc[i][j][4 * g + e] * kUnscale);
                            acc[i][j][4 * g + e] = 0.f;
                        }
                        *at = x;
                    }
            scale = 1.f;
            next_flush += kFlush;
        }
    }
    if (PAIRED && wave < NW / 2)
        __builtin_amdgcn_s_barrier();   // as many as the second four

    // A lane holds, of each 32 x 32 block, column `low` and rows
    // 8 g + 4 half + (0..3) for g = 0..3: 8 bytes of the transposed operand.
    // Four lanes' 4 x 4 halves are transposed for the 8 bytes of the other.
    // What a block reads is read before any of it is written: a load behind a
    // store to what may be the same place waits for it (20 us a 256 tile).
    if (MODE == kGramPart) {
        float *to = parts + (int64_t)tl.part * T * T + wave * TM * TN * 1024 + lane * 4;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<float4v *>(to + (i * TN + j) * 1024 + g * 256) =
                        float4v{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                                acc[i][j][4 * g + 3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t bi = i0 / 32 + wm * TM + i;
        if (MODE == kGram || MODE == kPoly) {
            half4 x[TN][4], rest[TN][4];
            if (MODE == kPoly)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int64_t bj = j0 / 32 + wn * TN + j;
                        const int64_t from = (bi * t.mp + bj * 32 + low) * 32 + half * 4 + g * 8;
                        x[j][g] = *reinterpret_cast<const half4 *>(t.A + from);
                        if (WIDE)
                            rest[j][g] = *reinterpret_cast<const half4 *>(t.Al + from);
                    }
            _Float16 *D = MODE == kGram ? t.A : t.B, *Dl = MODE == kGram ? t.Al : t.Bl;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int64_t bj = j0 / 32 + wn * TN + j;
                const int64_t at = (bi * t.mp + bj * 32 + low) * 32 + half * 4;
                const int64_t mirror = (bj * t.mp + bi * 32 + half * 4 + (lane & 3)) * 32 + (low & ~3);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    half4 h, l;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float v = acc[i][j][4 * g + k] * kUnscale;
                        if (MODE == kPoly) {
                            const float a = WIDE ? (float)x[j][g][k] + (float)rest[j][g][k] : (float)x[j][g][k];
                            v = fmaf(cc, v, cb * a);
                        }
                        h[k] = (_Float16)v;
                        if (WIDE)
                            l[k] = low_part(v);
                    }
                    *reinterpret_cast<half4 *>(D + at + g * 8) = h;
                    if (WIDE)
                        *reinterpret_cast<half4 *>(Dl + at + g * 8) = l;
                    if (tl.ti != tl.tj) {
                        *reinterpret_cast<half4 *>(D + mirror + g * 256) = quad_transpose(h);
                        if (WIDE)
                            *reinterpret_cast<half4 *>(Dl + mirror + g * 256) = quad_transpose(l);
                    }
                }
            }
        } else {
            // X is its operand copy (which this tile has just multiplied) plus
            // the low part, or with wide products kept as it is: 22 bits add
            // 1e-5 to the error of a low-rank U there, 32 half of that
            half4 hi[TN][4], lo[TN][4];
            float4v full[TN][4];
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int64_t bj = j0 / 32 + wn * TN + j;
                    if (WIDE) {
                        full[j][g] = *reinterpret_cast<const float4v *>(
                            t.F + (bi * (t.np >> 5) + bj) * 1024 + lane * 4 + g * 256);
                        continue;
                    }
                    hi[j][g] = *reinterpret_cast<const half4 *>(
                        t.Y[src] + (bi * t.np + bj * 32 + low) * 32 + half * 4 + g * 8);
                    lo[j][g] = *reinterpret_cast<const half4 *>(
                        t.L + (bi * (t.np >> 5) + bj) * 1024 + lane * 4 + g * 256);
                }
            float4v x[TN][4];
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[j][g][k] = fmaf(WIDE ? scale : ca, WIDE ? full[j][g][k] : (float)hi[j][g][k] + (float)lo[j][g][k],
                                          acc[i][j][4 * g + k] * kUnscale);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int64_t bj = j0 / 32 + wn * TN + j;
                if (MODE == kUpdate) {
                    const int64_t place = (bi * (t.np >> 5) + bj) * 1024 + lane * 4;
                    const int64_t y_at = (bi * t.np + bj * 32 + low) * 32 + half * 4;
                    const int64_t x_at = (bj * t.mp + bi * 32 + half * 4 + (lane & 3)) * 32 + (low & ~3);
                    _Float16 *rest = t.L + place, *yt = t.Y[src ^ 1] + y_at, *xt = t.X + x_at;
                    _Float16 *yl = t.Yl[src ^ 1] + y_at, *xl = t.Xl + x_at;
                    float *whole = t.F + place;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        half4 h, l;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            h[k] = (_Float16)x[j][g][k];
                            l[k] = low_part(x[j][g][k]);
                        }
                        if (WIDE) {
                            *reinterpret_cast<float4v *>(whole + g * 256) = x[j][g];
                            *reinterpret_cast<half4 *>(yl + g * 8) = l;
                            *reinterpret_cast<half4 *>(xl + g * 256) = quad_transpose(l);
                        } else {
                            *reinterpret_cast<half4 *>(rest + g * 256) = l;
                        }
                        *reinterpret_cast<half4 *>(yt + g * 8) = h;
                        *reinterpret_cast<half4 *>(xt + g * 256) = quad_transpose(h);
                    }
                } else {
                    put_block<MODE>(t, u, bi * 32, bj * 32, x[j]);
                }
            }
        }
    }
}

// A = X X^T from the pieces' sums, added in order: a workgroup of four waves
// per 64 x 64 tile, lanes as in the product.
template <bool WIDE>
__global__ __launch_bounds__(256) void k_muon_join(const MuonMat *mats, const MuonTile *tiles,
                                                   const float *parts, int splits)
{
    const MuonTile tl = tiles[blockIdx.x];
    const MuonMat &t = mats[tl.mat];
    const int lane = threadIdx.x & 63, half = lane >> 5, low = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t bi = tl.ti * 2 + wave / 2, bj = tl.tj * 2 + wave % 2;
    const float *from = parts + (int64_t)tl.part * splits * 4096 + wave * 1024 + lane * 4;
    float4v s[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
        s[g] = *reinterpret_cast<const float4v *>(from + g * 256);
#pragma unroll 4
    for (int q = 1; q < splits; ++q)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            s[g] += *reinterpret_cast<const float4v *>(from + (int64_t)q * 4096 + g * 256);
    const int64_t at = (bi * t.mp + bj * 32 + low) * 32 + half * 4;
    const int64_t mirror = (bj * t.mp + bi * 32 + half * 4 + (lane & 3)) * 32 + (low & ~3);
    _Float16 *A = t.A, *Al = t.Al;
    const bool both = tl.ti != tl.tj;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        half4 h, l;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = (_Float16)(s[g][k] * kUnscale);
            if (WIDE)
                l[k] = low_part(s[g][k] * kUnscale);
        }
        *reinterpret_cast<half4 *>(A + at + g * 8) = h;
        if (WIDE)
            *reinterpret_cast<half4 *>(Al + at + g * 8) = l;
        if (both) {
            *reinterpret_cast<half4 *>(A + mirror + g * 256) = quad_transpose(h);
            if (WIDE)
                *reinterpret_cast<half4 *>(Al + mirror + g * 256) = quad_transpose(l);
        }
    }
}

template <Mode MODE, bool WIDE>
void product(const MuonTables &t, const MuonUpdate &u, int src, hipStream_t s)
{
    const int p = MODE == kGram ? 0 : MODE == kPoly ? 1 : 2;
    const uint32_t n = (uint32_t)t.n_tiles[p];
    if (t.tile[p] == 256)
        k_muon_gemm<256, 2, 4, 1, 4, true, MODE, WIDE><<<n, 512, 0, s>>>(t.mats, t.tiles[p], src, t.a, t.b, t.c, u, nullptr, 1);
    else if (t.tile[p] == 128)
        k_muon_gemm<128, 2, 2, 1, 3, false, MODE, WIDE><<<n, 256, 0, s>>>(t.mats, t.tiles[p], src, t.a, t.b, t.c, u, nullptr, 1);
    else
        k_muon_gemm<64, 2, 2, 2, 3, false, MODE, WIDE><<<n, 256, 0, s>>>(t.mats, t.tiles[p], src, t.a, t.b, t.c, u, nullptr, 1);
}

template <bool WIDE>
void iterate(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s)
{
    for (int k = 0; k < ns_steps; ++k) {
        const int src = k & 1;
        if (t.splits > 1) {
            k_muon_gemm<64, 2, 2, 2, 3, false, kGramPart, WIDE><<<(uint32_t)(t.n_tiles[0] * t.splits), 256, 0, s>>>(
                t.mats, t.pieces, src, t.a, t.b, t.c, u, t.parts, t.splits);
            k_muon_join<WIDE><<<(uint32_t)t.n_tiles[0], 256, 0, s>>>(t.mats, t.tiles[0], t.parts, t.splits);
        } else {
            product<kGram, WIDE>(t, u, src, s);
        }
        product<kPoly, WIDE>(t, u, src, s);
        if (k + 1 < ns_steps)
            product<kUpdate, WIDE>(t, u, src, s);
        else if (u.step)
            product<kStep, WIDE>(t, u, src, s);
        else
            product<kOrtho, WIDE>(t, u, src, s);
    }
}

// D = f(P P^T, P) for a symmetric P P^T with `side` blocks a side, in LDS, the
// blocks shared out over 8 waves; f gets P's own element where D and P have
// the same shape.  What a block reads of a step's depth is read before the
// first of it is multiplied.  32 x 32 blocks read LDS half as often and are used
// from 64 a side (64 x 512: 33 us against 39 with 16 x 16 blocks); 16 x 16 ones
// give four waves work where the side is 32.
template <typename F>
__device__ __forceinline__ void square16(const _Float16 *P, int sp, int depth, _Float16 *D, int sd,
                                         int side, int wave, int lane, F &&f)
{
    const int l15 = lane & 15, l4 = lane >> 4;
    for (int bl = wave; bl < side * side; bl += 8) {
        const int i = bl / side * 16, j = bl % side * 16;
        const _Float16 *pa = P + (i + l15) * sp + l4 * 8, *pb = P + (j + l15) * sp + l4 * 8;
        float4v s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        int k = 0;
        for (; k + 128 <= depth; k += 128) {
            half8 a[4], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = *reinterpret_cast<const half8 *>(pa + k + 32 * q);
                b[q] = *reinterpret_cast<const half8 *>(pb + k + 32 * q);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                s[q & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[q], b[q], s[q & 1], 0, 0, 0);
        }
        for (; k < depth; k += 32)
            s[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const half8 *>(pa + k),
                                                          *reinterpret_cast<const half8 *>(pb + k), s[0], 0, 0, 0);
        // column j + l15, rows i + 4 l4 + (0..3): stored as the mirrored place
        const half4 own = *reinterpret_cast<const half4 *>(P + (j + l15) * sp + i + 4 * l4);
        half4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = (_Float16)f((s[0][e] + s[1][e]) * kUnscale, (float)own[e]);
        *reinterpret_cast<half4 *>(D + (j + l15) * sd + i + 4 * l4) = h;
    }
}

template <typename F>
__device__ __forceinline__ void square32(const _Float16 *P, int sp, int depth, _Float16 *D, int sd,
                                         int side, int wave, int lane, F &&f)
{
    const int half = lane >> 5, low = lane & 31;
    for (int bl = wave; bl < side * side; bl += 8) {
        const int i = bl / side * 32, j = bl % side * 32;
        const _Float16 *pa = P + (i + low) * sp + half * 8, *pb = P + (j + low) * sp + half * 8;
        float16v s;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            s[e] = 0.f;
        for (int k = 0; k < depth; k += 32) {
            half8 a[2], b[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                a[q] = *reinterpret_cast<const half8 *>(pa + k + 16 * q);
                b[q] = *reinterpret_cast<const half8 *>(pb + k + 16 * q);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
                s = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[q], b[q], s, 0, 0, 0);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int ii = i + 8 * g + 4 * half;
            const half4 own = *reinterpret_cast<const half4 *>(P + (j + low) * sp + ii);
            half4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = (_Float16)f(s[4 * g + e] * kUnscale, (float)own[e]);
            *reinterpret_cast<half4 *>(D + (j + low) * sd + ii) = h;
        }
    }
}

// A small matrix's whole update in one workgroup: nothing but the caller's
// tensors crosses memory, and the five steps' fifteen products are separated
// by barriers instead of launches (2 of 64 x 256: 27 us against 62 for 18
// launches of 2 to 5 us each; 128 x 160: 33 against 60; 2000 of them: 278
// against 1242).  What is left is latency: 2.8 us a step of 64 x 256.
template <bool BF, bool STEP>
__global__ __launch_bounds__(512) void k_muon_small(const MuonMat *mats, MuonUpdate u, int ns_steps,
                                                    float ca, float cb, float cc, double eps)
{
    __shared__ __align__(16) char lds[kSmallLds];
    __shared__ double red[8];
    const MuonMat &t = mats[blockIdx.x];
    const int mp = t.mp, np = t.np, sx = np + 8, sy = mp + 8, su = np + 4;
    _Float16 *X = reinterpret_cast<_Float16 *>(lds);   // [mp][sx]
    _Float16 *Y = X + mp * sx;                         // [np][sy]
    _Float16 *A = Y + np * sy, *B = A + mp * sy;       // [mp][sy]
    float *U = reinterpret_cast<float *>(lds);         // [mp][su], before X and Y
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, low = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int numel = t.rows * t.cols;
    if (numel < mp * np) {   // the padding
        for (int q = tid; q < mp * su; q += 512)
            U[q] = 0.f;
        __syncthreads();
    }
    const float c = STEP ? clip_factor(u) : 1.0f;
    double sum = 0.0;
    const auto put = [&](int row, int col, float grad, float &mom) {
        float x = c * grad;
        if (STEP) {
            mom = fmaf(u.mu, mom, x);
            x = u.nesterov ? fmaf(u.mu, mom, x) : mom;
        }
        U[t.flip ? col * su + row : row * su + col] = x;
        sum += (double)x * (double)x;
    };
    // N elements a load, 8 loads of a lane in flight (the momentum is written
    // behind them: a load after a store to what may be its place would wait)
    const auto take = [&](auto width) {
        constexpr int N = decltype(width)::value, kBatch = 8;
        for (int at = tid * N; at < numel; at += 512 * N * kBatch) {
            float g[kBatch][N], m[kBatch][N];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int e = at + 512 * N * q;
                if (e < numel) {
                    if (N == 4 && !BF)
                        *reinterpret_cast<float4v *>(g[q]) =
                            *reinterpret_cast<const float4v *>(static_cast<const float *>(t.grad) + e);
                    else if (N == 4) {
                        const uint2v p = *reinterpret_cast<const uint2v *>(static_cast<const uint16_t *>(t.grad) + e);
                        g[q][0] = __uint_as_float(p.x << 16);
                        g[q][N / 4] = __uint_as_float(p.x & 0xffff0000u);
                        g[q][N / 2] = __uint_as_float(p.y << 16);
                        g[q][N - 1] = __uint_as_float(p.y & 0xffff0000u);
                    } else
                        g[q][0] = load_grad<BF>(t, e);
                    if (STEP) {
                        if (N == 4)
                            *reinterpret_cast<float4v *>(m[q]) = *reinterpret_cast<const float4v *>(t.mom + e);
                        else
                            m[q][0] = t.mom[e];
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int e = at + 512 * N * q;
                if (e < numel) {
                    const int row = (int)((uint32_t)e / (uint32_t)t.cols), col = e - row * t.cols;
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        put(row, col + k, g[q][k], m[q][k]);
                    if (STEP) {
                        if (N == 4)
                            *reinterpret_cast<float4v *>(t.mom + e) = *reinterpret_cast<float4v *>(m[q]);
                        else
                            t.mom[e] = m[q][0];
                    }
                }
            }
        }
    };
    if (t.vec && t.cols % 4 == 0)
        take(std::integral_constant<int, 4>());
    else
        take(std::integral_constant<int, 1>());
    sum = block_sum(sum, red);   // its barriers also end the writes of U
    const double d = sqrt(sum) + eps;
    const double r = d == 0.0 ? 0.0 : (double)kScale / d;

    // block q of this wave: number wave + 8 q of the (mp / 32) x (np / 32)
    const int across = np / 32, blocks = (mp / 32) * across;
    float4v x[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int bl = wave + 8 * q;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            x[q][g] = float4v{0.f, 0.f, 0.f, 0.f};
        if (bl < blocks) {
            const int i = bl / across * 32 + 4 * half, j = bl % across * 32 + low;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[q][g][k] = (float)((double)U[(i + 8 * g + k) * su + j] * r);
        }
    }
    __syncthreads();

    for (int step = 0; step < ns_steps; ++step) {
        // the operand copies of X
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int bl = wave + 8 * q;
            if (bl < blocks) {
                const int i = bl / across * 32 + 4 * half, j = bl % across * 32 + low;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    half4 h;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = (_Float16)x[q][g][k];
                    *reinterpret_cast<half4 *>(Y + j * sy + i + 8 * g) = h;
                    *reinterpret_cast<half4 *>(X + (i + 8 * g + (lane & 3)) * sx + (j & ~3)) = quad_transpose(h);
                }
            }
        }
        __syncthreads();
        // A = X X^T
        if (mp >= 64)
            square32(X, sx, np, A, sy, mp / 32, wave, lane,
                     [&](float v, float) { return v; });
        else
            square16(X, sx, np, A, sy, mp / 16, wave, lane, [&](float v, float) { return v; });
        __syncthreads();
        // B = b A + c A A
        if (mp >= 64)
            square32(A, sy, mp, B, sy, mp / 32, wave, lane,
                     [&](float v, float s) { return fmaf(cc, v, cb * s); });
        else
            square16(A, sy, mp, B, sy, mp / 16, wave, lane,
                     [&](float v, float s) { return fmaf(cc, v, cb * s); });
        __syncthreads();
        // X = a X + B X, the wave's blocks side by side
        {
            float16v acc[4];
            const _Float16 *pa[4], *pb[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int bl = wave + 8 * q;
                pa[q] = B + (bl / across * 32 + low) * sy + half * 8;
                pb[q] = Y + (bl % across * 32 + low) * sy + half * 8;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[q][e] = 0.f;
            }
            for (int k = 0; k < mp; k += 32) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (wave + 8 * q < blocks) {
                        const half8 a0 = *reinterpret_cast<const half8 *>(pa[q] + k);
                        const half8 b0 = *reinterpret_cast<const half8 *>(pb[q] + k);
                        const half8 a1 = *reinterpret_cast<const half8 *>(pa[q] + k + 16);
                        const half8 b1 = *reinterpret_cast<const half8 *>(pb[q] + k + 16);
                        acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a0, b0, acc[q], 0, 0, 0);
                        acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a1, b1, acc[q], 0, 0, 0);
                    }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[q][g][k] = fmaf(ca, x[q][g][k], acc[q][4 * g + k] * kUnscale);
        }
        __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int bl = wave + 8 * q;
        if (bl < blocks)
            put_block<STEP ? kStep : kOrtho>(t, u, bl / across * 32, bl % across * 32, x[q]);
    }
}

template <bool BF, bool STEP>
void small(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s)
{
    k_muon_small<BF, STEP><<<(uint32_t)t.n_small, 512, 0, s>>>(t.mats + t.n, u, ns_steps, t.a, t.b, t.c, t.eps);
}

template <bool BF, bool STEP, bool WIDE>
void first(const MuonTables &t, const MuonUpdate &u, hipStream_t s)
{
    k_muon_momentum<BF, STEP><<<(uint32_t)t.n_chunks, 256, 0, s>>>(t.mats, t.chunks, t.partials, u);
    // one partial a lane: every tile of the cast adds them by itself, and a
    // launch is saved (8 x 576 x 1536: 239 -> 236 us, 200 x 300: 71.5 -> 70)
    const bool apart = t.n_part_most > 256;
    if (apart)
        k_muon_norm<<<(uint32_t)t.n, 256, 0, s>>>(t.mats, t.partials, t.inv, t.eps);
    k_muon_cast<BF, STEP, WIDE><<<(uint32_t)t.n_cast, 256, 0, s>>>(
        t.mats, t.cast, apart ? t.inv : nullptr, t.partials, t.eps, u);
}

template <bool WIDE>
void tiled(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s)
{
    if (t.grad_bf16)
        u.step ? first<true, true, WIDE>(t, u, s) : first<true, false, WIDE>(t, u, s);
    else
        u.step ? first<false, true, WIDE>(t, u, s) : first<false, false, WIDE>(t, u, s);
    iterate<WIDE>(t, u, ns_steps, s);
}

}  // namespace

hipError_t launch_muon(const MuonTables &t, const MuonUpdate &u, int ns_steps, hipStream_t s)
{
    if (t.n_small > 0) {
        if (t.grad_bf16)
            u.step ? small<true, true>(t, u, ns_steps, s) : small<true, false>(t, u, ns_steps, s);
        else
            u.step ? small<false, true>(t, u, ns_steps, s) : small<false, false>(t, u, ns_steps, s);
    }
    if (t.n == 0)
        return hipGetLastError();
    t.wide ? tiled<true>(t, u, ns_steps, s) : tiled<false>(t, u, ns_steps, s);
    return hipGetLastError();
}

}  // namespace ops
}  // namespace z1
